"""More operators of a serving step around a paged KV cache, as measurable cases.

* ``rotate``: rotate a step's q and K by their positions, write q out and K and V into their
  pages (``kvx_append_rotated``).
* ``four``: attention over a cache held in 4 bits (``kvx_attend``), single tokens to prefill
  chunks; with ``chain`` the step's q and K are rotated and K and V put into that cache before
  (``kvx_append_rotated``), as a layer of a model does.
* ``select``: the best continuations of every group of beams over beams and vocabulary
  (``kvx_select_beams``).
* ``reorder``: make every beam's pages those of the beam that it continues
  (``kvx_reorder_beams``).

``own`` selects the form ``run`` takes: False is elementary torch in 32 bits (64 for the angles
of far positions and for what candidates are ordered by), True the calls of this library.

The 4-bit cache: a token of a side is [kv_heads][head_dim / 2] bytes of e2m1 codes, element 2 i
in the low half of byte i, then [kv_heads][head_dim / 16] e4m3 scales, padded to 16 bytes; an
element is its code times its block's scale times k_scale (v_scale).
"""
import math
import random

import torch

own = False

DEV = "cuda"
LAYER = 1            # attention and append work on this layer of a two-layer pool
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn,
         "fp32": torch.float32}
ITEM = {"bf16": 2, "fp16": 2, "fp8": 1, "fp32": 4}
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)    # of an e2m1 code's low three bits
SCALES = {"fp8": (0.03, 0.05), "fp4": (0.01, 0.012)}     # of K and V in caches of few bits


# ------------------------------------------------------------------------------- cases

def _step(name, op, requests, new, length, kv_heads, group, head_dim, page, kv, dtype="bf16",
          rotary=0, interleaved=False, far=0, window=0, prefix=0, softcap=0.0, slopes=False,
          fused=False):
    """`rotary`: elements of a head that are rotated (0: the step only attends)."""
    return {"name": name, "op": op, "requests": requests, "new_min": new[0], "new_max": new[1],
            "len_min": length[0], "len_max": length[1], "kv_heads": kv_heads, "group": group,
            "head_dim": head_dim, "page": page, "kv": kv, "dtype": dtype, "rotary": rotary,
            "interleaved": interleaved, "far": far, "window": window, "prefix": prefix,
            "softcap": softcap, "slopes": slopes, "fused": fused}


def _select(name, groups, width, vocab, picks, dtype="bf16", done=0.0):
    return {"name": name, "op": "select", "groups": groups, "width": width, "vocab": vocab,
            "picks": picks, "dtype": dtype, "done": done}


def _reorder(name, groups, width, length, layers, kv_factor, token_bytes, page):
    return {"name": name, "op": "reorder", "groups": groups, "width": width,
            "len_min": length[0], "len_max": length[1], "layers": layers,
            "kv_factor": kv_factor, "token_bytes": token_bytes, "page": page}


def listed():
    return [
        # One new token for each of 64 requests, K and V cast to the fp8 cache: latency counts.
        _step("rotate_decode", "rotate", 64, (1, 1), (1024, 32768), 4, 7, 128, 16, "fp8",
              rotary=128, fused=True),
        # Prefill chunks of several requests, q, K and V taken out of a fused projection.
        _step("rotate_chunk", "rotate", 5, (1000, 2048), (2048, 16384), 8, 4, 128, 32, "bf16",
              rotary=128, fused=True),
        # A single token of one short request: the smallest attention.
        _step("four_one", "four", 1, (1, 1), (1000, 1000), 2, 4, 64, 16, "fp4", "fp16"),
        # A layer of a decoding step over ragged contexts: rotation, append and attention.
        _step("four_step", "four", 64, (1, 1), (1024, 32768), 4, 7, 128, 16, "fp4", rotary=128,
              fused=True),
        # A few drafted tokens of each request behind longer contexts, all of them verified.
        _step("four_drafts", "four", 24, (2, 2), (2048, 65536), 8, 8, 128, 32, "fp4"),
        # One request alone with a very long context.
        _step("four_long", "four", 1, (1, 1), (262144, 262144), 8, 8, 128, 16, "fp4"),
        # Several requests with a few new tokens up to a prefill chunk, every score option on.
        _step("four_ragged", "four", 6, (1, 700), (1, 9000), 4, 4, 128, 16, "fp4", window=2048,
              prefix=130, softcap=30.0, slopes=True, fused=True),
        # The largest: a layer of a prefill chunk behind a long context.
        _step("four_chunk", "four", 1, (2048, 2048), (32768, 32768), 8, 4, 128, 16, "fp4",
              rotary=128, fused=True),
        # One prompt searched with four beams: latency.
        _select("select_one", 1, 4, 32000, 4, "fp32"),
        # A batch of prompts with eight beams each over a large vocabulary, twice the beams
        # taken (half of the candidates may end a sequence), some beams done.
        _select("select_batch", 64, 8, 128256, 16, done=0.1),
        # The pages of those four beams, 8B-shaped cache: only partly filled last pages move.
        _reorder("reorder_one", 1, 4, (1001, 1001), 32, 2, 2048, 16),
        # A beam step of a batch of ragged groups on the fp8 cache.
        _reorder("reorder_batch", 32, 8, (512, 8192), 28, 2, 512, 16),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "rotate", "four", "four", "four", "select", "reorder"])
    if op == "select":
        vocab = _log_int(rng, 1000, 160000)
        width = rng.choice([1, 2, 3, 4, 5, 8, 10, 16])
        groups = _log_int(rng, 1, max(1, min(64, int(66e6 / (vocab * width)))))
        c = _select("", groups, width, vocab, rng.choice([width, 2 * width]),
                    rng.choice(["bf16", "fp16", "fp32"]), rng.choice([0.0, 0.2]))
    elif op == "reorder":
        page = rng.choice([1, 7, 16, 16, 32, 64])
        token_bytes = rng.choice([256, 512, 1152, 2048])
        kv_factor = 1 if token_bytes == 1152 else 2
        layers = rng.randint(4, 32)
        width = rng.choice([1, 2, 3, 4, 5, 8, 10, 16])
        # Tokens of the whole pool stay within 6 GB of K and V.
        room = int(6e9 / (layers * kv_factor * token_bytes)) // 2
        groups = _log_int(rng, 1, 32)
        hi = max(40, min(8192, room // (groups * width)))
        lo = _log_int(rng, 1, hi)
        c = _reorder("", groups, width, (lo, hi), layers, kv_factor, token_bytes, page)
    else:
        dtype = rng.choice(["bf16", "bf16", "fp16"])
        head_dim = rng.choice([64, 128, 128])
        kv_heads, group = rng.choice([1, 2, 3, 4, 8, 8]), rng.choice([1, 2, 4, 5, 7, 8])
        page = rng.choice([1, 5, 8, 16, 16, 24, 32, 64])
        rotary = rng.choice([head_dim, head_dim, head_dim // 2, 16, 48])
        interleaved = rng.random() < 0.3
        far = rng.choice([0, 0, 900000])
        fused = rng.random() < 0.5
        if op == "rotate":
            requests = _log_int(rng, 1, 64)
            new = (1, 1) if rng.random() < 0.5 else (1, _log_int(rng, 2, 8192 // requests + 2))
            hi = _log_int(rng, new[1], 16384)
            c = _step("", op, requests, new, (min(hi, 1 + rng.randint(0, 1000)), hi), kv_heads,
                      group, head_dim, page, rng.choice([dtype, "fp8"]), dtype, rotary,
                      interleaved, far, fused=fused)
        else:
            kind = rng.choice(["one", "few", "chunk"])
            if kind == "one":
                requests, new = _log_int(rng, 1, 64), (1, 1)
            elif kind == "few":
                requests, new = _log_int(rng, 1, 32), (1, rng.randint(2, 16))
            else:
                requests, new = _log_int(rng, 1, 8), (1, _log_int(rng, 17, 2048))
            # The plain form's scores and gathered K stay below the largest listed case's.
            hi = min(262144 if requests * new[1] == 1 else 65536,
                     int(2.0e9 / (requests * new[1] * kv_heads * group)),
                     int(0.9e9 / (requests * kv_heads * 128)))
            hi = _log_int(rng, min(hi, max(16, new[1], hi // 64)), hi)
            odd, chain = rng.random() < 0.5, rng.random() < 0.4
            c = _step("", op, requests, new, (_log_int(rng, 1, hi), hi), kv_heads, group,
                      head_dim, page, "fp4", dtype, rotary if chain else 0,
                      chain and interleaved, far if chain else 0,
                      window=_log_int(rng, 16, 8192) if odd and rng.random() < 0.6 else 0,
                      prefix=rng.randint(1, 300) if odd and rng.random() < 0.5 else 0,
                      softcap=rng.choice([0.0, 20.0, 50.0]) if odd else 0.0,
                      slopes=odd and rng.random() < 0.5, fused=fused)
    del c["name"]
    return c


def _lengths(c):
    """(tokens, new tokens, prefix) of each request: by the case's sizes alone."""
    r = random.Random("%d %d %d %d %d" % (c["requests"], c["len_min"], c["len_max"],
                                          c["new_min"], c["new_max"]))
    tokens, new = [], []
    for i in range(c["requests"]):
        n = c["len_max"] if i == 0 else _log_int(r, c["len_min"], c["len_max"])
        tokens.append(n)
        new.append(min(n, c["new_max"] if i == 0 else r.randint(c["new_min"], c["new_max"])))
    return tokens, new, [min(c["prefix"] * (i % 3), n) for i, n in enumerate(tokens)]


def _group_lengths(c):
    r = random.Random("%d %d %d" % (c["groups"], c["len_min"], c["len_max"]))
    return [c["len_max"] if i == 0 else _log_int(r, c["len_min"], c["len_max"])
            for i in range(c["groups"])]


def _token_bytes(c):
    row = c["kv_heads"] * c["head_dim"]
    return -(-(row // 2 + row // 16) // 16) * 16 if c["kv"] == "fp4" else row * ITEM[c["kv"]]


# ------------------------------------------------------------------------------- inputs

_context = []


def _ctx():
    """The library context that a program creates once."""
    if not _context:
        from paged_kv_gather_gb300 import kvx
        _context.append(kvx.kvx_create(0))
    return _context[0]


class _Plan:
    """An attention plan that is destroyed with the state that holds it."""

    def __init__(self, handle):
        self.handle = handle

    def __del__(self):
        from paged_kv_gather_gb300 import kvx
        kvx.kvx_attn_plan_destroy(self.handle)


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _random_cache(c, slots, g):
    """[slots, token_bytes] of typed values: a layer of one side."""
    H, D = c["kv_heads"], c["head_dim"]
    if c["kv"] != "fp4":
        x = torch.randn((slots, H * D), dtype=torch.bfloat16, device=DEV, generator=g)
        if c["kv"] == "fp8":  # codes are the values over a scale, as a calibrated cache keeps them
            x.mul_(25.0)
        return x.to(TYPES[c["kv"]]).view(torch.uint8)
    out = torch.zeros((slots, _token_bytes(c)), dtype=torch.uint8, device=DEV)
    some = max(1, (1 << 27) // (H * D))
    for at in range(0, slots, some):
        x = torch.randn((min(some, slots - at), H, D), device=DEV, generator=g)
        out[at:at + some, :H * D * 9 // 16] = _four_bytes(*_four_of(x, 0.01))
    return out


def _prepare_step(c, seed):
    """A two-layer pool, its page tables and the q, K and V of a step."""
    g = _generator(seed)
    tokens, new, prefix = _lengths(c)
    H, D, P, n_req = c["kv_heads"], c["head_dim"], c["page"], c["requests"]
    pages = [-(-n // P) for n in tokens]
    n_pages = sum(pages) + sum(pages) // 4 + 3
    perm = torch.randperm(n_pages, device=DEV, generator=g).to(torch.int32)
    tables = torch.full((n_req, max(pages)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for r, n in enumerate(pages):
        tables[r, :n] = perm[at:at + n]
        at += n
    qt, total, heads = TYPES[c["dtype"]], sum(new), H * c["group"]
    pool = torch.zeros((2, 2, n_pages, P, _token_bytes(c)), dtype=torch.uint8, device=DEV)
    for side in (0, 1):
        pool[side, LAYER].view(n_pages * P, -1).copy_(_random_cache(c, n_pages * P, g))
    k_scale, v_scale = SCALES.get(c["kv"], (1.0, 1.0))
    widths = (heads, H, H) if c["rotary"] else (heads,)
    if c["fused"]:
        x = torch.randn((total, (heads + 2 * H) * D), dtype=qt, device=DEV, generator=g)
        parts, at = [], 0
        for n in widths:
            parts.append(x[:, at * D:(at + n) * D].unflatten(1, (n, D)))
            at += n
    else:
        parts = [torch.randn((total, n, D), dtype=qt, device=DEV, generator=g) for n in widths]
    s = {"case": c, "tables": tables, "tokens": tokens, "new": new, "prefix": prefix,
         "pool": pool, "k_scale": k_scale, "v_scale": v_scale, "q": parts[0]}
    if c["rotary"]:
        s["k"], s["v"] = parts[1:]
        s["q_out"] = torch.empty((total, heads, D), dtype=qt, device=DEV)
        half = torch.arange(c["rotary"] // 2, device=DEV, dtype=torch.float64)
        s["freqs"] = torch.exp(half * (-2.0 / c["rotary"] * math.log(500000.0))).float()
        # Where positions are not places in the request, they come with the step.
        s["positions"] = (torch.cat([torch.arange(n - q, n) for n, q in zip(tokens, new)])
                          .to(torch.int32).to(DEV) + c["far"]) if c["far"] else None
    if c["op"] == "four":
        s["out"] = torch.empty((total, heads, D), dtype=qt, device=DEV)
        # Asked for where the cache is given: behind a rotation of few tokens it shows a last bit
        # of q at full size.
        s["lse"] = (None if c["rotary"] else
                    torch.empty((total, heads), dtype=torch.float32, device=DEV))
        s["slopes"] = (torch.exp2(-8.0 * torch.arange(1, heads + 1, device=DEV) / heads)
                       .float() if c["slopes"] else None)
    if own:
        from paged_kv_gather_gb300 import kvx
        s["kvx_pool"] = kvx.Pool.from_tensor(pool, P)
        reqs = kvx.requests_array([(tables[r].data_ptr(), None, n) for r, n in enumerate(tokens)])
        cfg = kvx.attn_config(q_heads=heads, kv_heads=H, head_dim=D, dtype=c["dtype"],
                              kv_dtype=c["kv"], window=c["window"], softcap=c["softcap"],
                              slopes=s["slopes"].data_ptr() if c["slopes"] else 0)
        s["stream"] = torch.cuda.current_stream().cuda_stream
        s["plan"] = _Plan(kvx.kvx_attn_plan_create(_ctx(), s["kvx_pool"], reqs, new, cfg,
                                                   prefix=prefix, stream=s["stream"]))
        if c["rotary"]:
            s["rope"] = kvx.rope_config(
                s["freqs"].data_ptr(), c["rotary"], interleaved=c["interleaved"],
                positions=s["positions"].data_ptr() if c["far"] else 0)
    else:
        # What the plain form keeps of the step: which row of the packed tokens is which.
        s["lens_dev"] = torch.tensor(tokens, device=DEV)
        s["new_dev"] = torch.tensor(new, device=DEV)
        s["prefix_dev"] = torch.tensor(prefix, device=DEV)
        s["row_request"] = torch.repeat_interleave(torch.arange(n_req, device=DEV), s["new_dev"])
        begin = torch.cumsum(s["new_dev"], 0) - s["new_dev"]
        s["row_index"] = torch.arange(total, device=DEV) - begin[s["row_request"]]
        s["begin"] = begin
        s["scales_dev"] = torch.tensor([k_scale, v_scale], device=DEV)
        s["magnitudes"] = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=DEV)
    return s


def _prepare_select(c, seed):
    """Logits as a model gives them, some tokens ruled out, and the beams' sums so far."""
    g = _generator(seed)
    G, W, V = c["groups"], c["width"], c["vocab"]
    logits = torch.randn((G * W, V), device=DEV, generator=g).mul_(2.0)
    # A few continuations stand out, as they do in text.
    top = torch.randint(0, V, (G * W, 12), device=DEV, generator=g)
    logits.scatter_add_(1, top, torch.rand((G * W, 12), device=DEV, generator=g) * 12.0)
    logits[:, torch.randint(0, V, (V // 50 + 1,), device=DEV, generator=g)] = -math.inf
    logits = logits.to(TYPES[c["dtype"]])
    scores = torch.rand((G, W), device=DEV, generator=g).mul_(-6.0).sub_(20.0)
    done = torch.rand((G, W), device=DEV, generator=g) < c["done"]
    s = {"case": c, "logits": logits, "scores": scores, "done": done.to(torch.uint8),
         "parents": torch.empty((G, c["picks"]), dtype=torch.int32, device=DEV),
         "tokens": torch.empty((G, c["picks"]), dtype=torch.int32, device=DEV),
         "new_scores": torch.empty((G, c["picks"]), device=DEV)}
    if own:
        from paged_kv_gather_gb300 import kvx
        s["cfg"] = kvx.select_config(G, W, V, c["picks"], dtype=c["dtype"], done_token=1)
        s["work"] = torch.empty(kvx.kvx_select_workspace(_ctx(), s["cfg"]), dtype=torch.uint8,
                                device=DEV)
        s["stream"] = torch.cuda.current_stream().cuda_stream
    return s


def _prepare_reorder(c, seed):
    """Beams that share the full pages of a prompt and went different ways after it, each with
    a last page of its own where that is partly filled; half of them are about to be dropped."""
    g = _generator(seed)
    G, W, P = c["groups"], c["width"], c["page"]
    lens = _group_lengths(c)
    pages = [-(-n // P) for n in lens]
    shared = [(n // P) * 3 // 4 for n in lens]      # of the pages, by all beams of the group
    fresh = [W * (p - s) + s for p, s in zip(pages, shared)]
    n_pages = sum(fresh) + sum(fresh) // 4 + 3
    perm = torch.randperm(n_pages, device=DEV, generator=g).to(torch.int32)
    tables = torch.full((G, W, max(pages)), -1, dtype=torch.int32, device=DEV)
    refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    at = 0
    for r in range(G):
        tables[r, :, :shared[r]] = perm[at:at + shared[r]]
        refs[perm[at:at + shared[r]].long()] = W
        at += shared[r]
        n = W * (pages[r] - shared[r])
        tables[r, :, shared[r]:pages[r]] = perm[at:at + n].view(W, -1)
        refs[perm[at:at + n].long()] = 1
        at += n
    order = torch.argsort(torch.rand((G, W), device=DEV, generator=g), 1)
    alive = W - W // 2
    extra = torch.randint(0, alive, (G, W // 2), device=DEV, generator=g)
    parents = torch.cat([order[:, :alive], torch.gather(order, 1, extra)], 1)
    parents = torch.gather(parents, 1, torch.argsort(torch.rand((G, W), device=DEV,
                                                                generator=g), 1))
    s = {"case": c, "tables": tables, "refs": refs, "parents": parents.to(torch.int32),
         "pool": torch.randint(-2**31, 2**31 - 1,
                               (c["kv_factor"], c["layers"], n_pages, P, c["token_bytes"] // 4),
                               dtype=torch.int32, device=DEV, generator=g)}
    if own:
        from paged_kv_gather_gb300 import kvx
        s["kvx_pool"] = kvx.Pool.from_tensor(
            s["pool"].view(torch.uint8).view(c["kv_factor"], c["layers"], n_pages, P,
                                             c["token_bytes"]), P)
        s["beams"] = kvx.beams_array([(tables[r].data_ptr(), tables.stride(1),
                                       s["parents"][r].data_ptr(), W, n)
                                      for r, n in enumerate(lens)])
        s["stream"] = torch.cuda.current_stream().cuda_stream
    else:
        s["lens_dev"] = torch.tensor(lens, device=DEV)
    return s


def prepare(case, seed):
    c = dict(case)
    if c["op"] == "select":
        return _prepare_select(c, seed)
    return _prepare_reorder(c, seed) if c["op"] == "reorder" else _prepare_step(c, seed)


# ------------------------------------------------------------------------------- plain forms

def _four_of(x, scale):
    """Blocks of 16 along the last axis of x / scale in 4 bits: codes (0 .. 15) and scales.  A
    block's scale is its largest magnitude over 6, an element the nearest code, ties to the
    even one."""
    b = x.unflatten(-1, (-1, 16))
    unit = (b.abs().amax(-1) * (1.0 / (6.0 * scale))).clamp(max=448.0).to(torch.float8_e4m3fn)
    u = unit.to(x.dtype)[..., None]
    y = torch.where(u > 0, b / (u * scale), 0.0)
    m = y.abs()
    code = (torch.signbit(y).to(torch.uint8) * 8 + (m > 0.25) + (m >= 0.75) + (m > 1.25)
            + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    return code.flatten(-2), unit


def _four_bytes(code, unit):
    """[tokens, heads, ..] codes and scales as the bytes of a token."""
    return torch.cat([(code[..., 0::2] | code[..., 1::2] << 4).flatten(1),
                      unit.view(torch.uint8).flatten(1)], 1)


def _four_values(raw, H, D, magnitudes):
    """Values of [..., token_bytes] in 4 bits, as [..., H, D] of the type of `magnitudes`."""
    codes = raw[..., :H * D // 2]
    both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    unit = raw[..., H * D // 2:H * D * 9 // 16].contiguous().view(torch.float8_e4m3fn)
    x = magnitudes[both.int()].unflatten(-1, (-1, 16))
    return (x * unit.to(magnitudes.dtype)[..., None]).flatten(-2).unflatten(-1, (H, D))


def _rotated(x, cos, sin, c):
    """x [rows, heads, D] in 32 or 64 bits, its first `rotary` elements turned by the angles."""
    n = c["rotary"]
    a, b = ((x[..., 0:n:2], x[..., 1:n:2]) if c["interleaved"]
            else (x[..., :n // 2], x[..., n // 2:n]))
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if c["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., n:]], -1)


def _places(s):
    return (s["lens_dev"] - s["new_dev"])[s["row_request"]] + s["row_index"]


def _plain_rotate(s):
    c, P = s["case"], s["case"]["page"]
    place = _places(s)
    at = place if s["positions"] is None else s["positions"]
    angle = at.double()[:, None] * s["freqs"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    s["q_out"].copy_(_rotated(s["q"].float(), cos, sin, c))
    slots = s["tables"][s["row_request"], place // P].long() * P + place % P
    for side, x in ((0, _rotated(s["k"].float(), cos, sin, c)), (1, s["v"].float())):
        if c["kv"] == "fp4":
            raw = _four_bytes(*_four_of(x, s["v_scale"] if side else s["k_scale"]))
        else:
            if c["kv"] == "fp8":
                x = (x / s["scales_dev"][side]).clamp(-448.0, 448.0)
            raw = x.to(TYPES[c["kv"]]).flatten(1).view(torch.uint8)
        s["pool"][side, LAYER].view(-1, _token_bytes(c))[slots, :raw.shape[1]] = raw


def _plain_attend(s, q):
    c = s["case"]
    B, H, G, D = c["requests"], c["kv_heads"], c["group"], c["head_dim"]
    T, Q = max(s["tokens"]), max(s["new"])
    j = torch.arange(T, device=DEV)
    slots = s["tables"].clamp(min=0)[:, j // c["page"]].long() * c["page"] + j % c["page"]
    k, v = (_four_values(s["pool"][side, LAYER].view(-1, _token_bytes(c))[slots], H, D,
                         s["magnitudes"]).mul_(s["v_scale"] if side else s["k_scale"])
            for side in (0, 1))
    v = v.masked_fill_((j >= s["lens_dev"][:, None])[:, :, None, None], 0.0)
    i = torch.arange(Q, device=DEV)
    rows = (s["begin"][:, None] + i).clamp(max=q.shape[0] - 1)
    q = q[rows].float().view(B, Q, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, Q * G, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(D))
    if c["softcap"]:
        x.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    x = x.view(B, H, Q, G, T)
    pos = (s["lens_dev"] - s["new_dev"])[:, None] + i                      # [B, Q]
    away = pos[:, :, None] - j                                             # [B, Q, T]
    if s["slopes"] is not None:
        x.addcmul_(s["slopes"].view(1, H, 1, G, 1), away.abs().float()[:, None, :, None],
                   value=-1.0)
    seen = away >= 0
    if c["window"]:
        seen &= away < c["window"]
    seen |= (j < s["prefix_dev"][:, None])[:, None, :]
    seen &= (j < s["lens_dev"][:, None])[:, None, :]
    x.masked_fill_(~seen[:, None, :, None], float("-inf"))
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)   # a padded row may see nothing
    x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, H, Q * G, T), v.permute(0, 2, 1, 3)).view(B, H, Q, G, D) / l
    o = o.permute(0, 2, 1, 3, 4).reshape(B, Q, H * G, D)
    pick = s["row_request"], s["row_index"]
    out = o[pick].to(TYPES[c["dtype"]])
    if s["lse"] is None:
        return {"out": out}
    lse = (m + torch.log(l))[..., 0].permute(0, 2, 1, 3).reshape(B, Q, H * G)
    return {"out": out, "lse": lse[pick]}


def _plain_select(s):
    """Within a beam candidates go by logit, then by token; across beams by their sums, which
    are taken in 64 bits, then by beam."""
    c = s["case"]
    G, W, V, K = c["groups"], c["width"], c["vocab"], c["picks"]
    x = s["logits"].float()
    m = x.amax(1)
    log_sum = torch.log(torch.exp(x - m[:, None]).sum(1, dtype=torch.float64)) + m.double()
    bits = x.view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() << 32
    order += V - 1 - torch.arange(V, device=DEV)
    best = torch.topk(order, min(K, V), 1).values
    token = V - 1 - (best & 0xFFFFFFFF)
    so_far = s["scores"].double().view(-1, 1)
    score = so_far + (x.gather(1, token).double() - log_sum[:, None])
    # A beam that is done stays as it is: one candidate, its own sum.
    done = s["done"].view(-1, 1) != 0
    first = torch.arange(min(K, V), device=DEV) == 0
    score = torch.where(done, torch.where(first, so_far, -math.inf), score).view(G, -1)
    token = torch.where(done, 1, token)
    token = torch.where(done & ~first, V, token).view(G, -1)
    beam = torch.arange(W, device=DEV).repeat_interleave(min(K, V)).expand(G, -1)
    by_index = torch.argsort(beam * (V + 1) + token, 1)
    score, token, beam = (t.gather(1, by_index) for t in (score, token, beam))
    top = torch.argsort(score, dim=1, descending=True, stable=True)[:, :K]
    score = score.gather(1, top)
    none = score == -math.inf           # fewer candidates than wanted
    s["parents"].copy_(torch.where(none, 0, beam.gather(1, top)))
    s["tokens"].copy_(torch.where(none, -1, token.gather(1, top)))
    s["new_scores"].copy_(score)


def _plain_reorder(s):
    """A beam takes its parent's full pages.  Of the beams that continue one parent, the first
    takes its partly filled last page too; the i-th of the others gets the last page of the
    i-th beam that nobody continues, and a copy of the parent's in it."""
    c = s["case"]
    G, W, P = c["groups"], c["width"], c["page"]
    tables, parents = s["tables"], s["parents"].long()
    n = torch.zeros_like(parents).scatter_add_(1, parents, torch.ones_like(parents))
    full = (s["lens_dev"] // P)[:, None, None]
    tail = s["lens_dev"] % P
    j = torch.arange(tables.shape[2], device=DEV)
    is_full = (j < full).expand_as(tables)
    s["refs"].scatter_add_(0, tables.clamp(min=0).long().flatten(),
                           torch.where(is_full, (n - 1)[:, :, None], 0).int().flatten())
    taken = torch.gather(tables, 1, parents[:, :, None].expand(-1, -1, tables.shape[2]))
    # Last pages, partly filled.
    beam = torch.arange(W, device=DEV)
    extra = ((parents[:, :, None] == parents[:, None]) & (beam < beam[:, None])).any(2)
    dropped = torch.argsort((n > 0).int(), dim=1, stable=True)
    rank = (torch.cumsum(extra.long(), 1) - 1).clamp(min=0)
    giver = torch.where(extra, torch.gather(dropped, 1, rank), parents)
    last = full[:, 0].expand(G, W).clamp(max=tables.shape[2] - 1)
    mine = torch.gather(tables, 2, last[:, :, None])[:, :, 0]
    source, target = torch.gather(mine, 1, parents), torch.gather(mine, 1, giver)
    is_last = (j == full) & (tail > 0)[:, None, None]
    tables.copy_(torch.where(is_full, taken, torch.where(is_last, target[:, :, None], tables)))
    t = torch.arange(P, device=DEV)
    moved = (extra & (tail > 0)[:, None])[:, :, None] & (t < tail[:, None, None])
    a = (source.long()[:, :, None] * P + t)[moved]
    b = (target.long()[:, :, None] * P + t)[moved]
    flat = s["pool"].view(c["kv_factor"], c["layers"], -1, c["token_bytes"] // 4)
    flat[:, :, b] = flat[:, :, a]


# ------------------------------------------------------------------------------- own forms

def _own_rotate(s):
    from paged_kv_gather_gb300 import kvx
    kvx.kvx_append_rotated(s["plan"].handle, LAYER, s["rope"], s["k"].data_ptr(),
                           s["v"].data_ptr(), q=s["q"].data_ptr(), q_out=s["q_out"].data_ptr(),
                           k_stride=s["k"].stride(0), v_stride=s["v"].stride(0),
                           q_stride=s["q"].stride(0), k_scale=s["k_scale"],
                           v_scale=s["v_scale"], stream=s["stream"])


def _own_attend(s, q):
    from paged_kv_gather_gb300 import kvx
    kvx.kvx_attend(s["plan"].handle, LAYER, q.data_ptr(), s["out"].data_ptr(),
                   q_stride=q.stride(0), lse=0 if s["lse"] is None else s["lse"].data_ptr(),
                   k_scale=s["k_scale"], v_scale=s["v_scale"], stream=s["stream"])
    return {"out": s["out"]} if s["lse"] is None else {"out": s["out"], "lse": s["lse"]}


def _own_select(s):
    from paged_kv_gather_gb300 import kvx
    kvx.kvx_select_beams(_ctx(), s["cfg"], s["logits"].data_ptr(), s["scores"].data_ptr(),
                         s["parents"].data_ptr(), s["tokens"].data_ptr(),
                         s["new_scores"].data_ptr(), s["work"].data_ptr(),
                         done=s["done"].data_ptr(), stream=s["stream"])


def _own_reorder(s):
    from paged_kv_gather_gb300 import kvx
    kvx.kvx_reorder_beams(_ctx(), s["kvx_pool"], s["refs"].data_ptr(), s["beams"],
                          stream=s["stream"])


def _cache_values(s):
    """What a step changed in the cache: the layer's K and V in its own type, and of a 4-bit
    cache the scales (its codes show in the attention that follows)."""
    c = s["case"]
    H, D = c["kv_heads"], c["head_dim"]
    if c["kv"] == "fp4":
        return {"kv"[side] + "_scales": s["pool"][side, LAYER, :, :, H * D // 2:H * D * 9 // 16]
                .view(torch.float8_e4m3fn) for side in (0, 1)}
    return {"kv"[side]: s["pool"][side, LAYER].view(TYPES[c["kv"]]) for side in (0, 1)}


def run(state):
    s = state
    op = s["case"]["op"]
    if op == "select":
        (_own_select if own else _plain_select)(s)
        return {"parents": s["parents"], "tokens": s["tokens"], "scores": s["new_scores"]}
    if op == "reorder":
        (_own_reorder if own else _plain_reorder)(s)
        return {"refs": s["refs"], "tables": s["tables"], "pool": s["pool"]}
    got, q = {}, s["q"]
    if s["case"]["rotary"]:
        (_own_rotate if own else _plain_rotate)(s)
        q = s["q_out"]
        got = {"q": q, **_cache_values(s)}
    if op == "four":
        got.update((_own_attend if own else _plain_attend)(s, q))
    return got


# ------------------------------------------------------------------------------- work

def _seen(pos, n, window, prefix):
    """Keys that the row at position `pos` of a request of n tokens sees."""
    low = max(0, pos - window + 1) if window else 0
    return pos + 1 - low + max(0, min(prefix, n) - pos - 1) + min(prefix, low)


def work(case):
    c = dict(case)
    if c["op"] == "select":
        rows = c["groups"] * c["width"] * (1.0 - c["done"])
        return {"bytes": rows * c["vocab"] * ITEM[c["dtype"]] + 12.0 * c["groups"] * c["picks"],
                "flops": 4.0 * rows * c["vocab"]}
    if c["op"] == "reorder":
        lens, P = _group_lengths(c), c["page"]
        moved = sum(n % P for n in lens) * (c["width"] // 2)
        entries = sum(-(-n // P) for n in lens) * c["width"]
        # Tables read and written, and a count per entry.
        return {"bytes": 2.0 * moved * c["layers"] * c["kv_factor"] * c["token_bytes"]
                + 16.0 * entries, "flops": 0.0}
    tokens, new, prefix = _lengths(c)
    rows, D, item = sum(new), c["head_dim"], ITEM[c["dtype"]]
    heads = c["kv_heads"] * c["group"]
    w = {"bytes": 0.0, "flops": 0.0}
    if c["rotary"]:
        w["bytes"] += rows * (2.0 * heads + 2.0 * c["kv_heads"]) * D * item
        w["bytes"] += 2.0 * rows * _token_bytes(c)
        w["flops"] += 3.0 * rows * (heads + c["kv_heads"]) * c["rotary"]
    if c["op"] == "four":
        keys, pairs = 0, 0
        for n, q, p in zip(tokens, new, prefix):
            first = max(0, n - q - c["window"] + 1) if c["window"] else 0
            keys += n - first + min(p, first)
            pairs += sum(_seen(pos, n, c["window"], p) for pos in range(n - q, n))
        w["bytes"] += (2.0 * keys * _token_bytes(c)
                       + rows * heads * (2.0 * D * item + (0 if c["rotary"] else 4)))
        w["flops"] += 4.0 * D * heads * pairs
    return w


# ------------------------------------------------------------------------------- 64 bits

def _exact_four(x, scale):
    """(scale, value) of the 4-bit cache's elements from x in 64 bits, by the nearest of all
    the values that a code may have."""
    block = x.reshape(*x.shape[:-1], -1, 16) / scale
    unit = (block.abs().max(-1).values / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn).double()
    grid = torch.tensor(MAGNITUDES, dtype=torch.float64, device=DEV)
    middle = (grid[1:] + grid[:-1]) / 2
    size = block.abs() / unit.clamp(min=1e-30)[..., None]
    # Above a middle the next code; on it the even one.
    code = torch.bucketize(size, middle)
    code += (torch.isin(size, middle) & (code % 2 == 1)).long()
    return unit, (grid[code] * block.sign() * unit[..., None] * scale).reshape(x.shape)


def exact(case, seed):
    """Rotation, the casts into the cache, attention and candidates' sums from their
    definitions, in 64 bits.  Pages, parents and tokens are whole numbers only."""
    c = dict(case)
    if c["op"] == "reorder" or work(c)["flops"] > 4e12:
        return None
    global own
    kept, own = own, False
    try:
        s = _prepare_select(c, seed) if c["op"] == "select" else _prepare_step(c, seed)
    finally:
        own = kept
    if c["op"] == "select":
        best = []
        for g in range(c["groups"]):
            rows = s["logits"][g * c["width"]:(g + 1) * c["width"]].double()
            sums = s["scores"][g].double()
            each = sums[:, None] + torch.log_softmax(rows, 1)
            stays = s["done"][g] != 0
            all_ = torch.cat([each[~stays].flatten(), sums[stays]])
            all_ = torch.cat([all_, all_.new_full((c["picks"],), -math.inf)])
            best.append(all_.sort(descending=True).values[:c["picks"]])
        return {"parents": None, "tokens": None, "scores": torch.stack(best)}
    H, D, G, P = c["kv_heads"], c["head_dim"], c["group"], c["page"]
    tables = s["tables"].cpu().long()
    scales = (s["k_scale"], s["v_scale"])
    double = s["magnitudes"].double()

    def cache(side):
        raw = s["pool"][side, LAYER]
        if c["kv"] == "fp4":
            return _four_values(raw, H, D, double) * scales[side]
        return raw.view(TYPES[c["kv"]]).double().unflatten(-1, (H, D))

    layer, got, q = [cache(0), cache(1)], {}, s["q"].double()
    if c["rotary"]:
        place = torch.cat([torch.arange(n - m, n) for n, m in zip(s["tokens"], s["new"])])
        request = torch.repeat_interleave(torch.arange(len(s["new"])), torch.tensor(s["new"]))
        page, slot = tables[request, place // P].to(DEV), (place % P).to(DEV)
        phase = (place + c["far"]).double().to(DEV)[:, None] * s["freqs"].double()[None]
        turn = torch.polar(torch.ones_like(phase), phase)[:, None]

        def turned(x):
            x = x.double().clone()
            n = c["rotary"]
            first, second = ((slice(0, n, 2), slice(1, n, 2)) if c["interleaved"]
                             else (slice(0, n // 2), slice(n // 2, n)))
            z = torch.complex(x[..., first], x[..., second]) * turn
            x[..., first], x[..., second] = z.real, z.imag
            return x

        q = turned(s["q"])
        got["q"] = q
        for side, x in ((0, turned(s["k"])), (1, s["v"].double())):
            if c["kv"] == "fp4":
                unit, x = _exact_four(x, scales[side])
                raw = s["pool"][side, LAYER, :, :, H * D // 2:H * D * 9 // 16].contiguous()
                units = raw.view(torch.float8_e4m3fn).double()
                units[page, slot] = unit.flatten(1)
                got["kv"[side] + "_scales"] = units
                layer[side][page, slot] = x
            else:
                if c["kv"] == "fp8":
                    x = (x / scales[side]).clamp(-448.0, 448.0)
                layer[side][page, slot] = x
                got["kv"[side]] = layer[side].flatten(2)
        q = q.to(TYPES[c["dtype"]]).double()     # q_out is of q's type
    if c["op"] == "rotate":
        return got
    out = torch.empty(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(q.shape[:2], dtype=torch.float64, device=DEV)
    row = 0
    for r, (n, m, prefix) in enumerate(zip(s["tokens"], s["new"], s["prefix"])):
        pages = tables[r, :-(-n // P)].to(DEV)
        key, val = (x[pages].flatten(0, 1)[:n] for x in layer)
        place = torch.arange(n, device=DEV, dtype=torch.float64)
        gap = torch.arange(n - m, n, device=DEV, dtype=torch.float64)[:, None] - place[None]
        hidden = gap < 0
        if c["window"]:
            hidden |= gap >= c["window"]
        hidden &= ~(place < prefix)[None]
        for h in range(H * G):
            z = q[row:row + m, h] @ key[:, h // G].T / math.sqrt(D)
            if c["softcap"]:
                z = c["softcap"] * torch.tanh(z / c["softcap"])
            if s["slopes"] is not None:
                z = z - s["slopes"][h].double() * gap.abs()
            z = z.masked_fill(hidden, -math.inf)
            norm = torch.logsumexp(z, dim=1)
            lse[row:row + m, h] = norm
            out[row:row + m, h] = torch.exp(z - norm[:, None]) @ val[:, h // G]
        row += m
    got["out"] = out
    if s["lse"] is not None:
        got["lse"] = lse
    return got
