"""The operators that work on a paged KV cache in place, as measurable cases.

Four operators of a serving step around the page pools of this library:

* ``fork``: give the pages of finished continuations back and fork requests into new ones
  (``kvx_free_pages`` + ``kvx_fork_pages``): full pages are shared by reference count, a
  partly filled last page is copied, or every page is (``copy``).
* ``compact``: move the live pages of a fragmented pool to its front and rewrite the page
  tables (``kvx_compact_pages``).
* ``append``: write the K and V of new tokens into their pages (``kvx_append_tokens``).
* ``attend``: attention of a chunk of new tokens over the paged cache (``kvx_attend``), with
  its single-token form, a cap on the scores, a bias by distance, a sliding window and a
  prefix that every row sees.

``own`` selects the form ``run`` takes: False is elementary torch in 32 bits, True the calls
of this library.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
LAYER = 1            # attend and append work on this layer of a two-layer pool
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}
ITEM = {"bf16": 2, "fp16": 2, "fp8": 1}


# ------------------------------------------------------------------------------- cases

def _attend(name, requests, new, length, kv_heads, group, head_dim, page, kv="bf16", dtype="bf16",
            window=0, prefix=0, softcap=0.0, slopes=False, fused=False):
    return {"name": name, "op": "attend", "requests": requests, "new_min": new[0],
            "new_max": new[1], "len_min": length[0], "len_max": length[1], "kv_heads": kv_heads,
            "group": group, "head_dim": head_dim, "page": page, "kv": kv, "dtype": dtype,
            "window": window, "prefix": prefix, "softcap": softcap, "slopes": slopes,
            "fused": fused}


def _append(name, requests, new, length, kv_heads, head_dim, page, kv="bf16", dtype="bf16",
            fused=False):
    return {"name": name, "op": "append", "requests": requests, "new_min": new[0],
            "new_max": new[1], "len_min": length[0], "len_max": length[1], "kv_heads": kv_heads,
            "head_dim": head_dim, "page": page, "kv": kv, "dtype": dtype, "fused": fused}


def _fork(name, parents, children, length, layers, kv_factor, token_bytes, page, copy=False):
    return {"name": name, "op": "fork", "parents": parents, "children": children,
            "len_min": length[0], "len_max": length[1], "layers": layers,
            "kv_factor": kv_factor, "token_bytes": token_bytes, "page": page, "copy": copy}


def _compact(name, requests, length, live, pages, layers, kv_factor, token_bytes, page):
    return {"name": name, "op": "compact", "requests": requests, "len_min": length[0],
            "len_max": length[1], "live": live, "pages": pages, "layers": layers,
            "kv_factor": kv_factor, "token_bytes": token_bytes, "page": page}


def listed():
    return [
        # One prompt of the 8B-shaped cache continued four ways (parallel sampling): only the
        # last page of each child is copied, so the call's latency is what counts.
        _fork("fork_one", 1, 4, (1001, 1001), 32, 2, 2048, 16),
        # A beam step of a batch of ragged requests on the fp8 cache.
        _fork("fork_batch", 32, 2, (512, 8192), 28, 2, 512, 16),
        # Requests copied outright, every page of them (a child that will be edited in place).
        _fork("fork_copy", 6, 1, (1000, 6000), 32, 2, 2048, 16, copy=True),
        # The small pool, half of it live: latency.
        _compact("compact_small", 3, (200, 800), 0.5, 256, 4, 2, 256, 16),
        # The 8B-shaped pool with 60 % of its pages live: gigabytes move.
        _compact("compact_large", 24, (512, 4096), 0.6, 4096, 32, 2, 2048, 16),
        # One new token for each of 64 requests, cast to the fp8 cache.
        _append("append_decode", 64, (1, 1), (1024, 32768), 4, 128, 16, kv="fp8"),
        # Prefill chunks of several requests, K and V taken out of a fused projection.
        _append("append_chunk", 5, (1000, 2048), (2048, 16384), 8, 128, 32, fused=True),
        # A single token of one short request: the smallest call.
        _attend("decode_one", 1, (1, 1), (1000, 1000), 2, 4, 64, 16, kv="fp16", dtype="fp16"),
        # A decoding batch over ragged fp8 contexts, 7 query heads to a KV head.
        _attend("decode_batch", 64, (1, 1), (1024, 32768), 4, 7, 128, 16, kv="fp8"),
        # Several requests with a few new tokens up to a prefill chunk, every score option on.
        _attend("chunk_ragged", 6, (1, 700), (1, 9000), 4, 4, 128, 16, window=2048, prefix=130,
                softcap=30.0, slopes=True, fused=True),
        # A small chunk at the end of a long context (chunked prefill beside decoding).
        _attend("chunk_long", 1, (512, 512), (32768, 32768), 8, 4, 128, 16),
        # The largest: a chunk with 64 query heads, 32-token pages.
        _attend("chunk_large", 1, (2048, 2048), (32768, 32768), 8, 8, 128, 32),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fork", "compact", "append", "attend", "attend", "attend"])
    if op == "fork":
        page = rng.choice([1, 7, 16, 16, 32, 64])
        token_bytes = rng.choice([256, 512, 1152, 2048])
        kv_factor = 1 if token_bytes == 1152 else 2
        layers = rng.randint(4, 32)
        copy = rng.random() < 0.4
        children = rng.randint(1, 4)
        # Tokens of the whole pool stay within 6 GB of K and V.
        room = int(6e9 / (layers * kv_factor * token_bytes) / (2.0 + children * copy) / 2)
        parents = _log_int(rng, 1, 32)
        hi = max(40, min(8192, room // parents))
        lo = _log_int(rng, 1, hi)
        c = _fork("", parents, children, (lo, hi), layers, kv_factor, token_bytes, page, copy)
    elif op == "compact":
        page = rng.choice([1, 7, 16, 32, 64])
        token_bytes = rng.choice([256, 512, 1152, 2048])
        kv_factor = 1 if token_bytes == 1152 else 2
        layers = rng.randint(2, 32)
        most = int(6e9 / (layers * kv_factor * token_bytes * page))
        pages = _log_int(rng, 64, max(65, min(65536, most)))
        live = rng.uniform(0.2, 0.9)
        per = max(1, int(pages * live * page / 6))
        c = _compact("", 24, (max(1, per // 4), per), round(live, 3), pages, layers, kv_factor,
                     token_bytes, page)
    elif op == "append":
        dtype = rng.choice(["bf16", "fp16"])
        kv = rng.choice([dtype, "fp8"])
        decode = rng.random() < 0.5
        requests = _log_int(rng, 1, 64)
        new = (1, 1) if decode else (1, _log_int(rng, 2, 8192 // requests + 2))
        hi = _log_int(rng, new[1], 16384)
        c = _append("", requests, new, (min(hi, 1 + rng.randint(0, 1000)), hi),
                    rng.choice([1, 2, 4, 8]), rng.choice([64, 128]),
                    rng.choice([1, 5, 16, 32, 64]), kv, dtype, rng.random() < 0.5)
    else:
        dtype = rng.choice(["bf16", "bf16", "fp16"])
        kv = rng.choice([dtype, dtype, "fp8"])
        kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8])
        kind = rng.choice(["one", "few", "chunk"])
        if kind == "one":
            requests, new = _log_int(rng, 1, 64), (1, 1)
        elif kind == "few":
            requests, new = _log_int(rng, 1, 32), (1, rng.randint(2, 16))
        else:
            requests, new = _log_int(rng, 1, 8), (1, _log_int(rng, 17, 2048))
        # The plain form's scores and gathered K stay below the largest listed case's.
        hi = min(32768, int(2.0e9 / (requests * new[1] * kv_heads * group)),
                 int(0.5e9 / (requests * kv_heads * 128)))
        hi = _log_int(rng, min(hi, max(16, new[1], hi // 64)), hi)
        odd = rng.random() < 0.5
        c = _attend("", requests, new, (_log_int(rng, 1, hi), hi), kv_heads, group,
                    rng.choice([64, 128, 128]), rng.choice([1, 5, 8, 16, 16, 24, 32, 64]), kv,
                    dtype, window=_log_int(rng, 16, 8192) if odd and rng.random() < 0.6 else 0,
                    prefix=rng.randint(1, 300) if odd and rng.random() < 0.5 else 0,
                    softcap=rng.choice([0.0, 20.0, 50.0]) if odd else 0.0,
                    slopes=odd and rng.random() < 0.5, fused=rng.random() < 0.5)
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
    p = c.get("prefix", 0)
    return tokens, new, [min(p * (i % 3), n) for i, n in enumerate(tokens)]


def _request_lengths(c):
    r = random.Random("%d %d %d" % (c.get("parents", 0) or c["requests"], c["len_min"],
                                    c["len_max"]))
    n = c["parents"] if c["op"] == "fork" else c["requests"]
    return [c["len_max"] if i == 0 else _log_int(r, c["len_min"], c["len_max"]) for i in range(n)]


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


def _normal(shape, dtype, g, scale=1.0):
    x = torch.randn(shape, dtype=torch.bfloat16 if dtype == torch.float8_e4m3fn else dtype,
                    device=DEV, generator=g)
    if scale != 1.0:
        x.mul_(scale)
    return x.to(dtype)


def _prepare_step(c, seed):
    """A two-layer pool, its page tables and the new tokens of a step."""
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
    kt, qt = TYPES[c["kv"]], TYPES[c["dtype"]]
    fp8 = c["kv"] == "fp8"
    # fp8 codes are the values over a scale, as a calibrated cache keeps them.
    s = {"case": c, "tables": tables, "tokens": tokens, "new": new, "prefix": prefix,
         "k_scale": 0.03 if fp8 else 1.0, "v_scale": 0.05 if fp8 else 1.0,
         "pool": _normal((2, 2, n_pages, P, H, D), kt, g, 25.0 if fp8 else 1.0)}
    total = sum(new)
    if c["op"] == "attend":
        heads = H * c["group"]
        width = (heads + 2 * H) * D if c["fused"] else heads * D
        x = _normal((total, width), qt, g, 1.5)
        s["q"] = x[:, :heads * D].unflatten(1, (heads, D))
        s["out"] = torch.empty((total, heads, D), dtype=qt, device=DEV)
        s["lse"] = torch.empty((total, heads), dtype=torch.float32, device=DEV)
        s["slopes"] = (torch.exp2(-8.0 * torch.arange(1, heads + 1, device=DEV) / heads)
                       .float() if c["slopes"] else None)
    else:
        if c["fused"]:
            x = _normal((total, 6 * H * D), qt, g)
            s["k"], s["v"] = (x[:, a * H * D:(a + 1) * H * D].unflatten(1, (H, D)) for a in (4, 5))
        else:
            s["k"], s["v"] = _normal((total, H, D), qt, g), _normal((total, H, D), qt, g)
    if own:
        from paged_kv_gather_gb300 import kvx
        raw = s["pool"].view(torch.uint8).view(2, 2, n_pages, P, H * D * ITEM[c["kv"]])
        s["kvx_pool"] = kvx.Pool.from_tensor(raw, P)
        reqs = kvx.requests_array([(tables[r].data_ptr(), None, n) for r, n in enumerate(tokens)])
        cfg = kvx.attn_config(q_heads=H * c.get("group", 1), kv_heads=H, head_dim=D,
                              dtype=c["dtype"], kv_dtype=c["kv"], window=c.get("window", 0),
                              softcap=c.get("softcap", 0.0),
                              slopes=s["slopes"].data_ptr() if c.get("slopes") else 0)
        s["stream"] = torch.cuda.current_stream().cuda_stream
        s["plan"] = _Plan(kvx.kvx_attn_plan_create(_ctx(), s["kvx_pool"], reqs, new, cfg,
                                                   prefix=prefix, stream=s["stream"]))
    else:
        # What the plain form keeps of the step: which row of the packed tokens is which.
        s["lens_dev"] = torch.tensor(tokens, device=DEV)
        s["new_dev"] = torch.tensor(new, device=DEV)
        s["prefix_dev"] = torch.tensor(prefix, device=DEV)
        s["row_request"] = torch.repeat_interleave(torch.arange(n_req, device=DEV), s["new_dev"])
        begin = torch.cumsum(s["new_dev"], 0) - s["new_dev"]
        s["row_index"] = torch.arange(total, device=DEV) - begin[s["row_request"]]
        s["begin"] = begin
    return s


def _random_pool(c, n_pages, g):
    words = c["token_bytes"] // 4
    return torch.randint(-2**31, 2**31 - 1, (c["kv_factor"], c["layers"], n_pages, c["page"], words),
                         dtype=torch.int32, device=DEV, generator=g)


def _prepare_fork(c, seed):
    """Parents on random pages of a pool, and children of an earlier step that still hold
    theirs: a pass frees those and forks the parents again."""
    g = _generator(seed)
    P, copy = c["page"], c["copy"]
    lens = _request_lengths(c)
    pages = [-(-n // P) for n in lens]
    # A child has room for 1..2 pages of tokens of its own.
    rows = [(i, lens[i], lens[i] + 1 + (7 * k + 3) % (2 * P)) for i in range(len(lens))
            for k in range(c["children"])]
    full = [0 if copy else n // P for _, n, _ in rows]
    total = [-(-t // P) for _, _, t in rows]
    fresh = sum(t - f for f, t in zip(full, total))
    n_pages = sum(pages) + fresh + fresh // 2 + 8
    perm = torch.randperm(n_pages, device=DEV, generator=g).to(torch.int32)
    parents = torch.full((len(lens), max(pages)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for r, n in enumerate(pages):
        parents[r, :n] = perm[at:at + n]
        at += n
    refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    refs[perm[:at].long()] = 1
    children = torch.full((len(rows), max(total)), -1, dtype=torch.int32, device=DEV)
    for r, (p, _, _) in enumerate(rows):
        children[r, :full[r]] = parents[p, :full[r]]
        refs[children[r, :full[r]].long()] += 1
        n = total[r] - full[r]
        children[r, full[r]:total[r]] = perm[at:at + n]
        refs[perm[at:at + n].long()] = 1
        at += n
    s = {"case": c, "refs": refs, "parents": parents, "children": children,
         "pool": _random_pool(c, n_pages, g)}
    if own:
        from paged_kv_gather_gb300 import kvx
        s["kvx_pool"] = kvx.Pool.from_tensor(
            s["pool"].view(torch.uint8).view(c["kv_factor"], c["layers"], n_pages, P,
                                             c["token_bytes"]), P)
        s["tables"] = kvx.tables_array([(children[r].data_ptr(), n) for r, n in enumerate(total)])
        s["forks"] = kvx.forks_array([(parents[p].data_ptr(), children[r].data_ptr(), n, t, copy)
                                      for r, (p, n, t) in enumerate(rows)])
        s["stream"] = torch.cuda.current_stream().cuda_stream
    else:
        s["fresh"] = fresh
        s["row_parent"] = torch.tensor([p for p, _, _ in rows], device=DEV)
        s["full"] = torch.tensor(full, device=DEV)
        s["total"] = torch.tensor(total, device=DEV)
        # Tokens that are copied, as (child, token) pairs.
        first = [f * P for f in full]
        s["copied"] = torch.tensor([n - f for (_, n, _), f in zip(rows, first)], device=DEV)
        s["copied_total"] = sum(n - f for (_, n, _), f in zip(rows, first))
    return s


def _prepare_compact(c, seed):
    g = _generator(seed)
    P, n_pages = c["page"], c["pages"]
    room = int(n_pages * c["live"])
    tables, at = [], 0
    for n in _request_lengths(c):
        k = min(-(-n // P), room - at)
        if k > 0:
            tables.append((at, k))
            at += k
    perm = torch.randperm(n_pages, device=DEV, generator=g).to(torch.int32)
    width = max(k for _, k in tables)
    t = torch.full((len(tables) + 1, width), -1, dtype=torch.int32, device=DEV)
    refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    for r, (a, k) in enumerate(tables):
        t[r, :k] = perm[a:a + k]
    refs[perm[:at].long()] = 1
    # The last table is a fork of the first: it names the same pages.
    half = tables[0][1] // 2 + 1 if tables[0][1] > 1 else 1
    t[-1, :half] = t[0, :half]
    refs[t[0, :half].long()] += 1
    counts = [k for _, k in tables] + [half]
    s = {"case": c, "refs0": refs, "tables0": t, "refs": refs.clone(), "tables": t.clone(),
         "n_live": torch.zeros(1, dtype=torch.int32, device=DEV),
         "pool": _random_pool(c, n_pages, g)}
    if own:
        from paged_kv_gather_gb300 import kvx
        s["kvx_pool"] = kvx.Pool.from_tensor(
            s["pool"].view(torch.uint8).view(c["kv_factor"], c["layers"], n_pages, P,
                                             c["token_bytes"]), P)
        s["table_args"] = kvx.tables_array([(s["tables"][r].data_ptr(), k)
                                            for r, k in enumerate(counts)])
        s["stream"] = torch.cuda.current_stream().cuda_stream
    return s


def prepare(case, seed):
    c = dict(case)
    if c["op"] == "fork":
        return _prepare_fork(c, seed)
    if c["op"] == "compact":
        return _prepare_compact(c, seed)
    return _prepare_step(c, seed)


# ------------------------------------------------------------------------------- plain forms

def _slots(tables, j, page):
    """Slot of logical token j of each table: its page's first slot plus its place there."""
    return tables[:, j // page].long() * page + j % page


def _plain_attend(s):
    c = s["case"]
    B, H, G, D = c["requests"], c["kv_heads"], c["group"], c["head_dim"]
    T, Q = max(s["tokens"]), max(s["new"])
    j = torch.arange(T, device=DEV)
    slots = _slots(s["tables"].clamp(min=0), j, c["page"])
    k = s["pool"][0, LAYER].reshape(-1, H, D)[slots].float() * s["k_scale"]
    v = s["pool"][1, LAYER].reshape(-1, H, D)[slots].float() * s["v_scale"]
    v = v.masked_fill((j >= s["lens_dev"][:, None])[:, :, None, None], 0.0)
    i = torch.arange(Q, device=DEV)
    rows = (s["begin"][:, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().view(B, Q, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, Q * G, D)
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
    lse = (m + torch.log(l))[..., 0]
    o = o.permute(0, 2, 1, 3, 4).reshape(B, Q, H * G, D)
    lse = lse.permute(0, 2, 1, 3).reshape(B, Q, H * G)
    pick = s["row_request"], s["row_index"]
    return {"out": o[pick].to(TYPES[c["dtype"]]), "lse": lse[pick]}


def _plain_append(s):
    c = s["case"]
    H, D, P = c["kv_heads"], c["head_dim"], c["page"]
    r = s["row_request"]
    pos = (s["lens_dev"] - s["new_dev"])[r] + s["row_index"]
    slots = s["tables"][r, pos // P].long() * P + pos % P
    out = []
    for side, x, scale in ((0, s["k"], s["k_scale"]), (1, s["v"], s["v_scale"])):
        layer = s["pool"][side, LAYER]
        if c["kv"] == "fp8":
            x = (x.float() / scale).clamp(-448.0, 448.0)
        # Indexed as bytes: torch has no scatter for 8-bit floats.
        layer.view(torch.uint8).view(-1, H * D * ITEM[c["kv"]])[slots] = (
            x.to(layer.dtype).contiguous().view(torch.uint8).view(-1, H * D * ITEM[c["kv"]]))
        out.append(layer)
    return {"k": out[0], "v": out[1]}


def _plain_fork(s):
    c = s["case"]
    P = c["page"]
    refs, children = s["refs"], s["children"]
    j = torch.arange(children.shape[1], device=DEV)
    held = j < s["total"][:, None]
    # Free the children of the last step.
    refs.scatter_add_(0, children.clamp(min=0).long().flatten(), -held.int().flatten())
    # Fresh pages are the free pages in ascending order.
    free = torch.argsort((refs != 0).int(), stable=True)[:s["fresh"]].int()
    fresh = held & (j >= s["full"][:, None])
    rank = (torch.cumsum(fresh.flatten().int(), 0) - 1).clamp(min=0).view_as(fresh)
    parents = torch.nn.functional.pad(s["parents"][s["row_parent"]],
                                      (0, children.shape[1] - s["parents"].shape[1]), value=-1)
    children.copy_(torch.where(fresh, free[rank], torch.where(held, parents, -1)))
    refs.scatter_add_(0, children.clamp(min=0).long().flatten(), held.int().flatten())
    # Copy the tokens of the pages that are not shared.
    row = torch.repeat_interleave(torch.arange(len(s["full"]), device=DEV), s["copied"],
                                  output_size=s["copied_total"])
    begin = torch.cumsum(s["copied"], 0) - s["copied"]
    t = torch.arange(s["copied_total"], device=DEV) - begin[row] + s["full"][row] * P
    flat = s["pool"].view(c["kv_factor"], c["layers"], -1, c["token_bytes"] // 4)
    flat[:, :, children[row, t // P].long() * P + t % P] = (
        flat[:, :, parents[row, t // P].long() * P + t % P])
    return {"refs": refs, "children": children, "pool": s["pool"]}


def _plain_compact(s):
    refs, tables = s["refs"], s["tables"]
    ids = torch.arange(refs.shape[0], device=DEV)
    live = refs > 0
    n_live = live.sum()
    holes = torch.nonzero(~live & (ids < n_live))[:, 0]
    moved = torch.nonzero(live & (ids >= n_live))[:, 0]
    new = ids.clone()
    new[moved] = holes
    s["pool"][:, :, holes] = s["pool"][:, :, moved]
    refs[holes] = refs[moved]
    refs[moved] = 0
    tables.copy_(torch.where(tables >= 0, new[tables.clamp(min=0).long()].int(), tables))
    s["n_live"].copy_(n_live)
    return {"refs": refs, "tables": tables, "n_live": s["n_live"], "pool": s["pool"]}


# ------------------------------------------------------------------------------- own forms

def _own_attend(s):
    from paged_kv_gather_gb300 import kvx
    kvx.kvx_attend(s["plan"].handle, LAYER, s["q"].data_ptr(), s["out"].data_ptr(),
                   q_stride=s["q"].stride(0), lse=s["lse"].data_ptr(), k_scale=s["k_scale"],
                   v_scale=s["v_scale"], stream=s["stream"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_append(s):
    from paged_kv_gather_gb300 import kvx
    kvx.kvx_append_tokens(s["plan"].handle, LAYER, s["k"].data_ptr(), s["v"].data_ptr(),
                          k_stride=s["k"].stride(0), v_stride=s["v"].stride(0),
                          k_scale=s["k_scale"], v_scale=s["v_scale"], stream=s["stream"])
    return {"k": s["pool"][0, LAYER], "v": s["pool"][1, LAYER]}


def _own_fork(s):
    from paged_kv_gather_gb300 import kvx
    kvx.kvx_free_pages(_ctx(), s["kvx_pool"], s["refs"].data_ptr(), s["tables"],
                       stream=s["stream"])
    kvx.kvx_fork_pages(_ctx(), s["kvx_pool"], s["refs"].data_ptr(), s["forks"],
                       stream=s["stream"])
    return {"refs": s["refs"], "children": s["children"], "pool": s["pool"]}


def _own_compact(s):
    from paged_kv_gather_gb300 import kvx
    kvx.kvx_compact_pages(_ctx(), s["kvx_pool"], s["refs"].data_ptr(), s["table_args"],
                          n_live=s["n_live"].data_ptr(), stream=s["stream"])
    return {"refs": s["refs"], "tables": s["tables"], "n_live": s["n_live"], "pool": s["pool"]}


def run(state):
    op = state["case"]["op"]
    if op == "compact":
        # The pool is fragmented again by putting the bookkeeping back; moved pages still
        # hold their bytes where they were.
        state["refs"].copy_(state["refs0"])
        state["tables"].copy_(state["tables0"])
    if own:
        return {"attend": _own_attend, "append": _own_append, "fork": _own_fork,
                "compact": _own_compact}[op](state)
    return {"attend": _plain_attend, "append": _plain_append, "fork": _plain_fork,
            "compact": _plain_compact}[op](state)


# ------------------------------------------------------------------------------- work

def _seen(pos, n, window, prefix):
    """Keys that the row at position `pos` of a request of n tokens sees."""
    low = max(0, pos - window + 1) if window else 0
    return pos + 1 - low + max(0, min(prefix, n) - pos - 1) + min(prefix, low)


def work(case):
    c = dict(case)
    if c["op"] in ("attend", "append"):
        tokens, new, prefix = _lengths(c)
        row = c["kv_heads"] * c["head_dim"]
        if c["op"] == "append":
            return {"bytes": 2.0 * sum(new) * row * (ITEM[c["kv"]] + ITEM[c["dtype"]]),
                    "flops": 0.0}
        heads = c["kv_heads"] * c["group"]
        keys, pairs = 0, 0
        for n, q, p in zip(tokens, new, prefix):
            first = max(0, n - q - c["window"] + 1) if c["window"] else 0
            keys += n - first + min(p, first)
            pairs += sum(_seen(pos, n, c["window"], p) for pos in range(n - q, n))
        return {"bytes": 2.0 * keys * row * ITEM[c["kv"]]
                + sum(new) * heads * (2.0 * c["head_dim"] * ITEM[c["dtype"]] + 4),
                "flops": 4.0 * c["head_dim"] * heads * pairs}
    token = c["layers"] * c["kv_factor"] * c["token_bytes"]
    P = c["page"]
    if c["op"] == "fork":
        lens = _request_lengths(c)
        moved = sum(n if c["copy"] else n % P for n in lens) * c["children"]
        entries = sum(-(-n // P) for n in lens) * c["children"]
        # Tables read and written, and a count per entry, in the free and in the fork.
        return {"bytes": 2.0 * moved * token + 16.0 * entries, "flops": 0.0}
    # Of the live pages, a share lies past the front that compaction fills: the free share.
    at = 0
    for n in _request_lengths(c):
        at += min(-(-n // P), int(c["pages"] * c["live"]) - at)
    moved = at * (1.0 - at / c["pages"])
    return {"bytes": 2.0 * moved * P * token + 8.0 * c["pages"] + 8.0 * at, "flops": 0.0}


# ------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    """Attention and the cast into the cache from their definitions, in 64 bits."""
    c = dict(case)
    if c["op"] not in ("attend", "append"):
        return None                     # pages and counts: whole numbers only
    global own
    kept, own = own, False
    try:
        s = _prepare_step(c, seed)
    finally:
        own = kept
    P, H, D = c["page"], c["kv_heads"], c["head_dim"]
    pages = s["tables"].cpu().numpy().astype(np.int64)
    row = 0
    if c["op"] == "append":
        layers = [s["pool"][side, LAYER].double() for side in (0, 1)]
        for r, (n, q) in enumerate(zip(s["tokens"], s["new"])):
            for pos in range(n - q, n):
                at = pages[r, pos // P], pos % P
                layers[0][at] = s["k"][row].double() / s["k_scale"]
                layers[1][at] = s["v"][row].double() / s["v_scale"]
                row += 1
        if c["kv"] == "fp8":
            layers = [x.clamp(-448.0, 448.0) for x in layers]
        return {"k": layers[0], "v": layers[1]}
    G = c["group"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    if any(q for q in s["new"]) and work(c)["flops"] > 6e12:
        return None
    for r, (n, q, prefix) in enumerate(zip(s["tokens"], s["new"], s["prefix"])):
        own_pages = torch.from_numpy(pages[r, :-(-n // P)]).to(DEV)
        key = s["pool"][0, LAYER][own_pages].flatten(0, 1)[:n].double() * s["k_scale"]
        val = s["pool"][1, LAYER][own_pages].flatten(0, 1)[:n].double() * s["v_scale"]
        place = torch.arange(n, device=DEV, dtype=torch.float64)
        mine = torch.arange(n - q, n, device=DEV, dtype=torch.float64)
        gap = mine[:, None] - place[None]
        hidden = gap < 0
        if c["window"]:
            hidden |= gap >= c["window"]
        hidden &= ~(place < prefix)[None]
        for h in range(H * G):
            z = s["q"][row:row + q, h].double() @ key[:, h // G].T / math.sqrt(D)
            if c["softcap"]:
                z = c["softcap"] * torch.tanh(z / c["softcap"])
            if s["slopes"] is not None:
                z = z - s["slopes"][h].double() * gap.abs()
            z = z.masked_fill(hidden, -math.inf)
            norm = torch.logsumexp(z, dim=1)
            lse[row:row + q, h] = norm
            out[row:row + q, h] = torch.exp(z - norm[:, None]) @ val[:, h // G]
        row += q
    return {"out": out, "lse": lse}
