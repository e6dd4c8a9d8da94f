"""kvx_append_rotated (and kvx_append_tokens into a 4-bit cache) against the definition in 64 bits.

Tolerance, derived before any run: a rotated element is p cos a - r sin a.  Cosine and sine are
off by at most 2^-22 (the angle's 4e-9 and a few roundings in 32 bits), products and their sum by
2^-23 (|p| + |r|) more: 2^-21 (|p| + |r|) magnitude in all, besides the rounding of the output's
type: bf16 2^-8, fp16 2^-11 (or half of 2^-24 near zero), e4m3 2^-4 (or half of 2^-9 near zero).
What is not rotated is copied, or cast exactly as torch casts it."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_gather_gb300.build import build  # noqa: E402

build()
from paged_kv_gather_gb300 import kvx  # noqa: E402
from tests.cache_common import ITEM, ROUNDOFF, TORCH  # noqa: E402
from tests.four_common import check_stored  # noqa: E402

TINY = {"bf16": 0.0, "fp16": 2.0 ** -25, "fp8": 2.0 ** -10}
STEP = {**ROUNDOFF, "fp8": 2.0 ** -4}


@pytest.fixture(scope="module")
def ctx():
    c = kvx.kvx_create(0)
    yield c
    kvx.kvx_destroy(c)


class Step:
    """Requests with room for their tokens on random pages of a pool filled with 0x5A."""

    def __init__(self, ctx, tokens, new, heads, group, dim, page, kv, dtype, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.tokens, self.new, self.heads, self.dim, self.page = tokens, new, heads, dim, page
        self.kv, self.dtype, self.rows = kv, dtype, sum(new)
        counts = [-(-n // page) for n in tokens]
        self.n_pages = sum(counts) + 3
        self.token_bytes = kvx.kvx_token_bytes(heads, dim, kv)
        self.pool = torch.full((2, 2, self.n_pages, page, self.token_bytes), 0x5A,
                               dtype=torch.uint8, device="cuda")
        perm = torch.randperm(self.n_pages, device="cuda", generator=g).to(torch.int32)
        self.tables = torch.full((len(tokens), max(counts + [1])), -1, dtype=torch.int32,
                                 device="cuda")
        at = 0
        for r, n in enumerate(counts):
            self.tables[r, :n] = perm[at:at + n]
            at += n
        self.kvx_pool = kvx.Pool.from_tensor(self.pool, page)
        cfg = kvx.attn_config(heads * group, heads, dim, dtype, kv)
        self.plan = kvx.kvx_attn_plan_create(
            ctx, self.kvx_pool, kvx.requests_array([(self.tables[r].data_ptr(), None, n)
                                                    for r, n in enumerate(tokens)]), new, cfg)
        self.place = torch.cat([torch.arange(n - m, n) for n, m in zip(tokens, new)])
        self.request = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new))

    def stored(self, layer):
        """Bytes of the step's K and V tokens [2, rows, token_bytes], and whether all others
        still are what they were."""
        page = self.tables.cpu().long()[self.request, self.place // self.page]
        slot = page * self.page + self.place % self.page
        flat = self.pool.view(2, 2, -1, self.token_bytes).cpu()
        got = flat[:, layer][:, slot]
        rest = torch.ones(flat.shape[2], dtype=torch.bool)
        rest[slot] = False
        clean = bool((flat[:, layer][:, rest] == 0x5A).all() and (flat[:, 1 - layer] == 0x5A).all())
        return got.numpy(), clean

    def close(self):
        kvx.kvx_attn_plan_destroy(self.plan)


def rotated(x, angle, rotary, interleaved, magnitude):
    """x [rows, heads, dim] and angles [rows, rotary / 2] in 64 bits; and the error's measure."""
    x, size = x.copy(), np.abs(x)
    a, b = ((slice(0, rotary, 2), slice(1, rotary, 2)) if interleaved else
            (slice(0, rotary // 2), slice(rotary // 2, rotary)))
    z = (x[..., a] + 1j * x[..., b]) * (magnitude * np.exp(1j * angle))[:, None]
    both = (size[..., a] + size[..., b]) * abs(magnitude)
    x[..., a], x[..., b] = z.real, z.imag
    off = np.zeros_like(x)
    off[..., a] = off[..., b] = both * 2.0 ** -21
    return x, off


def run_case(ctx, tokens, new, heads, group, dim, page, kv, dtype, rotary, interleaved=False,
             positions=None, magnitude=1.0, pad=0, in_place=False, with_q=True, seed=0, theta=1e4):
    s = Step(ctx, tokens, new, heads, group, dim, page, kv, dtype, seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    widths = [heads * group * dim, heads * dim, heads * dim]
    x = torch.randn((s.rows, sum(widths) + pad), device="cuda", generator=g).to(TORCH[dtype])
    q, k, v = x[:, :sum(widths)].split(widths, 1)
    keep = x.clone()
    freqs = torch.exp(torch.arange(rotary // 2, device="cuda", dtype=torch.float64)
                      * (-2 / rotary * math.log(theta))).float()
    at = None
    if positions:
        at = torch.randint(*positions, (s.rows,), device="cuda", generator=g, dtype=torch.int32)
    rope = kvx.rope_config(freqs.data_ptr(), rotary, interleaved, at.data_ptr() if positions else 0,
                           magnitude)
    guard = torch.full((s.rows + 1, widths[0] + 8), 7.0, dtype=TORCH[dtype], device="cuda")
    out = q if in_place else guard[:s.rows, :widths[0]]
    k_scale, v_scale = (1.0, 1.0) if kv == dtype else (0.03, 0.05)
    torch.cuda.synchronize()
    kvx.kvx_append_rotated(s.plan, 1, rope, k.data_ptr(), v.data_ptr(),
                           q=q.data_ptr() if with_q else 0,
                           q_out=out.data_ptr() if with_q else 0, k_stride=x.stride(0),
                           v_stride=x.stride(0), q_stride=x.stride(0), q_out_stride=out.stride(0),
                           k_scale=k_scale, v_scale=v_scale)
    torch.cuda.synchronize()
    assert kvx.kvx_get_status(ctx) == 0
    angle = (at.cpu() if positions else s.place).double().numpy()[:, None] \
        * freqs.double().cpu().numpy()[None]
    shape = lambda t: t.double().cpu().unflatten(1, (-1, dim)).numpy()  # noqa: E731
    if with_q:
        ref, off = rotated(shape(keep[:, :widths[0]]), angle, rotary, interleaved, magnitude)
        err = np.abs(shape(out) - ref)
        assert (err <= off + 1.01 * STEP[dtype] * np.abs(ref) + TINY[dtype]).all(), err.max()
        assert torch.equal(out.unflatten(1, (-1, dim))[..., rotary:],
                           keep[:, :widths[0]].unflatten(1, (-1, dim))[..., rotary:])
    if not in_place:
        assert torch.equal(x, keep)
        assert (guard[s.rows] == 7.0).all() and (guard[:, widths[0]:] == 7.0).all()
    got, clean = s.stored(1)
    assert clean
    ref, off = rotated(shape(keep[:, widths[0]:widths[0] + widths[1]]), angle, rotary, interleaved,
                       magnitude)
    value = shape(keep[:, widths[0] + widths[1]:sum(widths)])
    if kv == "fp4":
        check_stored(got[0], ref, heads, dim, k_scale, off.max())
        check_stored(got[1], value, heads, dim, v_scale)
    else:
        kk, vv = (torch.from_numpy(t.copy()).view(TORCH[kv]).double().numpy()
                  .reshape(s.rows, heads, dim) for t in got)
        want = (ref / k_scale).clip(-448, 448) if kv == "fp8" else ref
        tol = off / k_scale + 1.01 * STEP[kv] * np.abs(want) + TINY[kv]
        assert (np.abs(kk - want) <= tol).all()
        v_ref = keep[:, widths[0] + widths[1]:sum(widths)]
        if kv == "fp8":
            v_ref = (v_ref.float() / torch.full_like(v_ref, v_scale, dtype=torch.float32)) \
                .clamp(-448, 448).to(TORCH[kv])
        assert np.array_equal(v_ref.contiguous().view(torch.uint8).cpu().numpy().reshape(s.rows, -1),
                              got[1])
    s.close()


@pytest.mark.parametrize("kv", ["same", "fp8", "fp4"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,rotary", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 32),
                                        (128, 112), (128, 80)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_types(ctx, kv, dtype, dim, rotary, interleaved):
    run_case(ctx, [40, 3, 100], [5, 3, 1], 3, 2, dim, 16, dtype if kv == "same" else kv, dtype,
             rotary, interleaved)


@pytest.mark.parametrize("heads,group", [(1, 1), (2, 7), (5, 3), (8, 8), (16, 4)])
@pytest.mark.parametrize("page", [1, 7, 64])
def test_heads(ctx, heads, group, page):
    run_case(ctx, [1, 33, 300], [1, 0, 130], heads, group, 128, page, "fp4", "bf16", 128, pad=8)
    run_case(ctx, [1, 33, 300], [1, 0, 130], heads, group, 128, page, "bf16", "bf16", 64, pad=8)


@pytest.mark.parametrize("positions", [(0, 10), (900000, 1100000), (2 ** 30, 2 ** 31 - 1),
                                       (-2 ** 31, -1)])
@pytest.mark.parametrize("theta", [1e4, 5e5])
def test_far_positions(ctx, positions, theta):
    run_case(ctx, [64], [64], 2, 2, 128, 16, "bf16", "bf16", 128, positions=positions, theta=theta)


def test_options(ctx):
    run_case(ctx, [64, 20], [64, 7], 2, 2, 128, 16, "fp8", "fp16", 64, magnitude=1.3, pad=16)
    run_case(ctx, [64, 20], [64, 7], 2, 2, 64, 16, "fp4", "bf16", 64, magnitude=-0.7,
             in_place=True)
    run_case(ctx, [64, 20], [64, 7], 2, 2, 128, 16, "bf16", "bf16", 128, with_q=False)
    run_case(ctx, [5000], [4500], 8, 4, 128, 16, "fp4", "bf16", 128)


@pytest.mark.parametrize("dim,heads", [(64, 1), (64, 4), (128, 3)])
def test_append_tokens_to_four_bits(ctx, dim, heads):
    """Blocks of zeros, of one large element, of values past the largest scale, of NaN and of
    infinity."""
    s = Step(ctx, [50, 9], [50, 4], heads, 1, dim, 16, "fp4", "bf16")
    x = torch.randn((2, s.rows, heads, dim), device="cuda").bfloat16()
    x[0, 3, 0, :16] = 0.0
    x[0, 4, 0, :16] = 0.0
    x[0, 4, 0, 5] = 17.0
    x[1, 5] = 3e4
    x[0, 6, 0, 2] = float("nan")
    x[1, 7, 0, 3] = float("inf")
    x[1, 8, 0, :16] = 1e-30
    kvx.kvx_append_tokens(s.plan, 0, x[0].data_ptr(), x[1].data_ptr(), k_scale=0.5, v_scale=0.25)
    torch.cuda.synchronize()
    got, clean = s.stored(0)
    assert clean
    units = got[0, 6, heads * dim // 2:heads * dim * 9 // 16]
    assert units[0] == 0x7F and (units[1:] != 0x7F).all()
    ref = x.double().cpu().numpy()
    ref[0, 6] = 0
    ref[1, 7, 0, 3] = 1e9
    for side, scale in ((0, 0.5), (1, 0.25)):
        fine = np.array([r for r in range(s.rows) if (side, r) != (0, 6)])
        check_stored(got[side][fine], ref[side][fine], heads, dim, scale)
    s.close()


def test_rotating_equals_appending_what_was_rotated(ctx):
    """At position 0 nothing turns: the bytes are those of kvx_append_tokens."""
    for kv in ("bf16", "fp8", "fp4"):
        s = Step(ctx, [300], [300], 4, 2, 128, 16, kv, "bf16", seed=4)
        k, v = torch.randn((2, 300, 4 * 128), device="cuda").bfloat16()
        zero = torch.zeros(300, dtype=torch.int32, device="cuda")
        freqs = torch.ones(64, device="cuda")
        rope = kvx.rope_config(freqs.data_ptr(), 128, positions=zero.data_ptr())
        kvx.kvx_append_rotated(s.plan, 0, rope, k.data_ptr(), v.data_ptr(), k_scale=0.02,
                               v_scale=0.02)
        kvx.kvx_append_tokens(s.plan, 1, k.data_ptr(), v.data_ptr(), k_scale=0.02, v_scale=0.02)
        torch.cuda.synchronize()
        assert torch.equal(s.pool[:, 0], s.pool[:, 1])
        s.close()


def test_bad_page_and_refusals(ctx):
    s = Step(ctx, [40, 40], [1, 1], 2, 2, 128, 16, "bf16", "bf16")
    x = torch.randn((2, 8 * 128), device="cuda").bfloat16()
    q_out = torch.zeros((2, 4 * 128), device="cuda").bfloat16()
    freqs = torch.ones(64, device="cuda")

    def call(rope=None, layer=0, **kw):
        kvx.kvx_append_rotated(s.plan, layer, rope or kvx.rope_config(freqs.data_ptr(), 128),
                               kw.pop("k", x.data_ptr()), kw.pop("v", x.data_ptr()), **kw)

    for status, kw in [
            (kvx.KVX_ERR_INVALID_ARG, {"rope": kvx.rope_config(freqs.data_ptr(), 24)}),
            (kvx.KVX_ERR_INVALID_ARG, {"rope": kvx.rope_config(freqs.data_ptr(), 0)}),
            (kvx.KVX_ERR_INVALID_ARG, {"rope": kvx.rope_config(freqs.data_ptr(), 144)}),
            (kvx.KVX_ERR_INVALID_ARG, {"rope": kvx.rope_config(0, 128)}),
            (kvx.KVX_ERR_ALIGNMENT, {"rope": kvx.rope_config(freqs.data_ptr() + 2, 128)}),
            (kvx.KVX_ERR_INVALID_ARG,
             {"rope": kvx.rope_config(freqs.data_ptr(), 128, magnitude=float("nan"))}),
            (kvx.KVX_ERR_INVALID_ARG, {"layer": 2}), (kvx.KVX_ERR_INVALID_ARG, {"k": 0}),
            (kvx.KVX_ERR_ALIGNMENT, {"v": x.data_ptr() + 2}),
            (kvx.KVX_ERR_INVALID_ARG, {"q": x.data_ptr()}),
            (kvx.KVX_ERR_INVALID_ARG, {"q": x.data_ptr(), "q_out": x.data_ptr(),
                                       "q_stride": 1024, "q_out_stride": 512}),
            (kvx.KVX_ERR_INVALID_ARG, {"k_stride": 8}), (kvx.KVX_ERR_ALIGNMENT, {"k_stride": 260})]:
        with pytest.raises(kvx.KvxError) as e:
            call(**kw)
        assert e.value.status == status, kw
    s.tables[0, 2] = s.n_pages
    call(q=x.data_ptr(), q_out=q_out.data_ptr(), q_stride=8 * 128, k_stride=8 * 128,
         v_stride=8 * 128)
    torch.cuda.synchronize()
    assert kvx.kvx_get_status(ctx) == kvx.KVX_DEV_PAGE_OUT_OF_RANGE
    assert (q_out != 0).any(1).all()
    s.close()
    four = Step(ctx, [40], [1], 2, 2, 128, 16, "fp4", "bf16")
    for scale in (0.0, -1.0, float("inf"), 2.0 ** -101):
        with pytest.raises(kvx.KvxError):
            kvx.kvx_append_tokens(four.plan, 0, x.data_ptr(), x.data_ptr(), k_scale=scale)
    four.close()
