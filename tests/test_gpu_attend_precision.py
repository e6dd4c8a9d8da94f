"""kvx_attend where most is asked of 32 bits: caps far from the scores, many keys
of small weight beside a large one, rows of q that span many powers of two.  References are in
64 bits."""
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
from tests.cache_common import ROUNDOFF, TORCH, Cache, attend_reference  # noqa: E402

LAYER = 1


@pytest.fixture(scope="module")
def ctx():
    c = kvx.kvx_create(0)
    yield c
    kvx.kvx_destroy(c)


def attend(ctx, cache, reqs, new, q, cfg, k_scale=1.0, v_scale=1.0):
    """out and lse of one launch, as float64 arrays."""
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:2], device="cuda")
    plan = kvx.kvx_attn_plan_create(ctx, cache.kvx_pool, reqs, new, cfg)
    torch.cuda.synchronize()
    kvx.kvx_attend(plan, LAYER, q.data_ptr(), out.data_ptr(), lse=lse.data_ptr(),
                   k_scale=k_scale, v_scale=v_scale)
    torch.cuda.synchronize()
    assert kvx.kvx_get_status(ctx) == 0
    kvx.kvx_attn_plan_destroy(plan)
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


@pytest.mark.parametrize("dtype,kv", [("bf16", "bf16"), ("fp16", "fp8")])
@pytest.mark.parametrize("new", [1, 3, 150])
@pytest.mark.parametrize("softcap", [1e-3, 1.0, 200.0, 1e4, 1e6, 1e9])
def test_caps_of_every_size(ctx, softcap, new, dtype, kv):
    """A cap far above the scores leaves them as they are; one far below makes them signs.

    Tolerance: tanh is good to 2^-19 of itself (a polynomial below 1/2, 6e-7, and some eight
    roundings; the definition above, 2^-21 of 1), so a capped score is off by 2^-19 |s| beside the products'
    D 2^-24 sum|q k|.  That moves lse by as much, and weights by twice that relative to each
    other; the rest is the output's and the weights' rounding to the type, and 2^-18 for
    exponentials and sums."""
    ks = 0.05 if kv == "fp8" else 1.0
    tokens, heads, group, dim = [new, 700], 2, 4, 128
    cache = Cache(tokens, heads, dim, 16, kv, scale=8.0 if kv == "fp8" else 1.0, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    q = (3.0 * torch.randn((2 * new, heads * group, dim), device="cuda", generator=g)).to(
        TORCH[dtype])
    cfg = kvx.attn_config(heads * group, heads, dim, dtype, kv, softcap=softcap)
    got, got_lse = attend(ctx, cache, cache.requests(), [new, new], q, cfg, ks, ks)
    qd, u = q.double().cpu().numpy(), ROUNDOFF[dtype]
    for r in range(2):
        k, v = cache.values[r][0, LAYER] * ks, cache.values[r][1, LAYER] * ks
        rows = slice(r * new, (r + 1) * new)
        ref, ref_lse, spread, reach = attend_reference(qd[rows], k, v, new, group, dim ** -0.5,
                                                       softcap=softcap)
        d = dim * 2.0 ** -24 * reach + 2.0 ** -19 * np.minimum(softcap, reach)
        tol = 1.01 * u * (np.abs(ref) + spread) + (2 * d[..., None] + 2.0 ** -18) * spread
        if dtype == "fp16":
            tol += 2.0 ** -25 * (1 + tokens[r] * np.abs(v).max())
        assert (np.abs(got[rows] - ref) <= tol).all(), np.max(np.abs(got[rows] - ref) / tol)
        lt = d + 2.0 ** -20 * (1 + np.abs(ref_lse)) + 2.0 ** -20 * reach
        assert (np.abs(got_lse[rows] - ref_lse) <= lt).all(), np.max(
            np.abs(got_lse[rows] - ref_lse) / lt)


@pytest.mark.parametrize("dtype,kv", [("bf16", "fp8"), ("fp16", "fp8"), ("fp16", "fp16")])
@pytest.mark.parametrize("new,requests,tokens", [(1, 160, 20000), (4, 160, 20000), (40, 160, 3000)])
def test_many_small_weights_beside_a_large_one(ctx, new, requests, tokens, dtype, kv):
    """One key 17.5 above all the others, whose values alone make up the result.

    Half-precision weights are made 2^7 times their size, in steps of 2^-24 at the least: each
    is off by at most 2^-32 of the largest, or by its own 2^-11.  With n such keys of values
    up to V beside a sum of weights of at least 1, that is n 2^-32 V."""
    heads, group, dim, gap = 2, 2, 64, 17.5
    group = group if new < 40 else 4
    cache = Cache([tokens], heads, dim, 16, kv, seed=1)
    main = tokens - new      # seen by every row, in the first step of the walk
    slots = (cache.tables[0].long()[torch.arange(tokens, device="cuda") // 16] * 16
             + torch.arange(tokens, device="cuda") % 16)
    top = 440.0 if kv == "fp8" else 1000.0
    x = torch.zeros((2, tokens, heads, dim), device="cuda")
    x[0, main] = 1.0
    x[1] = top
    x[1, main] = 0.0
    x = x.to(TORCH[kv])
    flat = cache.pool.view(torch.uint8).view(2, 2, cache.n_pages * 16, -1)
    flat[:, LAYER, slots] = x.view(torch.uint8).view(2, tokens, -1)
    value = float(x[1, main - 1, 0, 0])
    q = torch.ones((requests * new, heads * group, dim), dtype=TORCH[dtype], device="cuda")
    cfg = kvx.attn_config(heads * group, heads, dim, dtype, kv, scale=gap / dim)
    reqs = kvx.requests_array([(cache.tables[0].data_ptr(), None, tokens)] * requests)
    got, got_lse = attend(ctx, cache, reqs, [new] * requests, q, cfg)
    n = np.tile(np.arange(tokens - new, tokens), requests)[:, None]  # keys beside the large one
    tail = n * math.exp(-gap)
    ref, ref_lse = (tail * value / (1 + tail))[..., None], gap + np.log1p(tail)
    d = dim * 2.0 ** -24 * gap
    tol = (2.02 * ROUNDOFF[dtype] + 2 * d + 2.0 ** -18) * ref + n[..., None] * 2.0 ** -32 * value
    err = np.abs(got - ref)
    assert (err <= tol).all(), (np.max(err / tol), np.max(err / ref))
    assert (np.abs(got_lse - ref_lse) <= d + 2.0 ** -18 * gap).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("new", [1, 4, 60])
def test_rows_of_q_that_span_many_powers_of_two(ctx, new, dtype):
    """An e4m3 cache is multiplied in half precision: q, scaled to at most 1, keeps its elements
    to 2^-25 of the row's largest.  Large elements meet zeros in K here, so that the small ones
    make the scores; tolerance: that 2^-25 for every element, and the products' 32 bits."""
    tokens, heads, group, dim, ks = [new, 900], 2, 3, 128, 2.0 ** 4
    cache = Cache(tokens, heads, dim, 16, "fp8", scale=8.0, seed=8)
    small = np.arange(dim) % 4 != 0
    for r, t in enumerate(tokens):
        cache.values[r][0, LAYER][:, :, ~small] = 0.0
        at = (cache.tables[r].long()[torch.arange(t, device="cuda") // 16] * 16
              + torch.arange(t, device="cuda") % 16)
        x = torch.tensor(cache.values[r][0, LAYER], device="cuda").float().to(TORCH["fp8"])
        flat = cache.pool.view(torch.uint8).view(2, 2, cache.n_pages * 16, -1)
        flat[0, LAYER, at] = x.view(torch.uint8).view(t, -1)
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    q = torch.randn((2 * new, heads * group, dim), device="cuda", generator=g)
    power = torch.randint(-22, -12, q.shape, device="cuda", generator=g).float()
    q = q * torch.where(torch.tensor(small, device="cuda"), torch.exp2(power),
                        torch.ones((), device="cuda"))
    q = q.to(TORCH[dtype])
    scale = 2.0 ** 6
    cfg = kvx.attn_config(heads * group, heads, dim, dtype, "fp8", scale=scale)
    got, got_lse = attend(ctx, cache, cache.requests(), [new, new], q, cfg, ks, 1.0)
    qd, u = q.double().cpu().numpy(), ROUNDOFF[dtype]
    for r in range(2):
        k, v = cache.values[r][0, LAYER] * ks, cache.values[r][1, LAYER]
        rows = slice(r * new, (r + 1) * new)
        ref, ref_lse, spread, reach = attend_reference(qd[rows], k, v, new, group, scale)
        most = np.abs(qd[rows]).max(-1)                                  # of a row of q
        size = np.abs(k).sum(-1).max(0)                                  # sum |k| per KV head
        d = (dim * 2.0 ** -24 * reach
             + 2.0 * 2.0 ** -25 * most * np.repeat(size, group)[None] * scale)
        tol = 1.01 * u * (np.abs(ref) + spread) + (2 * d[..., None] + 2.0 ** -18) * spread
        if dtype == "fp16":
            tol += 2.0 ** -25 * (1 + tokens[r] * np.abs(v).max())
        assert (np.abs(got[rows] - ref) <= tol).all(), np.max(np.abs(got[rows] - ref) / tol)
        assert (np.abs(got_lse[rows] - ref_lse) <= d + 2.0 ** -20 * (1 + np.abs(ref_lse))).all()
