"""kvx_attend and kvx_append_tokens against their definitions in 64 bits.

Tolerance of an output, derived before any run.  With u the relative rounding of the output
type, A = sum_j p_j |v_j| and n keys: the result is rounded once (u |o|); each weight is
rounded to the type for the product with V (u A, and 2^-25 n max|v| where half-precision
weights are subnormal, which bfloat16 ones are not); a score is a sum of D products in 32 bits, off by at most
D 2^-24 sum|q k| scale, which moves every weight by twice that relative to the rest (2 d A);
exponential, tanh and the running sums add a few 2^-22 (2^-18 A covers 9000 terms summed in
blocks).  A cap multiplies the tanh's own few 2^-23 by softcap.  lse is off by d plus the
same 32-bit terms, relative to its size.
"""
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
from tests.cache_common import (ITEM, ROUNDOFF, TORCH, Cache,  # noqa: E402
                                attend_reference, visible)

LAYER = 1


@pytest.fixture(scope="module")
def ctx():
    c = kvx.kvx_create(0)
    yield c
    kvx.kvx_destroy(c)


def make_q(rows, heads, dim, dtype, seed, scale=1.0, pad=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn((rows, heads * dim + pad), device="cuda", generator=g) * scale
    return x.to(TORCH[dtype])


def slopes_of(heads):
    return torch.exp2(-8.0 * torch.arange(1, heads + 1, device="cuda") / heads).float()


def check(cache, q, out, lse, new, group, scale, k_scale=1.0, v_scale=1.0, dtype="bf16", window=0,
          prefix=None, softcap=0.0, slopes=None):
    """Compare every row with the reference under the derived tolerance."""
    u = ROUNDOFF[dtype]
    heads, dim = cache.heads * group, cache.dim
    row = 0
    sl = None if slopes is None else slopes.double().cpu().numpy()
    qd = q.double().cpu().numpy()
    got, got_lse = out.double().cpu().numpy(), None if lse is None else lse.double().cpu().numpy()
    for r, n in enumerate(cache.tokens):
        m = new[r]
        k, v = cache.values[r][0, LAYER] * k_scale, cache.values[r][1, LAYER] * v_scale
        if m == 0:
            continue
        ref, ref_lse, spread, reach = attend_reference(
            qd[row:row + m], k, v, m, group, scale, window, prefix[r] if prefix else 0, softcap, sl)
        d = dim * 2.0 ** -24 * reach + softcap * 2.0 ** -21
        tol = (1.01 * u * (np.abs(ref) + spread) + (2 * d[..., None] + 2.0 ** -18) * spread)
        if dtype == "fp16":
            tol += 2.0 ** -25 * (1 + n * np.abs(v).max())
        err = np.abs(got[row:row + m] - ref)
        assert np.isfinite(got[row:row + m]).all(), f"request {r}: not finite"
        worst = np.unravel_index(np.argmax(err / tol), err.shape)
        assert (err <= tol).all(), (f"request {r}: row, head, dim {worst}: off by {err[worst]:.3g}, "
                                    f"bound {tol[worst]:.3g}, ref {ref[worst]:.3g}")
        if got_lse is not None:
            lt = d + 2.0 ** -20 * (1 + np.abs(ref_lse)) + 2.0 ** -20 * reach
            assert (np.abs(got_lse[row:row + m] - ref_lse) <= lt).all()
        row += m
    assert row == got.shape[0]


def run_case(ctx, tokens, new, heads, group, dim, page, kv="bf16", dtype="bf16", window=0,
             prefix=None, softcap=0.0, slopes=False, k_scale=1.0, v_scale=1.0, pad=0, out_pad=0,
             want_lse=True, seed=0, q_scale=1.0, scale=0.0, spoil=True):
    cache = Cache(tokens, heads, dim, page, kv, seed=seed, scale=8.0 if kv == "fp8" else 1.0)
    if spoil:  # pages that no row sees may be named by anything
        for r, n in enumerate(tokens):
            seen = visible(n, new[r], window, prefix[r] if prefix else 0).any(0)
            for j in range(-(-n // page)):
                if not seen[j * page:(j + 1) * page].any():
                    cache.tables[r, j] = (-1, 2 ** 31 - 1, cache.n_pages)[j % 3]
    rows, hq = sum(new), heads * group
    x = make_q(rows, hq, dim, dtype, seed + 1, q_scale, pad)
    q = x[:, :hq * dim].unflatten(1, (hq, dim))
    guard = torch.full((rows + 1, hq * dim + out_pad), 7.0, dtype=TORCH[dtype], device="cuda")
    out = guard[:rows, :hq * dim].unflatten(1, (hq, dim))
    lse = torch.full((rows + 1, hq), 7.0, device="cuda") if want_lse else None
    sl = slopes_of(hq) if slopes else None
    cfg = kvx.attn_config(hq, heads, dim, dtype, kv, window, scale, softcap,
                          sl.data_ptr() if slopes else 0)
    plan = kvx.kvx_attn_plan_create(ctx, cache.kvx_pool, cache.requests(), new, cfg, prefix)
    try:
        torch.cuda.synchronize()
        for _ in range(2):  # the second launch finds the workspace as the first left it
            kvx.kvx_attend(plan, LAYER, q.data_ptr(), out.data_ptr(), x.stride(0) if pad else 0,
                           guard.stride(0) if out_pad else 0, lse.data_ptr() if want_lse else 0,
                           k_scale, v_scale)
            first = out.clone()
        torch.cuda.synchronize()
        assert kvx.kvx_get_status(ctx) == 0
        assert torch.equal(first, out)
    finally:
        kvx.kvx_attn_plan_destroy(plan)
    assert (guard[rows] == 7.0).all() and (guard[:, hq * dim:] == 7.0).all()
    if want_lse:
        assert (lse[rows] == 7.0).all()
    check(cache, q, out, lse[:rows] if want_lse else None, new, group, scale or dim ** -0.5,
          k_scale, v_scale, dtype, window, prefix, softcap, sl)


TYPES = [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp8"), ("fp16", "fp8")]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype,kv", TYPES)
@pytest.mark.parametrize("page", [1, 5, 16, 24, 64, 200])
def test_single_tokens(ctx, dtype, kv, dim, page):
    """Decoding: one new token a request, from the first token of a request to long ones."""
    tokens = [1, 2, page, page + 1, 63, 64, 65, 127, 129, 700, 2049]
    run_case(ctx, tokens, [1] * len(tokens), 2, 4, dim, page, kv, dtype, k_scale=0.05
             if kv == "fp8" else 1.0, v_scale=0.1 if kv == "fp8" else 1.0)


@pytest.mark.parametrize("group", [1, 2, 3, 7, 8, 16, 20])
@pytest.mark.parametrize("new", [1, 2, 5, 16])
def test_few_rows_and_groups(ctx, group, new):
    """Rows per KV head from one to hundreds: every boundary of the tiles of rows."""
    run_case(ctx, [new, 40 + new, 333, 1500], [new, new, new, 1], 3, group, 128, 16)


@pytest.mark.parametrize("dtype,kv", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [1, 7, 16, 48, 128])
def test_chunks(ctx, dtype, kv, dim, page):
    """Prefill chunks: whole prompts, chunks behind a context, ragged with single tokens and
    requests that add nothing."""
    tokens = [300, 129, 1000, 128, 0, 77, 400, 31]
    new = [300, 129, 130, 1, 0, 0, 257, 31]
    run_case(ctx, tokens, new, 2, 4, dim, page, kv, dtype, k_scale=0.05 if kv == "fp8" else 1.0,
             v_scale=0.1 if kv == "fp8" else 1.0)


@pytest.mark.parametrize("new", [1, 3, 40, 300])
@pytest.mark.parametrize("window", [1, 17, 128, 1000])
@pytest.mark.parametrize("prefix", [None, 1, 130])
def test_window_and_prefix(ctx, new, window, prefix):
    """A sliding window, with and without a prefix that stays visible; pages outside both hold
    NaN and are named by invalid ids."""
    tokens = [new, 500 + new, 2000, 1290]
    pre = None if prefix is None else [min(prefix, n) for n in tokens]
    run_case(ctx, tokens, [new] * 4, 2, 4, 64, 16, window=window, prefix=pre)


@pytest.mark.parametrize("new,group", [(1, 4), (6, 5), (200, 2)])
@pytest.mark.parametrize("prefix", [0, 100, 10 ** 6])
def test_prefix_both_ways(ctx, new, group, prefix):
    """Inside the prefix rows see later tokens too, up to the whole request."""
    tokens = [new, 260, 901]
    run_case(ctx, tokens, [new] * 3, 2, group, 128, 16, prefix=[min(prefix, n) for n in tokens])


@pytest.mark.parametrize("dtype,kv", TYPES)
@pytest.mark.parametrize("softcap,slopes,window", [(20.0, False, 0), (0.0, True, 0),
                                                   (50.0, True, 300)])
def test_score_options(ctx, dtype, kv, softcap, slopes, window):
    ks = 0.05 if kv == "fp8" else 1.0
    for new in (1, 9, 150):
        run_case(ctx, [new, 200, 1100], [new] * 3, 2, 6, 128, 16, kv, dtype, window=window,
                 softcap=softcap, slopes=slopes, k_scale=ks, v_scale=2 * ks, q_scale=3.0)


@pytest.mark.parametrize("new", [1, 4, 200])
def test_large_scores(ctx, new):
    """Scores in the hundreds: one key takes the whole weight, the running maximum jumps."""
    run_case(ctx, [new, 500, 1500], [new] * 3, 2, 4, 128, 16, q_scale=40.0)


@pytest.mark.parametrize("new", [1, 150])
def test_strides_and_no_lse(ctx, new):
    run_case(ctx, [200, 777], [new, new], 2, 4, 128, 16, pad=2 * 2 * 128, out_pad=24,
             want_lse=False)


@pytest.mark.parametrize("new", [1, 12, 100])
def test_given_scale_and_negative(ctx, new):
    run_case(ctx, [300, 129], [new, new], 1, 8, 64, 16, scale=-0.3)


@pytest.mark.parametrize("new,kv", [(1, "bf16"), (64, "bf16"), (1, "fp8"), (64, "fp8")])
def test_long_context(ctx, new, kv):
    """Long enough that one KV head's keys are split over many SMs, few enough requests that
    every split is needed."""
    run_case(ctx, [20011, 300], [new, 1], 1, 4, 128, 16, kv, k_scale=0.05 if kv == "fp8" else 1.0)


@pytest.mark.parametrize("new", [1, 70])
def test_many_requests(ctx, new):
    """More (request, head) pairs than SMs, so that a CTA works through several."""
    rng = np.random.default_rng(5)
    tokens = [int(x) for x in rng.integers(new, 400, 150)]
    run_case(ctx, tokens, [new] * 150, 2, 2, 64, 16)


@pytest.mark.parametrize("new", [1, 40])
def test_offsets_past_32_bits(ctx, new):
    """Pages whose byte offset in a layer is past 4 GiB."""
    pages = (1 << 32) // (16 * 2048) + 200
    cache = Cache([333, 90], 8, 128, 16, layers=2, pages=pages, first_page=pages - 60)
    q = make_q(2 * new, 16, 128, "bf16", 3).unflatten(1, (16, 128))
    out = torch.empty_like(q)
    plan = kvx.kvx_attn_plan_create(ctx, cache.kvx_pool, cache.requests(), [new, new],
                                    kvx.attn_config(16, 8, 128))
    kvx.kvx_attend(plan, LAYER, q.data_ptr(), out.data_ptr())
    torch.cuda.synchronize()
    assert kvx.kvx_get_status(ctx) == 0
    kvx.kvx_attn_plan_destroy(plan)
    check(cache, q, out, None, [new, new], 2, 128 ** -0.5)


def test_update_other_stream_and_graph(ctx):
    """A plan refilled step after step on a stream of its own, and replayed from a graph."""
    cache = Cache([900, 450], 2, 128, 16)
    stream = torch.cuda.Stream()
    s = stream.cuda_stream
    cfg = kvx.attn_config(8, 2, 128)
    # The requests of a step are the first n tokens of the cache's.
    def reqs(tokens):
        return kvx.requests_array([(cache.tables[r].data_ptr(), None, n)
                                   for r, n in enumerate(tokens)])
    plan = kvx.kvx_attn_plan_create(ctx, cache.kvx_pool, reqs([5, 7]), [5, 7], cfg, stream=s)
    full = cache.tokens, cache.values
    for tokens, new in (([5, 7], [5, 7]), ([6, 8], [1, 1]), ([700, 8], [694, 0]), ([900], [130]),
                        ([701, 450], [1, 442])):
        q = make_q(sum(new), 8, 128, "bf16", 9).unflatten(1, (8, 128))
        out = torch.empty_like(q)
        torch.cuda.synchronize()
        kvx.kvx_attn_plan_update(plan, reqs(tokens), new, stream=s)
        kvx.kvx_attend(plan, LAYER, q.data_ptr(), out.data_ptr(), stream=s)
        torch.cuda.synchronize()
        cache.tokens = tokens
        cache.values = [v[:, :, :n] for v, n in zip(full[1], tokens)]
        check(cache, q, out, None, new, 4, 128 ** -0.5)
    out.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        kvx.kvx_attend(plan, LAYER, q.data_ptr(), out.data_ptr(), stream=s)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    check(cache, q, out, None, new, 4, 128 ** -0.5)
    assert kvx.kvx_get_status(ctx) == 0
    kvx.kvx_attn_plan_destroy(plan)


@pytest.mark.parametrize("new", [1, 33])
@pytest.mark.parametrize("bad", [-1, 10 ** 9])
def test_page_out_of_range_is_reported(ctx, new, bad):
    """A visible page id outside the pool sets the status bit; other requests are right."""
    cache = Cache([200, 300], 2, 64, 16)
    cache.tables[0, 3] = bad
    q = make_q(2 * new, 4, 64, "bf16", 1).unflatten(1, (4, 64))
    out = torch.zeros_like(q)
    plan = kvx.kvx_attn_plan_create(ctx, cache.kvx_pool, cache.requests(), [new, new],
                                    kvx.attn_config(4, 2, 64))
    kvx.kvx_attend(plan, LAYER, q.data_ptr(), out.data_ptr())
    torch.cuda.synchronize()
    assert kvx.kvx_get_status(ctx) == kvx.KVX_DEV_PAGE_OUT_OF_RANGE
    kvx.kvx_attn_plan_destroy(plan)
    cache.tokens, cache.values = cache.tokens[1:], cache.values[1:]
    check(cache, q[new:], out[new:], None, [new], 2, 64 ** -0.5)


def test_empty_step(ctx):
    cache = Cache([10, 20], 2, 64, 16)
    plan = kvx.kvx_attn_plan_create(ctx, cache.kvx_pool, cache.requests(), [0, 0],
                                    kvx.attn_config(4, 2, 64))
    kvx.kvx_attend(plan, 0, 0, 0)
    kvx.kvx_append_tokens(plan, 0, 0, 0)
    kvx.kvx_attn_plan_update(plan, None, [])
    kvx.kvx_attend(plan, 0, 0, 0)
    kvx.kvx_attn_plan_destroy(plan)
    assert kvx.kvx_get_status(ctx) == 0


def test_refusals_of_launches(ctx):
    cache = Cache([10, 20], 2, 64, 16, kv="fp8")
    plan = kvx.kvx_attn_plan_create(ctx, cache.kvx_pool, cache.requests(), [1, 2],
                                    kvx.attn_config(4, 2, 64, "bf16", "fp8"))
    x = torch.zeros(4096, dtype=torch.bfloat16, device="cuda")
    p = x.data_ptr()

    def refused(status, fn, *args, **kw):
        with pytest.raises(kvx.KvxError) as e:
            fn(plan, *args, **kw)
        assert e.value.status == status and e.value.message

    inv, al = kvx.KVX_ERR_INVALID_ARG, kvx.KVX_ERR_ALIGNMENT
    for fn in (kvx.kvx_attend, kvx.kvx_append_tokens):
        refused(inv, fn, 2, p, p)
        refused(inv, fn, -1, p, p)
        refused(inv, fn, 0, 0, p)
        refused(inv, fn, 0, p, 0)
        refused(al, fn, 0, p + 2, p)
        refused(al, fn, 0, p, p + 8)
    refused(inv, kvx.kvx_attend, 0, p, p, q_stride=128)
    refused(al, kvx.kvx_attend, 0, p, p, out_stride=260)
    refused(al, kvx.kvx_attend, 0, p, p, lse=p + 2)
    refused(inv, kvx.kvx_attend, 0, p, p, k_scale=math.inf)
    refused(inv, kvx.kvx_append_tokens, 0, p, p, k_stride=64)
    refused(inv, kvx.kvx_append_tokens, 0, p, p, v_scale=0.0)
    refused(inv, kvx.kvx_append_tokens, 0, p, p, k_scale=math.nan)
    with pytest.raises(kvx.KvxError) as e:
        kvx.kvx_attn_plan_update(plan, kvx.requests_array(
            [(cache.tables[0].data_ptr(), None, 5)] * 3), [1, 1, 1])
    assert e.value.status == kvx.KVX_ERR_CAPACITY
    kvx.kvx_attn_plan_destroy(plan)
    torch.cuda.synchronize()
    assert kvx.kvx_get_status(ctx) == 0


# ------------------------------------------------------------------------------- append

@pytest.mark.parametrize("dtype,kv", TYPES)
@pytest.mark.parametrize("page,dim,heads", [(1, 64, 1), (5, 128, 8), (16, 64, 3), (64, 128, 2)])
@pytest.mark.parametrize("pad", [0, 40])
def test_append(ctx, dtype, kv, page, dim, heads, pad):
    """Exactly the new tokens' slots of exactly one layer change, to the nearest code."""
    tokens, new = [1, 7, 100, 0, 64, 333], [1, 0, 33, 0, 64, 1]
    cache = Cache(tokens, heads, dim, page, kv, seed=4, scale=20.0 if kv == "fp8" else 1.0)
    before = cache.pool.view(torch.uint8).cpu().numpy().copy()
    rows = sum(new)
    k = make_q(rows, heads, dim, dtype, 5, 30.0, pad)
    v = make_q(rows, heads, dim, dtype, 6, 0.01, 2 * pad)
    k[0, :8] = torch.tensor([0.0, -0.0, 1e4, -1e4, math.inf, -math.inf, 2.0 ** -10, math.nan])
    ks, vs = (0.11, 0.003) if kv == "fp8" else (1.0, 1.0)
    plan = kvx.kvx_attn_plan_create(ctx, cache.kvx_pool, cache.requests(), new,
                                    kvx.attn_config(heads, heads, dim, dtype, kv))
    kvx.kvx_append_tokens(plan, LAYER, k.data_ptr(), v.data_ptr(), k.stride(0), v.stride(0), ks, vs)
    torch.cuda.synchronize()
    assert kvx.kvx_get_status(ctx) == 0
    kvx.kvx_attn_plan_destroy(plan)
    want = before.reshape(2, 2, -1, heads * dim * ITEM[kv])
    tables, row = cache.tables.cpu().numpy(), 0
    for r, n in enumerate(tokens):
        for p in range(n - new[r], n):
            slot = int(tables[r, p // page]) * page + p % page
            for side, x, s in ((0, k, ks), (1, v, vs)):
                y = x[row, :heads * dim].cpu()
                if kv == "fp8":
                    y = (y.float() / torch.tensor(s, dtype=torch.float32)).clamp(-448.0, 448.0)
                    y = y.to(TORCH[kv])
                want[side, LAYER, slot] = y.view(torch.uint8).numpy()
            row += 1
    got = cache.pool.view(torch.uint8).cpu().numpy().reshape(want.shape)
    if kv == "fp8":  # one code of NaN or the other
        got, want = got.copy(), want.copy()
        got[got == 0xFF], want[want == 0xFF] = 0x7F, 0x7F
    assert np.array_equal(got, want)


@pytest.mark.parametrize("bad", [-1, 10 ** 9])
def test_append_reports_pages_out_of_range(ctx, bad):
    cache = Cache([20, 40], 2, 64, 16)
    before = cache.pool.view(torch.uint8).clone()
    kept = cache.tables[1].clone()
    cache.tables[1, 2] = bad
    k = make_q(2, 2, 64, "bf16", 1)
    plan = kvx.kvx_attn_plan_create(ctx, cache.kvx_pool, cache.requests(), [1, 1],
                                    kvx.attn_config(2, 2, 64))
    kvx.kvx_append_tokens(plan, 0, k.data_ptr(), k.data_ptr())
    torch.cuda.synchronize()
    assert kvx.kvx_get_status(ctx) == kvx.KVX_DEV_PAGE_OUT_OF_RANGE
    kvx.kvx_attn_plan_destroy(plan)
    flat, was = (x.view(2, 2, -1, 256) for x in (cache.pool.view(torch.uint8), before))
    slot = int(cache.tables[0, 1]) * 16 + 3
    assert torch.equal(flat[0, 0, slot], k[0].view(torch.uint8))
    flat[:, 0, slot] = was[:, 0, slot]
    assert torch.equal(flat, was) and int(kept[2]) >= 0


def _steps(ctx, synchronize, steps=40):
    """Grow, append, attend, shrink the life of two requests again and again; every output."""
    page, heads, dim, group = 16, 2, 64, 8
    pages = torch.zeros((2, 1, 64, page, heads * dim * 2), dtype=torch.uint8, device="cuda")
    pool = kvx.Pool.from_tensor(pages, page)
    refs = torch.zeros(64, dtype=torch.int32, device="cuda")
    tables = torch.full((2, 64), -1, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn((steps, 2 * 24, (group + 2) * heads * dim), device="cuda",
                    generator=g).bfloat16()
    cfg = kvx.attn_config(heads * group, heads, dim)
    outs, now = [], [0, 0]
    plan = None

    def settle():
        if synchronize:
            torch.cuda.synchronize()

    for i in range(steps):
        new = [(1, 1), (20, 1), (3, 17)][i % 3]
        then = [n + m for n, m in zip(now, new)]
        rows = tables.data_ptr(), tables[1].data_ptr()
        kvx.kvx_fork_pages(ctx, pool, refs.data_ptr(), kvx.forks_array(
            [(p, p, n, t, False) for p, n, t in zip(rows, now, then)]))
        settle()
        reqs = kvx.requests_array([(p, None, t) for p, t in zip(rows, then)])
        if plan is None:
            plan = kvx.kvx_attn_plan_create(ctx, pool, reqs, new, cfg)
        else:
            kvx.kvx_attn_plan_update(plan, reqs, new)
        settle()
        # A copy first, then kernels that start while the one before them ends: what append
        # and attend read is written just ahead of them, on the same few pages every time.
        y = (x[i, :sum(new)] * 1.0).contiguous()
        width = heads * dim * 2
        at = y.data_ptr()
        stride = y.stride(0)
        out = torch.empty((sum(new), heads * group, dim), dtype=torch.bfloat16, device="cuda")
        settle()
        kvx.kvx_append_tokens(plan, 0, at + group * width, at + (group + 1) * width, stride, stride)
        settle()
        kvx.kvx_attend(plan, 0, at, out.data_ptr(), stride)
        settle()
        outs.append(out)
        now = then
        if i % 8 == 7:  # both end and begin anew on the pages they free
            kvx.kvx_free_pages(ctx, pool, refs.data_ptr(), kvx.tables_array(
                [(p, -(-n // page)) for p, n in zip(rows, now)]))
            now = [0, 0]
            settle()
    torch.cuda.synchronize()
    kvx.kvx_attn_plan_destroy(plan)
    assert kvx.kvx_get_status(ctx) == 0
    return outs


def test_back_to_back_calls_see_each_others_work(ctx):
    """The calls of a step, which may start while the one before them drains, give the same
    outputs as with the GPU idle between them."""
    want = _steps(ctx, True)
    for _ in range(3):
        for a, b in zip(_steps(ctx, False), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("tokens,new,heads,group", [
    ([700, 1, 450, 333, 90], [700, 1, 450, 333, 90], 8, 4),        # prompts
    ([900, 40, 260, 2000, 5], [300, 40, 130, 500, 5], 8, 5),       # chunks
    ([1 + 37 * r % 400 for r in range(38)], [1] * 38, 64, 17),     # many units, short
    ([1 + 37 * r % 400 for r in range(39)], [1] * 39, 64, 17)])    # and some more
def test_more_units_than_sms(ctx, tokens, new, heads, group):
    """Several units of unequal length for every SM, whole or cut."""
    run_case(ctx, tokens, new, heads, group, 64, 16)


def test_update_between_schedules(ctx):
    """A plan refilled with batches of few long and many short units gives what it gave."""
    tokens = [3000, 520, 300, 700, 64, 900]
    cache = Cache(tokens, 8, 128, 16)
    cfg = kvx.attn_config(32, 8, 128)
    news = [[3000, 520, 300, 700, 64, 900], [1, 0, 64, 0, 0, 1], [64, 0, 0, 0, 0, 0], [1] * 6]
    q = make_q(sum(tokens), 32, 128, "bf16", 5)
    plan = kvx.kvx_attn_plan_create(ctx, cache.kvx_pool, cache.requests(), news[0], cfg)
    outs = []
    for i in (0, 1, 2, 0, 3, 1, 0, 2, 3):
        if outs:
            kvx.kvx_attn_plan_update(plan, cache.requests(), news[i])
        out = torch.zeros((sum(news[i]), 32, 128), dtype=torch.bfloat16, device="cuda")
        kvx.kvx_attend(plan, LAYER, q.data_ptr(), out.data_ptr())
        outs.append((i, out))
    torch.cuda.synchronize()
    kvx.kvx_attn_plan_destroy(plan)
    assert kvx.kvx_get_status(ctx) == 0
    first = {}
    for i, out in outs:
        assert torch.equal(first.setdefault(i, out), out)
    for i, out in first.items():
        if i:
            check(cache, q[:sum(news[i])].unflatten(1, (32, 128)), out, None, news[i], 4, 128 ** -0.5)
