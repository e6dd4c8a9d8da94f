"""kvx_attend over a 4-bit cache against its definition in 64 bits.

Codes x scales are exact in half precision, in which they are multiplied, so the tolerance is
that of the other caches (tests/test_gpu_attend.py): an output's rounding, the weights' rounding
to half precision (which the bound of bfloat16 outputs covers), and scores of D products in 32
bits."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_gather_gb300.build import build  # noqa: E402

build()
from paged_kv_gather_gb300 import kvx  # noqa: E402
from tests.cache_common import TORCH, visible  # noqa: E402
from tests.four_common import FourCache  # noqa: E402
from tests.test_gpu_attend import LAYER, check, make_q, slopes_of  # noqa: E402


@pytest.fixture(scope="module")
def ctx():
    c = kvx.kvx_create(0)
    yield c
    kvx.kvx_destroy(c)


def run_case(ctx, tokens, new, heads, group, dim, page, dtype="bf16", window=0, prefix=None,
             softcap=0.0, slopes=False, k_scale=0.01, v_scale=0.012, pad=0, seed=0, q_scale=1.0,
             stream=None, spread=False):
    cache = FourCache(tokens, heads, dim, page, seed=seed, spread=spread)
    for r, n in enumerate(tokens):  # pages that no row sees may be named by anything
        seen = visible(n, new[r], window, prefix[r] if prefix else 0).any(0)
        for j in range(-(-n // page)):
            if not seen[j * page:(j + 1) * page].any():
                cache.tables[r, j] = (-1, 2 ** 31 - 1, cache.n_pages)[j % 3]
    rows, hq = sum(new), heads * group
    x = make_q(rows, hq, dim, dtype, seed + 1, q_scale, pad)
    q = x[:, :hq * dim].unflatten(1, (hq, dim))
    guard = torch.full((rows + 1, hq * dim + pad), 7.0, dtype=TORCH[dtype], device="cuda")
    out = guard[:rows, :hq * dim].unflatten(1, (hq, dim))
    lse = torch.full((rows + 1, hq), 7.0, device="cuda")
    sl = slopes_of(hq) if slopes else None
    cfg = kvx.attn_config(hq, heads, dim, dtype, "fp4", window, 0.0, softcap,
                          sl.data_ptr() if slopes else 0)
    torch.cuda.synchronize()
    s = stream.cuda_stream if stream else 0
    plan = kvx.kvx_attn_plan_create(ctx, cache.kvx_pool, cache.requests(), new, cfg, prefix,
                                    stream=s)
    try:
        for _ in range(2):  # the second launch finds the workspace as the first left it
            kvx.kvx_attend(plan, LAYER, q.data_ptr(), out.data_ptr(), x.stride(0),
                           guard.stride(0), lse.data_ptr(), k_scale, v_scale, stream=s)
            torch.cuda.synchronize()
            first = out.clone()
        kvx.kvx_attend(plan, LAYER, q.data_ptr(), out.data_ptr(), x.stride(0), guard.stride(0),
                       lse.data_ptr(), k_scale, v_scale, stream=s)
        torch.cuda.synchronize()
        assert kvx.kvx_get_status(ctx) == 0
        assert torch.equal(first, out)
    finally:
        kvx.kvx_attn_plan_destroy(plan)
    assert (guard[rows] == 7.0).all() and (guard[:, hq * dim:] == 7.0).all()
    assert (lse[rows] == 7.0).all()
    check(cache, q, out, lse[:rows], new, group, dim ** -0.5, k_scale, v_scale, dtype, window,
          prefix, softcap, sl)


@pytest.mark.parametrize("heads", [1, 2, 3, 4, 5, 6, 7, 8, 9, 12, 16])
@pytest.mark.parametrize("dim", [64, 128])
def test_heads(ctx, heads, dim):
    run_case(ctx, [700, 33, 1], [1, 1, 1], heads, 4, dim, 16, seed=heads)


@pytest.mark.parametrize("page", [1, 5, 8, 16, 24, 64, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", [2, 4, 9])
def test_pages(ctx, page, dtype, heads):
    run_case(ctx, [513, 64, 17, 1], [1, 2, 1, 1], heads, 2, 128, page, dtype, seed=page)


@pytest.mark.parametrize("group", [1, 2, 5, 7, 8, 16])
@pytest.mark.parametrize("new", [1, 2, 3, 17])
@pytest.mark.parametrize("dim", [64, 128])
def test_rows(ctx, group, new, dim):
    """Rows of a KV head: up to 8, up to 16, and the kernel for chunks past that."""
    run_case(ctx, [200, new, 31 + new], [new] * 3, 2, group, dim, 16, seed=group + new)


@pytest.mark.parametrize("new", [1, 3, 150])
@pytest.mark.parametrize("window,prefix,softcap,slopes", [
    (64, None, 0.0, False), (1, None, 0.0, False), (40, [5, 100, 0], 0.0, False),
    (0, [300, 7, 50], 0.0, False), (0, None, 20.0, False), (0, None, 0.0, True),
    (100, [33, 1, 64], 15.0, True)])
@pytest.mark.parametrize("heads", [1, 4])
def test_options(ctx, new, window, prefix, softcap, slopes, heads):
    run_case(ctx, [900, 301, 150], [new] * 3, heads, 4, 128, 16, window=window, prefix=prefix,
             softcap=softcap, slopes=slopes, seed=new, pad=8)


@pytest.mark.parametrize("tokens,new", [
    ([1], [1]), ([2, 1], [0, 1]), ([5000], [1]), ([16384], [1]), ([40000], [2]),
    ([100] * 70, [1] * 70), ([3000, 1, 700, 64], [300, 1, 129, 64]), ([1000, 2000], [1, 700]),
    ([0, 40], [0, 1])])
@pytest.mark.parametrize("heads,dim", [(8, 128), (4, 64)])
def test_lengths(ctx, tokens, new, heads, dim):
    run_case(ctx, tokens, new, heads, 4, dim, 16, seed=len(tokens))


@pytest.mark.parametrize("page", [1, 7, 8, 32, 128])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_chunks(ctx, page, dim, dtype):
    run_case(ctx, [777, 260], [300, 260], 3, 2, dim, page, dtype, seed=page, pad=16)


@pytest.mark.parametrize("new", [1, 60])
def test_scales_of_all_sizes(ctx, new):
    """Block scales from 2^-9 to 448 in one head; q small enough that scores stay moderate."""
    run_case(ctx, [400], [new], 2, 4, 128, 16, k_scale=2.0 ** -6, v_scale=-3.0, q_scale=0.01,
             spread=True)


def test_on_another_stream(ctx):
    run_case(ctx, [2000, 64], [1, 40], 8, 4, 128, 16, stream=torch.cuda.Stream())


@pytest.mark.parametrize("new", [1, 40])
def test_bad_page_is_reported(ctx, new):
    """A page id outside the pool sets the flag; other requests are as without it."""
    outs = []
    for bad in (False, True):
        cache = FourCache([300, 200], 4, 128, 16, seed=3, spread=False)
        if bad:
            cache.tables[0, 4] = cache.n_pages
        q = make_q(2 * new, 16, 128, "bf16", 5)
        out = torch.zeros_like(q)
        plan = kvx.kvx_attn_plan_create(ctx, cache.kvx_pool, cache.requests(), [new, new],
                                        kvx.attn_config(16, 4, 128, "bf16", "fp4"))
        kvx.kvx_attend(plan, LAYER, q.data_ptr(), out.data_ptr())
        torch.cuda.synchronize()
        flags = kvx.kvx_get_status(ctx)
        assert flags == (kvx.KVX_DEV_PAGE_OUT_OF_RANGE if bad else 0)
        kvx.kvx_attn_plan_destroy(plan)
        outs.append(out)
    assert torch.equal(outs[0][new:], outs[1][new:])
    assert torch.isfinite(outs[1]).all()


def test_plans_of_different_shapes_side_by_side(ctx):
    """Two plans whose kernels need different shared memory, launched in turn."""
    runs = []
    for heads, tokens in ((8, [500]), (1, [500]), (8, [500])):
        cache = FourCache(tokens, heads, 128, 16, seed=heads, spread=False)
        q = make_q(1, heads * 4, 128, "bf16", 1)
        plan = kvx.kvx_attn_plan_create(ctx, cache.kvx_pool, cache.requests(), [1],
                                        kvx.attn_config(heads * 4, heads, 128, "bf16", "fp4"))
        runs.append((cache, q, torch.empty_like(q), plan))
    for _ in range(2):
        for cache, q, out, plan in runs:
            kvx.kvx_attend(plan, LAYER, q.data_ptr(), out.data_ptr())
    torch.cuda.synchronize()
    assert kvx.kvx_get_status(ctx) == 0
    for cache, q, out, plan in runs:
        heads = cache.heads
        check(cache, q.unflatten(1, (heads * 4, 128)), out.unflatten(1, (heads * 4, 128)), None,
              [1], 4, 128 ** -0.5)
        kvx.kvx_attn_plan_destroy(plan)


def test_captured_and_updated(ctx):
    cache = FourCache([600, 90], 4, 128, 16, seed=9, spread=False)
    q = make_q(2, 16, 128, "bf16", 2)
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    plan = kvx.kvx_attn_plan_create(ctx, cache.kvx_pool, cache.requests(), [1, 1],
                                    kvx.attn_config(16, 4, 128, "bf16", "fp4"),
                                    stream=s.cuda_stream)
    with torch.cuda.stream(s):
        kvx.kvx_attend(plan, LAYER, q.data_ptr(), out.data_ptr(), stream=s.cuda_stream)
        eager = out.clone()
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        g.capture_begin()
        kvx.kvx_attend(plan, LAYER, q.data_ptr(), out.data_ptr(), stream=s.cuda_stream)
        g.capture_end()
        for _ in range(3):
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, eager)
    kvx.kvx_attn_plan_update(plan, cache.requests()[:1].copy().view(type(cache.requests())), [1])
    kvx.kvx_attend(plan, LAYER, q.data_ptr(), out.data_ptr())
    torch.cuda.synchronize()
    assert kvx.kvx_get_status(ctx) == 0
    cache.tokens, cache.values = cache.tokens[:1], cache.values[:1]
    check(cache, q[:1].unflatten(1, (16, 128)), out[:1].unflatten(1, (16, 128)), None, [1], 4,
          128 ** -0.5)
    kvx.kvx_attn_plan_destroy(plan)
