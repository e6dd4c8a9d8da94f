"""kvx_attend over a 4-bit cache in the forms that tests/test_gpu_attend_four.py leaves out: half
precision for up to 8 and up to 16 rows of a KV head and with score options, options at head_dim 64,
and several groups of KV heads (more than 8 of them, copied token by token) with 9 to 16 rows,
options, and pages that end inside a step.  The reference and its tolerance are that file's, but
for the lse of scores with a bias, whose tolerance there has no term for the bias's own rounding.

That term: the kernel for chunks takes 32 keys at a time and adds 2 slope to the bias of the first
two 15 times over.  With a key's distance a, all these numbers are at most slope (a + 31) in size,
so the slope in units of log 2 (2 roundings), the first product, the second key's sum and 15
additions leave a score off by at most 19 x 2^-24 slope (a + 31), and lse by the mean of that under
the weights.  The other kernels round less often."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_gather_gb300.build import build  # noqa: E402

build()
from paged_kv_gather_gb300 import kvx  # noqa: E402
from tests import test_gpu_attend_four  # noqa: E402
from tests.cache_common import attend_reference, visible  # noqa: E402
from tests.four_common import FourCache  # noqa: E402
from tests.test_gpu_attend import LAYER, check, make_q  # noqa: E402
from tests.test_gpu_attend_four import ctx, run_case  # noqa: E402,F401

OPTIONS = [(64, None, 0.0, False), (1, None, 0.0, False), (40, [5, 100, 0], 0.0, False),
           (0, [300, 7, 50], 0.0, False), (0, None, 20.0, False), (0, None, 0.0, True),
           (100, [33, 1, 64], 15.0, True)]


def check_with_bias(cache, q, out, lse, new, group, scale, k_scale, v_scale, dtype, window, prefix,
                    softcap, slopes):
    """tests.test_gpu_attend.check, but lse may be off by the bias's rounding too."""
    check(cache, q, out, None if slopes is not None else lse, new, group, scale, k_scale, v_scale,
          dtype, window, prefix, softcap, slopes)
    if slopes is None:
        return
    sl, qd = slopes.double().cpu().numpy(), q.double().cpu().numpy()
    got, row = lse.double().cpu().numpy(), 0
    for r, n in enumerate(cache.tokens):
        m, pre = new[r], prefix[r] if prefix else 0
        k, v = cache.values[r][0, LAYER] * k_scale, cache.values[r][1, LAYER] * v_scale
        _, ref, _, reach = attend_reference(qd[row:row + m], k, v, m, group, scale, window, pre,
                                            softcap, sl)
        away = np.abs(np.arange(n - m, n)[:, None] - np.arange(n)[None])
        seen = visible(n, m, window, pre)
        for h in range(q.shape[1]):
            s = qd[row:row + m, h] @ k[:, h // group].T * scale
            if softcap:
                s = softcap * np.tanh(s / softcap)
            p = np.where(seen, np.exp(s - sl[h] * away - ref[:, h:h + 1]), 0.0)
            bias = 19 * 2.0 ** -24 * sl[h] * (p * (away + 31)).sum(1)
            room = (q.shape[2] * 2.0 ** -24 * reach[:, h] + softcap * 2.0 ** -21
                    + 2.0 ** -20 * (1 + np.abs(ref[:, h]) + reach[:, h]) + bias)
            assert (np.abs(got[row:row + m, h] - ref[:, h]) <= room).all(), (r, h)
        row += m


@pytest.fixture(autouse=True)
def room_for_bias(monkeypatch):
    monkeypatch.setattr(test_gpu_attend_four, "check", check_with_bias)


@pytest.mark.parametrize("group", [1, 3, 5, 8])
@pytest.mark.parametrize("new", [1, 2, 3])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads", [2, 5, 9])
def test_half_precision_rows(ctx, group, new, dim, heads):  # noqa: F811
    """1 to 24 rows of a KV head: every kernel of few rows, and the one for chunks behind them."""
    run_case(ctx, [200, new, 31 + new], [new] * 3, heads, group, dim, 16, "fp16",
             seed=group + new)


@pytest.mark.parametrize("new", [1, 3, 150])
@pytest.mark.parametrize("window,prefix,softcap,slopes", OPTIONS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads", [1, 4])
def test_half_precision_options(ctx, new, window, prefix, softcap, slopes, dim,  # noqa: F811
                                heads):
    run_case(ctx, [900, 301, 150], [new] * 3, heads, 4, dim, 16, "fp16", window=window,
             prefix=prefix, softcap=softcap, slopes=slopes, seed=new, pad=8)


@pytest.mark.parametrize("new", [1, 3, 40])
@pytest.mark.parametrize("window,prefix,softcap,slopes", OPTIONS)
@pytest.mark.parametrize("dim,heads", [(64, 1), (64, 4), (64, 9), (128, 12)])
def test_options_of_other_shapes(ctx, new, window, prefix, softcap, slopes, dim,  # noqa: F811
                                 heads):
    """With 4 query heads to a KV head, 3 new tokens are 12 rows."""
    run_case(ctx, [700, 301, 150], [new] * 3, heads, 4, dim, 16, window=window, prefix=prefix,
             softcap=softcap, slopes=slopes, seed=new, pad=8)


@pytest.mark.parametrize("heads", [9, 11, 12, 16, 17, 25, 32])
@pytest.mark.parametrize("new", [1, 2])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [1, 7, 16, 40])
def test_groups_of_heads(ctx, heads, new, dim, page):  # noqa: F811
    """Two and more groups of KV heads, the last one smaller; with 8 query heads to one, 2 new
    tokens are 16 rows."""
    run_case(ctx, [333, 64, 1 + new], [new] * 3, heads, 8, dim, page, seed=heads, window=90)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("new", [1, 2])
def test_long_context_of_many_heads(ctx, dtype, new):  # noqa: F811
    """Units of two groups of heads, cut and joined."""
    run_case(ctx, [9000], [new], 12, 8, 128, 16, dtype, seed=3)


@pytest.mark.parametrize("heads,new", [(9, 1), (9, 2), (20, 2)])
def test_bad_page_of_many_heads(ctx, heads, new):  # noqa: F811
    """A page id outside the pool sets the flag; other requests are as without it."""
    outs = []
    for bad in (False, True):
        cache = FourCache([300, 200], heads, 128, 16, seed=3, spread=False)
        if bad:
            cache.tables[0, 4] = cache.n_pages
        q = make_q(2 * new, heads * 8, 128, "bf16", 5)
        out = torch.zeros_like(q)
        plan = kvx.kvx_attn_plan_create(ctx, cache.kvx_pool, cache.requests(), [new, new],
                                        kvx.attn_config(heads * 8, heads, 128, "bf16", "fp4"))
        kvx.kvx_attend(plan, LAYER, q.data_ptr(), out.data_ptr())
        torch.cuda.synchronize()
        assert kvx.kvx_get_status(ctx) == (kvx.KVX_DEV_PAGE_OUT_OF_RANGE if bad else 0)
        kvx.kvx_attn_plan_destroy(plan)
        outs.append(out)
    assert torch.equal(outs[0][new:], outs[1][new:])
    assert torch.isfinite(outs[1]).all()
