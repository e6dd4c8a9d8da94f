"""kvx_select_beams with many picks: logits without ties take no longer per pick than with few.

Where more candidates reach a bar than a list holds, they are taken one after the other, each round
looking through all of them again: meant for ties, hundreds of microseconds where counting takes
tens.  Ordinary logits must not get there.  Twice the picks are twice the candidates, so at most twice
the time of what depends on them; the bounds below are twice that again, and a bar that is far too
low misses them by another factor of two at least."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_gather_gb300.build import build  # noqa: E402

build()
from paged_kv_gather_gb300 import kvx  # noqa: E402
from tests.test_gpu_beams import check_selection, ctx, make, select  # noqa: E402,F401


def device_time(ctx, x, scores, picks, dtype):  # noqa: F811
    """Microseconds of a call, of the median of seven runs of ten."""
    groups, width = scores.shape
    cfg = kvx.select_config(groups, width, x.shape[1], picks, dtype)
    work = torch.empty(kvx.kvx_select_workspace(ctx, cfg), dtype=torch.uint8, device="cuda")
    parents, tokens = (torch.empty((groups, picks), dtype=torch.int32, device="cuda")
                       for _ in range(2))
    sums = torch.empty((groups, picks), device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    times = []
    with torch.cuda.stream(stream):
        for _ in range(8):
            begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            begin.record(stream)
            for _ in range(10):
                kvx.kvx_select_beams(ctx, cfg, x.data_ptr(), scores.data_ptr(),
                                     parents.data_ptr(), tokens.data_ptr(), sums.data_ptr(),
                                     work.data_ptr(), stream=stream.cuda_stream)
            end.record(stream)
            end.synchronize()
            times.append(begin.elapsed_time(end) * 100.0)
    return sorted(times[1:])[3]


@pytest.mark.parametrize("width,vocab", [(16, 500000), (32, 500000)])
def test_merging_many_lists(ctx, width, vocab):  # noqa: F811
    """32 parts of a row, 32 picks of each: the bar over all of a group's lists."""
    x, s = make(1, width, vocab, "bf16", 11)
    s.fill_(-3.0)
    check_selection(select(ctx, x, s, 32, "bf16"), x, s, 32)
    few, many = (device_time(ctx, x, s, picks, "bf16") for picks in (16, 32))
    assert many < 4 * few, (few, many)


@pytest.mark.parametrize("groups,width,vocab,dtype", [(16, 8, 128256, "bf16"),
                                                      (16, 8, 128256, "fp16"),
                                                      (1, 2, 128256, "fp32")])
def test_as_many_picks_as_there_may_be(ctx, groups, width, vocab, dtype):  # noqa: F811
    """A part's own bar, and what reaches it, at KVX_MAX_PICKS."""
    x, s = make(groups, width, vocab, dtype, 12)
    check_selection(select(ctx, x, s, 64, dtype), x, s, 64)
    few, many = (device_time(ctx, x, s, picks, dtype) for picks in (32, 64))
    assert many < 4 * few, (few, many)


@pytest.mark.parametrize("picks", [16, 17, 31, 32, 33, 47, 63])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_picks_around_every_choice(ctx, picks, dtype):  # noqa: F811
    for groups, width, vocab in ((1, 4, 3000), (3, 7, 40001), (20, 2, 17000)):
        x, s = make(groups, width, vocab, dtype, picks)
        check_selection(select(ctx, x, s, picks, dtype), x, s, picks)


@pytest.mark.parametrize("vocab,live", [(1000, 1000), (128256, 1000), (50257, 600)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_few_tokens_left(ctx, vocab, live, dtype):  # noqa: F811
    """Fewer groups of threads have a logit than there are picks: all that is left are candidates,
    up to 1000 instead of some 50, each compared with all."""
    x, s = make(1, 32, vocab, dtype, 13)
    x[:, live:] = -float("inf")
    check_selection(select(ctx, x, s, 64, dtype), x, s, 64)
    few, many = (device_time(ctx, x, s, picks, dtype) for picks in (32, 64))
    assert many < 6 * few, (few, many)
