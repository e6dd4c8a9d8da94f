"""kvx_select_beams where finite mask values outweigh everything else of a beam, against sums whose
norm is taken relative to the largest logit.

Of V equal logits each token has probability 1 / V, whatever their value, so its continuation's sum
is score - log V.  Beside a value of 1e12 or more log V is less than 64 bits resolve: a norm formed as
largest + log sum loses it, and a beam that is masked altogether would continue at its own score.
The tolerance is that of tests/test_gpu_beams.py."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_gather_gb300.build import build  # noqa: E402

build()
from tests.test_gpu_beams import CLOSE, TORCH, ctx, make, select  # noqa: E402,F401

MASKS = [-1e9, -1e12, -1e30, "lowest"]


def value_of(mask, dtype):
    return torch.finfo(TORCH[dtype]).min if mask == "lowest" else mask


def sums_of(logits, scores):
    """[groups, width, vocab] of sums in 64 bits, the norm relative to a beam's largest logit."""
    groups, width = scores.shape
    x = logits.double().cpu().view(groups, width, -1).numpy()
    away = x - x.max(-1, keepdims=True)
    norm = np.log(np.exp(away).sum(-1, keepdims=True))
    return scores.double().cpu().numpy()[..., None] + (away - norm)


def check(got, logits, scores, picks):
    """Best first, none twice, each with its own sum and as large as the one that belongs there."""
    parents, tokens, sums = (t.numpy() for t in got)
    for g, s in enumerate(sums_of(logits, scores)):
        best = np.sort(s.ravel())[::-1][:picks]
        took = s[parents[g], tokens[g]]
        assert len(set(zip(parents[g].tolist(), tokens[g].tolist()))) == picks
        assert (np.abs(took - best) <= CLOSE).all(), (g, took, best)
        assert (np.abs(sums[g] - took) <= CLOSE / 2 + 2.0 ** -24 * np.abs(took)).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("vocab", [2, 40, 5000, 40000, 130001])
def test_all_logits_a_mask_value(ctx, dtype, mask, vocab):  # noqa: F811
    _, s = make(2, 3, vocab, dtype, 1)
    x = torch.full((6, vocab), value_of(mask, dtype), dtype=TORCH[dtype], device="cuda")
    picks = min(8, vocab)
    parents, tokens, sums = got = select(ctx, x, s, picks, dtype)
    check(got, x, s, picks)
    for g in range(2):  # one beam's tokens in order, at its score less log V
        best = int(s[g].argmax())
        want = float(s[g, best]) - math.log(vocab)
        first = [k for k in range(picks) if int(parents[g, k]) == best]
        assert tokens[g, first].tolist() == list(range(len(first))) and first[0] == 0
        assert abs(float(sums[g, 0]) - want) <= CLOSE / 2 + 2.0 ** -24 * abs(want)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("groups", [1, 4])
def test_masked_beam_ranks_behind_live_ones(ctx, dtype, mask, groups):  # noqa: F811
    """The beam with the highest score so far is masked altogether: its continuations are log V
    lower, and the live beams' best come first."""
    vocab = 40000
    x, s = make(groups, 4, vocab, dtype, 2)
    x[1::4] = value_of(mask, dtype)
    s.copy_(torch.tensor([-3.0, -1.0, -3.5, -4.0]).expand(groups, 4))
    parents, _, _ = got = select(ctx, x, s, 8, dtype)
    check(got, x, s, 8)
    assert (parents[:, 0] != 1).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("mask", MASKS)
def test_masked_beams_and_masked_parts(ctx, dtype, mask):  # noqa: F811
    """Rows of mask values but for a few tokens, whole rows of them, and rows of two mask values."""
    vocab = 40000
    value = value_of(mask, dtype)
    x, s = make(3, 4, vocab, dtype, 8)
    y = torch.full_like(x, value)
    y[:, 17000:17100] = x[:, 17000:17100]
    y[1::4] = value
    y[2, :] = value
    y[2, 30000:30010] = value / 2
    check(select(ctx, y, s, 16, dtype), y, s, 16)
