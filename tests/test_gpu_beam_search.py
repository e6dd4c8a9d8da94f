"""A beam search as a user runs it: rotated append into 4-bit pages, attention, selection and
reordering in turn (examples/beam_search.py), against the same hypotheses decoded from their
tokens, and the selection of one step against all continuations in 64 bits."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_gather_gb300.build import build  # noqa: E402

build()

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "beam_search", os.path.join(ROOT, "examples", "beam_search.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("prompt,beams,steps", [(45, 4, 40), (16, 2, 17), (1, 8, 20), (100, 5, 3)])
def test_search(example, prompt, beams, steps):
    r = example.run(prompt, beams, steps)
    assert r["status"] == 0 and r["identical"] and r["counts_add_up"]
    assert r["distinct"] == beams and r["falling"]
    assert r["tokens"] == prompt + steps


def test_sums_are_those_of_the_tokens(example):
    """A hypothesis' sum is that of its tokens' log probabilities along the way: within what 32-bit
    sums of `steps` terms round (2^-24 of 6 per term, size 64) and the selection's own 2^-22."""
    model = example.Model()
    prompt = torch.arange(30, device="cuda") % example.VOCAB
    steps, beams = 12, 4
    e, said, sums, _, _ = example.search(model, prompt, beams, steps)
    e.close()
    e = example.Engine(model, beams)
    x = e.prefill(prompt).expand(beams, -1)
    e.spread(30)
    total = torch.zeros(beams, dtype=torch.float64, device="cuda")
    for step in range(steps):
        log_p = torch.log_softmax(example.rows(x, model.logits).double(), 1)
        total += log_p.gather(1, said[:, step:step + 1].long())[:, 0]
        x = e.decode(30 + step + 1, said[:, step].long())
    e.close()
    assert ((total - sums.double()).abs() <= steps * (2.0 ** -22 + 2.0 ** -24 * 64)).all()
