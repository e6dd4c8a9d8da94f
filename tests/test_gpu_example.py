"""The serving example: prefill, fork, decode, free, compact, evict and restore in one pool
give, to the last bit, what the same steps give on pages that nobody shares or moves."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_gather_gb300.build import build  # noqa: E402

build()
from examples import serve_step  # noqa: E402


@pytest.mark.parametrize("prompt,steps,children", [(77, 12, 4), (64, 5, 3), (200, 20, 2)])
def test_shared_pages_change_nothing(prompt, steps, children):
    r = serve_step.run(prompt, steps, children)
    assert r["status"] == 0 and r["identical"]
    assert r["survivors"] == children - children // 2
    assert r["tokens"] == prompt + 3 * steps
    # Shared full prompt pages once, the rest per survivor.
    full, total = prompt // 16, -(-r["tokens"] // 16)
    expect = full + r["survivors"] * (total - full)
    evicted_copy = full                      # the restored one no longer shares
    assert r["live_pages"] in (expect, expect + evicted_copy)
