import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a)")
    config.addinivalue_line("markers", "slow: full-size workload")


# Cases of tests/test_gpu_beams.py that expect wrong sums.  Their reference subtracts m + log s in
# one 64-bit number (m a beam's largest logit, s the sum of exp(logit - m)).  With m the lowest
# value of bf16 or fp32 that number is m: log s, at most 13, is below half a unit of its last place
# (2^74 at 2^127).  So it gives every token of a beam that is masked altogether the log probability
# 0, although V equal logits have 1 / V each, and expects those tokens ahead of all others.
# tests/test_gpu_beams_masks.py has the same inputs with (logit - m) - log s.
EXPECT_MASKED_BEAM_FIRST = {
    f"test_masks_infinities_and_nan[{vocab}-{dtype}]" for vocab in (40, 20000)
    for dtype in ("bf16", "fp32")} | {
    f"test_mask_values_of_whole_parts[{groups}-lowest-{dtype}]" for groups in (1, 4)
    for dtype in ("bf16", "fp32")}


def pytest_collection_modifyitems(items):
    for item in items:
        if item.path.name == "test_gpu_beams.py" and item.name in EXPECT_MASKED_BEAM_FIRST:
            item.add_marker(pytest.mark.xfail(
                strict=True, reason="expects log probability 0 of a masked beam's tokens"))
