"""Sizes at which the attention calls stop, by the host checks alone."""
import pytest

from paged_kv_gather_gb300.build import build

build()
from paged_kv_gather_gb300 import kvx  # noqa: E402

A = 1 << 40  # an aligned address that nothing dereferences


@pytest.mark.parametrize("last,status", [(1, kvx.KVX_OK), (2, kvx.KVX_ERR_CAPACITY)])
def test_rows_of_a_step(last, status):
    """Rows fit in 32 bits together with the empty end of a block of 256 of them: the kernel
    steps to the row past its last block."""
    heads = 127
    most = (2 ** 31 - 256) // heads          # whole tokens of so many heads
    new = (most - 1, last)
    assert (new[0] + 1) * heads <= 2 ** 31 - 256 < (new[0] + 2) * heads <= 2 ** 31 - 1
    p = kvx.Pool(1, 2, 16, 64, 128, [A], [A])
    reqs = kvx.requests_array([(A, None, n) for n in new])
    st, msg = kvx.kvx_attn_validate(p, reqs, new, kvx.attn_config(heads, 1, 64))
    assert st == status and bool(msg) == (status != kvx.KVX_OK)
