"""Page upkeep where its limits lie: pool sizes about the default limit of shared memory."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_gather_gb300.build import build  # noqa: E402

build()

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

ABOUT_THE_DEFAULT = """
import torch
from paged_kv_gather_gb300 import kvx
ctx = kvx.kvx_create(0)
for n in (321024, 321025, 330000, 347136, 347137):
    pool = torch.zeros((1, 1, n, 1, 16), dtype=torch.uint8, device="cuda")
    p = kvx.Pool.from_tensor(pool, 1)
    refs = torch.ones(n, dtype=torch.int32, device="cuda")
    refs[-2] = 0
    pool[0, 0, -1] = 5
    parent = torch.tensor([n - 1], dtype=torch.int32, device="cuda")
    child = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    kvx.kvx_fork_pages(ctx, p, refs.data_ptr(),
                       kvx.forks_array([(parent.data_ptr(), child.data_ptr(), 1, 1, 1)]))
    torch.cuda.synchronize()
    assert int(child) == n - 2 and (refs == 1).all() and (pool[0, 0, -2] == 5).all()
    refs[0] = 0
    torch.cuda.synchronize()
    kvx.kvx_compact_pages(ctx, p, refs.data_ptr(),
                          kvx.tables_array([(parent.data_ptr(), 1), (child.data_ptr(), 1)]))
    torch.cuda.synchronize()
    assert int(parent) == 0 and int(child) == n - 2
    assert int(refs[0]) == 1 and int(refs[-1]) == 0 and int(refs.sum()) == n - 1
    assert (pool[0, 0, 0] == 5).all()
    assert kvx.kvx_get_status(ctx) == 0
kvx.kvx_destroy(ctx)
"""


def test_pools_about_the_default_limit_of_shared_memory():
    """Bitmaps that end, with the kernels' static shared memory, just below and above what a
    launch gets without asking for more, in a process that has launched no larger one."""
    r = subprocess.run([sys.executable, "-c", ABOUT_THE_DEFAULT], cwd=ROOT, timeout=300,
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
