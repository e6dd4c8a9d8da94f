"""Page upkeep where its limits lie: pool sizes about the default limit of shared memory,
calls on several pools of one context at a time, and as many table entries as there may be."""
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
from paged_kv_gather_gb300 import kvx  # noqa: E402

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


class Copier:
    """A pool whose parent request is copied whole into a child and the child freed again:
    every round finds the pool as the one before it did."""

    def __init__(self, n_pages, pages, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.bytes = torch.randint(0, 256, (2, 3, n_pages, 4, 64), dtype=torch.uint8, device="cuda",
                                   generator=g)
        self.pool = kvx.Pool.from_tensor(self.bytes, 4)
        order = torch.randperm(n_pages, device="cuda", generator=g).int()
        self.parent = order[:pages].contiguous()
        self.refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        self.refs[self.parent.long()] = 1
        self.before = self.refs.clone()
        self.want = (self.refs == 0).nonzero()[:pages, 0].int()
        self.child = torch.full_like(self.parent, -1)
        self.forks = kvx.forks_array([(self.parent.data_ptr(), self.child.data_ptr(), 4 * pages,
                                       4 * pages, True)])
        self.tables = kvx.tables_array([(self.child.data_ptr(), pages)])

    def round(self, ctx, stream):
        """Returns the child's table and the counts after the copy, taken on the stream."""
        kvx.kvx_fork_pages(ctx, self.pool, self.refs.data_ptr(), self.forks,
                           stream=stream.cuda_stream)
        seen = self.child.clone(), self.refs.clone()
        kvx.kvx_free_pages(ctx, self.pool, self.refs.data_ptr(), self.tables,
                           stream=stream.cuda_stream)
        return seen

    def check(self, seen):
        held = self.before.clone()
        held[self.want.long()] = 1
        for child, refs in seen:
            assert torch.equal(child, self.want) and torch.equal(refs, held)
        assert torch.equal(self.refs, self.before)
        assert torch.equal(self.bytes[:, :, self.want.long()], self.bytes[:, :, self.parent.long()])


def test_calls_on_different_pools_at_the_same_time():
    """A captured call replayed on one stream beside more direct calls on another than a
    context keeps anything for, on one context: neither sees the other."""
    ctx = kvx.kvx_create(0)
    a, b = Copier(60000, 300, 1), Copier(20000, 37, 2)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=sa):
        last = a.round(ctx, sa)
    got_a, got_b = [], []
    for _ in range(150):
        with torch.cuda.stream(sa):
            graph.replay()
            got_a.append([x.clone() for x in last])
        with torch.cuda.stream(sb):
            got_b.append(b.round(ctx, sb))
    torch.cuda.synchronize()
    a.check(got_a)
    b.check(got_b)
    assert kvx.kvx_get_status(ctx) == 0
    kvx.kvx_destroy(ctx)


def test_as_many_entries_as_a_call_takes():
    """2^31 - 1 table entries in a call: a fork that shares them, a compaction that rewrites
    them and a free that gives them back."""
    total, n = 2 ** 31 - 1, 1 << 20
    ctx = kvx.kvx_create(0)
    pool = torch.zeros((1, 1, n, 1, 16), dtype=torch.uint8, device="cuda")
    p = kvx.Pool.from_tensor(pool, 1)
    parent = torch.arange(1, n, dtype=torch.int32, device="cuda")   # page 0 is free
    refs = torch.ones(n, dtype=torch.int32, device="cuda")
    refs[0] = 0
    table = torch.full((total + 1,), -7, dtype=torch.int32, device="cuda")
    n_live = torch.zeros(1, dtype=torch.int32, device="cuda")
    whole, rest = divmod(total, n - 1)
    at = [(i * (n - 1), n - 1) for i in range(whole)] + [(whole * (n - 1), rest)]

    def is_parent(last):
        for begin, m in at:
            want = parent[:m].clone()
            want[parent[:m] == n - 1] = last
            assert torch.equal(table[begin:begin + m], want)
        assert int(table[total]) == -7

    torch.cuda.synchronize()
    kvx.kvx_fork_pages(ctx, p, refs.data_ptr(), kvx.forks_array(
        [(parent.data_ptr(), table.data_ptr() + 4 * begin, m, m, False) for begin, m in at]))
    torch.cuda.synchronize()
    assert kvx.kvx_get_status(ctx) == 0
    is_parent(n - 1)
    held = torch.full_like(refs, 1 + whole)
    held[1:1 + rest] += 1
    held[0] = 0
    assert torch.equal(refs, held)
    tables = kvx.tables_array([(table.data_ptr(), total)])
    kvx.kvx_compact_pages(ctx, p, refs.data_ptr(), tables, n_live.data_ptr())
    torch.cuda.synchronize()
    assert kvx.kvx_get_status(ctx) == 0 and int(n_live) == n - 1
    is_parent(0)
    held[0], held[-1] = held[-1].clone(), 0
    assert torch.equal(refs, held)
    kvx.kvx_free_pages(ctx, p, refs.data_ptr(), tables)
    torch.cuda.synchronize()
    assert kvx.kvx_get_status(ctx) == 0
    assert int(table[:total].min()) == int(table[:total].max()) == -1 and int(table[total]) == -7
    assert torch.equal(refs, (torch.arange(n, device="cuda") < n - 1).int())
    kvx.kvx_destroy(ctx)


@pytest.mark.parametrize("children,tokens", [(1, 9), (4, 9), (4, 1), (40, 15)])
def test_copying_warps_of_a_fork(children, tokens):
    """No warp of a fork has a second copy while SMs are left over: 12 warps of a CTA copy."""
    ctx = kvx.kvx_create(0)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    bytes_ = torch.zeros((2, 32, 2 * children + 1, 16, 2048), dtype=torch.uint8, device="cuda")
    p = kvx.Pool.from_tensor(bytes_, 16)
    refs = torch.zeros(2 * children + 1, dtype=torch.int32, device="cuda")
    refs[0] = 1
    parent = torch.zeros(1, dtype=torch.int32, device="cuda")
    child = torch.zeros((children, 1), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    kvx.kvx_fork_pages(ctx, p, refs.data_ptr(), kvx.forks_array(
        [(parent.data_ptr(), c.data_ptr(), tokens, 16, False) for c in child]))
    items, ctas, threads, _ = kvx.kvx_last_launch(ctx)
    torch.cuda.synchronize()
    assert threads == 512 and items >= children * 64
    assert ctas == min(sms, -(-items // 12))
    assert child[:, 0].cpu().tolist() == list(range(1, children + 1))
    assert kvx.kvx_get_status(ctx) == 0
    kvx.kvx_destroy(ctx)
