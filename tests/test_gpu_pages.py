"""kvx_fork_pages, kvx_free_pages and kvx_compact_pages against a model on Python lists:
counts, tables and every byte of the pool are equal."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_gather_gb300.build import build  # noqa: E402

build()
from paged_kv_gather_gb300 import kvx  # noqa: E402
from tests.cache_common import PagesModel  # noqa: E402


@pytest.fixture(scope="module")
def ctx():
    c = kvx.kvx_create(0)
    yield c
    kvx.kvx_destroy(c)


class World:
    """A pool of random bytes with a model beside it."""

    def __init__(self, n_pages, page, layers=3, kv=2, token_bytes=48, seed=0):
        rng = np.random.default_rng(seed)
        self.rng, self.n_pages, self.page = rng, n_pages, page
        self.shape = (kv, layers, n_pages, page, token_bytes)
        self.pool = torch.randint(0, 256, self.shape, dtype=torch.uint8, device="cuda")
        self.kvx_pool = kvx.Pool.from_tensor(self.pool, page)
        self.bytes = self.pool.cpu().numpy()
        self.model = PagesModel([0] * n_pages, page)
        self.refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        self.free_order = rng.permutation(n_pages).tolist()

    def hold(self, n, seed=0):
        """A table of n random free pages, held once."""
        table = []
        while len(table) < n:
            p = self.free_order.pop()
            if self.model.refs[p] == 0:
                table.append(p)
                self.model.refs[p] = 1
        return table

    def upload(self):
        self.refs.copy_(torch.tensor(self.model.refs, dtype=torch.int32))

    def check(self, refs=True):
        for a, b, tokens in self.model.moves:
            self.bytes[:, :, b, :tokens] = self.bytes[:, :, a, :tokens]
        self.model.moves = []
        assert self.refs.cpu().tolist() == self.model.refs
        got = self.pool.cpu().numpy()
        assert np.array_equal(got, self.bytes)


def dev(table, extra=0):
    t = torch.full((len(table) + extra + 1,), -7, dtype=torch.int32, device="cuda")
    t[:len(table)] = torch.tensor(table, dtype=torch.int32)
    return t


def fork(ctx, w, entries):
    """entries: (parent list, shared, total, copy, grow) -> child device tables, model's."""
    w.upload()
    parents = {}
    args, children = [], []
    for parent, shared, total, copy, grow in entries:
        n = -(-total // w.page)
        if grow:
            c = dev(parent, n)
            args.append((c.data_ptr(), c.data_ptr(), shared, total, False))
        else:
            if id(parent) not in parents:
                parents[id(parent)] = dev(parent)
            c = dev([], n)
            args.append((parents[id(parent)].data_ptr() if shared else 0, c.data_ptr(), shared,
                         total, copy))
        children.append((c, n))
    want = w.model.fork_batch(entries)
    torch.cuda.synchronize()
    kvx.kvx_fork_pages(ctx, w.kvx_pool, w.refs.data_ptr(), kvx.forks_array(args))
    torch.cuda.synchronize()
    return children, want


@pytest.mark.parametrize("page", [1, 3, 16, 64])
@pytest.mark.parametrize("n_pages", [40, 256, 257, 5000, 70000])
def test_fork_grow_allocate_and_free(ctx, page, n_pages):
    """All kinds of entries in one batch, then all of it freed again."""
    w = World(n_pages, page, seed=page * n_pages, token_bytes=16 if n_pages > 6000 else 48)
    big = min(n_pages // 4, 300)
    a, b = w.hold(big), w.hold(3)
    na, nb = big * page - page // 2, 3 * page
    entries = [(a, na, na + 1, False, False), (a, na, na + 2 * page, False, False),
               (a, max(1, na // 2), na // 2 + page, False, False), ([], 0, 2 * page + 1, False, False),
               (b, nb, nb + page, False, True), (b, 2 * page, 2 * page, True, False),
               (b, 0, 0, False, False)]
    children, want = fork(ctx, w, entries)
    assert kvx.kvx_get_status(ctx) == 0
    for (c, n), t in zip(children, want):
        assert c[:n].cpu().tolist() == t and (c[n:] == -7).all()
    w.check()
    held = [(a, dev(a)), (want[4], children[4][0])] + [(t, c) for i, ((c, n), t) in
                                                      enumerate(zip(children, want)) if i != 4]
    kvx.kvx_free_pages(ctx, w.kvx_pool, w.refs.data_ptr(),
                       kvx.tables_array([(c.data_ptr(), len(t)) for t, c in held]))
    torch.cuda.synchronize()
    assert kvx.kvx_get_status(ctx) == 0
    for t, c in held:
        w.model.free(t)
        assert (c[:len(t)] == -1).all()
    w.check()
    assert not any(w.model.refs)


@pytest.mark.parametrize("entries", [3, 200])
def test_fork_whole_copies(ctx, entries):
    """Copies of whole requests; 200 entries go through a descriptor slot."""
    w = World(20 * entries + 20, 16, layers=4, token_bytes=256, seed=entries)
    parents = [w.hold(int(n)) for n in w.rng.integers(1, 9, entries)]
    batch = [(t, int(w.rng.integers(1, 16 * len(t) + 1)), 16 * len(t) + 5, i % 3 != 0, False)
             for i, t in enumerate(parents)]
    children, want = fork(ctx, w, batch)
    assert kvx.kvx_get_status(ctx) == 0
    for (c, n), t in zip(children, want):
        assert c[:n].cpu().tolist() == t
    w.check()


def test_fork_without_enough_pages_changes_nothing(ctx):
    w = World(300, 16)
    t = w.hold(290)
    children, want = fork(ctx, w, [(t, 16 * 290, 16 * 295, False, False), (t, 40, 40, True, False),
                                   ([], 0, 16 * 3, False, False)])
    assert want is None
    assert kvx.kvx_get_status(ctx) == kvx.KVX_DEV_NO_FREE_PAGE
    for c, n in children:
        assert (c == -7).all()
    w.check()
    # Exactly enough is enough, and the next call finds everything as it should be.
    children, want = fork(ctx, w, [(t, 16 * 290, 16 * 297, False, False), (t, 40, 40, True, False)])
    assert kvx.kvx_get_status(ctx) == 0 and all(n > 0 for n in w.model.refs)
    for (c, n), x in zip(children, want):
        assert c[:n].cpu().tolist() == x
    w.check()


def test_fork_and_free_report_bad_entries(ctx):
    w = World(100, 16)
    t = w.hold(6)
    free = next(p for p in range(100) if w.model.refs[p] == 0)
    w.upload()
    parent = dev([t[0], -1, t[2], 100, 99 if w.model.refs[99] == 0 else 98, t[5]])
    child = dev([], 8)
    kvx.kvx_fork_pages(ctx, w.kvx_pool, w.refs.data_ptr(),
                       kvx.forks_array([(parent.data_ptr(), child.data_ptr(), 85, 86, 0)]))
    torch.cuda.synchronize()
    got = child.cpu().tolist()
    assert got[:6] == [t[0], -1, t[2], -1, -1, free]
    assert kvx.kvx_get_status(ctx) == (kvx.KVX_DEV_PAGE_OUT_OF_RANGE | kvx.KVX_DEV_PAGE_NOT_HELD)
    w.model.refs[t[0]] += 1
    w.model.refs[t[2]] += 1
    w.model.refs[free] = 1
    w.model.moves.append((t[5], free, 5))
    w.check()
    # Freed three times, held twice: one report, and the count ends at zero.
    c = dev([t[0]] * 3)
    kvx.kvx_free_pages(ctx, w.kvx_pool, w.refs.data_ptr(), kvx.tables_array([(c.data_ptr(), 3)]))
    torch.cuda.synchronize()
    assert kvx.kvx_get_status(ctx) == kvx.KVX_DEV_PAGE_NOT_HELD
    w.model.refs[t[0]] = 0
    c = dev([-1, 10 ** 9])
    kvx.kvx_free_pages(ctx, w.kvx_pool, w.refs.data_ptr(), kvx.tables_array([(c.data_ptr(), 2)]))
    torch.cuda.synchronize()
    assert kvx.kvx_get_status(ctx) == kvx.KVX_DEV_PAGE_OUT_OF_RANGE
    assert (c[:2] == -1).all()
    w.check()


@pytest.mark.parametrize("live", [0.0, 0.1, 0.5, 0.9, 1.0])
@pytest.mark.parametrize("n_pages,page,token_bytes", [(1, 4, 32), (64, 16, 512), (700, 5, 48),
                                                      (9001, 2, 16)])
def test_compact(ctx, live, n_pages, page, token_bytes):
    w = World(n_pages, page, token_bytes=token_bytes, seed=int(live * 10) + n_pages)
    n = int(live * n_pages)
    tables = [t for t in (w.hold(n // 3), w.hold(n // 2), w.hold(n - n // 3 - n // 2)) if t]
    if tables:
        shared = tables[0][::2]
        for p in shared:
            w.model.refs[p] += 1
        tables.append(shared)
    w.upload()
    d = [dev(t) for t in tables]
    n_live = torch.full((2,), -7, dtype=torch.int32, device="cuda")
    remap = torch.full((n_pages + 1,), -7, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    kvx.kvx_compact_pages(ctx, w.kvx_pool, w.refs.data_ptr(),
                          kvx.tables_array([(x.data_ptr(), len(t)) for x, t in zip(d, tables)]),
                          n_live.data_ptr(), remap.data_ptr())
    torch.cuda.synchronize()
    assert kvx.kvx_get_status(ctx) == 0
    before = [x > 0 for x in w.model.refs]
    count, to, want = w.model.compact(tables)
    assert n_live.cpu().tolist() == [count, -7] and count == n
    assert remap.cpu().tolist() == [to[p] if before[p] else -1 for p in range(n_pages)] + [-7]
    for x, t in zip(d, want):
        assert x.cpu().tolist() == t + [-7]
    assert all((c > 0) == (p < n) for p, c in enumerate(w.model.refs))
    w.check()


def test_compact_reports_entries_that_hold_nothing(ctx):
    w = World(50, 4)
    t = w.hold(10)
    w.upload()
    free = next(p for p in range(50) if w.model.refs[p] == 0)
    d = dev(t + [free, -1, 50])
    torch.cuda.synchronize()
    kvx.kvx_compact_pages(ctx, w.kvx_pool, w.refs.data_ptr(),
                          kvx.tables_array([(d.data_ptr(), 13)]))
    torch.cuda.synchronize()
    assert kvx.kvx_get_status(ctx) == (kvx.KVX_DEV_PAGE_OUT_OF_RANGE | kvx.KVX_DEV_PAGE_NOT_HELD)
    _, _, (want,) = w.model.compact([t])
    assert d.cpu().tolist() == want + [free, -1, 50, -7]
    w.check()


def test_largest_pool(ctx):
    """KVX_MAX_UPKEEP_PAGES pages: the bitmap fills shared memory; one more is refused."""
    n = kvx.KVX_MAX_UPKEEP_PAGES
    pool = torch.zeros((1, 1, n, 1, 16), dtype=torch.uint8, device="cuda")
    p = kvx.Pool.from_tensor(pool, 1)
    refs = torch.ones(n, dtype=torch.int32, device="cuda")
    refs[1::2] = 0
    pool.view(n, 16)[:, 0] = (torch.arange(n, device="cuda") % 251).to(torch.uint8)
    table = torch.arange(0, n, 2, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    kvx.kvx_compact_pages(ctx, p, refs.data_ptr(), kvx.tables_array([(table.data_ptr(), n // 2)]))
    torch.cuda.synchronize()
    assert kvx.kvx_get_status(ctx) == 0
    assert torch.equal(refs, (torch.arange(n, device="cuda") < n // 2).int())
    assert torch.equal(table.sort().values, torch.arange(n // 2, device="cuda").int())
    where = pool.view(n, 16)[table.long(), 0]
    assert torch.equal(where, (torch.arange(0, n, 2, device="cuda") % 251).to(torch.uint8))
    child = torch.zeros(9, dtype=torch.int32, device="cuda")
    refs[:] = 1
    refs[-9:] = 0
    torch.cuda.synchronize()
    kvx.kvx_fork_pages(ctx, p, refs.data_ptr(), kvx.forks_array([(0, child.data_ptr(), 0, 9, 0)]))
    torch.cuda.synchronize()
    assert kvx.kvx_get_status(ctx) == 0
    assert child.cpu().tolist() == list(range(n - 9, n)) and (refs == 1).all()


def test_offsets_past_32_bits(ctx):
    """Pages whose byte offset in a layer is past 4 GiB are copied and moved."""
    page_bytes = 64 << 10
    n = (1 << 32) // page_bytes + 40
    pool = torch.zeros((1, 1, n, 16, 4096), dtype=torch.uint8, device="cuda")
    p = kvx.Pool.from_tensor(pool, 16)
    refs = torch.ones(n, dtype=torch.int32, device="cuda")
    refs[-30:-1] = 0                     # the last page is live, those before it free
    pool[0, 0, -1] = torch.randint(0, 256, (16, 4096), dtype=torch.uint8, device="cuda")
    parent = torch.tensor([n - 1], dtype=torch.int32, device="cuda")
    child = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    kvx.kvx_fork_pages(ctx, p, refs.data_ptr(), kvx.forks_array(
        [(parent.data_ptr(), child.data_ptr(), 15, 16, 0)]))
    torch.cuda.synchronize()
    assert kvx.kvx_get_status(ctx) == 0 and int(child) == n - 30
    assert torch.equal(pool[0, 0, n - 30, :15], pool[0, 0, -1, :15])
    assert not pool[0, 0, n - 30, 15].any()
    want = pool[0, 0, -1].clone()
    kvx.kvx_compact_pages(ctx, p, refs.data_ptr(), kvx.tables_array([(parent.data_ptr(), 1)]))
    torch.cuda.synchronize()
    assert int(parent) == n - 29 and torch.equal(pool[0, 0, n - 29], want)
    assert kvx.kvx_get_status(ctx) == 0


def test_capture_of_a_small_call(ctx):
    """A call whose descriptors travel in the launch can be captured and replayed."""
    w = World(100, 16)
    t = w.hold(4)
    w.upload()
    parent, child = dev(t), dev([], 5)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        kvx.kvx_fork_pages(ctx, w.kvx_pool, w.refs.data_ptr(), kvx.forks_array(
            [(parent.data_ptr(), child.data_ptr(), 60, 70, 0)]), stream=stream.cuda_stream)
        kvx.kvx_free_pages(ctx, w.kvx_pool, w.refs.data_ptr(), kvx.tables_array(
            [(child.data_ptr(), 5)]), stream=stream.cuda_stream)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert kvx.kvx_get_status(ctx) == 0
    assert w.refs.cpu().tolist() == w.model.refs
    free = next(p for p in range(100) if w.model.refs[p] == 0)
    w.model.moves.append((t[3], free, 12))
    w.check()
