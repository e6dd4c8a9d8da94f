"""kvx_select_beams against its definition in 64 bits, kvx_reorder_beams against a model of the
bookkeeping on Python lists.

Tolerance of a selection: a sum is so_far + logit - log sum exp.  The sum of exponentials is off
by about 2^-22 of itself (an exponential's few 2^-23, and 2^-24 per addition inside a thread), so
sums are off by 2^-22 and, as they are given in 32 bits, by 2^-24 of their size.  Continuations
closer than 2^-21 may change places."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_gather_gb300.build import build  # noqa: E402

build()
from paged_kv_gather_gb300 import kvx  # noqa: E402

TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CLOSE = 2.0 ** -21


@pytest.fixture(scope="module")
def ctx():
    c = kvx.kvx_create(0)
    yield c
    kvx.kvx_destroy(c)


# ---------------------------------------------------------------------------- selection

def select(ctx, logits, scores, picks, dtype, done=None, done_token=-7, stride=0, ptr=None,
           vocab=None, stream=0):
    groups, width = scores.shape
    vocab = vocab or logits.shape[-1]
    cfg = kvx.select_config(groups, width, vocab, picks, dtype, done_token)
    nbytes = kvx.kvx_select_workspace(ctx, cfg)
    work = torch.full((nbytes + 16,), 0xA5, dtype=torch.uint8, device="cuda")
    parents, tokens = (torch.full((groups * picks + 1,), -99, dtype=torch.int32, device="cuda")
                       for _ in range(2))
    sums = torch.full((groups * picks + 1,), 55.0, device="cuda")
    torch.cuda.synchronize()
    for _ in range(2):
        kvx.kvx_select_beams(ctx, cfg, ptr or logits.data_ptr(), scores.data_ptr(),
                             parents.data_ptr(), tokens.data_ptr(), sums.data_ptr(),
                             work.data_ptr(), logits_stride=stride,
                             done=done.data_ptr() if done is not None else 0, stream=stream)
        torch.cuda.synchronize()
        now = [t.clone() for t in (parents, tokens, sums)]
    assert (work[nbytes:] == 0xA5).all()
    assert int(parents[-1]) == -99 and int(tokens[-1]) == -99 and float(sums[-1]) == 55.0
    kvx.kvx_select_beams(ctx, cfg, ptr or logits.data_ptr(), scores.data_ptr(), parents.data_ptr(),
                         tokens.data_ptr(), sums.data_ptr(), work.data_ptr(), logits_stride=stride,
                         done=done.data_ptr() if done is not None else 0, stream=stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(now, (parents, tokens, sums)))
    return [t[:-1].view(groups, picks).cpu() for t in (parents, tokens, sums)]


def all_sums(logits, scores, done, done_token):
    """[groups][(sum, beam, token)] of every continuation, best first, and sums by (beam, token)."""
    groups, width = scores.shape
    x = logits.double().cpu().view(groups, width, -1).numpy().copy()
    x[~(x < np.inf)] = -np.inf
    so_far = scores.double().cpu().numpy()
    out = []
    for g in range(groups):
        s, b, t = [], [], []
        for w in range(width):
            if not so_far[g, w] > -np.inf:
                continue
            if done is not None and done[g, w]:
                s.append(np.array([so_far[g, w]])), b.append(np.array([w]))
                t.append(np.array([done_token]))
                continue
            row = x[g, w]
            live = np.flatnonzero(row > -np.inf)
            if len(live) == 0:
                continue
            m = row.max()
            s.append(so_far[g, w] + (row[live] - (m + np.log(np.exp(row[live] - m).sum()))))
            b.append(np.full(len(live), w)), t.append(live)
        if s:
            s, b, t = (np.concatenate(v) for v in (s, b, t))
            order = np.lexsort((t, b, -s))
            out.append((s[order], b[order], t[order]))
        else:
            out.append((np.zeros(0), np.zeros(0, int), np.zeros(0, int)))
    return out


def check_selection(got, logits, scores, picks, done=None, done_token=-7):
    parents, tokens, sums = got
    for g, (s, b, t) in enumerate(all_sums(logits, scores, done, done_token)):
        n = min(picks, len(s))
        place = {(int(bb), int(tt)): k for k, (bb, tt) in enumerate(zip(b, t))}
        took = [place[(int(parents[g, k]), int(tokens[g, k]))] for k in range(n)]
        assert len(set(took)) == n
        for k, at in enumerate(took):
            assert abs(s[at] - s[k]) <= CLOSE, (g, k, s[at], s[k])
            if at != k:  # only among sums that are close and not the same beam's
                assert s[at] != s[k] or b[at] != b[k]
            assert abs(float(sums[g, k]) - s[at]) <= CLOSE / 2 + 2.0 ** -24 * abs(s[at])
        assert (parents[g, n:] == 0).all() and (tokens[g, n:] == -1).all()
        assert (sums[g, n:] == -float("inf")).all()


def make(groups, width, vocab, dtype, seed=0, spread=3.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = (torch.randn((groups * width, vocab), device="cuda", generator=g) * spread).to(TORCH[dtype])
    scores = -10.0 * torch.rand((groups, width), device="cuda", generator=g)
    return x, scores


@pytest.mark.parametrize("vocab", [1, 2, 7, 63, 1000, 4095, 4096, 4097, 16385, 32000, 131071])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("groups,width,picks", [(1, 4, 4), (3, 5, 10)])
def test_sizes(ctx, vocab, dtype, groups, width, picks):
    x, s = make(groups, width, vocab, dtype, vocab)
    check_selection(select(ctx, x, s, picks, dtype), x, s, picks)


@pytest.mark.parametrize("groups,width,picks,vocab", [
    (1, 1, 1, 50257), (1, 1, 64, 50257), (1, 32, 64, 20011), (40, 8, 16, 30000), (200, 2, 3, 5000),
    (1, 2, 2, 524000), (2, 32, 32, 200003)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_shapes(ctx, groups, width, picks, vocab, dtype):
    x, s = make(groups, width, vocab, dtype, picks)
    check_selection(select(ctx, x, s, picks, dtype), x, s, picks)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("pad,off", [(0, 1), (3, 0), (5, 3), (8, 2)])
def test_strides_and_alignment(ctx, dtype, pad, off):
    """Rows that begin anywhere; what lies between them is not looked at."""
    groups, width, vocab = 2, 3, 9001
    x, s = make(groups, width, vocab, dtype)
    stride = vocab + pad
    flat = torch.full((off + groups * width * stride,), 30000.0, dtype=TORCH[dtype], device="cuda")
    rows = flat[off:].view(groups * width, stride)
    rows[:, :vocab] = x
    got = select(ctx, flat, s, 6, dtype, stride=stride, vocab=vocab,
                 ptr=flat.data_ptr() + off * flat.element_size())
    check_selection(got, x, s, 6)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("vocab", [5, 4000, 70000])
def test_ties_go_by_beam_and_token(ctx, dtype, vocab):
    """All logits alike, all sums alike; a few values only; two beams with the same logits."""
    s = torch.full((2, 4), -3.0, device="cuda")
    x = torch.full((8, vocab), 1.25, dtype=TORCH[dtype], device="cuda")
    parents, tokens, _ = got = select(ctx, x, s, 9, dtype)
    check_selection(got, x, s, 9)
    want = [(b, t) for b in range(4) for t in range(vocab)][:9]
    assert [(int(a), int(b)) for a, b in zip(parents[0], tokens[0])] == want
    x = torch.randint(-2, 3, (8, vocab), device="cuda").to(TORCH[dtype])
    x[1], x[3] = x[0], x[0]
    for picks in (9, 64):
        got = select(ctx, x, s, picks, dtype)
        check_selection(got, x, s, picks)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("vocab", [40, 20000])
def test_masks_infinities_and_nan(ctx, dtype, vocab):
    x, s = make(3, 4, vocab, dtype, 3)
    lowest = torch.finfo(TORCH[dtype]).min
    x[0] = -float("inf")                         # nothing left
    x[1, : vocab - 2] = -float("inf")            # two tokens left
    x[2, ::2] = lowest
    x[3] = lowest                                # all alike
    x[4, 5] = float("nan")
    x[5, 7] = float("inf")
    x[6] = float("nan")
    x[7, : vocab // 2] = float("inf")
    x[8:] = -float("inf")                        # a group of which nothing is left
    s[1, 0] = -float("inf")
    s[1, 3] = float("nan")
    check_selection(select(ctx, x, s, 8, dtype), x, s, 8)
    # The first step: one beam counts.
    x, s = make(2, 4, vocab, dtype, 4)
    s[:, 0], s[:, 1:] = 0.0, -float("inf")
    check_selection(select(ctx, x, s, 4, dtype), x, s, 4)
    # -0 and 0 are alike.
    x, s = make(1, 1, vocab, dtype, 5)
    x[:] = -1.0
    x[0, 3], x[0, 9], x[0, 20] = 0.0, -0.0, 0.0
    _, tokens, _ = select(ctx, x, s, 3, dtype)
    assert tokens[0].tolist() == [3, 9, 20]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("mask", [-1e6, -1e9, -1e12, "lowest"])
@pytest.mark.parametrize("groups", [1, 4])
def test_mask_values_of_whole_parts(ctx, dtype, mask, groups):
    """Finite mask values everywhere but at a few tokens: whatever of a row a CTA takes, some have
    nothing else.  One beam of each group has nothing but mask values, one the largest of all."""
    vocab = 40000
    value = torch.finfo(TORCH[dtype]).min if mask == "lowest" else mask
    x, s = make(groups, 4, vocab, dtype, 8)
    y = torch.full_like(x, value)
    y[:, 17000:17100] = x[:, 17000:17100]
    y[1::4] = value
    y[3::4, 50] = -value
    check_selection(select(ctx, y, s, 8, dtype), y, s, 8)


@pytest.mark.parametrize("at", [3e4, -3e4, 1e6, -1e6, 3e7, -1e9])
def test_logits_far_from_zero(ctx, at):
    """All logits around `at`.  Near 2^20 the sum's correction is an exponential of its own, 2^-22
    off: within what a beam's sum is compared by, 2^-22 and 2^-24 of its size (about 10)."""
    x, s = make(2, 3, 30000, "fp32", 9)
    x = x.double().add(at).float()
    check_selection(select(ctx, x, s, 6, "fp32"), x, s, 6)


def test_done_beams(ctx):
    x, s = make(4, 5, 3001, "bf16", 6)
    done = torch.zeros((4, 5), dtype=torch.uint8, device="cuda")
    done[0, 1] = done[1, 0] = done[1, 4] = 1
    done[2] = 255
    x[done.view(-1) != 0] = float("nan")         # not read
    got = select(ctx, x, s, 10, "bf16", done=done, done_token=2)
    check_selection(got, x, s, 10, done.cpu().numpy(), 2)


def test_in_place_graph_and_stream(ctx):
    """out_scores is scores; a captured selection gives what an eager one gives, on new logits."""
    x, s0 = make(6, 4, 32000, "bf16", 7)
    want = select(ctx, x, s0, 4, "bf16")
    s = s0.clone()
    st = torch.cuda.Stream()
    cfg = kvx.select_config(6, 4, 32000, 4)
    work = torch.empty(kvx.kvx_select_workspace(ctx, cfg), dtype=torch.uint8, device="cuda")
    p, t = (torch.empty((6, 4), dtype=torch.int32, device="cuda") for _ in range(2))
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        g = torch.cuda.CUDAGraph()
        g.capture_begin()
        kvx.kvx_select_beams(ctx, cfg, x.data_ptr(), s.data_ptr(), p.data_ptr(), t.data_ptr(),
                             s.data_ptr(), work.data_ptr(), stream=st.cuda_stream)
        g.capture_end()
    for _ in range(2):
        s.copy_(s0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.cpu(), want[0]) and torch.equal(t.cpu(), want[1])
        assert torch.equal(s.cpu(), want[2])
        x2, s0 = make(6, 4, 32000, "bf16", 8)
        x.copy_(x2)
        want = select(ctx, x, s0, 4, "bf16")


def test_selection_refusals(ctx):
    x, s = make(1, 2, 100, "bf16")
    out = torch.zeros(64, dtype=torch.int32, device="cuda")
    work = torch.zeros(4096, dtype=torch.uint8, device="cuda")

    def call(cfg=None, logits=None, scores=None, work_at=None, **kw):
        a = out.data_ptr()
        kvx.kvx_select_beams(ctx, cfg or kvx.select_config(1, 2, 100, 2),
                             x.data_ptr() if logits is None else logits,
                             s.data_ptr() if scores is None else scores, kw.pop("parents", a),
                             a + 64, kw.pop("out", a + 128), work.data_ptr() if work_at is None
                             else work_at, **kw)

    for status, kw in [
            (kvx.KVX_ERR_INVALID_ARG, {"cfg": kvx.select_config(0, 2, 100, 2)}),
            (kvx.KVX_ERR_INVALID_ARG, {"cfg": kvx.select_config(1, 33, 100, 2)}),
            (kvx.KVX_ERR_INVALID_ARG, {"cfg": kvx.select_config(1, 2, 0, 2)}),
            (kvx.KVX_ERR_INVALID_ARG, {"cfg": kvx.select_config(1, 2, 524001, 2)}),
            (kvx.KVX_ERR_INVALID_ARG, {"cfg": kvx.select_config(1, 2, 100, 65)}),
            (kvx.KVX_ERR_INVALID_ARG, {"cfg": kvx.select_config(1, 2, 100, 2, "fp8")}),
            (kvx.KVX_ERR_INVALID_ARG, {"logits": 0}), (kvx.KVX_ERR_INVALID_ARG, {"work_at": 0}),
            (kvx.KVX_ERR_INVALID_ARG, {"logits_stride": 99}),
            (kvx.KVX_ERR_ALIGNMENT, {"logits": x.data_ptr() + 1}),
            (kvx.KVX_ERR_ALIGNMENT, {"work_at": work.data_ptr() + 8}),
            (kvx.KVX_ERR_ALIGNMENT, {"parents": out.data_ptr() + 2}),
            (kvx.KVX_ERR_INVALID_ARG, {"cfg": kvx.select_config(1, 2, 100, 4),
                                       "out": s.data_ptr()})]:
        with pytest.raises(kvx.KvxError) as e:
            call(**kw)
        assert e.value.status == status, kw
    call()
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------- reordering

class Beams:
    """Groups of beams over one pool: full pages partly shared, last pages their own."""

    def __init__(self, groups, page, layers=3, kv=2, token_bytes=48, seed=0, spare=2):
        """groups: (width, tokens)."""
        rng = np.random.default_rng(seed)
        self.groups, self.page, self.rng = groups, page, rng
        counts = [-(-n // page) for _, n in groups]
        total = sum(w * c for (w, _), c in zip(groups, counts)) + 5
        self.n_pages = total
        ids = iter(rng.permutation(total).tolist())
        self.refs = [0] * total
        self.tables = []
        for (w, n), c in zip(groups, counts):
            full = n // page
            shared = int(rng.integers(0, full + 1))
            common = [next(ids) for _ in range(shared)]
            rows = [common + [next(ids) for _ in range(c - shared)] for _ in range(w)]
            for row in rows:
                for p in row:
                    self.refs[p] += 1
            self.tables.append(rows)
        self.stride = max(counts + [1]) + spare
        self.dev = torch.full((len(groups), 32, self.stride), -5, dtype=torch.int32, device="cuda")
        for g, rows in enumerate(self.tables):
            for b, row in enumerate(rows):
                if row:
                    self.dev[g, b, :len(row)] = torch.tensor(row, dtype=torch.int32)
        self.dev_refs = torch.tensor(self.refs, dtype=torch.int32, device="cuda")
        self.pool = torch.randint(0, 256, (kv, layers, total, page, token_bytes),
                                  dtype=torch.uint8, device="cuda")
        self.model = self.pool.cpu().numpy().copy()
        self.kvx_pool = kvx.Pool.from_tensor(self.pool, page)
        self.parents = torch.zeros((len(groups), 32), dtype=torch.int32, device="cuda")

    def choose(self):
        for g, (w, _) in enumerate(self.groups):
            self.parents[g, :w] = torch.from_numpy(self.rng.integers(0, w, w).astype(np.int32))

    def array(self):
        return kvx.beams_array([(self.dev[g].data_ptr(), self.stride, self.parents[g].data_ptr(),
                                 w, n) for g, (w, n) in enumerate(self.groups)])

    def step(self, skip=()):
        """The bookkeeping of one call, beam by beam."""
        parents = self.parents.cpu().tolist()
        for g, (w, n) in enumerate(self.groups):
            if g in skip:
                continue
            old, par = [list(r) for r in self.tables[g]], parents[g][:w]
            full, tail = n // self.page, n % self.page
            for row in old:
                for p in row[:full]:
                    self.refs[p] -= 1
            dropped = iter(b for b in range(w) if b not in par)
            first = set()
            for b in range(w):
                new = old[par[b]][:full]
                for p in new:
                    self.refs[p] += 1
                if tail:
                    source = old[par[b]][full]
                    if par[b] in first:
                        target = old[next(dropped)][full]
                        self.model[:, :, target, :tail] = self.model[:, :, source, :tail]
                    else:
                        target = source
                    new = new + [target]
                first.add(par[b])
                self.tables[g][b] = new

    def check(self):
        torch.cuda.synchronize()
        dev = self.dev.cpu()
        for g, rows in enumerate(self.tables):
            for b, row in enumerate(rows):
                assert dev[g, b, :len(row)].tolist() == row, (g, b)
                assert (dev[g, b, len(row):] == -5).all()
            assert (dev[g, len(rows):] == -5).all()
        assert self.dev_refs.cpu().tolist() == self.refs
        assert np.array_equal(self.pool.cpu().numpy(), self.model)

    def run(self, ctx, stream=0):
        torch.cuda.synchronize()
        kvx.kvx_reorder_beams(ctx, self.kvx_pool, self.dev_refs.data_ptr(), self.array(),
                              stream=stream)


@pytest.mark.parametrize("page", [1, 3, 16, 64])
@pytest.mark.parametrize("groups", [
    [(1, 10)], [(4, 1)], [(4, 16)], [(2, 100), (5, 33), (3, 0), (8, 64)], [(32, 70)],
    [(16, 3000), (3, 129 * 16)], [(3, 20)] * 100])
def test_reorder(ctx, page, groups):
    b = Beams(groups, page)
    for _ in range(3):
        b.choose()
        b.run(ctx)
        b.step()
        b.check()
    assert kvx.kvx_get_status(ctx) == 0


@pytest.mark.parametrize("layers,kv,token_bytes", [(1, 1, 16), (40, 2, 256), (5, 2, 2048),
                                                   (61, 1, 1152)])
def test_reorder_pools(ctx, layers, kv, token_bytes):
    b = Beams([(6, 61), (4, 5), (10, 200)], 16, layers, kv, token_bytes)
    for _ in range(2):
        b.choose()
        b.run(ctx)
        b.step()
        b.check()


@pytest.mark.parametrize("parents", [[0, 1, 2, 3], [3, 2, 1, 0], [2, 2, 2, 2], [1, 1, 0, 0],
                                     [3, 3, 3, 0]])
@pytest.mark.parametrize("tokens", [5, 16, 40])
def test_reorder_orders(ctx, parents, tokens):
    b = Beams([(4, tokens)], 16)
    b.parents[0, :4] = torch.tensor(parents, dtype=torch.int32)
    b.run(ctx)
    b.step()
    b.check()


def test_reorder_reports_and_skips(ctx):
    b = Beams([(4, 40), (3, 30), (2, 25)], 16)
    b.choose()
    b.parents[1, 2] = 3                       # not a beam of the group
    b.run(ctx)
    b.step(skip=(1,))
    b.check()
    assert kvx.kvx_get_status(ctx) == kvx.KVX_DEV_BEAM_OUT_OF_RANGE
    b.parents[1, 2] = -1
    b.run(ctx)
    b.step(skip=(1,))
    b.check()
    assert kvx.kvx_get_status(ctx) == kvx.KVX_DEV_BEAM_OUT_OF_RANGE
    # A page id outside the pool, and one that nobody holds, among a dropped beam's full pages.
    b = Beams([(2, 40)], 16, seed=1)
    b.parents[0, :2] = 0
    b.dev[0, 1, 0] = b.n_pages
    b.run(ctx)
    torch.cuda.synchronize()
    assert kvx.kvx_get_status(ctx) & kvx.KVX_DEV_PAGE_OUT_OF_RANGE
    b = Beams([(2, 40)], 16, seed=2)
    b.parents[0, :2] = 0
    free = b.refs.index(0)
    b.dev[0, 1, 0] = free
    b.run(ctx)
    torch.cuda.synchronize()
    assert kvx.kvx_get_status(ctx) == kvx.KVX_DEV_PAGE_NOT_HELD
    assert int(b.dev_refs[free]) == 0


def test_reorder_captured_and_chained(ctx):
    """Replays of a captured call with new parents, and calls right behind one another."""
    b = Beams([(4, 45), (8, 30)], 16, layers=4)
    s = torch.cuda.Stream()
    b.choose()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        g.capture_begin()
        kvx.kvx_reorder_beams(ctx, b.kvx_pool, b.dev_refs.data_ptr(), b.array(),
                              stream=s.cuda_stream)
        g.capture_end()
    for _ in range(3):
        b.choose()
        torch.cuda.synchronize()
        g.replay()
        b.step()
        b.check()
    b.choose()
    torch.cuda.synchronize()
    beams = b.array()
    for _ in range(4):
        kvx.kvx_reorder_beams(ctx, b.kvx_pool, b.dev_refs.data_ptr(), beams, stream=s.cuda_stream)
        b.step()
    b.check()
    assert kvx.kvx_get_status(ctx) == 0
