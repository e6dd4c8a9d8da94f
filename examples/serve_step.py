"""A serving engine's life of one prompt, on a paged KV cache that never leaves its pages.

1. A prompt is prefilled in chunks: each layer appends the chunk's K and V to the request's
   pages and attends over everything so far.
2. The prompt is forked into several continuations: full pages are shared, the partly filled
   last page is copied.
3. The continuations decode: their tables grow page by page, each step appends one token and
   attends.
4. Some are given up, the pool is compacted, and the others decode on.
5. One is evicted to host memory and brought back into fresh pages.

The projections are stand-ins (fixed random matrices); every operator on the cache is the
library's.  The same batches run once more with a prefill of its own for every continuation and
nothing shared, freed, compacted or evicted: the hidden states agree to the last bit, because
which page holds a token never enters the arithmetic.

    python examples/serve_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from paged_kv_gather_gb300 import kvx  # noqa: E402
from paged_kv_gather_gb300 import workloads as wl  # noqa: E402

LAYERS, HEADS, GROUP, DIM, PAGE = 3, 2, 4, 128, 16
WIDTH = HEADS * GROUP * DIM
TOKEN_BYTES = HEADS * DIM * 2


class Model:
    """Random projections into q, k and v, and a mixing of the attention's output."""

    def __init__(self, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def matrix(n, m):
            return (torch.randn((n, m), device="cuda", generator=g) / n ** 0.5).bfloat16()

        self.embed = torch.randn((64, WIDTH), device="cuda", generator=g).bfloat16()
        self.qkv = [matrix(WIDTH, WIDTH + 2 * HEADS * DIM) for _ in range(LAYERS)]
        self.mix = [matrix(WIDTH, WIDTH) for _ in range(LAYERS)]


def rows(x, w):
    """x @ w one row at a time: what a row gives does not depend on its neighbours."""
    return torch.cat([r[None] @ w for r in x])


class Engine:
    """One pool of pages with its counts, and the calls of a step."""

    def __init__(self, model, num_pages=256):
        self.model, self.num_pages = model, num_pages
        self.ctx = kvx.kvx_create(0)
        self.pages = torch.zeros((2, LAYERS, num_pages, PAGE, TOKEN_BYTES), dtype=torch.uint8,
                                 device="cuda")
        self.pool = kvx.Pool.from_tensor(self.pages, PAGE)
        self.refs = torch.zeros(num_pages, dtype=torch.int32, device="cuda")
        self.stream = torch.cuda.current_stream().cuda_stream
        self.plan, self.plan_size = None, 0

    def close(self):
        if self.plan:
            kvx.kvx_attn_plan_destroy(self.plan)
        kvx.kvx_destroy(self.ctx)

    def table(self):
        return torch.full((self.num_pages,), -1, dtype=torch.int32, device="cuda")

    def fork(self, entries):
        """entries: (parent table or None, child table, shared tokens, room in tokens)."""
        kvx.kvx_fork_pages(self.ctx, self.pool, self.refs.data_ptr(), kvx.forks_array(
            [(p.data_ptr() if p is not None else 0, c.data_ptr(), s, t, False)
             for p, c, s, t in entries]), stream=self.stream)

    def grow(self, tables, tokens, room):
        """Room for `room` tokens in requests of `tokens`."""
        self.fork([(t, t, n, r) for t, n, r in zip(tables, tokens, room)])

    def free(self, tables, tokens):
        kvx.kvx_free_pages(self.ctx, self.pool, self.refs.data_ptr(), kvx.tables_array(
            [(t.data_ptr(), -(-n // PAGE)) for t, n in zip(tables, tokens)]), stream=self.stream)

    def compact(self, tables, tokens):
        n_live = torch.zeros(1, dtype=torch.int32, device="cuda")
        kvx.kvx_compact_pages(self.ctx, self.pool, self.refs.data_ptr(), kvx.tables_array(
            [(t.data_ptr(), -(-n // PAGE)) for t, n in zip(tables, tokens)]),
            n_live=n_live.data_ptr(), stream=self.stream)
        return n_live

    def step(self, tables, tokens, new, ids):
        """Run the new tokens `ids` (packed) of every request, whose lengths are `tokens` with
        them; returns their hidden states."""
        reqs = kvx.requests_array([(t.data_ptr(), None, n) for t, n in zip(tables, tokens)])
        if self.plan is None or len(tables) > self.plan_size:
            if self.plan:
                kvx.kvx_attn_plan_destroy(self.plan)
            self.plan_size = len(tables)
            self.plan = kvx.kvx_attn_plan_create(
                self.ctx, self.pool, reqs, new, kvx.attn_config(HEADS * GROUP, HEADS, DIM),
                stream=self.stream)
        else:
            kvx.kvx_attn_plan_update(self.plan, reqs, new, stream=self.stream)
        x = self.model.embed[ids]
        for layer in range(LAYERS):
            qkv = rows(x, self.model.qkv[layer])
            q, k, v = qkv.split([WIDTH, HEADS * DIM, HEADS * DIM], dim=1)
            kvx.kvx_append_tokens(self.plan, layer, k.data_ptr(), v.data_ptr(), qkv.stride(0),
                                  qkv.stride(0), stream=self.stream)
            out = torch.empty_like(x)
            kvx.kvx_attend(self.plan, layer, q.data_ptr(), out.data_ptr(), qkv.stride(0),
                           stream=self.stream)
            x = x + rows(out, self.model.mix[layer])
        return x

    def prefill(self, table, ids, chunk):
        for at in range(0, len(ids), chunk):
            n = min(at + chunk, len(ids))
            self.grow([table], [at], [n])
            x = self.step([table], [n], [n - at], ids[at:n])
        return x[-1:]

    def decode(self, tables, tokens, ids):
        """One new token for each request; `tokens` counts them in."""
        self.grow(tables, [n - 1 for n in tokens], tokens)
        return self.step(tables, tokens, [1] * len(tables), ids)

    def evict(self, table, tokens):
        """Store a request's pages in host memory and free them."""
        shape = wl.KVShape(LAYERS, 2, HEADS, DIM, "bf16", PAGE, self.num_pages)
        chunks = wl.split_tokens(0, 0, tokens, 64, 0, LAYERS, wl.LAYER_MAJOR)
        wl.place_chunks(chunks, shape)
        host = kvx.HostBuffer(wl._arena_bytes(chunks, shape))
        kvx.kvx_store_chunks(self.ctx, self.pool, kvx.requests_array(
            [(table.data_ptr(), None, tokens)]), kvx.chunks_array(chunks, host.ptr),
            stream=self.stream)
        self.free([table], [tokens])
        return host, chunks

    def restore(self, table, tokens, kept):
        host, chunks = kept
        self.grow([table], [0], [tokens])
        kvx.kvx_load_chunks(self.ctx, self.pool, kvx.requests_array(
            [(table.data_ptr(), None, tokens)]), kvx.chunks_array(chunks, host.ptr),
            stream=self.stream)
        torch.cuda.synchronize()
        host.close()

    def status(self):
        return kvx.kvx_get_status(self.ctx, self.stream)


def run(prompt_tokens=77, steps=12, children=4):
    model = Model()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    prompt = torch.randint(0, 64, (prompt_tokens,), device="cuda", generator=g)
    said = torch.randint(0, 64, (3 * steps, children), device="cuda", generator=g)

    # The whole life in one pool.
    e = Engine(model)
    parent = e.table()
    e.prefill(parent, prompt, 32)
    tables = [e.table() for _ in range(children)]
    e.fork([(parent, t, prompt_tokens, prompt_tokens) for t in tables])
    e.free([parent], [prompt_tokens])
    alive, n = list(range(children)), prompt_tokens
    last = {}
    for step in range(3 * steps):
        if step == steps:                       # the first half is given up
            gone = alive[:children // 2]
            e.free([tables[c] for c in gone], [n] * len(gone))
            alive = alive[children // 2:]
            e.compact([tables[c] for c in alive], [n] * len(alive))
        if step == 2 * steps:                   # one leaves for host memory and comes back
            kept = e.evict(tables[alive[0]], n)
            e.restore(tables[alive[0]], n, kept)
        n += 1
        x = e.decode([tables[c] for c in alive], [n] * len(alive), said[step, alive])
        last = {c: x[i] for i, c in enumerate(alive)}
    live_pages = int((e.refs > 0).sum())
    flags = e.status()
    e.close()

    # The same batches on pages that nobody shares or moves.
    e = Engine(model, 4 * 256)
    tables = [e.table() for _ in range(children)]
    for t in tables:
        e.prefill(t, prompt, 32)
    alive, n, same = list(range(children)), prompt_tokens, True
    for step in range(3 * steps):
        if step == steps:
            alive = alive[children // 2:]
        n += 1
        x = e.decode([tables[c] for c in alive], [n] * len(alive), said[step, alive])
    for i, c in enumerate(alive):
        same &= torch.equal(x[i], last[c])
    flags |= e.status()
    e.close()
    return {"survivors": len(alive), "tokens": n, "live_pages": live_pages, "status": flags,
            "identical": same}


if __name__ == "__main__":
    r = run()
    print(f"{r['survivors']} continuations of {r['tokens']} tokens on {r['live_pages']} live pages; "
          f"status {r['status']}; "
          + ("identical to" if r["identical"] else "DIFFERENT from")
          + " the same steps on pages of their own")
    sys.exit(0 if r["identical"] and r["status"] == 0 else 1)
