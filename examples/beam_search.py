"""A beam search on a paged KV cache held in 4 bits, without reading anything back on the way.

A prompt is prefilled, forked into beams (full pages shared, the last one copied), and every step
then rotates and appends the new tokens' K, attends over the pages, selects the best continuations
over beams and vocabulary, and reorders the beams' pages after them.  The step's launches take
everything that depends on the search (parents, tokens, sums, tables) from device memory.

The projections are stand-ins (fixed random matrices); every operator on the cache is the
library's.  The hypotheses that survive are then decoded again from their tokens, on pages that
nobody shares or reorders: the caches agree to the last byte and the hidden states to the last bit.

    python examples/beam_search.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from paged_kv_gather_gb300 import kvx  # noqa: E402

LAYERS, HEADS, GROUP, DIM, PAGE, VOCAB = 2, 4, 2, 128, 16, 500
QUERIES = HEADS * GROUP
WIDTH = QUERIES * DIM
TOKEN_BYTES = kvx.kvx_token_bytes(HEADS, DIM, "fp4")
K_SCALE, V_SCALE = 0.02, 0.02


class Model:
    """Random projections into q, k and v, a mixing of the attention's output, and logits."""

    def __init__(self, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def matrix(n, m, scale=1.0):
            return (torch.randn((n, m), device="cuda", generator=g) * scale / n ** 0.5).bfloat16()

        self.embed = torch.randn((VOCAB, WIDTH), device="cuda", generator=g).bfloat16()
        self.qkv = [matrix(WIDTH, WIDTH + 2 * HEADS * DIM) for _ in range(LAYERS)]
        self.mix = [matrix(WIDTH, WIDTH) for _ in range(LAYERS)]
        self.logits = matrix(WIDTH, VOCAB, 2.0)
        self.freqs = torch.exp(torch.arange(DIM // 2, device="cuda") * (-2.0 / DIM * 9.21)).float()


def rows(x, w):
    """x @ w one row at a time: what a row gives does not depend on its neighbours."""
    return torch.cat([r[None] @ w for r in x])


class Engine:
    """One pool of 4-bit pages with its counts, and the tables of up to `beams` beams."""

    def __init__(self, model, beams, num_pages=512, table_pages=64):
        self.model, self.beams = model, beams
        self.ctx = kvx.kvx_create(0)
        self.pages = torch.zeros((2, LAYERS, num_pages, PAGE, TOKEN_BYTES), dtype=torch.uint8,
                                 device="cuda")
        self.pool = kvx.Pool.from_tensor(self.pages, PAGE)
        self.refs = torch.zeros(num_pages, dtype=torch.int32, device="cuda")
        self.tables = torch.full((beams, table_pages), -1, dtype=torch.int32, device="cuda")
        self.stream = torch.cuda.current_stream().cuda_stream
        self.rope = kvx.rope_config(model.freqs.data_ptr(), DIM)
        self.plan = None

    def close(self):
        if self.plan:
            kvx.kvx_attn_plan_destroy(self.plan)
        kvx.kvx_destroy(self.ctx)

    def fork(self, entries):
        """entries: (parent table or None, child table, shared tokens, room in tokens)."""
        kvx.kvx_fork_pages(self.ctx, self.pool, self.refs.data_ptr(), kvx.forks_array(
            [(p.data_ptr() if p is not None else 0, c.data_ptr(), s, t, False)
             for p, c, s, t in entries]), stream=self.stream)

    def step(self, tables, tokens, new, ids):
        """Run the new tokens `ids` (packed) of requests of `tokens` tokens with them; returns
        their hidden states."""
        reqs = kvx.requests_array([(t.data_ptr(), None, n) for t, n in zip(tables, tokens)])
        if self.plan is None:
            cfg = kvx.attn_config(QUERIES, HEADS, DIM, "bf16", "fp4")
            # Room for every beam: the first batch is filled up with requests without tokens.
            empty = [(0, None, 0)] * (self.beams - len(tables))
            first = kvx.requests_array([(t.data_ptr(), None, n)
                                        for t, n in zip(tables, tokens)] + empty)
            self.plan = kvx.kvx_attn_plan_create(self.ctx, self.pool, first,
                                                 new + [0] * len(empty), cfg, stream=self.stream)
        else:
            kvx.kvx_attn_plan_update(self.plan, reqs, new, stream=self.stream)
        x = self.model.embed[ids]
        for layer in range(LAYERS):
            qkv = rows(x, self.model.qkv[layer])
            q, k, v = qkv.split([WIDTH, HEADS * DIM, HEADS * DIM], dim=1)
            turned, out = torch.empty_like(x), torch.empty_like(x)
            kvx.kvx_append_rotated(self.plan, layer, self.rope, k.data_ptr(), v.data_ptr(),
                                   q=q.data_ptr(), q_out=turned.data_ptr(),
                                   k_stride=qkv.stride(0), v_stride=qkv.stride(0),
                                   q_stride=qkv.stride(0), k_scale=K_SCALE, v_scale=V_SCALE,
                                   stream=self.stream)
            kvx.kvx_attend(self.plan, layer, turned.data_ptr(), out.data_ptr(), k_scale=K_SCALE,
                           v_scale=V_SCALE, stream=self.stream)
            x = x + rows(out, self.model.mix[layer])
        return x

    def grow(self, tables, tokens, room):
        self.fork([(t, t, n, room) for t, n in zip(tables, tokens)])

    def prefill(self, ids, chunk=32):
        """The prompt in table 0; returns its last hidden state."""
        for at in range(0, len(ids), chunk):
            n = min(at + chunk, len(ids))
            self.grow(self.tables[:1], [at], n)
            x = self.step([self.tables[0]], [n], [n - at], ids[at:n])
        return x[-1:]

    def spread(self, tokens):
        """Fork the prompt in table 0 into all beams, beam 0 among them."""
        self.fork([(self.tables[0], t, tokens, tokens) for t in self.tables[1:]])

    def decode(self, n, ids):
        """One new token for every beam, n tokens with it."""
        self.grow(list(self.tables), [n - 1] * self.beams, n)
        return self.step(list(self.tables), [n] * self.beams, [1] * self.beams, ids)

    def cached(self, n):
        """The bytes of every beam's tokens, [beams, 2, LAYERS, n, bytes in use]."""
        j = torch.arange(n, device="cuda")
        slots = self.tables[:, j // PAGE].long() * PAGE + j % PAGE
        flat = self.pages.view(2, LAYERS, -1, TOKEN_BYTES)
        return torch.stack([flat[:, :, s, :HEADS * DIM * 9 // 16] for s in slots])


def search(model, prompt, beams, steps):
    """Histories [beams, steps] on the device, their sums, and the engine with their cache."""
    e = Engine(model, beams)
    cfg = kvx.select_config(1, beams, VOCAB, beams)
    work = torch.empty(kvx.kvx_select_workspace(e.ctx, cfg), dtype=torch.uint8, device="cuda")
    x = e.prefill(prompt).expand(beams, -1)
    e.spread(len(prompt))
    # The first step continues one beam: the others are copies of it.
    sums = torch.full((beams,), -float("inf"), device="cuda")
    sums[0] = 0.0
    parents, ids = (torch.zeros(beams, dtype=torch.int32, device="cuda") for _ in range(2))
    said = torch.zeros((beams, 0), dtype=torch.int32, device="cuda")
    n = len(prompt)
    for _ in range(steps):
        logits = rows(x, model.logits)
        kvx.kvx_select_beams(e.ctx, cfg, logits.data_ptr(), sums.data_ptr(), parents.data_ptr(),
                             ids.data_ptr(), sums.data_ptr(), work.data_ptr(), stream=e.stream)
        kvx.kvx_reorder_beams(e.ctx, e.pool, e.refs.data_ptr(), kvx.beams_array(
            [(e.tables.data_ptr(), e.tables.stride(0), parents.data_ptr(), beams, n)]),
            stream=e.stream)
        said = torch.cat([said[parents.long()], ids[:, None]], 1)
        n += 1
        x = e.decode(n, ids.long())
    return e, said, sums, x, n


def run(prompt_tokens=45, beams=4, steps=40):
    model = Model()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    prompt = torch.randint(0, VOCAB, (prompt_tokens,), device="cuda", generator=g)
    e, said, sums, x, n = search(model, prompt, beams, steps)
    found, live = e.cached(n), int((e.refs > 0).sum())
    held = int(e.refs.sum()) == beams * -(-n // PAGE)
    flags = kvx.kvx_get_status(e.ctx, e.stream)

    # The same hypotheses from their tokens alone.
    again = Engine(model, beams)
    again.prefill(prompt)
    again.spread(prompt_tokens)
    for step in range(steps):
        y = again.decode(prompt_tokens + step + 1, said[:, step].long())
    same = torch.equal(found, again.cached(n)) and torch.equal(x, y)
    flags |= kvx.kvx_get_status(again.ctx, again.stream)
    e.close()
    again.close()
    return {"tokens": n, "live_pages": live, "counts_add_up": held, "status": flags,
            "identical": same, "distinct": len({tuple(s) for s in said.tolist()}),
            "falling": bool((sums[:-1] >= sums[1:]).all())}


if __name__ == "__main__":
    r = run()
    print(f"{r['distinct']} hypotheses of {r['tokens']} tokens on {r['live_pages']} live pages; "
          f"status {r['status']}; caches and hidden states "
          + ("identical to" if r["identical"] else "DIFFERENT from")
          + " those of the same tokens decoded without sharing or reordering")
    sys.exit(0 if r["identical"] and r["counts_add_up"] and r["status"] == 0 else 1)
