"""Plain references and inputs for the operators that work on a paged KV cache in place.

attend_reference is the definition of kvx_attend in 64-bit numpy, one query head and one
request at a time; pages_model is the bookkeeping of fork, free and compact on Python lists.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from paged_kv_gather_gb300 import kvx

TORCH = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
ITEM = {"fp16": 2, "bf16": 2, "fp8": 1}
ROUNDOFF = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}  # half a unit in the last place, relative


class Cache:
    """A pool of typed K and V pages with page tables for a batch of requests.

    Every byte of the pool that no token of a request owns is NaN, and so is every page no
    table names, unless `spare` gives a fill."""

    def __init__(self, tokens, heads, dim, page, kv="bf16", layers=2, seed=0, scale=1.0,
                 pages=None, first_page=0):
        self.tokens, self.heads, self.dim, self.page, self.kv = tokens, heads, dim, page, kv
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        counts = [-(-n // page) for n in tokens]
        self.n_pages = pages or sum(counts) + 5
        dtype = TORCH[kv]
        self.pool = torch.empty((2, layers, self.n_pages, page, heads, dim), dtype=dtype,
                                device="cuda")
        if pages is None:
            self.pool.view(torch.uint8).fill_(0x7F if kv == "fp8" else 0xFF)  # NaN
        perm = torch.randperm(self.n_pages - first_page, device="cuda", generator=g)
        perm = (perm + first_page).to(torch.int32)
        self.width = max(counts + [1])
        self.tables = torch.full((len(tokens), self.width), -1, dtype=torch.int32, device="cuda")
        self.values = []  # per request [2, layers, tokens, heads, dim] float64
        at = 0
        for r, n in enumerate(tokens):
            table = perm[at:at + counts[r]]
            at += counts[r]
            self.tables[r, :counts[r]] = table
            x = (torch.randn((2, layers, n, heads, dim), device="cuda", generator=g)
                 * scale).to(torch.bfloat16).to(dtype)
            slots = (table.long()[torch.arange(n, device="cuda") // page] * page
                     + torch.arange(n, device="cuda") % page)
            # Bytes: 8-bit floats have no indexed assignment.
            flat = self.pool.view(torch.uint8).view(2, layers, self.n_pages * page, -1)
            if n:
                flat[:, :, slots] = x.view(torch.uint8).view(2, layers, n, -1)
            self.values.append(x.double().cpu().numpy())
        torch.cuda.synchronize()
        self.kvx_pool = kvx.Pool.from_tensor(
            self.pool.view(torch.uint8).view(2, layers, self.n_pages, page,
                                             heads * dim * ITEM[kv]), page)

    def requests(self):
        return kvx.requests_array([(self.tables[r].data_ptr(), None, n)
                                   for r, n in enumerate(self.tokens)])


def visible(n, n_new, window, prefix):
    """[n_new, n] which keys each row sees."""
    j = np.arange(n)[None]
    p = np.arange(n - n_new, n)[:, None]
    seen = j <= p
    if window:
        seen &= p - j < window
    return seen | (j < prefix)


def attend_reference(q, k, v, n_new, group, scale, window=0, prefix=0, softcap=0.0, slopes=None):
    """q [n_new, heads, D], k and v [n, kv_heads, D], all float64.  Returns out, lse, and what
    a tolerance is made of: sum_j p_j |v_j| per output and the largest sum_d |q_d k_d| * scale
    per row."""
    n = k.shape[0]
    seen = visible(n, n_new, window, prefix)
    away = np.abs(np.arange(n - n_new, n)[:, None] - np.arange(n)[None])
    out, spread = np.empty_like(q), np.empty_like(q)
    lse, reach = np.empty(q.shape[:2]), np.empty(q.shape[:2])
    for h in range(q.shape[1]):
        key, val = k[:, h // group], v[:, h // group]
        s = q[:, h] @ key.T * scale
        reach[:, h] = (np.abs(q[:, h]) @ np.abs(key).T * abs(scale)).max(1)
        if softcap:
            s = softcap * np.tanh(s / softcap)
        if slopes is not None:
            s = s - slopes[h] * away
        s[~seen] = -math.inf
        m = s.max(1, keepdims=True)
        p = np.exp(s - m)
        l = p.sum(1, keepdims=True)
        out[:, h] = p @ val / l
        spread[:, h] = p @ np.abs(val) / l
        lse[:, h] = (m + np.log(l))[:, 0]
    return out, lse, spread, reach


class PagesModel:
    """Counts, tables and page contents of fork, free and compact, one entry at a time."""

    def __init__(self, refs, page_size):
        self.refs = list(refs)
        self.page_size = page_size
        self.moves = []     # (from page, to page, tokens) in order

    def fork(self, parent, shared, total, copy=False, grow=False):
        """Child table of one entry; fresh pages come from self.fresh (see fork_batch)."""
        P = self.page_size
        held = -(-shared // P)
        full = held if grow else 0 if copy else shared // P
        child = []
        for j in range(-(-total // P)):
            if j < full:
                if not grow:
                    self.refs[parent[j]] += 1
                child.append(parent[j])
            else:
                p = self.fresh.pop(0)
                if j < held:
                    self.moves.append((parent[j], p, min(P, shared - j * P)))
                child.append(p)
        return child

    def fork_batch(self, entries):
        """entries: (parent, shared, total, copy, grow).  None when pages run out."""
        P = self.page_size
        need = sum(-(-t // P) - (-(-s // P) if g else 0 if c else s // P)
                   for _, s, t, c, g in entries)
        free = [p for p, n in enumerate(self.refs) if n == 0]
        if len(free) < need:
            return None
        self.fresh = free[:need]
        taken = list(self.fresh)
        out = [self.fork(*e) for e in entries]
        for p in taken:
            self.refs[p] = 1
        return out

    def free(self, table):
        for p in table:
            if self.refs[p] > 0:
                self.refs[p] -= 1

    def compact(self, tables):
        live = [p for p, n in enumerate(self.refs) if n > 0]
        n = len(live)
        holes = [p for p in range(n) if self.refs[p] == 0]
        late = [p for p in live if p >= n]
        remap = {p: p for p in live if p < n}
        for a, b in zip(late, holes):
            remap[a] = b
            self.moves.append((a, b, self.page_size))
            self.refs[b], self.refs[a] = self.refs[a], 0
        return n, remap, [[remap[p] for p in t] for t in tables]
