"""A 4-bit cache for tests: its layout, what its codes stand for, and the nearest ones.

An element is an e2m1 code times its block's e4m3 scale; MAGNITUDES are the codes' values."""
from __future__ import annotations

import numpy as np
import torch

from paged_kv_gather_gb300 import kvx

MAGNITUDES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
CODES = np.concatenate([MAGNITUDES, -MAGNITUDES])
E4M3 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
FINITE = np.sort(E4M3[:127])  # 0 .. 448


def split(raw, heads, dim):
    """Codes [..., heads, dim] (0 .. 15) and scale bytes [..., heads, dim / 16] of token bytes."""
    raw = np.asarray(raw)
    codes = raw[..., :heads * dim // 2]
    both = np.stack([codes & 15, codes >> 4], -1).reshape(*raw.shape[:-1], heads, dim)
    units = raw[..., heads * dim // 2:heads * dim * 9 // 16]
    return both, units.reshape(*raw.shape[:-1], heads, dim // 16)


def values(raw, heads, dim):
    codes, units = split(raw, heads, dim)
    return CODES[codes] * np.repeat(E4M3[units], 16, -1)


def check_stored(raw, x, heads, dim, scale, slack=0.0):
    """The bytes are what the cache should hold of x [tokens, heads, dim] (64 bits).  The stored
    scale is a nearest one to max / (6 scale) and each code a nearest one to x / (stored x scale),
    both up to 2^-19 relative: reciprocals and products in 32 bits are off by a few 2^-24.
    `slack`: by how much x itself may be off, absolutely."""
    codes, units = split(raw, heads, dim)
    b = x.reshape(*x.shape[:-1], dim // 16, 16)
    want = np.minimum(np.abs(b).max(-1) / (6.0 * scale), 448.0)
    stored = E4M3[units]
    off = np.abs(FINITE[:, None] - want.ravel()[None]).min(0).reshape(want.shape)
    assert (np.abs(stored - want) <= off + want * 2.0 ** -19 + slack / scale).all()
    unit = np.repeat(stored, 16, -1) * scale
    t = np.where(unit > 0, x / np.where(unit > 0, unit, 1.0), 0.0).clip(-6, 6)
    off = np.abs(CODES[:, None] - t.ravel()[None]).min(0).reshape(t.shape)
    room = 6 * 2.0 ** -19 + slack / np.where(unit > 0, unit, 1.0)
    assert (np.abs(CODES[codes] - t) <= off + room).all()


class FourCache:
    """A pool of pages in 4 bits with page tables for a batch of requests; every byte that no
    token owns is 0xFF, a scale of NaN.  `values` as tests.cache_common.Cache has them."""

    def __init__(self, tokens, heads, dim, page, layers=2, seed=0, spread=True):
        self.tokens, self.heads, self.dim, self.page, self.kv = tokens, heads, dim, page, "fp4"
        self.token_bytes = kvx.kvx_token_bytes(heads, dim, "fp4")
        rng = np.random.default_rng(seed)
        counts = [-(-n // page) for n in tokens]
        self.n_pages = sum(counts) + 5
        pool = np.full((2, layers, self.n_pages * page, self.token_bytes), 0xFF, np.uint8)
        perm = rng.permutation(self.n_pages).astype(np.int32)
        tables = np.full((len(tokens), max(counts + [1])), -1, np.int32)
        self.values = []
        at, row = 0, heads * dim
        for r, n in enumerate(tokens):
            tables[r, :counts[r]] = perm[at:at + counts[r]]
            at += counts[r]
            raw = np.empty((2, layers, n, row * 9 // 16), np.uint8)
            raw[..., :row // 2] = rng.integers(0, 256, raw[..., :row // 2].shape)
            # Scales from 2^-9 to 448 where they spread, else around 1.
            raw[..., row // 2:] = (rng.integers(1, 127, raw[..., row // 2:].shape) if spread else
                                   rng.integers(0x30, 0x40, raw[..., row // 2:].shape))
            slots = (tables[r, np.arange(n) // page].astype(np.int64) * page + np.arange(n) % page)
            pool[:, :, slots, :row * 9 // 16] = raw
            self.values.append(values(raw, heads, dim))
        self.pool = torch.from_numpy(pool).cuda().view(2, layers, self.n_pages, page, -1)
        self.tables = torch.from_numpy(tables).cuda()
        self.kvx_pool = kvx.Pool.from_tensor(self.pool, page)

    def requests(self):
        return kvx.requests_array([(self.tables[r].data_ptr(), None, n)
                                   for r, n in enumerate(self.tokens)])
