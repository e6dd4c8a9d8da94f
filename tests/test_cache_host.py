"""Refusals of page upkeep and attention that need no GPU: the host checks through the C ABI,
and the new structs' layout as a C compiler sees it."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from paged_kv_gather_gb300.build import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
build()
from paged_kv_gather_gb300 import kvx  # noqa: E402

A = 1 << 40  # an aligned address that nothing dereferences
INV, ALIGN, OK = kvx.KVX_ERR_INVALID_ARG, kvx.KVX_ERR_ALIGNMENT, kvx.KVX_OK


def pool(page=16, pages=64, token_bytes=2 * 64 * 2, kv=2, layers=2):
    return kvx.Pool(layers, kv, page, pages, token_bytes, [A] * layers, [A] * layers)


def forks(*entries):
    return kvx.forks_array(entries)


@pytest.mark.parametrize("entry,status", [
    ((A, A + 4096, 100, 120, 0), OK),
    ((A, A + 4096, 100, 120, 1), OK),
    ((0, A, 0, 120, 0), OK),
    ((0, 0, 0, 0, 0), OK),
    ((A, A, 100, 120, 0), OK),
    ((A, A, 100, 120, 1), INV),
    ((A, A + 4096, -1, 120, 0), INV),
    ((A, A + 4096, 100, 99, 0), INV),
    ((0, A + 4096, 100, 120, 0), INV),
    ((A, 0, 100, 120, 0), INV),
    ((A, A + 4096, 100, 16 * 64 + 1, 0), INV),
    ((A, A + 4096, 100, 16 * 64, 0), OK),
    ((A + 2, A + 4096, 100, 120, 0), ALIGN),
    ((A, A + 4097, 100, 120, 0), ALIGN),
    ((A, A + 4096, 100, 120, 2), INV),
])
def test_fork_entries(entry, status):
    f = forks(entry[:4] + (0,))
    f[0]["copy"] = entry[4]
    st, msg = kvx.kvx_upkeep_validate(pool(), A, f)
    assert st == status and bool(msg) == (status != OK)


@pytest.mark.parametrize("entries,status", [
    ([(A, A + 4096, 100, 120, 0), (A, A + 8192, 100, 120, 0)], OK),        # one parent, twice
    ([(A, A + 4096, 100, 120, 0), (A, A + 4096, 100, 120, 0)], kvx.KVX_ERR_OVERLAP),
    ([(A, A + 4096, 100, 120, 0), (A + 4096, A + 8192, 100, 120, 0)], kvx.KVX_ERR_OVERLAP),
    ([(A, A + 4096, 100, 120, 0), (A + 512, A + 4096 + 28, 100, 120, 0)], kvx.KVX_ERR_OVERLAP),
    ([(A, A + 4096, 100, 128, 0), (A + 512, A + 4096 + 32, 100, 120, 0)], OK),  # side by side
    ([(A, A, 100, 120, 0), (A, A + 4096, 100, 120, 0)], kvx.KVX_ERR_OVERLAP),
])
def test_fork_tables_that_meet(entries, status):
    assert kvx.kvx_upkeep_validate(pool(), A, forks(*entries), level=2)[0] == status
    assert kvx.kvx_upkeep_validate(pool(), A, forks(*entries), level=1)[0] == OK


def test_upkeep_arguments():
    t = kvx.tables_array([(A, 10), (0, 0)])
    assert kvx.kvx_upkeep_validate(pool(), A, tables=t)[0] == OK
    assert kvx.kvx_upkeep_validate(pool(), 0, tables=t)[0] == INV
    assert kvx.kvx_upkeep_validate(pool(), A + 2, tables=t)[0] == INV
    assert kvx.kvx_upkeep_validate(pool(), A, tables=kvx.tables_array([(0, 1)]))[0] == INV
    assert kvx.kvx_upkeep_validate(pool(), A, tables=kvx.tables_array([(A, -1)]))[0] == INV
    assert kvx.kvx_upkeep_validate(pool(), A, tables=kvx.tables_array([(A + 1, 1)]))[0] == ALIGN
    twice = kvx.tables_array([(A, 10), (A + 36, 10)])
    assert kvx.kvx_upkeep_validate(pool(), A, tables=twice, level=2)[0] == kvx.KVX_ERR_OVERLAP
    big = pool(pages=kvx.KVX_MAX_UPKEEP_PAGES + 1)
    assert kvx.kvx_upkeep_validate(big, A, tables=t)[0] == kvx.KVX_ERR_CAPACITY
    assert kvx.kvx_upkeep_validate(pool(pages=kvx.KVX_MAX_UPKEEP_PAGES), A, tables=t)[0] == OK
    assert kvx.kvx_upkeep_validate(pool(token_bytes=24), A, tables=t)[0] == ALIGN
    assert kvx.kvx_upkeep_validate(pool(kv=1), A, tables=t)[0] == OK


def attn(n_tokens=(100, 50), n_new=(1, 50), prefix=None, p=None, table=A, level=1, host=None,
         **cfg):
    c = dict(q_heads=8, kv_heads=2, head_dim=64, dtype="bf16")
    c.update(cfg)
    reqs = kvx.requests_array([(table, host, n) for n in n_tokens])
    return kvx.kvx_attn_validate(p or pool(), reqs, n_new, kvx.attn_config(**c), prefix, level)


@pytest.mark.parametrize("kw,status", [
    ({}, OK),
    ({"n_new": (0, 0), "table": 0}, OK),
    ({"n_tokens": (0, 0), "n_new": (0, 0), "table": 0}, OK),
    ({"n_new": (101, 1)}, INV),
    ({"n_new": (-1, 1)}, INV),
    ({"n_tokens": (-1, 5), "n_new": (0, 1)}, INV),
    ({"prefix": (100, 0)}, OK),
    ({"prefix": (101, 0)}, INV),
    ({"prefix": (-1, 0)}, INV),
    ({"table": 0}, INV),
    ({"table": A + 2}, ALIGN),
    ({"q_heads": 7}, INV),
    ({"q_heads": 0}, INV),
    ({"kv_heads": 0}, INV),
    ({"kv_heads": 4, "p": None}, INV),             # token_bytes says 2 heads of 64
    ({"head_dim": 96}, INV),
    ({"dtype": "fp8"}, INV),
    ({"dtype": "fp16"}, OK),
    ({"dtype": "fp16", "kv_dtype": "bf16"}, INV),
    ({"kv_dtype": "fp8"}, INV),                    # half the bytes a token
    ({"kv_dtype": "fp8", "p": "fp8"}, OK),
    ({"p": "latent"}, INV),
    ({"window": -1}, INV),
    ({"softcap": -1.0}, INV),
    ({"softcap": float("inf")}, INV),
    ({"softcap": float("nan")}, INV),
    ({"scale": float("nan")}, INV),
    ({"slopes": A + 2}, ALIGN),
    ({"n_tokens": (2 ** 31 - 1,) * 2, "n_new": (2 ** 27, 2 ** 27)}, kvx.KVX_ERR_CAPACITY),
    ({"n_tokens": (2 ** 30,) * 2, "n_new": (2 ** 27, 2 ** 27)}, kvx.KVX_ERR_CAPACITY),
    ({"n_tokens": (2 ** 30 + 1, 1), "n_new": (1, 1)}, kvx.KVX_ERR_CAPACITY),
    ({"n_tokens": (2 ** 30, 1), "n_new": (1, 1), "window": 2 ** 31 - 1}, OK),
])
def test_attention_arguments(kw, status):
    kw = dict(kw)
    kw["p"] = {"fp8": pool(token_bytes=128), "latent": pool(kv=1)}.get(kw.get("p"))
    st, msg = attn(**kw)
    assert st == status and bool(msg) == (status != OK)


def test_attention_pages_that_a_row_sees():
    """Level 2 checks the page ids of what some row sees, and no others."""
    table = np.array([-1, 3, 99, 5, 6, 7, 8], np.int32)
    kw = dict(n_tokens=(100,), n_new=(4,), host=table, level=2)
    assert attn(**kw)[0] == kvx.KVX_ERR_PAGE_OUT_OF_RANGE
    assert attn(window=49, **kw)[0] == OK               # rows 96..99 see 48 and later
    assert attn(window=50, **kw)[0] == kvx.KVX_ERR_PAGE_OUT_OF_RANGE
    assert attn(window=49, prefix=(1,), **kw)[0] == kvx.KVX_ERR_PAGE_OUT_OF_RANGE


def test_struct_layouts(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = (kvx.kvx_table, kvx.kvx_fork, kvx.kvx_attn_cfg)
    lines = []
    for s in structs:
        lines.append(f'printf("%zu\\n", sizeof({s.__name__}));')
        lines += [f'printf("%zu\\n", offsetof({s.__name__}, {n}));' for n, _ in s._fields_]
    src = tmp_path / "t.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"kvx.h\"\n"
                   "int main(void) {\n" + "\n".join(lines) + "\nreturn 0; }\n")
    exe = str(tmp_path / "t")
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I",
                    os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], check=True, capture_output=True,
                                          text=True).stdout.split()]
    want = []
    for s in structs:
        want += [ctypes.sizeof(s)] + [getattr(s, n).offset for n, _ in s._fields_]
    assert got == want
