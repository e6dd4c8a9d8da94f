"""Refusals that need no GPU: 4-bit caches in the attention's checks, groups of beams; and the new
structs' layout as a C compiler sees it."""
import ctypes
import os
import shutil
import subprocess

import pytest

from paged_kv_gather_gb300.build import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
build()
from paged_kv_gather_gb300 import kvx  # noqa: E402

A = 1 << 40  # an aligned address that nothing dereferences
INV, ALIGN, OK = kvx.KVX_ERR_INVALID_ARG, kvx.KVX_ERR_ALIGNMENT, kvx.KVX_OK


def pool(page=16, pages=64, token_bytes=288, kv=2, layers=2):
    return kvx.Pool(layers, kv, page, pages, token_bytes, [A] * layers, [A] * layers)


@pytest.mark.parametrize("heads,dim,dtype,want", [
    (4, 128, "fp4", 288), (1, 128, "fp4", 80), (8, 64, "fp4", 288), (1, 64, "fp4", 48),
    (3, 64, "fp4", 112), (4, 128, "fp8", 512), (4, 128, "bf16", 1024), (4, 64, "fp16", 512),
    (0, 128, "fp4", 0), (4, 120, "fp4", 0), (4, 128, "fp32", 0)])
def test_token_bytes(heads, dim, dtype, want):
    assert kvx.kvx_token_bytes(heads, dim, dtype) == want


@pytest.mark.parametrize("token_bytes,heads,dim,dtype,kv,status", [
    (288, 4, 128, "bf16", "fp4", OK), (288, 4, 128, "fp16", "fp4", OK),
    (256, 4, 128, "bf16", "fp4", INV), (288, 8, 64, "bf16", "fp4", OK),
    (288, 4, 128, "fp4", "fp4", INV), (1024, 4, 128, "bf16", "fp32", INV),
    (2048, 4, 128, "fp32", "fp32", INV), (80, 1, 128, "bf16", "fp4", OK)])
def test_attention_over_four_bits(token_bytes, heads, dim, dtype, kv, status):
    cfg = kvx.attn_config(4 * heads, heads, dim, dtype, kv)
    reqs = kvx.requests_array([(A, None, 100)])
    st, msg = kvx.kvx_attn_validate(pool(token_bytes=token_bytes), reqs, [1], cfg)
    assert st == status and bool(msg) == (status != OK)


@pytest.mark.parametrize("entry,status", [
    ((A, 8, A, 4, 100), OK), ((A, 7, A, 4, 100), OK), ((A, 6, A, 4, 100), INV),
    ((A, 0, A, 1, 100), OK), ((0, 0, A, 4, 0), OK), ((0, 8, A, 4, 100), INV),
    ((A, 8, 0, 4, 100), INV), ((A, 8, A, 0, 100), INV), ((A, 8, A, 33, 100), INV),
    ((A, 8, A, 4, -1), INV), ((A, 65, A, 4, 16 * 64 + 1), INV), ((A, 64, A, 4, 16 * 64), OK),
    ((A + 2, 8, A, 4, 100), ALIGN), ((A, 8, A + 1, 4, 100), ALIGN),
    ((A, 1 << 62, A, 4, 100), INV), ((A, -1, A, 2, 0), INV)])
def test_groups_of_beams(entry, status):
    st, msg = kvx.kvx_beams_validate(pool(), A, kvx.beams_array([entry]))
    assert st == status and bool(msg) == (status != OK)


def test_beams_that_meet():
    two = lambda b: kvx.beams_array([(A, 8, A, 4, 100), (b, 8, A, 4, 100)])  # noqa: E731
    for at, status in ((A + 4 * 32, OK), (A + 4 * 24, kvx.KVX_ERR_OVERLAP), (A, kvx.KVX_ERR_OVERLAP),
                       (A + 4 * 7, kvx.KVX_ERR_OVERLAP)):
        assert kvx.kvx_beams_validate(pool(), A, two(at), level=1)[0] == OK
        assert kvx.kvx_beams_validate(pool(), A, two(at), level=2)[0] == status
    assert kvx.kvx_beams_validate(pool(), 0, two(A))[0] == INV
    assert kvx.kvx_beams_validate(pool(), A + 2, two(A))[0] == INV
    assert kvx.kvx_beams_validate(pool(), A, None)[0] == OK


def test_struct_layout(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lines = []
    for struct in (kvx.kvx_rope, kvx.kvx_select_cfg, kvx.kvx_beams):
        name = struct.__name__
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in struct._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "kvx.h"\n'
                   "int main(void)\n{\n" + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I",
                    os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(line.split() for line in
               subprocess.run([str(exe)], check=True, capture_output=True,
                              text=True).stdout.splitlines())
    for struct in (kvx.kvx_rope, kvx.kvx_select_cfg, kvx.kvx_beams):
        assert int(got[struct.__name__]) == ctypes.sizeof(struct)
        for f, _ in struct._fields_:
            assert int(got[f"{struct.__name__}.{f}"]) == getattr(struct, f).offset, f
