"""CPU: what spec_attend.h declares is exported and laid out as the binding has it, and wrong arguments
are refused before anything touches a GPU (every pointer here is fake)."""
import ctypes
import os
import re
import shutil
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_43_gb300 import build
    build.build()
    from speculative_decoding_verification_43_gb300 import _lib
    return _lib


def test_every_declared_symbol_is_exported(lib):
    from speculative_decoding_verification_43_gb300 import build
    src = open(os.path.join(ROOT, "include", "spec_attend.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?[A-Za-z_][A-Za-z0-9_]*\s*\*?\s*([a-z_][a-z0-9_]*)\s*\(", src, flags=re.M))
    assert names == set(lib.ATTEND_EXPORTS)
    for path in (build.LIB_PATH, build.DEBUG_LIB_PATH):
        raw = ctypes.CDLL(path)
        for n in names:
            assert hasattr(raw, n), n


def test_ctypes_structs_match_the_header_layout(lib):
    cuda_inc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    if not shutil.which("gcc") or not os.path.exists(os.path.join(cuda_inc, "cuda_runtime_api.h")):
        pytest.skip("gcc or the CUDA headers are missing")
    structs = (("spec_kv_append_args", lib.SpecKvAppendArgs), ("spec_attend_args", lib.SpecAttendArgs))
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "spec_attend.h"', "int main(void) {"]
    for cname, cls in structs:
        lines.append(f'printf("{cname} sizeof %zu\\n", sizeof({cname}));')
        for f, _ in cls._fields_:
            lines.append(f'printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));')
    lines += ["return 0;", "}"]
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "layout.c"), os.path.join(d, "layout")
        open(src, "w").write("\n".join(lines))
        subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), "-I", cuda_inc, src, "-o", exe])
        out = subprocess.check_output([exe], text=True)
    got = {(a, b): int(c) for a, b, c in (ln.split() for ln in out.splitlines())}
    for cname, cls in structs:
        assert got[(cname, "sizeof")] == ctypes.sizeof(cls), cname
        for f, _ in cls._fields_:
            assert got[(cname, f)] == getattr(cls, f).offset, (cname, f)


FAKE = 0x10000


def append_args(lib, **kw):
    a = lib.SpecKvAppendArgs()
    a.B, a.total_rows, a.n_q_heads, a.n_kv_heads, a.head_dim, a.rot_dim = 4, 8, 4, 2, 64, 64
    a.page_size, a.max_blocks, a.n_pages, a.n_pos, a.dtype = 16, 8, 32, 128, lib.SPEC_BF16
    for f in ("q", "k", "v", "q_out", "cos_sin", "k_cache", "v_cache", "row_off", "kv_len", "block_table"):
        setattr(a, f, FAKE)
    a.q_stride = a.q_out_stride = 256
    a.k_stride = a.v_stride = 128
    a.page_stride, a.slot_stride, a.head_stride = 2048, 128, 64
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), -1), (dict(total_rows=-1), -1), (dict(n_q_heads=-1), -1), (dict(n_kv_heads=0), -1),
    (dict(head_dim=0), -1), (dict(rot_dim=63), -1), (dict(rot_dim=66), -1), (dict(rot_dim=-2), -1),
    (dict(page_size=0), -1), (dict(max_blocks=0), -1), (dict(n_pages=0), -1), (dict(n_pos=-1), -1),
    (dict(dtype=7), -1), (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(q_out=None), -1),
    (dict(cos_sin=None), -1), (dict(k_cache=None), -1), (dict(v_cache=None), -1), (dict(row_off=None), -1),
    (dict(kv_len=None), -1), (dict(block_table=None), -1), (dict(q_stride=255), -1), (dict(k_stride=0), -1),
    (dict(q_out_stride=512), -1),  # in place, but with another stride
    (dict(page_stride=-1), -1), (dict(head_dim=520, rot_dim=0, q_stride=1 << 20, q_out_stride=1 << 20,
                                      k_stride=1 << 20, v_stride=1 << 20), -4),
])
def test_append_refuses(lib, kw, want):
    assert lib.lib.spec_kv_append(ctypes.byref(append_args(lib, **kw)), None) == want
    assert lib.lib.spec_kv_append(None, None) == -1


def attend_args(lib, **kw):
    a = lib.SpecAttendArgs()
    a.B, a.total_rows, a.n_q_heads, a.n_kv_heads, a.head_dim = 4, 8, 4, 2, 64
    a.page_size, a.max_blocks, a.n_pages, a.dtype, a.scale = 16, 8, 32, lib.SPEC_BF16, 0.125
    for f in ("q", "k_cache", "v_cache", "row_off", "kv_len", "block_table", "out", "lse"):
        setattr(a, f, FAKE)
    a.q_stride = a.out_stride = 256
    a.page_stride, a.slot_stride, a.head_stride = 2048, 128, 64
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), -1), (dict(total_rows=-1), -1), (dict(n_q_heads=3), -1), (dict(n_q_heads=0), -1),
    (dict(n_kv_heads=0), -1), (dict(head_dim=0), -1), (dict(page_size=0), -1), (dict(max_blocks=0), -1),
    (dict(n_pages=0), -1), (dict(window=-1), -1), (dict(n_sink=-1), -1), (dict(shared_len=-1), -1),
    (dict(shared_len=16), -1),  # no table for it
    (dict(dtype=9), -1), (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=float("nan")), -1),
    (dict(scale=float("inf")), -1), (dict(q=None), -1), (dict(out=None), -1), (dict(k_cache=None), -1),
    (dict(v_cache=None), -1), (dict(row_off=None), -1), (dict(kv_len=None), -1), (dict(block_table=None), -1),
    (dict(q_stride=248), -1), (dict(out_stride=0), -1), (dict(slot_stride=-8), -1),
    (dict(head_dim=260), -4), (dict(head_dim=60), -4), (dict(q=FAKE + 8), -4), (dict(out=FAKE + 2), -4),
    (dict(k_cache=FAKE + 4), -4), (dict(q_stride=260), -4), (dict(slot_stride=132), -4), (dict(head_stride=68), -4),
    (dict(max_blocks=1 << 28), -4),
])
def test_attend_refuses(lib, kw, want):
    a = attend_args(lib, **kw)
    assert lib.lib.spec_attend(ctypes.byref(a), 0x20000, 1 << 40, None) == want
    assert lib.lib.spec_attend(None, 0x20000, 1 << 40, None) == -1


def test_attend_workspace(lib):
    a = attend_args(lib)
    need = lib.lib.spec_attend_workspace_size(ctypes.byref(a))
    assert need > 0 and need % 256 == 0
    assert lib.lib.spec_attend(ctypes.byref(a), None, need, None) == -2
    assert lib.lib.spec_attend(ctypes.byref(a), 0x20000, need - 1, None) == -2
    assert lib.lib.spec_attend(ctypes.byref(a), 0x20010, need, None) == -2
    assert lib.lib.spec_attend_workspace_size(ctypes.byref(attend_args(lib, B=0))) == 0
    assert lib.lib.spec_attend_plan(ctypes.byref(attend_args(lib, n_q_heads=3))) is None
    # the sizes alone decide: more rows or a shared prefix never need less
    more = lib.lib.spec_attend_workspace_size(ctypes.byref(attend_args(lib, total_rows=64)))
    shared = lib.lib.spec_attend_workspace_size(ctypes.byref(attend_args(lib, total_rows=64, shared_len=64)))
    assert need <= more <= shared
