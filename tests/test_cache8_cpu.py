"""CPU: what spec_cache8.h and spec_tables.h declare is exported and laid out as the binding has it, and wrong
arguments are refused before anything touches a GPU (every pointer here is fake)."""
import ctypes
import os
import re
import shutil
import subprocess
import tempfile

import pytest
from test_attend_cpu import FAKE, append_args

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_43_gb300 import build
    build.build()
    from speculative_decoding_verification_43_gb300 import _lib
    return _lib


@pytest.mark.parametrize("header,exports", [("spec_cache8.h", "CACHE8_EXPORTS"), ("spec_tables.h", "TABLES_EXPORTS")])
def test_every_declared_symbol_is_exported(lib, header, exports):
    from speculative_decoding_verification_43_gb300 import build
    src = open(os.path.join(ROOT, "include", header)).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = set(re.findall(r"^\s*(?:const\s+)?[A-Za-z_][A-Za-z0-9_]*\s*\*?\s*([a-z_][a-z0-9_]*)\s*\(", src, flags=re.M))
    assert names == set(getattr(lib, exports))
    for path in (build.LIB_PATH, build.DEBUG_LIB_PATH):
        raw = ctypes.CDLL(path)
        for n in names:
            assert hasattr(raw, n), n


def test_ctypes_structs_match_the_header_layout(lib):
    cuda_inc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    if not shutil.which("gcc") or not os.path.exists(os.path.join(cuda_inc, "cuda_runtime_api.h")):
        pytest.skip("gcc or the CUDA headers are missing")
    structs = (("spec_kv_append8_args", lib.SpecKvAppend8Args), ("spec_attend8_args", lib.SpecAttend8Args),
               ("spec_block_tables_args", lib.SpecBlockTablesArgs))
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "spec_cache8.h"', '#include "spec_tables.h"',
             "int main(void) {"]
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


def append8_args(lib, **kw):
    a = lib.SpecKvAppend8Args()
    a.k_scale = a.v_scale = FAKE
    inner = {k: v for k, v in kw.items() if k not in ("k_scale", "v_scale")}
    a.append = append_args(lib, **inner)
    for k in ("k_scale", "v_scale"):
        if k in kw:
            setattr(a, k, kw[k])
    return a


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), -1), (dict(total_rows=-1), -1), (dict(n_q_heads=-1), -1), (dict(n_kv_heads=0), -1),
    (dict(head_dim=0), -1), (dict(rot_dim=63), -1), (dict(rot_dim=66), -1), (dict(page_size=0), -1),
    (dict(max_blocks=0), -1), (dict(n_pages=0), -1), (dict(n_pos=-1), -1), (dict(dtype=7), -1), (dict(q=None), -1),
    (dict(k=None), -1), (dict(v=None), -1), (dict(cos_sin=None), -1), (dict(k_cache=None), -1), (dict(v_cache=None), -1),
    (dict(row_off=None), -1), (dict(kv_len=None), -1), (dict(block_table=None), -1), (dict(k_scale=None), -1),
    (dict(v_scale=None), -1), (dict(k_stride=100), -1), (dict(page_stride=-1), -1), (dict(head_dim=600), -4),
    (dict(total_rows=(1 << 20) + 1), -4), (dict(page_size=(1 << 16) + 1), -4), (dict(B=1 << 28), -4),
])
def test_append8_refuses(lib, kw, want):
    a = append8_args(lib, **kw)
    if kw.get("head_dim") == 600:
        a.append.k_stride = a.append.v_stride = 1200
        a.append.q_stride = a.append.q_out_stride = 2400
    assert lib.lib.spec_kv_append8(ctypes.byref(a), None) == want


def test_append8_refuses_null(lib):
    assert lib.lib.spec_kv_append8(None, None) == -1


def attend8_args(lib, **kw):
    x = lib.SpecAttend8Args()
    x.k_scale = x.v_scale = FAKE
    a = x.attend
    a.B, a.total_rows, a.n_q_heads, a.n_kv_heads, a.head_dim = 4, 8, 4, 2, 64
    a.page_size, a.max_blocks, a.n_pages, a.dtype, a.scale = 16, 8, 32, lib.SPEC_BF16, 0.125
    for f in ("q", "k_cache", "v_cache", "row_off", "kv_len", "block_table", "out", "lse", "req_status"):
        setattr(a, f, FAKE)
    a.q_stride = a.out_stride = 256
    a.page_stride, a.slot_stride, a.head_stride = 2048, 128, 64
    for k, v in kw.items():
        setattr(x if k in ("k_scale", "v_scale") else a, k, v)
    return x


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), -1), (dict(total_rows=-1), -1), (dict(n_q_heads=3), -1), (dict(n_kv_heads=0), -1), (dict(head_dim=0), -1),
    (dict(page_size=0), -1), (dict(max_blocks=0), -1), (dict(n_pages=0), -1), (dict(window=-1), -1), (dict(n_sink=-1), -1),
    (dict(shared_len=-1), -1), (dict(shared_len=5), -1), (dict(dtype=9), -1), (dict(scale=0.0), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(q=None), -1), (dict(out=None), -1),
    (dict(k_cache=None), -1), (dict(v_cache=None), -1), (dict(row_off=None), -1), (dict(kv_len=None), -1),
    (dict(block_table=None), -1), (dict(k_scale=None), -1), (dict(v_scale=None), -1), (dict(q_stride=100), -1),
    (dict(slot_stride=-16), -1), (dict(head_dim=72), -4), (dict(head_dim=272), -4), (dict(q=FAKE + 8), -4),
    (dict(k_cache=FAKE + 8), -4), (dict(v_cache=FAKE + 4), -4), (dict(slot_stride=120), -4), (dict(page_stride=2056), -4),
    (dict(head_stride=72), -4), (dict(total_rows=1 << 28), -4),
])
def test_attend8_refuses(lib, kw, want):
    a = attend8_args(lib, **kw)
    assert lib.lib.spec_attend8(ctypes.byref(a), FAKE * 256, 1 << 40, None) == want


def test_attend8_workspace(lib):
    a = attend8_args(lib)
    n = lib.lib.spec_attend8_workspace_size(ctypes.byref(a))
    assert n > 0
    assert lib.lib.spec_attend8(ctypes.byref(a), None, n, None) == -2
    assert lib.lib.spec_attend8(ctypes.byref(a), FAKE * 256, n - 1, None) == -2
    assert lib.lib.spec_attend8(ctypes.byref(a), FAKE * 256 + 16, n, None) == -2
    assert lib.lib.spec_attend8_workspace_size(ctypes.byref(attend8_args(lib, head_dim=72))) == 0
    assert lib.lib.spec_attend8_workspace_size(None) == 0 and lib.lib.spec_attend8(None, None, 0, None) == -1


def table_args(lib, **kw):
    a = lib.SpecBlockTablesArgs()
    a.B, a.total_rows, a.page_size, a.max_blocks, a.n_pages, a.n_shared = 4, 8, 16, 8, 32, 2
    for f in ("kv_len", "row_off", "shared_table", "n_blocks", "block_table", "free_pages", "n_free", "slot_map", "positions",
              "req_status"):
        setattr(a, f, FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,want", [
    (dict(B=0), -1), (dict(total_rows=-1), -1), (dict(page_size=0), -1), (dict(max_blocks=0), -1), (dict(n_pages=0), -1),
    (dict(n_shared=-1), -1), (dict(n_shared=9), -1), (dict(kv_len=None), -1), (dict(row_off=None), -1),
    (dict(shared_table=None), -1), (dict(n_blocks=None), -1), (dict(block_table=None), -1), (dict(free_pages=None), -1),
    (dict(n_free=None), -1), (dict(B=1 << 20, max_blocks=1 << 12), -4), (dict(n_pages=1 << 20, page_size=1 << 12), -4),
])
def test_tables_refuse(lib, kw, want):
    a = table_args(lib, **kw)
    assert lib.lib.spec_block_tables(ctypes.byref(a), FAKE * 256, 1 << 40, None) == want


def test_tables_workspace(lib):
    a = table_args(lib)
    n = lib.lib.spec_block_tables_workspace_size(ctypes.byref(a))
    assert n > 0
    assert lib.lib.spec_block_tables(ctypes.byref(a), None, n, None) == -2
    assert lib.lib.spec_block_tables(ctypes.byref(a), FAKE * 256, n - 1, None) == -2
    assert lib.lib.spec_block_tables(ctypes.byref(a), FAKE * 256 + 8, n, None) == -2
    assert lib.lib.spec_block_tables_workspace_size(ctypes.byref(table_args(lib, B=0))) == 0
    assert lib.lib.spec_block_tables_workspace_size(None) == 0 and lib.lib.spec_block_tables(None, None, 0, None) == -1


# the most rows, and entries of all tables, that are taken (rows and entries are stepped through in 32 bits)
TABLES_MOST = (1 << 31) - (1 << 19)


@pytest.mark.parametrize("kw", [dict(total_rows=TABLES_MOST + 1), dict(total_rows=(1 << 31) - 1),
                                dict(total_rows=(1 << 31) - 300000, slot_map=None, positions=None),
                                dict(B=TABLES_MOST + 1, max_blocks=1, n_shared=1), dict(B=(1 << 31) - 1, max_blocks=1, n_shared=0),
                                dict(B=1, max_blocks=(1 << 31) - 1), dict(B=1 << 12, max_blocks=(1 << 19) - 127)])
def test_tables_refuse_steps_beyond_32_bits(lib, kw):
    a = table_args(lib, **kw)
    assert lib.lib.spec_block_tables_workspace_size(ctypes.byref(a)) == 0
    assert lib.lib.spec_block_tables(ctypes.byref(a), FAKE * 256, 1 << 40, None) == -4


@pytest.mark.parametrize("kw,B", [(dict(total_rows=TABLES_MOST), 4), (dict(B=TABLES_MOST, max_blocks=1, n_shared=0), TABLES_MOST),
                                  (dict(B=1 << 12, max_blocks=(1 << 19) - 128), 1 << 12)])
def test_tables_take_the_largest_sizes(lib, kw, B):
    """Up to the workspace, which is too small by one byte here, so that nothing is enqueued."""
    a = table_args(lib, **kw)
    n = lib.lib.spec_block_tables_workspace_size(ctypes.byref(a))
    assert n >= 20 * (B + 1)
    assert lib.lib.spec_block_tables(ctypes.byref(a), FAKE * 256, n - 1, None) == -2
