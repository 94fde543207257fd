"""GPU: the index-checked build of the 8-bit cache's operators and of the block tables against the release build,
every output set back before each of the two calls."""
import ctypes

import pytest
import torch
from cache8_ref import E4M3, Batch8
from test_gpu_debug_cache import both, dbg  # noqa: F401 (a fixture)
from test_gpu_tables import Pool

import test_gpu_append8 as A
import test_gpu_target_pass as R
from speculative_decoding_verification_43_gb300 import _lib, api

pytestmark = pytest.mark.gpu


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("name", list(A.CASES))
def test_append8(dbg, name):  # noqa: F811
    rows, kv, Hq, Hkv, D, dt, page, rot, inter, order, pad = A.CASES[name]
    a, _ = A.make(rows, kv, Hq, Hkv, D, dt, page, rot, order, pad=pad)
    c = api.KvAppender8(len(rows), sum(rows), Hq, Hkv, D, dt, rot_dim=rot, interleaved=inter).bind(**a)
    c.out.q.fill_(9.0)
    c.out.req_status.fill_(-1)
    outs = [c.out.q, c.out.req_status, *(a[n].view(torch.uint8) if a[n].dtype == E4M3 else a[n]
                                         for n in ("k_cache", "v_cache", "k_scale", "v_scale"))]
    both(dbg, outs, [t.clone() for t in outs], c.run,
         lambda: _lib.check(dbg.spec_kv_append8(ctypes.byref(c.args8), stream()), "spec_kv_append8"))


@pytest.mark.parametrize("name", list(R.CASES))
def test_attend8(dbg, name):  # noqa: F811
    b = Batch8(*R.CASES[name], seed=5).place()
    a = b.attention()
    a.out.out.fill_(9.0)
    a.out.lse.fill_(9.0)
    a.out.req_status.fill_(-1)
    a.workspace.fill_(0xFF)
    outs = [a.out.out, a.out.lse, a.out.req_status]

    def debug():
        a.workspace.fill_(0xFF)
        _lib.check(dbg.spec_attend8(ctypes.byref(a.args8), a.workspace.data_ptr(), a.workspace.numel(), stream()), "spec_attend8")

    both(dbg, outs, [t.clone() for t in outs], a.run, debug)


@pytest.mark.parametrize("B", [3, 700])
def test_tables(dbg, B):  # noqa: F811
    pool = Pool([2 + i % 3 for i in range(B)], 8, 40 * B, width=30).device()
    i32 = dict(dtype=torch.int32, device="cuda")
    kv = torch.tensor([(7 * i) % 90 + 3 for i in range(B)], **i32)
    ro = torch.arange(0, 3 * B + 1, 3, **i32)
    t = api.BlockTables(B, 3 * B, 8, pool.n_pages).bind(kv, *pool.d.values(), row_off=ro)
    outs = [*vars(t.out).values(), *pool.d.values()]
    for x in vars(t.out).values():
        x.fill_(-7)

    def debug():
        t.workspace.fill_(0xFF)
        _lib.check(dbg.spec_block_tables(ctypes.byref(t.args), t.workspace.data_ptr(), t.workspace.numel(), stream()),
                   "spec_block_tables")

    both(dbg, outs, [x.clone() for x in outs], t.run, debug)
