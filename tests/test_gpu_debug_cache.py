"""GPU: the index-checked build of the cache operators against the release build, every output and both caches
set back before each of the two calls, so that a row or an element the debug kernels leave out shows."""
import ctypes

import numpy as np
import pytest
import torch

from speculative_decoding_verification_43_gb300 import _lib, api, build

from attend_ref import Batch
import test_gpu_append as A
import test_gpu_target_pass as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dbg():
    build.build()
    return _lib.load_library(build.DEBUG_LIB_PATH)


def fetch(lib):
    words = np.zeros(4, np.uint32)
    assert lib.spec_debug_fetch(words.ctypes.data_as(ctypes.c_void_p)) == _lib.SPEC_OK
    return words.tolist()


def both(dbg, outputs, start, release, debug):
    """The outputs of the two builds from the same start."""
    fetch(dbg)
    got = []
    for call in (release, debug):
        for t, s in zip(outputs, start):
            t.copy_(s)
        torch.cuda.synchronize()
        call()
        torch.cuda.synchronize()
        got.append([t.clone() for t in outputs])
        assert any(not torch.equal(t, s) for t, s in zip(outputs, start)), "a call that writes something"
    assert fetch(dbg) == [0, 0, 0, 0]
    bits = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
    for x, y in zip(*got):
        assert torch.equal(bits(x), bits(y))


@pytest.mark.parametrize("name", list(A.CASES))
def test_append(dbg, name):
    rows, kv, Hq, Hkv, D, dt, page, rot, inter, order, pad = A.CASES[name]
    a, _ = A.make(rows, kv, Hq, Hkv, D, dt, page, rot, order, pad=pad)
    c = api.KvAppender(len(rows), sum(rows), Hq, Hkv, D, dt, rot_dim=rot, interleaved=inter).bind(**a)
    c.out.q.fill_(9.0)
    c.out.req_status.fill_(-1)
    outs = [c.out.q, c.out.req_status, a["k_cache"], a["v_cache"]]
    st = torch.cuda.current_stream().cuda_stream
    both(dbg, outs, [t.clone() for t in outs], c.run,
         lambda: _lib.check(dbg.spec_kv_append(ctypes.byref(c.args), st), "spec_kv_append"))


@pytest.mark.parametrize("name", list(R.CASES))
def test_attend(dbg, name):
    b = Batch(*R.CASES[name], seed=5).place()
    a = b.attention()
    a.out.out.fill_(9.0)
    a.out.lse.fill_(9.0)
    a.out.req_status.fill_(-1)
    a.workspace.fill_(0xFF)
    outs = [a.out.out, a.out.lse, a.out.req_status]
    st = torch.cuda.current_stream().cuda_stream

    def debug():
        a.workspace.fill_(0xFF)
        _lib.check(dbg.spec_attend(ctypes.byref(a.args), a.workspace.data_ptr(), a.workspace.numel(), st), "spec_attend")

    both(dbg, outs, [t.clone() for t in outs], a.run, debug)
