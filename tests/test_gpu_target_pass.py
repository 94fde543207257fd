"""GPU: the example's rounds (append, attend, verify) end to end, and the index-checked build of the
cache operators against the release build."""
import ctypes
import os
import sys

import numpy as np
import pytest
import torch

from speculative_decoding_verification_43_gb300 import _lib, api, build

from attend_ref import Batch
import test_gpu_append as A

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def plain_logits(m, tokens):
    """The example's model on one text, from the definition, in float64 on bf16 weights."""
    x = m.embed[torch.tensor(tokens, device="cuda")].double()
    n, G = len(tokens), m.Hq // m.Hkv
    norm = lambda y: y * torch.rsqrt(y.pow(2).mean(-1, keepdim=True) + 1e-30)  # noqa: E731
    cos, sin = m.cos_sin[:n].double().chunk(2, 1)
    turn = lambda y: torch.cat([y[..., :m.D // 2] * cos[:, None] - y[..., m.D // 2:] * sin[:, None],  # noqa: E731
                                y[..., m.D // 2:] * cos[:, None] + y[..., :m.D // 2] * sin[:, None]], -1)
    at = torch.arange(n, device="cuda")
    hidden = at[None] > at[:, None]
    if m.window:
        hidden |= (at[None] <= at[:, None] - m.window) & (at[None] >= m.n_sink)
    for w in m.layers:
        qkv = norm(x) @ w["qkv"].double()
        q, k, v = (t.unflatten(1, (-1, m.D)) for t in qkv.split([m.Hq * m.D, m.Hkv * m.D, m.Hkv * m.D], 1))
        q, k = turn(q), turn(k).repeat_interleave(G, 1)
        z = torch.einsum("ihd,jhd->hij", q, k) / m.D ** 0.5
        z[:, hidden] = -torch.inf
        o = torch.einsum("hij,jhd->ihd", torch.softmax(z, -1), v.repeat_interleave(G, 1))
        x = x + o.flatten(1) @ w["out"].double()
        a, b = (norm(x) @ w["up"].double()).chunk(2, 1)
        x = x + (torch.nn.functional.silu(a) * b) @ w["down"].double()
    return norm(x) @ m.head.double()


@pytest.mark.parametrize("kw", [dict(), dict(shared=False), dict(window=24, n_sink=3)], ids=["shared", "own pages", "window"])
def test_rounds_follow_the_texts(kw):
    """After several rounds with rejected drafts, the cached model's logits are those of the plain model on
    the requests' texts. The model runs in bf16 (some thirty roundings of 2^-8 relative on the way to a
    logit): its error is held to 5 % of the logits' spread in the mean and 40 % at the largest."""
    import target_pass as ex
    kw = {**dict(B=5, gamma=3, rounds=3, prompt=37, seed=3), **kw}
    texts, logits, o = ex.run(**kw)
    m = ex.Target(seed=kw["seed"], window=kw.get("window", 0), n_sink=kw.get("n_sink", 0))
    n, A_len = o.n_emitted.tolist(), o.accept_len.tolist()
    at = 0
    for i, t in enumerate(texts):
        K = min(3, i % 4)
        # rows of the last round that are part of the text: the pending token and the accepted drafts
        want = plain_logits(m, t[:-1] if n[i] else t)[-(A_len[i] + 1):]
        got = logits[at:at + A_len[i] + 1].double()
        err, spread = (got - want).abs(), want.std()
        assert err.mean() <= 0.05 * spread and err.max() <= 0.4 * spread, (i, err.mean() / spread, err.max() / spread)
        at += K + 1


def fetch(lib):
    words = np.zeros(4, np.uint32)
    assert lib.spec_debug_fetch(words.ctypes.data_as(ctypes.c_void_p)) == _lib.SPEC_OK
    return words


@pytest.fixture(scope="module")
def dbg():
    build.build()
    return _lib.load_library(build.DEBUG_LIB_PATH)


BF, F32 = torch.bfloat16, torch.float32
CASES = {
    "round": ([1, 8, 3], [1, 300, 130], 8, 2, 128, BF, 16, 0, 0, 0),
    "round f32": ([1, 8, 3], [1, 300, 130], 8, 2, 128, F32, 16, 0, 0, 0),
    "window, odd page": ([2, 5], [400, 77], 6, 2, 80, BF, 7, 50, 3, 0),
    "shared": ([2, 1, 5], [300, 258, 262], 8, 2, 64, BF, 16, 0, 0, 250),
    "shared f32": ([2, 1, 5], [300, 258, 262], 8, 2, 64, F32, 16, 0, 0, 250),
    "prompts": ([170, 300], [170, 400], 4, 2, 128, BF, 16, 0, 0, 0),
    "prompts behind a prefix": ([170, 100], [370, 300], 4, 2, 128, BF, 16, 0, 0, 150),
    "nothing": ([3, 0, 2], [0, 5, 1], 4, 2, 128, BF, 16, 0, 0, 0),
}


@pytest.mark.parametrize("name", list(CASES))
def test_debug_build_of_attend(dbg, name):
    fetch(dbg)
    b = Batch(*CASES[name], seed=5).place()
    a = b.attention()
    r = a.run()
    want = r.out.clone(), r.lse.clone(), r.req_status.clone()
    r.out.fill_(3.0)
    st = torch.cuda.current_stream().cuda_stream
    _lib.check(dbg.spec_attend(ctypes.byref(a.args), a.workspace.data_ptr(), a.workspace.numel(), st), "spec_attend")
    torch.cuda.synchronize()
    assert torch.equal(r.out, want[0]) and torch.equal(r.lse, want[1]) and torch.equal(r.req_status, want[2])
    words = fetch(dbg)
    assert words[3] == 0, words


@pytest.mark.parametrize("name", ["ragged", "ragged f32", "interleaved", "rows off the vectors", "padding rows"])
def test_debug_build_of_append(dbg, name):
    rows, kv, Hq, Hkv, D, dt, page, rot, inter, order, pad = A.CASES[name]
    fetch(dbg)
    a, _ = A.make(rows, kv, Hq, Hkv, D, dt, page, rot, order, pad=pad)
    c = api.KvAppender(len(rows), sum(rows), Hq, Hkv, D, dt, rot_dim=rot, interleaved=inter).bind(**a)
    q = c.run().q.clone()
    k, v = a["k_cache"].clone(), a["v_cache"].clone()
    st = torch.cuda.current_stream().cuda_stream
    _lib.check(dbg.spec_kv_append(ctypes.byref(c.args), st), "spec_kv_append")
    torch.cuda.synchronize()
    if pad == 0 and min(kv) >= max(rows):
        assert torch.equal(c.out.q, q)
    assert torch.equal(a["k_cache"], k) and torch.equal(a["v_cache"], v)
    assert fetch(dbg)[3] == 0


def test_plan_names_the_kernel():
    plans = {}
    for name, c in CASES.items():
        plans[name] = Batch(*c, seed=5).place().attention().plan()
    assert plans["round"] == "spec_attend_round_kernel" and plans["round f32"] == "spec_attend_fma_kernel"
    assert plans["prompts"] == "spec_attend_pair_kernel" and plans["window, odd page"] == "spec_attend_round_kernel"
