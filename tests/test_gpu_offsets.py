"""GPU: spec_attend and spec_kv_append with row offsets that are out of range or out of order. A request holds
its rows when 0 <= row_off[i] <= row_off[i+1] <= T and none of the offsets within [0, T] contradicts it; every
other request reports SPEC_REQ_BAD_SHAPE, and those that hold theirs are served as if nothing were wrong."""
import math

import pytest
import torch

from speculative_decoding_verification_43_gb300 import api

from attend_ref import Batch, check
import test_gpu_append as A

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
TYPES = pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
BIG = 10 ** 9

ROWS = [3, 2, 1, 4, 2, 1]
OFF = [0, 3, 5, 6, 10, 12, 13]
# changed offsets, and the requests that hold their rows then
CASES = {
    "in order": ({}, [0, 1, 2, 3, 4, 5]),
    "one goes back": ({2: 1}, [3, 4, 5]),
    "one goes back to its neighbour": ({3: 4}, [0, 4, 5]),
    "one far ahead": ({1: 12}, [5]),
    "one beyond the rows": ({2: BIG}, [0, 3, 4, 5]),
    "one negative": ({3: -7}, [0, 1, 4, 5]),
    "both ways": ({2: -5, 3: BIG}, [0, 4, 5]),
    "a run beyond the rows": ({1: 14, 2: BIG, 3: BIG, 4: BIG, 5: 14}, []),
    "a run in the middle": ({2: 14, 3: -1, 4: BIG}, [0, 5]),
    "the first": ({0: -1}, [1, 2, 3, 4, 5]),
    "the last": ({6: 99}, [0, 1, 2, 3, 4]),
    "the last goes back": ({6: 0}, []),
    "again and again": ({1: 13, 2: 0, 3: 13, 4: 0, 5: 13}, [5]),
}


def held(off, T):
    """From the definition."""
    out = []
    for i, (a, b) in enumerate(zip(off, off[1:])):
        if 0 <= a <= b <= T and not any(0 <= v <= T and (v > a if j <= i else v < b) for j, v in enumerate(off)):
            out.append(i)
    return out


def changed(change):
    off = list(OFF)
    for j, v in change.items():
        off[j] = v
    return off


@pytest.mark.parametrize("name", list(CASES))
def test_the_cases_follow_the_definition(name):
    change, want = CASES[name]
    assert held(changed(change), 13) == want


def attend_with(b, off):
    """Runs the batch with these offsets (workspace and outputs hold garbage before) and checks it."""
    keep = held(off, b.T)
    b.place()
    b.row_off.copy_(torch.tensor(off, dtype=torch.int32))
    a = b.attention()
    a.workspace.fill_(0xFF)
    for t in (a.out.out, a.out.lse):
        t.fill_(7.0)
    got = a.run()
    torch.cuda.synchronize()
    assert got.req_status.tolist() == [0 if i in keep else 4 for i in range(b.B)]
    rows = torch.zeros(b.T, dtype=torch.bool)
    for i in keep:
        rows[off[i]:off[i + 1]] = True
    b.rows = [off[i + 1] - off[i] if i in keep else 0 for i in range(b.B)]
    b.off = [max(x, 0) for x in off]
    ref = b.reference()
    # rows of requests in error are 0 / -inf where their own offsets are right, and nobody's rows are left alone
    zeroed = torch.zeros(b.T, dtype=torch.bool)
    for i, (x, y) in enumerate(zip(off, off[1:])):
        if i not in keep and 0 <= x <= y <= b.T:
            zeroed[x:y] = True
    assert not (rows & zeroed).any()
    assert (got.out.cpu()[zeroed] == 0).all() and (got.lse.cpu()[zeroed] == -math.inf).all()
    got.out[~rows], got.lse[~rows] = 0, -math.inf
    check(b, got, ref)


@TYPES
@pytest.mark.parametrize("shared", [0, 40])
@pytest.mark.parametrize("name", list(CASES))
def test_attend(dtype, shared, name):
    b = Batch(ROWS, [n + 50 + 20 * i for i, n in enumerate(ROWS)], 8, 2, 64, dtype, 16, shared=shared, seed=7)
    attend_with(b, changed(CASES[name][0]))


@pytest.mark.parametrize("shared", [0, 40])
@pytest.mark.parametrize("name", ["one goes back", "both ways", "again and again"])
def test_attend_with_many_rows(shared, name):
    """The same shapes with 30 rows for one."""
    rows = [30 * n for n in ROWS]
    b = Batch(rows, [n + 50 + 20 * i for i, n in enumerate(rows)], 8, 2, 64, BF, 16, shared=shared, seed=7)
    attend_with(b, [30 * x if 0 <= x <= 13 else x for x in changed(CASES[name][0])])


def wide():
    """1100 requests of one row; offsets beyond the rows where a search looks first, a run of them, one that
    goes back by two."""
    off = list(range(1101))
    for j in (35, 70, 350, 700, 1050):
        off[j] = BIG if j % 20 else -3
    for j in range(500, 560):
        off[j] = -1 - j
    off[812] = 810
    return off


@TYPES
@pytest.mark.parametrize("shared", [0, 20])
def test_attend_with_many_requests(dtype, shared):
    b = Batch([1] * 1100, [shared + 1 + i % 30 for i in range(1100)], 4, 2, 64, dtype, 16, shared=shared, seed=7)
    attend_with(b, wide())


def append_with(rows, off, dtype):
    T, B = sum(rows), len(rows)
    kv = [n + 20 + 7 * (i % 5) for i, n in enumerate(rows)]
    a, _ = A.make(rows, kv, 4, 2, 64, dtype, 16, 64)
    keep = held(off, T)
    a["row_off"].copy_(torch.tensor(off, dtype=torch.int32))
    before = a["k_cache"].clone(), a["v_cache"].clone()
    out = torch.full((T, 4, 64), 9.0, dtype=dtype, device="cuda")
    o = api.kv_append(**a, q_out=out)
    torch.cuda.synchronize()
    assert o.req_status.tolist() == [0 if i in keep else 4 for i in range(B)]
    own = torch.zeros(T, dtype=torch.bool)
    for i in keep:
        own[off[i]:off[i + 1]] = True
    assert (out.cpu()[~own] == 9.0).all()
    a["q0"] = None
    A.verify(a, [max(x, 0) for x in off], [off[i + 1] - off[i] if i in keep else 0 for i in range(B)], kv, 16, 64, False,
             o.q, before)


@TYPES
@pytest.mark.parametrize("name", list(CASES))
def test_append(dtype, name):
    append_with(ROWS, changed(CASES[name][0]), dtype)


@pytest.mark.parametrize("name", ["one goes back", "both ways", "again and again"])
def test_append_with_many_rows(name):
    append_with([150 * n for n in ROWS], [150 * x if 0 <= x <= 13 else x for x in changed(CASES[name][0])], BF)


def test_append_with_many_requests():
    append_with([1] * 1100, wide(), BF)
