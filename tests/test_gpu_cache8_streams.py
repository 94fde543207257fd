"""GPU: the 8-bit cache's calls and the block tables' on another stream than the one their tensors belong to
(tests/test_gpu_streams.py has the method)."""
import pytest
import torch
from cache8_ref import E4M3, Batch8
from test_gpu_streams import busy_stream, fills, untouched
from test_gpu_tables import Pool

import test_gpu_append8 as A
from speculative_decoding_verification_43_gb300 import api

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def batch():
    return Batch8([3, 5, 1], [900, 1300, 40], 8, 2, 128, BF, 16, shared=32, seed=1).place()


def settled(b):
    a = b.attention()
    o = a.run()
    want = o.out.clone(), o.lse.clone()
    like = [torch.empty_like(t) for t in (a.workspace, o.out, o.lse, o.req_status)]
    torch.cuda.synchronize()
    return want, like


@pytest.mark.parametrize("keep", [True, False], ids=["kept", "dropped"])
def test_attend8_on_a_busy_stream(keep):
    b = batch()
    want, like = settled(b)
    st = busy_stream()
    o = api.attend8(b.qd, *b.cache(), b.row_off, b.kv_len, b.table, shared_len=b.shared, shared_table=b.shared_table, stream=st)
    if not keep:
        del o
    f = fills(*like)
    torch.cuda.synchronize()
    assert untouched(f)
    if keep:
        assert torch.equal(o.out, want[0]) and torch.equal(o.lse, want[1])


def test_prepared_attention8_dropped_while_it_runs():
    b = batch()
    _, like = settled(b)
    a = b.attention()
    st = busy_stream()
    a.run(st)
    del a
    f = fills(*like)
    torch.cuda.synchronize()
    assert untouched(f)


def bits(a):
    return [a[n].view(torch.uint8) if a[n].dtype == E4M3 else a[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")]


def test_kv_append8_on_a_busy_stream():
    a, _ = A.make([3, 2], [60, 70], 4, 2, 64, BF, 16, 64)
    start = [t.clone() for t in bits(a)]
    o = api.kv_append8(**a)
    want = [o.q.clone(), *(t.clone() for t in bits(a))]
    like = [torch.empty_like(o.q), torch.empty_like(o.req_status)]
    for t, s in zip(bits(a), start):
        t.copy_(s)
    torch.cuda.synchronize()
    st = busy_stream()
    o = api.kv_append8(**a, stream=st)
    f = fills(*like)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip([o.q, *bits(a)], want)) and untouched(f)
    c = api.KvAppender8(2, 5, 4, 2, 64, BF).bind(**a)
    st = busy_stream()
    c.run(st)
    del c
    f = fills(*like)
    torch.cuda.synchronize()
    assert untouched(f)


def test_block_tables_on_a_busy_stream():
    pool = Pool([2, 5, 1], 8, 40, width=12).device()
    i32 = dict(dtype=torch.int32, device="cuda")
    kv, ro = torch.tensor([40, 8, 33], **i32), torch.tensor([0, 3, 4, 8], **i32)
    args = dict(row_off=ro, total_rows=8)
    start = [t.clone() for t in pool.d.values()]
    o = api.block_tables(kv, *pool.d.values(), 8, **args)
    want = [o.slot_map.clone(), o.positions.clone(), *(t.clone() for t in pool.d.values())]
    like = [torch.empty_like(t) for t in vars(o).values()]
    for t, s in zip(pool.d.values(), start):
        t.copy_(s)
    torch.cuda.synchronize()
    st = busy_stream()
    o = api.block_tables(kv, *pool.d.values(), 8, **args, stream=st)
    f = fills(*like)
    torch.cuda.synchronize()
    assert untouched(f)
    assert all(torch.equal(x, y) for x, y in zip([o.slot_map, o.positions, *pool.d.values()], want))


def test_tables_made_on_a_busy_stream_and_run_on_another():
    """Nothing that making a prepared call left on its stream comes after the run."""
    i32 = dict(dtype=torch.int32, device="cuda")
    pool = Pool([1, 2], 8, 10, width=6).device()
    kv, row_off = torch.tensor([20, 25], **i32), torch.tensor([0, 3, 5], **i32)
    torch.cuda.synchronize()
    st = busy_stream()
    with torch.cuda.stream(st):
        t = api.BlockTables(2, 5, 8, pool.n_pages)
    t.bind(kv, *pool.d.values(), row_off=row_off)
    o = t.run()
    torch.cuda.synchronize()
    pool.step([20, 25])
    pool.same()
    slots, pos = pool.rows([3, 2], [20, 25], [0, 0])
    assert o.slot_map.cpu().tolist() == slots and o.positions.cpu().tolist() == pos
