"""GPU: spec_attend against float64 (tests/attend_ref.py has the reference and the bounds): lengths from
zero up, odd sizes, group sizes, head layouts, page sizes that end inside a tile, windows and
sinks, shared prefixes, rows that see nothing, values that are not finite in places nobody sees."""
import math

import pytest
import torch

from attend_ref import Batch, check

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32

# rows, kv, Hq, Hkv, D, dtype, page, window, sinks, shared, order
CASES = {
    "one token": ([1], [1], 4, 4, 128, BF, 16, 0, 0, 0, "slot"),
    "one round": ([5], [1005], 32, 8, 128, BF, 16, 0, 0, 0, "slot"),
    "one round f32": ([5], [1005], 32, 8, 128, F32, 16, 0, 0, 0, "slot"),
    "ragged": ([1, 8, 3, 2, 6], [1, 8, 130, 257, 1023], 8, 2, 128, BF, 16, 0, 0, 0, "slot"),
    "ragged f32": ([1, 8, 3, 2, 6], [1, 8, 130, 257, 1023], 8, 2, 128, F32, 16, 0, 0, 0, "head"),
    "heads of 64": ([4, 7, 1], [300, 129, 64], 12, 4, 64, BF, 24, 0, 0, 0, "head"),
    "heads of 80, group 3": ([2, 9], [500, 77], 6, 2, 80, BF, 7, 0, 0, 0, "slot"),
    "heads of 96": ([3, 1, 2], [200, 400, 128], 8, 8, 96, BF, 64, 0, 0, 0, "slot"),
    "heads of 72": ([3, 1, 2], [200, 40, 128], 8, 4, 72, BF, 16, 0, 0, 0, "slot"),
    "heads of 256": ([2, 3], [300, 70], 4, 2, 256, BF, 16, 40, 3, 0, "slot"),
    "heads of 256 f32": ([2, 3], [300, 70], 4, 2, 256, F32, 16, 0, 0, 0, "head"),
    "heads of 4 f32": ([2, 3], [30, 70], 2, 1, 4, F32, 3, 0, 0, 0, "slot"),
    "heads of 16": ([2, 3], [300, 70], 4, 2, 16, BF, 16, 0, 0, 0, "slot"),
    "one head for all": ([6, 2], [300, 513], 40, 1, 128, BF, 16, 0, 0, 0, "slot"),
    "pages of one": ([2, 3], [140, 33], 4, 2, 64, BF, 1, 0, 0, 0, "slot"),
    "window": ([5, 8, 1, 2], [900, 1024, 33, 400], 8, 2, 128, BF, 16, 100, 0, 0, "slot"),
    "window and sinks": ([5, 8, 1, 2], [900, 1024, 33, 400], 8, 2, 128, BF, 16, 100, 4, 0, "slot"),
    "window and sinks f32": ([5, 8, 1, 2], [900, 1024, 33, 400], 8, 2, 64, F32, 16, 100, 4, 0, "slot"),
    "window of one": ([3, 4], [50, 300], 4, 2, 64, BF, 16, 1, 0, 0, "slot"),
    "window of one, many sinks": ([3, 4], [50, 700], 4, 2, 64, BF, 16, 1, 290, 0, "slot"),
    "window longer than the text": ([3, 4], [50, 300], 4, 2, 64, BF, 16, 10000, 2, 0, "slot"),
    "prompt": ([200], [200], 4, 2, 128, BF, 16, 0, 0, 0, "slot"),
    "prompts": ([70, 1, 333], [170, 90, 460], 8, 2, 64, BF, 16, 0, 0, 0, "head"),
    "prompts, window": ([70, 1, 333], [170, 90, 460], 8, 2, 128, BF, 16, 50, 5, 0, "slot"),
    "prompts f32": ([70, 1, 133], [170, 90, 260], 4, 2, 64, F32, 16, 0, 0, 0, "slot"),
    "nothing to see": ([3, 2, 4, 0, 1], [0, 1, 2, 40, 0], 4, 2, 128, BF, 16, 0, 0, 0, "slot"),
    "nothing to see f32": ([3, 2, 4, 0, 1], [0, 1, 2, 40, 0], 4, 2, 128, F32, 16, 0, 0, 0, "slot"),
    "no rows at all": ([0, 0], [5, 40], 4, 2, 128, BF, 16, 0, 0, 0, "slot"),
    "shared": ([2, 1, 5], [300, 258, 262], 8, 2, 128, BF, 16, 0, 0, 256, "slot"),
    "shared f32": ([2, 1, 5], [300, 258, 262], 8, 2, 128, F32, 16, 0, 0, 256, "slot"),
    "shared, ends inside a page": ([2, 1, 5, 3], [350, 340, 345, 601], 12, 4, 96, BF, 16, 0, 0, 333, "head"),
    "shared, rows inside the prefix": ([4, 2, 3, 0, 2], [100, 201, 250, 200, 0], 8, 2, 64, BF, 16, 0, 0, 200, "slot"),
    "shared, window behind it": ([4, 2], [700, 460], 8, 2, 64, BF, 16, 50, 3, 300, "slot"),
    "shared, window across": ([4, 2], [330, 340], 8, 2, 128, BF, 16, 100, 3, 300, "slot"),
    "shared, many rows": ([8] * 30, [600 + 3 * i for i in range(30)], 16, 2, 64, BF, 16, 0, 0, 520, "slot"),
    "shared, many rows f32": ([3] * 9, [300 + 3 * i for i in range(9)], 8, 2, 64, F32, 16, 0, 0, 290, "slot"),
    "shared only": ([1, 1], [64, 64], 4, 2, 64, BF, 16, 0, 0, 64, "slot"),
}


@pytest.mark.parametrize("name", list(CASES))
def test_against_float64(name):
    rows, kv, Hq, Hkv, D, dt, page, W, S, L, order = CASES[name]
    b = Batch(rows, kv, Hq, Hkv, D, dt, page, W, S, L, seed=len(name), order=order).place()
    a = b.attention()
    for t in (a.out.out, a.out.lse):
        t.fill_(7.0)
    got = a.run()
    torch.cuda.synchronize()
    assert (got.req_status.cpu() == 0).all()
    check(b, got)


def test_many_requests_and_uneven_lengths():
    """More requests than workers, from one token to many tiles: items cut by the workers' borders."""
    g = torch.Generator().manual_seed(5)
    B = 300
    rows = torch.randint(0, 4, (B,), generator=g).tolist()
    kv = [r + int(x) for r, x in zip(rows, (torch.rand(B, generator=g) ** 6 * 2000).tolist())]
    b = Batch(rows, kv, 4, 2, 64, BF, 16, seed=3).place()
    got = b.attention().run()
    torch.cuda.synchronize()
    check(b, got)


def _ramp(dtype, D):
    """Scores that grow along the text, to far beyond a fixed reference's range, then fall."""
    b = Batch([3, 2], [700, 400], 4, 2, D, dtype, 16, seed=9)
    for i, kv in enumerate(b.kv):
        t = torch.linspace(0.0, 1.0, kv)
        up = torch.where(t < 0.7, t / 0.7, (1 - t) / 0.3)[:, None, None]
        b.keys[i] = (up * 12.0 * torch.ones(kv, b.Hkv, D) + 0.1 * b.keys[i].float()).to(dtype)
    b.q = (0.9 + 0.05 * b.q.float()).to(dtype)
    return b


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_growing_scores(dtype):
    b = _ramp(dtype, 128).place()
    got = b.attention().run()
    torch.cuda.synchronize()
    check(b, got)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("what", ["nan value", "inf value", "nan key", "inf key"])
def test_not_finite_where_only_later_rows_see_it(dtype, what):
    """The last positions' keys and values are not finite: rows before them are as if these did not
    exist, rows that see them get what the formula gives."""
    b = Batch([5, 2], [140, 130], 4, 2, 128, dtype, 16, seed=11)
    x = float("nan") if what.startswith("nan") else float("inf")
    clean = b.reference()
    for i in range(2):
        (b.vals if what.endswith("value") else b.keys)[i][-1, :, 3] = x
    b.place()
    got = b.attention().run()
    torch.cuda.synchronize()
    out, lse = got.out.cpu(), got.lse.cpu()
    last = [4, 6]
    keep = [t for t in range(7) if t not in last]
    want, wl = clean[0], clean[1]
    assert torch.isfinite(out[keep].float()).all()
    tol = clean[2][keep] * 2.0 ** -7
    assert ((out[keep].double() - want[keep]).abs() <= tol).all()
    assert ((lse[keep].double() - wl[keep]).abs() <= 1e-3).all()
    if what.endswith("value"):
        assert (~torch.isfinite(out[last][..., 3].float())).all()
        rest = [d for d in range(128) if d != 3]
        assert torch.isfinite(out[last][..., rest].float()).all()
        assert ((lse[last].double() - wl[last]).abs() <= 1e-3).all()
    elif what == "nan key":
        assert torch.isnan(out[last].float()).all() and torch.isnan(lse[last]).all()


def test_window_edge_not_finite():
    """A value just behind one row's window and inside the row before's."""
    W = 60
    b = Batch([4], [300], 4, 2, 64, BF, 16, window=W, seed=2)
    clean = b.reference()
    b.vals[0][300 - 4 - W + 1] = float("nan")  # the first row's oldest position, nobody else's
    b.place()
    got = b.attention().run()
    torch.cuda.synchronize()
    out = got.out.cpu().double()
    assert torch.isnan(out[0]).all()
    assert ((out[1:] - clean[0][1:]).abs() <= clean[2][1:] * 2.0 ** -7).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_requests_in_error_leave_the_others_alone(dtype):
    b = Batch([2, 3, 1, 2], [200, 300, 50, 90], 4, 2, 128, dtype, 16, seed=4).place()
    ref = b.reference()
    b.table[1, 5] = -1                 # a visible position without a page
    b.table[2, 1] = 10 ** 6            # an id outside the cache
    b.kv_len[3] = -3
    got = b.attention().run()
    torch.cuda.synchronize()
    assert got.req_status.tolist() == [0, 16, 16, 4]
    out, lse = got.out.cpu(), got.lse.cpu()
    assert (out[2:] == 0).all() and (lse[2:] == -math.inf).all()
    assert ((out[:2].double() - ref[0][:2]).abs() <= ref[2][:2] * 2.0 ** -7).all()
    b.kv_len[3] = 10 ** 6
    got = b.attention().run()
    torch.cuda.synchronize()
    assert got.req_status.tolist() == [0, 16, 16, 16] and (got.out[2:] == 0).all()


def test_shared_page_missing():
    b = Batch([2, 1], [100, 80], 4, 2, 64, BF, 16, shared=64, seed=4).place()
    b.shared_table[2] = -5
    got = b.attention().run()
    torch.cuda.synchronize()
    assert got.req_status.tolist() == [16, 16] and (got.out == 0).all()


def test_inconsistent_offsets():
    b = Batch([2, 3, 2], [60, 70, 80], 4, 2, 64, BF, 16, seed=4).place()
    b.row_off.copy_(torch.tensor([0, 5, 2, 7], dtype=torch.int32))
    got = b.attention().run()
    torch.cuda.synchronize()
    assert got.req_status.tolist()[1] == 4
    b.row_off.copy_(torch.tensor([0, 2, 5, 9], dtype=torch.int32))  # beyond the rows there are
    got = b.attention().run()
    torch.cuda.synchronize()
    assert got.req_status.tolist() == [0, 0, 4]


def test_shared_prefix_equals_own_pages():
    """A shared prefix is a way to compute, not another result: the same batch with every page in
    each request's own table agrees within the bounds."""
    b = Batch([3, 1, 4], [400, 350, 333], 8, 2, 128, BF, 16, shared=320, seed=6).place()
    got = b.attention().run()
    b.shared, keep = 0, b.shared_table
    b.place()
    alone = b.attention().run()
    torch.cuda.synchronize()
    ref = b.reference()
    check(b, got, ref)
    check(b, alone, ref)
    assert keep is not None


def test_runs_repeat_bit_for_bit_and_share_a_workspace():
    big = Batch([3, 5, 1], [900, 1300, 40], 8, 2, 128, BF, 16, seed=1).place()
    small = Batch([1, 2], [70, 300], 8, 2, 128, BF, 16, shared=64, seed=2).place()
    a, s = big.attention(), small.attention()
    if s.workspace.numel() > a.workspace.numel():
        a.workspace = s.workspace
    else:
        s.workspace = a.workspace
    x, y = [t.clone() for t in (a.run().out, s.run().out)]
    s.workspace.fill_(0xFF)
    for _ in range(3):
        assert torch.equal(a.run().out, x) and torch.equal(s.run().out, y)
    torch.cuda.synchronize()


def test_other_stream_and_graph():
    b = Batch([3, 5, 1], [900, 300, 40], 8, 2, 128, BF, 16, shared=32, seed=1).place()
    a = b.attention()
    want = a.run().out.clone()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    a.out.out.zero_()
    st.wait_stream(torch.cuda.current_stream())
    a.run(st)
    st.synchronize()
    assert torch.equal(a.out.out, want)
    a.out.out.zero_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.out.out, want)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_strided_rows_and_caches(dtype):
    """Queries inside a wider projection, outputs inside a wider row, keys and values in one tensor."""
    b = Batch([3, 2], [120, 300], 8, 2, 64, dtype, 16, seed=8).place()
    n = b.k_cache.shape[0]
    kv = torch.full((n, 2, 16, 2, 64), float("nan"), dtype=dtype, device="cuda")
    kv[:, 0], kv[:, 1] = b.k_cache, b.v_cache
    b.k_cache, b.v_cache = kv[:, 0], kv[:, 1]
    wide = torch.full((b.T, 12 * 64), float("nan"), dtype=dtype, device="cuda")
    wide[:, :8 * 64] = b.qd.flatten(1)
    b.qd = wide[:, :8 * 64].unflatten(1, (8, 64))
    a = b.attention()
    out = torch.full((b.T, 16 * 64), 5.0, dtype=dtype, device="cuda")
    a.bind(b.qd, b.k_cache, b.v_cache, b.row_off, b.kv_len, b.table, out=out[:, 8 * 64:].unflatten(1, (8, 64)))
    got = a.run()
    torch.cuda.synchronize()
    check(b, got)
    assert (out[:, :8 * 64] == 5.0).all()


@pytest.mark.parametrize("dtype,pages", [(BF, 270000), (F32, 270000)], ids=["bf16", "f32"])
def test_offsets_beyond_32_bits(dtype, pages):
    """Pages whose elements lie past 2^32 in the cache."""
    b = Batch([3], [100], 8, 8, 128, dtype, 16, seed=8).place(extra_pages=0)
    n = b.k_cache.shape[0]
    big = [torch.empty(pages, 16, 8, 128, dtype=dtype, device="cuda") for _ in range(2)]
    assert big[0].numel() > 2 ** 32
    for t, c in zip(big, (b.k_cache, b.v_cache)):
        t[:64].fill_(float("nan"))
        t[pages - n:] = c
    b.k_cache, b.v_cache = big
    b.table = torch.where((b.table >= 0) & (b.table < n), b.table + (pages - n), -1).int()
    got = b.attention().run()
    torch.cuda.synchronize()
    check(b, got)


def test_scale():
    b = Batch([3, 1], [100, 40], 4, 2, 64, BF, 16, seed=8)
    b.place()
    got = b.attention(scale=0.5 * 64 ** -0.5).run()
    torch.cuda.synchronize()
    b.q = b.q * 0.5
    check(b, got)
