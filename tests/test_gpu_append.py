"""GPU: spec_kv_append against float64: rotation forms and widths, types, cache orders, strides that
leave 16-byte boundaries, padding rows, positions without a page or a table row; everything else in the
cache keeps its bits."""
import pytest
import torch

from speculative_decoding_verification_43_gb300 import api

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def make(rows, kv, Hq, Hkv, D, dtype, page, rot, order="slot", seed=0, pad=0, n_pos=None):
    g = torch.Generator().manual_seed(seed)
    T, B = sum(rows), len(rows)
    width = max(1, max((max(x, 0) + page - 1) // page for x in kv))
    n_pages = B * width + 2
    table = torch.randperm(n_pages, generator=g)[:B * width].view(B, width).int()
    n = (Hq + 2 * Hkv) * D + pad
    qkv = torch.randn(T, n, generator=g).to(dtype).cuda()
    cut = [Hq * D, (Hq + Hkv) * D, (Hq + 2 * Hkv) * D]
    q = qkv[:, :cut[0]].unflatten(1, (Hq, D)) if Hq else None
    k, v = (qkv[:, a:b].unflatten(1, (Hkv, D)) for a, b in zip(cut, cut[1:]))
    shape = (n_pages, Hkv, page, D) if order == "head" else (n_pages, page, Hkv, D)
    kc, vc = (torch.randn(*shape, generator=g).to(dtype).cuda() for _ in range(2))
    if order == "head":
        kc, vc = kc.permute(0, 2, 1, 3), vc.permute(0, 2, 1, 3)
    ang = torch.rand(n_pos or max([1, *kv]), rot // 2, generator=g, dtype=torch.float64) * 6.3
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    off = [0]
    for r in rows:
        off.append(off[-1] + r)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(q=q, k=k, v=v, cos_sin=cs, row_off=i32(off), kv_len=i32(kv), k_cache=kc, v_cache=vc,
                block_table=table.cuda()), off


def turned(x, cs, rot, interleaved):
    """One row [H][D] in float64, pair by pair; and the sum of the magnitudes that enter."""
    y, mag = x.double().clone(), x.double().abs()
    for c in range(rot // 2):
        a, b = (2 * c, 2 * c + 1) if interleaved else (c, c + rot // 2)
        co, si = cs[c].double(), cs[rot // 2 + c].double()
        xa, xb = x[:, a].double(), x[:, b].double()
        y[:, a], y[:, b] = xa * co - xb * si, xb * co + xa * si
        mag[:, a], mag[:, b] = (xa * co).abs() + (xb * si).abs(), (xb * co).abs() + (xa * si).abs()
    return y, mag


def close(got, y, mag):
    """The products and their sum in 32 bits may be off by 2^-22 of the magnitudes; rounding to the
    type is monotonous, so the result lies between the roundings of that interval's ends."""
    lo, hi = ((y + s * mag * 2.0 ** -22).to(got.dtype) for s in (-1.0, 1.0))
    return ((got >= lo) & (got <= hi)).all()


def verify(a, off, rows, kv, page, rot, interleaved, out, before, skip=()):
    kc, vc = (t.cpu() for t in before)
    cs, table = a["cos_sin"].cpu(), a["block_table"].cpu()
    kw, km = kc.double(), torch.zeros(kc.shape, dtype=torch.float64)
    for i, n in enumerate(rows):
        for j in range(n):
            p, t = kv[i] - n + j, off[i] + j
            if p < 0 or (i, j) in skip:
                continue
            y, mag = turned(a["k"][t].cpu(), cs[p] if rot else None, rot, interleaved)
            at = (int(table[i, p // page]), p % page)
            kw[at], km[at], vc[at] = y, mag, a["v"][t].cpu()
            if out is not None:
                y, mag = turned(a["q"][t].cpu() if a["q0"] is None else a["q0"][t], cs[p] if rot else None, rot,
                                interleaved)
                assert close(out[t].cpu(), y, mag), (i, j)
    assert torch.equal(a["v_cache"].cpu(), vc)
    assert close(a["k_cache"].cpu(), kw, km)


# rows, kv, Hq, Hkv, D, dtype, page, rot, interleaved, order, pad
CASES = {
    "one row": ([1], [1], 1, 1, 64, BF, 16, 64, False, "slot", 0),
    "one round": ([5], [1005], 32, 8, 128, BF, 16, 128, False, "slot", 0),
    "ragged": ([1, 8, 0, 3], [40, 8, 17, 1000], 6, 2, 96, BF, 24, 96, False, "head", 0),
    "ragged f32": ([1, 8, 0, 3], [40, 8, 17, 1000], 6, 2, 80, F32, 7, 80, False, "slot", 0),
    "interleaved": ([3, 2], [60, 70], 4, 2, 128, BF, 16, 128, True, "slot", 0),
    "interleaved, half, f32": ([3, 2], [60, 70], 4, 2, 128, F32, 16, 64, True, "head", 0),
    "part of the head": ([3, 2], [60, 70], 4, 2, 128, BF, 16, 64, False, "slot", 0),
    "part, off the vectors": ([3, 2], [60, 70], 4, 2, 80, BF, 16, 40, False, "slot", 0),
    "interleaved, off the vectors": ([3, 2], [60, 70], 4, 2, 80, BF, 16, 6, True, "slot", 0),
    "rows off the vectors": ([3, 2], [60, 70], 4, 2, 64, BF, 16, 64, False, "slot", 3),
    "rows off the vectors f32": ([3, 2], [60, 70], 4, 2, 64, F32, 16, 64, True, "slot", 1),
    "odd heads": ([3, 2], [60, 70], 3, 1, 33, BF, 16, 32, False, "slot", 0),
    "no rotation": ([3, 2], [60, 70], 4, 2, 64, BF, 16, 0, False, "slot", 0),
    "no queries": ([3, 2], [60, 70], 0, 2, 64, BF, 16, 64, False, "slot", 0),
    "padding rows": ([5, 3, 2], [3, 0, 2], 4, 2, 64, BF, 16, 64, False, "slot", 0),
    "prompts": ([700, 1, 300], [700, 20, 555], 4, 2, 64, BF, 16, 64, False, "slot", 0),
    "many requests": ([2] * 1100, [2 + i % 50 for i in range(1100)], 2, 1, 16, BF, 16, 16, False, "slot", 0),
}


@pytest.mark.parametrize("name", list(CASES))
def test_against_float64(name):
    rows, kv, Hq, Hkv, D, dt, page, rot, inter, order, pad = CASES[name]
    a, off = make(rows, kv, Hq, Hkv, D, dt, page, rot, order, seed=len(name), pad=pad)
    before = a["k_cache"].clone(), a["v_cache"].clone()
    o = api.kv_append(**a, rot_dim=rot, interleaved=inter)
    torch.cuda.synchronize()
    assert (o.req_status.cpu() == 0).all()
    a["q0"] = None
    verify(a, off, rows, kv, page, rot, inter, o.q if Hq else None, before)


def test_queries_in_place():
    rows, kv = [3, 2], [60, 70]
    a, off = make(rows, kv, 4, 2, 64, BF, 16, 64)
    before, q0 = (a["k_cache"].clone(), a["v_cache"].clone()), a["q"].cpu()
    o = api.kv_append(**a, q_out=a["q"])
    torch.cuda.synchronize()
    assert o.q.data_ptr() == a["q"].data_ptr()
    a["q0"] = q0
    verify(a, off, rows, kv, 16, 64, False, o.q, before)


def test_positions_without_a_page_or_a_table_row():
    rows, kv = [4, 4, 3, 2, 2], [50, 64, 70, 40, 33]
    a, off = make(rows, kv, 4, 2, 64, BF, 16, 64, n_pos=69)
    a["block_table"][0, 2] = -1             # positions 46, 47 of request 0
    a["block_table"][3, 2] = 10 ** 6        # positions 38, 39 of request 3
    a["kv_len"][4] = 16 * 5 + 1             # its last row lies beyond the table's five blocks
    kv[4] = 81
    before = a["k_cache"].clone(), a["v_cache"].clone()
    out = torch.full((sum(rows), 4, 64), 9.0, dtype=BF, device="cuda")
    o = api.kv_append(**a, q_out=out)
    torch.cuda.synchronize()
    assert a["block_table"].shape[1] == 5
    # request 2's last row has no table row; request 4's rows are past both
    assert o.req_status.tolist() == [16, 0, 4, 16, 20]
    skip = [(0, 0), (0, 1), (2, 2), (3, 0), (3, 1), (4, 0), (4, 1)]
    a["q0"] = None
    verify_rows = [(i, j) for i, n in enumerate(rows) for j in range(n) if (i, j) in skip]
    for i, j in verify_rows:
        assert (o.q[off[i] + j] == 9.0).all()
        o.q[off[i] + j] = 0
    verify(a, off, rows, kv, 16, 64, False, o.q, before, skip=skip)


def test_inconsistent_offsets_write_nothing():
    a, _ = make([2, 2, 2], [20, 30, 40], 4, 2, 64, BF, 16, 64)
    a["row_off"].copy_(torch.tensor([0, 2, 1, 99], dtype=torch.int32))
    a["kv_len"][0] = -1
    before = a["k_cache"].clone(), a["v_cache"].clone()
    o = api.kv_append(**a)
    torch.cuda.synchronize()
    assert o.req_status.tolist() == [4, 4, 4]
    assert torch.equal(a["k_cache"], before[0]) and torch.equal(a["v_cache"], before[1])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_offsets_beyond_32_bits(dtype):
    pages = 270000
    a, off = make([3], [40], 8, 8, 128, dtype, 16, 128)
    big = [torch.zeros(pages, 16, 8, 128, dtype=dtype, device="cuda") for _ in range(2)]
    n = a["k_cache"].shape[0]
    for t, c in zip(big, (a["k_cache"], a["v_cache"])):
        t[pages - n:] = c
    small = a["block_table"].clone()
    a["k_cache"], a["v_cache"] = big
    a["block_table"] = small + (pages - n)
    before = big[0][pages - n:].clone(), big[1][pages - n:].clone()
    o = api.kv_append(**a)
    torch.cuda.synchronize()
    assert not big[0][:pages - n].any()
    a["k_cache"], a["v_cache"], a["block_table"], a["q0"] = big[0][pages - n:], big[1][pages - n:], small, None
    verify(a, off, [3], [40], 16, 128, False, o.q, before)


def test_other_stream():
    a, _ = make([3, 2], [60, 70], 4, 2, 64, BF, 16, 64)
    want = api.kv_append(**a).q.clone()
    k = a["k_cache"].clone()
    a["k_cache"].zero_()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    o = api.kv_append(**a, stream=st)
    st.synchronize()
    assert torch.equal(o.q, want)
    for p in (57, 58, 59):
        page = int(a["block_table"][0, p // 16])
        assert torch.equal(a["k_cache"][page, p % 16], k[page, p % 16])
