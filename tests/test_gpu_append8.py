"""GPU: spec_kv_append8 against float64: scales of new pages and of pages that hold earlier tokens, elements
brought to a larger scale, rotation forms and widths, types, cache orders, strides that leave 16-byte boundaries,
padding rows, positions without a page, values that are not finite; everything else in the cache keeps its
bits."""
import math

import pytest
import torch
from cache8_ref import E4M3, least_scale
from test_gpu_append import CASES, close, turned

from speculative_decoding_verification_43_gb300 import api

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def make(rows, kv, Hq, Hkv, D, dtype, page, rot, order="slot", seed=0, pad=0, n_pos=None, spread=2.0):
    """As in test_gpu_append; every request's rows differ in magnitude, and earlier tokens' scales too."""
    g = torch.Generator().manual_seed(seed)
    T, B = sum(rows), len(rows)
    width = max(1, max((max(x, 0) + page - 1) // page for x in kv))
    n_pages = B * width + 2
    table = torch.randperm(n_pages, generator=g)[:B * width].view(B, width).int()
    n = (Hq + 2 * Hkv) * D + pad
    loud = torch.exp2(torch.randn(T, 1, generator=g) * spread)
    qkv = (torch.randn(T, n, generator=g) * loud).to(dtype).cuda()
    cut = [Hq * D, (Hq + Hkv) * D, (Hq + 2 * Hkv) * D]
    q = qkv[:, :cut[0]].unflatten(1, (Hq, D)) if Hq else None
    k, v = (qkv[:, a:b].unflatten(1, (Hkv, D)) for a, b in zip(cut, cut[1:]))
    shape = (n_pages, Hkv, page, D) if order == "head" else (n_pages, page, Hkv, D)
    bits = [torch.randint(0, 256, shape, generator=g, dtype=torch.uint8) for _ in range(2)]
    bits = [torch.where((b & 127) == 127, 0, b).to(torch.uint8).cuda() for b in bits]
    if order == "head":
        bits = [b.permute(0, 2, 1, 3) for b in bits]
    scales = [torch.exp2(torch.randint(-12, 4, (n_pages, Hkv), generator=g).float()).cuda() for _ in range(2)]
    ang = torch.rand(n_pos or max([1, *kv]), max(rot // 2, 1), generator=g, dtype=torch.float64) * 6.3
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    off = [0]
    for r in rows:
        off.append(off[-1] + r)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(q=q, k=k, v=v, cos_sin=cs, row_off=i32(off), kv_len=i32(kv), k_cache=bits[0].view(E4M3),
                v_cache=bits[1].view(E4M3), k_scale=scales[0], v_scale=scales[1], block_table=table.cuda()), off


def saved(a):
    return {n: a[n].view(torch.uint8).clone().cpu() if a[n].dtype == E4M3 else a[n].clone().cpu()
            for n in ("k_cache", "v_cache", "k_scale", "v_scale")}


def between(got, lo, hi):
    """Elements (bytes) between the roundings of two float64 values: rounding is monotonous."""
    x = got.view(E4M3).float()
    a, b = (t.clamp(-448, 448).float().to(E4M3).float() for t in (lo, hi))
    return ((x >= a) & (x <= b)).all()


def verify(a, off, rows, kv, page, rot, interleaved, out, before, skip=()):
    """Against the definition, page by page. A turned value may be off by 2^-22 of the magnitudes that enter; the
    scale is that of an amax within these bounds, and the elements are checked under the scale found."""
    cs, table = a["cos_sin"].cpu(), a["block_table"].cpu()
    after = saved(a)
    rows_cpu = {c: a[c].cpu() for c in "qkv" if a.get(c) is not None}
    expect = {n: t.clone() for n, t in before.items()}
    for i, n in enumerate(rows):
        first = max(kv[i] - n, 0)
        new = {}
        for j in range(n):
            p, t = kv[i] - n + j, off[i] + j
            if p < 0 or (i, j) in skip:
                continue
            new.setdefault(p // page, []).append((p, t))
            if out is not None:
                y, mag = turned(rows_cpu["q"][t], cs[p] if rot else None, rot, interleaved)
                assert close(out[t].cpu(), y, mag), (i, j)
        for blk, pts in new.items():
            pid = int(table[i, blk])
            kept = max(first - blk * page, 0)
            for c in "kv":
                vals = []
                for p, t in pts:
                    vals.append(turned(rows_cpu[c][t], cs[p], rot, interleaved) if c == "k" and rot else
                                (rows_cpu[c][t].double(), torch.zeros(1, dtype=torch.float64)))
                y = torch.stack([v[0] for v in vals])
                err = torch.stack([v[1].expand_as(v[0]) for v in vals]) * 2.0 ** -22
                fin = torch.where(torch.isfinite(y), y.abs(), 0.0)
                for h in range(y.shape[1]):
                    got = float(after[c + "_scale"][pid, h])
                    old = float(before[c + "_scale"][pid, h]) if kept else 0.0
                    ends = [max(least_scale(float((fin[:, h] + s * err[:, h]).clamp_min(0).max())), old) for s in (-1, 0, 1)]
                    assert got in ends, (i, blk, c, h, got, ends)
                    expect[c + "_scale"][pid, h] = got
                    for (p, _), yy, ee in zip(pts, y[:, h], err[:, h]):
                        e = after[c + "_cache"][pid, p % page, h]
                        ok = torch.isfinite(yy)
                        assert between(e[ok], ((yy - ee) / got)[ok], ((yy + ee) / got)[ok]), (i, blk, c, h, p)
                        assert ((e[~ok] & 127) == 127).all()
                        expect[c + "_cache"][pid, p % page, h] = e
                    if kept and got != old:
                        was = before[c + "_cache"][pid, :kept, h].view(E4M3).double()
                        expect[c + "_cache"][pid, :kept, h] = (was * (old / got)).float().to(E4M3).view(torch.uint8)
    for n in before:
        assert torch.equal(after[n], expect[n]), n


@pytest.mark.parametrize("name", list(CASES))
def test_against_float64(name):
    rows, kv, Hq, Hkv, D, dt, page, rot, inter, order, pad = CASES[name]
    a, off = make(rows, kv, Hq, Hkv, D, dt, page, rot, order, seed=len(name), pad=pad)
    before = saved(a)
    o = api.kv_append8(**a, rot_dim=rot, interleaved=inter)
    torch.cuda.synchronize()
    assert (o.req_status.cpu() == 0).all()
    verify(a, off, rows, kv, page, rot, inter, o.q if Hq else None, before)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("D,rot,pad", [(64, 64, 0), (128, 32, 0), (36, 20, 1), (512, 512, 0)], ids=str)
def test_more_rows_than_a_page_has_slots(D, rot, pad, inter, dtype):
    """Every form of the kernel for prompts; their queries in place."""
    rows, kv = [50, 1, 33], [60, 5, 33]
    a, off = make(rows, kv, 3, 2, D, dtype, 16, rot, seed=D + inter, pad=pad)
    before, q0 = saved(a), a["q"].cpu()
    o = api.kv_append8(**a, rot_dim=rot, interleaved=inter, q_out=a["q"])
    torch.cuda.synchronize()
    assert o.q.data_ptr() == a["q"].data_ptr()
    verify({**a, "q": q0}, off, rows, kv, 16, rot, inter, o.q, before)


@pytest.mark.parametrize("page", [1, 2, 5, 8, 24, 128])
def test_page_sizes(page):
    rows, kv = [9, 1, 130, 3], [70, 128, 200, 3]
    a, off = make(rows, kv, 2, 3, 48, BF, page, 48, seed=page)
    before = saved(a)
    api.kv_append8(**a)
    torch.cuda.synchronize()
    verify(a, off, rows, kv, page, 48, False, None, before)


def test_zeros_small_and_large_values():
    """Pages of zeros, of the smallest and of the largest values, and an earlier page that is louder."""
    rows, kv = [2, 2, 2, 2, 1], [2, 2, 2, 18, 20]
    a, off = make(rows, kv, 1, 1, 16, BF, 16, 0, seed=4)
    k = a["k"]
    k[0:2] = 0.0
    k[2:4] = 1e-38
    k[4:6] = 3.3e38
    k[6:8] = 448.0
    a["k_scale"][a["block_table"][4, 1].long()] = 2.0 ** 20
    before = saved(a)
    api.kv_append8(**a, rot_dim=0)
    torch.cuda.synchronize()
    verify(a, off, rows, kv, 16, 0, False, None, before)
    t = a["block_table"].cpu()
    s = a["k_scale"].cpu()
    assert s[t[0, 0]] == 2.0 ** -60 and s[t[1, 0]] == 2.0 ** -60
    assert s[t[3, 1]] == 1.0 and s[t[4, 1]] == 2.0 ** 20


def test_not_finite():
    rows, kv = [4, 3], [20, 3]
    a, off = make(rows, kv, 2, 2, 32, F32, 16, 0, seed=6)
    a["k"][1, 0, 5], a["k"][5, 1, :] = math.nan, math.inf
    a["v"][2, 1, 31], a["v"][4:, 0, :] = -math.inf, math.nan
    before = saved(a)
    o = api.kv_append8(**a, rot_dim=0)
    torch.cuda.synchronize()
    assert (o.req_status.cpu() == 0).all()
    verify(a, off, rows, kv, 16, 0, False, None, before)
    assert a["v_scale"][a["block_table"][1, 0].long(), 0] == 2.0 ** -60


def test_scale_that_is_no_power_of_two_stays():
    rows, kv = [2], [21]
    a, off = make(rows, kv, 1, 2, 16, F32, 16, 0, seed=8)
    pid = a["block_table"][0, 1].long()
    a["k_scale"][pid] = torch.tensor([0.3, 1e-6], device="cuda")
    before = saved(a)
    a["k"].clamp_(-20, 20)
    api.kv_append8(**a, rot_dim=0)
    torch.cuda.synchronize()
    verify(a, off, rows, kv, 16, 0, False, None, before)
    assert a["k_scale"][pid, 0] == before["k_scale"][pid.cpu(), 0]


def test_again_is_the_same():
    """The same rows once more: a page's scale has what it needs, the elements stay."""
    rows, kv = [5, 3], [41, 70]
    a, off = make(rows, kv, 4, 2, 64, BF, 16, 64, seed=3)
    c = api.KvAppender8(2, 8, 4, 2, 64, BF)
    c.bind(a["q"], a["k"], a["v"], a["cos_sin"], a["row_off"], a["kv_len"], a["k_cache"], a["v_cache"], a["k_scale"],
           a["v_scale"], a["block_table"])
    c.run()
    torch.cuda.synchronize()
    once = saved(a)
    c.run()
    torch.cuda.synchronize()
    for n, t in saved(a).items():
        assert torch.equal(t, once[n]), n


def test_refused_drafts_are_written_over():
    """A round of five rows whose last three are refused, then a round at their positions: what stays is the two
    accepted rows, under a scale that no refused row lowers."""
    a, off = make([5], [25], 2, 2, 32, BF, 16, 0, seed=12)
    api.kv_append8(**a, rot_dim=0)
    torch.cuda.synchronize()
    before = saved(a)
    b, off2 = make([4], [26], 2, 2, 32, BF, 16, 0, seed=13)
    for n in ("k_cache", "v_cache", "k_scale", "v_scale", "block_table"):
        b[n] = a[n]
    api.kv_append8(**b, rot_dim=0)
    torch.cuda.synchronize()
    verify(b, off2, [4], [26], 16, 0, False, None, before)


def test_errors_of_one_request_leave_the_others():
    rows, kv = [2, 3, 2, 2, 1], [40, 35, 37, 500, -3]
    a, off = make(rows, [40, 35, 37, 48, 3], 4, 2, 64, BF, 16, 64, n_pos=64)
    a["kv_len"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
    t = a["block_table"]
    t[1, 2] = -1     # request 1: positions 32.. have no page
    before = saved(a)
    o = api.kv_append8(**a, rot_dim=64)
    torch.cuda.synchronize()
    assert o.req_status.cpu().tolist() == [0, 16, 0, 4 | 16, 4]
    skip = {(1, j) for j in range(3)} | {(3, j) for j in range(2)} | {(4, 0)}
    verify(a, off, rows, [40, 35, 37, 48, 3], 16, 64, False, None, before, skip)


def test_rows_of_nobody_and_offsets_out_of_order():
    a, off = make([2, 2, 2, 2], [40, 35, 37, 48], 4, 2, 64, BF, 16, 64)
    a["row_off"] = torch.tensor([1, 3, 99, 5, 7], dtype=torch.int32, device="cuda")  # rows 0 and 7 are nobody's
    before = saved(a)
    q0 = torch.full_like(a["q"].contiguous(), 9.0)
    o = api.kv_append8(**a, q_out=q0.clone())
    torch.cuda.synchronize()
    assert o.req_status.cpu().tolist() == [0, 4, 4, 0]
    skip = {(1, 0), (1, 1), (2, 0), (2, 1)}
    verify(a, [1, 3, 5, 5], [2, 2, 2, 2], [40, 35, 37, 48], 16, 64, False, None, before, skip)
    assert (o.q[[0, 3, 4, 7]] == 9.0).all()


def test_no_rows():
    a, off = make([0, 0], [5, 0], 2, 2, 32, BF, 16, 32)
    before = saved(a)
    o = api.kv_append8(**a)
    torch.cuda.synchronize()
    assert (o.req_status.cpu() == 0).all()
    for n, t in saved(a).items():
        assert torch.equal(t, before[n]), n
