"""GPU: spec_attend8 against float64 (tests/cache8_ref.py has the reference and the bounds): spec_attend's
lengths, sizes, layouts, windows and prefixes over a cache in e4m3, scales of all magnitudes, elements and scales
that are no numbers in places nobody sees."""
import math

import pytest
import torch
from cache8_ref import Batch8, check8
from test_gpu_attend import CASES as ATTEND_CASES

from speculative_decoding_verification_43_gb300 import api

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32

CASES = {n: c for n, c in ATTEND_CASES.items() if c[4] % 16 == 0}


@pytest.mark.parametrize("name", list(CASES))
def test_against_float64(name):
    rows, kv, Hq, Hkv, D, dt, page, W, S, L, order = CASES[name]
    b = Batch8(rows, kv, Hq, Hkv, D, dt, page, W, S, L, seed=len(name), order=order).place()
    a = b.attention()
    for t in (a.out.out, a.out.lse):
        t.fill_(7.0)
    got = a.run()
    torch.cuda.synchronize()
    assert (got.req_status.cpu() == 0).all()
    check8(b, got)
    again = [t.clone() for t in (got.out, got.lse)]
    got = a.run()
    torch.cuda.synchronize()
    assert torch.equal(got.out, again[0]) and torch.equal(got.lse, again[1])


# rows, kv, Hq, Hkv, D, page, window, sinks, shared, order
MORE = {
    "a long text cut up": ([5], [20000], 16, 8, 64, 16, 0, 0, 0, "slot"),
    "a long text, one head": ([2], [9000], 4, 1, 128, 8, 0, 0, 0, "head"),
    "three heads": ([3, 7], [500, 1200], 6, 3, 128, 16, 0, 0, 0, "slot"),
    "six heads": ([3, 7], [500, 1200], 12, 6, 64, 32, 0, 0, 0, "head"),
    "sixteen heads": ([3, 1], [300, 700], 16, 16, 64, 16, 0, 0, 0, "slot"),
    "33 to 64 rows a head": ([12, 9, 16], [600, 1000, 300], 8, 2, 128, 16, 0, 0, 0, "slot"),
    "33 to 64 rows, window": ([12, 9, 16], [600, 1000, 300], 8, 2, 80, 24, 130, 7, 0, "head"),
    "rows between": ([8, 7, 6, 5, 4, 3, 2, 1], [130 * i for i in range(1, 9)], 12, 4, 96, 16, 0, 0, 0, "slot"),
    "prompts of 1000 rows": ([1000, 300], [1100, 300], 4, 1, 128, 64, 0, 0, 0, "slot"),
    "prompts, heads of 80": ([300, 260], [500, 260], 8, 2, 80, 24, 0, 0, 0, "head"),
    "prompts, window and sinks": ([400, 100], [900, 100], 4, 2, 64, 16, 150, 20, 0, "slot"),
    "prompts behind a prefix": ([170, 100], [370, 300], 4, 2, 128, 16, 0, 0, 150, "slot"),
    "rounds behind a prefix": ([4] * 40, [1100 + 11 * i for i in range(40)], 32, 8, 128, 16, 0, 0, 1001, "slot"),
    "pages of 128": ([4, 2], [1000, 130], 8, 2, 128, 128, 0, 0, 0, "slot"),
    "pages of 40": ([4, 2], [1000, 130], 8, 2, 128, 40, 0, 0, 0, "slot"),
}


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", list(MORE))
def test_layouts(name, dtype):
    rows, kv, Hq, Hkv, D, page, W, S, L, order = MORE[name]
    b = Batch8(rows, kv, Hq, Hkv, D, dtype, page, W, S, L, seed=len(name), order=order).place()
    got = b.attention().run()
    torch.cuda.synchronize()
    assert (got.req_status.cpu() == 0).all()
    check8(b, got)


@pytest.mark.parametrize("rows,kernel", [([4], "round"), ([12], "round"), ([13], "pair"), ([100], "pair")], ids=str)
def test_plan_names_the_kernel(rows, kernel):
    b = Batch8(rows, [200], 8, 2, 64, BF, 16, seed=1).place()
    assert b.attention().plan() == f"spec_attend8_{kernel}_kernel"
    assert Batch8(rows, [200], 8, 2, 64, F32, 16, seed=1).place().attention().plan() == "spec_attend8_round_kernel"
    for page, D in ((7, 64), (16, 144)):
        for dtype in (BF, F32):
            b = Batch8(rows, [200], 8, 2, D, dtype, page, seed=1).place()
            assert b.attention().plan() == "spec_attend_fma_kernel"


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("loud", [0.0, 12.0], ids=["alike", "apart"])
def test_scales(dtype, loud):
    """Scales that are no powers of two, and heads whose magnitudes are far apart."""
    b = Batch8([5, 2, 1], [300, 130, 17], 8, 4, 128, dtype, 16, seed=21, odd_scales=True, loud=loud).place()
    got = b.attention().run()
    torch.cuda.synchronize()
    check8(b, got)


def test_many_requests_and_uneven_lengths():
    g = torch.Generator().manual_seed(5)
    B = 300
    rows = torch.randint(0, 4, (B,), generator=g).tolist()
    kv = [r + int(x) for r, x in zip(rows, (torch.rand(B, generator=g) ** 6 * 2000).tolist())]
    b = Batch8(rows, kv, 4, 2, 64, BF, 16, seed=3).place()
    got = b.attention().run()
    torch.cuda.synchronize()
    check8(b, got)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows", [[3, 2], [20, 22], [40, 70], [300, 1]], ids=str)
def test_growing_scores(dtype, rows):
    """Scores that grow along the text, far beyond a fixed reference's range, then fall; the values' scales fall
    and grow."""
    b = Batch8(rows, [700, 400], 4, 2, 128, dtype, 16, seed=9)
    _reshape(b, lambda t: torch.where(t < 0.7, t / 0.7, (1 - t) / 0.3) * 12.0, lambda t: torch.exp2(20.0 * (t - 0.5).abs()))
    b.q = (0.9 + 0.05 * b.q.float()).to(dtype)
    b.place()
    got = b.attention().run()
    torch.cuda.synchronize()
    check8(b, got)


def _reshape(b, key_level, value_scale):
    """Keys about key_level(t) in every element, values times value_scale(t), t = 0 .. 1 along each text."""
    g = torch.Generator().manual_seed(1)
    for i, kv in enumerate(b.kv):
        t = torch.linspace(0.0, 1.0, kv, dtype=torch.float64)[:, None, None]
        k = key_level(t) + 0.1 * torch.randn(kv, b.Hkv, b.D, generator=g, dtype=torch.float64)
        v = value_scale(t) * torch.randn(kv, b.Hkv, b.D, generator=g, dtype=torch.float64)
        b.loud = {c: torch.ones(b.Hkv) for c in "kv"}
        for c, whole, x in (("k", b.keys, k), ("v", b.vals, v)):
            for a in range(0, kv, b.page):
                e, s = b.own8[i][c][a] = b.quantise(c, x[a:a + b.page])
                whole[i][a:a + b.page] = e.to(torch.float64) * s.to(torch.float64)[:, None]


def test_one_heavy_position_and_a_long_tail():
    """One position that outweighs each of the others 2^15 times, and 20000 others that together weigh half of it:
    what each of them adds must not vanish."""
    b = Batch8([1, 3], [20000, 6000], 4, 1, 64, BF, 16, seed=2)
    for i, kv in enumerate(b.kv):
        x = torch.zeros(kv, 1, 64, dtype=torch.float64)
        x[2] = math.log(2.0 ** 15) / 8 / 1.0   # 64 elements of 1 in q: score = 64 x / 8
        v = torch.ones(kv, 1, 64, dtype=torch.float64)
        v[2] = -1.0
        b.loud = {c: torch.ones(1) for c in "kv"}
        for c, whole, y in (("k", b.keys, x), ("v", b.vals, v)):
            for a in range(0, kv, b.page):
                e, s = b.own8[i][c][a] = b.quantise(c, y[a:a + b.page])
                whole[i][a:a + b.page] = e.to(torch.float64) * s.to(torch.float64)[:, None]
    b.q = torch.ones_like(b.q)
    b.place()
    got = b.attention().run()
    torch.cuda.synchronize()
    check8(b, got)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows", [[5, 2], [21, 20], [150, 40]], ids=str)
@pytest.mark.parametrize("what", ["value", "key"])
def test_no_number_where_only_later_rows_see_it(dtype, rows, what):
    kv = [rows[0] + 135, rows[1] + 128]
    b = Batch8(rows, kv, 4, 2, 128, dtype, 16, seed=11)
    clean = b.reference()
    for i in range(2):
        a = (kv[i] - 1) // 16 * 16
        b.own8[i]["v" if what == "value" else "k"][a][0].view(torch.uint8)[-1, :, 3] = 0x7f if i else 0xff
    b.place()
    got = b.attention().run()
    torch.cuda.synchronize()
    out, lse = got.out.cpu(), got.lse.cpu()
    last = [rows[0] - 1, sum(rows) - 1]
    keep = [t for t in range(sum(rows)) if t not in last]

    class Part:
        pass
    part, kept = Part(), Part()
    part.dtype, kept.out, kept.lse = dtype, out[keep], lse[keep]
    check8(part, kept, [t[keep] for t in clean])
    if what == "value":
        assert torch.isnan(out[last][..., 3].float()).all()
        assert torch.isfinite(out[last][..., [d for d in range(128) if d != 3]].float()).all()
        assert ((lse[last].double() - clean[1][last]).abs() <= 1e-3).all()
    else:
        assert torch.isnan(out[last].float()).all() and torch.isnan(lse[last]).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows", [[5], [13], [150], [400]], ids=str)
def test_scale_that_is_no_number_spoils_those_who_see_it(rows, dtype):
    """The page of the last positions: rows before them are as if it did not exist."""
    n = rows[0]
    b = Batch8(rows, [160 + n], 4, 2, 64, dtype, 16, seed=5)
    clean = b.reference()
    b.place()
    first = (160 + n - 1) // 16 * 16           # the last page's first position
    page = int(b.table[0, first // 16])
    for t in (b.k_scale, b.v_scale):
        t[page] = math.nan
    got = b.attention().run()
    torch.cuda.synchronize()
    keep = [t for t in range(n) if 160 + t < first]

    class Part:
        pass
    part, kept = Part(), Part()
    part.dtype, kept.out, kept.lse = dtype, got.out.cpu()[keep], got.lse.cpu()[keep]
    check8(part, kept, [t[keep] for t in clean])


def test_window_edge_no_number():
    W = 60
    b = Batch8([4], [300], 4, 2, 64, BF, 16, window=W, seed=2)
    clean = b.reference()
    x = 300 - 4 - W + 1                        # the first row's oldest position, nobody else's
    b.own8[0]["v"][x // 16 * 16][0].view(torch.uint8)[x % 16] = 0x7f
    b.place()
    got = b.attention().run()
    torch.cuda.synchronize()
    assert torch.isnan(got.out[0].float()).all()

    class Part:
        pass
    part, kept = Part(), Part()
    part.dtype, kept.out, kept.lse = BF, got.out.cpu()[1:], got.lse.cpu()[1:]
    check8(part, kept, [t[1:] for t in clean])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows", [[3], [100]], ids=str)
def test_queries_that_are_not_finite(rows, dtype):
    """A head of one row: that head's output is no number, the others are as before."""
    b = Batch8(rows, [200], 4, 2, 64, dtype, 16, seed=6)
    ref = b.reference()
    b.place()
    b.qd[1, 2, 7] = math.inf
    b.qd[2, 0, 0] = math.nan
    got = b.attention().run()
    torch.cuda.synchronize()
    out = got.out.cpu()
    assert torch.isnan(out[1, 2].float()).all() and torch.isnan(out[2, 0].float()).all()
    ok = torch.ones(rows[0], 4, dtype=torch.bool)
    ok[1, 2] = ok[2, 0] = False

    class Part:
        pass
    part, kept = Part(), Part()
    part.dtype, kept.out, kept.lse = dtype, out[ok], got.lse.cpu()[ok]
    check8(part, kept, [t[ok] if t.shape[1] == 4 else t.expand(-1, 4)[ok] for t in ref])


def test_errors_of_one_request_leave_the_others():
    b = Batch8([2, 3, 2, 1, 2], [40, 35, 200, 60, 33], 4, 2, 64, BF, 16, seed=7).place()
    ref = b.reference()
    b.table[1, 1] = -1
    b.kv_len[2] = -5
    b.kv_len[3] = 10 ** 6
    a = b.attention()
    a.out.out.fill_(3.0)
    got = a.run()
    torch.cuda.synchronize()
    assert got.req_status.cpu().tolist() == [0, 16, 4, 16, 0]
    assert (got.out[2:8] == 0).all() and (got.lse[2:8] == -math.inf).all()
    keep = [0, 1, 8, 9]

    class Part:
        pass
    part, kept = Part(), Part()
    part.dtype, kept.out, kept.lse = BF, got.out.cpu()[keep], got.lse.cpu()[keep]
    check8(part, kept, [t[keep] for t in ref])


def test_long_sums_of_one_sign_in_fp32():
    """Values of one sign and even weights over a long text, in fp32, 96 requests on the same pages, so that a worker
    has some 70 tiles: an accumulator that cuts every sum off instead of rounding it would be off by 2^-15. The sum of
    n weighted values in groups that are added up in turn may be off by the additions' cuts and roundings, fewer than
    64 on the way of each value (a group's instructions, the groups' sums and the workers', whose errors go both
    ways), 2^-24 each, and by the weights': together 2^-17."""
    n, B, D, page = 30000, 96, 64, 16
    g = torch.Generator().manual_seed(1)
    pages = n // page
    kc, vc = (torch.randint(0x28, 0x40, (pages, page, 1, D), generator=g, dtype=torch.uint8) for _ in range(2))
    ks, vs = (torch.exp2(torch.randint(-1, 2, (pages, 1), generator=g).float()) for _ in range(2))
    q = torch.randn(B, 2, D, generator=g) * 0.01
    K, V = ((c.view(torch.float8_e4m3fn).float() * s[:, :, None, None]).double().view(n, D) for c, s in ((kc, ks), (vc, vs)))
    z = q.double() @ K.T * D ** -0.5
    want, lse = torch.softmax(z, 2) @ V, torch.logsumexp(z, 2)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.arange(pages, **i32).repeat(B, 1)
    got = api.attend8(q.cuda(), kc.cuda().view(torch.float8_e4m3fn), vc.cuda().view(torch.float8_e4m3fn), ks.cuda(), vs.cuda(),
                      torch.arange(B + 1, **i32), torch.full((B,), n, **i32), table)
    torch.cuda.synchronize()
    assert (got.req_status == 0).all()
    assert ((got.out.cpu().double() - want).abs() <= want.abs() * 2.0 ** -17).all()
    assert ((got.lse.cpu().double() - lse).abs() <= lse.abs() * 2.0 ** -17).all()
