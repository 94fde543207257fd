"""GPU: spec_attend8 where the pages' value scales differ as far as they may, 2^-60 .. 2^30, against float64: rows that
see a quiet page alone beside a loud one of the same tile, loud pages behind the window, softmax sums whose terms come
from quiet pages and outputs that come from loud ones, in one worker's tiles and in parts of several workers."""
import math

import pytest
import torch

from speculative_decoding_verification_43_gb300 import api

pytestmark = pytest.mark.gpu
BF, F32, E4M3, F64 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float64
PAGE, D, HKV, KSCALE = 16, 64, 2, 2.0 ** -3
# rows of two query heads a key head: the round kernel's items of 32 rows and of 64, the pair kernel; fp32: the first
KINDS = [(5, BF), (20, BF), (100, BF), (5, F32), (100, F32)]
NAMES = ["round", "round 64", "pair", "round f32", "many f32"]


class Texts:
    """B requests of `rows` rows on the same n positions, whose pages lie anywhere in the cache. level[x]: log2 of
    position x's weight, about; vlog[page]: log2 of the values' scale. The first query element is 8 and meets the key's level;
    the others are small, and held whole by two parts."""

    def __init__(self, B, rows, n, dtype, level, vlog, G=2, seed=0, adds=None):
        """adds: at most so many sums on the way of a weight into the row's sum; then keys have the level alone, to two
        elements' precision."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=F64)  # noqa: E731
        self.B, self.rows, self.n, self.dtype, self.G = B, rows, n, dtype, G
        pages = (n + PAGE - 1) // PAGE
        self.table = torch.randperm(pages, generator=g, device="cuda").int()
        key = rnd(pages * PAGE, HKV, D) * 0.125
        key[..., 0] = 0.0
        key[:n, :, 0] = torch.tensor([level(x) for x in range(n)], device="cuda", dtype=F64)[:, None] * math.log(2.0)
        if adds:
            at = key[..., 0].clone()
            key.zero_()
            key[..., 0] = (at / KSCALE).float().to(E4M3).to(F64) * KSCALE
            key[..., 1] = 8 * (at - key[..., 0])
        self.adds = adds
        kq, vq = (key / KSCALE).float().to(E4M3), (rnd(pages * PAGE, HKV, D) * 100).clamp(-448, 448).float().to(E4M3)
        vs = torch.tensor([[2.0 ** vlog(b)] * HKV for b in range(pages)], device="cuda", dtype=F64)
        self.K, self.V = kq.to(F64)[:n] * KSCALE, vq.to(F64)[:n] * vs.repeat_interleave(PAGE, 0)[:n, :, None]
        self.loudness = 448 * vs.repeat_interleave(PAGE, 0)[:n]
        place = self.table.long()
        self.kc, self.vc = (torch.zeros(pages, PAGE, HKV, D, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.vs = torch.zeros(pages, HKV, device="cuda")
        self.kc[place], self.vc[place] = (t.view(torch.uint8).view(pages, PAGE, HKV, D) for t in (kq, vq))
        self.vs[place] = vs.float()
        self.ks = torch.full((pages, HKV), KSCALE, device="cuda")
        q = rnd(B * rows, HKV * G, D).clamp(-4, 4) * 0.0625
        q = torch.where(q.abs() < 2.0 ** -8, 0.0, q).to(BF)
        q[..., 0], q[..., 1] = 8.0, 1.0
        self.q = q.to(dtype)

    def run(self, window=0, shared=0):
        i32 = dict(dtype=torch.int32, device="cuda")
        B, n = self.B, self.n
        got = api.attend8(self.q, self.kc.view(E4M3), self.vc.view(E4M3), self.ks, self.vs,
                          torch.arange(B + 1, **i32) * self.rows, torch.full((B,), n, **i32), self.table.repeat(B, 1), window=window,
                          shared_len=shared, shared_table=self.table[:(shared + PAGE - 1) // PAGE].clone() if shared else None)
        torch.cuda.synchronize()
        assert (got.req_status == 0).all()
        return got

    def check(self, got, window=0):
        """Bounds. Queries are held whole (fp32: to 2^-19), so a score is off by its additions: at most `ulps` * 2^-22, as
        in attend_ref.check, and a weight and the weights' sum by that each. A weight's logarithm is the sum of score,
        log2 of the scale and reference: three roundings of numbers below 2^8, 2^-17 each. The exponential unit adds 2^-21, the
        sums over n keys n 2^-24 each (or `adds`; a score of two products is off by the roundings of four numbers no larger). In bf16 a weight is a 16-bit float (2^-11 of itself), and the output is rounded, 2^-8.
        What the tensor cores add is cut off at 2^-24 of an instruction's largest product, and small weights at 2^-28 of the
        largest: fewer than n / 4 instructions, and n weights, so n 2^-26 of the largest contribution p * 448 * scale."""
        rows, n, scale = self.rows, self.n, D ** -0.5
        pos = torch.arange(n - rows, n, device="cuda")[:, None]
        x = torch.arange(n, device="cuda")[None]
        seen = ((x <= pos) & ((x > pos - window) if window else True))[:, None, None]
        nk = seen.sum(3)[..., None]
        for i in range(self.B):
            part = slice(i * rows, (i + 1) * rows)
            q = self.q[part].to(F64).view(rows, HKV, self.G, D)
            z = (torch.einsum("rhgd,xhd->rhgx", q, self.K) * scale).masked_fill(~seen, -math.inf)
            lse, p = torch.logsumexp(z, 3, keepdim=True), torch.softmax(z, 3)
            out, mag = (torch.einsum("rhgx,xhd->rhgd", p, v) for v in (self.V, self.V.abs()))
            most = (p * self.loudness.T[None, :, None]).amax(3, keepdim=True)
            ulps = torch.einsum("rhgd,xhd->rhgx", q.abs(), self.K.abs()).masked_fill(~seen, 0).amax(3, keepdim=True) * scale
            ulps = ulps * (4 if self.adds else D) + 4 * z.abs().masked_fill(~seen, 0).amax(3, keepdim=True)
            weight = 2 * ulps * 2.0 ** -22 + 3 * 2.0 ** -17 + 2.0 ** -20 + (self.adds or nk) * 2.0 ** -23
            tol = mag * weight + nk * 2.0 ** -26 * most + out.abs() * 2.0 ** -24
            if self.dtype == BF:
                tol = tol + mag * 2.0 ** -11 + out.abs() * 2.0 ** -8
            go, gl = got.out[part].to(F64).view_as(out), got.lse[part].to(F64).view_as(lse)
            bad = ~((go - out).abs() <= tol)
            assert not bad.any(), (i, int(bad.sum()), bad.nonzero()[:3].tolist(), float(((go - out).abs() / tol).max()))
            bad = ~((gl - lse).abs() <= weight + lse.abs() * 2.0 ** -22)
            assert not bad.any(), (i, int(bad.sum()), bad.nonzero()[:3].tolist(), float((gl - lse).abs().max()))


@pytest.mark.parametrize("apart", [26, 40, 90])
@pytest.mark.parametrize("rows,n,dtype", [(5, 18, BF), (20, 30, BF), (200, 200, BF), (300, 420, BF), (200, 200, F32)], ids=str)
def test_quiet_page_before_a_loud_one(rows, n, dtype, apart):
    """The rows that see the quiet page alone do not know of the loud one behind it in the same tile."""
    t = Texts(1, rows, n, dtype, lambda x: 0.25 * (x % 5), lambda b: 30 - apart if b % 8 == 0 else 30)
    first = max(0, n - rows)
    if first >= PAGE:  # (nobody sees it alone: the rows of the next page see it with that one)
        t = Texts(1, rows, n, dtype, lambda x: 0.25 * (x % 5), lambda b: 30 - apart if b < (n - 100) // PAGE else 30)
    t.check(t.run())


@pytest.mark.parametrize("rows,dtype", KINDS, ids=NAMES)
@pytest.mark.parametrize("window", [40, 100])
def test_loud_page_behind_the_window(rows, dtype, window):
    """Pages 9 and 14 are 2^50 louder than the others; rows whose window has left them behind, or that see them with
    hardly any weight, have the quiet values alone."""
    def level(x):
        return -80.0 if x // PAGE == 14 else 0.5 * (x % 3)
    n = max(rows + 60, 16 * 9 + 30 + window)
    t = Texts(1, rows, n, dtype, level, lambda b: 30 if b in (9, 14) else -20, seed=1)
    t.check(t.run(window), window)


@pytest.mark.parametrize("rows,dtype", KINDS, ids=NAMES)
@pytest.mark.parametrize("low", [-30, -60])
def test_what_positions_contribute(rows, dtype, low):
    """Weights as far apart as the scales, the other way round: every position contributes to the output alike."""
    r = torch.Generator().manual_seed(5)
    vlog = [int(torch.randint(low, 31, (1,), generator=r)) for _ in range(40)]
    vlog[7], vlog[8], vlog[20] = low, 30, low
    t = Texts(20, rows, 640, dtype, lambda x: -float(vlog[x // PAGE]), lambda b: vlog[b], seed=3)
    t.check(t.run())
@pytest.mark.parametrize("rows,dtype", KINDS, ids=NAMES)
@pytest.mark.parametrize("loud", ["first", "last"])
@pytest.mark.parametrize("level", [-7.0, -18.0, -30.0])
@pytest.mark.parametrize("many", [True, False], ids=["one worker", "workers"])
def test_sums_from_quiet_pages(many, level, loud, rows, dtype):
    """One position of a page at scale 2^30 and all others, 2^level of its weight each, at 2^-60: the output is the
    first's, the softmax sum is nearly the others'. Many requests on the same positions give a worker several tiles each; one request
    over 20000 positions falls to many workers."""
    B, n = (80 if rows == 100 else 300, 1000) if many else (1, 20000)
    at = 3 if loud == "first" else n - 3
    page = at // PAGE

    def weight(x):
        return 0.0 if x == at else -50.0 if x // PAGE == page else level
    t = Texts(B, rows, n, dtype, weight, lambda b: 30 if b == page else -60, seed=2)
    t.check(t.run())




@pytest.mark.parametrize("rows,dtype", KINDS, ids=NAMES)
def test_sums_of_parts_far_below(rows, dtype):
    """The parts of 400000 positions at 2^-60, beside one at 2^30 that outweighs each of them 2^29 times and more: a part's
    reference, which its first tile sets, lies 2^126 below that one's, its sum counts. A worker has 1 / 75 of the positions at
    most (two items, 152 workers or more), and adds 64 or fewer at a time; 512 parts and steps of a tile's own sum beside."""
    n = 400000
    t = Texts(1, rows, n, dtype, lambda x: (0.0 if x == 3 else -50.0 if x < PAGE else -36.6 if x // 128 % 2 == 0 else -29.0),
              lambda b: 30 if b == 0 else -60, seed=4, adds=n // 75 // 64 + 512)
    t.check(t.run())


@pytest.mark.parametrize("rows,dtype", KINDS, ids=NAMES)
@pytest.mark.parametrize("loud", ["prefix", "own"])
@pytest.mark.parametrize("level", [-7.0, -18.0])
def test_loud_page_on_one_side_of_the_prefix(level, loud, rows, dtype):
    """Quiet positions and the loud one in a shared prefix and behind it, whose parts other kernels may leave."""
    n, shared = 1100, 505
    at = 40 if loud == "prefix" else 900
    t = Texts(20, rows, n, dtype, lambda x: 0.0 if x == at else -50.0 if x // PAGE == at // PAGE else level,
              lambda b: 30 if b == at // PAGE else -60, seed=6)
    t.check(t.run(shared=shared))
