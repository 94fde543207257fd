"""Calls of the 8-bit cache's operators at the ends of their ranges: windows and sinks beyond every position, pages whose
scales are far apart, no rows at all, caches beyond 2^32 bytes, the same page in several places, many random batches bit
for bit."""
import math

import pytest
import torch
from cache8_ref import Batch8, check8

from speculative_decoding_verification_43_gb300 import api

pytestmark = pytest.mark.gpu
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
INT_MAX = 2 ** 31 - 1


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(INT_MAX, 0), (INT_MAX, INT_MAX), (7, INT_MAX)], ids=["window", "both", "sinks"])
@pytest.mark.parametrize("rows,shared,page,D", [([5, 2], 0, 16, 64), ([5, 2], 100, 16, 64), ([150, 90], 0, 16, 64),
                                                ([150, 90], 100, 16, 64), ([5, 2], 0, 5, 64)], ids=str)
def test_windows_beyond_every_position(rows, shared, page, D, window, sinks, dtype):
    """Every earlier position is visible, so the call without a window and sinks gives the same."""
    b = Batch8(rows, [400, 300], 4, 2, D, dtype, page, 0, 0, shared, seed=3).place()
    plain = b.attention().run()
    b.window, b.sinks = window, sinks
    wide = b.attention().run()
    torch.cuda.synchronize()
    assert torch.equal(wide.out, plain.out) and torch.equal(wide.lse, plain.lse)
    assert torch.equal(wide.req_status, plain.req_status)


class Apart(Batch8):
    """Pages whose values differ in magnitude, 2^-spread .. 2^spread."""
    spread = 10

    def quantise(self, c, x):
        f = 2.0 ** int(torch.randint(-self.spread, self.spread + 1, (1,), generator=self.g))
        return super().quantise(c, x * f if c == "v" else x)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows", [[5, 1, 3], [14, 15, 16], [150, 90, 200]], ids=str)
@pytest.mark.parametrize("odd", [False, True], ids=["powers of two", "odd"])
def test_pages_far_apart(rows, odd, dtype):
    b = Apart(rows, [300, 290, 270], 8, 2, 64, dtype, 16, seed=9, odd_scales=odd).place()
    got = b.attention().run()
    torch.cuda.synchronize()
    check8(b, got)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_no_rows(dtype):
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.empty(0, 4, 64, dtype=dtype, device="cuda")
    cache = torch.zeros(4, 16, 2, 64, dtype=torch.uint8, device="cuda").view(E4M3)
    scale = torch.ones(4, 2, device="cuda")
    got = api.attend8(q, cache, cache, scale, scale, torch.zeros(4, **i32), torch.tensor([0, 20, -1], **i32),
                      torch.zeros(3, 2, **i32))
    torch.cuda.synchronize()
    assert got.out.shape == (0, 4, 64) and got.req_status.tolist() == [0, 0, 4]


@pytest.mark.parametrize("order", ["slot", "head"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_cache_beyond_four_gigabytes(dtype, order):
    """The last pages of a cache of 2^32 bytes and more hold what the first ones of a small one do."""
    page, H, D, n = 64, 8, 128, 80
    many = 2 ** 32 // (page * H * D) + n
    g = torch.Generator(device="cuda").manual_seed(4)
    i32 = dict(dtype=torch.int32, device="cuda")
    T, kv = 10, [40 * page - 3, 39 * page + 10]
    row_off, kv_len = torch.tensor([0, 4, T], **i32), torch.tensor(kv, **i32)
    table = torch.randperm(n, generator=g, device="cuda").int().view(2, 40)
    qkv = torch.randn(T, 4 * H, D, generator=g, device="cuda").to(dtype)
    ang = torch.rand(kv[0], D // 2, generator=g, device="cuda") * 6
    cos_sin = torch.cat([ang.cos(), ang.sin()], 1)
    small = torch.randint(0, 0x78, (2, n, page, H, D), generator=g, device="cuda", dtype=torch.uint8)
    got = []
    for pages in (n, many):
        shape = (2, pages, page, H, D) if order == "slot" else (2, pages, H, page, D)
        cache = torch.empty(shape, dtype=torch.uint8, device="cuda")
        cache = cache if order == "slot" else cache.transpose(2, 3)
        cache[:, pages - n:] = small
        scale = torch.full((2, pages, H), 2.0 ** -7, device="cuda")
        kc, vc = cache.view(E4M3)
        at = table + (pages - n)
        q = api.kv_append8(qkv[:, :2 * H], qkv[:, 2 * H:3 * H], qkv[:, 3 * H:], cos_sin, row_off, kv_len, kc, vc, scale[0],
                           scale[1], at).q
        o = api.attend8(q, kc, vc, scale[0], scale[1], row_off, kv_len, at)
        torch.cuda.synchronize()
        assert (o.req_status == 0).all()
        got.append((q, o.out, o.lse, cache[:, pages - n:].clone(), scale[:, pages - n:].clone()))
        del cache, kc, vc
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows", [1, 5, 14, 100])
def test_a_page_in_several_places(rows):
    """Two requests that name one page for all their blocks: every block holds the same."""
    i32 = dict(dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    kc, vc = (torch.randint(0, 0x78, (3, 16, 2, 64), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2))
    ks, vs = (torch.rand(3, 2, generator=g, device="cuda") + 0.5 for _ in range(2))
    ks *= 2.0 ** -9
    q = torch.randn(2 * rows, 4, 64, generator=g, device="cuda")
    got = api.attend8(q, kc.view(E4M3), vc.view(E4M3), ks, vs, torch.tensor([0, rows, 2 * rows], **i32),
                      torch.full((2,), 20 * 16, **i32), torch.full((2, 20), 1, **i32))
    torch.cuda.synchronize()
    k, v = ((c.view(E4M3)[1].double() * s[1].double()[:, None]).repeat(20, 1, 1) for c, s in ((kc, ks), (vc, vs)))
    qd = q.double().view(2, rows, 2, 2, 64)
    z = torch.einsum("brhgd,xhd->brhgx", qd, k) * 64 ** -0.5
    pos = torch.arange(320 - rows, 320, device="cuda")
    z = z.masked_fill(torch.arange(320, device="cuda")[None, :] > pos[:, None, None, None], -math.inf)
    want = torch.einsum("brhgx,xhd->brhgd", torch.softmax(z, 4), v).reshape(2 * rows, 4, 64)
    # scores: 2^-19 of each element (64 of |q k| in all) and 64 additions of 2^-24; sums and weights alike
    mag = torch.einsum("brhgd,xhd->brhgx", qd.abs(), k.abs()).amax(4).reshape(2 * rows, 4, 1) * 64 ** -0.5
    vmax = v.abs().amax()
    assert ((got.out.double() - want).abs() <= vmax * (mag * 2.0 ** -17 + 2.0 ** -16)).all()


@pytest.mark.parametrize("seed", range(4))
def test_random_batches_bit_for_bit(seed):
    """A call gives the same bits each time, whichever waits its warps meet; and what fp32 rows give, to their
    roundings. Query elements lie between 2^-7 and 1 of 4, or are 0, which two e4m3 hold whole; four hold the fp32 rows'
    to 2^-19 of themselves. With |k| up to 448 2^-6 a score is at most 4 * 448 2^-6 * D^1/2 <= 317, and off by 317 (2^-19
    + 2^-22 for its sums): a weight by twice that, 2^-9.8, and by 2^-11 for its 16-bit float; together 2^-9 of the largest
    value. The output is rounded once, 2^-8 of itself."""
    r = torch.Generator().manual_seed(seed)

    def pick(a, b):
        return int(torch.randint(a, b + 1, (1,), generator=r))
    i32 = dict(dtype=torch.int32, device="cuda")
    for _ in range(60):
        D, page, Hkv, G = 16 * pick(1, 8), 8 * pick(1, 9), pick(1, 3), pick(1, 5)
        B, most = pick(1, 8), [2, 8, 40, 300][pick(0, 3)]
        rows = [pick(0, most) for _ in range(B)]
        kv = [n + (pick(0, 1500) if pick(0, 2) else 0) for n in rows]
        window, sinks = (pick(1, 300), pick(0, 5)) if pick(0, 1) else (0, 0)
        T, width = sum(rows), max(1, max((x + page - 1) // page for x in kv))
        pages = width * 2
        g = torch.Generator(device="cuda").manual_seed(pick(0, 10 ** 6))
        kc, vc = (torch.randint(0, 256, (pages, page, Hkv, D), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2))
        for c in (kc, vc):
            c[(c & 0x7f) == 0x7f] = 0
        ks, vs = (torch.exp2(torch.randint(-9, -5, (pages, Hkv), generator=g, device="cuda").float()) for _ in range(2))
        q = torch.randn(T, Hkv * G, D, generator=g, device="cuda").clamp(-4, 4)
        q = torch.where(q.abs() < 2.0 ** -5, 0.0, q).to(BF)
        off = [0]
        for n in rows:
            off.append(off[-1] + n)
        row_off, kv_len = torch.tensor(off, **i32), torch.tensor(kv, **i32)
        table = torch.randint(0, pages, (B, width), generator=g, device="cuda", dtype=torch.int32)
        more = dict(window=window, n_sink=sinks)
        args = (kc.view(E4M3), vc.view(E4M3), ks, vs, row_off, kv_len, table)
        first = api.attend8(q, *args, **more)
        again = [api.attend8(q, *args, **more) for _ in range(4)]
        wide = api.attend8(q.float(), *args, **more)
        torch.cuda.synchronize()
        assert (first.req_status == 0).all()
        for a in again:
            assert torch.equal(a.out, first.out) and torch.equal(a.lse, first.lse)
        vmax = float((vc.view(E4M3).float() * vs[:, None, :, None]).abs().amax()) if T else 0.0
        assert torch.isfinite(wide.out).all()
        off_by = (first.out.float() - wide.out).abs()
        assert (off_by <= wide.out.abs() * 2.0 ** -8 + vmax * 2.0 ** -9).all(), float(off_by.max() / max(vmax, 1e-30))
