"""spec_attend8's queries, which enter the tensor cores in parts of 8 bits: quiet channels beside a loud one, and what the
last part holds. On the CPU: the bounds see a part that is missing or of the wrong type."""
import math

import pytest
import torch

from speculative_decoding_verification_43_gb300 import api

BF, F32, E4M3, E5M2, F64 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e5m2, torch.float64
PAGE, HKV, G = 16, 2, 2


def in_parts(q, types):
    """q [.., D] as the sum of its parts, after division by the power of two that brings the largest between 224 and 448:
    each part is the nearest to what the ones before leave; from the third on to 2^8 times that."""
    top = q.abs().amax(-1, keepdim=True).to(F64)
    s = torch.exp2(torch.ceil(torch.log2(top / 448)))
    y, total = q.to(F64) / s, 0.0
    for i, t in enumerate(types):
        by = 256.0 if i >= 2 else 1.0
        p = (y * by).float().to(t).to(F64) / by
        total, y = total + p, y - p
    return total * s


def loud_channel(rows, D, loud, seed=1):
    """bf16 queries whose first element is 2^loud, the others 1 .. 2, against keys that have nothing there."""
    g = torch.Generator().manual_seed(seed)
    q = (1 + torch.rand(rows, HKV * G, D, generator=g, dtype=F64)).to(BF)
    q[..., 0] = 2.0 ** loud
    n = rows + 150
    kq = (0.5 + 0.5 * torch.rand(n, HKV, D, generator=g, dtype=F64)).mul(64).float().to(E4M3)
    kq[..., 0] = 0
    return q, kq, 2.0 ** -6


def last_part(rows, D, seed=2):
    """fp32 queries whose elements are all one value, of which three parts of four leave much: that adds up over a head."""
    g = torch.Generator().manual_seed(seed)
    x = (1 + torch.rand(20000, 1, generator=g)).to(F32)
    left = ((x.to(F64) - in_parts(x, [E4M3] * 3)) / x.to(F64)).squeeze(1)
    few = left.argsort(descending=True)[:rows * HKV * G]
    q = x[few].view(rows, HKV * G, 1).expand(-1, -1, D).contiguous()
    n = rows + 150
    kq = (0.5 + 0.5 * torch.rand(n, HKV, D, generator=g, dtype=F64)).mul(64).float().to(E4M3)
    return q, kq, 2.0 ** -5


def scores(q, K):
    rows, D = q.shape[0], q.shape[2]
    z = torch.einsum("rhgd,xhd->rhgx", q.to(F64).view(rows, HKV, G, D), K) * D ** -0.5
    seen = torch.arange(K.shape[0])[None] <= torch.arange(K.shape[0] - rows, K.shape[0])[:, None]
    return z.masked_fill(~seen[:, None, None], -math.inf)


def off_by(lse, z, held):
    """lse against the scores', in units of its bound. All products have one sign, so that a score's roundings are counted
    in it. A query element is off by 2^-19 of itself (fp32) or by nothing; an instruction of 32 products cuts sums off at
    2^-23 of the score, and there are 16 at most (4 parts, 128 elements; twice that is allowed); factors and scale are three
    roundings of 2^-24, the exponential and the logarithm 2^-20 together, reference and logarithm of the scale roundings of
    numbers below 64, 2^-18 each; the weights' sum over fewer than 512 keys, in fewer than 64 steps, 2^-18."""
    top = z.amax(-1)
    bound = top * ((0.0 if held else 2.0 ** -19) + 32 * 2.0 ** -23 + 3 * 2.0 ** -24) + 2.0 ** -20 + 3 * 2.0 ** -18
    return float(((lse.to(F64) - torch.logsumexp(z, -1)).abs() / bound).max())


@pytest.mark.parametrize("D", [64, 128])
def test_the_bound_sees_a_missing_part(D):
    q, kq, ks = last_part(20, D)
    K = kq.to(F64) * ks
    z = scores(q, K)
    for n, ok in ((4, True), (3, False), (2, False)):
        assert (off_by(torch.logsumexp(scores(in_parts(q, [E4M3] * n), K), -1), z, False) < 1) == ok, n


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("loud", [12, 14])
def test_the_bound_sees_quiet_channels(D, loud):
    q, kq, ks = loud_channel(20, D, loud)
    K = kq.to(F64) * ks
    z = scores(q, K)
    for types, ok in (([E4M3, E5M2], True), ([E4M3, E4M3], False), ([E4M3], False)):
        assert (off_by(torch.logsumexp(scores(in_parts(q, types), K), -1), z, True) < 1) == ok, types


def run(q, kq, ks):
    """lse of one request's last rows; pages in any order."""
    rows, (n, _, D) = q.shape[0], kq.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    pages = (n + PAGE - 1) // PAGE
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(0))
    cache = torch.zeros(pages, PAGE, HKV, D, dtype=torch.uint8)
    flat = torch.zeros(pages * PAGE, HKV, D, dtype=torch.uint8)
    flat[:n] = kq.view(torch.uint8)
    cache[table] = flat.view(pages, PAGE, HKV, D)
    cache = cache.cuda().view(E4M3)
    one = torch.ones(pages, HKV, device="cuda")
    got = api.attend8(q.cuda(), cache, cache, one * ks, one, torch.tensor([0, rows], **i32), torch.tensor([n], **i32),
                      table.int().cuda()[None])
    torch.cuda.synchronize()
    assert (got.req_status == 0).all()
    return got.lse.cpu().view(rows, HKV, G)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [5, 20, 100])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("loud", [12, 14])
def test_quiet_channels_beside_a_loud_one(loud, D, rows):
    q, kq, ks = loud_channel(rows, D, loud)
    assert off_by(run(q, kq, ks), scores(q, kq.to(F64) * ks), True) < 1


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [5, 100])
@pytest.mark.parametrize("D", [64, 128])
def test_four_parts_of_an_fp32_query(D, rows):
    q, kq, ks = last_part(rows, D)
    assert off_by(run(q, kq, ks), scores(q, kq.to(F64) * ks), False) < 1
