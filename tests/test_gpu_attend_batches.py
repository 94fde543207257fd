"""GPU: spec_attend on batches of other shapes, against float64 (tests/attend_ref.py): more requests than a
CTA's warps walk at once, prompts and single tokens in one batch, values that are not finite inside and behind a
shared prefix and in parts whose weight vanishes when they are joined."""
import pytest
import torch

from attend_ref import Batch, check

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
TYPES = pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])


def _run(b):
    a = b.attention()
    for t in (a.out.out, a.out.lse):
        t.fill_(7.0)
    got = a.run()
    torch.cuda.synchronize()
    assert (got.req_status.cpu() == 0).all()
    return got


def _tol(b, ref):
    """attend_ref.check's bound, for the elements that stay finite."""
    _, _, mag, ulps, nk = ref
    unit = 2.0 ** -7 if b.dtype == BF else 0.0
    return mag * (unit + 2 * ulps * 2.0 ** -22 + 2.0 ** -20 + nk * 2.0 ** -23)[..., None] + 1e-30


@TYPES
@pytest.mark.parametrize("shared", [0, 37])
def test_more_than_a_thousand_requests(dtype, shared):
    g = torch.Generator().manual_seed(8)
    B = 1100
    rows = torch.randint(0, 3, (B,), generator=g).tolist()
    kv = [shared + r + int(x) for r, x in zip(rows, torch.randint(0, 60, (B,), generator=g).tolist())]
    b = Batch(rows, kv, 4, 2, 64, dtype, 16, shared=shared, seed=3).place()
    check(b, _run(b))


@TYPES
@pytest.mark.parametrize("shared", [0, 130])
@pytest.mark.parametrize("rows", [[1] * 40 + [300] + [5] * 6, [3, 200, 1, 1, 90]], ids=["rounds", "prompts"])
def test_prompts_and_rounds_in_one_batch(dtype, shared, rows):
    kv = [shared + n + 17 * (i % 13) for i, n in enumerate(rows)]
    b = Batch(rows, kv, 8, 2, 64, dtype, 16, shared=shared, seed=len(rows)).place()
    check(b, _run(b))


@TYPES
@pytest.mark.parametrize("rows,kv", [([4, 2, 3], [100, 201, 250]), ([8] * 12, [100] + [205 + 7 * i for i in range(11)])],
                         ids=["few", "many"])
@pytest.mark.parametrize("x", [50, 98, 199])
def test_not_finite_inside_a_shared_prefix(dtype, rows, kv, x):
    """Position x of the prefix has a value that is not finite: rows before it are as if it did not exist."""
    b = Batch(rows, kv, 8, 2, 64, dtype, 16, shared=200, seed=4)
    ref = b.reference()
    b.pv[x, :, 5] = float("nan")
    got = _run(b.place())
    pos = torch.tensor([b.kv[i] - n + j for i, n in enumerate(rows) for j in range(n)])
    sees, rest = pos >= x, [d for d in range(64) if d != 5]
    assert sees.any()
    out, lse, tol = got.out.cpu().double(), got.lse.cpu().double(), _tol(b, ref)
    assert ((out[~sees] - ref[0][~sees]).abs() <= tol[~sees]).all()
    assert torch.isnan(out[sees][..., 5]).all()
    assert ((out[sees] - ref[0][sees]).abs() <= tol[sees])[..., rest].all()
    assert ((lse - ref[1]).abs() <= 1e-3).all()


@TYPES
@pytest.mark.parametrize("back", [1, 3])
def test_not_finite_behind_a_shared_prefix(dtype, back):
    """A position of the requests' own text, seen by their last rows only."""
    rows = [4, 5, 12, 3]
    b = Batch(rows, [n + 150 + 40 * i for i, n in enumerate(rows)], 8, 2, 64, dtype, 16, shared=140, seed=4)
    ref = b.reference()
    for i in range(b.B):
        b.vals[i][-back, :, 5] = float("inf")
    got = _run(b.place())
    sees, rest = torch.tensor([j >= n - back for n in rows for j in range(n)]), [d for d in range(64) if d != 5]
    out, tol = got.out.cpu().double(), _tol(b, ref)
    assert ((out[~sees] - ref[0][~sees]).abs() <= tol[~sees]).all()
    assert (~torch.isfinite(out[sees][..., 5])).all()
    assert ((out[sees] - ref[0][sees]).abs() <= tol[sees])[..., rest].all()


@TYPES
@pytest.mark.parametrize("shared", [0, 4000])
@pytest.mark.parametrize("rows", [2, 12, 200])
def test_not_finite_in_a_part_of_vanishing_weight(dtype, rows, shared):
    """The first half of the text scores 2^184 times less than the second, so that parts taken over it count for
    nothing in 32 bits. A value there that is not a number reaches its column all the same, as 0 times it does in
    a text that is not cut; the other columns are the formula's."""
    n = 9000
    b = Batch([rows], [n], 4, 1, 64, dtype, 16, shared=shared, seed=21)
    b.keys[0] = torch.where(torch.arange(n) < n // 2, -8.0, 8.0)[:, None, None].expand(n, 1, 64).to(dtype).contiguous()
    b.pk = b.keys[0][:shared]
    b.q = torch.ones_like(b.q)
    ref = b.reference()
    (b.pv if shared else b.vals[0])[100, :, 3] = float("nan")
    got = _run(b.place())
    out, rest = got.out.cpu().double(), [d for d in range(64) if d != 3]
    assert torch.isnan(out[..., 3]).all()
    assert ((out - ref[0]).abs() <= _tol(b, ref))[..., rest].all()


@TYPES
def test_every_visible_page_is_checked(dtype):
    """One bad entry of a table with 1500 (pages of one slot), at ends and in the middle; the request next to it
    is served. Entries behind the window and past the text may be anything."""
    n = 1500
    whole = Batch([2, 1], [n, 40], 2, 1, 64, dtype, 1, seed=2).place()
    cut = Batch([2, 1], [n, 40], 2, 1, 64, dtype, 1, 300, 5, seed=2).place()
    for b, seen in ((whole, range(n)), (cut, [*range(5), *range(n - 2 - 300 + 1, n)])):
        a = b.attention()
        good = a.run().out.clone()
        assert a.out.req_status.tolist() == [0, 0]
        for x in (0, 4, 5, 31, 32, 511, 512, 513, 543, 1023, 1024, 1197, 1198, 1199, 1230, 1498, 1499, 1500):
            for bad in (-1, b.k_cache.shape[0]):
                keep = b.table[0, x].item()
                b.table[0, x] = bad
                a.run()
                torch.cuda.synchronize()
                assert a.out.req_status.tolist() == [16 if x in seen else 0, 0], x
                assert torch.equal(a.out.out[2:], good[2:])
                assert (a.out.out[:2] == 0).all() if x in seen else torch.equal(a.out.out, good)
                b.table[0, x] = keep
