"""GPU: spec_attend in bf16 with more rows than a round has, against float64 (tests/attend_ref.py): scores that
outgrow a softmax's reference, values that are not finite where only some rows see them, windows' edges,
strided tensors, workers' borders inside a text. "middle" keeps 40 rows of a head together in one request,
"many" some hundred, "across" has requests on both sides of an item's end."""
import pytest
import torch

from attend_ref import Batch, check

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
ROWS = {"middle": [10, 9], "many": [90, 33], "across": [65, 3, 64, 1, 127]}
FORM = {"middle": "spec_attend_round_kernel", "many": "spec_attend_pair_kernel", "across": "spec_attend_pair_kernel"}


def _run(b):
    a = b.attention()
    for t in (a.out.out, a.out.lse):
        t.fill_(7.0)
    got = a.run()
    torch.cuda.synchronize()
    assert (got.req_status.cpu() == 0).all()
    return got


def _tol(ref):
    """attend_ref.check's bound, for the elements that stay finite."""
    _, _, mag, ulps, nk = ref
    return mag * (2.0 ** -7 + 2 * ulps * 2.0 ** -22 + 2.0 ** -20 + nk * 2.0 ** -23)[..., None] + 1e-30


def _kv(rows, *more):
    return [n + more[i % len(more)] for i, n in enumerate(rows)]


@pytest.mark.parametrize("form", list(ROWS))
@pytest.mark.parametrize("D,page", [(128, 16), (64, 7), (96, 64), (80, 1)])
def test_against_float64(form, D, page):
    rows = ROWS[form]
    b = Batch(rows, _kv(rows, 300, 0, 129), 8, 2, D, BF, page, seed=D).place()
    check(b, _run(b))
    assert b.attention().plan() == FORM[form]


@pytest.mark.parametrize("form", list(ROWS))
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 140), (64, 4), (130, 0), (5000, 3)])
def test_windows(form, window, sinks):
    rows = ROWS[form]
    b = Batch(rows, _kv(rows, 400, 3), 8, 2, 128, BF, 16, window, sinks, seed=window, order="head").place()
    check(b, _run(b))


@pytest.mark.parametrize("shared", [128, 333])
def test_shared_prefix_of_requests_with_many_rows(shared):
    """Rows inside the prefix, at its end and behind it, in one batch."""
    rows = [40, 1, 80, 12]
    b = Batch(rows, [shared - 60, shared + 1, shared + 30, shared + 200], 8, 2, 64, BF, 16, 0, 0, shared, seed=5).place()
    check(b, _run(b))


@pytest.mark.parametrize("form", list(ROWS))
def test_growing_scores(form):
    """Scores that grow along the text, far beyond the slack of a reference, then fall."""
    rows = ROWS[form]
    b = Batch(rows, _kv(rows, 700, 300), 4, 1, 128, BF, 16, seed=9)
    for i, kv in enumerate(b.kv):
        t = torch.linspace(0.0, 1.0, kv)
        up = torch.where(t < 0.7, t / 0.7, (1 - t) / 0.3)[:, None, None]
        b.keys[i] = (up * 12.0 * torch.ones(kv, b.Hkv, 128) + 0.1 * b.keys[i].float()).to(BF)
    b.q = (0.9 + 0.05 * b.q.float()).to(BF)
    b.place()
    check(b, _run(b))


@pytest.mark.parametrize("form", list(ROWS))
@pytest.mark.parametrize("what", ["nan value", "inf value", "nan key", "inf key"])
@pytest.mark.parametrize("back", [1, 5])
def test_not_finite_where_only_later_rows_see_it(form, what, back):
    """One position near each text's end is not finite: rows before it do not see it, rows from it on get
    what the formula gives. The bound for the others is that of attend_ref.check."""
    rows, rest = ROWS[form], [d for d in range(128) if d != 3]
    b = Batch(rows, _kv(rows, 140, 37, 0), 8, 2, 128, BF, 16, seed=11)
    clean = b.reference()
    x = float("nan") if what.startswith("nan") else float("inf")
    for i in range(b.B):
        (b.vals if what.endswith("value") else b.keys)[i][-back, :, 3] = x
    sees = torch.tensor([j > b.rows[i] - 1 - back for i in range(b.B) for j in range(b.rows[i])])
    # a request with fewer rows than `back` has the position in every row's sight
    got = _run(b.place())
    out, lse = got.out.cpu(), got.lse.cpu()
    want, wl, tol = clean[0], clean[1], _tol(clean)
    assert torch.isfinite(out[~sees].float()).all() and torch.isfinite(lse[~sees]).all()
    assert ((out[~sees].double() - want[~sees]).abs() <= tol[~sees]).all()
    assert ((lse[~sees].double() - wl[~sees]).abs() <= 1e-3).all()
    if what.endswith("value"):
        assert (~torch.isfinite(out[sees][..., 3].float())).all()
        diff = (out[sees].double() - want[sees]).abs()[..., rest]
        assert (diff <= tol[sees][..., rest]).all()
        assert ((lse[sees].double() - wl[sees]).abs() <= 1e-3).all()
    elif what == "nan key":
        assert torch.isnan(out[sees].float()).all() and torch.isnan(lse[sees]).all()


@pytest.mark.parametrize("form", list(ROWS))
def test_window_edge_not_finite(form):
    """The first row's oldest position holds a value that is not finite; no other row sees it."""
    W, rows = 60, ROWS[form]
    b = Batch(rows, _kv(rows, 300, 100), 4, 1, 64, BF, 16, window=W, seed=2)
    clean = b.reference()
    for i in range(b.B):
        b.vals[i][b.kv[i] - rows[i] - W + 1] = float("nan")
    got = _run(b.place())
    out = got.out.cpu().double()
    first = torch.zeros(b.T, dtype=torch.bool)
    first[[b.off[i] for i in range(b.B)]] = True
    assert torch.isnan(out[first]).all()
    assert ((out[~first] - clean[0][~first]).abs() <= _tol(clean)[~first]).all()


@pytest.mark.parametrize("form", list(ROWS))
def test_strided_rows_and_caches(form):
    """Queries inside a wider projection, outputs inside a wider row, keys and values in one tensor."""
    rows = ROWS[form]
    b = Batch(rows, _kv(rows, 120, 300), 8, 2, 64, BF, 16, seed=8).place()
    n = b.k_cache.shape[0]
    kv = torch.full((n, 2, 16, 2, 64), float("nan"), dtype=BF, device="cuda")
    kv[:, 0], kv[:, 1] = b.k_cache, b.v_cache
    b.k_cache, b.v_cache = kv[:, 0], kv[:, 1]
    wide = torch.full((b.T, 12 * 64), float("nan"), dtype=BF, device="cuda")
    wide[:, :8 * 64] = b.qd.flatten(1)
    b.qd = wide[:, :8 * 64].unflatten(1, (8, 64))
    a = b.attention()
    out = torch.full((b.T, 16 * 64), 5.0, dtype=BF, device="cuda")
    a.bind(b.qd, b.k_cache, b.v_cache, b.row_off, b.kv_len, b.table, out=out[:, 8 * 64:].unflatten(1, (8, 64)))
    got = a.run()
    torch.cuda.synchronize()
    check(b, got)
    assert (out[:, :8 * 64] == 5.0).all()


def test_texts_longer_than_a_workers_share():
    """Items cut by the workers' borders many times over, joined: 2 heads' items over 152 workers."""
    b = Batch([60], [20000], 8, 2, 64, BF, 16, seed=21).place()
    a = b.attention()
    first = a.run()
    torch.cuda.synchronize()
    one, lse = first.out.clone(), first.lse.clone()
    check(b, first)
    again = a.run()
    torch.cuda.synchronize()
    assert torch.equal(one, again.out) and torch.equal(lse, again.lse)
