"""GPU: rounds over the 8-bit cache as a server runs them: block tables brought to the round's lengths, rows
appended, attended to, some refused, their pages given back. The cache is followed on the CPU by its definition
(no rotation, so that every element is exact) and the attention's outputs by float64 on what it stands for. The
same captured into a graph and replayed; the example with its cache in 8 bits."""
import os
import sys

import pytest
import torch
from cache8_ref import E4M3, least_scale

from speculative_decoding_verification_43_gb300 import api
from test_gpu_tables import blocks

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


class Server:
    """B requests over a pool of pages; what each page holds by the definition, in `sim`."""

    def __init__(self, B, Hq, Hkv, D, page, n_pages, width, dtype, seed=0):
        self.B, self.Hq, self.Hkv, self.D, self.page, self.n_pages, self.dtype = B, Hq, Hkv, D, page, n_pages, dtype
        self.g = torch.Generator().manual_seed(seed)
        i32 = dict(dtype=torch.int32, device="cuda")
        order = torch.randperm(n_pages, generator=self.g)
        self.pool = dict(n_blocks=torch.zeros(B, **i32), block_table=torch.full((B, width), -1, **i32),
                         free_pages=order.to(**i32), n_free=torch.tensor([n_pages], **i32))
        nan = torch.full((n_pages, page, Hkv, D), 0x7f, dtype=torch.uint8)
        self.kc, self.vc = nan.cuda().view(E4M3), nan.cuda().view(E4M3)
        self.ks, self.vs = (torch.full((n_pages, Hkv), float("nan"), device="cuda") for _ in range(2))
        self.sim = {c: (torch.zeros(n_pages, page, Hkv, D), torch.zeros(n_pages, Hkv)) for c in "kv"}
        self.length = [0] * B

    def rows(self, n):
        T = sum(n)
        loud = torch.exp2(torch.randn(T, 1, 1, generator=self.g) * 2)
        q = torch.randn(T, self.Hq, self.D, generator=self.g).to(self.dtype)
        k, v = ((torch.randn(T, self.Hkv, self.D, generator=self.g) * loud).to(self.dtype) for _ in range(2))
        return q, k, v

    def inputs(self, n):
        off = [0]
        for c in n:
            off.append(off[-1] + c)
        i32 = dict(dtype=torch.int32, device="cuda")
        kv = [x + c for x, c in zip(self.length, n)]
        return torch.tensor(off, **i32), torch.tensor(kv, **i32), off, kv

    def follow(self, n, kv, off, k, v, table):
        for i, c in enumerate(n):
            first = kv[i] - c
            for blk in range(first // self.page, blocks(kv[i], self.page)):
                a, b = max(first, blk * self.page), min(kv[i], (blk + 1) * self.page)
                if a >= b:
                    continue
                pid, kept = int(table[i, blk]), a - blk * self.page
                for name, x in (("k", k), ("v", v)):
                    e, s = self.sim[name]
                    new = x[off[i] + a - first:off[i] + b - first].float()
                    for h in range(self.Hkv):
                        scale = max(least_scale(float(new[:, h].abs().max())), float(s[pid, h]) if kept else 0.0)
                        e[pid, :kept, h] = (e[pid, :kept, h] * (float(s[pid, h]) / scale)).to(E4M3).float()
                        e[pid, kept:kept + b - a, h] = (new[:, h] / scale).to(E4M3).float()
                        s[pid, h] = scale

    def check(self, n, kv, off, q, table, out, lse):
        for i, c in enumerate(n):
            at = torch.arange(kv[i])
            pid, slot = table[i].long()[at // self.page], at % self.page
            for c_, cache, scale in (("k", self.kc, self.ks), ("v", self.vc, self.vs)):
                e, s = self.sim[c_]
                assert torch.equal(cache.float().cpu()[pid, slot], e[pid, slot]), (i, c_)
                assert torch.equal(scale.cpu()[pid], s[pid]), (i, c_)
            K, V = ((self.sim[c_][0][pid, slot] * self.sim[c_][1][pid][:, :, None]).to(F64) for c_ in "kv")
            G = self.Hq // self.Hkv
            K, V = K.repeat_interleave(G, 1), V.repeat_interleave(G, 1)
            rows = slice(off[i], off[i] + c)
            z = torch.einsum("ihd,jhd->hij", q[rows].to(F64), K) * self.D ** -0.5
            z.masked_fill_(at > torch.arange(kv[i] - c, kv[i])[:, None], -torch.inf)
            p = torch.softmax(z, 2)
            want, mag = torch.einsum("hij,jhd->ihd", p, V), torch.einsum("hij,jhd->ihd", p, V.abs())
            # as in check8, with the scores' and the queries' errors (2^-18 of a head's largest element each) bounded together
            cut = (q[rows].to(F64).abs().amax(2) * K.abs().sum(2).amax(0) * self.D ** -0.5)[..., None]
            big = 0.0 if self.dtype == F32 else 1.0
            tol = want.abs() * 2.0 ** (-8 if big else -23) + mag * (big * 2.0 ** -11 + cut * 2.0 ** (-17 if big else -20) + 2.0 ** -16)
            tol = tol + big * V.abs().amax() * kv[i] * 2.0 ** -22
            assert ((out[rows].cpu().to(F64) - want).abs() <= tol).all(), i
            assert ((lse[rows].cpu().to(F64) - torch.logsumexp(z, 2).T).abs() <= (cut[..., 0] * 2.0 ** -17 + 2.0 ** -15)).all()


@pytest.mark.parametrize("dtype,page,D", [(BF, 16, 128), (BF, 8, 64), (F32, 16, 64), (BF, 5, 32)], ids=str)
def test_rounds(dtype, page, D):
    s = Server(4, 8, 2, D, page, 400, 80, dtype, seed=page)
    no_turn = torch.zeros(1, 0, device="cuda")
    for rnd in range(5):
        # the prompts, then rounds; a request pauses now and then
        n = [37, 5, 90, 1] if rnd == 0 else [int(x) for x in torch.randint(0, 6, (4,), generator=s.g)]
        q, k, v = s.rows(n)
        ro, kvl, off, kv = s.inputs(n)
        t = api.block_tables(kvl, *s.pool.values(), page, row_off=ro, total_rows=sum(n))
        a = api.kv_append8(q.cuda(), k.cuda(), v.cuda(), no_turn, ro, kvl, s.kc, s.vc, s.ks, s.vs, s.pool["block_table"], rot_dim=0)
        o = api.attend8(a.q, s.kc, s.vc, s.ks, s.vs, ro, kvl, s.pool["block_table"])
        torch.cuda.synchronize()
        for x in (t, a, o):
            assert (x.req_status == 0).all()
        table = s.pool["block_table"].cpu()
        assert s.pool["n_blocks"].tolist() == [blocks(x, page) for x in kv]
        held = [int(p) for i in range(4) for p in table[i, :blocks(kv[i], page)]]
        assert len(set(held)) == len(held) and set(held).isdisjoint(s.pool["free_pages"].tolist()[:int(s.pool["n_free"])])
        for i in range(4):
            for j in range(n[i]):
                p = kv[i] - n[i] + j
                assert int(t.slot_map[off[i] + j]) == int(table[i, p // page]) * page + p % page
        assert torch.equal(a.q.cpu(), q)
        s.follow(n, kv, off, k, v, table)
        s.check(n, kv, off, q, table, o.out, o.lse)
        # some of the rows are refused: their pages go back, the next rows take their positions
        s.length = [x - min(c, int(torch.randint(0, 4, (1,), generator=s.g))) if rnd else x for x, c in zip(kv, n)]
        api.block_tables(torch.tensor(s.length, dtype=torch.int32, device="cuda"), *s.pool.values(), page)
        torch.cuda.synchronize()
        assert s.pool["n_blocks"].tolist() == [blocks(x, page) for x in s.length]


def test_captured_round():
    """Tables, append and attention of a round in one graph, replayed on new values and lengths."""
    page, B, n = 16, 3, [4, 1, 3]
    s = Server(B, 8, 2, 64, page, 100, 20, BF, seed=9)
    s.length = [30, 0, 100]
    ro, kvl, off, kv = s.inputs(n)
    T = sum(n)
    cs = torch.zeros(400, 64, device="cuda")
    cs[:, :32] = 1.0  # (no rotation: cosines of 1)
    q, k, v = (torch.zeros(T, h, 64, dtype=BF, device="cuda") for h in (8, 2, 2))
    s.kc.view(torch.uint8).zero_(), s.vc.view(torch.uint8).zero_(), s.ks.fill_(1.0), s.vs.fill_(1.0)
    tables = api.BlockTables(B, T, page, s.n_pages).bind(kvl, *s.pool.values(), row_off=ro)
    append = api.KvAppender8(B, T, 8, 2, 64, BF)
    append.bind(q, k, v, cs, ro, kvl, s.kc, s.vc, s.ks, s.vs, s.pool["block_table"])
    attend = api.Attention8(B, T, 8, 2, 64, BF)
    attend.bind(append.out.q, s.kc, s.vc, s.ks, s.vs, ro, kvl, s.pool["block_table"])

    def step():
        tables.run()
        append.run()
        attend.run()

    state = [*s.pool.values(), s.kc.view(torch.uint8), s.vc.view(torch.uint8), s.ks, s.vs]
    start = [t.clone() for t in state]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()

    def put_back():
        for t, x in zip(state, start):
            t.copy_(x)

    for seed in range(3):
        g = torch.Generator().manual_seed(seed)
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g))
        kvl.copy_(torch.tensor([30 + 7 * seed, 1 + seed, 103 - 20 * seed], dtype=torch.int32))
        got = []
        for call in (step, graph.replay):
            put_back()
            for t in (attend.out.out, attend.out.lse, tables.out.slot_map):
                t.fill_(7)
            call()
            torch.cuda.synchronize()
            got.append([t.clone() for t in (*state, attend.out.out, attend.out.lse, tables.out.slot_map, append.out.q)])
        assert all(torch.equal(x, y) for x, y in zip(*got))
        assert (attend.out.req_status == 0).all() and not torch.equal(got[0][-4], torch.full_like(got[0][-4], 7))


def test_two_attentions_at_once():
    """Two streams, each call with a workspace of its own."""
    from cache8_ref import Batch8
    bs = [Batch8([5, 3] * 8, [900 + 50 * i for i in range(16)], 8, 2, 128, BF, 16, seed=i).place() for i in range(2)]
    calls = [b.attention() for b in bs]
    want = []
    for a in calls:
        o = a.run()
        torch.cuda.synchronize()
        want.append((o.out.clone(), o.lse.clone()))
    streams = [torch.cuda.Stream() for _ in bs]
    for _ in range(20):
        for a, st in zip(calls, streams):
            a.run(st)
    torch.cuda.synchronize()
    for a, w in zip(calls, want):
        assert torch.equal(a.out.out, w[0]) and torch.equal(a.out.lse, w[1])


@pytest.mark.parametrize("kw", [dict(), dict(shared=False), dict(window=24, n_sink=3)], ids=["shared", "own pages", "window"])
def test_example_with_its_cache_in_8_bits(kw):
    import target_pass as ex
    texts, logits, o = ex.run(B=5, gamma=3, rounds=3, prompt=37, seed=3, cache8=True, **kw)
    assert torch.isfinite(logits.float()).all() and (o.req_status == 0).all()
    assert all(len(t) > 38 for t in texts)
