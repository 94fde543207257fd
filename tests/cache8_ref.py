"""The ragged batch of attend_ref over a cache in e4m3 with a scale for each page and head. What the cache
stands for (element * scale, in float64) takes the place of the batch's keys and values, so that the reference
of attend_ref is the reference here too. Everything a kernel may not use holds NaN: elements of slots that no
row sees, and the scales of pages that none sees."""
import math

import torch
from attend_ref import Batch

from speculative_decoding_verification_43_gb300 import api

E4M3, F64 = torch.float8_e4m3fn, torch.float64


def least_scale(amax):
    """The least power of two s with amax <= 448 s, at least 2^-60 (a Python float in, one out)."""
    if amax == 0:
        return 2.0 ** -60
    f, e = math.frexp(amax / 448.0)  # f in [0.5, 1): 2^(e-1) holds it only when f = 0.5
    return max(math.ldexp(1.0, e - 1 if f == 0.5 else e), 2.0 ** -60)


class Batch8(Batch):
    """odd_scales: scales that are no powers of two. loud: factors of the heads' magnitudes, 2^-loud .. 2^loud."""

    def __init__(self, *args, odd_scales=False, loud=3.0, **kw):
        super().__init__(*args, **kw)
        g = torch.Generator().manual_seed(kw.get("seed", 0) + 77)
        self.loud = {c: torch.exp2((torch.rand(self.Hkv, generator=g) * 2 - 1) * loud) for c in "kv"}
        self.odd, self.g = odd_scales, g
        # q is divided by the keys' magnitude, so that the scores stay what they are
        G = self.Hq // self.Hkv
        self.q = (self.q.float() / self.loud["k"].repeat_interleave(G)[None, :, None]).to(self.dtype)
        pages = lambda n, first: [(x, min(n, (x // self.page + 1) * self.page))  # noqa: E731
                                  for x in [first, *range((first // self.page + 1) * self.page, n, self.page)] if x < n]
        self.prefix8 = {c: [self.quantise(c, t[a:b]) for a, b in pages(self.shared, 0)]
                        for c, t in (("k", self.pk), ("v", self.pv))}
        self.own8 = []
        for i in range(self.B):
            n = max(self.kv[i], 0)
            own = {}
            for c, t in (("k", self.keys), ("v", self.vals)):
                own[c] = {}
                whole = torch.zeros(n, self.Hkv, self.D, dtype=F64)
                for (a, b), (e, s) in zip(pages(self.shared, 0), self.prefix8[c]):
                    if a < n:
                        whole[a:b] = (e.to(F64) * s.to(F64)[:, None])[:min(b, n) - a]
                for a, b in pages(n, self.shared):
                    e, s = own[c][a] = self.quantise(c, t[i][a:b])
                    whole[a:b] = e.to(F64) * s.to(F64)[:, None]
                t[i] = whole
            self.own8.append(own)

    def quantise(self, c, x):
        """e4m3 elements [slots, H, D] and scales [H] of the values x [slots, H, D]."""
        x = x.double() * self.loud[c].double()[:, None]
        s = torch.tensor([least_scale(float(t)) for t in x.abs().amax((0, 2))], dtype=F64)
        if self.odd:
            s = s * (1 + torch.rand(self.Hkv, generator=self.g, dtype=F64))
        s = s.float()
        return (x / s.double()[:, None]).float().to(E4M3), s

    def place(self, device="cuda", extra_pages=3):
        page, g = self.page, torch.Generator().manual_seed(self.perm_seed)
        blocks = [(max(x, 0) + page - 1) // page for x in self.kv]
        width = max(max(blocks), 1) + 2
        n_sh = (self.shared + page - 1) // page
        n_pages = n_sh + sum(blocks) + extra_pages
        ids = torch.randperm(n_pages, generator=g).tolist()
        nan = math.nan if self.poison else 0.0
        cache = {c: torch.full((n_pages, page, self.Hkv, self.D), nan).to(E4M3).view(torch.uint8) for c in "kv"}
        scale = {c: torch.full((n_pages, self.Hkv), math.nan if self.poison else 1.0) for c in "kv"}
        table = torch.full((self.B, width), -1, dtype=torch.int32)
        table[:, 1::2] = n_pages + 7
        for c in "kv":
            for b, (e, s) in enumerate(self.prefix8[c]):
                cache[c][ids[b], :len(e)] = e.view(torch.uint8)
                scale[c][ids[b]] = s
        nxt = n_sh
        for i, kv in enumerate(self.kv):
            first = kv - self.rows[i]
            seen = [self.rows[i] > 0 and (self.window == 0 or x > max(first, 0) - self.window or x < self.sinks)
                    for x in range(max(kv, 0))]
            for b in range(blocks[i]):
                pid = ids[nxt]
                nxt += 1
                a, e = max(b * page, self.shared), min(kv, (b + 1) * page)
                xs = [x for x in range(a, e) if seen[x]]
                if not xs:
                    continue  # no row sees this page, or the shared one serves it
                table[i, b] = pid
                for c in "kv":
                    val, s = self.own8[i][c][a]
                    scale[c][pid] = s
                    for x in xs:
                        cache[c][pid, x % page] = val[x - a].view(torch.uint8)
        to = lambda t: t.to(device)  # noqa: E731
        for c in "kv":
            t = cache[c]
            if self.order == "head":  # a page keeps each head's slots together
                t = to(t.permute(0, 2, 1, 3).contiguous()).permute(0, 2, 1, 3)
            else:
                t = to(t)
            setattr(self, c + "_cache", t.view(E4M3))
            setattr(self, c + "_scale", to(scale[c]))
        self.table = to(table)
        self.row_off = to(torch.tensor(self.off, dtype=torch.int32))
        self.kv_len = to(torch.tensor(self.kv, dtype=torch.int32))
        self.shared_table = to(torch.tensor(ids[:n_sh], dtype=torch.int32)) if self.shared else None
        self.qd = to(self.q)
        return self

    def cache(self):
        return self.k_cache, self.v_cache, self.k_scale, self.v_scale

    def attention(self, **kw):
        a = api.Attention8(self.B, self.T, self.Hq, self.Hkv, self.D, self.dtype, window=self.window,
                           n_sink=self.sinks, shared_len=self.shared, **kw)
        return a.bind(self.qd, *self.cache(), self.row_off, self.kv_len, self.table, shared_table=self.shared_table)

    def reference(self):
        """attend_ref's, and per row a bound on what the queries' two parts leave of the scores, and the largest
        |v| that the row sees."""
        out, lse, mag, ulps, nk = super().reference()
        cut, vmax = torch.zeros_like(lse), torch.zeros(self.T, self.Hq, 1, dtype=F64)
        G, scale = self.Hq // self.Hkv, self.D ** -0.5
        for i in range(self.B):
            if not len(self.keys[i]):
                continue
            ksum, vm = self.keys[i].abs().sum(2), self.vals[i].abs().amax(2)
            for t in range(self.off[i], self.off[i + 1]):
                q = self.q[t].double().abs().amax(1)
                cut[t] = q * ksum.amax(0).repeat_interleave(G) * scale
                vmax[t, :, 0] = vm.amax(0).repeat_interleave(G)
        return out, lse, mag, ulps, nk, cut, vmax


def check8(batch, got, ref=None):
    """The kernel's out and lse against the reference.

    Bounds, beside those of attend_ref.check (`ulps`, the exponentials, the sums; fp32 rows' queries have 19 bits
    and their weights 22 on the tensor cores, which `ulps` holds as well). bf16 rows on the tensor cores: a query element is off by at most 2^-18 of its head's largest, which moves a score by at most 2^-18 * `cut`. A
    product of a position's scale and a row's factor is rounded, 2^-23 of the score (4 |z| of `ulps` has it). The
    logarithms of the v scales are off by 2^-20 at most (|log2| below 64, 2^-22 of it each way). A weight is
    rounded to 11 bits, 2^-11 of itself, or by at most 2^-27 of the row's reference, which is at most the largest
    weight * 2^5 away from it: n keys move the output by at most n 2^-22 of the largest |v|. The output is rounded
    once, 2^-8 of itself (2^-24 in fp32)."""
    out, lse, mag, ulps, nk, cut, vmax = ref or batch.reference()
    got_out, got_lse = got.out.cpu().double(), got.lse.cpu().double()
    weight = 2 * ulps * 2.0 ** -22 + 2.0 ** -20 + nk * 2.0 ** -23
    tol = torch.zeros_like(out)
    if batch.dtype == torch.bfloat16:
        weight = weight + 2 * cut * 2.0 ** -18 + 2.0 ** -17
        tol = mag * 2.0 ** -11 + out.abs() * 2.0 ** -8 + vmax * nk[..., None] * 2.0 ** -22
    tol = tol + mag * weight[..., None]
    bad = ~((got_out - out).abs() <= tol + 1e-30)
    assert not bad.any(), (bad.sum().item(), bad.nonzero()[:4].tolist(), (got_out - out).abs().max().item())
    empty = lse == -math.inf
    assert torch.equal(got_lse == -math.inf, empty)
    assert (got_out[empty] == 0).all()
    ltol = weight + lse.abs() * 2.0 ** -22
    lbad = ~((got_lse - lse).abs() <= ltol) & ~empty
    assert not lbad.any(), (lbad.sum().item(), lbad.nonzero()[:4].tolist(), (got_lse - lse)[lbad][:4])
