"""Ragged batches over a paged cache and their attention in float64, for the tests of spec_kv_append
and spec_attend. The reference works on one row and one head at a time from the definition; it shares
nothing with the kernels. Everything a kernel may not use is poisoned: slots past a request's
length, pages nobody refers to and positions behind every row's window hold NaN, and the block table
has no valid id for pages that no row sees."""
import math

import torch

from speculative_decoding_verification_43_gb300 import api


class Batch:
    """rows[i] rows and kv[i] positions for each request; the values of every position are kept in
    `keys` and `vals` ([kv][Hkv][D] per request) and placed in the cache by place()."""

    def __init__(self, rows, kv, Hq, Hkv, D, dtype, page, window=0, sinks=0, shared=0, seed=0, order="slot",
                 spread=1.5, poison=True):
        g = torch.Generator().manual_seed(seed)
        self.rows, self.kv, self.Hq, self.Hkv, self.D, self.dtype, self.page = rows, kv, Hq, Hkv, D, dtype, page
        self.window, self.sinks, self.shared, self.order, self.poison = window, sinks, shared, order, poison
        self.B, self.T = len(rows), sum(rows)
        self.off = [0]
        for n in rows:
            self.off.append(self.off[-1] + n)
        rnd = lambda *s: torch.randn(*s, generator=g).to(dtype)  # noqa: E731
        self.q = (torch.randn(self.T, Hq, D, generator=g) * spread).to(dtype)
        pk, pv = rnd(shared, Hkv, D), rnd(shared, Hkv, D)
        self.keys, self.vals = [], []
        for x in kv:
            x = max(x, 0)
            self.keys.append(torch.cat([pk[:x], rnd(max(x - shared, 0), Hkv, D)]))
            self.vals.append(torch.cat([pv[:x], rnd(max(x - shared, 0), Hkv, D)]))
        self.pk, self.pv = pk, pv
        self.perm_seed = seed + 1

    def sees(self, p, x):
        return x <= p and (self.window == 0 or x > p - self.window or x < self.sinks)

    def place(self, device="cuda", extra_pages=3):
        page, g = self.page, torch.Generator().manual_seed(self.perm_seed)
        blocks = [(max(x, 0) + page - 1) // page for x in self.kv]
        width = max(max(blocks), 1) + 2
        n_sh = (self.shared + page - 1) // page
        n_pages = n_sh + sum(blocks) + extra_pages
        ids = torch.randperm(n_pages, generator=g).tolist()
        fill = float("nan") if self.poison else 0.0
        k = torch.full((n_pages, page, self.Hkv, self.D), fill, dtype=self.dtype)
        v = k.clone()
        table = torch.full((self.B, width), -1, dtype=torch.int32)
        table[:, 1::2] = n_pages + 7
        nxt = n_sh
        for x in range(self.shared):
            k[ids[x // page], x % page], v[ids[x // page], x % page] = self.pk[x], self.pv[x]
        for i, kv in enumerate(self.kv):
            first = kv - self.rows[i]
            seen = [self.rows[i] > 0 and (self.window == 0 or x > max(first, 0) - self.window or x < self.sinks)
                    for x in range(max(kv, 0))]
            for b in range(blocks[i]):
                pid = ids[nxt]
                nxt += 1
                xs = [x for x in range(b * page, min(kv, (b + 1) * page)) if seen[x]]
                if not xs or xs[-1] < self.shared:
                    continue  # no row sees this page, or the shared one serves it
                table[i, b] = pid
                for x in xs:
                    k[pid, x % page], v[pid, x % page] = self.keys[i][x], self.vals[i][x]
        if self.order == "head":  # a page keeps each head's slots together
            k = k.permute(0, 2, 1, 3).contiguous().to(device).permute(0, 2, 1, 3)
            v = v.permute(0, 2, 1, 3).contiguous().to(device).permute(0, 2, 1, 3)
        to = lambda t: t.to(device)  # noqa: E731
        self.k_cache, self.v_cache, self.table = to(k), to(v), to(table)
        self.row_off = to(torch.tensor(self.off, dtype=torch.int32))
        self.kv_len = to(torch.tensor(self.kv, dtype=torch.int32))
        self.shared_table = to(torch.tensor(ids[:n_sh], dtype=torch.int32)) if self.shared else None
        self.qd = to(self.q)
        return self

    def attention(self, **kw):
        a = api.Attention(self.B, self.T, self.Hq, self.Hkv, self.D, self.dtype, window=self.window,
                          n_sink=self.sinks, shared_len=self.shared, **kw)
        return a.bind(self.qd, self.k_cache, self.v_cache, self.row_off, self.kv_len, self.table,
                      shared_table=self.shared_table)

    def reference(self):
        """out, lse, and per element sum p |v| and per row a bound on the scores' rounding in units of
        the last place of 32 bits."""
        f = torch.float64
        G = self.Hq // self.Hkv
        out = torch.zeros(self.T, self.Hq, self.D, dtype=f)
        mag = torch.zeros_like(out)
        lse = torch.full((self.T, self.Hq), -math.inf, dtype=f)
        ulps = torch.zeros(self.T, self.Hq, dtype=f)
        nk = torch.zeros(self.T, 1, dtype=f)
        scale = self.D ** -0.5
        for i in range(self.B):
            K, V = self.keys[i].to(f), self.vals[i].to(f)
            for j in range(self.rows[i]):
                p, t = self.kv[i] - self.rows[i] + j, self.off[i] + j
                x = torch.tensor([x for x in range(p + 1) if self.sees(p, x)], dtype=torch.long)
                if not len(x):
                    continue
                nk[t] = len(x)
                for h in range(self.Hkv):
                    q = self.q[t, h * G:(h + 1) * G].to(f)
                    z = q @ K[x, h].T * scale
                    w = torch.softmax(z, 1)
                    s = slice(h * G, (h + 1) * G)
                    out[t, s], mag[t, s] = w @ V[x, h], w @ V[x, h].abs()
                    lse[t, s] = torch.logsumexp(z, 1)
                    ulps[t, s] = (q.abs() @ K[x, h].abs().T * scale).amax(1) * self.D + 4 * z.abs().amax(1)
        return out, lse, mag, ulps, nk


def check(batch, got, ref=None):
    """The kernel's out and lse against the reference.

    Bounds. A score is a sum of D exact products (bf16) or rounded ones (fp32) accumulated in 32 bits
    and scaled: its error is at most `ulps` * 2^-22 in the exponent's units (2^-24 per addition, and a
    factor four for a tensor core's truncating accumulation), and so is the relative error of a
    weight, twice (its own and the sum's). The exponential unit adds 2^-21, the sums over n keys
    n * 2^-24. In bf16 (8 significant bits: half a unit in the last place is up to 2^-8) each weight is
    rounded and the output once more: together at most 2^-7 of sum p |v|."""
    out, lse, mag, ulps, nk = ref or batch.reference()
    got_out, got_lse = got.out.cpu().double(), got.lse.cpu().double()
    weight = 2 * ulps * 2.0 ** -22 + 2.0 ** -20 + nk * 2.0 ** -23
    tol = mag * ((2.0 ** -7 if batch.dtype == torch.bfloat16 else 0.0) + weight)[..., None]
    bad = ~((got_out - out).abs() <= tol + 1e-30)
    assert not bad.any(), (bad.sum().item(), bad.nonzero()[:4].tolist(), (got_out - out).abs().max().item())
    empty = lse == -math.inf
    assert torch.equal(got_lse == -math.inf, empty)
    assert (got_out[empty] == 0).all()
    ltol = weight + lse.abs() * 2.0 ** -22
    lbad = ~((got_lse - lse).abs() <= ltol) & ~empty
    assert not lbad.any(), (lbad.sum().item(), lbad.nonzero()[:4].tolist(), (got_lse - lse)[lbad][:4])
