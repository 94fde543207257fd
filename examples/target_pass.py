"""Verification rounds of a small target model over a paged cache: what goes into spec_verify, computed
with the same library.

Each round the target takes, for every request, the pending token and its drafts: per layer their
keys and values are appended to the cache (rotated on the way) and the rows attend to it, with the
system prompt that all requests share read once for the whole batch. The logits go to the verifier
with the drafter's, and what it accepts moves each request's length on. Rejected drafts need no undoing:
the next round's rows take their positions. With --cache8 the cache is held in 8 bits, and its pages are
handed out on the device: tables are brought to each round's lengths, and to what was accepted after it.

The model is random (two layers, rotary attention and a gated feed-forward block); the drafter is the
target's own output projection over noisy embeddings. One GPU:

    python examples/target_pass.py [--cache8]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from speculative_decoding_verification_43_gb300 import api  # noqa: E402


class Target:
    """Two layers with grouped query heads; bf16 weights from a seed."""

    def __init__(self, vocab=512, layers=2, Hq=8, Hkv=2, D=64, page=16, pages=512, seed=0, window=0, n_sink=0,
                 cache8=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda *s: (torch.randn(*s, generator=g, device="cuda") * s[0] ** -0.5).bfloat16()  # noqa: E731
        self.Hq, self.Hkv, self.D, self.page, self.window, self.n_sink = Hq, Hkv, D, page, window, n_sink
        width = Hq * D
        self.embed, self.head = w(vocab, width) * vocab ** 0.5, w(width, vocab) * 4
        self.layers = [dict(qkv=w(width, (Hq + 2 * Hkv) * D), out=w(width, width), up=w(width, 4 * width),
                            down=w(2 * width, width)) for _ in range(layers)]
        self.pages, self.cache8 = pages, cache8
        self.cache = [tuple(torch.zeros(pages, page, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
                      for _ in range(layers)]
        if cache8:  # elements and, for each page and head, their scale
            self.cache = [tuple(torch.zeros(pages, page, Hkv, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
                                for _ in range(2)) + tuple(torch.ones(pages, Hkv, device="cuda") for _ in range(2))
                          for _ in range(layers)]
        angle = torch.arange(pages * page, device="cuda")[:, None] * 10000.0 ** (
            -torch.arange(D // 2, device="cuda") / (D // 2))
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()

    def forward(self, tokens, row_off, kv_len, table, shared_len=0, shared_table=None):
        """Logits of the rows (tokens [T], rows of request i at row_off[i]..); kv_len includes them."""
        T, B, Hq, Hkv, D = tokens.numel(), kv_len.numel(), self.Hq, self.Hkv, self.D
        norm = lambda x: torch.nn.functional.rms_norm(x, (x.shape[-1],))  # noqa: E731
        x = self.embed[tokens.long()]
        kinds = (api.KvAppender8, api.Attention8) if self.cache8 else (api.KvAppender, api.Attention)
        append = kinds[0](B, T, Hq, Hkv, D, torch.bfloat16)
        attend = kinds[1](B, T, Hq, Hkv, D, torch.bfloat16, window=self.window, n_sink=self.n_sink,
                          shared_len=shared_len)
        for w, cache in zip(self.layers, self.cache):
            qkv = norm(x) @ w["qkv"]
            q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
            q = append.bind(q, k, v, self.cos_sin, row_off, kv_len, *cache, table).run().q
            o = attend.bind(q, *cache, row_off, kv_len, table, shared_table=shared_table).run().out
            x = x + o.flatten(1) @ w["out"]
            a, b = (norm(x) @ w["up"]).chunk(2, 1)
            x = x + (torch.nn.functional.silu(a) * b) @ w["down"]
        return norm(x) @ self.head


def run(B=6, gamma=3, rounds=4, prompt=37, seed=0, temperature=0.8, shared=True, window=0, n_sink=0,
        cache8=False):
    """A few rounds; returns each request's tokens and the last round's target logits with their rows."""
    m = Target(seed=seed, window=window, n_sink=n_sink, cache8=cache8)
    V = m.head.shape[1]
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    # the system prompt, prefilled once into pages of its own; every request's table names them
    system = torch.randint(0, V, (prompt,), generator=g, device="cuda")
    n_sys = (prompt + m.page - 1) // m.page
    sys_table = i32(list(range(n_sys)))
    m.forward(system, i32([0, prompt]), i32([prompt]), sys_table[None])
    whole = prompt // m.page * m.page  # whole pages are shared as they are; the rest is copied per request
    per = (prompt + rounds * (gamma + 1) + gamma) // m.page + 1
    table = torch.stack([i32([b if b < whole // m.page else n_sys + i * per + b for b in range(per)]) for i in range(B)])
    pages = None
    if cache8:  # the pages behind the system prompt's are handed out as they are needed
        free = list(range(n_sys, m.pages))
        pages = (i32([0] * B), i32([[-1] * per] * B), i32(free + [-1] * n_sys), i32([len(free)]))
        table, whole_pages = pages[1], sys_table[:whole // m.page].contiguous()
        bring = lambda lengths, **kw: api.block_tables(lengths, *pages, m.page, shared_table=whole_pages, **kw)  # noqa: E731
        bring(i32([prompt] * B))
    for cache in m.cache:
        for c in cache:
            if whole < prompt:
                c = c.view(torch.uint8) if c.dtype == torch.float8_e4m3fn else c
                c[table[:, whole // m.page].long()] = c[n_sys - 1].clone()
    texts = [system.tolist() + [int(torch.randint(0, V, (1,), generator=g, device="cuda"))] for _ in range(B)]
    K = [min(gamma, i % (gamma + 1)) for i in range(B)]  # some requests draft less, some nothing
    row_off = [0]
    for k in K:
        row_off.append(row_off[-1] + k + 1)
    T = row_off[-1]
    ro = i32(row_off)
    logits = None
    for _ in range(rounds):
        # the drafter: tokens from a noisy bigram law of the target's own embeddings
        rows, draft_logits, drafts = [], [], []
        for i in range(B):
            last = texts[i][-1]
            rows.append(last)
            for _ in range(K[i]):
                z = (m.embed[last].float() @ m.head.float() * 0.2 + torch.randn(V, generator=g, device="cuda")).bfloat16()
                last = int(torch.multinomial(torch.softmax(z.float() / temperature, 0), 1, generator=g))
                draft_logits.append(z)
                drafts.append(last)
                rows.append(last)
        kv_len = i32([len(texts[i]) + K[i] for i in range(B)])
        if cache8:
            t = bring(kv_len, row_off=ro, total_rows=T)
            assert (t.req_status == 0).all() and (t.slot_map >= 0).all()
        logits = m.forward(i32(rows), ro, kv_len, table, shared_len=whole if shared else 0,
                           shared_table=sys_table if shared else None).contiguous()
        u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
        o = api.verify(logits, torch.stack(draft_logits), ro, i32(drafts), u, temperature, K_max=gamma)
        torch.cuda.synchronize()
        assert (o.req_status == 0).all()
        out, n = o.out_tokens.tolist(), o.n_emitted.tolist()
        for i in range(B):
            texts[i] += out[row_off[i]:row_off[i] + n[i]]
        if cache8:  # (the last token of a text has no keys yet)
            bring(i32([len(t) - 1 for t in texts]))
    return texts, logits, o


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--requests", type=int, default=6)
    p.add_argument("--gamma", type=int, default=3)
    p.add_argument("--rounds", type=int, default=4)
    p.add_argument("--cache8", action="store_true")
    a = p.parse_args()
    texts, logits, o = run(a.requests, a.gamma, a.rounds, cache8=a.cache8)
    for i, t in enumerate(texts):
        print(f"request {i}: {len(t)} tokens, the last round accepted {int(o.accept_len[i])}: ...", t[-8:])


if __name__ == "__main__":
    main()
