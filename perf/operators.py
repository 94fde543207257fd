"""Cases of the target pass's operators over a paged cache: appending a round's keys and values
with their position rotation, attention of the round's rows with a sliding window and sinks, and
the same attention for a batch whose requests share a long prefix.

Layout, as for the verifier: request i owns rows row_off[i] .. row_off[i+1]-1 of the batch; its
n_i rows are the last n_i of its kv_len[i] positions; position x lies in slot x % page of page
block_table[i][x // page].

A case's shapes (rows and lengths of each request) follow from its own numbers ("shape" seeds
them); the values follow from the seed given to prepare().
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------- cases

def _append(name, shape, B, rows, ctx, Hq, Hkv, D, page, dtype, rot, interleaved=False, order="slot"):
    return dict(name=name, op="append", shape=shape, B=B, rows_lo=rows[0], rows_hi=rows[1], ctx_lo=ctx[0],
                ctx_hi=ctx[1], Hq=Hq, Hkv=Hkv, D=D, page=page, dtype=dtype, rot=rot, interleaved=interleaved,
                order=order)


def _attend(name, shape, B, rows, ctx, Hq, Hkv, D, page, dtype, window=0, sinks=0, shared=0, order="slot"):
    return dict(name=name, op="attend", shape=shape, B=B, rows_lo=rows[0], rows_hi=rows[1], ctx_lo=ctx[0],
                ctx_hi=ctx[1], Hq=Hq, Hkv=Hkv, D=D, page=page, dtype=dtype, window=window, sinks=sinks,
                shared=shared, order=order)


def listed():
    return [
        # one user's round of four drafts: five rows, a thousand tokens in; latency is all that counts
        _append("append_one", 1, 1, (5, 5), (1000, 1000), 32, 8, 128, 16, "bf16", 128),
        # the ragged batch of 64 requests with up to seven drafts, at any point of their texts
        _append("append_round", 2, 64, (1, 8), (1, 16000), 32, 8, 128, 16, "bf16", 128),
        # 256 requests of three drafts after 4096-token prefixes in fp32; part of each head rotated, as
        # interleaved pairs; the cache holds each head's slots together
        _append("append_round_f32", 3, 256, (4, 4), (4096, 4096), 16, 4, 128, 16, "f32", 64, True, "head"),
        # whole prompts entering the cache, heads of 64 without sharing
        _append("append_prompts", 4, 6, (500, 4000), (0, 700), 16, 16, 64, 64, "bf16", 64),
        # one user's round of four drafts after a thousand tokens
        _attend("attend_one", 5, 1, (5, 5), (1000, 1000), 32, 8, 128, 16, "bf16"),
        # the ragged batch under a sliding window with four sinks
        _attend("attend_round_window", 6, 64, (1, 8), (1, 16000), 32, 8, 128, 16, "bf16", 1024, 4),
        # few users deep in long texts, every token visible: the cache's bytes are the work
        _attend("attend_round_long", 7, 16, (1, 8), (4000, 65000), 32, 8, 128, 16, "bf16"),
        # 256 requests of three drafts after 4096-token prefixes in fp32, a narrow window
        _attend("attend_round_f32", 8, 256, (4, 4), (4096, 4096), 16, 4, 128, 16, "f32", 500, 4, 0, "head"),
        # prompts of a few thousand tokens, some continuing a cached part: arithmetic is the work
        _attend("attend_prompts", 9, 4, (1000, 2500), (0, 6000), 32, 8, 128, 64, "bf16"),
        # a handful of requests behind one instruction text
        _attend("shared_small", 10, 8, (1, 4), (1, 200), 12, 4, 96, 16, "bf16", 0, 0, 1001),
        # the ragged batch behind an 8192-token document
        _attend("shared_round", 11, 64, (1, 8), (1, 1000), 32, 8, 128, 16, "bf16", 0, 0, 8192),
        # 512 requests with zero to two drafts behind a long document
        _attend("shared_large", 12, 512, (1, 3), (1, 250), 32, 8, 128, 16, "bf16", 0, 0, 32768),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ranges."""
    ref = listed()
    while True:
        kind = rng.choice(["append", "append", "attend", "attend", "attend", "shared", "shared"])
        f32 = rng.random() < 0.2
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 3, 4, 8])
        page = rng.choice([8, 16, 24, 32, 64])
        order = rng.choice(["slot", "slot", "head"])
        D = rng.choice([64, 80, 96, 128, 128])
        shape = rng.randrange(1 << 30)
        dtype = "f32" if f32 else "bf16"
        if kind == "append":
            if rng.random() < 0.3:
                B, hi = _log_int(rng, 1, 8), _log_int(rng, 200, 4000)
                rows, ctx = (max(1, hi // 8), hi), (0, _log_int(rng, 1, 700))
            else:
                B = _log_int(rng, 1, 512)
                rows, ctx = (1, rng.randint(1, 8)), (1, _log_int(rng, 10, 16000))
            rot = rng.choice([D, D, D // 2])
            case = _append("", shape, B, rows, ctx, Hkv * G, Hkv, D, page, dtype, rot, rng.random() < 0.4, order)
        elif kind == "attend":
            window = rng.choice([0, 0, _log_int(rng, 1, 4000)])
            sinks = rng.choice([0, 4, rng.randint(1, 300)]) if window else 0
            if rng.random() < 0.25:
                B, hi = _log_int(rng, 1, 4), _log_int(rng, 200, 2500)
                rows, ctx = (max(1, hi // 8), hi), (0, _log_int(rng, 1, 6000))
            else:
                B = _log_int(rng, 1, 256)
                rows, ctx = (1, rng.randint(1, 8)), (1, _log_int(rng, 50, 65000))
            case = _attend("", shape, B, rows, ctx, Hkv * G, Hkv, D, page, dtype, window, sinks, 0, order)
        else:
            B = _log_int(rng, 2, 512)
            window = rng.choice([0, 0, 0, _log_int(rng, 100, 4000)])
            sinks = rng.choice([4, 100]) if window else 0
            case = _attend("", shape, B, (1, rng.randint(1, 8)), (1, _log_int(rng, 1, 1000)), Hkv * G, Hkv, D, page,
                           dtype, window, sinks, _log_int(rng, 200, 32768), order)
        del case["name"]
        same = [c for c in ref if c["op"] == case["op"] and (case["dtype"] == "bf16" or c["dtype"] == "f32")
                and bool(c.get("shared")) == bool(case.get("shared")) or
                (case.get("shared") and case["dtype"] == "f32" and c["name"] == "attend_round_f32")]
        w = work(case)
        if all(w[k] <= max(work(c)[k] for c in same) for k in ("bytes", "flops")) and _pool_tokens(case) <= 1100000:
            return case


# -------------------------------------------------------------------------- shapes and work

def _shape(case):
    """(rows, ctx) of each request: rows of this call, and positions before them (the requests'
    own ones, after the shared prefix)."""
    r = random.Random(case["shape"])
    rows = [r.randint(case["rows_lo"], case["rows_hi"]) for _ in range(case["B"])]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) + case.get("shared", 0) for _ in range(case["B"])]
    return rows, ctx


def _pool_tokens(case):
    rows, ctx = _shape(case)
    if case["op"] == "append":
        return sum(rows) + case["B"] * case["page"] * 2
    return sum(rows) + sum(ctx) - (case["B"] - 1) * case["shared"]


def _count_visible(n, c, lo, W, S):
    """(pairs, keys) of a request's n rows at positions c .. c+n-1 over positions >= lo."""
    pairs = 0
    for p in range(c, c + n):
        w0 = max(lo, p - W + 1) if W else lo
        pairs += max(0, p + 1 - w0) + (max(0, min(S, w0) - lo) if W else 0)
    w0 = max(lo, c - W + 1) if W else lo
    keys = max(0, c + n - w0) + (max(0, min(S, w0) - lo) if W else 0)
    return pairs, keys


def work(case):
    rows, ctx = _shape(case)
    T, B = sum(rows), case["B"]
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    eb = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "append":
        byt = 2 * T * (Hq + 2 * Hkv) * D * eb + T * case["rot"] * 4 + (B + 1 + B) * 4
        byt += 4 * sum((c + n - 1) // case["page"] - c // case["page"] + 1 for n, c in zip(rows, ctx))
        return {"bytes": byt, "flops": 3 * T * (Hq + Hkv) * case["rot"]}
    W, S, L = case["window"], case["sinks"], case["shared"]
    pairs = keys = 0
    pre = 0  # keys of the prefix that some row sees
    for n, c in zip(rows, ctx):
        a, b = _count_visible(n, c, L, W, S)
        pairs, keys = pairs + a, keys + b
        if L:
            for p in range(c, c + n):
                w0 = min(L, max(0, p - W + 1)) if W else 0
                seen = L - w0 + (min(S, w0) if W else 0)
                pairs += seen
                pre = max(pre, seen)
    keys += pre
    byt = 2 * T * Hq * D * eb + 4 * T * Hq + 2 * keys * Hkv * D * eb + 4 * (keys // case["page"] + 2 * B)
    return {"bytes": byt, "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------------------------ inputs

def _cache(n_pages, case, gen, dev):
    """A pool of earlier tokens' values, [pages, slots, heads, D]; "head" keeps a head's slots of a page
    together in memory."""
    dt = DTYPES[case["dtype"]]
    page, H, D = case["page"], case["Hkv"], case["D"]
    if case["order"] == "head":
        return torch.randn(n_pages, H, page, D, generator=gen, device=dev, dtype=dt).permute(0, 2, 1, 3)
    return torch.randn(n_pages, page, H, D, generator=gen, device=dev, dtype=dt)


def _inputs(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 1000003 + case["shape"])
    r = random.Random(seed * 7919 + case["shape"])
    rows, ctx = _shape(case)
    B, page, L = case["B"], case["page"], case.get("shared", 0)
    off = [0]
    for n in rows:
        off.append(off[-1] + n)
    kv = [c + n for n, c in zip(rows, ctx)]
    T = off[-1]
    width = max((x + page - 1) // page for x in kv)
    tab = [[-1] * width for _ in range(B)]
    # pages: first the ones all requests share, then each request's own; a request's own part that
    # begins inside a shared page has a page of its own there, with the same tokens before it
    if case["op"] == "append":  # only the tail is written: pages before it are common to all
        common = [c // page for c in ctx]
    else:
        common = [L // page] * B
    n_shared = max([*common, (L + page - 1) // page])
    if case["op"] == "append":
        n_shared = min(n_shared, 64)  # what they hold does not matter here: few pages stand for all
    own_pages = sum((x + page - 1) // page - c for x, c in zip(kv, common))
    ids = list(range(n_shared + own_pages))
    r.shuffle(ids)
    nxt = n_shared
    for i in range(B):
        for b in range((kv[i] + page - 1) // page):
            if b < common[i]:
                tab[i][b] = ids[b % max(n_shared, 1)]
            else:
                tab[i][b] = ids[nxt]
                nxt += 1
    i32 = dict(dtype=torch.int32, device=dev)
    s = dict(case=case, rows=rows, kv=kv, off=off, T=T)
    s["row_off"] = torch.tensor(off, **i32)
    s["kv_len"] = torch.tensor(kv, **i32)
    s["table"] = torch.tensor(tab, **i32)
    s["k_cache"] = _cache(len(ids), case, gen, dev)
    s["v_cache"] = _cache(len(ids), case, gen, dev)
    dt = DTYPES[case["dtype"]]
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if L:
        s["shared_table"] = torch.tensor(ids[:(L + page - 1) // page], **i32)
        if L % page:  # the requests' own copies of the last shared page hold the same tokens
            last = torch.tensor([tab[i][L // page] for i in range(B)], device=dev)
            for c in (s["k_cache"], s["v_cache"]):
                c[last, :L % page] = c[ids[L // page], :L % page].clone()
    if case["op"] == "append":
        # the rows come out of one projection: q, k and v side by side
        qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=gen, device=dev, dtype=dt)
        s["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        s["v"] = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
        half = case["rot"] // 2
        ang = torch.arange(max(kv), dtype=torch.float64, device=dev)[:, None] * \
            (10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half))[None]
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
    else:
        s["q"] = (torch.randn(T, Hq, D, generator=gen, device=dev) * 1.5).to(dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from speculative_decoding_verification_43_gb300 import api
        dims = (case["B"], s["T"], case["Hq"], case["Hkv"], case["D"], DTYPES[case["dtype"]])
        if case["op"] == "append":
            s["call"] = api.KvAppender(*dims, rot_dim=case["rot"], interleaved=case["interleaved"])
            s["call"].bind(s["q"], s["k"], s["v"], s["cos_sin"], s["row_off"], s["kv_len"], s["k_cache"],
                           s["v_cache"], s["table"])
        else:
            s["call"] = api.Attention(*dims, window=case["window"], n_sink=case["sinks"], shared_len=case["shared"])
            s["call"].bind(s["q"], s["k_cache"], s["v_cache"], s["row_off"], s["kv_len"], s["table"],
                           shared_table=s.get("shared_table"))
    return s


# ------------------------------------------------------------------------------ one pass

def run(state):
    s, case = state, state["case"]
    if case["op"] == "append":
        if own:
            return s["call"].run().q, s["k_cache"], s["v_cache"]
        return _plain_append(s, case)
    if own:
        o = s["call"].run()
        return o.out, o.lse
    return _plain_attend(s, case)


def _positions(s):
    """Position and request of every row."""
    row_off, kv_len = s["row_off"].long(), s["kv_len"].long()
    n = row_off[1:] - row_off[:-1]
    req = torch.repeat_interleave(torch.arange(n.numel(), device=n.device), n, output_size=s["T"])
    return kv_len[req] - n[req] + torch.arange(s["T"], device=n.device) - row_off[req], req


def _rotate(x, cos, sin, rot, interleaved):
    x = x.float()
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([r, x[..., rot:]], -1)


def _plain_append(s, case):
    rot, page = case["rot"], case["page"]
    pos, req = _positions(s)
    cos, sin = s["cos_sin"][pos][:, None, :rot // 2], s["cos_sin"][pos][:, None, rot // 2:]
    dt = s["q"].dtype
    q = _rotate(s["q"], cos, sin, rot, case["interleaved"]).to(dt)
    k = _rotate(s["k"], cos, sin, rot, case["interleaved"]).to(dt)
    pages, slots = s["table"][req, pos // page].long(), pos % page
    s["k_cache"][pages, slots] = k
    s["v_cache"][pages, slots] = s["v"]
    return q, s["k_cache"], s["v_cache"]


def _part(q, k, v, seen, scale):
    """Softmax parts of rows q [n, Hkv, G, D] over keys k, v [x, Hkv, D] (seen [n, x]): row maxima,
    sums and unnormalised outputs, [Hkv, n, G] and [Hkv, n, G, D]."""
    n, H, G, D = q.shape
    z = torch.matmul(q.permute(1, 0, 2, 3).reshape(H, n * G, D), k.permute(1, 2, 0)).view(H, n, G, -1) * scale
    z = z.masked_fill(~seen[None, :, None, :], -math.inf)
    m = z.amax(-1)
    p = torch.exp(z - torch.where(m == -math.inf, 0.0, m)[..., None])
    return m, p.sum(-1), torch.matmul(p.view(H, n * G, -1), v.permute(1, 0, 2)).view(H, n, G, D)


def _plain_attend(s, case):
    W, S, L, page = case["window"], case["sinks"], case["shared"], case["page"]
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    scale = D ** -0.5
    dev = s["q"].device
    kc, vc = s["k_cache"], s["v_cache"]
    q = s["q"].float().view(s["T"], Hkv, Hq // Hkv, D)
    pos, _ = _positions(s)

    def keys(table, x):
        pages, slots = table[x // page].long(), x % page
        return kc[pages, slots].float(), vc[pages, slots].float()

    def seen(p, x):
        ok = x[None] <= p[:, None]
        return ok & ((x[None] > p[:, None] - W) | (x[None] < S)) if W else ok

    if L:
        x = torch.arange(L, device=dev)
        pm, pl, po = _part(q, *keys(s["shared_table"], x), seen(pos, x), scale)
    out = torch.empty(s["T"], Hq, D, dtype=s["q"].dtype, device=dev)
    lse = torch.empty(s["T"], Hq, dtype=torch.float32, device=dev)
    for i, (n, kv) in enumerate(zip(s["rows"], s["kv"])):
        a, b = s["off"][i], s["off"][i + 1]
        w0 = max(L, kv - n - W + 1) if W else L
        x = torch.arange(w0, kv, device=dev)
        if W and L < min(S, w0):
            x = torch.cat([torch.arange(L, min(S, w0), device=dev), x])
        m, l, o = _part(q[a:b], *keys(s["table"][i], x), seen(pos[a:b], x), scale)
        if L:
            m1, l1, o1 = pm[:, a:b], pl[:, a:b], po[:, a:b]
            mm = torch.maximum(m, m1)
            e, e1 = torch.exp(m - mm), torch.exp(m1 - mm)
            m, l, o = mm, l * e + l1 * e1, o * e[..., None] + o1 * e1[..., None]
        out[a:b] = (o / l[..., None]).permute(1, 0, 2, 3).reshape(n, Hq, D).to(out.dtype)
        lse[a:b] = (m + torch.log(l)).permute(1, 0, 2).reshape(n, Hq)
    return out, lse


# ------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    f64 = torch.float64
    dev = s["q"].device
    page, Hq, Hkv, D = case["page"], case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "append":
        rot = case["rot"]
        half = rot // 2
        # dimension d turns with partner[d]: x[d] cos + sign[d] x[partner[d]] sin
        d = torch.arange(rot, device=dev)
        if case["interleaved"]:
            partner, freq, sign = d ^ 1, d // 2, torch.where(d % 2 == 0, -1.0, 1.0).to(f64)
        else:
            partner, freq, sign = (d + half) % rot, d % half, torch.where(d < half, -1.0, 1.0).to(f64)
        q, kc, vc = s["q"].to(f64), s["k_cache"].to(f64), s["v_cache"].to(f64)
        for i in range(case["B"]):
            a, b = s["off"][i], s["off"][i + 1]
            x = torch.arange(s["kv"][i] - (b - a), s["kv"][i], device=dev)
            cos = s["cos_sin"][x][:, freq].to(f64)[:, None]
            sin = s["cos_sin"][x][:, half + freq].to(f64)[:, None]
            k = s["k"][a:b].to(f64)
            for t in (q[a:b], k):
                t[..., :rot] = t[..., :rot] * cos + sign * t[..., :rot][..., partner] * sin
            at = s["table"][i][x // page].long()
            kc[at, x % page] = k
            vc[at, x % page] = s["v"][a:b].to(f64)
        return q, kc, vc
    W, S = case["window"], case["sinks"]
    G = Hq // Hkv
    out = torch.zeros(s["T"], Hq, D, dtype=f64, device=dev)
    lse = torch.zeros(s["T"], Hq, dtype=f64, device=dev)
    for i in range(case["B"]):
        a, b = s["off"][i], s["off"][i + 1]
        kv = s["kv"][i]
        pages = s["table"][i][:(kv + page - 1) // page].long()
        x = torch.arange(kv, device=dev)
        p = torch.arange(kv - (b - a), kv, device=dev)[:, None]
        hidden = x > p
        if W:
            hidden = hidden | ((x <= p - W) & (x >= S))
        live = (~hidden).any(0)
        for h in range(Hkv):
            k = s["k_cache"][:, :, h][pages].flatten(0, 1)[:kv][live].to(f64)
            v = s["v_cache"][:, :, h][pages].flatten(0, 1)[:kv][live].to(f64)
            for g in range(h * G, h * G + G):
                z = (s["q"][a:b, g].to(f64) @ k.T) / math.sqrt(D)
                z[hidden[:, live]] = -math.inf
                lse[a:b, g] = torch.logsumexp(z, 1)
                out[a:b, g] = torch.softmax(z, 1) @ v
    return out, lse
