"""Cases of the paged cache held in 8 bits and of its pages: appending a round's keys and values to
e4m3 blocks with a scale for each page and head, attention of the round's rows over that cache, and the
block tables and slot maps that the two go by, built from the requests' lengths.

Layout, as for the verifier: request i owns rows row_off[i] .. row_off[i+1]-1 of the batch; its
n_i rows are the last n_i of its kv_len[i] positions; position x lies in slot x % page of page
block_table[i][x // page]. Element (b, s, h, d) of the cache stands for cache[b, s, h, d] * scale[b, h].

A case's shapes (rows and lengths of each request) follow from its own numbers ("shape" seeds
them); the values follow from the seed given to prepare().
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
TOP = 448.0        # the largest e4m3
LEAST = 2.0 ** -60  # the least scale an append sets


# ------------------------------------------------------------------------------------- cases

def _append(name, shape, B, rows, ctx, Hq, Hkv, D, page, dtype, rot, interleaved=False, order="slot"):
    return dict(name=name, op="append", shape=shape, B=B, rows_lo=rows[0], rows_hi=rows[1], ctx_lo=ctx[0],
                ctx_hi=ctx[1], Hq=Hq, Hkv=Hkv, D=D, page=page, dtype=dtype, rot=rot, interleaved=interleaved,
                order=order)


def _attend(name, shape, B, rows, ctx, Hq, Hkv, D, page, dtype, window=0, sinks=0, shared=0, order="slot"):
    return dict(name=name, op="attend", shape=shape, B=B, rows_lo=rows[0], rows_hi=rows[1], ctx_lo=ctx[0],
                ctx_hi=ctx[1], Hq=Hq, Hkv=Hkv, D=D, page=page, dtype=dtype, window=window, sinks=sinks,
                shared=shared, order=order)


def _tables(name, shape, B, rows, ctx, page, shared=0):
    return dict(name=name, op="tables", shape=shape, B=B, rows_lo=rows[0], rows_hi=rows[1], ctx_lo=ctx[0],
                ctx_hi=ctx[1], page=page, shared=shared)


def listed():
    return [
        # one user's round of four drafts: five rows, a thousand tokens in; latency is all that counts
        _append("append8_one", 1, 1, (5, 5), (1000, 1000), 32, 8, 128, 16, "bf16", 128),
        # the ragged batch of 64 requests with up to seven drafts, at any point of their texts
        _append("append8_round", 2, 64, (1, 8), (1, 16000), 32, 8, 128, 16, "bf16", 128),
        # 256 requests of three drafts after 4096-token prefixes, rows in fp32; part of each head rotated, as
        # interleaved pairs; the cache holds each head's slots together
        _append("append8_round_f32", 3, 256, (4, 4), (4096, 4096), 12, 4, 128, 16, "f32", 64, True, "head"),
        # whole prompts entering the cache, heads of 64 without sharing
        _append("append8_prompts", 4, 6, (500, 4000), (0, 700), 12, 12, 64, 64, "bf16", 64),
        # one user's round of four drafts after a thousand tokens
        _attend("attend8_one", 5, 1, (5, 5), (1000, 1000), 32, 8, 128, 16, "bf16"),
        # the ragged batch under a sliding window with four sinks
        _attend("attend8_round_window", 6, 64, (1, 8), (1, 16000), 32, 8, 128, 16, "bf16", 1024, 4),
        # few users deep in long texts, every token visible: the cache's bytes are the work
        _attend("attend8_round_long", 7, 16, (1, 8), (4000, 65000), 32, 8, 128, 16, "bf16"),
        # rows in fp32 after up to 4096 tokens, heads' slots together
        _attend("attend8_round_f32", 8, 64, (1, 4), (1, 4096), 12, 4, 128, 16, "f32", 0, 0, 0, "head"),
        # prompts of a few thousand tokens, some continuing a cached part: arithmetic is the work
        _attend("attend8_prompts", 9, 4, (1000, 2500), (0, 6000), 32, 8, 128, 64, "bf16"),
        # the ragged batch behind an 8192-token document that is kept once
        _attend("attend8_shared", 10, 64, (1, 8), (1, 1000), 32, 8, 128, 16, "bf16", 0, 0, 8192),
        # the ragged batch's tables before a round, and again when the round has been refused
        _tables("tables_round", 11, 64, (1, 8), (1, 16000), 16),
        # 512 prompts admitted behind one instruction text, and their pages given back
        _tables("tables_prompts", 12, 512, (1, 2000), (0, 0), 16, 1000),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ranges."""
    ref = listed()
    while True:
        kind = rng.choice(["append", "append", "attend", "attend", "attend", "shared", "tables"])
        dtype = "f32" if rng.random() < 0.2 else "bf16"
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 3, 4, 8])
        page = rng.choice([8, 16, 24, 32, 64])
        order = rng.choice(["slot", "slot", "head"])
        D = rng.choice([64, 80, 96, 128, 128])
        shape = rng.randrange(1 << 30)
        if kind == "tables":
            B = _log_int(rng, 1, 512)
            if rng.random() < 0.5:
                rows, ctx = (1, rng.randint(1, 8)), (1, _log_int(rng, 10, 16000))
            else:
                rows, ctx = (1, _log_int(rng, 50, 2000)), (0, rng.choice([0, _log_int(rng, 1, 6000)]))
            case = _tables("", shape, B, rows, ctx, page, rng.choice([0, 0, _log_int(rng, 1, 8192)]))
        elif kind == "append":
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
        same = [c for c in ref if c["op"] == case["op"] and (case.get("dtype") != "f32" or c["dtype"] == "f32")]
        w = work(case)
        if all(w[k] <= max(work(c)[k] for c in same) for k in ("bytes", "flops")) and _pool_tokens(case) <= 1100000:
            return case


# -------------------------------------------------------------------------- shapes and work

def _shape(case):
    """(rows, ctx) of each request: rows of this call, and positions before them (the shared
    prefix among them)."""
    r = random.Random(case["shape"])
    rows = [r.randint(case["rows_lo"], case["rows_hi"]) for _ in range(case["B"])]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) + case.get("shared", 0) for _ in range(case["B"])]
    return rows, ctx


def _blocks(x, page):
    return (x + page - 1) // page


def _pool_tokens(case):
    rows, ctx = _shape(case)
    if case["op"] == "append":
        return sum(rows) + case["B"] * case["page"] * 2
    if case["op"] == "tables":
        return 0
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
    T, B, page = sum(rows), case["B"], case["page"]
    if case["op"] == "tables":
        new = sum(_blocks(c + n, page) - (_blocks(c, page) if case["ctx_hi"] else case["shared"] // page)
                  for n, c in zip(rows, ctx))
        # two calls: lengths, counts and offsets in, counts out; pages to the tables and back; the rows' slots
        # and positions
        return {"bytes": 2 * (4 * B * 4 + 8 * new) + 8 * T, "flops": 0}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    eb = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "append":
        pages = sum((c + n - 1) // page - c // page + 1 for n, c in zip(rows, ctx))
        byt = 2 * T * Hq * D * eb + 2 * T * Hkv * D * (eb + 1) + T * case["rot"] * 4 + (B + 1 + B) * 4
        byt += pages * (4 + 2 * Hkv * 4) + sum(2 * Hkv * 4 for c in ctx if c % page)
        return {"bytes": byt, "flops": 3 * T * (Hq + Hkv) * case["rot"] + 4 * T * Hkv * D}
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
    byt = 2 * T * Hq * D * eb + 4 * T * Hq + 2 * keys * Hkv * D + (4 + 8 * Hkv) * (keys // page + 2 * B)
    return {"bytes": byt, "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------------------------ inputs

def _scale_for(amax):
    """The least power of two s with amax <= 448 s (frexp: amax / 448 = f 2^e, f in [0.5, 1))."""
    f, e = torch.frexp(amax.double() / TOP)
    s = torch.ldexp(torch.ones_like(f), torch.where(f == 0.5, e - 1, e))
    return torch.where(amax == 0, torch.zeros_like(s), s).clamp_min(LEAST).float()


def _cache(n_pages, case, gen, dev):
    """A pool of earlier tokens' values in e4m3 [pages, slots, heads, D] and their scales [pages, heads]; the
    heads' magnitudes differ. "head" keeps a head's slots of a page together in memory."""
    page, H, D = case["page"], case["Hkv"], case["D"]
    loud = torch.exp2(torch.randn(H, generator=gen, device=dev))[:, None, None]
    x = torch.randn(n_pages, H, page, D, generator=gen, device=dev) * loud
    scale = _scale_for(x.abs().amax((2, 3)))
    x = (x / scale[:, :, None, None]).to(E4M3)
    x = x.permute(0, 2, 1, 3)
    if case["order"] == "slot":  # (copied as bytes)
        x = x.view(torch.uint8).contiguous().view(E4M3)
    return x, scale


def _lengths(case):
    rows, ctx = _shape(case)
    off = [0]
    for n in rows:
        off.append(off[-1] + n)
    kv = [c + n for n, c in zip(rows, ctx)]
    dev = torch.device("cuda")
    i32 = dict(dtype=torch.int32, device=dev)
    return dict(case=case, rows=rows, ctx=ctx, kv=kv, off=off, T=off[-1], row_off=torch.tensor(off, **i32),
                kv_len=torch.tensor(kv, **i32)), i32, dev


def _table_inputs(case, seed):
    """Requests in mid-text (or, with no text of their own yet, without any page) with pages from all over the
    pool, the rest of the pool on the free stack."""
    s, i32, dev = _lengths(case)
    r = random.Random(seed * 7919 + case["shape"])
    page, B, sh = case["page"], case["B"], case["shared"] // case["page"]
    s["before"] = [c if case["ctx_hi"] else 0 for c in s["ctx"]]
    held = [_blocks(c, page) for c in s["before"]]
    s["width"] = width = max(_blocks(x, page) for x in s["kv"]) + 8
    own_pages = sum(max(h - sh, 0) for h in held)
    new = sum(max(_blocks(x, page) - max(h, sh), 0) for x, h in zip(s["kv"], held))
    s["n_pages"] = n_pages = sh + own_pages + new + 100
    ids = list(range(n_pages))
    r.shuffle(ids)
    tab, nxt = [], sh
    for h in held:
        k = max(h - sh, 0)
        tab.append((ids[:sh] if h else [-1] * sh) + ids[nxt:nxt + k] + [-1] * (width - sh - k))
        nxt += k
    free = ids[nxt:]
    s["shared_table"] = torch.tensor(ids[:sh], **i32) if sh else None
    s["table"] = torch.tensor(tab, **i32)
    s["n_blocks"] = torch.tensor(held, **i32)
    s["free"] = torch.tensor(free + [-1] * (n_pages - len(free)), **i32)
    s["n_free"] = torch.tensor([len(free)], **i32)
    s["before_len"] = torch.tensor(s["before"], **i32)
    return s


def _inputs(case, seed):
    if case["op"] == "tables":
        return _table_inputs(case, seed)
    s, i32, dev = _lengths(case)
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 1000003 + case["shape"])
    r = random.Random(seed * 7919 + case["shape"])
    kv, ctx, T = s["kv"], s["ctx"], s["T"]
    B, page, L = case["B"], case["page"], case.get("shared", 0)
    width = max(_blocks(x, page) for x in kv)
    tab = [[-1] * width for _ in range(B)]
    # pages: first the ones all requests share, then each request's own; a request's own part that
    # begins inside a shared page has a page of its own there, with the same tokens before it
    if case["op"] == "append":  # only the tail is written: pages before it are common to all
        common = [c // page for c in ctx]
    else:
        common = [L // page] * B
    n_shared = max([*common, _blocks(L, page)])
    if case["op"] == "append":
        n_shared = min(n_shared, 64)  # what they hold does not matter here: few pages stand for all
    ids = list(range(n_shared + sum(_blocks(x, page) - c for x, c in zip(kv, common))))
    r.shuffle(ids)
    nxt = n_shared
    for i in range(B):
        for b in range(_blocks(kv[i], page)):
            if b < common[i]:
                tab[i][b] = ids[b % max(n_shared, 1)]
            else:
                tab[i][b] = ids[nxt]
                nxt += 1
    s["table"] = torch.tensor(tab, **i32)
    s["k_cache"], s["k_scale"] = _cache(len(ids), case, gen, dev)
    s["v_cache"], s["v_scale"] = _cache(len(ids), case, gen, dev)
    dt = DTYPES[case["dtype"]]
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if L:
        s["shared_table"] = torch.tensor(ids[:_blocks(L, page)], **i32)
        if L % page:  # the requests' own copies of the last shared page hold the same tokens
            last = torch.tensor([tab[i][L // page] for i in range(B)], device=dev)
            for c in ("k", "v"):
                bits = s[c + "_cache"].view(torch.uint8)
                bits[last, :L % page] = bits[ids[L // page], :L % page].clone()
                s[c + "_scale"][last] = s[c + "_scale"][ids[L // page]].clone()
    if case["op"] == "append":
        # the rows come out of one projection: q, k and v side by side, some tokens louder than others
        loud = torch.where(torch.rand(T, 1, generator=gen, device=dev) < 0.1, 5.0, 1.0)
        qkv = (torch.randn(T, (Hq + 2 * Hkv) * D, generator=gen, device=dev) * loud).to(dt)
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
        if case["op"] == "tables":
            grow = api.BlockTables(case["B"], s["T"], case["page"], s["n_pages"])
            back = api.BlockTables(case["B"], 0, case["page"], s["n_pages"])
            pool = (s["n_blocks"], s["table"], s["free"], s["n_free"])
            s["call"] = (grow.bind(s["kv_len"], *pool, row_off=s["row_off"], shared_table=s["shared_table"]),
                         back.bind(s["before_len"], *pool, shared_table=s["shared_table"]))
            return s
        dims = (case["B"], s["T"], case["Hq"], case["Hkv"], case["D"], DTYPES[case["dtype"]])
        cache = (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        if case["op"] == "append":
            s["call"] = api.KvAppender8(*dims, rot_dim=case["rot"], interleaved=case["interleaved"])
            s["call"].bind(s["q"], s["k"], s["v"], s["cos_sin"], s["row_off"], s["kv_len"], *cache, s["table"])
        else:
            s["call"] = api.Attention8(*dims, window=case["window"], n_sink=case["sinks"], shared_len=case["shared"])
            s["call"].bind(s["q"], *cache, s["row_off"], s["kv_len"], s["table"], shared_table=s.get("shared_table"))
    return s


# ------------------------------------------------------------------------------ one pass

def run(state):
    s, case = state, state["case"]
    if case["op"] == "tables":
        # pages for the round's rows, and back again: the second call undoes the first
        if own:
            grow, back = s["call"]
            o = grow.run()
            back.run()
            slot_map, positions = o.slot_map, o.positions
        else:
            slot_map, positions = _plain_tables(s, case, s["kv_len"], s["T"])
            _plain_tables(s, case, s["before_len"], 0)
        return slot_map, positions, s["table"], s["n_blocks"], s["free"], s["n_free"]
    if case["op"] == "append":
        q = s["call"].run().q if own else _plain_append(s, case)
        return q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
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


def _store8(x, cache, scale, pages, slots, first_pages, kept):
    """Rows x [T, H, D] to the cache's slots. A page's scale is the least power of two that holds the new
    values, but not less than what it was where earlier tokens stay in the page (first_pages [B], of which
    the first `kept` slots): they are brought to the new scale."""
    amax = torch.zeros_like(scale).index_reduce_(0, pages, x.abs().amax(-1), "amax")
    touched = torch.zeros(scale.shape[0], dtype=torch.bool, device=x.device)
    touched[pages] = True
    stays = torch.zeros_like(touched)
    stays[first_pages] = kept > 0
    was = scale.clone()
    new = torch.maximum(_scale_for(amax), torch.where(stays[:, None], was, 0.0))
    scale.copy_(torch.where(touched[:, None], new, was))
    by = (was / scale)[first_pages][:, None, :, None]
    old = cache[first_pages]
    mine = (torch.arange(cache.shape[1], device=x.device)[None] < kept[:, None])[:, :, None, None]
    cache[first_pages] = torch.where(mine, old.float() * by, old.float()).to(E4M3)
    cache[pages, slots] = (x / scale[pages][..., None]).to(E4M3)


def _plain_append(s, case):
    rot, page = case["rot"], case["page"]
    pos, req = _positions(s)
    cos, sin = s["cos_sin"][pos][:, None, :rot // 2], s["cos_sin"][pos][:, None, rot // 2:]
    q = _rotate(s["q"], cos, sin, rot, case["interleaved"]).to(s["q"].dtype)
    k = _rotate(s["k"], cos, sin, rot, case["interleaved"])
    pages, slots = s["table"][req, pos // page].long(), pos % page
    base = (s["kv_len"] - (s["row_off"][1:] - s["row_off"][:-1])).long()
    first = torch.gather(s["table"].long(), 1, (base // page)[:, None])[:, 0]
    _store8(k, s["k_cache"], s["k_scale"], pages, slots, first, base % page)
    _store8(s["v"].float(), s["v_cache"], s["v_scale"], pages, slots, first, base % page)
    return q


def _part(q, k, v, seen, scale):
    """Softmax parts of rows q [.., n, D] over keys k, v [.., x, D] (seen [.., n, x]): row maxima, sums and
    unnormalised outputs."""
    z = (torch.matmul(q, k.transpose(-1, -2)) * scale).masked_fill(~seen, -math.inf)
    m = z.amax(-1)
    p = torch.exp(z - torch.where(m == -math.inf, 0.0, m)[..., None])
    return m, p.sum(-1), torch.matmul(p, v)


def _plain_attend(s, case):
    W, S, L, page = case["window"], case["sinks"], case["shared"], case["page"]
    Hq, Hkv, D, B, T = case["Hq"], case["Hkv"], case["D"], case["B"], s["T"]
    G, n = Hq // Hkv, max(s["rows"])
    dev = s["q"].device
    q = s["q"].float().view(T, Hkv, G, D)
    pos, req = _positions(s)

    def keys(pages, x):
        """Keys and values of positions x [.., X] in pages [.., X]: [.., Hkv, X, D]."""
        return [(s[c + "_cache"][pages, x % page].float() * s[c + "_scale"][pages][..., None]).transpose(-2, -3)
                for c in ("k", "v")]

    # the rows of each request side by side, up to the longest's
    j = torch.arange(T, device=dev) - s["row_off"].long()[req]
    qb = torch.zeros(B, n, Hkv, G, D, device=dev)
    qb[req, j] = q
    p = torch.full((B, n), -1, dtype=torch.long, device=dev)
    p[req, j] = pos
    # the positions that some row of a request sees, from L on: the window's (or all), then the sinks
    kv = s["kv_len"].long()
    rows = (s["row_off"][1:] - s["row_off"][:-1]).long()
    w0 = (kv - rows - W + 1).clamp_min(L) if W else torch.full_like(kv, L)
    span = min(max(s["kv"]) - L, W - 1 + n) if W else max(s["kv"]) - L
    x = w0[:, None] + torch.arange(span, device=dev)
    live = x < kv[:, None]
    if W and S > L:
        sink = L + torch.arange(S - L, device=dev)[None].expand(B, -1)
        x, live = torch.cat([x, sink], 1), torch.cat([live, (sink < S) & (sink < w0[:, None])], 1)
    x = torch.where(live, x, 0)
    pages = torch.gather(s["table"].long(), 1, x // page).clamp_min(0)
    seen = live[:, None] & (x[:, None] <= p[..., None])
    if W:
        seen &= (x[:, None] > p[..., None] - W) | (x[:, None] < S)
    k, v = keys(pages, x)
    grouped = seen[:, None, :, None].expand(-1, Hkv, -1, G, -1).reshape(B, Hkv, n * G, -1)
    m, l, o = _part(qb.permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D), k, v, grouped, D ** -0.5)
    m, l = (t.view(B, Hkv, n, G).permute(0, 2, 1, 3)[req, j] for t in (m, l))  # [T, Hkv, G]
    o = o.view(B, Hkv, n, G, D).permute(0, 2, 1, 3, 4)[req, j]
    if L:
        x = torch.arange(L, device=dev)
        seen = x[None] <= pos[:, None]
        if W:
            seen &= (x[None] > pos[:, None] - W) | (x[None] < S)
        k, v = keys(s["shared_table"].long()[x // page], x)
        m1, l1, o1 = _part(q.permute(1, 0, 2, 3).reshape(Hkv, T * G, D), k, v,
                           seen.repeat_interleave(G, 0)[None], D ** -0.5)
        m1, l1 = (t.view(Hkv, T, G).transpose(0, 1) for t in (m1, l1))
        o1 = o1.view(Hkv, T, G, D).transpose(0, 1)
        mm = torch.maximum(m, m1)
        e, e1 = torch.exp(m - mm), torch.exp(m1 - mm)
        m, l, o = mm, l * e + l1 * e1, o * e[..., None] + o1 * e1[..., None]
    return (o / l[..., None]).reshape(T, Hq, D).to(s["q"].dtype), (m + torch.log(l)).reshape(T, Hq)


def _plain_tables(s, case, lengths, T):
    """Brings every request's table to its length: pages are given back (the last request's last page
    first) and then taken from the top of the stack, request after request."""
    page, sh, width = case["page"], case["shared"] // case["page"], s["width"]
    table, held, free, n_free = s["table"], s["n_blocks"], s["free"], s["n_free"]
    dev = table.device
    need = (lengths + page - 1) // page
    have, want = (held - sh).clamp_min(0), (need - sh).clamp_min(0)
    back, take = (have - want).clamp_min(0), (want - have).clamp_min(0)
    b = torch.arange(width, device=dev)[None]
    # given back: request i's block b goes to the stack behind those of the requests after it and of the
    # blocks after it
    after = back.flip(0).cumsum(0).flip(0) - back
    going = (b >= sh + want[:, None]) & (b < sh + have[:, None])
    at = torch.where(going, n_free + after[:, None] + sh + have[:, None] - 1 - b, free.numel())
    stack = torch.cat([free, free.new_zeros(1)]).scatter(0, at.flatten(), table.flatten())
    # taken: block b of request i is the stack's entry below those of the requests before it
    before = take.cumsum(0) - take
    total = n_free + back.sum()
    coming = (b >= sh + have[:, None]) & (b < sh + want[:, None])
    at = torch.where(coming, total - 1 - before[:, None] - (b - sh - have[:, None]), 0)
    table.copy_(torch.where(coming, stack[at], table))
    if sh:
        first = (b < sh) & (b >= held[:, None]) & (b < need[:, None])
        table.copy_(torch.where(first, torch.cat([s["shared_table"], s["shared_table"].new_zeros(width - sh)]), table))
    free.copy_(stack[:-1])
    n_free.copy_(total - take.sum())
    held.copy_(need)
    if not T:
        return None
    pos, req = _positions(s)
    return (table[req, pos // page] * page + pos % page).int(), pos.int()


# ------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "tables":
        return _exact_tables(s, case)
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
        q = s["q"].to(f64)
        caches = [s[c + "_cache"].to(f64) for c in ("k", "v")]
        scales = [s[c + "_scale"].to(f64) for c in ("k", "v")]
        for i in range(case["B"]):
            a, b = s["off"][i], s["off"][i + 1]
            c0 = s["ctx"][i]
            x = torch.arange(c0, s["kv"][i], device=dev)
            cos = s["cos_sin"][x][:, freq].to(f64)[:, None]
            sin = s["cos_sin"][x][:, half + freq].to(f64)[:, None]
            k = s["k"][a:b].to(f64)
            for t in (q[a:b], k):
                t[..., :rot] = t[..., :rot] * cos + sign * t[..., :rot][..., partner] * sin
            ids = s["table"][i].tolist()
            for y, cache, scale in zip((k, s["v"][a:b].to(f64)), caches, scales):
                for blk in range(c0 // page, (s["kv"][i] - 1) // page + 1):
                    x0, x1 = max(c0, blk * page), min(s["kv"][i], (blk + 1) * page)
                    rows, kept = y[x0 - c0:x1 - c0], x0 - blk * page
                    least = torch.exp2(torch.ceil(torch.log2(rows.abs().amax((0, 2)) / TOP)))
                    new = least.clamp_min(LEAST)
                    if kept:
                        new = torch.maximum(new, scale[ids[blk]])
                        cache[ids[blk], :kept] *= (scale[ids[blk]] / new)[None, :, None]
                    scale[ids[blk]] = new
                    cache[ids[blk], kept:kept + x1 - x0] = rows / new[None, :, None]
        return q, caches[0], caches[1], scales[0], scales[1]
    W, S = case["window"], case["sinks"]
    G = Hq // Hkv
    out = torch.zeros(s["T"], Hq, D, dtype=f64, device=dev)
    lse = torch.zeros(s["T"], Hq, dtype=f64, device=dev)
    for i in range(case["B"]):
        a, b = s["off"][i], s["off"][i + 1]
        kv = s["kv"][i]
        pages = s["table"][i][:_blocks(kv, page)].long()
        x = torch.arange(kv, device=dev)
        p = torch.arange(kv - (b - a), kv, device=dev)[:, None]
        hidden = x > p
        if W:
            hidden = hidden | ((x <= p - W) & (x >= S))
        live = (~hidden).any(0)
        for h in range(Hkv):
            k, v = ((s[c + "_cache"][pages, :, h].to(f64) * s[c + "_scale"][pages, h].to(f64)[:, None, None])
                    .flatten(0, 1)[:kv][live] for c in ("k", "v"))
            for g in range(h * G, h * G + G):
                z = (s["q"][a:b, g].to(f64) @ k.T) / math.sqrt(D)
                z[hidden[:, live]] = -math.inf
                lse[a:b, g] = torch.logsumexp(z, 1)
                out[a:b, g] = torch.softmax(z, 1) @ v
    return out, lse


def _exact_tables(s, case):
    """The same by hand: one stack of page numbers, popped and pushed."""
    page, sh = case["page"], case["shared"] // case["page"]
    table, held = s["table"].tolist(), s["n_blocks"].tolist()
    n_free = int(s["n_free"])
    tail = s["free"].tolist()
    stack = tail[:n_free]
    shared = s["shared_table"].tolist() if sh else []
    slot_map, positions = [], []
    for lengths in (s["kv"], s["before"]):
        need = [_blocks(x, page) for x in lengths]
        for i in reversed(range(case["B"])):
            for b in reversed(range(max(need[i], sh), held[i])):
                stack.append(table[i][b])
                tail[len(stack) - 1] = table[i][b]
        for i in range(case["B"]):
            for b in range(held[i], need[i]):
                table[i][b] = shared[b] if b < sh else stack.pop()
        held = need
        if lengths is s["kv"]:
            for i in range(case["B"]):
                for x in range(s["ctx"][i], s["kv"][i]):
                    positions.append(x)
                    slot_map.append(table[i][x // page] * page + x % page)
    i32 = dict(dtype=torch.int32, device=s["table"].device)
    return (torch.tensor(slot_map, **i32), torch.tensor(positions, **i32), torch.tensor(table, **i32),
            torch.tensor(held, **i32), torch.tensor(tail, **i32), torch.tensor([n_free], **i32))
