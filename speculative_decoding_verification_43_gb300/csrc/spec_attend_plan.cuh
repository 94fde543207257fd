// How the attention of a ragged batch over the paged cache is cut into work, computed on the device
// (lengths and offsets are device arrays).
//
// Rows that share a key/value head are packed: row r of a request's head is (row j, query head g of
// the group) = (r / G, r % G). An item is up to RT packed rows of one head; its keys, in tiles of KT
// positions, are its units, behind some that stand for the time an item takes whatever its keys are (its
// queries, its first references, its way out). Units are numbered item after item, and worker w of NW takes its
// share of consecutive units: every worker gets the same amount of work, give or take a tile, whatever the
// lengths are, a long context is split over many workers, and the cut depends on the inputs alone. An item
// that falls to several workers leaves a part (output, maximum, sum) per worker, and the joining
// kernel adds the parts in the order of the workers.
//
// Two classes of items. A call without a shared prefix has "own" items: a request's rows over its
// positions. With one, the own items begin at shared_len, and "prefix" items take the rows of the
// whole batch over the positions below it.
#pragma once

#include <climits>
#include <cstdint>

#include "spec_attend.h"
#include "spec_device.cuh"
#include "spec_paged.cuh"

namespace spec {

// An item that several workers share, as the joining kernel needs it: written by the worker that begins it
// (calls without a shared prefix; nrows = 0: this worker begins none).
struct CutItem {
    int req, t0, row0, nrows, head;
    int parts;      // workers (every head_step-th), this one first
    int slot;       // this worker's slot of two; the others have their first
    int pad;
};

struct AttendParams {
    int32_t B, T, Hq, Hkv, G, D;
    int32_t page_size;
    FastDiv by_page, by_group;      // by page_size and G
    int32_t box_log2;               // slots copied as one box (a divisor of page_size), as a power of two
    int32_t max_blocks, n_pages, window, n_sink, shared_len;
    float scale_log2;  // scale * log2(e): the softmax is taken in base 2
    const void *q, *k_cache, *v_cache;
    const float *k_scale, *v_scale;  // [n_pages][Hkv], a cache in 8 bits
    int64_t q_stride, page_stride, slot_stride, head_stride;
    const int32_t *row_off, *kv_len, *block_table, *shared_table;
    void *out;
    int64_t out_stride;
    float *lse;
    int32_t *req_status;
    // workspace
    int32_t *status;       // [B]
    int32_t *unit_prefix;  // [B+1] units of the own items before each request
    CutItem *cut;          // [own workers]
    int32_t *prefix_units; // units of a prefix item
    int32_t *broken;       // 1: some request's offsets are wrong
    float2 *part_ml;       // [part rows] maximum (base 2, scaled) and sum
    float *part_o;         // [part rows][D] unnormalised output
    int32_t *err;          // [workers of both classes] 1: a bounded wait gave up
    int32_t own_workers, prefix_workers;
    int32_t own_rt_log2, prefix_rt_log2;  // packed rows of an item (RT), as a power of two
    int32_t own_pitch, prefix_pitch;      // rows of a worker's part
    int32_t own_extra, prefix_extra;      // units of an item beside its tiles
    int32_t head_step;  // heads that workers side by side take in step (a divisor of Hkv and own_workers; 1 with a
                        // shared prefix): they number the units of every head_step-th head alone
    int64_t part_rows;
};

// ---------------------------------------------------------------- positions and pages

struct ReqRows {
    int r0, n, kv;  // first row, rows, positions; n = 0 / kv = 0 where the batch is inconsistent
};
__device__ __forceinline__ ReqRows load_request(const AttendParams &P, int i) {
    const int r0 = P.row_off[i], r1 = P.row_off[i + 1];
    int kv = P.kv_len[i];
    if (!offsets_right(r0, r1, P.T)) return {0, 0, 0};
    if (kv < 0 || kv > static_cast<int64_t>(P.max_blocks) * P.page_size) kv = 0;
    return {r0, r1 - r0, kv};
}

// The same without rows that other offsets leave in doubt, which are looked for where some request's offsets
// are wrong (broken).
__device__ __forceinline__ ReqRows held_request(const AttendParams &P, int i, bool broken) {
    const ReqRows q = load_request(P, i);
    if (broken && q.n > 0 && offsets_contradict(P.row_off, P.B, P.T, i, q.r0, q.r0 + q.n, 0, 1)) return {0, 0, 0};
    return q;
}

// Element offset of position x's slot (head 0), or -1 when it has no page.
__device__ __forceinline__ int64_t slot_offset(const AttendParams &P, const int32_t *table, int x) {
    const int b = P.by_page(x);
    const int page = table[b];
    if (page < 0 || page >= P.n_pages) return -1;
    return page * P.page_stride + (x - b * P.page_size) * P.slot_stride;
}

// The key tiles an item visits: of the tiles of KT positions from lo, the first s (the sinks), then
// those from w_first on (the window); n in all. Some row of the item sees a position of [from, hi) that is
// at or above win, or below the sinks. lo is from, rounded down so that a copied box of slots
// (P.box_log2) lies in one page.
struct KeyTiles {
    int lo, from, hi, win, s, w_first, n;
};
template <int KT>
__device__ __forceinline__ KeyTiles key_tiles(const AttendParams &P, int from, int hi, int pmin) {
    const int lo = from >> P.box_log2 << P.box_log2;
    KeyTiles t = {lo, from, hi, from, 0, 0, 0};
    if (hi <= from) return t;
    const int total = (hi - lo + KT - 1) / KT;
    if (P.window > 0) {
        t.win = max(from, pmin - P.window + 1);
        const int sinks = min(P.n_sink, hi) - lo;
        t.w_first = t.win < hi ? (t.win - lo) / KT : total;
        t.s = P.n_sink > from ? min((sinks + KT - 1) / KT, t.w_first) : 0;
    }
    t.n = t.s + total - t.w_first;
    return t;
}
template <int KT>
__device__ __forceinline__ int tile_begin(const KeyTiles &t, int i) {
    return t.lo + (i < t.s ? i : i - t.s + t.w_first) * KT;
}
// True when some row of the item may see a position of [x, x + n).
__device__ __forceinline__ bool item_sees(const AttendParams &P, const KeyTiles &t, int x, int n = 1) {
    const int a = max(x, t.from), b = min(x + n, t.hi);
    return a < b && (b > t.win || a < P.n_sink);
}

// ---------------------------------------------------------------- items and units
// Unit numbers are 32-bit: the host refuses sizes that could have more.

template <int KT>
__device__ __forceinline__ KeyTiles own_tiles(const AttendParams &P, const ReqRows &q, int k) {
    const int base = q.kv - q.n, r0 = k << P.own_rt_log2, r1 = r0 + (1 << P.own_rt_log2), end = q.n * P.G;
    const int j0 = P.by_group(r0), j1 = P.by_group(min(r1, end) - 1);
    return key_tiles<KT>(P, P.shared_len, base + j1 + 1, max(base + j0, 0));
}
// Row tiles of n rows of G query heads.
__device__ __forceinline__ int row_tiles(int rows, int rt_log2) { return (rows + (1 << rt_log2) - 1) >> rt_log2; }
// Tiles of an item, one at least (an item without keys has rows to write too).
__device__ __forceinline__ int item_tiles(const KeyTiles &t) { return max(t.n, 1); }
// Units of one head of a request.
template <int KT>
__device__ __forceinline__ int own_units(const AttendParams &P, const ReqRows &q) {
    int u = 0;
    const int tiles = row_tiles(q.n * P.G, P.own_rt_log2);
#pragma unroll 1
    for (int k = 0; k < tiles; ++k) u += item_tiles(own_tiles<KT>(P, q, k)) + P.own_extra;
    return u;
}

// A class's units over its workers: as many workers as there are units at most, the first `more` of them
// with one unit more than the others' `each`.
struct Shares {
    int each, more, workers;
    __device__ __forceinline__ Shares(int total, int limit) {
        workers = min(total, limit);
        each = workers > 0 ? total / workers : 0;
        more = total - each * workers;
    }
    // The first unit of worker w (total, past the last one).
    __device__ __forceinline__ int first(int w) const {
        const int x = min(w, workers);
        return each * x + min(x, more);
    }
    // The worker of unit u.
    __device__ __forceinline__ int owner(int u) const {
        const int longer = more * (each + 1);
        return u < longer ? u / (each + 1) : more + (u - longer) / each;
    }
};

// The batch as a whole, by one warp: units of the own items, least and greatest position of the rows
// (padding aside), and whether some request's offsets are wrong (then a second pass leaves out the rows in
// doubt: with them the units need not stay within the host's bound). Lane l has requests [l * per, (l + 1) * per),
// and `before` units lie before them.
struct Totals {
    int units, before, per, pmin, pmax;
    bool broken;
};
template <int KT>
__device__ __forceinline__ Totals batch_totals(const AttendParams &P, int lane) {
    Totals t = {0, 0, (P.B + kWarp - 1) / kWarp, INT_MAX, -1, false};
    int mine;
#pragma unroll 1
    for (;;) {
        bool wrong = false;
        mine = 0;
#pragma unroll 1
        for (int i = lane * t.per; i < min(P.B, (lane + 1) * t.per); ++i) {
            const ReqRows q = held_request(P, i, t.broken);
            if (q.n > 0 && q.kv > 0) {
                t.pmin = min(t.pmin, max(q.kv - q.n, 0));
                t.pmax = max(t.pmax, q.kv - 1);
            }
            mine += P.Hkv / P.head_step * own_units<KT>(P, q);
            wrong |= !offsets_right(P.row_off[i], P.row_off[i + 1], P.T);
        }
        if (t.broken || !__any_sync(0xffffffffu, wrong)) break;
        t.broken = true;
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < kWarp; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    t.before = incl - mine;
    t.units = __shfl_sync(0xffffffffu, incl, kWarp - 1);
    t.pmin = __reduce_min_sync(0xffffffffu, t.pmin);
    t.pmax = __reduce_max_sync(0xffffffffu, t.pmax);
    return t;
}
// Leaves the units before each request, and those of all, to the joining kernel of a call with a shared
// prefix (one warp).
template <int KT>
__device__ __forceinline__ void record_units(const AttendParams &P, int lane) {
    const Totals t = batch_totals<KT>(P, lane);
    int u = t.before;
#pragma unroll 1
    for (int i = lane * t.per; i < min(P.B, (lane + 1) * t.per); ++i) {
        if (SPEC_IN(i, P.B, DBG_ATTEND)) P.unit_prefix[i] = u;
        u += P.Hkv * own_units<KT>(P, held_request(P, i, t.broken));
    }
    if (lane == 0) P.unit_prefix[P.B] = t.units;
}
template <int KT>
__device__ __forceinline__ KeyTiles prefix_tiles(const AttendParams &P, const Totals &t) {
    return key_tiles<KT>(P, 0, min(P.shared_len, t.pmax + 1), t.pmin);
}

// A run of units of one item, as a worker takes it.
struct Segment {
    int row0;        // first packed row (own: within the request's head; prefix: within the batch)
    int nrows;       // packed rows, at most RT (0: the worker has no more)
    int t0;          // first row of the request in the batch (prefix: 0)
    int base;        // position of row t0 (prefix: unused, rows have their own)
    int head;        // key/value head
    int req;         // request, -1 for prefix items
    int tile, ntile; // first tile and number of tiles of this run
    int pmin, pmax;  // bounds of the rows' positions (padding aside)
    int64_t part;    // first row of its part in the workspace, or -1: the whole item, written out
    KeyTiles keys;
};

// Walks a worker's segments. Used by whole warps; every lane holds the same state.
// Own items in order. Prefix items are all alike and as long as a worker's share, roughly: a worker begins
// with its last item, whose tiles start with the prefix, and goes on with the first, which it takes up where
// the worker before has left it; so all workers are near the same position of the prefix at any time,
// and what one head's row tiles read of it comes from L2.
template <int KT, bool PREFIX>
struct Walker {
    int u, u_end, emitted;
    int worker;
    int i, head, k, tile;  // request, head, row tile, unit within the item
    int head_tiles;        // row tiles of a head
    bool broken;           // some request's offsets are wrong
    ReqRows q;
    KeyTiles shared;       // prefix items: all alike
    int pmin, pmax;
    Shares share = Shares(0, 1);

    __device__ __forceinline__ void start(const AttendParams &P, int w, int lane) {
        worker = w;
        const Totals t = batch_totals<KT>(P, lane);
        broken = t.broken;
        head = k = tile = i = head_tiles = 0;
        q = {0, 0, 0};
        if constexpr (PREFIX) {
            shared = prefix_tiles<KT>(P, t);
            pmin = t.pmin;
            pmax = t.pmax;
            q.n = P.T;
            head_tiles = row_tiles(P.T * P.G, P.prefix_rt_log2);
            share = Shares(P.Hkv * head_tiles * (item_tiles(shared) + P.prefix_extra), P.prefix_workers);
            if (w == 0 && lane == 0) *P.prefix_units = item_tiles(shared);
            u = share.first(w);
            u_end = share.first(w + 1);
            i = 0;  // segments so far
        } else {
            share = Shares(t.units, P.own_workers / P.head_step);
            u = share.first(w / P.head_step);
            u_end = share.first(w / P.head_step + 1);
            if (u < u_end) {
                // the lane whose requests have unit u (the last one with no more before it), then the request
                const int l = __popc(__ballot_sync(0xffffffffu, t.before <= u)) - 1;
                int rem = u - __shfl_sync(0xffffffffu, t.before, l), per_head;
#pragma unroll 1
                for (i = l * t.per;; ++i) {
                    q = held_request(P, i, broken);
                    per_head = own_units<KT>(P, q);
                    if (rem < P.Hkv / P.head_step * per_head || i + 1 >= P.B) break;
                    rem -= P.Hkv / P.head_step * per_head;
                }
                head_tiles = row_tiles(q.n * P.G, P.own_rt_log2);
                head = rem / per_head;
                rem -= head * per_head;
                head = head * P.head_step + w % P.head_step;
#pragma unroll 1
                for (; k + 1 < head_tiles; ++k) {
                    const int len = item_tiles(own_tiles<KT>(P, q, k)) + P.own_extra;
                    if (rem < len) break;
                    rem -= len;
                }
                tile = rem;
            }
        }
        emitted = 0;
        if (!PREFIX && P.shared_len == 0 && lane == 0) P.cut[w].nrows = 0;
        if (!PREFIX && w == 0 && lane == 0) *P.broken = broken;
    }

    // The next segment, or false at the end of the worker's units.
    __device__ __forceinline__ bool next(const AttendParams &P, Segment &s, int lane) {
#pragma unroll 1
        for (;;) {
            s.keys = PREFIX ? shared : own_tiles<KT>(P, q, k);
            const int extra = PREFIX ? P.prefix_extra : P.own_extra, tiles = item_tiles(s.keys), len = tiles + extra;
            int take;
            if constexpr (PREFIX) {
                const int first = u / len, last = (u_end - 1) / len, item = i == 0 ? last : first + i - 1;
                if (u >= u_end || (i > 0 && item >= last)) return false;
                tile = item == first ? u - first * len : 0;
                take = (item == last ? u_end - last * len : len) - tile;
                head = item / head_tiles;
                k = item - head * head_tiles;
                ++i;
            } else {
                if (u >= u_end) return false;
                take = min(len - tile, u_end - u);
            }
            const int rt_log2 = PREFIX ? P.prefix_rt_log2 : P.own_rt_log2;
            // the tiles among these units
            const int a = max(tile - extra, 0), b = max(tile + take - extra, 0), begin = u - tile;
            s.row0 = k << rt_log2;
            s.nrows = min(1 << rt_log2, q.n * P.G - s.row0);
            s.t0 = q.r0;
            s.base = q.kv - q.n;
            s.head = head;
            s.req = PREFIX ? -1 : i;
            s.tile = a;
            s.ntile = s.keys.n > 0 ? b - a : 0;
            s.pmin = PREFIX ? pmin : max(s.base + P.by_group(s.row0), 0);
            s.pmax = PREFIX ? pmax : s.keys.hi - 1;
            const bool whole = a == 0 && b == tiles;
            if (P.shared_len > 0) {
                // along a class's units either the item or the worker grows from one part to the next, so
                // (rows of the items before) + worker * pitch gives every part rows of its own
                const int64_t rows = (static_cast<int64_t>(q.r0) * P.Hkv + static_cast<int64_t>(head) * q.n) * P.G + s.row0;
                s.part = rows + static_cast<int64_t>(worker) * (PREFIX ? P.prefix_pitch : P.own_pitch);
                if (!PREFIX)
                    s.part += static_cast<int64_t>(P.T) * P.Hq + static_cast<int64_t>(P.prefix_workers) * P.prefix_pitch;
            } else {
                // only a worker's first and last segment can be part of an item
                const int slot = emitted > 0 ? 1 : 0;
                s.part = whole ? -1 : static_cast<int64_t>(2 * worker + slot) * P.own_pitch;
                if (!whole && a == 0 && b > 0 && lane == 0)
                    P.cut[worker] = {i, q.r0, s.row0, s.nrows, head, share.owner(begin + len - 1) - worker / P.head_step + 1, slot, 0};
            }
            if constexpr (!PREFIX) {
                u += take;
                tile += take;
                if (tile >= len) {
                    tile = 0;
                    if (++k >= head_tiles) {
                        k = 0;
                        if ((head += P.head_step) >= P.Hkv) {
                            head = worker % P.head_step;
                            if (u < u_end) {
#pragma unroll 1
                                do {
                                    q = held_request(P, ++i, broken);
                                } while (q.n == 0 && i + 1 < P.B);
                                head_tiles = row_tiles(q.n * P.G, P.own_rt_log2);
                            }
                        }
                    }
                }
            }
            if (b > a) {
                ++emitted;
                return true;
            }
        }
    }
};

// ---------------------------------------------------------------- requests' status

// Table entries a lane asks for at a time when a text's pages are checked. One at a time, the warp that checks a
// long text took longer than its CTA's share of the attention (in the round kernel it issues the matrix
// instructions afterwards): 5 rows after a million positions 1390 us, after 65000 86 us; with 16, 701 and 62;
// with 8 the 16 requests of up to 65000 take 320 us instead of 317.
constexpr int kCheckAtOnce = 16;

// Status of request i, by one warp: offsets and length that are right by themselves, and a page for every
// position that a row sees. (Rows that other requests' offsets leave in doubt: the joining kernel.)
__device__ __forceinline__ int attend_status(const AttendParams &P, int i, int lane) {
    const int r0 = P.row_off[i], r1 = P.row_off[i + 1], kv = P.kv_len[i];
    if (!offsets_right(r0, r1, P.T) || kv < 0) return SPEC_REQ_BAD_SHAPE;
    if (r1 == r0 || kv == 0) return SPEC_REQ_OK;
    if (kv > static_cast<int64_t>(P.max_blocks) * P.page_size) return SPEC_REQ_BAD_BLOCKS;
    const int32_t *table = P.block_table + static_cast<int64_t>(i) * P.max_blocks;
    const int win = P.window > 0 ? max(max(kv - (r1 - r0), 0) - P.window + 1, 0) : 0;
    const int sinks = min(min(P.n_sink, win), kv);
    const int L = P.shared_len;
    bool bad = false;
    // the positions seen: window and sinks, of the request's own part and of the shared prefix
#pragma unroll 1
    for (int part = 0; part < (L > 0 ? 4 : 2); ++part) {
        const int a = part == 0 ? max(win, L) : part == 1 ? L : part == 2 ? win : 0;
        const int b = part == 0 ? kv : part == 1 ? sinks : part == 2 ? min(L, kv) : min(sinks, L);
        if (a >= b) continue;
        const int32_t *pages = part < 2 ? table : P.shared_table;
        const int last = P.by_page(b - 1);
        // kCheckAtOnce entries a lane are under way together (page 0 stands for those past the end)
#pragma unroll 1
        for (int x = P.by_page(a) + lane; x <= last; x += kCheckAtOnce * kWarp) {
            int page[kCheckAtOnce];
#pragma unroll
            for (int k = 0; k < kCheckAtOnce; ++k) page[k] = x <= last - k * kWarp ? pages[x + k * kWarp] : 0;
#pragma unroll
            for (int k = 0; k < kCheckAtOnce; ++k) bad |= page[k] < 0 || page[k] >= P.n_pages;
        }
    }
    return __any_sync(0xffffffffu, bad) ? SPEC_REQ_BAD_BLOCKS : SPEC_REQ_OK;
}

// How the kernels of a call overlap. The prefix kernel waits for what came before it in the stream and only
// then lets the next be launched; so the kernel of own items behind it may read the call's inputs at once,
// and works on the SMs that the prefix kernel leaves. It waits for it at its own end, for the joining
// kernel's sake, which waits for this one alone. The joining kernel is not launched early: its blocks,
// waiting beside the workers, kept the next call's workers from filling the SMs (three workers an SM: 408
// instead of 267 us for 256 fp32 requests, call after call).
template <bool PREFIX>
__device__ __forceinline__ void begin_kernel(const AttendParams &P) {
    if (PREFIX || P.shared_len == 0) griddep_wait();
    if (PREFIX) griddep_launch_dependents();
}
template <bool PREFIX>
__device__ __forceinline__ void end_kernel(const AttendParams &P) {
    if (!PREFIX && P.shared_len > 0) griddep_wait();
}

// What a kernel of own items leaves to the joining kernel, by one warp of each CTA: the requests' status,
// and (with a shared prefix, the last CTA) the units before each request.
template <int KT>
__device__ __forceinline__ void keep_books(const AttendParams &P, int lane) {
    if (P.shared_len > 0 && blockIdx.x == gridDim.x - 1) record_units<KT>(P, lane);
#pragma unroll 1
    for (int i = blockIdx.x; i < P.B; i += gridDim.x) {
        const int st = attend_status(P, i, lane);
        if (lane == 0 && SPEC_IN(i, P.B, DBG_ATTEND)) P.status[i] = st;
    }
}

}  // namespace spec
