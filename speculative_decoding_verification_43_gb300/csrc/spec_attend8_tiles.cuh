// What the two tensor-core kernels over the cache in 8 bits share: the ring of key and value tiles with their
// scales, the warp that fills it, the queries in two parts, and the care for values that are no numbers.
//
// A tile holds 128 positions' keys or values of one head as they lie in the cache: 128 rows of 128 bytes in the
// 128-byte swizzle, columns from head_dim on zero. The matrix instructions read e4m3 straight from it; nothing is
// converted. The scales of the tile's boxes of slots come along with the values and are applied to the scores (a
// column of K) and to the weights (a row of V).
#pragma once

#include <cuda.h>

#include "spec_attend_tiles.cuh"
#include "spec_fp8.cuh"

namespace spec {
namespace tiles8 {

using tiles::edge_tile;
using tiles::kHintNs;
using tiles::kKT;
using tiles::kTries;
using tiles::Ring;
using tiles::wait_one;
using tiles::wait_warp;

constexpr int kTile = kKT * 128;  // bytes
constexpr int kBoxes = kKT / 8;   // of a tile, at most

// Where heads and pages lie in the tensor maps (head_dim x heads x slots): slot s of page b, head h is plane
// b * page_rows + h * head_rows + s, row h * head_step.
struct CacheMap {
    int32_t page_rows, head_rows, head_step;
};

// A ring of key tiles and one of value tiles with their scales (of the keys and of the values), and the segments they
// belong to: written by the loading warp. Two rings, because a tile's keys are let go as soon as its scores are
// taken, a tile ahead of the softmax, and its values a tile's time later: in one ring of five slots, in order, three
// tiles were on their way while one was worked on, in rings of two and three four are.
template <int KEYS, int VALUES>
struct Pipe {
    static constexpr int kKeys = KEYS, kValues = VALUES;
    uint64_t k_full[KEYS], k_empty[KEYS], v_full[VALUES], v_empty[VALUES];
    uint64_t desc_full[2], desc_empty[2];
    Segment desc[2];
    float2 scale[VALUES][kBoxes];
    int32_t abort;  // a wait gave up: everyone leaves
};

// Positions of a tile that are used: up to the item's end, in whole groups of 32.
__device__ __forceinline__ int tile_keys(const KeyTiles &k, int x0) { return min(kKT, (k.hi - x0 + 31) & ~31); }

// Waits of a whole warp for several barriers at once: those that have completed cost one round trip together (some 130
// cycles) instead of one each.
__device__ __forceinline__ bool wait_two(int32_t *abort, uint64_t *a, uint32_t a_phase, uint64_t *b, uint32_t b_phase) {
    const bool x = mbar_try_wait(a, a_phase), y = mbar_try_wait(b, b_phase);
    if (__all_sync(0xffffffffu, x && y)) return true;
    return wait_warp(abort, a, a_phase) && wait_warp(abort, b, b_phase);
}

// ---------------------------------------------------------------- loading
// In boxes of the largest power of two of slots that divides the page, a box per lane. Boxes that no row of the
// item sees are not copied (their pages may be gone), and have no scales.

struct TilePlan {
    int row, page;
    bool on;
};

__device__ __forceinline__ TilePlan plan_tile(const AttendParams &P, const CacheMap &M, const Segment &s,
                                              const int32_t *table, int x0, int n, int lane) {
    TilePlan t = {};
    const int x = x0 + (lane << P.box_log2);
    t.on = lane < kKT >> P.box_log2 && x - x0 < n && item_sees(P, s.keys, x, 1 << P.box_log2);
    if (t.on) {
        const int b = P.by_page(x);
        t.page = table[b];
        if (t.page < 0 || t.page >= P.n_pages) t.page = 0;  // (its request is in error: any will do)
        t.row = t.page * M.page_rows + s.head * M.head_rows + (x - b * P.page_size);
        // (the debug build's check) the box's slots are the cache's
        t.on = SPEC_IN(t.row, (P.n_pages - 1) * M.page_rows + (P.Hkv - 1) * M.head_rows + P.page_size - (1 << P.box_log2) + 1,
                       DBG_CACHE);
    }
    return t;
}

// ring_mem: the slots of keys, then those of values.
template <bool PREFIX, int KEYS, int VALUES>
__device__ __forceinline__ void load_role(const AttendParams &P, const CacheMap &M, const CUtensorMap *kmap,
                                          const CUtensorMap *vmap, Pipe<KEYS, VALUES> &pipe, unsigned char *ring_mem, int worker,
                                          int lane) {
    Ring keys = {0, KEYS, 0}, values = {0, VALUES, 0}, desc = {0, 2, 0};
    Walker<kKT, PREFIX> walk;
    walk.start(P, worker, lane);
    Segment s = {};
    bool ok = true;
    int used_keys = 0, used_values = 0;
    auto copy_tile = [&](const CUtensorMap *map, const TilePlan &t, uint64_t *full, unsigned char *dst) {
        const int boxes = __popc(__ballot_sync(0xffffffffu, t.on));
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(full, static_cast<uint32_t>(boxes * (128 << P.box_log2)));
        __syncwarp();
        if (t.on) copy_box3(dst + (lane << (P.box_log2 + 7)), map, 0, s.head * M.head_step, t.row, full);
    };
    while (ok && walk.next(P, s, lane)) {
        ok = wait_warp(&pipe.abort, &pipe.desc_empty[desc.slot], desc.phase ^ 1u);
        if (!ok) break;
        if (lane == 0) {
            pipe.desc[desc.slot] = s;
            mbar_arrive(&pipe.desc_full[desc.slot]);
        }
        __syncwarp();
        desc.step();
        const int32_t *table = PREFIX ? P.shared_table : P.block_table + static_cast<int64_t>(s.req) * P.max_blocks;
        auto plan = [&](int t) {
            const int x0 = tile_begin<kKT>(s.keys, s.tile + t);
            return plan_tile(P, M, s, table, x0, tile_keys(s.keys, x0), lane);
        };
        TilePlan now;
        if (s.ntile > 0) now = plan(0);
#pragma unroll 1
        for (int t = 0; t < s.ntile; ++t) {
            ok = wait_warp(&pipe.abort, &pipe.k_empty[keys.slot], keys.phase ^ 1u);
            if (!ok) break;
            copy_tile(kmap, now, &pipe.k_full[keys.slot], ring_mem + keys.slot * kTile);
            keys.step();
            ++used_keys;
            TilePlan next;
            if (t + 1 < s.ntile) next = plan(t + 1);  // its page ids arrive while this tile's slot is awaited
            ok = wait_warp(&pipe.abort, &pipe.v_empty[values.slot], values.phase ^ 1u);
            if (!ok) break;
            uint64_t *full = &pipe.v_full[values.slot];
            if (now.on) {
                const int64_t at = static_cast<int64_t>(now.page) * P.Hkv + s.head;
                copy_word(&pipe.scale[values.slot][lane].x, P.k_scale + at);
                copy_word(&pipe.scale[values.slot][lane].y, P.v_scale + at);
                copy_words_arrive(full);  // (the phase waits for lane 0's arrival, in copy_tile)
            }
            copy_tile(vmap, now, full, ring_mem + (KEYS + values.slot) * kTile);
            values.step();
            ++used_values;
            now = next;
        }
    }
    // the end of the stream
    if (ok) ok = wait_warp(&pipe.abort, &pipe.desc_empty[desc.slot], desc.phase ^ 1u);
    if (ok && lane == 0) {
        pipe.desc[desc.slot].nrows = 0;
        mbar_arrive(&pipe.desc_full[desc.slot]);
    }
    __syncwarp();
    // every copy has landed and every tile has been let go before the CTA may end
    auto drain = [&](uint64_t *full, uint64_t *empty, int n, int used) {
        Ring back = {0, n, 0};
#pragma unroll 1
        for (int i = 0; i < used; ++i) {
            if (i + n >= used) {
#pragma unroll 1
                for (int t = 0; t < kTries && !mbar_try_wait_sleep(&full[back.slot], back.phase, kHintNs); ++t) {
                }
                if (ok) wait_one(&pipe.abort, &empty[back.slot], back.phase);
            }
            back.step();
        }
    };
    drain(pipe.k_full, pipe.k_empty, KEYS, used_keys);
    drain(pipe.v_full, pipe.v_empty, VALUES, used_values);
    __syncwarp();
}
template <int KEYS, int VALUES>
__device__ __forceinline__ void init_pipe(Pipe<KEYS, VALUES> &pipe, int value_readers, int desc_readers) {
    for (int i = 0; i < KEYS; ++i) {
        mbar_init(&pipe.k_full[i], 1);
        mbar_init(&pipe.k_empty[i], 1);
    }
    for (int i = 0; i < VALUES; ++i) {
        mbar_init(&pipe.v_full[i], 1);
        mbar_init(&pipe.v_empty[i], value_readers);
    }
    for (int i = 0; i < 2; ++i) {
        mbar_init(&pipe.desc_full[i], 1);
        mbar_init(&pipe.desc_empty[i], desc_readers);
    }
    pipe.abort = 0;
}

// ---------------------------------------------------------------- queries
// A row of a head is divided by the power of two s that brings its largest element between 224 and 448, and each
// element becomes hi + lo, hi the nearest e4m3 (four bits) and lo the nearest e5m2 to what that leaves: of a bf16 element of
// eight bits at most 8 of its last places, which three bits hold. So hi + lo is the element exactly while hi has its four
// bits, from 2^-6 on (2^-13 of the largest and more), and off by 2^-14 at most below, where what is left is 2^-10 or less
// (lo as e4m3, whose least is 2^-9, was off by 2^-10 from 2^-2 on). Both products go to the same scores, which are then
// taken times s.

constexpr int kLeastQueryLog2 = -100;

// The greatest magnitude of eight bf16, as bits, in both halves of `top`.
__device__ __forceinline__ uint32_t top_bits(uint32_t top, const uint4 &v) {
    return __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
}
// s for a row whose greatest magnitude has these bits (of fp32); what is not finite gives 1.
__device__ __forceinline__ float query_scale(uint32_t bits) {
    if (bits >= 0x7f800000u) return 1.0f;
    const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float(static_cast<uint32_t>(max(e, kLeastQueryLog2) + 127) << 23);
}
// 1 / s for such an s.
__device__ __forceinline__ float power_inverse(float s) { return __uint_as_float(0x7f000000u - __float_as_uint(s)); }
// Eight bf16 times inv as hi and lo.
__device__ __forceinline__ void split_query(const uint4 &v, float inv, uint2 &hi, uint2 &lo) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = __uint_as_float(w[i] << 16) * inv, b = __uint_as_float(w[i] & 0xffff0000u) * inv;
        const uint16_t p = to_e4m3(a, b);
        const float2 f = e4m3_to_float2(p);
        h[i] = p;
        l[i] = to_e5m2(a - f.x, b - f.y);
    }
    hi = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
    lo = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
}

// Four fp32 times inv in four parts: two as above, and two of what they leave (at most 1/2: a part of four bits is off by
// at most 2^4 of 448, the next by 2^-1) times 2^SHIFT. The first part has four bits, each further one adds five (the
// sign is one): 19 in all, down to 2^-18.
template <int SHIFT>
__device__ __forceinline__ void split_query_wide(const float4 &x, float inv, uint32_t (&parts)[4]) {
    static_assert(SHIFT <= 9, "what is left stays within e4m3");
    float y[4] = {x.x * inv, x.y * inv, x.z * inv, x.w * inv};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t p = to_e4m3(y[0], y[1]) | static_cast<uint32_t>(to_e4m3(y[2], y[3])) << 16;
        const float4 f = e4m3_to_float4(p);
        parts[i] = p;
        const float times = i == 1 ? static_cast<float>(1 << SHIFT) : 1.0f;
        y[0] = (y[0] - f.x) * times;
        y[1] = (y[1] - f.y) * times;
        y[2] = (y[2] - f.z) * times;
        y[3] = (y[3] - f.w) * times;
    }
}

// ---------------------------------------------------------------- values that are no numbers
// As in spec_attend_tiles.cuh: 0 * NaN is NaN.

// By 128 threads: the values of positions that no row sees become 0; true when this thread has found a NaN among
// those that some rows see and others do not.
__device__ __forceinline__ bool clean_values(const AttendParams &P, const Segment &s, unsigned char *v_tile, int x0, int n,
                                             int tid) {
    const KeyTiles &k = s.keys;
    if (tid < n && !item_sees(P, k, x0 + tid)) {
        unsigned char *row = v_tile + tid * 128;
#pragma unroll 1
        for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4 *>(row + c * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    // positions after the first row's, and positions that leave the window between the first row and the last
    const int end = min(x0 + n, k.hi), a0 = max(x0, s.pmin + 1), a = max(min(end, s.pmax + 1) - a0, 0);
    const int b0 = max(x0, s.pmin - P.window + 1), b = P.window > 0 ? max(min(end, s.pmax - P.window + 1) - b0, 0) : 0;
    const int c = tid & 7;
    uint32_t found = 0u;
    if (c < P.D / 16)
#pragma unroll 1
        for (int y = tid >> 3; y < a + b; y += 16) {
            const int x = y < a ? a0 + y : b0 + y - a, r = x - x0;
            if (!item_sees(P, k, x)) continue;
            const uint4 v = *reinterpret_cast<const uint4 *>(v_tile + r * 128 + ((c ^ (r & 7)) << 4));
            found |= __vcmpeq4(v.x & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(v.y & 0x7f7f7f7fu, 0x7f7f7f7fu) |
                     __vcmpeq4(v.z & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(v.w & 0x7f7f7f7fu, 0x7f7f7f7fu);
        }
    return found != 0u;
}

// Column d of position k's values in a tile.
__device__ __forceinline__ float tile_value(const unsigned char *v_tile, int k, int d) {
    return e4m3_to_float2(v_tile[k * 128 + (((d >> 4) ^ (k & 7)) << 4) + (d & 15)]).x;
}

// A position's weight for the output has its value's scale in it, w = 2^(z + log2 v - reference), its part of the row's sum is
// w / v, and 0 where w is, below 2^-126. With scales up to 2^90 apart such a part is less than 2^-43 of its sum: the largest
// weight is 2^7 or more, so z + log2 v lies 133 below that one's, log2 v at most 90. (With weights kept 2^40 larger until
// they are rounded, scales might be 2^120 apart; it cost rounds under a window and fp32 rounds a twentieth.)
// log2 of a scale and the reciprocal that goes with it: a weight times the scale, and back (exact for powers of two).
// The reciprocal is finite whatever the scale is: rows that do not see its position add 0 times it to their sums.
struct ValueScale {
    float log2, inv;
};
__device__ __forceinline__ ValueScale value_scale(float s) {
    const uint32_t bits = __float_as_uint(s);
    if (bits - 0x00800000u >= 0x7f000000u) return {__log2f(s), 1.0f};  // no positive normal number
    const int e = static_cast<int>(bits >> 23) - 127;
    const float part = __log2f(__uint_as_float((bits & 0x7fffffu) | 0x3f800000u));
    return {static_cast<float>(e) + part, ex2(-part) * ex2(static_cast<float>(-e))};
}

}  // namespace tiles8
}  // namespace spec
