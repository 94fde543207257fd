// What the two tensor-core attention kernels share: bounded waits, the ring of key and value tiles, the
// warp that fills it, and the care for values that are not finite.
//
// A tile holds 128 positions' keys or values of one head: blocks of 64 columns, each 128 rows of 128
// bytes in the 128-byte swizzle, as the matrix instructions read them.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "spec_attend_plan.cuh"
#include "spec_tcgen05.cuh"

namespace spec {
namespace tiles {

constexpr int kKT = 128;                // positions of a tile
constexpr int kBlock = kKT * 128;       // bytes of a block of 64 columns
constexpr int kMaxStages = 12;
constexpr uint32_t kHintNs = 1000000;   // a wait sleeps up to 1 ms at a time,
constexpr int kTries = 2000;            // and gives up after 2 s

__host__ __device__ constexpr int blocks(int D) { return D > 64 ? 2 : 1; }
__host__ __device__ constexpr int tile_bytes(int D) { return blocks(D) * kBlock; }

// Where heads and pages lie in the tensor maps: slot s of page b, head h is row
// b * page_rows + h * head_rows + s, from column h * head_cols on.
struct CacheMap {
    int32_t page_rows, head_rows, head_cols;
};

// A ring of tiles, and the segments they belong to: written by the loading warp.
template <int STAGES>
struct Pipe {
    uint64_t full[STAGES], empty[STAGES];
    uint64_t desc_full[2], desc_empty[2];
    Segment desc[2];
    int32_t abort;  // a wait gave up: everyone leaves
};

// A wait by one thread that gives up, and that ends when another thread of the CTA has.
__device__ __forceinline__ bool wait_one(int32_t *abort, uint64_t *bar, uint32_t phase) {
    if (mbar_try_wait_sleep(bar, phase, kHintNs)) return true;
#pragma unroll 1
    for (int t = 0; t < kTries; ++t) {
        if (mbar_try_wait_sleep(bar, phase, kHintNs)) return true;
        if (*reinterpret_cast<volatile int32_t *>(abort)) return false;
    }
    *reinterpret_cast<volatile int32_t *>(abort) = 1;
    return false;
}
// The same by a whole warp, with one answer.
__device__ __forceinline__ bool wait_warp(int32_t *abort, uint64_t *bar, uint32_t phase) {
    return __all_sync(0xffffffffu, wait_one(abort, bar, phase));
}

// A position in a ring of n slots.
struct Ring {
    int slot, n;
    uint32_t phase;
    __device__ __forceinline__ void step() {
        if (++slot == n) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

// Positions of a tile that are used: up to the item's end, in whole groups of 16.
__device__ __forceinline__ int tile_keys(const KeyTiles &k, int x0) { return min(kKT, (k.hi - x0 + 15) & ~15); }

// True when rows of the item differ in what they see of the tile at x0, or it holds positions none sees.
__device__ __forceinline__ bool edge_tile(const AttendParams &P, const Segment &s, int x0) {
    return x0 + kKT - 1 > min(s.pmin, s.keys.hi - 1) || x0 < s.keys.from ||
           (P.window > 0 && x0 <= s.pmax - P.window && x0 + kKT > P.n_sink);
}

// ---------------------------------------------------------------- loading
//
// Pages of a multiple of eight slots are copied in boxes of the largest power of two that divides the
// page (8 to 128 slots: 1 to 16 KB a copy), a box per lane; other pages by gathering copies of four
// slots. A gathering copy of 512 bytes takes the copy engine some 40 cycles, so that it alone would hold
// a stream of tiles to half the memory's rate; boxes of 16 slots do not.
// Boxes that no row of the item sees are not copied (their pages may be gone).

struct TilePlan {
    int row[4];  // box: its first row; gathering: four rows
    bool on;
};

__device__ __forceinline__ TilePlan plan_tile(const AttendParams &P, const CacheMap &M, const Segment &s,
                                              const int32_t *table, int x0, int n, int lane) {
    TilePlan t = {};
    // the map's row of position x; where it has no page (its request is in error) any will do
    auto row_of = [&](int x) {
        const int b = P.by_page(x);
        int page = table[b];
        if (page < 0 || page >= P.n_pages) page = 0;
        return page * M.page_rows + s.head * M.head_rows + (x - b * P.page_size);
    };
    // (the debug build's check) slots row .. row + n - 1 of the map are the cache's
    auto inside = [&](int row, int n) -> bool {
        return SPEC_IN(row, (P.n_pages - 1) * M.page_rows + (P.Hkv - 1) * M.head_rows + P.page_size - n + 1, DBG_CACHE);
    };
    if (P.box_log2 > 0) {
        const int box = lane & ((kKT >> P.box_log2) - 1), half = lane >> (7 - P.box_log2);
        const int x = x0 + (box << P.box_log2);
        t.on = half < blocks(P.D) && x - x0 < n && item_sees(P, s.keys, x, 1 << P.box_log2);
        if (t.on) t.row[0] = row_of(x);
        t.on = t.on && inside(t.row[0], 1 << P.box_log2);
    } else {
        t.on = 4 * lane < n;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (t.on && item_sees(P, s.keys, x0 + 4 * lane + j)) {
                const int row = row_of(x0 + 4 * lane + j);
                if (inside(row, 1)) t.row[j] = row;
            }
    }
    return t;
}

template <bool PREFIX, int STAGES>
__device__ __forceinline__ void load_role(const AttendParams &P, const CacheMap &M, const CUtensorMap *kmap,
                                          const CUtensorMap *vmap, Pipe<STAGES> &pipe, unsigned char *ring_mem, int stages,
                                          int worker, int lane) {
    Ring ring = {0, stages, 0}, desc = {0, 2, 0};
    Walker<kKT, PREFIX> walk;
    walk.start(P, worker, lane);
    Segment s = {};
    bool ok = true;
    int used = 0;
    auto copy_tile = [&](const CUtensorMap *map, const TilePlan &t) {
        uint64_t *full = &pipe.full[ring.slot];
        ok = wait_warp(&pipe.abort, &pipe.empty[ring.slot], ring.phase ^ 1u);
        if (!ok) return;
        const int lanes = __popc(__ballot_sync(0xffffffffu, t.on));
        if (lane == 0)
            mbar_arrive_expect_tx(full, static_cast<uint32_t>(P.box_log2 > 0 ? lanes * (128 << P.box_log2)
                                                                             : lanes * 512 * blocks(P.D)));
        __syncwarp();
        unsigned char *dst = ring_mem + ring.slot * tile_bytes(P.D);
        if (t.on) {
            const int x = s.head * M.head_cols;
            if (P.box_log2 > 0) {
                const int box = lane & ((kKT >> P.box_log2) - 1), half = lane >> (7 - P.box_log2);
                copy_box(dst + half * kBlock + (box << (P.box_log2 + 7)), map, x + 64 * half, t.row[0], full);
            } else {
                gather4(dst + lane * 512, map, x, t.row[0], t.row[1], t.row[2], t.row[3], full);
                if (blocks(P.D) == 2)
                    gather4(dst + lane * 512 + kBlock, map, x + 64, t.row[0], t.row[1], t.row[2], t.row[3], full);
            }
        }
        ring.step();
        ++used;
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
        for (int t = 0; ok && t < s.ntile; ++t) {
            copy_tile(kmap, now);
            if (!ok) break;
            TilePlan next;
            if (t + 1 < s.ntile) next = plan(t + 1);  // its page ids arrive while this tile's slot is awaited
            copy_tile(vmap, now);
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
    Ring back = {0, stages, 0};
#pragma unroll 1
    for (int i = 0; i < used; ++i) {
        if (i + stages >= used) {
#pragma unroll 1
            for (int t = 0; t < kTries && !mbar_try_wait_sleep(&pipe.full[back.slot], back.phase, kHintNs); ++t) {
            }
            if (ok) wait_one(&pipe.abort, &pipe.empty[back.slot], back.phase);
        }
        back.step();
    }
    __syncwarp();
}

// ---------------------------------------------------------------- values that are not finite
//
// A position that a row does not see has weight 0 for it, but 0 * inf is not 0. In an edge tile the
// values of positions that no row of the item sees (behind the window, past the end, not copied) are
// therefore set to 0, and those that some rows see and others do not (the rows' own positions, the
// window's edge) are searched for one that is not finite. If there is one, the tile's second product is
// taken on the fp32 units, each row with the positions it sees.

// By 128 threads: the first part a thread a position, the second 16 threads a position. True when this
// thread has found a value that is not finite.
__device__ __forceinline__ bool clean_values(const AttendParams &P, const Segment &s, unsigned char *v_tile, int x0, int n,
                                             int tid) {
    const KeyTiles &k = s.keys;
    if (tid < n && !item_sees(P, k, x0 + tid)) {
        unsigned char *row = v_tile + tid * 128;
#pragma unroll 1
        for (int c = 0; c < 8 * blocks(P.D); ++c)
            *reinterpret_cast<uint4 *>(row + (c >> 3) * kBlock + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    // positions after the first row's, and positions that leave the window between the first row and the last
    const int end = min(x0 + n, k.hi), a0 = max(x0, s.pmin + 1), a = max(min(end, s.pmax + 1) - a0, 0);
    const int b0 = max(x0, s.pmin - P.window + 1), b = P.window > 0 ? max(min(end, s.pmax - P.window + 1) - b0, 0) : 0;
    const int c = tid & 15;
    uint32_t top = 0u;  // the greatest magnitude as bit patterns, by halves
    if (c < P.D / 8)
#pragma unroll 1
        for (int y = tid >> 4; y < a + b; y += 8) {
            const int x = y < a ? a0 + y : b0 + y - a, r = x - x0;
            if (!item_sees(P, k, x)) continue;
            const uint4 v = *reinterpret_cast<const uint4 *>(v_tile + (c >> 3) * kBlock + r * 128 + (((c & 7) ^ (r & 7)) << 4));
            top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                         __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
        }
    return (top & 0xffffu) >= 0x7f80u || (top >> 16) >= 0x7f80u;
}

// Column d of position k's values in a tile.
__device__ __forceinline__ float tile_value(const unsigned char *v_tile, int k, int d) {
    const unsigned char *at = v_tile + (d >> 6) * kBlock + k * 128 + ((((d & 63) >> 3) ^ (k & 7)) << 4) + (d & 7) * 2;
    return __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(at));
}

}  // namespace tiles
}  // namespace spec
