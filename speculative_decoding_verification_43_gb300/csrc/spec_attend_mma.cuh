// Attention in bf16 on the tensor cores: head sizes that are multiples of 16 up to 128.
//
// One CTA per SM with two 128-row accumulators. Per tile of 128 keys and accumulator:
//   S = Q K^T      tcgen05.mma, both operands in shared memory, S (fp32) in tensor memory
//   P = 2^(S - m)  a warpgroup, one row per thread; P (bf16) goes back over S's columns
//   O += P V       tcgen05.mma, P read from tensor memory, V from shared memory
// A row's maximum m is a reference, not the running maximum: O and the sum are rescaled only when the
// maximum has grown by more than 2^8 beyond it (P then stays below 2^8, whose bf16 rounding is relative
// all the same), so the output hardly ever leaves tensor memory before the end.
//
// Warps: 0-3 and 4-7 the two warpgroups, 8 and 9 load tiles, 10 and 11 issue matrix instructions (for
// accumulator 0 and 1). They meet at mbarriers: tiles full / empty, S ready, P ready, O ready, queries
// ready, and the descriptors of the segments that the loader hands out.
//
// PAIR: an item is 256 packed rows, both accumulators use the same tiles (long prompts, the shared
// prefix): 64 flops per byte of shared memory read more, and one accumulator's matrix instructions run
// while the other's softmax does. Otherwise each accumulator is a worker of its own with its own items
// and tiles: with the few rows of a verification round the keys' bytes are the bound, and two chains
// keep copies in flight while each waits for its own products.
//
// Keys and values come by gathering tensor copies, four slots of 128 bytes a copy, each lane of the
// loading warp naming four positions: pages of any size end anywhere. Positions that no row of the item
// sees are replaced by one that some row does, so that no foreign value enters (a weight of zero
// times a NaN would be a NaN). The last such case, a value that is not finite at a position some
// rows see and others do not, is looked for in the tiles where rows differ (see mixed_tile).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "spec_attend_plan.cuh"
#include "spec_tcgen05.cuh"

namespace spec {
namespace mma {

constexpr int kKT = 128, kRows = 128;         // keys of a tile, rows of an accumulator
constexpr int kThreads = 384;                 // 8 softmax warps, 2 loading, 2 issuing
constexpr int kBlock = 128 * 128;             // bytes of 128 rows of 64 bf16
constexpr int kMaxStages = 12;
constexpr uint32_t kHintNs = 1000000;         // a wait sleeps up to 1 ms at a time,
constexpr int kTries = 2000;                  // and gives up after 2 s
constexpr float kSlack = 8.0f;                // log2 growth of the maximum that O and l absorb

// Where heads and pages lie in the tensor maps: slot s of page b, head h is row
// b * page_rows + h * head_rows + s, from column h * head_cols on.
struct CacheMap {
    int32_t page_rows, head_rows, head_cols;
};

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t desc_full[2][2], desc_empty[2][2];
    uint64_t q_full[2], s_full[2], p_full[2], o_full[2], v_seen[2], drain[2];
    Segment desc[2][2];
    uint32_t tmem;
    uint32_t bad[2][2][4];  // per warp: its quarter of the values holds one that is not finite
    uint32_t skip[2];       // the warpgroup has done this tile's second product itself
    int32_t abort;
};

__host__ __device__ constexpr int tile_bytes(int D) { return (D > 64 ? 2 : 1) * kBlock; }
__host__ constexpr int stages(int D) {
    const int n = (227 * 1024 - 2048 - static_cast<int>(sizeof(Shared)) - 2 * tile_bytes(D)) / tile_bytes(D);
    return n < kMaxStages ? n : kMaxStages;
}
__host__ constexpr int smem_bytes(int D) {
    return 1024 + 2 * tile_bytes(D) + stages(D) * tile_bytes(D) + static_cast<int>(sizeof(Shared));
}

// A wait by one thread that gives up, and that ends when another thread of the CTA has.
__device__ __forceinline__ bool wait_one(Shared &sh, uint64_t *bar, uint32_t phase) {
    for (int t = 0; t < kTries; ++t) {
        if (mbar_try_wait_sleep(bar, phase, kHintNs)) return true;
        if (*reinterpret_cast<volatile int32_t *>(&sh.abort)) return false;
    }
    *reinterpret_cast<volatile int32_t *>(&sh.abort) = 1;
    return false;
}
// The same by a whole warp, with one answer.
__device__ __forceinline__ bool wait_warp(Shared &sh, uint64_t *bar, uint32_t phase) {
    return __all_sync(0xffffffffu, wait_one(sh, bar, phase));
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

// Keys of tile i of an item that are used: up to the item's end, in whole groups of 16.
__device__ __forceinline__ int tile_keys(const KeyTiles &k, int x0) { return min(kKT, (k.hi - x0 + 15) & ~15); }

// ---------------------------------------------------------------- loading

// Rows of the maps of the four positions from x on.
__device__ __forceinline__ void slot_rows(const AttendParams &P, const CacheMap &M, const KeyTiles &k,
                                          const int32_t *table, int head, int x, int (&row)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int y = item_sees(P, k, x + j) ? x + j : k.pad;
        const int b = P.page_shift >= 0 ? y >> P.page_shift : y / P.page_size;
        int page = table[b];
        // a position without a page puts its request in error: any slot will do
        if (page < 0 || page >= P.n_pages) page = 0;
        row[j] = page * M.page_rows + head * M.head_rows + (y - b * P.page_size);
    }
}

template <bool PREFIX>
__device__ __forceinline__ void load_role(const AttendParams &P, const CacheMap &M, const CUtensorMap *kmap,
                                          const CUtensorMap *vmap, Shared &sh, unsigned char *tiles, int chain, int worker,
                                          int first, int count, int lane) {
    const int tb = tile_bytes(P.D), blocks = tb / kBlock;
    Ring ring = {0, count, 0}, desc = {0, 2, 0};
    Walker<kKT, PREFIX> walk;
    walk.start(P, worker, lane);
    Segment s;
    bool ok = true;
    int used = 0;
    auto copy_tile = [&](const CUtensorMap *map, const int (&row)[4], int n) {
        uint64_t *full = &sh.full[first + ring.slot];
        ok = wait_warp(sh, &sh.empty[first + ring.slot], ring.phase ^ 1u);
        if (!ok) return;
        if (lane == 0) mbar_arrive_expect_tx(full, static_cast<uint32_t>(blocks * n * 128));
        __syncwarp();
        unsigned char *dst = tiles + (first + ring.slot) * tb + lane * 512;
        if (4 * lane < n) {
            const int x = s.head * M.head_cols;
            gather4(dst, map, x, row[0], row[1], row[2], row[3], full);
            if (blocks == 2) gather4(dst + kBlock, map, x + 64, row[0], row[1], row[2], row[3], full);
        }
        ring.step();
        ++used;
    };
    while (ok && walk.next(P, s)) {
        ok = wait_warp(sh, &sh.desc_empty[chain][desc.slot], desc.phase ^ 1u);
        if (!ok) break;
        if (lane == 0) {
            sh.desc[chain][desc.slot] = s;
            mbar_arrive(&sh.desc_full[chain][desc.slot]);
        }
        __syncwarp();
        desc.step();
        const int32_t *table =
            PREFIX ? P.shared_table : P.block_table + static_cast<int64_t>(s.req) * P.max_blocks;
        int row[4];
        for (int t = 0; ok && t < s.ntile; ++t) {
            const int x0 = tile_begin<kKT>(s.keys, s.tile + t), n = tile_keys(s.keys, x0);
            slot_rows(P, M, s.keys, table, s.head, x0 + 4 * lane, row);
            copy_tile(kmap, row, n);
            if (ok) copy_tile(vmap, row, n);
        }
    }
    // the end of the stream: a descriptor without rows
    if (ok) ok = wait_warp(sh, &sh.desc_empty[chain][desc.slot], desc.phase ^ 1u);
    if (ok && lane == 0) {
        sh.desc[chain][desc.slot].nrows = 0;
        mbar_arrive(&sh.desc_full[chain][desc.slot]);
    }
    __syncwarp();
    // every copy has landed and every tile has been let go before the CTA may end
    Ring back = {0, count, 0};
    for (int i = 0; i < used; ++i) {
        if (i + count >= used) {
            for (int t = 0; t < kTries && !mbar_try_wait_sleep(&sh.full[first + back.slot], back.phase, kHintNs); ++t) {
            }
            if (ok) wait_one(sh, &sh.empty[first + back.slot], back.phase);
        }
        back.step();
    }
    __syncwarp();
}

// ---------------------------------------------------------------- matrix instructions (one thread)

__device__ __forceinline__ void mma_role(const AttendParams &P, Shared &sh, unsigned char *q_tile, unsigned char *tiles,
                                         int w, int chain, int first, int count, bool pair) {
    const int tb = tile_bytes(P.D);
    const uint32_t s_col = sh.tmem + w * 256, o_col = s_col + 128, p_col = s_col;
    const uint32_t q_addr = smem_addr(q_tile), t_addr = smem_addr(tiles);
    Ring ring = {0, count, 0}, desc = {0, 2, 0};
    uint32_t q_phase = 0, p_phase = 0;
    auto score = [&](int n) {  // S = Q K^T
        const uint32_t k_addr = t_addr + (first + ring.slot) * tb;
        const uint32_t shape = mma_shape(n, false);
        for (int d = 0; d < P.D; d += 16) {
            const uint32_t at = (d >> 6) * kBlock + (d & 63) * 2;
            mma_ss(s_col, smem_operand(q_addr + at, 16), smem_operand(k_addr + at, 16), shape, d > 0);
        }
        mma_commit(&sh.s_full[w]);
        mma_commit(&sh.empty[first + ring.slot]);
        ring.step();
    };
    for (;;) {
        if (!wait_one(sh, &sh.desc_full[chain][desc.slot], desc.phase)) return;
        const Segment &s = sh.desc[chain][desc.slot];
        if (s.nrows == 0) return;
        const int nt = s.ntile;
        if (nt > 0 && pair && s.nrows <= w * kRows) {
            for (int t = 0; t < 2 * nt; ++t) {  // no rows for this accumulator: let the tiles go by
                if (!wait_one(sh, &sh.full[first + ring.slot], ring.phase)) return;
                mbar_arrive(&sh.empty[first + ring.slot]);
                ring.step();
            }
        } else if (nt > 0) {
            if (!wait_one(sh, &sh.q_full[w], q_phase)) return;
            q_phase ^= 1u;
            if (!wait_one(sh, &sh.full[first + ring.slot], ring.phase)) return;
            tc_fence_after();
            int n = tile_keys(s.keys, tile_begin<kKT>(s.keys, s.tile));
            score(n);
            for (int t = 0; t < nt; ++t) {
                if (!wait_one(sh, &sh.full[first + ring.slot], ring.phase)) return;
                if (!wait_one(sh, &sh.p_full[w], p_phase)) return;
                p_phase ^= 1u;
                tc_fence_after();
                if (!*reinterpret_cast<volatile uint32_t *>(&sh.skip[w])) {  // O += P V
                    const uint32_t v_addr = t_addr + (first + ring.slot) * tb;
                    const uint32_t shape = mma_shape(P.D, true);
                    for (int k = 0; k < n; k += 16)
                        mma_ts(o_col, p_col + k / 2, smem_operand(v_addr + k * 128, kBlock), shape, t > 0 || k > 0);
                }
                mma_commit(&sh.empty[first + ring.slot]);
                ring.step();
                if (t + 1 < nt) {
                    if (!wait_one(sh, &sh.full[first + ring.slot], ring.phase)) return;
                    tc_fence_after();
                    // S and P share columns: matrix instructions of one thread run in the order of
                    // their issue, so this one follows the product that reads P
                    n = tile_keys(s.keys, tile_begin<kKT>(s.keys, s.tile + t + 1));
                    score(n);
                } else {
                    mma_commit(&sh.o_full[w]);
                }
            }
        }
        mbar_arrive(&sh.desc_empty[chain][desc.slot]);
        desc.step();
    }
}

// ---------------------------------------------------------------- softmax (one row per thread)

__device__ __forceinline__ bool not_finite2(uint32_t w) {  // either bf16 of a word
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// The second product of a tile with a value that is not finite at a position that some rows see and
// others do not: on the fp32 units, each row taking the positions it sees. Rows' weights are in tensor
// memory already; O is complete up to the tile before. first: O holds nothing yet.
__device__ __noinline__ void mixed_tile(int D, uint32_t p_addr, uint32_t o_addr, const unsigned char *v_tile, int x0, int n,
                                        int lim, int wlo, int sinks, bool first) {
#pragma unroll 1
    for (int d = 0; d < D; d += 16) {
        float o[16];
        __syncwarp();
        tmem_ld16(o, o_addr + d);
        tmem_wait_ld();
        if (first)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = 0.0f;
#pragma unroll 1
        for (int k = 0; k < n; k += 32) {
            float p[16];
            __syncwarp();
            tmem_ld16(p, p_addr + k / 2);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                const int x = x0 + k + e;
                if (k + e < n && x <= lim && (x >= wlo || x < sinks)) {
                    const uint32_t pw = __float_as_uint(p[e / 2]);
                    const float w = __uint_as_float(e % 2 ? pw & 0xffff0000u : pw << 16);
                    const unsigned char *row = v_tile + (d >> 6) * kBlock + (k + e) * 128;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(row + (((((d & 63) >> 3) + c) ^ ((k + e) & 7)) << 4));
                        const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            o[8 * c + 2 * i] = fmaf(w, __uint_as_float(vw[i] << 16), o[8 * c + 2 * i]);
                            o[8 * c + 2 * i + 1] = fmaf(w, __uint_as_float(vw[i] & 0xffff0000u), o[8 * c + 2 * i + 1]);
                        }
                    }
                }
            }
        }
        uint32_t ow[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) ow[e] = __float_as_uint(o[e]);
        __syncwarp();
        tmem_st16(o_addr + d, ow);
        tmem_wait_st();
    }
}

template <bool PAIR, bool PREFIX>
__device__ __forceinline__ void softmax_role(const AttendParams &P, Shared &sh, unsigned char *q_tile,
                                             unsigned char *tiles, int w, int chain, int first, int count) {
    const int tid = threadIdx.x % 128, warp = tid / kWarp, lane = tid % kWarp;
    const int tb = tile_bytes(P.D);
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t s_addr = sh.tmem + w * 256 + lanes, o_addr = s_addr + 128;
    Ring ring = {0, count, 0}, desc = {0, 2, 0};
    uint32_t s_phase = 0, o_phase = 0, seen_phase = 0;
    for (;;) {
        if (!wait_warp(sh, &sh.desc_full[chain][desc.slot], desc.phase)) return;
        const Segment &s = sh.desc[chain][desc.slot];
        if (s.nrows == 0) return;
        const int off = PAIR ? w * kRows : 0;
        const int mine = min(max(s.nrows - off, 0), kRows);  // rows of this accumulator
        const bool have = tid < mine;
        const bool warp_has = warp * kWarp < mine;
        const int nt = s.ntile, hi = s.keys.hi;
        // this thread's row
        const int pr = s.row0 + off + tid, j = pr / P.G, g = pr - j * P.G;
        const int t = s.t0 + j, h = s.head * P.G + g;
        float m = -INFINITY, l = 0.0f;  // reference (scores, unscaled) and sum
        bool dead = true;               // no position, or no keys at all
        if (mine > 0 && nt > 0) {
            // its query into the swizzled tile
            if (have && SPEC_IN(t, P.T, DBG_ATTEND)) {
                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(P.q) +
                                                                   t * P.q_stride + static_cast<int64_t>(h) * P.D);
                for (int c = 0; c < P.D / 8; ++c)
                    *reinterpret_cast<uint4 *>(q_tile + (c >> 3) * kBlock + tid * 128 + (((c & 7) ^ (tid & 7)) << 4)) =
                        src[c];
            }
            fence_proxy_async_smem();
            mbar_arrive(&sh.q_full[w]);
            int p = -1;
            if (have) {
                if constexpr (PREFIX) {
                    int lo = 0, n = P.B;  // the row's request
                    while (n > 1) {
                        const int half = n / 2;
                        if (P.row_off[lo + half] <= t) {
                            lo += half;
                            n -= half;
                        } else {
                            n = half;
                        }
                    }
                    const ReqRows q = load_request(P, lo);
                    if (t >= q.r0 && t < q.r0 + q.n) p = q.kv - q.n + (t - q.r0);
                } else {
                    p = s.base + j;
                }
            }
            dead = p < 0;
            const int lim = min(p, hi - 1), wlo = P.window > 0 ? p - P.window + 1 : 0;
            for (int i = 0; i < nt; ++i) {
                const int x0 = tile_begin<kKT>(s.keys, s.tile + i), n = tile_keys(s.keys, x0);
                // rows differ in what they see of this tile (or it has fewer keys)
                const bool edge = x0 + kKT - 1 > min(s.pmin, hi - 1) ||
                                  (P.window > 0 && x0 <= s.pmax - P.window && x0 + kKT > P.n_sink);
                const int v_stage = ring.slot + 1 == ring.n ? 0 : ring.slot + 1;
                const uint32_t v_phase = ring.slot + 1 == ring.n ? ring.phase ^ 1u : ring.phase;
                bool skip = false;
                if (edge) {
                    if (!wait_warp(sh, &sh.full[first + v_stage], v_phase)) return;
                    bool bad = false;
                    if (tid < n) {
                        const unsigned char *row = tiles + (first + v_stage) * tb + tid * 128;
                        for (int c = 0; c < P.D / 8; ++c) {
                            const uint4 v =
                                *reinterpret_cast<const uint4 *>(row + (c >> 3) * kBlock + (((c & 7) ^ (tid & 7)) << 4));
                            bad |= not_finite2(v.x) | not_finite2(v.y) | not_finite2(v.z) | not_finite2(v.w);
                        }
                    }
                    // the four warps' findings (two sets, used in turn)
                    bad = __any_sync(0xffffffffu, bad);
                    volatile uint32_t *found = sh.bad[w][seen_phase];
                    if (lane == 0) {
                        found[warp] = bad;
                        mbar_arrive(&sh.v_seen[w]);
                    }
                    __syncwarp();
                    if (!wait_warp(sh, &sh.v_seen[w], seen_phase)) return;
                    seen_phase ^= 1u;
                    skip = (found[0] | found[1] | found[2] | found[3]) != 0;
                }
                if (!wait_warp(sh, &sh.s_full[w], s_phase)) return;
                s_phase ^= 1u;
                tc_fence_after();
                if (warp_has) {
                    float z[kKT];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (c * 32 < n) tmem_ld32(z + 32 * c, s_addr + 32 * c);
                    tmem_wait_ld();
                    if (edge) {
#pragma unroll
                        for (int e = 0; e < kKT; ++e) {
                            const int x = x0 + e;
                            if (!(x <= lim && (x >= wlo || x < P.n_sink))) z[e] = -INFINITY;
                        }
                    }
                    float mx[4] = {z[0], z[1], z[2], z[3]};
#pragma unroll
                    for (int e = 4; e < kKT; e += 8)
#pragma unroll
                        for (int a = 0; a < 4; ++a)
                            mx[a] = e + 4 + a < kKT ? fmaxf(mx[a], fmaxf(z[e + a], z[e + 4 + a])) : fmaxf(mx[a], z[e + a]);
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    // a new reference when the old one is too low (or there was none)
                    const bool grow = top > m && !((top - m) * P.scale_log2 <= kSlack);
                    if (__any_sync(0xffffffffu, grow && m != -INFINITY)) {
                        const float a = grow && m != -INFINITY ? ex2((m - top) * P.scale_log2) : 1.0f;
                        l *= a;
                        // S is complete, and with it the product of the tile before: O is at rest
                        for (int d = 0; d < P.D; d += 16) {
                            float o[16];
                            uint32_t ow[16];
                            tmem_ld16(o, o_addr + d);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) ow[e] = __float_as_uint(o[e] * a);
                            tmem_st16(o_addr + d, ow);
                        }
                        tmem_wait_st();
                    }
                    if (grow) m = top;
                    const float ref = m == -INFINITY ? 0.0f : m;
                    const float2 sc = make_float2(P.scale_log2, P.scale_log2);
                    const float2 rf = make_float2(-ref * P.scale_log2, -ref * P.scale_log2);
                    float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (c * 32 < n) {
                            uint32_t pw[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float2 y = fma2(make_float2(z[32 * c + 2 * e], z[32 * c + 2 * e + 1]), sc, rf);
                                y.x = ex2(y.x);
                                y.y = ex2(y.y);
                                sum[e & 1] = add2(sum[e & 1], y);
                                pw[e] = pack_bf16(y.x, y.y);
                            }
                            tmem_st16(s_addr + 16 * c, pw);
                        }
                    }
                    sum[0] = add2(sum[0], sum[1]);
                    l += sum[0].x + sum[0].y;
                    tmem_wait_st();
                    if (skip)
                        mixed_tile(P.D, s_addr, o_addr, tiles + (first + v_stage) * tb, x0, n, lim, wlo, P.n_sink, i == 0);
                }
                if (tid == 0) *reinterpret_cast<volatile uint32_t *>(&sh.skip[w]) = skip;
                tc_fence_before();
                mbar_arrive(&sh.p_full[w]);
                ring.step();
                ring.step();
            }
            if (!wait_warp(sh, &sh.o_full[w], o_phase)) return;
            o_phase ^= 1u;
            tc_fence_after();
        } else {
            for (int i = 0; i < 2 * nt; ++i) ring.step();
        }
        if (dead) {
            m = -INFINITY;
            l = 0.0f;
        }
        const bool none = l == 0.0f;
        const float inv = s.part >= 0 ? 1.0f : 1.0f / l;
        if (warp_has) {
            for (int d = 0; d < P.D; d += 16) {
                float o[16];
                __syncwarp();
                if (nt > 0) {
                    tmem_ld16(o, o_addr + d);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = none ? 0.0f : o[e] * inv;
                if (!have) continue;
                if (s.part >= 0) {
                    if (SPEC_IN(s.part + off + tid, P.part_rows, DBG_ATTEND)) {
                        float4 *dst = reinterpret_cast<float4 *>(P.part_o + (s.part + off + tid) * P.D + d);
#pragma unroll
                        for (int e = 0; e < 4; ++e) dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    }
                } else if (SPEC_IN(t, P.T, DBG_ATTEND)) {
                    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(P.out) + t * P.out_stride +
                                                           static_cast<int64_t>(h) * P.D + d);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        dst[e] = make_uint4(pack_bf16(o[8 * e], o[8 * e + 1]), pack_bf16(o[8 * e + 2], o[8 * e + 3]),
                                            pack_bf16(o[8 * e + 4], o[8 * e + 5]), pack_bf16(o[8 * e + 6], o[8 * e + 7]));
                }
            }
            if (have) {
                const float ms = m * P.scale_log2;
                if (s.part >= 0) {
                    // a sum that is not a number must reach the joined row, whatever the other parts' maxima
                    if (SPEC_IN(s.part + off + tid, P.part_rows, DBG_ATTEND))
                        P.part_ml[s.part + off + tid] = make_float2(isnan(l) ? INFINITY : ms, l);
                } else if (P.lse && SPEC_IN(t, P.T, DBG_ATTEND)) {
                    P.lse[static_cast<int64_t>(t) * P.Hq + h] =
                        none ? -INFINITY : (ms + log2f(l)) * 0.6931471805599453f;
                }
            }
        }
        tc_fence_before();  // O may be written again once the next segment's P is ready
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.desc_empty[chain][desc.slot]);
        desc.step();
    }
}

// ---------------------------------------------------------------- the kernel

template <bool PAIR, bool PREFIX>
__global__ void __launch_bounds__(kThreads, 1)
    spec_attend_mma_kernel(const __grid_constant__ AttendParams P, const CacheMap M, const __grid_constant__ CUtensorMap kmap,
                           const __grid_constant__ CUtensorMap vmap, const int n_stages) {
    extern __shared__ unsigned char raw[];
    unsigned char *base = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    const int tb = tile_bytes(P.D);
    unsigned char *tiles = base + 2 * tb;
    Shared &sh = *reinterpret_cast<Shared *>(tiles + n_stages * tb);
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
    // chains of tiles: one for both accumulators, or one each
    const int count = PAIR ? n_stages : n_stages / 2;

    griddep_launch_dependents();
    if (warp == 10) tmem_alloc(&sh.tmem, 512);
    if (threadIdx.x == 0) {
        for (int i = 0; i < n_stages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], PAIR ? 2 : 1);
        }
        for (int c = 0; c < 2; ++c) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(&sh.desc_full[c][i], 1);
                mbar_init(&sh.desc_empty[c][i], PAIR ? 10 : 5);  // four warps and the issuing thread, of each reader
            }
            mbar_init(&sh.q_full[c], 128);
            mbar_init(&sh.s_full[c], 1);
            mbar_init(&sh.p_full[c], 128);
            mbar_init(&sh.o_full[c], 1);
            mbar_init(&sh.v_seen[c], 4);
            mbar_init(&sh.drain[c], 1);
            sh.skip[c] = 0;
        }
        sh.abort = 0;
        fence_mbar_init();
        prefetch_map(&kmap);
        prefetch_map(&vmap);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();

    if (warp < 8) {
        const int w = warp / 4, chain = PAIR ? 0 : w;
        if constexpr (!PREFIX)
            for (int i = blockIdx.x * 8 + warp; i < P.B; i += gridDim.x * 8) {
                const int st = attend_status(P, i, lane);
                if (lane == 0 && SPEC_IN(i, P.B, DBG_ATTEND)) P.status[i] = st;
            }
        softmax_role<PAIR, PREFIX>(P, sh, base + w * tb, tiles, w, chain, chain * count, count);
    } else if (warp < 10) {
        const int c = warp - 8;
        if (!PAIR || c == 0)
            load_role<PREFIX>(P, M, &kmap, &vmap, sh, tiles, c, PAIR ? blockIdx.x : 2 * blockIdx.x + c, c * count, count,
                              lane);
    } else if (lane == 0) {
        const int w = warp - 10, chain = PAIR ? 0 : w;
        mma_role(P, sh, base + w * tb, tiles, w, chain, chain * count, count, PAIR);
        // nothing this thread issued is in flight when the CTA ends
        mma_commit(&sh.drain[w]);
        for (int t = 0; t < kTries && !mbar_try_wait_sleep(&sh.drain[w], 0, kHintNs); ++t) {
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 10) tmem_free(sh.tmem, 512);
    // a worker's word: PAIR one per CTA, else both accumulators' alike
    if (threadIdx.x == 0) {
        int32_t *err = P.err + (PREFIX ? P.own_workers : 0);
        if (PAIR) {
            err[blockIdx.x] = sh.abort;
        } else {
            err[2 * blockIdx.x] = err[2 * blockIdx.x + 1] = sh.abort;
        }
    }
}

}  // namespace mma
}  // namespace spec
