// Attention of many rows on the tensor cores (bf16, head sizes that are multiples of 16 up to 128): long
// prompts, and the shared prefix, whose rows are those of the whole batch.
//
// One CTA per SM, an item of 256 packed rows in two accumulators of 128 that use the same tiles. Per
// tile of 128 keys and accumulator:
//   S = Q K^T      tcgen05.mma, both operands in shared memory, S (fp32) in tensor memory
//   P = 2^(S - m)  a warpgroup, one row per thread; P (bf16) goes back over S's columns, in two halves
//   O += P V       tcgen05.mma, P read from tensor memory, V from shared memory
// One warp issues the products of both accumulators in turn, so that one's run while the other's softmax
// does: a product of 128 x 128 x 128 takes 512 cycles of the tensor cores, four of them a tile. Issued
// by a warp each, both would wait for the tensor cores at the same time and then for the softmax.
// (S of half tiles in two buffers hides the products' latency altogether, but 64 columns of keys take
// as long as 128: the queries' 128 rows are read again. It took 4000 cycles a tile.)
// A row's m is a reference, not the running maximum: O and the sum are rescaled only when the maximum
// has grown by more than 2^8 beyond it (P then stays below 2^8, whose bf16 rounding is relative all the
// same), so the output hardly ever leaves tensor memory before the end.
//
// Measured: 372 GFLOP of prompts (4 requests, 32 query and 8 key heads of 128) 371 us, 0.51 of the measured
// bf16 rate; 550 GFLOP of a 32768-position prefix under 1031 rows 447 us, 0.63. A pair of tiles takes some
// 3500 cycles by its time, 2048 of them products; on 2000 rows after 6000 positions the counters have the tensor
// pipe active in 48 % of the cycles, instructions issued in 36 % and DRAM in 3 %, and warps waiting on loads and
// barriers most of the rest. What is left is taken to be the chain from a warpgroup's weights over the
// issuing warp's waits to the next scores, and an item's queries and way out (six tiles' time).
//
// Warps: 0-3 and 4-7 the two warpgroups, 8 loads tiles, 9 keeps the books (the requests' status), 10
// issues matrix instructions.
#pragma once

#include "spec_attend_tiles.cuh"

namespace spec {
namespace pair {

using namespace tiles;

constexpr int kRTLog2 = 8, kRows = 128;  // rows of an item, of an accumulator
constexpr int kHalf = kKT / 2;           // positions whose scores are taken at a time
constexpr int kThreads = 352;
constexpr float kSlack = 8.0f;           // log2 growth of the maximum that O and the sum absorb

struct Shared {
    Pipe<kMaxStages> pipe;
    uint64_t q_full[2], s_full[2], p_full[2][2], o_half[2], o_full[2], agree[2], drain;
    uint32_t bad[2][2][4];  // per warp: its quarter of the values holds one that is not finite
    uint32_t skip[2];       // the warpgroup does this tile's second product itself
    uint32_t tmem;
};

// An accumulator's queries, and its output on the way out: two blocks.
constexpr int kQBytes = 2 * kBlock;
__host__ constexpr int stages(int D) {
    const int n = (227 * 1024 - 1024 - static_cast<int>(sizeof(Shared)) - 2 * kQBytes) / tile_bytes(D);
    return n < kMaxStages ? n : kMaxStages;
}
__host__ constexpr int smem_bytes(int D) {
    return 1024 + 2 * kQBytes + stages(D) * tile_bytes(D) + static_cast<int>(sizeof(Shared));
}

// ---------------------------------------------------------------- matrix instructions (one warp)

__device__ __forceinline__ void mma_role(const AttendParams &P, Shared &sh, unsigned char *q_mem, unsigned char *ring_mem,
                                         int n_stages) {
    const int tb = tile_bytes(P.D);
    int32_t *ab = &sh.pipe.abort;
    const uint32_t tmem = sh.tmem, pv_shape = mma_shape(P.D, false, true);
    const uint64_t q_op = smem_operand(smem_addr(q_mem), 16), k_op = smem_operand(smem_addr(ring_mem), 16),
                   v_op = smem_operand(smem_addr(ring_mem), kBlock);
    const int steps = P.D / 16;
    Ring ring = {0, n_stages, 0}, desc = {0, 2, 0};
    uint32_t q_phases = 0, p_phases = 0;
    // (by the elected lane) S = Q K^T of accumulator w; n positions of the tile are used
    auto score = [&](int w, const Ring &at, int n) {
        const uint64_t k = operand_at(k_op, at.slot * tb), q = operand_at(q_op, w * kQBytes);
        const uint32_t shape = mma_shape(n, false, false);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t in = (i >> 2) * kBlock + (i & 3) * 32;
            if (i < steps) mma_ss(tmem + w * 256, operand_at(q, in), operand_at(k, in), shape, i > 0);
        }
        mma_commit(&sh.s_full[w]);
    };
    // (by the elected lane) O += P V of accumulator w and half u; n positions of the half are used
    auto weigh = [&](int w, int u, const Ring &at, int n, bool add) {
        const uint64_t v = operand_at(v_op, at.slot * tb + u * (kHalf * 128));
        const uint32_t p = tmem + w * 256 + u * kHalf, o = tmem + w * 256 + 128;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i * 16 < n) mma_ts(o, p + 8 * i, operand_at(v, i * 2048), pv_shape, add || i > 0);
    };
    for (;;) {
        if (!wait_warp(ab, &sh.pipe.desc_full[desc.slot], desc.phase)) return;
        const Segment &s = sh.pipe.desc[desc.slot];
        if (s.nrows == 0) return;
        const int nt = s.ntile, first = s.tile, accs = s.nrows > kRows ? 2 : 1;
        const KeyTiles keys = s.keys;
        if (nt > 0) {
            int n = tile_keys(keys, tile_begin<kKT>(keys, first));
            if (!wait_warp(ab, &sh.pipe.full[ring.slot], ring.phase)) return;
            for (int w = 0; w < accs; ++w) {
                if (!wait_warp(ab, &sh.q_full[w], q_phases >> w & 1u)) return;
                q_phases ^= 1u << w;
                tc_fence_after();
                if (elect_lane()) {
                    score(w, ring, n);
                    if (w == accs - 1) mma_commit(&sh.pipe.empty[ring.slot]);
                }
                __syncwarp();
            }
            ring.step();
            // Between the waits only one stretch of instructions by the elected lane: what this warp does
            // beside issuing, the tensor cores wait for.
#pragma unroll 1
            for (int t = 0; t < nt; ++t) {
                const Ring v = ring;  // this tile's values; the next tile's keys follow them
                ring.step();
                const bool more = t + 1 < nt;
                const int next = more ? tile_keys(keys, tile_begin<kKT>(keys, first + t + 1)) : 0;
                if (!wait_warp(ab, &sh.pipe.full[v.slot], v.phase)) return;
                if (more && !wait_warp(ab, &sh.pipe.full[ring.slot], ring.phase)) return;
#pragma unroll 1
                for (int w = 0; w < accs; ++w) {
                    if (!wait_warp(ab, &sh.p_full[w][0], p_phases >> w & 1u)) return;
                    p_phases ^= 1u << w;
                    tc_fence_after();
                    const bool take = !*reinterpret_cast<volatile uint32_t *>(&sh.skip[w]);
                    if (n > kHalf) {
                        if (elect_lane()) {
                            if (take) weigh(w, 0, v, kHalf, t > 0);
                            mma_commit(&sh.o_half[w]);
                        }
                        __syncwarp();
                        if (!wait_warp(ab, &sh.p_full[w][1], p_phases >> (2 + w) & 1u)) return;
                        p_phases ^= 4u << w;
                        tc_fence_after();
                    }
                    if (elect_lane()) {
                        if (take) weigh(w, n > kHalf ? 1 : 0, v, n > kHalf ? n - kHalf : n, t > 0 || n > kHalf);
                        // S and P share columns: matrix instructions of one thread run in the order of
                        // their issue, so the next scores follow the product that reads P
                        if (more)
                            score(w, ring, next);
                        else
                            mma_commit(&sh.o_full[w]);
                        if (w == accs - 1) {
                            mma_commit(&sh.pipe.empty[v.slot]);
                            if (more) mma_commit(&sh.pipe.empty[ring.slot]);
                        }
                    }
                    __syncwarp();
                }
                if (more) ring.step();
                n = next;
            }
        }
        if (elect_lane()) mbar_arrive(&sh.pipe.desc_empty[desc.slot]);
        __syncwarp();
        desc.step();
    }
}

// ---------------------------------------------------------------- softmax (one row per thread)

// The second product of a tile with values that are not finite, on the fp32 units: the row's weights
// are in tensor memory already, O is complete up to the tile before. first: O holds nothing yet.
__device__ __noinline__ void mixed_tile(int D, uint32_t p_addr, uint32_t o_addr, const unsigned char *v_tile, int k0, int x0, int n,
                                        int from, int lim, int wlo, int sinks, bool first) {
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
                if (k + e < n && x >= from && x <= lim && (x >= wlo || x < sinks)) {
                    const uint32_t pw = __float_as_uint(p[e / 2]);
                    const float w = __uint_as_float(e % 2 ? pw & 0xffff0000u : pw << 16);
#pragma unroll 4
                    for (int i = 0; i < 16; ++i) o[i] = fmaf(w, tile_value(v_tile, k0 + k + e, d + i), o[i]);
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

template <bool PREFIX>
__device__ __forceinline__ void softmax_role(const AttendParams &P, Shared &sh, unsigned char *q_tile,
                                             unsigned char *ring_mem, int w, int n_stages) {
    const int tid = threadIdx.x % 128, warp = tid / kWarp, lane = tid % kWarp;
    const int tb = tile_bytes(P.D);
    int32_t *ab = &sh.pipe.abort;
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t s_addr = sh.tmem + w * 256 + lanes, o_addr = s_addr + 128;
    Ring ring = {0, n_stages, 0}, desc = {0, 2, 0};
    uint32_t s_phase = 0, o_phase = 0, half_phase = 0, agree_phase = 0;
    bool behind = false;  // tiles have gone by that this warpgroup has not waited for
    for (;;) {
        if (!wait_warp(ab, &sh.pipe.desc_full[desc.slot], desc.phase)) return;
        const Segment &s = sh.pipe.desc[desc.slot];
        if (s.nrows == 0) return;
        const int off = w * kRows;
        const int mine = min(max(s.nrows - off, 0), kRows);  // rows of this accumulator
        const bool have = tid < mine;
        const bool warp_has = warp * kWarp < mine;
        const int nt = s.ntile;
        // this thread's row
        const int pr = s.row0 + off + tid, j = P.by_group(pr), g = pr - j * P.G;
        const int t = s.t0 + j, h = s.head * P.G + g;
        float m = -INFINITY, l = 0.0f;  // reference (scores, unscaled) and sum
        bool dead = true;               // no position, or no keys at all
        if (mine > 0 && nt > 0) {
            // the warp's queries into the swizzled tile, some rows at a time: lanes side by side along a row
            // (a request of one sector per row and lane would take four times the time)
            const int per = P.D / 8, at_once = kWarp / per, piece = lane % per;
            const int64_t src = t * P.q_stride + static_cast<int64_t>(h) * P.D;
#pragma unroll 4
            for (int r0 = 0; r0 < kWarp; r0 += at_once) {
                const int r = r0 + lane / per;
                const int64_t row = __shfl_sync(0xffffffffu, src, r & 31);
                const int at = warp * kWarp + r;
                if (lane < at_once * per && r < kWarp && at < mine && SPEC_IN(row + 8 * piece, P.T * P.q_stride, DBG_ATTEND))
                    *reinterpret_cast<uint4 *>(q_tile + (piece >> 3) * kBlock + at * 128 + (((piece & 7) ^ (at & 7)) << 4)) =
                        reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(P.q) + row)[piece];
            }
            fence_proxy_async_smem();
            mbar_arrive(&sh.q_full[w]);
            int p = -1;
            if (have) {
                if constexpr (PREFIX) {
                    const ReqRows q = load_request(P, find_request(P.row_off, P.B, P.T, t));
                    if (t >= q.r0 && t < q.r0 + q.n) p = q.kv - q.n + (t - q.r0);
                } else {
                    p = s.base + j;
                }
            }
            dead = p < 0;
            const int lim = min(p, s.keys.hi - 1), wlo = P.window > 0 ? p - P.window + 1 : 0, from = s.keys.from;
            if (!have) m = 0.0f;  // lanes without a row never ask for another reference
            const KeyTiles keys = s.keys;
            const int first = s.tile;
            // a tile is seen whole by all rows from x0 = from on to here, when no window cuts it off
            const int whole = min(s.pmin, keys.hi - 1) - (kKT - 1), cut = P.window > 0 ? s.pmax - P.window : -1;
            const float2 sc = make_float2(P.scale_log2, P.scale_log2);
#pragma unroll 1
            for (int i = 0; i < nt; ++i) {
                const int x0 = tile_begin<kKT>(keys, first + i), n = tile_keys(keys, x0);
                const bool edge = x0 > whole || x0 < from || (x0 <= cut && x0 + kKT > P.n_sink);
                unsigned char *v_tile = ring_mem + (ring.slot + 1 == ring.n ? 0 : ring.slot + 1) * tb;
                bool skip = false, scored = false;
                auto scores = [&]() -> bool {
                    if (scored) return true;
                    scored = true;
                    if (!wait_warp(ab, &sh.s_full[w], s_phase)) return false;
                    s_phase ^= 1u;
                    tc_fence_after();
                    behind = false;
                    return true;
                };
                if (edge) {
                    // A wait by parity tells this use of the slot from the one before only when that one is known to
                    // have arrived: its scores or the next tile's, issued behind its product, have been waited for.
                    // After items without rows for this accumulator, this item's first scores say so.
                    if (behind && !scores()) return;
                    const int v_slot = ring.slot + 1 == ring.n ? 0 : ring.slot + 1;
                    if (!wait_warp(ab, &sh.pipe.full[v_slot], ring.slot + 1 == ring.n ? ring.phase ^ 1u : ring.phase)) return;
                    const bool bad = __any_sync(0xffffffffu, clean_values(P, s, v_tile, x0, n, tid));
                    fence_proxy_async_smem();
                    // the four warps' findings (two sets, used in turn)
                    volatile uint32_t *found = sh.bad[w][agree_phase];
                    __syncwarp();
                    if (lane == 0) {
                        found[warp] = bad;
                        mbar_arrive(&sh.agree[w]);
                    }
                    if (!wait_warp(ab, &sh.agree[w], agree_phase)) return;
                    agree_phase ^= 1u;
                    skip = (found[0] | found[1] | found[2] | found[3]) != 0;
                }
                if (!scores()) return;
                // (the tile before has been read out of this word: its products were issued before S)
                if (tid == 0) *reinterpret_cast<volatile uint32_t *>(&sh.skip[w]) = skip;
#pragma unroll 1
                for (int u = 0; u * kHalf < n; ++u) {
                    const int xu = x0 + u * kHalf, nu = min(n - u * kHalf, kHalf);
                    const uint32_t s_at = s_addr + u * kHalf;
                    if (warp_has) {
                        float za[32], zb[32];
                        uint32_t pw[32];
                        tmem_ld32(za, s_at);
                        if (nu > 32) tmem_ld32(zb, s_at + 32);
                        tmem_wait_ld32(za);
                        tmem_wait_ld32(zb);
                        if (edge) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const int xa = xu + e, xb = xu + 32 + e;
                                if (!(xa >= from && xa <= lim && (xa >= wlo || xa < P.n_sink))) za[e] = -INFINITY;
                                if (!(xb >= from && xb <= lim && (xb >= wlo || xb < P.n_sink))) zb[e] = -INFINITY;
                            }
                        }
                        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            mx[0] = fmaxf(mx[0], fmaxf(za[e], za[e + 1]));
                            mx[1] = fmaxf(mx[1], fmaxf(za[e + 2], za[e + 3]));
                            mx[2] = fmaxf(mx[2], fmaxf(zb[e], zb[e + 1]));
                            mx[3] = fmaxf(mx[3], fmaxf(zb[e + 2], zb[e + 3]));
                        }
                        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                        // a new reference when the old one is too low (or there was none)
                        const bool grow = top > m && !((top - m) * P.scale_log2 <= kSlack) && have;
                        if (__any_sync(0xffffffffu, grow)) {
                            if (__any_sync(0xffffffffu, grow && m != -INFINITY)) {
                                // O is at rest: with S came the end of the tiles before, and the first half's
                                // product has a barrier of its own
                                if (u > 0 && !wait_warp(ab, &sh.o_half[w], half_phase)) return;
                                tc_fence_after();
                                const float a = grow && m != -INFINITY ? ex2((m - top) * P.scale_log2) : 1.0f;
                                l *= a;
#pragma unroll 1
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
                        }
                        const float ref = m == -INFINITY ? 0.0f : -m * P.scale_log2;
                        const float2 rf = make_float2(ref, ref);
                        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float2 y = fma2(make_float2(za[2 * e], za[2 * e + 1]), sc, rf);
                            y.x = ex2(y.x);
                            y.y = ex2(y.y);
                            sum[e & 1] = add2(sum[e & 1], y);
                            pw[e] = pack_bf16(y.x, y.y);
                        }
                        tmem_st16(s_at, pw);  // over columns that have been read
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float2 y = fma2(make_float2(zb[2 * e], zb[2 * e + 1]), sc, rf);
                            y.x = ex2(y.x);
                            y.y = ex2(y.y);
                            sum[e & 1] = add2(sum[e & 1], y);
                            pw[16 + e] = pack_bf16(y.x, y.y);
                        }
                        tmem_st16(s_at + 16, pw + 16);
                        sum[0] = add2(sum[0], sum[1]);
                        l += sum[0].x + sum[0].y;
                        tmem_wait_st();
                        if (skip) {
                            if (u > 0 && !wait_warp(ab, &sh.o_half[w], half_phase)) return;
                            tc_fence_after();
                            mixed_tile(P.D, s_at, o_addr, v_tile, u * kHalf, xu, nu, from, lim, wlo, P.n_sink, i + u == 0);
                        }
                    }
                    tc_fence_before();
                    mbar_arrive(&sh.p_full[w][u]);
                }
                if (n > kHalf) half_phase ^= 1u;
                ring.step();
                ring.step();
            }
            if (!wait_warp(ab, &sh.o_full[w], o_phase)) return;
            o_phase ^= 1u;
            tc_fence_after();
        } else {
            for (int i = 0; i < 2 * nt; ++i) ring.step();
            behind = behind || nt > 0;
        }
        if (dead) {
            m = -INFINITY;
            l = 0.0f;
        }
        const bool none = l == 0.0f;
        const float inv = s.part >= 0 ? 1.0f : 1.0f / l;
        if (warp_has) {
            // O leaves through a quarter of the query memory (every product with it is done), 8 KB: rows of
            // 256 bytes, the 16-byte pieces of row r at (piece ^ (r % 8)); out of it the lanes go side by side
            // along the rows (see the queries)
            unsigned char *mem = q_tile + warp * (kQBytes / 4);
            const bool part = s.part >= 0;
            const int span = part ? 64 : 128;  // columns at a time
            const int64_t row_out = part ? (s.part + off + tid) * static_cast<int64_t>(P.D)
                                         : t * P.out_stride + static_cast<int64_t>(h) * P.D;
#pragma unroll 1
            for (int d0 = 0; d0 < P.D; d0 += span) {
                const int width = min(span, P.D - d0);
                __syncwarp();
#pragma unroll 1
                for (int d = 0; d < width; d += 16) {
                    float o[16];
                    if (nt > 0) {
                        tmem_ld16(o, o_addr + d0 + d);
                        tmem_wait_ld();
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = none ? 0.0f : o[e] * inv;
                    unsigned char *row = mem + lane * 256;
                    const int p0 = part ? d >> 2 : d >> 3;
                    if (part) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *reinterpret_cast<float4 *>(row + (((p0 + e) ^ (lane & 7)) << 4)) =
                                make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            *reinterpret_cast<uint4 *>(row + (((p0 + e) ^ (lane & 7)) << 4)) =
                                make_uint4(pack_bf16(o[8 * e], o[8 * e + 1]), pack_bf16(o[8 * e + 2], o[8 * e + 3]),
                                           pack_bf16(o[8 * e + 4], o[8 * e + 5]), pack_bf16(o[8 * e + 6], o[8 * e + 7]));
                    }
                }
                __syncwarp();
                const int per = part ? width / 4 : width / 8, at_once = kWarp / per, piece = lane % per;
#pragma unroll 4
                for (int r0 = 0; r0 < kWarp; r0 += at_once) {
                    const int r = r0 + lane / per;
                    const int64_t dst = __shfl_sync(0xffffffffu, row_out, r & 31);
                    if (lane < at_once * per && r < kWarp && warp * kWarp + r < mine) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(mem + r * 256 + ((piece ^ (r & 7)) << 4));
                        if (part) {
                            if (SPEC_IN(dst + d0 + 4 * piece, P.part_rows * P.D, DBG_ATTEND))
                                *reinterpret_cast<uint4 *>(P.part_o + dst + d0 + 4 * piece) = v;
                        } else if (SPEC_IN(dst + d0 + 8 * piece, P.T * P.out_stride, DBG_ATTEND)) {
                            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(P.out) + dst + d0 + 8 * piece) = v;
                        }
                    }
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
        // the query memory may be written again once all four warps are through
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.agree[w]);
        if (!wait_warp(ab, &sh.agree[w], agree_phase)) return;
        agree_phase ^= 1u;
        if (lane == 0) mbar_arrive(&sh.pipe.desc_empty[desc.slot]);
        desc.step();
    }
}

// ---------------------------------------------------------------- the kernel

template <bool PREFIX>
__global__ void __launch_bounds__(kThreads, 1)
    spec_attend_pair_kernel(const __grid_constant__ AttendParams P, const CacheMap M, const __grid_constant__ CUtensorMap kmap,
                            const __grid_constant__ CUtensorMap vmap, const int n_stages) {
    extern __shared__ unsigned char raw[];
    unsigned char *base = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    const int tb = tile_bytes(P.D);
    unsigned char *ring_mem = base + 2 * kQBytes;
    Shared &sh = *reinterpret_cast<Shared *>(ring_mem + n_stages * tb);
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;

    if (warp == 10) tmem_alloc(&sh.tmem, 512);
    if (threadIdx.x == 0) {
        for (int i = 0; i < n_stages; ++i) {
            mbar_init(&sh.pipe.full[i], 1);
            mbar_init(&sh.pipe.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.pipe.desc_full[i], 1);
            mbar_init(&sh.pipe.desc_empty[i], 9);  // eight softmax warps and the issuing one
            mbar_init(&sh.q_full[i], 128);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i][0], 128);
            mbar_init(&sh.p_full[i][1], 128);
            mbar_init(&sh.o_half[i], 1);
            mbar_init(&sh.o_full[i], 1);
            mbar_init(&sh.agree[i], 4);
            sh.skip[i] = 0;
        }
        mbar_init(&sh.drain, 1);
        sh.pipe.abort = 0;
        fence_mbar_init();
        prefetch_map(&kmap);
        prefetch_map(&vmap);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    begin_kernel<PREFIX>(P);

    if (warp < 8) {
        softmax_role<PREFIX>(P, sh, base + (warp / 4) * kQBytes, ring_mem, warp / 4, n_stages);
    } else {
        if (warp == 8) {
            load_role<PREFIX>(P, M, &kmap, &vmap, sh.pipe, ring_mem, n_stages, blockIdx.x, lane);
        } else if (warp == 9) {
            if constexpr (!PREFIX) keep_books<kKT>(P, lane);
        } else {
            mma_role(P, sh, base, ring_mem, n_stages);
            // nothing this warp issued is in flight when the CTA ends
            if (elect_lane()) mma_commit(&sh.drain);
            __syncwarp();
#pragma unroll 1
            for (int t = 0; t < kTries && !mbar_try_wait_sleep(&sh.drain, 0, kHintNs); ++t) {
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 10) tmem_free(sh.tmem, 512);
    end_kernel<PREFIX>(P);
    if (threadIdx.x == 0) P.err[(PREFIX ? P.own_workers : 0) + blockIdx.x] = sh.pipe.abort;
}

}  // namespace pair
}  // namespace spec
