// Attention of many rows over the cache in 8 bits on the tensor cores (bf16 rows, head sizes that are multiples of
// 16 up to 128): long prompts, and the shared prefix. The work is laid out as in spec_attend_pair.cuh: an item of
// 256 packed rows in two accumulators of 128 that use the same tiles, a row a thread, one warp issuing the
// products of both in turn.
//   S = Q K^T      Q in two parts, K as it lies in the cache (spec_attend8_tiles.cuh)
//   O += P V       P in three parts of 8 bits, over S's columns in tensor memory; V as it lies in the cache
// That is 8 + 12 instructions of 65 cycles a tile and accumulator (128 x 128 x 32; bf16: 8 + 8 of the same time).
//
// A column of S has its position's scales: of the key (a factor of the score) and of the value (which goes into
// the weight as its logarithm, and out of it again in the row's sum, as in spec_attend8_round.cuh). They are the
// same for a box of at least eight columns.
#pragma once

#include "spec_attend8_tiles.cuh"

namespace spec {
namespace pair8 {

using namespace tiles8;

constexpr int kRTLog2 = 8, kRows = 128;  // rows of an item, of an accumulator
constexpr int kHalf = kKT / 2;           // positions whose scores are taken at a time
constexpr int kPart = kHalf / 4;         // columns of tensor memory of a part of a half's weights
constexpr int kThreads = 352;
constexpr float kTop = 11.0f;            // log2 of the largest weight under a new reference, and of what may be
constexpr float kMost = 15.0f;           // reached before the next

struct Shared {
    Pipe<kMaxStages> pipe;
    uint64_t q_full[2], s_full[2], p_full[2][2], o_half[2], o_full[2], agree[2], drain;
    uint32_t bad[2][2][4];  // per warp: its quarter of the values holds one that is not finite
    uint32_t skip[2];       // the warpgroup does this tile's second product itself
    float factor[2][kRows]; // of the rows' scores
    uint32_t tmem;
};

// An accumulator's queries in two parts, and its output on the way out.
constexpr int kQPart = kRows * 128, kQBytes = 2 * kQPart;
__host__ constexpr int stages() {
    constexpr int n = (227 * 1024 - 1024 - static_cast<int>(sizeof(Shared)) - 2 * kQBytes) / kTile;
    return n < kMaxStages ? n : kMaxStages;
}
__host__ constexpr int smem_bytes() {
    return 1024 + 2 * kQBytes + stages() * kTile + static_cast<int>(sizeof(Shared));
}

// ---------------------------------------------------------------- matrix instructions (one warp)

__device__ __forceinline__ void mma_role(const AttendParams &P, Shared &sh, unsigned char *q_mem, unsigned char *ring_mem,
                                         int n_stages) {
    int32_t *ab = &sh.pipe.abort;
    const uint32_t tmem = sh.tmem, pv_shape = mma8_shape(P.D, true, false, false, true);
    const uint64_t q_op = smem_operand(smem_addr(q_mem), 16), ring_op = smem_operand(smem_addr(ring_mem), 16);
    const int steps = (P.D + 31) / 32;
    Ring ring = {0, n_stages, 0}, desc = {0, 2, 0};
    uint32_t q_phases = 0, p_phases = 0;
    // (by the elected lane) S = Q K^T of accumulator w; n positions of the tile are used
    auto score = [&](int w, const Ring &at, int n) {
        const uint64_t k = operand_at(ring_op, at.slot * kTile), q = operand_at(q_op, w * kQBytes);
        const uint32_t shape = mma8_shape(n, false, false, false, false);
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < steps)
                    mma8_ss(tmem + w * 256, operand_at(q, p * kQPart + i * 32), operand_at(k, i * 32), shape, p + i > 0);
        mma_commit(&sh.s_full[w]);
    };
    // (by the elected lane) O += P V of accumulator w and half u; n positions of the half are used
    auto weigh = [&](int w, int u, const Ring &at, int n, bool add) {
        const uint64_t v = operand_at(ring_op, at.slot * kTile + u * (kHalf * 128));
        const uint32_t p = tmem + w * 256 + u * kHalf, o = tmem + w * 256 + 128;
#pragma unroll
        for (int part = 0; part < 3; ++part)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (i * 32 < n) mma8_ts(o, p + part * kPart + 8 * i, operand_at(v, i * 4096), pv_shape, add || part + i > 0);
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
        for (int k = 0; k < n; k += 16) {
            float p[3][4];
            __syncwarp();
#pragma unroll
            for (int part = 0; part < 3; ++part) tmem_ld4(p[part], p_addr + part * kPart + k / 4);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int x = x0 + k + e;
                if (k + e < n && x >= from && x <= lim && (x >= wlo || x < sinks)) {
                    float w = 0.0f;
#pragma unroll
                    for (int part = 0; part < 3; ++part)
                        w += e5m2_to_float(__float_as_uint(p[part][e / 4]) >> (e % 4 * 8) & 0xffu);
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
        float m = -INFINITY, l = 0.0f;  // reference and sum
        bool dead = true;               // no position, or no keys at all
        if (mine > 0 && nt > 0) {
            // the warp's queries into the swizzled tiles, two rows at a time: 16 lanes side by side along a row (a
            // request of one sector per row and lane would take four times the time)
            const int piece = lane % 16;
            const int64_t src = t * P.q_stride + static_cast<int64_t>(h) * P.D;
#pragma unroll 4
            for (int r0 = 0; r0 < kWarp; r0 += 2) {
                const int r = r0 + lane / 16;
                const int64_t row = __shfl_sync(0xffffffffu, src, r);
                const int at = warp * kWarp + r;
                const bool there = at < mine && piece < P.D / 8 && SPEC_IN(row + 8 * piece, P.T * P.q_stride, DBG_ATTEND);
                const uint4 x = there ? reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(P.q) + row)[piece]
                                      : make_uint4(0u, 0u, 0u, 0u);
                uint32_t top = top_bits(0u, x);
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
                const uint32_t bits = max(top & 0xffffu, top >> 16);
                const float qs = query_scale(bits);
                if (at < mine) {
                    uint2 hi, lo;
                    split_query(x, 1.0f / qs, hi, lo);
                    unsigned char *to = q_tile + at * 128 + (((piece >> 1) ^ (at & 7)) << 4) + (piece & 1) * 8;
                    *reinterpret_cast<uint2 *>(to) = hi;
                    *reinterpret_cast<uint2 *>(to + kQPart) = lo;
                    if (piece == 0) sh.factor[w][at] = bits < 0x7f80u ? qs * P.scale_log2 : NAN;
                }
            }
            __syncwarp();
            const float factor = have ? sh.factor[w][tid] : 0.0f;
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
#pragma unroll 1
            for (int i = 0; i < nt; ++i) {
                const int x0 = tile_begin<kKT>(keys, first + i), n = tile_keys(keys, x0);
                const bool edge = x0 > whole || x0 < from || (x0 <= cut && x0 + kKT > P.n_sink);
                const int v_slot = ring.slot + 1 == ring.n ? 0 : ring.slot + 1;
                unsigned char *v_tile = ring_mem + v_slot * kTile;
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
                auto landed = [&]() -> bool {
                    return wait_warp(ab, &sh.pipe.full[v_slot], ring.slot + 1 == ring.n ? ring.phase ^ 1u : ring.phase);
                };
                if (edge) {
                    // A wait by parity tells this use of the slot from the one before only when that one is known to
                    // have arrived: its scores or the next tile's, issued behind its product, have been waited for.
                    // After items without rows for this accumulator, this item's first scores say so.
                    if (behind && !scores()) return;
                    if (!landed()) return;
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
                if (!edge && !landed()) return;  // the scales come with the values
                // (the tile before has been read out of this word: its products were issued before S)
                if (tid == 0) *reinterpret_cast<volatile uint32_t *>(&sh.skip[w]) = skip;
#pragma unroll 1
                for (int u = 0; u * kHalf < n; ++u) {
                    const int xu = x0 + u * kHalf, nu = min(n - u * kHalf, kHalf);
                    const uint32_t s_at = s_addr + u * kHalf;
                    if (warp_has) {
                        float z[64];
                        tmem_ld32(z, s_at);
                        if (nu > 32) tmem_ld32(z + 32, s_at + 32);
                        tmem_wait_ld32(z);
                        tmem_wait_ld32(z + 32);
                        // scores in base 2, and the scales' logarithms with them: eight columns share them
                        float2 by[8];
                        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const int x = xu + 8 * c;
                            float2 sk = make_float2(1.0f, 1.0f);
                            if (!edge || item_sees(P, keys, x, 8)) sk = sh.pipe.scale[v_slot][(u * kHalf + 8 * c) >> P.box_log2];
                            const ValueScale vs = value_scale(sk.y);
                            by[c] = make_float2(vs.log2, vs.inv);
                            const float kf = sk.x * factor;
#pragma unroll
                            for (int e = 8 * c; e < 8 * c + 8; e += 2) {
                                const float2 y = fma2(make_float2(z[e], z[e + 1]), make_float2(kf, kf), make_float2(vs.log2, vs.log2));
                                z[e] = y.x;
                                z[e + 1] = y.y;
                            }
                            if (edge)
#pragma unroll
                                for (int e = 8 * c; e < 8 * c + 8; ++e) {
                                    const int xe = xu + e;
                                    if (!(xe >= from && xe <= lim && (xe >= wlo || xe < P.n_sink))) z[e] = -INFINITY;
                                }
#pragma unroll
                            for (int e = 8 * c; e < 8 * c + 8; e += 2)
                                mx[(e >> 1) & 3] = fmaxf(mx[(e >> 1) & 3], fmaxf(z[e], z[e + 1]));
                        }
                        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                        // a new reference when the old one is too low (or there was none): m is kTop below it
                        const bool grow = top > m && !(top - m <= kMost) && have;
                        if (__any_sync(0xffffffffu, grow)) {
                            if (__any_sync(0xffffffffu, grow && m != -INFINITY)) {
                                // O is at rest: with S came the end of the tiles before, and the first half's
                                // product has a barrier of its own
                                if (u > 0 && !wait_warp(ab, &sh.o_half[w], half_phase)) return;
                                tc_fence_after();
                                const float a = grow && m != -INFINITY ? ex2(m - (top - kTop)) : 1.0f;
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
                            if (grow) m = top - kTop;
                        }
                        const float ref = m == -INFINITY ? 0.0f : -m;
                        const float2 rf = make_float2(ref, ref);
                        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                        uint32_t pw[3][16];
#pragma unroll
                        for (int e = 0; e < 64; e += 4) {
                            float2 a = add2(make_float2(z[e], z[e + 1]), rf), c = add2(make_float2(z[e + 2], z[e + 3]), rf);
                            a.x = ex2(a.x);
                            a.y = ex2(a.y);
                            c.x = ex2(c.x);
                            c.y = ex2(c.y);
                            const float2 inv = make_float2(by[e >> 3].y, by[e >> 3].y);
                            sum[0] = fma2(a, inv, sum[0]);
                            sum[1] = fma2(c, inv, sum[1]);
                            uint32_t parts[3];
                            split_e5m2(a.x, a.y, c.x, c.y, parts);
#pragma unroll
                            for (int part = 0; part < 3; ++part) pw[part][e / 4] = parts[part];
                        }
                        // over columns that have been read
#pragma unroll
                        for (int part = 0; part < 3; ++part) tmem_st16(s_at + part * kPart, pw[part]);
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
                const float ms = m;
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
    spec_attend8_pair_kernel(const __grid_constant__ AttendParams P, const CacheMap M, const __grid_constant__ CUtensorMap kmap,
                            const __grid_constant__ CUtensorMap vmap, const int n_stages) {
    extern __shared__ unsigned char raw[];
    unsigned char *base = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    unsigned char *ring_mem = base + 2 * kQBytes;
    Shared &sh = *reinterpret_cast<Shared *>(ring_mem + n_stages * kTile);
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

}  // namespace pair8
}  // namespace spec
