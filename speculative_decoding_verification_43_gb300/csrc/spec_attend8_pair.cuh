// Attention of many rows over the cache in 8 bits on the tensor cores (bf16 rows, head sizes that are multiples of
// 16 up to 128): long prompts, and the shared prefix. The work is laid out as in spec_attend_pair.cuh: an item of
// 256 packed rows in two accumulators of 128 that use the same tiles, a row a thread, one warp issuing the
// products of both in turn. Per tile of 128 keys and accumulator:
//   S = Q K^T      Q in two parts, e4m3 and e5m2 (spec_attend8_tiles.cuh), K as it lies in the cache, in two halves of
//                  64 keys
//   P = 2^(S - m)  a warpgroup, one row per thread; P (16-bit floats) goes back over S's columns, a half at a time
//   O += P V       V as 16-bit floats, to which two warps bring each tile once for all 256 rows
// Taking V as it is would need P in three parts of 8 bits: 12 instructions instead of 8, and five operations a weight
// on top of four (prompts 870 us that way, 621 this way when it came, with tiles fetched without the next head's bytes);
// converting V is one operation for two values, and exact. 16-bit floats hold weights from 2^15 down to 2^-14 to 11
// bits, below to 2^-25, so a row's reference m may stay 2^8 behind its maximum.
//
// Measured (us a call): 4 prompts of 1000-2500 rows on up to 6000 positions, 32 / 8 heads of 128 (372 GFLOP) 420-450, 0.45 of
// the measured rate; 64 requests behind 8192 shared positions 106, of which the shared ones some 50. Two tiles (both
// accumulators) take some 4200 cycles, 2600 of them products (QK by halves: 8 of 49 cycles where whole tiles take 65 for twice
// the columns, a price for scores that are there before they are needed: 574 us -> 545). The rest is the issuing warp's
// hand-overs, which find the weights ready but cost it 250 cycles and more each; a softmax thread works 2600. An item's queries and
// outputs take 9400 + 7900 cycles (once 21000 + 8500: prompts 545 us). Tried: a second issuing warp, with registers moved
// between warpgroups for it (470 -> 500), a look at the next weights between product and scores (545 -> 557),
// conversions without bank conflicts (no difference). Left out one at a time, the exponentials, three quarters of PV,
// the queries' lower parts or the conversions change the time by 0 to 4 %: no unit is the limit, their chain is.
//
// Scales: a column of S has its key's scale as a factor, the same for a box of at least eight columns. Its value's scale v
// goes into the weight, 2^(S + log2 v - m), so that what counts is what a position contributes, and its part of the row's
// sum is the weight / v. So values are e4m3 as 16-bit floats, exactly, and a row's reference comes from positions
// that it sees alone. (Scales applied to the values, as fractions of the tile's largest, rounded away a quiet page's values
// beside a loud page, for rows that did not see that one, too.) The converting warps also set the values of positions that
// no row sees to 0.
//
// Warps: 0-3 and 4-7 the two warpgroups, 8 loads tiles, 9 issues matrix instructions, 10 and 11 convert values
// (11 keeps the books first: the requests' status).
#pragma once

#include "spec_attend8_tiles.cuh"

namespace spec {
namespace pair8 {

using namespace tiles8;

constexpr int kRTLog2 = 8, kRows = 128;  // rows of an item, of an accumulator
constexpr int kHalf = kKT / 2;           // positions whose scores are taken at a time
constexpr int kThreads = 384;
constexpr int kStages = 4;               // tiles of keys and of values, two each
constexpr int kBlock = kKT * 128, kValues = 2 * kBlock;  // values as 16-bit floats: two blocks of 64 columns
constexpr float kTop = 7.0f;             // log2 of the largest weight under a new reference, and of what may be
constexpr float kMost = 15.0f;           // reached before the next

struct Shared {
    Pipe<kStages / 2, kStages / 2> pipe;
    uint64_t q_full[2], s_full[2][2], p_full[2][2], o_done[2][2], agree[2], drain;  // [accumulator][half of a tile]
    uint64_t v_full[2], v_empty[2];     // converted values
    uint32_t skip[2][2];                // the warpgroup does this half's second product itself
    uint32_t no_number[2][2];           // per slot of values and converting warp: it has found a NaN
    uint32_t tmem;
    // per slot of values and eight columns: scale of the keys, log2 of the values' scale, and its reciprocal
    alignas(16) float key_scale[2][kBoxes], value_log2[2][kBoxes], value_inv[2][kBoxes];
    float factor[2][kRows];             // of the rows' scores
};

// An accumulator's queries in two parts, and its output on the way out.
constexpr int kQPart = kRows * 128, kQBytes = 2 * kQPart;
constexpr int kSmem = 1024 + 2 * kQBytes + 2 * kValues + kStages * kTile + static_cast<int>(sizeof(Shared));
static_assert(kSmem <= 227 * 1024, "fits");

// ---------------------------------------------------------------- matrix instructions (one warp)

__device__ __forceinline__ void mma_role(const AttendParams &P, Shared &sh, unsigned char *q_mem, unsigned char *v_mem,
                                         unsigned char *ring_mem) {
    int32_t *ab = &sh.pipe.abort;
    const uint32_t tmem = sh.tmem, pv_shape = mma_shape_f16(P.D, false, true);
    const uint64_t q_op = smem_operand(smem_addr(q_mem), 16), k_op = smem_operand(smem_addr(ring_mem), 16),
                   v_op = smem_operand(smem_addr(v_mem), kBlock);
    const int steps = (P.D + 31) / 32;
    Ring ring = {0, kStages / 2, 0}, values = {0, 2, 0}, desc = {0, 2, 0};
    uint32_t q_phases = 0, p_phases = 0;
    // (by the elected lane) S = Q K^T of accumulator w and half u; n positions of the tile are used
    auto score = [&](int w, int u, const Ring &at, int n) {
        const uint64_t k = operand_at(k_op, at.slot * kTile + u * (kHalf * 128)), q = operand_at(q_op, w * kQBytes);
        const uint32_t shapes[2] = {mma8_shape(min(n - u * kHalf, kHalf), false, false, false, false),
                                    mma8_shape(min(n - u * kHalf, kHalf), true, false, false, false)};
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < steps)
                    mma8_ss(tmem + w * 256 + u * kHalf, operand_at(q, p * kQPart + i * 32), operand_at(k, i * 32),
                            shapes[p], p + i > 0);
        mma_commit(&sh.s_full[w][u]);
    };
    // (by the elected lane) O += P V of accumulator w and half u; n positions of the half are used
    auto weigh = [&](int w, int u, const Ring &at, int n, bool add) {
        const uint64_t v = operand_at(v_op, at.slot * kValues + u * (kHalf * 128));
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
            if (!wait_warp(ab, &sh.pipe.k_full[ring.slot], ring.phase)) return;
            for (int w = 0; w < accs; ++w) {
                if (!wait_warp(ab, &sh.q_full[w], q_phases >> w & 1u)) return;
                q_phases ^= 1u << w;
                tc_fence_after();
                if (elect_lane()) {
                    score(w, 0, ring, n);
                    if (n > kHalf) score(w, 1, ring, n);
                    if (w == accs - 1) mma_commit(&sh.pipe.k_empty[ring.slot]);
                }
                __syncwarp();
            }
            ring.step();
            // Between the waits only one stretch of instructions by the elected lane: what this warp does beside issuing, the
            // tensor cores wait for. So the four stretches of a tile are written out: their operands and barriers are
            // constants (prompts 452 us -> 430).
#pragma unroll 1
            for (int t = 0; t < nt; ++t) {
                const bool more = t + 1 < nt;  // (only a segment's last tile may be short)
                const int next = more ? tile_keys(keys, tile_begin<kKT>(keys, first + t + 1)) : 0;
                // (this warp has waited for every use of these slots before)
                if (!(more ? wait_two(ab, &sh.v_full[values.slot], values.phase, &sh.pipe.k_full[ring.slot], ring.phase)
                           : wait_warp(ab, &sh.v_full[values.slot], values.phase)))
                    return;
                const int halves = n > kHalf ? 2 : 1;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (u >= halves) break;
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        if (w >= accs) break;
                        if (!wait_warp(ab, &sh.p_full[w][u], p_phases >> (2 * u + w) & 1u)) return;
                        p_phases ^= 1u << (2 * u + w);
                        tc_fence_after();
                        const bool take = !*reinterpret_cast<volatile uint32_t *>(&sh.skip[w][u]);
                        if (elect_lane()) {
                            if (take) weigh(w, u, values, min(n - u * kHalf, kHalf), t + u > 0);
                            mma_commit(&sh.o_done[w][u]);
                            // S and P share columns: matrix instructions of one thread run in the order of
                            // their issue, so the next scores follow the product that reads P
                            if (next > u * kHalf) score(w, u, ring, next);
                            if (u == halves - 1 && w == accs - 1) {
                                mma_commit(&sh.v_empty[values.slot]);
                                if (more) mma_commit(&sh.pipe.k_empty[ring.slot]);
                            }
                        }
                        __syncwarp();
                    }
                }
                if (more) ring.step();
                values.step();
                n = next;
            }
        }
        if (elect_lane()) mbar_arrive(&sh.pipe.desc_empty[desc.slot]);
        __syncwarp();
        desc.step();
    }
}

// ---------------------------------------------------------------- values (two warps)

__device__ __forceinline__ void convert_role(const AttendParams &P, Shared &sh, unsigned char *v_mem,
                                             const unsigned char *ring_mem, int which, int lane) {
    int32_t *ab = &sh.pipe.abort;
    Ring ring = {0, kStages / 2, 0}, values = {0, 2, 0}, desc = {0, 2, 0};
    const int c = lane & 7;
    for (;;) {
        if (!wait_warp(ab, &sh.pipe.desc_full[desc.slot], desc.phase)) return;
        const Segment &s = sh.pipe.desc[desc.slot];
        if (s.nrows == 0) return;
        const int nt = s.ntile;
#pragma unroll 1
        for (int t = 0; t < nt; ++t) {
            const int x0 = tile_begin<kKT>(s.keys, s.tile + t), n = tile_keys(s.keys, x0);
            const bool edge = edge_tile(P, s, x0);
            if (!wait_warp(ab, &sh.v_empty[values.slot], values.phase ^ 1u)) return;
            if (!wait_warp(ab, &sh.pipe.v_full[ring.slot], ring.phase)) return;
            // lane x < 16: eight positions (no scales were copied for boxes that no row sees)
            const float2 *scales = sh.pipe.scale[ring.slot];
            const int group = lane & (kBoxes - 1);
            const bool used = !edge || item_sees(P, s.keys, x0 + 8 * group >> P.box_log2 << P.box_log2, 1 << P.box_log2);
            const float2 by = used ? scales[8 * group >> P.box_log2] : make_float2(1.0f, 1.0f);
            if (which == 0 && lane < kBoxes) {
                const ValueScale vs = value_scale(by.y);
                sh.key_scale[values.slot][lane] = by.x;
                sh.value_log2[values.slot][lane] = vs.log2;
                sh.value_inv[values.slot][lane] = vs.inv;
            }
            // 16 values a lane, eight lanes a row: two pieces of eight 16-bit floats in the row's block of columns
            const unsigned char *from = ring_mem + (kStages / 2 + ring.slot) * kTile;
            unsigned char *to = v_mem + values.slot * kValues + (c >> 2) * kBlock;
            const int piece = (c & 3) * 2, first = which * 4 + (lane >> 3);
            uint32_t found = 0u;
            auto fetch = [&](int r) { return *reinterpret_cast<const uint4 *>(from + r * 128 + ((c ^ (r & 7)) << 4)); };
            auto put = [&](int r, const uint4 &v) {
                unsigned char *row = to + r * 128;
                *reinterpret_cast<uint4 *>(row + ((piece ^ (r & 7)) << 4)) =
                    make_uint4(e4m3_to_half2(v.x), e4m3_to_half2(v.x >> 16), e4m3_to_half2(v.y), e4m3_to_half2(v.y >> 16));
                *reinterpret_cast<uint4 *>(row + (((piece + 1) ^ (r & 7)) << 4)) =
                    make_uint4(e4m3_to_half2(v.z), e4m3_to_half2(v.z >> 16), e4m3_to_half2(v.w), e4m3_to_half2(v.w >> 16));
            };
            if (c < P.D / 16) {
                if (!edge) {
                    // (half of a warp's rows at a time: their loads are under way together)
#pragma unroll 1
                    for (int r = first; r < kKT; r += 64) {
                        uint4 v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] = fetch(r + 8 * i);
#pragma unroll
                        for (int i = 0; i < 8; ++i) put(r + 8 * i, v[i]);
                    }
                } else {
#pragma unroll 1
                    for (int r = first; r < n; r += 32) {
                        uint4 v[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[i] = item_sees(P, s.keys, x0 + r + 8 * i) ? fetch(r + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            found |= __vcmpeq4(v[i].x & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(v[i].y & 0x7f7f7f7fu, 0x7f7f7f7fu) |
                                     __vcmpeq4(v[i].z & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(v[i].w & 0x7f7f7f7fu, 0x7f7f7f7fu);
                            put(r + 8 * i, v[i]);
                        }
                    }
                }
            }
            found = __any_sync(0xffffffffu, found != 0u);
            if (lane == 0) sh.no_number[values.slot][which] = found;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh.v_full[values.slot]);
                mbar_arrive(&sh.pipe.v_empty[ring.slot]);
            }
            ring.step();
            values.step();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.pipe.desc_empty[desc.slot]);
        desc.step();
    }
}

// ---------------------------------------------------------------- softmax (one row per thread)

// The lowest n of 64 bits.
__device__ __forceinline__ uint64_t below(int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; }

// The second product of a tile with values that are no numbers, on the fp32 units: the row's weights are in tensor
// memory already, O is complete up to the tile before. first: O holds nothing yet.
__device__ __noinline__ void mixed_tile(int D, uint32_t p_addr, uint32_t o_addr, const unsigned char *values, int k0, int x0, int n,
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
                    const float w = __half2float(__ushort_as_half(static_cast<unsigned short>(e % 2 ? pw >> 16 : pw)));
                    const int row = k0 + k + e;
#pragma unroll 4
                    for (int i = 0; i < 16; ++i) {
                        const unsigned char *at = values + ((d + i) >> 6) * kBlock + row * 128 +
                                                  (((((d + i) & 63) >> 3) ^ (row & 7)) << 4) + ((d + i) & 7) * 2;
                        o[i] = fmaf(w, __half2float(*reinterpret_cast<const __half *>(at)), o[i]);
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

template <bool PREFIX>
__device__ __forceinline__ void softmax_role(const AttendParams &P, Shared &sh, unsigned char *q_tile,
                                             const unsigned char *v_mem, int w) {
    const int tid = threadIdx.x % 128, warp = tid / kWarp, lane = tid % kWarp;
    int32_t *ab = &sh.pipe.abort;
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t s_addr = sh.tmem + w * 256 + lanes, o_addr = s_addr + 128;
    Ring values = {0, 2, 0}, desc = {0, 2, 0};
    uint32_t s_phases = 0, o_phases = 0, agree_phase = 0;  // (a bit per half; o_phases: of the product to come)
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
            // request of one sector per row and lane would take four times the time). Sixteen rows' loads are under way
            // together: one after the other, with the shuffles between them, they took 21000 cycles of an item.
            constexpr int kAtOnce = 8;
            const int piece = lane % 16;
            const int64_t src = t * P.q_stride + static_cast<int64_t>(h) * P.D;
#pragma unroll 1
            for (int r0 = lane / 16; r0 < kWarp; r0 += 2 * kAtOnce) {
                uint4 x[kAtOnce];
#pragma unroll
                for (int y = 0; y < kAtOnce; ++y) {
                    const int r = r0 + 2 * y;
                    const int64_t row = __shfl_sync(0xffffffffu, src, r);
                    const bool there =
                        warp * kWarp + r < mine && piece < P.D / 8 && SPEC_IN(row + 8 * piece, P.T * P.q_stride, DBG_ATTEND);
                    x[y] = there ? reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(P.q) + row)[piece]
                                 : make_uint4(0u, 0u, 0u, 0u);
                }
                uint32_t bits[kAtOnce];
#pragma unroll
                for (int y = 0; y < kAtOnce; ++y) bits[y] = top_bits(0u, x[y]);
#pragma unroll
                for (int o = 8; o > 0; o >>= 1)
#pragma unroll
                    for (int y = 0; y < kAtOnce; ++y)
                        bits[y] = __vmaxu2(bits[y], __shfl_xor_sync(0xffffffffu, bits[y], o));
#pragma unroll
                for (int y = 0; y < kAtOnce; ++y) {
                    const int at = warp * kWarp + r0 + 2 * y;
                    const uint32_t top = max(bits[y] & 0xffffu, bits[y] >> 16) << 16;
                    const float qs = query_scale(top);
                    uint2 hi, lo;
                    split_query(x[y], power_inverse(qs), hi, lo);
                    unsigned char *to = q_tile + at * 128 + (((piece >> 1) ^ (at & 7)) << 4) + (piece & 1) * 8;
                    *reinterpret_cast<uint2 *>(to) = hi;  // (rows that are not there: zeros)
                    *reinterpret_cast<uint2 *>(to + kQPart) = lo;
                    if (piece == 0) sh.factor[w][at] = top < 0x7f800000u ? qs * P.scale_log2 : NAN;
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
            const int lim = min(p, s.keys.hi - 1), wlo = P.window > 0 ? max(p - P.window + 1, 0) : 0, from = s.keys.from;
            if (!have) m = 0.0f;  // lanes without a row never ask for another reference
            const KeyTiles keys = s.keys;
            const int first = s.tile;
            int last = 0;  // the half that came last
            // a tile is seen whole by all rows from x0 = from on to here, when no window cuts it off
            const int whole = min(s.pmin, keys.hi - 1) - (kKT - 1), cut = P.window > 0 ? s.pmax - P.window : -1;
#pragma unroll 1
            for (int i = 0; i < nt; ++i) {
                const int x0 = tile_begin<kKT>(keys, first + i), n = tile_keys(keys, x0);
                const bool edge = x0 > whole || x0 < from || (x0 <= cut && x0 + kKT > P.n_sink);
                // A wait by parity tells this use of a slot of values from the one before, two tiles ago, once that one is
                // known to have arrived: its products were issued before these scores. So what an early look at the values
                // says counts only if the scores are there, looked at first.
                if (!wait_two(ab, &sh.s_full[w][0], s_phases & 1u, &sh.v_full[values.slot], values.phase)) return;
                const unsigned char *v_tile = v_mem + values.slot * kValues;
                const float *key_scale = sh.key_scale[values.slot], *value_log2 = sh.value_log2[values.slot],
                            *value_inv = sh.value_inv[values.slot];
                const bool skip = edge && (sh.no_number[values.slot][0] | sh.no_number[values.slot][1]) != 0;
#pragma unroll 1
                for (int u = 0; u * kHalf < n; ++u) {
                    const int xu = x0 + u * kHalf, nu = min(n - u * kHalf, kHalf);
                    const uint32_t s_at = s_addr + u * kHalf;
                    if (u > 0 && !wait_warp(ab, &sh.s_full[w][1], s_phases >> 1 & 1u)) return;
                    s_phases ^= 1u << u;
                    tc_fence_after();
                    // (what the half before left here has been read: its product was issued before these scores)
                    if (tid == 0) *reinterpret_cast<volatile uint32_t *>(&sh.skip[w][u]) = skip;
                    // O is at rest once the product of the half before is done; those before that one were issued
                    // before these scores (so that a wait by parity knows it from them)
                    auto at_rest = [&]() -> bool {
                        if (i + u > 0 && !wait_warp(ab, &sh.o_done[w][u ^ 1], (o_phases >> (u ^ 1) & 1u) ^ 1u)) return false;
                        tc_fence_after();
                        return true;
                    };
                    if (warp_has) {
                        float z[64];
                        tmem_ld32(z, s_at);
                        if (nu > 32) tmem_ld32(z + 32, s_at + 32);
                        tmem_wait_ld32(z);
                        tmem_wait_ld32(z + 32);
                        // the weights' logarithms under the reference that there is; eight columns share a scale
                        const float ref = m == -INFINITY ? 0.0f : m;
                        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int c = 0; c < 8; c += 4) {
                            const float4 k4 = *reinterpret_cast<const float4 *>(key_scale + u * (kHalf / 8) + c);
                            const float4 v4 = *reinterpret_cast<const float4 *>(value_log2 + u * (kHalf / 8) + c);
                            const float k[4] = {k4.x * factor, k4.y * factor, k4.z * factor, k4.w * factor};
                            const float less[4] = {v4.x - ref, v4.y - ref, v4.z - ref, v4.w - ref};
#pragma unroll
                            for (int e = 8 * c; e < 8 * c + 32; e += 2) {
                                const float kf = k[e / 8 - c], lf = less[e / 8 - c];
                                const float2 y = fma2(make_float2(z[e], z[e + 1]), make_float2(kf, kf), make_float2(lf, lf));
                                z[e] = y.x;
                                z[e + 1] = y.y;
                            }
                        }
                        if (edge) {
                            // the positions that the row sees, as bits: up to its own, in the window or among the sinks
                            const uint64_t seen = below(lim + 1 - xu) & ~below(from - xu) & (~below(wlo - xu) | below(P.n_sink - xu));
#pragma unroll
                            for (int e = 0; e < 64; ++e)
                                if (!(seen >> e & 1u)) z[e] = -INFINITY;
                        }
#pragma unroll
                        for (int e = 0; e < 64; e += 8) {
                            mx[0] = fmaxf(mx[0], fmaxf(z[e], z[e + 1]));
                            mx[1] = fmaxf(mx[1], fmaxf(z[e + 2], z[e + 3]));
                            mx[2] = fmaxf(mx[2], fmaxf(z[e + 4], z[e + 5]));
                            mx[3] = fmaxf(mx[3], fmaxf(z[e + 6], z[e + 7]));
                        }
                        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                        // a new reference when the old one is too low (or there was none): the largest weight is 2^kTop
                        const bool grow = have && (m == -INFINITY ? top > -INFINITY : top > kMost);
                        if (__any_sync(0xffffffffu, grow)) {
                            if (__any_sync(0xffffffffu, grow && m != -INFINITY)) {
                                if (!at_rest()) return;
                                // (by its root: a sum, divided by scales, may count where 2^(kTop - top) is 0)
                                const float root = grow && m != -INFINITY ? ex2(0.5f * (kTop - top)) : 1.0f, a = root * root;
                                l = l * root * root;
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
                            const float by = grow ? kTop - top : 0.0f;
                            if (grow) m = (m == -INFINITY ? 0.0f : m) - by;
#pragma unroll
                            for (int e = 0; e < 64; e += 2) {
                                const float2 y = add2(make_float2(z[e], z[e + 1]), make_float2(by, by));
                                z[e] = y.x;
                                z[e + 1] = y.y;
                            }
                        }
                        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                        uint32_t pw[32];
#pragma unroll
                        for (int c = 0; c < 8; c += 4) {
                            const float4 i4 = *reinterpret_cast<const float4 *>(value_inv + u * (kHalf / 8) + c);
                            const float inv[4] = {i4.x, i4.y, i4.z, i4.w};
#pragma unroll
                            for (int g = c; g < c + 4; ++g) {  // eight columns of one scale
                                float2 y[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    y[e] = make_float2(ex2(z[8 * g + 2 * e]), ex2(z[8 * g + 2 * e + 1]));
                                    pw[4 * g + e] = pack_f16(y[e].x, y[e].y);
                                }
                                sum[g & 1] = fma2(add2(add2(y[0], y[1]), add2(y[2], y[3])), make_float2(inv[g - c], inv[g - c]),
                                                  sum[g & 1]);
                            }
                            if (c == 0) tmem_st16(s_at, pw);  // over columns that have been read
                        }
                        tmem_st16(s_at + 16, pw + 16);
                        sum[0] = add2(sum[0], sum[1]);
                        l += sum[0].x + sum[0].y;
                        tmem_wait_st();
                        if (skip) {
                            if (!at_rest()) return;
                            mixed_tile(P.D, s_at, o_addr, v_tile, u * kHalf, xu, nu, from, lim, wlo, P.n_sink, i + u == 0);
                        }
                    }
                    tc_fence_before();
                    mbar_arrive(&sh.p_full[w][u]);
                    o_phases ^= 1u << u;
                    last = u;
                }
                values.step();
            }
            if (!wait_warp(ab, &sh.o_done[w][last], (o_phases >> last & 1u) ^ 1u)) return;
            tc_fence_after();
        } else {
            for (int i = 0; i < nt; ++i) values.step();
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
                for (int d = 0; d < width; d += 32) {
                    float o[32];
                    if (nt > 0) {
                        tmem_ld32(o, o_addr + d0 + d);
                        tmem_wait_ld32(o);
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = none ? 0.0f : o[e] * inv;
                    unsigned char *row = mem + lane * 256;
                    const int p0 = part ? d >> 2 : d >> 3;  // (pieces behind the width lie in the row, unused)
                    if (part) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            *reinterpret_cast<float4 *>(row + (((p0 + e) ^ (lane & 7)) << 4)) =
                                make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *reinterpret_cast<uint4 *>(row + (((p0 + e) ^ (lane & 7)) << 4)) =
                                make_uint4(pack_bf16(o[8 * e], o[8 * e + 1]), pack_bf16(o[8 * e + 2], o[8 * e + 3]),
                                           pack_bf16(o[8 * e + 4], o[8 * e + 5]), pack_bf16(o[8 * e + 6], o[8 * e + 7]));
                    }
                }
                __syncwarp();
                const int per = part ? width / 4 : width / 8, at_once = kWarp / per, piece = lane % per;
#pragma unroll 1
                for (int r0 = lane / per; r0 - lane / per < kWarp; r0 += 8 * at_once) {
                    uint4 v[8];
                    int64_t dst[8];
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        const int r = (r0 + y * at_once) & 31;  // (beyond the warp's rows: not stored)
                        dst[y] = __shfl_sync(0xffffffffu, row_out, r);
                        v[y] = *reinterpret_cast<const uint4 *>(mem + r * 256 + ((piece ^ (r & 7)) << 4));
                    }
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        const int r = r0 + y * at_once;
                        if (lane >= at_once * per || r >= kWarp || warp * kWarp + r >= mine) continue;
                        if (part) {
                            if (SPEC_IN(dst[y] + d0 + 4 * piece, P.part_rows * P.D, DBG_ATTEND))
                                *reinterpret_cast<uint4 *>(P.part_o + dst[y] + d0 + 4 * piece) = v[y];
                        } else if (SPEC_IN(dst[y] + d0 + 8 * piece, P.T * P.out_stride, DBG_ATTEND)) {
                            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(P.out) + dst[y] + d0 + 8 * piece) = v[y];
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
                             const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ unsigned char raw[];
    unsigned char *base = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    unsigned char *v_mem = base + 2 * kQBytes, *ring_mem = v_mem + 2 * kValues;
    Shared &sh = *reinterpret_cast<Shared *>(ring_mem + kStages * kTile);
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;

    if (warp == 9) tmem_alloc(&sh.tmem, 512);
    if (threadIdx.x == 0) {
        init_pipe(sh.pipe, 2, 11);  // values: the converting warps; segments: eight softmax warps, the issuing one and these
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.q_full[i], 128);
            for (int u = 0; u < 2; ++u) {
                mbar_init(&sh.s_full[i][u], 1);
                mbar_init(&sh.p_full[i][u], 128);
                mbar_init(&sh.o_done[i][u], 1);
                sh.skip[i][u] = 0;
            }
            mbar_init(&sh.agree[i], 4);
            mbar_init(&sh.v_full[i], 2);
            mbar_init(&sh.v_empty[i], 1);
        }
        mbar_init(&sh.drain, 1);
        fence_mbar_init();
        prefetch_map(&kmap);
        prefetch_map(&vmap);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    begin_kernel<PREFIX>(P);

    if (warp < 8) {
        softmax_role<PREFIX>(P, sh, base + (warp / 4) * kQBytes, v_mem, warp / 4);
    } else if (warp == 8) {
        load_role<PREFIX>(P, M, &kmap, &vmap, sh.pipe, ring_mem, blockIdx.x, lane);
    } else if (warp == 9) {
        mma_role(P, sh, base, v_mem, ring_mem);
        // nothing this warp issued is in flight when the CTA ends
        if (elect_lane()) mma_commit(&sh.drain);
        __syncwarp();
#pragma unroll 1
        for (int t = 0; t < kTries && !mbar_try_wait_sleep(&sh.drain, 0, kHintNs); ++t) {
        }
    } else {
        if constexpr (!PREFIX)
            if (warp == 11) keep_books<kKT>(P, lane);
        convert_role(P, sh, v_mem, ring_mem, warp - 10, lane);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_free(sh.tmem, 512);
    end_kernel<PREFIX>(P);
    if (threadIdx.x == 0) P.err[(PREFIX ? P.own_workers : 0) + blockIdx.x] = sh.pipe.abort;
}

}  // namespace pair8
}  // namespace spec
