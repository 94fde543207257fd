// Attention of few rows over the cache in 8 bits on the tensor cores (head sizes that are multiples of 16 up to 128): a
// verification round, single tokens; fp32 rows also in larger numbers. The work is laid out as in spec_attend_round.cuh: positions and
// output columns along the lanes, the item's rows along the columns,
//   S^T = K Q^T     K as it lies in the cache, Q in two parts (spec_attend8_tiles.cuh)
//   O^T += V^T P^T  V as it lies in the cache, P in three parts, each with rows of RT bytes a position
// Half the bytes of bf16 make the time between two tiles half as long, while the products take 20 instructions a
// tile instead of 16, of 42 cycles each (a product's time follows its 128 lanes until it has 64 columns). So one
// warp issues them together (a single thread took 126 cycles an instruction to issue them).
//
// Measured (us a call, back to back; heads 32 / 8 of 128): 16 requests of 1-8 rows with texts to 65000 (1.0 GB) 188, 0.81
// of the copy rate, and 0.90 with 4 rows each; 64 requests under a window of 1024 (137 MB) 61; 5 rows of one request 12.6.
// A tile takes a CTA 2500-2800 cycles with 32 rows, of which the tensor cores work 840 and the softmax threads the
// rest, two CTAs an SM in turn; the copies alone take 159-189 us for the long texts, by the order of the pages. So the long
// ones are bound by bytes and, with rows above 16, by the weights' arithmetic (three e5m2 a weight: eight instructions);
// the window's items of nine tiles by their ends: some 3 us for the plan, 2 for the first tile's references.
// What brought it here: hardware barriers between the softmax warps, and keys and values in rings of their own (226 ->
// 191), heads of the same positions read in step, an edge tile's visible rows as bits (window 74 -> 61).
// Two softmax warpgroups of 96 registers spilled and were twice as slow; three CTAs an SM spilled too.
//
// Scales. A thread has one position: its key's scale is one factor of all its scores, and a row's factor (the
// query's own scale, the softmax's and log2 e) comes from shared memory beside the row's reference. The value's
// scale v goes into the weight, w = 2^(z + log2 v - reference), so that the weights' range follows what they
// contribute; the row's sum takes w / v. The reference puts the first tile's largest weight at 2^11, and is renewed
// when one passes 2^15: e5m2 holds weights from 2^15 down to 2^-16, that is 2^-27 of the reference.
#pragma once

#include "spec_attend8_tiles.cuh"

namespace spec {
namespace round8 {

using namespace tiles8;

constexpr int kThreads = 192, kPerSM = 2;
constexpr float kTop = 11.0f;  // log2 of the largest weight under a new reference, and of what may be reached
constexpr float kMost = 15.0f; // before the next

// What a row's type asks for. bf16: queries in two parts, weights in three, one accumulator each. fp32: two more parts
// of the queries and three of the weights, which hold what the first ones leave times 2^kQueryShift and 2^kWeightShift,
// each in an accumulator of its own, so that e4m3 and e5m2 need not reach down to it: 19 and 22 bits in all, and 25
// bits below a query's largest element. 40 instructions a tile instead of 20, and still a fifth of the fp32 units' time:
// 64 requests of up to 4096 positions, 12 / 4 heads (128 MB) 246 -> 56 us, 0.34 of the copy rate, bound by the softmax threads, which make
// six parts of a weight.
template <bool WIDE>
struct Parts {
    static constexpr int kSets = WIDE ? 2 : 1, kQ = 2, kP = 3;  // accumulators, and parts in each
    // Tiles whose products are summed by the tensor cores, which cut sums off instead of rounding them: each
    // instruction takes about 2^-23.5 off an accumulator of one sign, 12 of them a tile. bf16 rows can bear that (2^-13
    // after a hundred tiles); fp32 rows' sums go to columns of their own every few tiles, added up in fp32, and the
    // smaller parts are taken first, while there is little to cut.
    static constexpr int kGroup = WIDE ? 2 : 1 << 30;
};
constexpr int kQueryShift = 8, kWeightShift = 11;

template <int RT, bool WIDE>
struct Shared {
    Pipe<2, RT == 32 && !WIDE ? 3 : 2> pipe;
    uint64_t q_full, s_full[2], p_full, o_done, drain;
    uint32_t found[4];     // per warp: what it brings to a meeting
    uint32_t skip;         // the warpgroup has done this tile's second product itself
    uint32_t tmem;
    // of this segment's rows and the next one's, in turn
    int pos[2][RT];                 // positions (-1: none)
    alignas(16) float nref[2][RT];  // minus the reference; kNoRef before there is one (read four at a time)
    alignas(16) float factor[2][RT];  // of the scores
};
// What the row operations of a warpgroup need now and then, in the weights' memory while that is unused.
template <int RT>
struct Scratch {
    float warp[4][RT];
    alignas(16) float row[RT];
    int64_t to[RT];  // where a row goes (-1: nowhere)
};
// A reference that every finite score exceeds and that leaves -inf alone.
constexpr float kNoRef = 3e38f;

// Queries: parts of 128 bytes a row; weights: parts of a byte a row and position.
__host__ __device__ constexpr int q_part(int RT) { return RT * 128; }
__host__ __device__ constexpr int p_part(int RT) { return kKT * RT; }
template <bool WIDE>
__host__ __device__ constexpr int q_bytes(int RT) {
    return Parts<WIDE>::kSets * Parts<WIDE>::kQ * q_part(RT);
}
template <bool WIDE>
__host__ __device__ constexpr int p_bytes(int RT) {
    return Parts<WIDE>::kSets * Parts<WIDE>::kP * p_part(RT);
}
template <int RT, bool WIDE>
__host__ __device__ constexpr int stages() {
    return decltype(Shared<RT, WIDE>::pipe)::kKeys + decltype(Shared<RT, WIDE>::pipe)::kValues;
}
template <int RT, bool WIDE>
__host__ constexpr int smem_bytes() {
    return stages<RT, WIDE>() * kTile + q_bytes<WIDE>(RT) + p_bytes<WIDE>(RT) + static_cast<int>(sizeof(Shared<RT, WIDE>));
}
// 228 KB of shared memory, 1 KB of it taken per CTA
constexpr int kMostSmem = 228 * 1024 / kPerSM - 1024;
static_assert(smem_bytes<32, false>() <= kMostSmem && smem_bytes<64, false>() <= kMostSmem && smem_bytes<32, true>() <= kMostSmem,
              "fits");
static_assert(sizeof(Scratch<64>) <= p_bytes<false>(64) && sizeof(Scratch<32>) <= p_bytes<false>(32), "fits the weights' memory");

// ---------------------------------------------------------------- matrix instructions (one warp)

template <int RT, bool WIDE>
__device__ __forceinline__ void mma_role(const AttendParams &P, Shared<RT, WIDE> &sh, unsigned char *ring_mem,
                                         unsigned char *q_tile, unsigned char *p_tile) {
    int32_t *ab = &sh.pipe.abort;
    constexpr int kKeys = decltype(Shared<RT, WIDE>::pipe)::kKeys, kValues = decltype(Shared<RT, WIDE>::pipe)::kValues;
    constexpr int kSets = Parts<WIDE>::kSets, kQ = Parts<WIDE>::kQ, kP = Parts<WIDE>::kP, kGroup = Parts<WIDE>::kGroup;
    const uint32_t s_col = sh.tmem, o_col = sh.tmem + 2 * kSets * RT;
    const uint64_t q_op = smem_operand(smem_addr(q_tile), 16), k_op = smem_operand(smem_addr(ring_mem), 16),
                   v_op = smem_operand(smem_addr(ring_mem + kKeys * kTile), 16),
                   p_op = RT == 64 ? smem_operand64(smem_addr(p_tile)) : smem_operand32(smem_addr(p_tile));
    const int steps = (P.D + 31) / 32;
    Ring next = {0, kKeys, 0}, v = {0, kValues, 0}, desc = {0, 2, 0};
    uint32_t q_phase = 0, p_phase = 0;
    for (;;) {
        if (!wait_warp(ab, &sh.pipe.desc_full[desc.slot], desc.phase)) return;
        const Segment &s = sh.pipe.desc[desc.slot];
        const int nrows = s.nrows, nt = s.ntile, first = s.tile;
        const KeyTiles keys = s.keys;
        if (nrows == 0) return;
        if (nt > 0) {
            const int n16 = (nrows + 15) & ~15;
            // (a bf16 query's second part is e5m2)
            const uint32_t qk_shapes[2] = {mma8_shape(n16, false, false, false, false),
                                           mma8_shape(n16, false, !WIDE, false, false)},
                           pv_shape = mma8_shape(n16, false, true, true, true);
            if (!wait_warp(ab, &sh.q_full, q_phase)) return;
            q_phase ^= 1u;
            // step t: tile t's product, and tile t + 1's scores (step -1: the first scores alone). The scores
            // go first if their keys are there.
#pragma unroll 1
            for (int t = -1; t < nt; ++t) {
                const bool more = t + 1 < nt;
                const bool ahead = more && __all_sync(0xffffffffu, mbar_try_wait(&sh.pipe.k_full[next.slot], next.phase));
#pragma unroll 1
                for (int part = 0; part < 2; ++part) {
                    if (part == (ahead ? 0 : 1)) {
                        if (!more) continue;
                        if (!ahead && !wait_warp(ab, &sh.pipe.k_full[next.slot], next.phase)) return;
                        tc_fence_after();
                        const int b = (t + 1) & 1;  // S^T = K Q^T
                        const uint64_t k = operand_at(k_op, next.slot * kTile);
                        if (elect_lane()) {
#pragma unroll
                            for (int q = kSets * kQ - 1; q >= 0; --q)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    if (i < steps)
                                        mma8_ss(s_col + (b * kSets + q / kQ) * RT, operand_at(k, i * 32),
                                                operand_at(q_op, q * q_part(RT) + i * 32), qk_shapes[q % kQ],
                                                q % kQ < kQ - 1 || i > 0);
                            mma_commit(&sh.s_full[b]);
                            mma_commit(&sh.pipe.k_empty[next.slot]);
                        }
                        __syncwarp();
                    } else if (t >= 0) {
                        if (!wait_warp(ab, &sh.pipe.v_full[v.slot], v.phase)) return;
                        if (!wait_warp(ab, &sh.p_full, p_phase)) return;
                        p_phase ^= 1u;
                        tc_fence_after();
                        const bool take = !*reinterpret_cast<volatile uint32_t *>(&sh.skip);
                        const uint64_t values = operand_at(v_op, v.slot * kTile);
                        const int n = tile_keys(keys, tile_begin<kKT>(keys, first + t));
                        if (elect_lane()) {
                            if (take) {  // O^T += V^T P^T
#pragma unroll
                                for (int p = kSets * kP - 1; p >= 0; --p)
#pragma unroll
                                    for (int i = 0; i < 4; ++i)
                                        if (i * 32 < n)
                                            mma8_ss(o_col + p / kP * RT, operand_at(values, i * 4096),
                                                    operand_at(p_op, p * p_part(RT) + i * 32 * RT), pv_shape,
                                                    t % kGroup > 0 || p % kP < kP - 1 || i > 0);
                            }
                            mma_commit(&sh.o_done);
                            mma_commit(&sh.pipe.v_empty[v.slot]);
                        }
                        __syncwarp();
                    }
                }
                if (more) next.step();
                if (t >= 0) v.step();
            }
        }
        if (elect_lane()) mbar_arrive(&sh.pipe.desc_empty[desc.slot]);
        __syncwarp();
        desc.step();
    }
}

// ---------------------------------------------------------------- softmax (one position per thread)

// The four warps meet at a hardware barrier: true when some thread brings a flag. A meeting has no limit of its own, so
// all four come to every one: a warp whose bounded wait has given up goes on with what it has (`gone`), brings that
// to the next meeting, and there they leave together. (At an mbarrier, with words in shared memory, a meeting
// took some 1000 cycles of a tile's 4000.)
__device__ __forceinline__ bool meet(bool flag) { return bar_any(1, 128, flag); }
// The same with a word each, of which all get the union.
__device__ __forceinline__ uint32_t meet_words(uint32_t *found, uint32_t mine) {
    if (!meet(mine != 0u)) return 0u;
    if (threadIdx.x % kWarp == 0) found[threadIdx.x / kWarp] = mine;
    bar_sync(1, 128);
    const uint32_t all = found[0] | found[1] | found[2] | found[3];
    bar_sync(1, 128);
    return all;
}
constexpr uint32_t kBeyond = 1, kNoNumber = 2, kGone = 4;  // a weight too large, a value that is no number, a wait given up

// The second product of a tile with values that are not finite, on the fp32 units: thread d has output
// column d, the weights lie in shared memory, O is complete up to the tile before (what this adds goes to its first
// accumulator; the others begin with 0 if the tile is the first).
template <int RT, bool WIDE>
__device__ __noinline__ void mixed_tile(const AttendParams &P, const int *pos, uint32_t o_addr,
                                        const unsigned char *v_tile, const unsigned char *p_tile, const KeyTiles &keys,
                                        int x0, int n, int nrows, int d, bool first) {
#pragma unroll 1
    for (int r0 = 0; r0 < nrows; r0 += 16) {
        float o[16];
        __syncwarp();
        tmem_ld16(o, o_addr + r0);
        tmem_wait_ld();
        if (first)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = 0.0f;
#pragma unroll 1
        for (int k = 0; k < n; ++k) {
            const int x = x0 + k;
            if (!item_sees(P, keys, x)) continue;
            const float v = d < P.D ? tile_value(v_tile, k, d) : 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int r = r0 + e, p = r < nrows ? pos[r] : -1;
                if (x <= p && (P.window == 0 || x > p - P.window || x < P.n_sink)) {
                    const int piece = RT == 64 ? (r >> 4) ^ ((k >> 1) & 3) : (r >> 4) ^ ((k >> 2) & 1);
                    const unsigned char *at = p_tile + k * RT + piece * 16 + (r & 15);
                    float w = e5m2_to_float(at[0]) + e5m2_to_float(at[p_part(RT)]) + e5m2_to_float(at[2 * p_part(RT)]);
                    if constexpr (WIDE)
                        w += 0x1p-11f * (e5m2_to_float(at[3 * p_part(RT)]) + e5m2_to_float(at[4 * p_part(RT)]) +
                                         e5m2_to_float(at[5 * p_part(RT)]));
                    o[e] = fmaf(w, v, o[e]);
                }
            }
        }
        uint32_t ow[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) ow[e] = __float_as_uint(o[e]);
        __syncwarp();
        tmem_st16(o_addr + r0, ow);
        if (WIDE && first) {
#pragma unroll
            for (int e = 0; e < 16; ++e) ow[e] = 0u;
            tmem_st16(o_addr + RT + r0, ow);
        }
        tmem_wait_st();
    }
}

template <int RT, bool PREFIX, bool WIDE>
__device__ __forceinline__ void softmax_role(const AttendParams &P, Shared<RT, WIDE> &sh, unsigned char *ring_mem,
                                             unsigned char *q_tile, unsigned char *p_tile) {
    constexpr int kKeys = decltype(Shared<RT, WIDE>::pipe)::kKeys, kValues = decltype(Shared<RT, WIDE>::pipe)::kValues;
    const int tid = threadIdx.x, warp = tid / kWarp, lane = tid % kWarp;
    int32_t *ab = &sh.pipe.abort;
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    constexpr int kSets = Parts<WIDE>::kSets, kP = Parts<WIDE>::kP, kGroup = Parts<WIDE>::kGroup;
    const uint32_t s_addr = sh.tmem + lanes, o_addr = s_addr + 2 * kSets * RT, sum_addr = o_addr + kSets * RT;
    Scratch<RT> &scratch = *reinterpret_cast<Scratch<RT> *>(p_tile);
    Ring values = {0, kValues, 0}, desc = {0, 2, 0};
    uint32_t s_phases = 0, o_phase = 0;
    int buf = 0;
    bool gone = false;
    // Brings a segment's queries: 128 / RT threads each row's (rows up to a multiple of 16: zeros), and its
    // position.
    auto bring = [&](const Segment &s, int to) {
        constexpr int kPer = 128 / RT, kPieces = 16 / kPer;  // of eight elements
        const int r = tid / kPer, pr = s.row0 + r, j = P.by_group(pr), g = pr - j * P.G;
        const int t = s.t0 + j, h = s.head * P.G + g;
        const bool have = r < s.nrows && SPEC_IN(t, P.T, DBG_ATTEND);
        const int64_t row = t * P.q_stride + static_cast<int64_t>(h) * P.D;
        auto whole = [&](uint32_t top) {
#pragma unroll
            for (int o = 1; o < kPer; o <<= 1) top = WIDE ? max(top, __shfl_xor_sync(0xffffffffu, top, o))
                                                          : __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
            return top;
        };
        auto at = [&](int c) { return q_tile + r * 128 + (((c >> 1) ^ (r & 7)) << 4) + (c & 1) * 8; };
        const bool taken = r < ((s.nrows + 15) & ~15);
        float qs;
        bool finite;
        if constexpr (!WIDE) {
            const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(P.q) + row);
            uint4 x[kPieces];
            uint32_t top = 0u;
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int c = tid % kPer + i * kPer;
                x[i] = have && c < P.D / 8 ? src[c] : make_uint4(0u, 0u, 0u, 0u);
                top = top_bits(top, x[i]);
            }
            top = whole(top);
            const uint32_t bits = max(top & 0xffffu, top >> 16) << 16;
            finite = bits < 0x7f800000u;
            qs = query_scale(bits);
            if (taken)
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const int c = tid % kPer + i * kPer;
                    uint2 hi, lo;
                    split_query(x[i], power_inverse(qs), hi, lo);
                    *reinterpret_cast<uint2 *>(at(c)) = hi;
                    *reinterpret_cast<uint2 *>(at(c) + q_part(RT)) = lo;
                }
        } else {
            const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(P.q) + row);
            uint32_t top = 0u;
            auto piece = [&](int i, int half) {
                const int c = tid % kPer + i * kPer;
                return have && c < P.D / 8 ? src[2 * c + half] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            };
#pragma unroll
            for (int i = 0; i < 2 * kPieces; ++i) {
                const float4 x = piece(i / 2, i % 2);
                top = max(top, max(max(__float_as_uint(x.x) & 0x7fffffffu, __float_as_uint(x.y) & 0x7fffffffu),
                                   max(__float_as_uint(x.z) & 0x7fffffffu, __float_as_uint(x.w) & 0x7fffffffu)));
            }
            top = whole(top);
            finite = top < 0x7f800000u;
            qs = query_scale(top);
            if (taken)
#pragma unroll 2
                for (int i = 0; i < 2 * kPieces; ++i) {  // (read again, from L1)
                    uint32_t parts[4];
                    split_query_wide<kQueryShift>(piece(i / 2, i % 2), power_inverse(qs), parts);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        *reinterpret_cast<uint32_t *>(at(tid % kPer + i / 2 * kPer) + q * q_part(RT) + i % 2 * 4) = parts[q];
                }
        }
        if (taken) {
            if (tid % kPer == 0) {
                int p = -1;
                if (have) {
                    if constexpr (PREFIX) {
                        const ReqRows q = load_request(P, find_request(P.row_off, P.B, P.T, t));
                        if (t >= q.r0 && t < q.r0 + q.n) p = q.kv - q.n + (t - q.r0);
                    } else {
                        p = s.base + j;
                    }
                }
                sh.pos[to][r] = p;
                sh.nref[to][r] = kNoRef;
                sh.factor[to][r] = finite ? qs * P.scale_log2 : NAN;
            }
        }
        if (s.ntile > 0) {
            fence_proxy_async_smem();
            mbar_arrive(&sh.q_full);
        }
    };
    bool first_segment = true;
    for (;;) {
        const Segment &s = sh.pipe.desc[desc.slot];
        if (first_segment) {
            gone = !wait_warp(ab, &sh.pipe.desc_full[0], 0);
            if (meet(gone)) return;
            if (s.nrows == 0) return;
            bring(s, 0);
            bar_sync(1, 128);
            first_segment = false;
        }
        const int nrows = s.nrows, nt = s.ntile, n16 = (nrows + 15) & ~15;
        const int *pos = sh.pos[buf];
        float *nref = sh.nref[buf];
        const float *factor = sh.factor[buf];

        float2 l[RT / 2];  // this thread's share of the rows' sums
#pragma unroll
        for (int e = 0; e < RT / 2; ++e) l[e] = make_float2(0.0f, 0.0f);
#pragma unroll 1
        for (int i = 0; i < nt; ++i) {
            const int b = i & 1;
            const int x0 = tile_begin<kKT>(s.keys, s.tile + i), n = tile_keys(s.keys, x0), x = x0 + tid;
            const bool edge = edge_tile(P, s, x0);
            unsigned char *v_tile = ring_mem + (kKeys + values.slot) * kTile;
            uint32_t mine = 0u;
            bool rested = i == 0;
            auto rest = [&]() {
                if (rested) return;
                rested = true;
                gone |= !wait_warp(ab, &sh.o_done, o_phase);
                o_phase ^= 1u;
                tc_fence_after();
            };
            // The scales come with the values. (A wait by parity cannot take the use of the slot before for this one: that
            // was two tiles ago or more, and the product of its values has been waited for.)
            if (edge) {
                gone |= !wait_warp(ab, &sh.pipe.v_full[values.slot], values.phase);
                if (__any_sync(0xffffffffu, clean_values(P, s, v_tile, x0, n, tid))) mine = kNoNumber;
                fence_proxy_async_smem();
            }
            gone |= !(edge ? wait_warp(ab, &sh.s_full[b], s_phases >> b & 1u)
                           : wait_two(ab, &sh.s_full[b], s_phases >> b & 1u, &sh.pipe.v_full[values.slot], values.phase));
            s_phases ^= 1u << b;
            tc_fence_after();
            // this position's scales (1 where no row sees it and none were copied)
            const bool used = !edge || item_sees(P, s.keys, x);
            const float2 by = used ? sh.pipe.scale[values.slot][tid >> P.box_log2] : make_float2(1.0f, 1.0f);
            const ValueScale vs = value_scale(by.y);
            const float2 kf = make_float2(by.x, by.x), vl = make_float2(vs.log2, vs.log2), vi = make_float2(vs.inv, vs.inv);
            // in an edge tile, the rows that see this position
            uint32_t seen[RT / 32];
            if (edge) {
                const bool in = x >= s.keys.from && x < s.keys.hi, sink = x < P.n_sink;
                if constexpr (PREFIX) {
                    const int back = P.window > 0 ? P.window : INT_MAX;
#pragma unroll
                    for (int c = 0; c < RT / 32; ++c) {
                        seen[c] = 0u;
#pragma unroll 4
                        for (int y = 0; y < 32; ++y) {
                            const int p = 32 * c + y < n16 ? pos[32 * c + y] : -1;
                            if (in && x <= p && (sink || p - x < back)) seen[c] |= 1u << y;
                        }
                    }
                } else {
                    // positions grow with the packed rows, by one every G: those from the position's own on, up to where the
                    // window has gone by
                    const int64_t first = in ? (static_cast<int64_t>(x) - s.base) * P.G - s.row0 : RT;
                    const int64_t last = P.window > 0 && !sink ? first + static_cast<int64_t>(P.window) * P.G : RT;
                    const int a = static_cast<int>(min(max(first, static_cast<int64_t>(0)), static_cast<int64_t>(RT))),
                              z = static_cast<int>(min(max(last, static_cast<int64_t>(0)), static_cast<int64_t>(RT)));
#pragma unroll
                    for (int c = 0; c < RT / 32; ++c) {
                        const int lo = min(max(a - 32 * c, 0), 32), hi = min(max(z - 32 * c, 0), 32);
                        seen[c] = hi > lo ? 0xffffffffu >> (32 - (hi - lo)) << lo : 0u;
                    }
                }
            }
            // from 16 rows' products (from row e on) to the logarithms of this position's weights, references aside
            auto finish = [&](float *z, int e) {
#pragma unroll
                for (int y = 0; y < 16; y += 4) {
                    const float4 fc = *reinterpret_cast<const float4 *>(factor + e + y);
                    const float2 a = fma2(mul2(make_float2(z[y], z[y + 1]), kf), make_float2(fc.x, fc.y), vl),
                                 c = fma2(mul2(make_float2(z[y + 2], z[y + 3]), kf), make_float2(fc.z, fc.w), vl);
                    z[y] = a.x;
                    z[y + 1] = a.y;
                    z[y + 2] = c.x;
                    z[y + 3] = c.y;
                }
                if (edge) {
#pragma unroll
                    for (int y = 0; y < 16; ++y)
                        if (!(seen[(e + y) / 32] >> (e + y) % 32 & 1u)) z[y] = -INFINITY;
                }
            };
            // 32 rows' scores stay in registers; 64 rows' would not, beside their sums, and are read anew
            constexpr bool kHeld = RT == 32;
            float held[kHeld ? RT : 16];
            if constexpr (kHeld) {
                const uint32_t from = s_addr + b * kSets * RT;
                if (nrows > 16)
                    tmem_ld32(held, from);
                else
                    tmem_ld16(held, from);
                if constexpr (WIDE) {
                    float rest[RT];
                    if (nrows > 16)
                        tmem_ld32(rest, from + RT);
                    else
                        tmem_ld16(rest, from + RT);
                    tmem_wait_ld32(held);
                    tmem_wait_ld32(rest);
#pragma unroll
                    for (int e = 0; e < RT; ++e) held[e] = fmaf(rest[e], 1.0f / (1 << kQueryShift), held[e]);
                } else {
                    tmem_wait_ld32(held);
                }
#pragma unroll
                for (int e = 0; e < RT; e += 16)
                    if (e < nrows) finish(held + e, e);
            }
            auto scores = [&](int e) -> float * {
                if constexpr (kHeld) return held + e;
                tmem_ld16(held, s_addr + b * RT + e);
                tmem_wait_ld();
                finish(held, e);
                return held;
            };
            // the logarithms of four weights
            auto against = [&](const float *z, int e, float2 &a, float2 &c) {
                const float4 rf = *reinterpret_cast<const float4 *>(nref + e);
                a = add2(make_float2(z[0], z[1]), make_float2(rf.x, rf.y));
                c = add2(make_float2(z[2], z[3]), make_float2(rf.z, rf.w));
            };
            if (i > 0) {
                float top = -INFINITY;
#pragma unroll
                for (int e = 0; e < RT; e += 16)
                    if (e < nrows) {
                        const float *z = scores(e);
#pragma unroll
                        for (int y = 0; y < 16; y += 4) {
                            float2 a, c;
                            against(z + y, e + y, a, c);
                            top = fmaxf(fmaxf(top, fmaxf(a.x, a.y)), fmaxf(c.x, c.y));
                        }
                    }
                mine |= __any_sync(0xffffffffu, top > kMost) ? kBeyond : 0u;
            }
            mine |= gone ? kGone : 0u;
            uint32_t word = meet_words(sh.found, mine);
            if (word & kGone) return;
            rest();  // the product before this tile: the weights' memory is free, O at rest
            if (WIDE && i > 0 && i % kGroup == 0) {
#pragma unroll 1
                for (int r0 = 0; r0 < nrows; r0 += 16) {
                    float o[16], more[16], sum[16];
                    uint32_t ow[16];
                    tmem_ld16(o, o_addr + r0);
                    tmem_ld16(more, o_addr + RT + r0);
                    tmem_ld16(sum, sum_addr + r0);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        ow[e] = __float_as_uint((i > kGroup ? sum[e] : 0.0f) + fmaf(more[e], 1.0f / (1 << kWeightShift), o[e]));
                    tmem_st16(sum_addr + r0, ow);
                }
                tmem_wait_st();
            }
            if (i == 0 || word & kBeyond) {
                // new references: the rows' maxima over the tile, where they are larger
#pragma unroll
                for (int e = 0; e < RT; e += 16)
                    if (e < nrows) {
                        const float *z = scores(e);
#pragma unroll
                        for (int y = 0; y < 16; ++y) {
                            const float v = redux_max(z[y]);
                            if (lane == 0) scratch.warp[warp][e + y] = v;
                        }
                    }
                bar_sync(1, 128);
                if (tid < n16) {
                    const float v = fmaxf(fmaxf(scratch.warp[0][tid], scratch.warp[1][tid]),
                                          fmaxf(scratch.warp[2][tid], scratch.warp[3][tid]));
                    const float old = nref[tid], nw = kTop - v;
                    const bool grow = v != -INFINITY && (old == kNoRef || nw < old);
                    // A row without weights so far has nothing to rescale. Where 2^(nw - old) is 0, sums vanish whose terms
                    // are below 2^-32 of the new ones' (scales up to 2^90 apart, references up to 2^4 behind their maxima).
                    // By the root twice, as in the pair kernel, whose references may lag 2^8, windows take 62.3 us for 61.1.
                    scratch.row[tid] = grow && old != kNoRef ? ex2(nw - old) : 1.0f;
                    if (grow) nref[tid] = nw;
                }
                bar_sync(1, 128);
                if (i > 0) {
#pragma unroll
                    for (int e = 0; e < RT; e += 2)
                        if ((e & ~15) < nrows) {
                            l[e / 2].x *= scratch.row[e];
                            l[e / 2].y *= scratch.row[e + 1];
                        }
#pragma unroll 1
                    for (int c0 = 0; c0 < (WIDE ? kSets + 1 : 1) * RT; c0 += 16) {  // (and the sums)
                        const int r0 = c0 % RT;
                        if (r0 >= nrows) continue;
                        float o[16];
                        uint32_t ow[16];
                        tmem_ld16(o, o_addr + c0);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) ow[e] = __float_as_uint(o[e] * scratch.row[r0 + e]);
                        tmem_st16(o_addr + c0, ow);
                    }
                    tmem_wait_st();
                    bar_sync(1, 128);  // the scratch has been read
                }
            }
            const bool skip = (word & kNoNumber) != 0;
            unsigned char *prow = p_tile + tid * RT;
#pragma unroll
            for (int e = 0; e < RT; e += 16)
                if (e < nrows) {
                    const float *z = scores(e);
                    uint32_t pw[4][kSets * kP];
#pragma unroll
                    for (int y = 0; y < 16; y += 4) {
                        float2 a, c;
                        against(z + y, e + y, a, c);
                        a.x = ex2(a.x);
                        a.y = ex2(a.y);
                        c.x = ex2(c.x);
                        c.y = ex2(c.y);
                        if (edge) {
                            // (the logarithm of a scale that is no number must not reach rows that do not see it)
                            a.x = z[y] == -INFINITY ? 0.0f : a.x;
                            a.y = z[y + 1] == -INFINITY ? 0.0f : a.y;
                            c.x = z[y + 2] == -INFINITY ? 0.0f : c.x;
                            c.y = z[y + 3] == -INFINITY ? 0.0f : c.y;
                        }
                        l[(e + y) / 2] = fma2(a, vi, l[(e + y) / 2]);
                        l[(e + y) / 2 + 1] = fma2(c, vi, l[(e + y) / 2 + 1]);
                        if constexpr (WIDE)
                            split_e5m2_wide<kWeightShift>(a.x, a.y, c.x, c.y, pw[y / 4]);
                        else
                            split_e5m2(a.x, a.y, c.x, c.y, pw[y / 4]);
                    }
                    const int piece = RT == 64 ? (e >> 4) ^ ((tid >> 1) & 3) : (e >> 4) ^ ((tid >> 2) & 1);
#pragma unroll
                    for (int p = 0; p < kSets * kP; ++p)
                        *reinterpret_cast<uint4 *>(prow + p * p_part(RT) + piece * 16) =
                            make_uint4(pw[0][p], pw[1][p], pw[2][p], pw[3][p]);
                }
            if (skip) {
                bar_sync(1, 128);  // all weights are there
                mixed_tile<RT, WIDE>(P, pos, o_addr, v_tile, p_tile, s.keys, x0, n, nrows, tid, i % kGroup == 0);
            }
            if (tid == 0) *reinterpret_cast<volatile uint32_t *>(&sh.skip) = skip;
            fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive(&sh.p_full);
            values.step();
        }
        // the next segment's queries; this one's scores have all been taken
        Ring then = desc;
        then.step();
        gone |= !wait_warp(ab, &sh.pipe.desc_full[then.slot], then.phase);
        if (meet(gone)) return;
        const bool more = sh.pipe.desc[then.slot].nrows > 0;
        if (more) bring(sh.pipe.desc[then.slot], buf ^ 1);
        if (nt > 0) {
            gone |= !wait_warp(ab, &sh.o_done, o_phase);
            o_phase ^= 1u;
            tc_fence_after();
        }
        // the sums: over the lanes, lane x ending with row x (and 32 + x) of its chunk, then over the warps
#pragma unroll
        for (int c = 0; c < RT; c += 32) {
            float v[32];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                v[2 * e] = l[c / 2 + e].x;
                v[2 * e + 1] = l[c / 2 + e].y;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const bool up = lane & o;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (e < o) {
                        const float send = up ? v[e] : v[e + o], keep = up ? v[e + o] : v[e];
                        v[e] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                    }
            }
            scratch.warp[warp][c + lane] = v[0];
        }
        if (meet(gone)) return;
        if (tid < nrows) {
            float sum = scratch.warp[0][tid] + scratch.warp[1][tid] + scratch.warp[2][tid] + scratch.warp[3][tid];
            if (pos[tid] < 0) sum = 0.0f;  // padding
            const bool none = sum == 0.0f;
            const float m = none ? -INFINITY : -nref[tid];
            int64_t to = -1;
            if (s.part >= 0) {
                // a sum that is not a number must reach the joined row, whatever the other parts' maxima
                if (SPEC_IN(s.part + tid, P.part_rows, DBG_ATTEND)) {
                    P.part_ml[s.part + tid] = make_float2(isnan(sum) ? INFINITY : m, sum);
                    to = (s.part + tid) * P.D;
                }
                scratch.row[tid] = none ? 0.0f : 1.0f;
            } else {
                const int j = P.by_group(s.row0 + tid), g = s.row0 + tid - j * P.G, h = s.head * P.G + g;
                if (SPEC_IN(s.t0 + j, P.T, DBG_ATTEND)) {
                    if (P.lse)
                        P.lse[static_cast<int64_t>(s.t0 + j) * P.Hq + h] =
                            none ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
                    to = (s.t0 + j) * P.out_stride + static_cast<int64_t>(h) * P.D;
                }
                scratch.row[tid] = none ? 0.0f : 1.0f / sum;
            }
            scratch.to[tid] = to;
        }
        bar_sync(1, 128);
        const bool part = s.part >= 0;
#pragma unroll 1
        for (int r0 = 0; r0 < nrows; r0 += 16) {
            float o[16];
            __syncwarp();
            if (nt > 0) {
                tmem_ld16(o, o_addr + r0);
                if constexpr (WIDE) {
                    float rest[16], sum[16];
                    tmem_ld16(rest, o_addr + RT + r0);
                    tmem_ld16(sum, sum_addr + r0);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        o[e] = fmaf(rest[e], 1.0f / (1 << kWeightShift), o[e]) + (nt > kGroup ? sum[e] : 0.0f);
                } else {
                    tmem_wait_ld();
                }
            }
            if (tid < P.D) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int r = r0 + e;
                    if (r >= nrows) break;
                    const float a = scratch.row[r], y = a == 0.0f ? 0.0f : o[e] * a;
                    const int64_t to = scratch.to[r];
                    if (to < 0) continue;
                    if (part)
                        P.part_o[to + tid] = y;
                    else if constexpr (WIDE)
                        static_cast<float *>(P.out)[to + tid] = y;
                    else
                        static_cast<__nv_bfloat16 *>(P.out)[to + tid] = __float2bfloat16_rn(y);
                }
            }
        }
        // (the next segment meets at least once before it writes where slower warps may still read)
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.pipe.desc_empty[desc.slot]);
        if (!more) return;
        desc = then;
        buf ^= 1;
    }
}

// ---------------------------------------------------------------- the kernel

template <int RT, bool PREFIX, bool WIDE>
__global__ void __launch_bounds__(kThreads, kPerSM)
    spec_attend8_round_kernel(const __grid_constant__ AttendParams P, const CacheMap M,
                             const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ __align__(1024) unsigned char ring_mem[];  // tiles, queries, weights, the rest
    unsigned char *q_tile = ring_mem + stages<RT, WIDE>() * kTile;
    unsigned char *p_tile = q_tile + q_bytes<WIDE>(RT);
    Shared<RT, WIDE> &sh = *reinterpret_cast<Shared<RT, WIDE> *>(p_tile + p_bytes<WIDE>(RT));
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
    constexpr int kColumns = RT == 64 || WIDE ? 256 : 128;  // 3 RT a set, and the sums' RT, as a power of two

    if (warp == 5) tmem_alloc(&sh.tmem, kColumns);
    if (threadIdx.x == 0) {
        init_pipe(sh.pipe, 1, 5);  // values: the products; segments: four softmax warps and the issuing one
        for (int i = 0; i < 2; ++i) mbar_init(&sh.s_full[i], 1);
        mbar_init(&sh.q_full, 128);
        mbar_init(&sh.p_full, 128);
        mbar_init(&sh.o_done, 1);
        mbar_init(&sh.drain, 1);
        sh.skip = 0;
        fence_mbar_init();
        prefetch_map(&kmap);
        prefetch_map(&vmap);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    begin_kernel<PREFIX>(P);

    if (warp < 4) {
        softmax_role<RT, PREFIX, WIDE>(P, sh, ring_mem, q_tile, p_tile);
    } else if (warp == 4) {
        load_role<PREFIX>(P, M, &kmap, &vmap, sh.pipe, ring_mem, blockIdx.x, lane);
    } else {
        if constexpr (!PREFIX) keep_books<kKT>(P, lane);
        mma_role<RT, WIDE>(P, sh, ring_mem, q_tile, p_tile);
        // nothing this warp issued is in flight when the CTA ends
        if (elect_lane()) mma_commit(&sh.drain);
        __syncwarp();
#pragma unroll 1
        for (int t = 0; t < kTries && !mbar_try_wait_sleep(&sh.drain, 0, kHintNs); ++t) {
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 5) tmem_free(sh.tmem, kColumns);
    end_kernel<PREFIX>(P);
    if (threadIdx.x == 0) P.err[(PREFIX ? P.own_workers : 0) + blockIdx.x] = sh.pipe.abort;
}

}  // namespace round8
}  // namespace spec
