// Attention of few rows on the tensor cores (bf16, head sizes that are multiples of 16 up to 128): a
// verification round, single tokens. The bytes of the keys and values are the bound, and between a tile's
// arrival and its release stands a chain of products, softmax and products that must stay short.
//
// The products are taken the other way round, positions and output columns along the 128 lanes, the
// item's rows (RT = 32 or 64, in steps of 16) along the columns:
//   S^T = K Q^T     128 positions x rows: every thread of the warpgroup has one position, all rows, so
//                   that the exponentials of a tile are spread over 128 threads however few rows there are
//   O^T += V^T P^T  output columns x rows: P^T, a position's weights side by side, goes to shared memory
//                   as the threads hold it, and V is read along its columns
// and the matrix instructions' time follows the rows that there are. S has two buffers, so that the next
// tile's scores are there when this tile's weights are done.
// A row's maximum is a reference shared by the 128 threads: set from the item's first tile, and anew when
// some score lies more than 2^8 above it (the threads agree on that each tile); else no maximum is
// taken at all. Each thread sums its own weights, and the sums meet at the end. The next segment's queries
// are brought in, and their first scores taken, while a segment ends.
//
// Two CTAs per SM, each a worker: while one begins or ends an item the other keeps copies in flight.
// Warps: 0-3 softmax, 4 loads tiles, 5 keeps the books, then issues the matrix instructions.
//
// Measured: 16 requests of 4 to 65 thousand tokens (2.0 GB of keys and values) 312 to 323 us, 0.93 to 0.96
// of the measured copy rate; 64 requests of up to 16 thousand under a 1024-token window with 4 sinks (0.27 GB,
// items of 9 tiles) 82 us, where items' beginnings and ends (some 4 us each, mostly the chain from queries to first
// weights and from sums to rows) are as long as their tiles. With rows along the lanes, as in the pair
// kernel, the first took 567 us and the second 227.
#pragma once

#include "spec_attend_tiles.cuh"

namespace spec {
namespace round_ {

using namespace tiles;

constexpr int kThreads = 192, kPerSM = 2, kStages = 6;
constexpr float kSlack = 8.0f;  // log2 growth of the maximum that the output and the sums absorb

template <int RT>
struct Shared {
    Pipe<kStages> pipe;
    uint64_t q_full, s_full[2], p_full, o_done, agree, drain;
    uint32_t found[2][4];  // per warp: a score beyond the reference (1), a value that is not finite (2)
    uint32_t skip;         // the warpgroup has done this tile's second product itself
    uint32_t tmem;
    // of this segment's rows and the next one's, in turn
    int pos[2][RT];                 // positions (-1: none)
    alignas(16) float nref[2][RT];  // minus the reference, scaled; kNoRef before there is one (read four at a time)
};
// What the row operations of a warpgroup need now and then, in the weights' memory while that is unused.
template <int RT>
struct Scratch {
    float warp[4][RT];
    float row[RT];
};
// A reference that every finite score exceeds and that leaves -inf alone.
constexpr float kNoRef = 3e38f;

__host__ __device__ constexpr int q_bytes(int D, int RT) { return blocks(D) * RT * 128; }
__host__ __device__ constexpr int p_bytes(int RT) { return kKT * RT * 2; }
template <int RT>
__host__ constexpr int stages(int D) {
    // 228 KB of shared memory, 1 KB of it taken per CTA
    const int n = (228 * 1024 / kPerSM - 1024 - static_cast<int>(sizeof(Shared<RT>)) - q_bytes(D, RT) - p_bytes(RT)) /
                  tile_bytes(D);
    return n < kStages ? n : kStages;
}
template <int RT>
__host__ constexpr int smem_bytes(int D) {
    return stages<RT>(D) * tile_bytes(D) + q_bytes(D, RT) + p_bytes(RT) + static_cast<int>(sizeof(Shared<RT>));
}
static_assert(stages<32>(128) >= 3 && stages<64>(128) >= 2, "a tile of keys and one of values at least");
static_assert(sizeof(Scratch<64>) <= p_bytes(64) && sizeof(Scratch<32>) <= p_bytes(32), "fits the weights' memory");

// ---------------------------------------------------------------- matrix instructions (one thread)

template <int RT>
__device__ __forceinline__ void mma_role(const AttendParams &P, Shared<RT> &sh, unsigned char *ring_mem,
                                         unsigned char *q_tile, unsigned char *p_tile, int n_stages) {
    const int tb = tile_bytes(P.D);
    int32_t *ab = &sh.pipe.abort;
    const uint32_t s_col = sh.tmem, o_col = sh.tmem + 2 * RT;
    // with up to 64 columns the output's lanes 64.. repeat the first 64 (unused)
    const uint64_t q_op = smem_operand(smem_addr(q_tile), 16), k_op = smem_operand(smem_addr(ring_mem), 16),
                   v_op = smem_operand(smem_addr(ring_mem), blocks(P.D) == 2 ? kBlock : 0),
                   p_op = RT == 64 ? smem_operand(smem_addr(p_tile), 16) : smem_operand64(smem_addr(p_tile));
    const int steps = P.D / 16;
    Ring ring = {0, n_stages, 0}, desc = {0, 2, 0};
    uint32_t q_phase = 0, p_phase = 0;
    for (;;) {
        if (!wait_one(ab, &sh.pipe.desc_full[desc.slot], desc.phase)) return;
        const Segment &s = sh.pipe.desc[desc.slot];
        const int nrows = s.nrows, nt = s.ntile;
        if (nrows == 0) return;
        if (nt > 0) {
            const int n16 = (nrows + 15) & ~15;
            const uint32_t qk_shape = mma_shape(n16, false, false), pv_shape = mma_shape(n16, true, true);
            if (!wait_one(ab, &sh.q_full, q_phase)) return;
            q_phase ^= 1u;
            // step t: tile t's product, and tile t + 1's scores (step -1: the first scores alone). The scores
            // go first if their keys are there.
#pragma unroll 1
            for (int t = -1; t < nt; ++t) {
                const bool more = t + 1 < nt;
                const Ring v = ring;  // this tile's values; the next tile's keys follow them
                if (t >= 0) ring.step();
                const bool ahead = more && mbar_try_wait(&sh.pipe.full[ring.slot], ring.phase);
#pragma unroll 1
                for (int part = 0; part < 2; ++part) {
                    if (part == (ahead ? 0 : 1)) {
                        if (!more) continue;
                        if (!ahead && !wait_one(ab, &sh.pipe.full[ring.slot], ring.phase)) return;
                        tc_fence_after();
                        const int b = (t + 1) & 1;  // S^T = K Q^T
                        const uint64_t k = operand_at(k_op, ring.slot * tb);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint32_t in = (i & 3) * 32;
                            if (i < steps)
                                mma_ss(s_col + b * RT, operand_at(k, (i >> 2) * kBlock + in),
                                       operand_at(q_op, (i >> 2) * (RT * 128) + in), qk_shape, i > 0);
                        }
                        mma_commit(&sh.s_full[b]);
                        mma_commit(&sh.pipe.empty[ring.slot]);
                    } else if (t >= 0) {
                        if (!wait_one(ab, &sh.pipe.full[v.slot], v.phase)) return;
                        if (!wait_one(ab, &sh.p_full, p_phase)) return;
                        p_phase ^= 1u;
                        tc_fence_after();
                        if (!*reinterpret_cast<volatile uint32_t *>(&sh.skip)) {  // O^T += V^T P^T
                            const uint64_t values = operand_at(v_op, v.slot * tb);
                            const int n = tile_keys(s.keys, tile_begin<kKT>(s.keys, s.tile + t));
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                if (i * 16 < n)
                                    mma_ss(o_col, operand_at(values, i * 2048), operand_at(p_op, i * 16 * RT * 2), pv_shape,
                                           t > 0 || i > 0);
                        }
                        mma_commit(&sh.o_done);
                        mma_commit(&sh.pipe.empty[v.slot]);
                    }
                }
                if (more) ring.step();
            }
        }
        mbar_arrive(&sh.pipe.desc_empty[desc.slot]);
        desc.step();
    }
}

// ---------------------------------------------------------------- softmax (one position per thread)

// The four warps meet; each leaves a word, and all get the words' union (-1: a wait gave up).
__device__ __forceinline__ int meet(int32_t *abort, uint64_t *bar, uint32_t (*found)[4], uint32_t phase, uint32_t mine) {
    const int warp = threadIdx.x / kWarp;
    volatile uint32_t *words = found[phase];
    __syncwarp();
    if (threadIdx.x % kWarp == 0) {
        words[warp] = mine;
        mbar_arrive(bar);
    }
    if (!wait_warp(abort, bar, phase)) return -1;
    return static_cast<int>(words[0] | words[1] | words[2] | words[3]);
}
// Out of line for the meetings that come once per item.
__device__ __noinline__ int meet_far(int32_t *abort, uint64_t *bar, uint32_t (*found)[4], uint32_t phase, uint32_t mine) {
    return meet(abort, bar, found, phase, mine);
}
template <int RT, bool FAR = true>
__device__ __forceinline__ bool agree(Shared<RT> &sh, uint32_t &phase, uint32_t mine, uint32_t &all) {
    const int r = FAR ? meet_far(&sh.pipe.abort, &sh.agree, sh.found, phase, mine)
                      : meet(&sh.pipe.abort, &sh.agree, sh.found, phase, mine);
    phase ^= 1u;
    all = static_cast<uint32_t>(r);
    return r >= 0;
}

// The second product of a tile with values that are not finite, on the fp32 units: thread d has output
// column d, the weights lie in shared memory, O is complete up to the tile before.
template <int RT>
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
                    const int piece = RT == 64 ? (r >> 3) ^ (k & 7) : (r >> 3) ^ ((k >> 1) & 3);
                    const float w = __bfloat162float(
                        *reinterpret_cast<const __nv_bfloat16 *>(p_tile + k * RT * 2 + piece * 16 + (r & 7) * 2));
                    o[e] = fmaf(w, v, o[e]);
                }
            }
        }
        uint32_t ow[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) ow[e] = __float_as_uint(o[e]);
        __syncwarp();
        tmem_st16(o_addr + r0, ow);
        tmem_wait_st();
    }
}

template <int RT, bool PREFIX>
__device__ __forceinline__ void softmax_role(const AttendParams &P, Shared<RT> &sh, unsigned char *ring_mem,
                                             unsigned char *q_tile, unsigned char *p_tile, int n_stages) {
    const int tid = threadIdx.x, warp = tid / kWarp, lane = tid % kWarp;
    const int tb = tile_bytes(P.D);
    int32_t *ab = &sh.pipe.abort;
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t s_addr = sh.tmem + lanes, o_addr = s_addr + 2 * RT;
    Scratch<RT> &scratch = *reinterpret_cast<Scratch<RT> *>(p_tile);
    Ring ring = {0, n_stages, 0}, desc = {0, 2, 0};
    uint32_t s_phases = 0, o_phase = 0, a_phase = 0, word = 0;
    int buf = 0;
    // Brings a segment's queries: 128 / RT threads each row's (rows up to a multiple of 16: zeros), and its
    // position.
    auto bring = [&](const Segment &s, int to) {
        constexpr int kPer = 128 / RT;
        const int r = tid / kPer, pr = s.row0 + r, j = P.by_group(pr), g = pr - j * P.G;
        const int t = s.t0 + j, h = s.head * P.G + g;
        if (r < ((s.nrows + 15) & ~15)) {
            const bool have = r < s.nrows && SPEC_IN(t, P.T, DBG_ATTEND);
            const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(P.q) + t * P.q_stride +
                                                               static_cast<int64_t>(h) * P.D);
#pragma unroll 4
            for (int c = tid % kPer; c < P.D / 8; c += kPer)
                *reinterpret_cast<uint4 *>(q_tile + (c >> 3) * (RT * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
                    have ? src[c] : make_uint4(0u, 0u, 0u, 0u);
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
            if (!wait_warp(ab, &sh.pipe.desc_full[0], 0)) return;
            if (s.nrows == 0) return;
            bring(s, 0);
            if (!agree(sh, a_phase, 0u, word)) return;
            first_segment = false;
        }
        const int nrows = s.nrows, nt = s.ntile, n16 = (nrows + 15) & ~15;
        const int *pos = sh.pos[buf];
        float *nref = sh.nref[buf];

        float2 l[RT / 2];  // this thread's share of the rows' sums
#pragma unroll
        for (int e = 0; e < RT / 2; ++e) l[e] = make_float2(0.0f, 0.0f);
#pragma unroll 1
        for (int i = 0; i < nt; ++i) {
            const int b = i & 1;
            const int x0 = tile_begin<kKT>(s.keys, s.tile + i), n = tile_keys(s.keys, x0), x = x0 + tid;
            const bool edge = edge_tile(P, s, x0);
            const int v_slot = ring.slot + 1 == ring.n ? 0 : ring.slot + 1;
            unsigned char *v_tile = ring_mem + v_slot * tb;
            uint32_t mine = 0u;
            // A wait by parity tells this use of a slot from the one before only when that one is known to have
            // arrived. In rings of three slots or more it is: it held keys whose scores, or values whose product,
            // have been waited for. In a ring of two (64 rows, more than 64 columns) it held the values of the
            // tile before, which only that tile's product says.
            bool rested = i == 0;
            auto rest = [&]() -> bool {
                if (rested) return true;
                rested = true;
                if (!wait_warp(ab, &sh.o_done, o_phase)) return false;
                o_phase ^= 1u;
                tc_fence_after();
                return true;
            };
            if (edge) {
                if (ring.n == 2 && !rest()) return;
                if (!wait_warp(ab, &sh.pipe.full[v_slot], ring.slot + 1 == ring.n ? ring.phase ^ 1u : ring.phase)) return;
                if (__any_sync(0xffffffffu, clean_values(P, s, v_tile, x0, n, tid))) mine = 2u;
                fence_proxy_async_smem();
            }
            if (!wait_warp(ab, &sh.s_full[b], s_phases >> b & 1u)) return;
            s_phases ^= 1u << b;
            tc_fence_after();
            // this position's scores with 16 rows from row e on
            auto read = [&](float *z, int e) {
                tmem_ld16(z, s_addr + b * RT + e);
                tmem_wait_ld();
                if (edge) {
                    const bool in = x >= s.keys.from && x < s.keys.hi, sink = x < P.n_sink;
                    const int back = P.window > 0 ? P.window : INT_MAX;
#pragma unroll
                    for (int y = 0; y < 16; ++y) {
                        const int p = pos[e + y];
                        if (!(in && x <= p && (sink || p - x < back))) z[y] = -INFINITY;
                    }
                }
            };
            // 32 rows' scores stay in registers; 64 rows' would not, beside their sums, and are read anew
            constexpr bool kHeld = RT == 32;
            float held[kHeld ? RT : 16];
            if constexpr (kHeld) {
#pragma unroll
                for (int e = 0; e < RT; e += 16)
                    if (e < nrows) read(held + e, e);
            }
            auto scores = [&](int e) -> float * {
                if constexpr (kHeld) return held + e;
                read(held, e);
                return held;
            };
            const float2 sc = make_float2(P.scale_log2, P.scale_log2);
            // four scores against their references
            auto against = [&](const float *z, int e, float2 &a, float2 &c) {
                const float4 rf = *reinterpret_cast<const float4 *>(nref + e);
                a = fma2(make_float2(z[0], z[1]), sc, make_float2(rf.x, rf.y));
                c = fma2(make_float2(z[2], z[3]), sc, make_float2(rf.z, rf.w));
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
                mine |= __any_sync(0xffffffffu, top > kSlack) ? 1u : 0u;
                if (!agree<RT, false>(sh, a_phase, mine, word)) return;
            } else {
                word = 1u;  // the first references (the values' flag comes with their meetings)
            }
            if (!rest()) return;  // the product before this tile: the weights' memory is free, O at rest
            if (word & 1u) {
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
                if (!agree(sh, a_phase, 0u, word)) return;
                if (tid < n16) {
                    const float v = fmaxf(fmaxf(scratch.warp[0][tid], scratch.warp[1][tid]),
                                          fmaxf(scratch.warp[2][tid], scratch.warp[3][tid]));
                    const float old = nref[tid], nw = -v * P.scale_log2;
                    const bool grow = v != -INFINITY && (old == kNoRef || nw < old);
                    // a row without weights so far has nothing to rescale
                    scratch.row[tid] = grow && old != kNoRef ? ex2(nw - old) : 1.0f;
                    if (grow) nref[tid] = nw;
                }
                if (!agree(sh, a_phase, mine & 2u, word)) return;
                if (i > 0) {
#pragma unroll
                    for (int e = 0; e < RT; e += 2)
                        if ((e & ~15) < nrows) {
                            l[e / 2].x *= scratch.row[e];
                            l[e / 2].y *= scratch.row[e + 1];
                        }
#pragma unroll 1
                    for (int r0 = 0; r0 < nrows; r0 += 16) {
                        float o[16];
                        uint32_t ow[16];
                        tmem_ld16(o, o_addr + r0);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) ow[e] = __float_as_uint(o[e] * scratch.row[r0 + e]);
                        tmem_st16(o_addr + r0, ow);
                    }
                    tmem_wait_st();
                    const uint32_t keep = word;
                    if (!agree(sh, a_phase, 0u, word)) return;  // the scratch has been read
                    word = keep;
                }
            }
            const bool skip = (word & 2u) != 0;
            unsigned char *prow = p_tile + tid * (RT * 2);
#pragma unroll
            for (int e = 0; e < RT; e += 16)
                if (e < nrows) {
                    const float *z = scores(e);
#pragma unroll
                    for (int y = 0; y < 16; y += 8) {
                        uint32_t pw[4];
#pragma unroll
                        for (int u = y; u < y + 8; u += 4) {
                            float2 a, c;
                            against(z + u, e + u, a, c);
                            a.x = ex2(a.x);
                            a.y = ex2(a.y);
                            c.x = ex2(c.x);
                            c.y = ex2(c.y);
                            l[(e + u) / 2] = add2(l[(e + u) / 2], a);
                            l[(e + u) / 2 + 1] = add2(l[(e + u) / 2 + 1], c);
                            pw[(u - y) / 2] = pack_bf16(a.x, a.y);
                            pw[(u - y) / 2 + 1] = pack_bf16(c.x, c.y);
                        }
                        const int piece = RT == 64 ? ((e + y) >> 3) ^ (tid & 7) : ((e + y) >> 3) ^ ((tid >> 1) & 3);
                        *reinterpret_cast<uint4 *>(prow + piece * 16) = make_uint4(pw[0], pw[1], pw[2], pw[3]);
                    }
                }
            if (skip) {
                if (!agree(sh, a_phase, 0u, word)) return;  // all weights are there
                mixed_tile<RT>(P, pos, o_addr, v_tile, p_tile, s.keys, x0, n, nrows, tid, i == 0);
            }
            if (tid == 0) *reinterpret_cast<volatile uint32_t *>(&sh.skip) = skip;
            fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive(&sh.p_full);
            ring.step();
            ring.step();
        }
        // the next segment's queries; this one's scores have all been taken
        Ring then = desc;
        then.step();
        if (!wait_warp(ab, &sh.pipe.desc_full[then.slot], then.phase)) return;
        const bool more = sh.pipe.desc[then.slot].nrows > 0;
        if (more) bring(sh.pipe.desc[then.slot], buf ^ 1);
        if (nt > 0) {
            if (!wait_warp(ab, &sh.o_done, o_phase)) return;
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
        if (!agree(sh, a_phase, 0u, word)) return;
        if (tid < nrows) {
            float sum = scratch.warp[0][tid] + scratch.warp[1][tid] + scratch.warp[2][tid] + scratch.warp[3][tid];
            if (pos[tid] < 0) sum = 0.0f;  // padding
            const bool none = sum == 0.0f;
            const float m = none ? -INFINITY : -nref[tid];
            if (s.part >= 0) {
                // a sum that is not a number must reach the joined row, whatever the other parts' maxima
                if (SPEC_IN(s.part + tid, P.part_rows, DBG_ATTEND))
                    P.part_ml[s.part + tid] = make_float2(isnan(sum) ? INFINITY : m, sum);
                scratch.row[tid] = none ? 0.0f : 1.0f;
            } else {
                const int j = P.by_group(s.row0 + tid), g = s.row0 + tid - j * P.G;
                if (P.lse && SPEC_IN(s.t0 + j, P.T, DBG_ATTEND))
                    P.lse[static_cast<int64_t>(s.t0 + j) * P.Hq + s.head * P.G + g] =
                        none ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
                scratch.row[tid] = none ? 0.0f : 1.0f / sum;
            }
        }
        if (!agree(sh, a_phase, 0u, word)) return;
#pragma unroll 1
        for (int r0 = 0; r0 < nrows; r0 += 4) {
            float o[4];
            __syncwarp();
            if (nt > 0) {
                tmem_ld4(o, o_addr + r0);
                tmem_wait_ld();
            }
            if (tid < P.D) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = r0 + e;
                    if (r >= nrows) break;
                    const float a = scratch.row[r], y = a == 0.0f ? 0.0f : o[e] * a;
                    if (s.part >= 0) {
                        if (SPEC_IN(s.part + r, P.part_rows, DBG_ATTEND)) P.part_o[(s.part + r) * P.D + tid] = y;
                    } else {
                        const int j = P.by_group(s.row0 + r), g = s.row0 + r - j * P.G;
                        if (SPEC_IN(s.t0 + j, P.T, DBG_ATTEND))
                            static_cast<__nv_bfloat16 *>(P.out)[(s.t0 + j) * P.out_stride + (s.head * P.G + g) * P.D + tid] =
                                __float2bfloat16_rn(y);
                    }
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

template <int RT, bool PREFIX>
__global__ void __launch_bounds__(kThreads, kPerSM)
    spec_attend_round_kernel(const __grid_constant__ AttendParams P, const CacheMap M,
                             const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                             const int n_stages) {
    extern __shared__ __align__(1024) unsigned char ring_mem[];  // tiles, queries, weights, the rest
    unsigned char *q_tile = ring_mem + n_stages * tile_bytes(P.D);
    unsigned char *p_tile = q_tile + q_bytes(P.D, RT);
    Shared<RT> &sh = *reinterpret_cast<Shared<RT> *>(p_tile + p_bytes(RT));
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
    constexpr int kColumns = RT == 64 ? 256 : 128;  // 3 RT, as a power of two

    if (warp == 5) tmem_alloc(&sh.tmem, kColumns);
    if (threadIdx.x == 0) {
        for (int i = 0; i < n_stages; ++i) {
            mbar_init(&sh.pipe.full[i], 1);
            mbar_init(&sh.pipe.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.pipe.desc_full[i], 1);
            mbar_init(&sh.pipe.desc_empty[i], 5);  // four softmax warps and the issuing thread
            mbar_init(&sh.s_full[i], 1);
        }
        mbar_init(&sh.q_full, 128);
        mbar_init(&sh.p_full, 128);
        mbar_init(&sh.o_done, 1);
        mbar_init(&sh.agree, 4);
        mbar_init(&sh.drain, 1);
        sh.skip = 0;
        sh.pipe.abort = 0;
        fence_mbar_init();
        prefetch_map(&kmap);
        prefetch_map(&vmap);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    begin_kernel<PREFIX>(P);

    if (warp < 4) {
        softmax_role<RT, PREFIX>(P, sh, ring_mem, q_tile, p_tile, n_stages);
    } else if (warp == 4) {
        load_role<PREFIX>(P, M, &kmap, &vmap, sh.pipe, ring_mem, n_stages, blockIdx.x, lane);
    } else {
        if constexpr (!PREFIX) keep_books<kKT>(P, lane);
        if (lane == 0) {
            mma_role<RT>(P, sh, ring_mem, q_tile, p_tile, n_stages);
            // nothing this thread issued is in flight when the CTA ends
            mma_commit(&sh.drain);
#pragma unroll 1
            for (int t = 0; t < kTries && !mbar_try_wait_sleep(&sh.drain, 0, kHintNs); ++t) {
            }
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

}  // namespace round_
}  // namespace spec
