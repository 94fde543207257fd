// Attention on the fp32 units: the kernel for fp32, for the bf16 shapes the tensor-core kernel does
// not take, and, over the cache in 8 bits, for the shapes that its tensor-core kernels do not take. One CTA of four warps per worker; a warp owns up to four of the item's 16 packed rows.
//
// Per tile of 32 keys: lane x forms the scores of key x with the warp's rows (keys padded by 16 bytes
// a row in shared memory, so that eight lanes' 16-byte reads cover all banks; queries are broadcast),
// the running maximum and sum follow by shuffles, and for the second product the lanes turn to the
// columns of the output, four (or eight, beyond 128) each, with the weights broadcast. The next tile is
// copied in while this one is used (fp32: by asynchronous copies; bf16 values pass through registers on their
// way to fp32, and each lane waits for its loads; 8-bit elements wait in registers while the tile before is used: 64 fp32
// requests of up to 4096 positions over them 246 us, 354 with loads that are waited for).
//
// Bound by shared memory, whose reads take twice the arithmetic's time (each warp reads every key and
// value): 256 requests of 4 rows and 16 query heads of 128 under a 500-token window (0.55 GB) 248 us, a
// third of the measured copy rate. Items have 16 rows however many a request has, so that a prompt of 2000
// rows (16 query heads of 128) reads its keys 500 times over: 888 us in fp32, 18 TFLOP/s. In bf16 with heads
// of 256, 16 requests of 4 rows after 16000 positions (1 GB) take 2.48 ms, 0.06 of the copy rate, and a prompt
// of 1000 rows 1.06 ms: one CTA of four warps an SM, and loads that are waited for. Keys split over the warps,
// with all 16 rows in each, halve the reads but take 255 registers a thread and with them the warps that hide
// the latency: 290 us.
#pragma once

#include <cuda_bf16.h>

#include "spec_attend_plan.cuh"
#include "spec_fp8.cuh"

namespace spec {
namespace fma {

constexpr int kRTLog2 = 4, kRT = 1 << kRTLog2, kKT = 32, kWarps = 4, kThreads = kWarps * kWarp, kRows = kRT / kWarps;

// Shared memory: queries, two tiles of keys and values, the weights.
__host__ __device__ constexpr int smem_floats(int D) {
    return kRT * D + 2 * kKT * (D + 4) + 2 * kKT * D + kRT * kKT;
}
// CTAs an SM holds (228 KB of shared memory, 1 KB of it taken per CTA; four CTAs are enough).
__host__ constexpr int ctas_per_sm(int D) {
    const int n = (228 * 1024) / (smem_floats(D) * 4 + 1024);
    return n < 4 ? n : 4;
}

__device__ __forceinline__ void copy16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 16 bytes of a head into shared memory as fp32.
__device__ __forceinline__ void bring(float *dst, const float *src) { copy16(dst, src); }
__device__ __forceinline__ void bring(float *dst, const __nv_bfloat16 *src) {
    const uint4 x = *reinterpret_cast<const uint4 *>(src);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        *reinterpret_cast<float2 *>(dst + 2 * j) =
            make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
}

__device__ __forceinline__ void store4(float *dst, float4 v) { *reinterpret_cast<float4 *>(dst) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16 *dst, float4 v) {
    __nv_bfloat162 p[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
    *reinterpret_cast<uint2 *>(dst) = *reinterpret_cast<const uint2 *>(p);
}

// One warp's rows: their positions, softmax state and outputs (columns c*128 + 4*lane ..).
template <int NC>
struct Rows {
    int pos[kRows];
    float m[kRows], l[kRows];
    float4 o[kRows][NC];
};

// One tile for NR of the warp's rows. full: every row sees every key of the tile.
template <int NR, int NC>
__device__ __forceinline__ void tile_step(const AttendParams &P, Rows<NC> &R, const float *sQ, const float *sK,
                                          const float *sV, float *sP, int x0, const KeyTiles &keys, int warp, int lane) {
    const int D = P.D;
    float s[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) s[r] = 0.0f;
    const float *kp = sK + lane * (D + 4);
    for (int d = 0; d < D; d += 4) {
        const float4 k = *reinterpret_cast<const float4 *>(kp + d);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const float4 q = *reinterpret_cast<const float4 *>(sQ + (r * kWarps + warp) * D + d);
            s[r] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, s[r]))));
        }
    }
    const int x = x0 + lane;
    unsigned seen[NR];
    unsigned all = 0xffffffffu;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int p = R.pos[r];
        const bool vis = x >= keys.from && x < keys.hi && x <= p && (P.window == 0 || x > p - P.window || x < P.n_sink);
        seen[r] = __ballot_sync(0xffffffffu, vis);
        all &= seen[r];
        const float z = vis ? s[r] * P.scale_log2 : -INFINITY;
        const float m = fmaxf(R.m[r], warp_max(z));
        // a row that has seen nothing so far keeps the reference 0: its weights are 2^-inf = 0
        const float ref = m == -INFINITY ? 0.0f : m;
        const float w = ex2(z - ref);
        const float a = R.m[r] == -INFINITY ? 0.0f : ex2(R.m[r] - ref);
        R.m[r] = m;
        R.l[r] = R.l[r] * a + warp_sum(w);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            R.o[r][c].x *= a;
            R.o[r][c].y *= a;
            R.o[r][c].z *= a;
            R.o[r][c].w *= a;
        }
        sP[(r * kWarps + warp) * kKT + lane] = w;
    }
    __syncwarp();
    const bool full = all == 0xffffffffu;
#pragma unroll 4
    for (int k = 0; k < kKT; ++k) {
        float4 v[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (c * 128 + 4 * lane < D) v[c] = *reinterpret_cast<const float4 *>(sV + k * D + c * 128 + 4 * lane);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            // a value at a position the row does not see takes no part, whatever it is
            if (full || (seen[r] >> k & 1u)) {
                const float w = sP[(r * kWarps + warp) * kKT + k];
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    R.o[r][c].x = fmaf(w, v[c].x, R.o[r][c].x);
                    R.o[r][c].y = fmaf(w, v[c].y, R.o[r][c].y);
                    R.o[r][c].z = fmaf(w, v[c].z, R.o[r][c].z);
                    R.o[r][c].w = fmaf(w, v[c].w, R.o[r][c].w);
                }
            }
        }
    }
    __syncwarp();
}

// The warps' share of copying one tile in: eight keys a warp.
template <typename C>
__device__ __forceinline__ void load_tile(const AttendParams &P, const Segment &s, float *sK, float *sV, int x0, int warp,
                                          int lane) {
    constexpr int V = 16 / sizeof(C);
    const int D = P.D, per = D / V;
    int64_t off = -1;
    const int x = x0 + warp * 8 + lane;
    if (lane < 8 && item_sees(P, s.keys, x)) {
        const int32_t *table = s.req < 0 ? P.shared_table : P.block_table + static_cast<int64_t>(s.req) * P.max_blocks;
        off = slot_offset(P, table, x);
        if (off >= 0) off += static_cast<int64_t>(s.head) * P.head_stride;
    }
    const C *kc = static_cast<const C *>(P.k_cache), *vc = static_cast<const C *>(P.v_cache);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t o = __shfl_sync(0xffffffffu, off, j);
        if (o < 0) continue;  // seen by no row (or its request is in error): never used
        const int key = warp * 8 + j;
        for (int c = lane; c < per; c += kWarp) {
            if (!SPEC_IN(o + c * V + V - 1, cache_extent(P), DBG_CACHE)) continue;
            bring(sK + key * (D + 4) + c * V, kc + o + c * V);
            bring(sV + key * D + c * V, vc + o + c * V);
        }
    }
}

// The same of a cache in 8 bits, in two steps: the warp's eight keys' elements and scales on their way into registers
// while the tile before is used, then into shared memory as fp32. A lane has the same 16 elements of every 32 / per-th key
// (per = D / 16 pieces a key; lanes left over have none).
template <int NC>
struct Tile8 {
    static constexpr int kPieces = 2 * NC;  // of a lane: 8 keys, 32 / per >= 4 / NC of them at a time
    uint4 k[kPieces], v[kPieces];
    float ks, vs;  // lane j < 8: key j's scales
    unsigned on;   // bit j: key j is used

    __device__ __forceinline__ void fetch(const AttendParams &P, const Segment &s, int x0, int warp, int lane) {
        const int per = P.D / 16, at_once = kWarp / per, j0 = lane / per, c = lane - j0 * per;
        const int x = x0 + warp * 8 + lane;
        int64_t off = -1;
        ks = vs = 1.0f;
        if (lane < 8 && item_sees(P, s.keys, x)) {
            const int32_t *table = s.req < 0 ? P.shared_table : P.block_table + static_cast<int64_t>(s.req) * P.max_blocks;
            off = slot_offset(P, table, x);
            if (off >= 0) {
                off += static_cast<int64_t>(s.head) * P.head_stride;
                const int64_t at = static_cast<int64_t>(table[P.by_page(x)]) * P.Hkv + s.head;
                ks = P.k_scale[at];
                vs = P.v_scale[at];
            }
        }
        on = __ballot_sync(0xffffffffu, off >= 0);
        const unsigned char *kc = static_cast<const unsigned char *>(P.k_cache), *vc = static_cast<const unsigned char *>(P.v_cache);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int j = j0 + i * at_once;
            const int64_t o = __shfl_sync(0xffffffffu, off, j & 31);
            if (j0 < at_once && j < 8 && o >= 0 && SPEC_IN(o + c * 16 + 15, cache_extent(P), DBG_CACHE)) {
                k[i] = *reinterpret_cast<const uint4 *>(kc + o + c * 16);
                v[i] = *reinterpret_cast<const uint4 *>(vc + o + c * 16);
            }
        }
    }
    __device__ __forceinline__ void put(const AttendParams &P, float *sK, float *sV, int warp, int lane) const {
        const int D = P.D, per = D / 16, at_once = kWarp / per, j0 = lane / per, c = lane - j0 * per;
        auto widen = [](float *dst, const uint4 &x, float by) {
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 f = e4m3_to_float4(w[e]);
                *reinterpret_cast<float4 *>(dst + 4 * e) = make_float4(f.x * by, f.y * by, f.z * by, f.w * by);
            }
        };
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int j = j0 + i * at_once, key = warp * 8 + j;
            const float kb = __shfl_sync(0xffffffffu, ks, j & 31), vb = __shfl_sync(0xffffffffu, vs, j & 31);
            if (j0 < at_once && j < 8 && (on >> j & 1u)) {  // (others are seen by no row, or their request is in error)
                widen(sK + key * (D + 4) + c * 16, k[i], kb);
                widen(sV + key * D + c * 16, v[i], vb);
            }
        }
    }
};

// E: the type of the rows; C: the cache's.
template <typename E, typename C, int NC, bool PREFIX>
__global__ void __launch_bounds__(kThreads) spec_attend_fma_kernel(const AttendParams P) {
    extern __shared__ float4 smem4[];
    float *sQ = reinterpret_cast<float *>(smem4);
    const int D = P.D;
    float *sK = sQ + kRT * D, *sV = sK + 2 * kKT * (D + 4), *sP = sV + 2 * kKT * D;
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
    begin_kernel<PREFIX>(P);

    Walker<kKT, PREFIX> walk;
    walk.start(P, blockIdx.x, lane);
    Segment s;
    while (walk.next(P, s, lane)) {
        constexpr int V = 16 / sizeof(E);
        const int per = D / V;
        __syncthreads();  // the last segment's queries and tiles have been used
        for (int c = threadIdx.x; c < s.nrows * per; c += kThreads) {
            const int r = c / per, d = (c - r * per) * V;
            const int j = P.by_group(s.row0 + r), g = s.row0 + r - j * P.G;
            if (SPEC_IN(s.t0 + j, P.T, DBG_ATTEND))
                bring(sQ + r * D + d, static_cast<const E *>(P.q) + (s.t0 + j) * P.q_stride +
                                          static_cast<int64_t>(s.head * P.G + g) * D + d);
        }
        // rows warp, warp + 4, ..: a warp has nr of them
        const int nr = s.nrows > warp ? (s.nrows - warp + kWarps - 1) / kWarps : 0;
        Rows<NC> R;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            R.m[r] = -INFINITY;
            R.l[r] = 0.0f;
            R.pos[r] = -1;
#pragma unroll
            for (int c = 0; c < NC; ++c) R.o[r][c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (r < nr) {
                const int j = P.by_group(s.row0 + r * kWarps + warp);
                if constexpr (PREFIX) {
                    const ReqRows q = load_request(P, find_request(P.row_off, P.B, P.T, j, lane));
                    R.pos[r] = j >= q.r0 && j < q.r0 + q.n ? q.kv - q.n + (j - q.r0) : -1;
                } else {
                    R.pos[r] = s.base + j;
                }
            }
        }
        auto use = [&](int t, int b) {
            const int x0 = tile_begin<kKT>(s.keys, s.tile + t);
            const float *k = sK + b * kKT * (D + 4), *v = sV + b * kKT * D;
            switch (nr) {
                case 1: tile_step<1, NC>(P, R, sQ, k, v, sP, x0, s.keys, warp, lane); break;
                case 2: tile_step<2, NC>(P, R, sQ, k, v, sP, x0, s.keys, warp, lane); break;
                case 3: tile_step<3, NC>(P, R, sQ, k, v, sP, x0, s.keys, warp, lane); break;
                case 4: tile_step<4, NC>(P, R, sQ, k, v, sP, x0, s.keys, warp, lane); break;
                default: break;
            }
        };
        if constexpr (sizeof(C) == 1) {
            copy_commit();
            Tile8<NC> tile;
            if (s.ntile > 0) {
                tile.fetch(P, s, tile_begin<kKT>(s.keys, s.tile), warp, lane);
                tile.put(P, sK, sV, warp, lane);
            }
            copy_wait<0>();  // the queries
            for (int t = 0; t < s.ntile; ++t) {
                const int b = t & 1;
                __syncthreads();  // the tile is there, and the one before has been used
                const bool more = t + 1 < s.ntile;
                if (more) tile.fetch(P, s, tile_begin<kKT>(s.keys, s.tile + t + 1), warp, lane);
                use(t, b);
                if (more) tile.put(P, sK + (b ^ 1) * kKT * (D + 4), sV + (b ^ 1) * kKT * D, warp, lane);
            }
        } else {
            if (s.ntile > 0) load_tile<C>(P, s, sK, sV, tile_begin<kKT>(s.keys, s.tile), warp, lane);
            copy_commit();
            for (int t = 0; t < s.ntile; ++t) {
                const int b = t & 1;
                if (t + 1 < s.ntile)
                    load_tile<C>(P, s, sK + (b ^ 1) * kKT * (D + 4), sV + (b ^ 1) * kKT * D,
                                 tile_begin<kKT>(s.keys, s.tile + t + 1), warp, lane);
                copy_commit();
                copy_wait<1>();
                __syncthreads();
                use(t, b);
                __syncthreads();
            }
        }
        copy_wait<0>();
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (r >= nr) continue;
            const int row = r * kWarps + warp;
            if (s.part >= 0) {
                if (!SPEC_IN(s.part + row, P.part_rows, DBG_ATTEND)) continue;
                float *o = P.part_o + (s.part + row) * D;
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    if (c * 128 + 4 * lane < D) store4(o + c * 128 + 4 * lane, R.o[r][c]);
                // a sum that is not a number must reach the joined row, whatever the other parts' maxima
                if (lane == 0) P.part_ml[s.part + row] = make_float2(isnan(R.l[r]) ? INFINITY : R.m[r], R.l[r]);
            } else {
                const int j = P.by_group(s.row0 + row), g = s.row0 + row - j * P.G;
                const int t = s.t0 + j, h = s.head * P.G + g;
                if (!SPEC_IN(t, P.T, DBG_ATTEND)) continue;
                const float inv = R.l[r] == 0.0f ? 0.0f : 1.0f / R.l[r];
                E *o = static_cast<E *>(P.out) + t * P.out_stride + static_cast<int64_t>(h) * D;
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    if (c * 128 + 4 * lane < D)
                        store4(o + c * 128 + 4 * lane, make_float4(R.o[r][c].x * inv, R.o[r][c].y * inv,
                                                                   R.o[r][c].z * inv, R.o[r][c].w * inv));
                if (lane == 0 && P.lse)
                    P.lse[static_cast<int64_t>(t) * P.Hq + h] =
                        R.l[r] == 0.0f ? -INFINITY : (R.m[r] + log2f(R.l[r])) * 0.6931471805599453f;
            }
        }
    }
    if (!PREFIX && warp == kWarps - 1) keep_books<kKT>(P, lane);
    end_kernel<PREFIX>(P);
    if (threadIdx.x == 0) P.err[(PREFIX ? P.own_workers : 0) + blockIdx.x] = 0;
}

}  // namespace fma
}  // namespace spec
