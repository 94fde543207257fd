// Appending a round's keys and values to the paged cache with their position rotation
// (spec_kv_append). See include/spec_attend.h for the contract.
//
// Rotary positions turn pair c of a head by the angle p * w_c, (a, b) -> (a cos - b sin,
// b cos + a sin), so that a rotated query's product with a rotated key depends on the difference of
// their positions alone. The cosines and sines come from the caller's table in 32 bits: an angle
// formed here as a 32-bit product would be off by p * 2^-24 radians, which at long positions is more
// than the type's rounding.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "spec_attend.h"
#include "spec_device.cuh"
#include "spec_paged.cuh"

namespace spec {

struct AppendParams {
    int32_t B, T, Hq, Hkv, D, rot, page_size, max_blocks, n_pages, n_pos;
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    void *q_out;
    int64_t q_out_stride;
    const float *cos_sin;
    void *k_cache, *v_cache;
    int64_t page_stride, slot_stride, head_stride;
    const int32_t *row_off, *kv_len, *block_table;
    int32_t *req_status;
    int32_t copy_blocks;  // blocks along x that move rows; one more after them checks the requests
};

constexpr int kAppendThreads = 256;

// N consecutive elements of E moved as one access (N * sizeof(E) a power of two up to 16 bytes).
template <typename E, int N>
struct alignas(sizeof(E) * N) Pack {
    E e[N];
};

template <typename E>
__device__ __forceinline__ float to_f32(E x);
template <>
__device__ __forceinline__ float to_f32(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename E>
__device__ __forceinline__ E from_f32(float x);
template <>
__device__ __forceinline__ float from_f32(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float x) { return __float2bfloat16_rn(x); }

// Floats of the cos_sin table, as wide as their alignment allows.
template <int N>
__device__ __forceinline__ void load_floats(float (&out)[N], const float *p) {
    constexpr int W = N % 4 == 0 ? 4 : (N % 2 == 0 ? 2 : 1);
#pragma unroll
    for (int i = 0; i < N; i += W) {
        const Pack<float, W> x = *reinterpret_cast<const Pack<float, W> *>(p + i);
#pragma unroll
        for (int j = 0; j < W; ++j) out[i + j] = x.e[j];
    }
}

// One thread moves the same piece of a row (its task) for every row of its column of blocks: a pair
// of packs c and c + rot/2 that turn together, a pack of interleaved pairs, or a pack that is
// copied. V: elements per pack (16 bytes, or 1 when something is not on 16-byte boundaries).
//
// Bound by latency when there are few rows (offsets -> length -> page -> store is a chain of
// dependent loads; the row's own values are requested before it), by DRAM when there are many.
template <typename E, int V, bool INTER>
__global__ void __launch_bounds__(kAppendThreads) spec_append_kernel(const AppendParams P) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x % kWarp;
    if (blockIdx.x == static_cast<unsigned>(P.copy_blocks)) {
        // the requests' status, a warp each
        constexpr int kWarps = kAppendThreads / kWarp;
        for (int i = blockIdx.y * kWarps + threadIdx.x / kWarp; i < P.B; i += gridDim.y * kWarps) {
            const int r0 = P.row_off[i], r1 = P.row_off[i + 1], kv = P.kv_len[i];
            int st = 0;
            if (r0 < 0 || r1 < r0 || r1 > P.T || kv < 0) {
                st = SPEC_REQ_BAD_SHAPE;
            } else if (r1 > r0 && kv > 0) {
                if (kv > P.n_pos) st = SPEC_REQ_BAD_SHAPE;
                const int b1 = (kv - 1) / P.page_size;
                if (b1 >= P.max_blocks) st |= SPEC_REQ_BAD_BLOCKS;
                bool bad = false;
                for (int b = max(0, kv - (r1 - r0)) / P.page_size + lane; b <= min(b1, P.max_blocks - 1); b += kWarp) {
                    const int page = P.block_table[static_cast<int64_t>(i) * P.max_blocks + b];
                    bad |= page < 0 || page >= P.n_pages;
                }
                if (__any_sync(0xffffffffu, bad)) st |= SPEC_REQ_BAD_BLOCKS;
            }
            if (lane == 0 && P.req_status && SPEC_IN(i, P.B, DBG_OUT_REQS)) P.req_status[i] = st;
        }
        return;
    }

    // this thread's task: head, first element(s), kind
    constexpr bool kPairs = !INTER || V == 1;  // a task turns elements d0.. with elements d1..
    const int turn = kPairs ? P.rot / 2 / V : P.rot / V;
    const int per_head = turn + (P.D - P.rot) / V, per_v = P.D / V;
    const int n_qk = (P.Hq + P.Hkv) * per_head;
    const int task = blockIdx.x * kAppendThreads + threadIdx.x;
    const bool have = task < n_qk + P.Hkv * per_v;
    int head = 0, d0 = 0, d1 = 0, c0 = 0;
    bool rotates = false;
    enum { Q, K, VAL } what = VAL;
    if (task < n_qk) {
        head = task / per_head;
        const int x = task - head * per_head;
        rotates = x < turn;
        if (!rotates) {
            d0 = P.rot + (x - turn) * V;
        } else if (!INTER) {
            d0 = c0 = x * V;
            d1 = d0 + P.rot / 2;
        } else {
            d0 = V == 1 ? 2 * x : x * V;
            d1 = d0 + 1;
            c0 = d0 / 2;
        }
        what = head < P.Hq ? Q : K;
        if (what == K) head -= P.Hq;
    } else if (have) {
        head = (task - n_qk) / per_v;
        d0 = (task - n_qk - head * per_v) * V;
    }
    const bool two = kPairs && rotates;
    const E *src = static_cast<const E *>(what == Q ? P.q : what == K ? P.k : P.v);
    const int64_t src_stride = what == Q ? P.q_stride : what == K ? P.k_stride : P.v_stride;
    src += static_cast<int64_t>(head) * P.D;
    E *cache = static_cast<E *>(what == K ? P.k_cache : P.v_cache);
    using Vec = Pack<E, V>;

    for (int r = blockIdx.y; r < P.T; r += gridDim.y) {
        Vec a = {}, b = {};
        if (have) {
            a = *reinterpret_cast<const Vec *>(src + r * src_stride + d0);
            if (two) b = *reinterpret_cast<const Vec *>(src + r * src_stride + d1);
        }
        const int i = find_request(P.row_off, P.B, r, lane);
        const int r0 = P.row_off[i], r1 = P.row_off[i + 1], kv = P.kv_len[i];
        if (!have || r0 < 0 || r < r0 || r >= r1 || r1 > P.T || kv < 0) continue;
        const int pos = kv - (r1 - r0) + (r - r0);
        if (pos < 0 || pos >= P.n_pos) continue;
        const int blk = pos / P.page_size;
        if (blk >= P.max_blocks) continue;
        const int page = P.block_table[static_cast<int64_t>(i) * P.max_blocks + blk];
        if (page < 0 || page >= P.n_pages) continue;
        if (rotates) {
            constexpr int NC = kPairs ? V : (V + 1) / 2;
            float c[NC], s[NC];
            const float *cs = P.cos_sin + static_cast<int64_t>(pos) * P.rot + c0;
            load_floats(c, cs);
            load_floats(s, cs + P.rot / 2);
            if constexpr (kPairs) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float x = to_f32(a.e[e]), y = to_f32(b.e[e]);
                    a.e[e] = from_f32<E>(x * c[e] - y * s[e]);
                    b.e[e] = from_f32<E>(y * c[e] + x * s[e]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < NC; ++e) {
                    const float x = to_f32(a.e[2 * e]), y = to_f32(a.e[2 * e + 1]);
                    a.e[2 * e] = from_f32<E>(x * c[e] - y * s[e]);
                    a.e[2 * e + 1] = from_f32<E>(y * c[e] + x * s[e]);
                }
            }
        }
        E *dst;
        if (what == Q)
            dst = static_cast<E *>(P.q_out) + r * P.q_out_stride + static_cast<int64_t>(head) * P.D;
        else
            dst = cache + page * P.page_stride + (pos - blk * P.page_size) * P.slot_stride + head * P.head_stride;
        if (!SPEC_IN(page, P.n_pages, DBG_CACHE) || !SPEC_IN(d0 + V - 1, P.D, DBG_CACHE)) continue;
        *reinterpret_cast<Vec *>(dst + d0) = a;
        if (two && SPEC_IN(d1 + V - 1, P.D, DBG_CACHE)) *reinterpret_cast<Vec *>(dst + d1) = b;
    }
}

template <typename E, int V, bool INTER>
static spec_status launch_append(AppendParams &P, cudaStream_t stream) {
    constexpr bool kPairs = !INTER || V == 1;
    const int turn = kPairs ? P.rot / 2 / V : P.rot / V;
    const int tasks = (P.Hq + P.Hkv) * (turn + (P.D - P.rot) / V) + P.Hkv * (P.D / V);
    P.copy_blocks = (tasks + kAppendThreads - 1) / kAppendThreads;
    // a block a row until the device is full (8 blocks of 256 threads on each of 152 SMs), then
    // blocks walk rows: the task's decoding is paid once
    const int rows = std::max(1, std::min(P.T, 152 * 8 / P.copy_blocks));
    const dim3 grid(static_cast<unsigned>(P.copy_blocks) + (P.req_status ? 1u : 0u), static_cast<unsigned>(rows));
    return launch_after(spec_append_kernel<E, V, INTER>, grid, dim3(kAppendThreads), 0, stream, P) == cudaSuccess
               ? SPEC_OK
               : SPEC_ERR_CUDA;
}

template <typename E>
static spec_status dispatch_append(AppendParams &P, bool inter, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(E);
    auto aligned = [](const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    const int64_t strides = P.k_stride | P.v_stride | P.page_stride | P.slot_stride | P.head_stride |
                            (P.Hq ? P.q_stride | P.q_out_stride : 0);
    const bool vec = strides % V == 0 && P.D % V == 0 && P.rot % (inter ? V : 2 * V) == 0 && aligned(P.k) &&
                     aligned(P.v) && aligned(P.k_cache) && aligned(P.v_cache) && (!P.rot || aligned(P.cos_sin)) &&
                     (!P.Hq || (aligned(P.q) && aligned(P.q_out)));
    if (inter) return vec ? launch_append<E, V, true>(P, stream) : launch_append<E, 1, true>(P, stream);
    return vec ? launch_append<E, V, false>(P, stream) : launch_append<E, 1, false>(P, stream);
}

}  // namespace spec

using namespace spec;

extern "C" spec_status spec_kv_append(const spec_kv_append_args *a, cudaStream_t stream) {
    if (!a) return SPEC_ERR_INVALID_ARG;
    if (a->B < 1 || a->total_rows < 0 || a->n_q_heads < 0 || a->n_kv_heads < 1 || a->head_dim < 1 ||
        a->page_size < 1 || a->max_blocks < 1 || a->n_pages < 1 || a->n_pos < 0)
        return SPEC_ERR_INVALID_ARG;
    if (a->rot_dim < 0 || a->rot_dim > a->head_dim || a->rot_dim % 2 != 0) return SPEC_ERR_INVALID_ARG;
    if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
    if (!a->row_off || !a->kv_len || !a->block_table || !a->k_cache || !a->v_cache) return SPEC_ERR_INVALID_ARG;
    if (a->rot_dim > 0 && !a->cos_sin) return SPEC_ERR_INVALID_ARG;
    if (a->total_rows > 0 && (!a->k || !a->v || (a->n_q_heads > 0 && (!a->q || !a->q_out)))) return SPEC_ERR_INVALID_ARG;
    const int64_t D = a->head_dim;
    if (a->total_rows > 1 && (a->k_stride < a->n_kv_heads * D || a->v_stride < a->n_kv_heads * D ||
                              (a->n_q_heads > 0 && (a->q_stride < a->n_q_heads * D || a->q_out_stride < a->n_q_heads * D))))
        return SPEC_ERR_INVALID_ARG;
    if (a->n_q_heads > 0 && a->q_out == a->q && a->q_out_stride != a->q_stride) return SPEC_ERR_INVALID_ARG;
    if (a->page_stride < 0 || a->slot_stride < 0 || a->head_stride < 0) return SPEC_ERR_INVALID_ARG;
    if (a->head_dim > 512 || a->n_q_heads > 4096 || a->n_kv_heads > 4096) return SPEC_ERR_UNSUPPORTED;

    AppendParams P = {};
    P.B = a->B;
    P.T = a->total_rows;
    P.Hq = a->n_q_heads;
    P.Hkv = a->n_kv_heads;
    P.D = a->head_dim;
    P.rot = a->rot_dim;
    P.page_size = a->page_size;
    P.max_blocks = a->max_blocks;
    P.n_pages = a->n_pages;
    // without a rotation no table row is read: every position is served
    P.n_pos = a->rot_dim > 0 ? a->n_pos : INT32_MAX;
    P.q = a->q;
    P.k = a->k;
    P.v = a->v;
    P.q_stride = a->q_stride;
    P.k_stride = a->k_stride;
    P.v_stride = a->v_stride;
    P.q_out = a->q_out;
    P.q_out_stride = a->q_out_stride;
    P.cos_sin = a->cos_sin;
    P.k_cache = a->k_cache;
    P.v_cache = a->v_cache;
    P.page_stride = a->page_stride;
    P.slot_stride = a->slot_stride;
    P.head_stride = a->head_stride;
    P.row_off = a->row_off;
    P.kv_len = a->kv_len;
    P.block_table = a->block_table;
    P.req_status = a->req_status;
    return a->dtype == SPEC_BF16 ? dispatch_append<__nv_bfloat16>(P, a->interleaved != 0, stream)
                                 : dispatch_append<float>(P, a->interleaved != 0, stream);
}

#ifdef SPEC_DEBUG
namespace spec {
// The debug words of this translation unit's kernel.
cudaError_t debug_take_append(unsigned int out[4]) { return spec_dbg_take(out); }
}  // namespace spec
#endif
