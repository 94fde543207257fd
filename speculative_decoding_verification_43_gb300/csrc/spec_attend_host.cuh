// What the calls of the attention over the paged cache share on the host, whatever type the cache has, and the
// kernels that join the parts.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "spec_attend.h"
#include "spec_attend_fma.cuh"
#include "spec_attend_plan.cuh"
#include "spec_device.cuh"
#include "spec_paged.cuh"

namespace spec {

// ---------------------------------------------------------------- joining the parts

constexpr int kJoinWarps = 4, kJoinThreads = kJoinWarps * kWarp;

// Parts of one row: part x < n lies `pitch` rows after part x - 1 (part 1 after `later`, where the first
// worker's slot differs from the others').
struct PartRun {
    int n, pitch;
    int64_t base, later;
    __device__ __forceinline__ int64_t row(int x) const { return x == 0 ? base : later + static_cast<int64_t>(x) * pitch; }
};

// A sum l of a part times w = 2^d, d <= 0. Over a cache in 8 bits a sum is divided by the values' scales and its reference is
// not, so that l may be 2^75 and count where 2^d itself is 0.
__device__ __forceinline__ float scaled_sum(float l, float d, float w) {
    if (d >= -120.0f) return w == 0.0f ? 0.0f : w * l;
    const float half = ex2(0.5f * d);
    return half == 0.0f ? 0.0f : l * half * half;
}

// Joins the parts of one row and writes it; a warp per row. The parts' outputs are asked for together with
// their maxima, four at a time, and weighed when both are there.
template <typename E>
__device__ __forceinline__ void join_row(const AttendParams &P, const PartRun &a, const PartRun &b, int t, int h,
                                         int lane) {
    const int n = a.n + b.n;
    float M = -INFINITY, L = 0.0f;
    float4 o[2] = {};
#pragma unroll 1
    for (int x0 = 0; x0 < n; x0 += kWarp) {
        const int x = x0 + lane;
        float2 ml = make_float2(-INFINITY, 0.0f);
        if (x < n) {
            const int64_t r = x < a.n ? a.row(x) : b.row(x - a.n);
            if (SPEC_IN(r, P.part_rows, DBG_ATTEND)) ml = P.part_ml[r];
        }
        const float top = fmaxf(M, warp_max(ml.x));
        const float ref = top == -INFINITY ? 0.0f : top;
        // weights of these parts, and of what has been joined so far
        const float w = ex2(ml.x - ref), keep = M == -INFINITY ? 0.0f : ex2(M - ref);
        L = scaled_sum(L, M - ref, keep) + warp_sum(scaled_sum(ml.y, ml.x - ref, w));
        M = top;
#pragma unroll
        for (int c = 0; c < 2; ++c) o[c] = make_float4(o[c].x * keep, o[c].y * keep, o[c].z * keep, o[c].w * keep);
        const int cnt = min(kWarp, n - x0);
#pragma unroll 1
        for (int j0 = 0; j0 < cnt; j0 += 4) {
            float4 v[4][2];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int y = x0 + min(j0 + j, cnt - 1);
                const int64_t r = y < a.n ? a.row(y) : b.row(y - a.n);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int d = c * 128 + 4 * lane;
                    v[j][c] = d < P.D && SPEC_IN(r, P.part_rows, DBG_ATTEND)
                                  ? *reinterpret_cast<const float4 *>(P.part_o + r * P.D + d)
                                  : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j0 + j >= cnt) break;
                // (a part whose weight vanishes takes part all the same: what is not finite in it has been seen)
                const float wj = __shfl_sync(0xffffffffu, w, j0 + j);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    o[c].x = fmaf(wj, v[j][c].x, o[c].x);
                    o[c].y = fmaf(wj, v[j][c].y, o[c].y);
                    o[c].z = fmaf(wj, v[j][c].z, o[c].z);
                    o[c].w = fmaf(wj, v[j][c].w, o[c].w);
                }
            }
        }
    }
    if (!SPEC_IN(t, P.T, DBG_ATTEND)) return;
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    E *dst = static_cast<E *>(P.out) + t * P.out_stride + static_cast<int64_t>(h) * P.D;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int d = c * 128 + 4 * lane;
        if (d < P.D) fma::store4(dst + d, make_float4(o[c].x * inv, o[c].y * inv, o[c].z * inv, o[c].w * inv));
    }
    if (lane == 0 && P.lse)
        P.lse[static_cast<int64_t>(t) * P.Hq + h] = L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

// Request i's status goes out, and the rows of a request in error become 0 / -inf (a block). Rows in doubt
// belong to requests in error only, so that no other's rows are touched.
template <typename E>
__device__ __forceinline__ void finish_request(const AttendParams &P, int i) {
    int bad = 0;
    const bool broken = *P.broken;
#pragma unroll 1
    for (int w = threadIdx.x; w < P.own_workers + P.prefix_workers; w += kJoinThreads) bad |= P.err[w];
    int st = P.status[i] | (__syncthreads_or(bad) ? SPEC_REQ_TIMEOUT : 0);
    if (broken) {
        const int r0 = P.row_off[i], r1 = P.row_off[i + 1];
        if (offsets_right(r0, r1, P.T) &&
            __syncthreads_or(offsets_contradict(P.row_off, P.B, P.T, i, r0, r1, threadIdx.x, kJoinThreads)))
            st |= SPEC_REQ_BAD_SHAPE;
    }
    if (threadIdx.x == 0 && P.req_status) P.req_status[i] = st;
    if (st == SPEC_REQ_OK) return;
    const ReqRows q = load_request(P, i);
#pragma unroll 1
    for (int j = 0; j < q.n; ++j) {
        E *o = static_cast<E *>(P.out) + (q.r0 + j) * P.out_stride;
#pragma unroll 1
        for (int d = 4 * threadIdx.x; d < P.Hq * P.D; d += 4 * kJoinThreads)
            fma::store4(o + d, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
        if (P.lse)
#pragma unroll 1
            for (int h = threadIdx.x; h < P.Hq; h += kJoinThreads)
                P.lse[static_cast<int64_t>(q.r0 + j) * P.Hq + h] = -INFINITY;
    }
}

// Calls without a shared prefix: a warp for each row that an item begun by a worker may have (worker x,
// rows 4 y ..), after the requests' blocks. Its first read says what there is to join; two round trips to
// memory in all.
template <typename E>
static __global__ void __launch_bounds__(kJoinThreads) spec_attend_join_kernel(const AttendParams P) {
    griddep_launch_dependents();
    griddep_wait();
    if (blockIdx.x < static_cast<unsigned>(P.B)) return finish_request<E>(P, blockIdx.x);
    const int blk = blockIdx.x - P.B, per = (P.own_pitch + kJoinWarps - 1) / kJoinWarps;
    const int w = blk / per, r = (blk - w * per) * kJoinWarps + threadIdx.x / kWarp;
    const CutItem c = P.cut[w];
    if (r >= c.nrows || P.status[c.req] != SPEC_REQ_OK) return;
    PartRun run, none = {};
    run.n = c.parts;
    run.pitch = 2 * P.own_pitch * P.head_step;
    run.later = static_cast<int64_t>(2 * w) * P.own_pitch + r;
    run.base = run.later + c.slot * P.own_pitch;
    const int j = P.by_group(c.row0 + r), g = c.row0 + r - j * P.G;
    join_row<E>(P, run, none, c.t0 + j, c.head * P.G + g, threadIdx.x % kWarp);
}

// Calls with a shared prefix: every row has parts of both classes. A warp for the rows of one token that
// share a key/value head.
template <typename E, int KT>
static __global__ void __launch_bounds__(kJoinThreads) spec_attend_join_shared_kernel(const AttendParams P) {
    griddep_launch_dependents();
    griddep_wait();
    if (blockIdx.x < static_cast<unsigned>(P.B)) return finish_request<E>(P, blockIdx.x);
    const int lane = threadIdx.x % kWarp;
    const bool broken = *P.broken;
    const int64_t unit = static_cast<int64_t>(blockIdx.x - P.B) * kJoinWarps + threadIdx.x / kWarp;
    if (unit >= static_cast<int64_t>(P.T) * P.Hkv) return;
    const int tok = static_cast<int>(unit / P.Hkv), head = static_cast<int>(unit - static_cast<int64_t>(tok) * P.Hkv);
    const int i = find_request(P.row_off, P.B, P.T, tok, lane);
    const ReqRows q = load_request(P, i);
    if (tok < q.r0 || tok >= q.r0 + q.n || P.status[i] != SPEC_REQ_OK) return;
    if (broken && __any_sync(0xffffffffu, offsets_contradict(P.row_off, P.B, P.T, i, q.r0, q.r0 + q.n, lane, kWarp)))
        return;
    const int pre_units = *P.prefix_units, tiles = row_tiles(P.T * P.G, P.prefix_rt_log2);
    const int pre_len = pre_units + P.prefix_extra;
    const Shares share(P.unit_prefix[P.B], P.own_workers), pre_share(P.Hkv * tiles * pre_len, P.prefix_workers);
    // items of the row tiles before this row's: they are walked through with it
    int start = P.unit_prefix[i] + head * own_units<KT>(P, q), k = 0, units = item_tiles(own_tiles<KT>(P, q, 0));
    const int64_t pre_rows = static_cast<int64_t>(head) * P.T * P.G;
    const int64_t own_rows = static_cast<int64_t>(P.T) * P.Hq + static_cast<int64_t>(P.prefix_workers) * P.prefix_pitch +
                             (static_cast<int64_t>(q.r0) * P.Hkv + static_cast<int64_t>(head) * q.n) * P.G;
    PartRun pre = {}, own = {};
    int pre_k = -1, own_k = -1;
#pragma unroll 1
    for (int g = 0; g < P.G; ++g) {
        const int pr = tok * P.G + g, ow = (tok - q.r0) * P.G + g;
        if (pr >> P.prefix_rt_log2 != pre_k) {
            pre_k = pr >> P.prefix_rt_log2;
            const int first = (head * tiles + pre_k) * pre_len + P.prefix_extra, w0 = pre_share.owner(first);
            pre.n = pre_share.owner(first + pre_units - 1) - w0 + 1;
            pre.pitch = P.prefix_pitch;
            pre.base = pre.later = pre_rows + static_cast<int64_t>(w0) * P.prefix_pitch;
        }
        if (ow >> P.own_rt_log2 != own_k) {
            own_k = ow >> P.own_rt_log2;
#pragma unroll 1
            for (; k < own_k; ++k) {
                start += units + P.own_extra;
                units = item_tiles(own_tiles<KT>(P, q, k + 1));
            }
            const int w0 = share.owner(start + P.own_extra);
            own.n = share.owner(start + P.own_extra + units - 1) - w0 + 1;
            own.pitch = P.own_pitch;
            own.base = own.later = own_rows + static_cast<int64_t>(w0) * P.own_pitch;
        }
        PartRun a = pre, b = own;
        a.base = a.later += pr;
        b.base = b.later += ow;
        join_row<E>(P, a, b, tok, head * P.G + g, lane);
    }
}

// ---------------------------------------------------------------- host side

struct AttendLayout {
    size_t status, unit_prefix, cut, prefix_units, broken, err, ml, o, total;
};

static AttendLayout attend_layout(const AttendParams &P) {
    AttendLayout L = {};
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off = (off + bytes + 255) / 256 * 256;
        return o;
    };
    L.status = take(static_cast<size_t>(P.B) * 4);
    L.unit_prefix = take((static_cast<size_t>(P.B) + 1) * 4);
    L.cut = take(static_cast<size_t>(P.own_workers) * sizeof(CutItem));
    L.prefix_units = take(4);
    L.broken = take(4);
    L.err = take(static_cast<size_t>(P.own_workers + P.prefix_workers) * 4);
    L.ml = take(static_cast<size_t>(P.part_rows) * 8);
    L.o = take(static_cast<size_t>(P.part_rows) * P.D * 4);
    L.total = off;
    return L;
}

// The sizes of a call, checked; workers and parts of the kernel that serves it.
static spec_status attend_sizes(const spec_attend_args *a, AttendParams &P) {
    if (!a) return SPEC_ERR_INVALID_ARG;
    if (a->B < 1 || a->total_rows < 0 || a->n_kv_heads < 1 || a->n_q_heads < 1 || a->n_q_heads % a->n_kv_heads != 0 ||
        a->head_dim < 1 || a->page_size < 1 || a->max_blocks < 1 || a->n_pages < 1 || a->window < 0 || a->n_sink < 0 ||
        a->shared_len < 0)
        return SPEC_ERR_INVALID_ARG;
    if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
    if (!(a->scale > 0.0f) || !std::isfinite(a->scale)) return SPEC_ERR_INVALID_ARG;
    const int vec = a->dtype == SPEC_BF16 ? 8 : 4;
    if (a->head_dim > 256 || a->head_dim % vec != 0) return SPEC_ERR_UNSUPPORTED;
    // packed rows and positions are 32-bit
    if (static_cast<int64_t>(a->total_rows) * a->n_q_heads > INT_MAX / 4 ||
        static_cast<int64_t>(a->max_blocks) * a->page_size > INT_MAX / 2 || a->shared_len > INT_MAX / 2 ||
        a->n_q_heads > 65536)
        return SPEC_ERR_UNSUPPORTED;
    // and so are the units of work, at their most with the smallest items and tiles (16 rows, 32 positions)
    const int64_t most_tiles = std::max<int64_t>(static_cast<int64_t>(a->max_blocks) * a->page_size, a->shared_len) / 32 + 8;
    const int64_t head_tiles =
        static_cast<int64_t>(a->total_rows) * (a->n_q_heads / a->n_kv_heads) / fma::kRT + a->B + 1;
    if (head_tiles * a->n_kv_heads > INT_MAX / most_tiles) return SPEC_ERR_UNSUPPORTED;
    P.B = a->B;
    P.T = a->total_rows;
    P.Hq = a->n_q_heads;
    P.Hkv = a->n_kv_heads;
    P.G = a->n_q_heads / a->n_kv_heads;
    P.D = a->head_dim;
    P.page_size = a->page_size;
    P.by_page = FastDiv(a->page_size);
    P.by_group = FastDiv(P.G);
    P.max_blocks = a->max_blocks;
    P.n_pages = a->n_pages;
    P.window = a->window;
    P.n_sink = a->n_sink;
    P.shared_len = a->shared_len;
    P.head_step = 1;
    P.scale_log2 = a->scale * 1.4426950408889634f;

    return SPEC_OK;
}

// Pointers and strides, with `vec` elements of q and out and `cache_vec` of the cache in 16 bytes; the sizes are in P.
static spec_status attend_pointers(const spec_attend_args *a, AttendParams &P, int vec, int cache_vec) {
    if (!a->row_off || !a->kv_len || !a->block_table || !a->k_cache || !a->v_cache) return SPEC_ERR_INVALID_ARG;
    if (P.T > 0 && (!a->q || !a->out)) return SPEC_ERR_INVALID_ARG;
    if (P.shared_len > 0 && !a->shared_table) return SPEC_ERR_INVALID_ARG;
    const int64_t width = static_cast<int64_t>(P.Hq) * P.D;
    if (P.T > 1 && (a->q_stride < width || a->out_stride < width)) return SPEC_ERR_INVALID_ARG;
    if (a->page_stride < 0 || a->slot_stride < 0 || a->head_stride < 0) return SPEC_ERR_INVALID_ARG;
    auto aligned = [](const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    if ((a->q_stride | a->out_stride) % vec != 0 || (a->page_stride | a->slot_stride | a->head_stride) % cache_vec != 0 ||
        !aligned(a->q) || !aligned(a->out) || !aligned(a->k_cache) || !aligned(a->v_cache))
        return SPEC_ERR_UNSUPPORTED;
    P.q = a->q;
    P.k_cache = a->k_cache;
    P.v_cache = a->v_cache;
    P.q_stride = a->q_stride;
    P.page_stride = a->page_stride;
    P.slot_stride = a->slot_stride;
    P.head_stride = a->head_stride;
    P.row_off = a->row_off;
    P.kv_len = a->kv_len;
    P.block_table = a->block_table;
    P.shared_table = a->shared_table;
    P.out = a->out;
    P.out_stride = a->out_stride;
    P.lse = a->lse;
    P.req_status = a->req_status;
    return SPEC_OK;
}

// The workspace's parts.
static void attend_place(AttendParams &P, void *workspace) {
    const AttendLayout L = attend_layout(P);
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    P.status = reinterpret_cast<int32_t *>(ws + L.status);
    P.unit_prefix = reinterpret_cast<int32_t *>(ws + L.unit_prefix);
    P.cut = reinterpret_cast<CutItem *>(ws + L.cut);
    P.prefix_units = reinterpret_cast<int32_t *>(ws + L.prefix_units);
    P.broken = reinterpret_cast<int32_t *>(ws + L.broken);
    P.err = reinterpret_cast<int32_t *>(ws + L.err);
    P.part_ml = reinterpret_cast<float2 *>(ws + L.ml);
    P.part_o = reinterpret_cast<float *>(ws + L.o);
}

// Slots copied as one box by the tensor-core kernels: the largest power of two that divides the page, from 8 to
// a tile of 128 (0: there is none).
static int box_log2_of(int page_size) {
    int log2 = 0;
    for (int b = 3; b <= 7; ++b)
        if (page_size % (1 << b) == 0) log2 = b;
    return log2;
}

// Workers of the fp32 units' kernel.
static void attend_fma_work(AttendParams &P) {
    P.own_rt_log2 = P.prefix_rt_log2 = fma::kRTLog2;
    P.own_workers = P.prefix_workers = kSMs * fma::ctas_per_sm(P.D);
    P.box_log2 = 0;
    // at 0, 1, 2, 4, 8: 250, 248, 248, 252, 256 us (256 fp32 requests under a window), 411, 408, 412, 417, 427
    // (64 fp32 requests of up to 8000 positions), 894, 875, 888, 912, 956 (an fp32 prompt of 2000 rows)
    P.own_extra = P.prefix_extra = 2;
}

// The parts that the workers leave, with the workers and items known.
static void attend_parts(AttendParams &P) {
    const int64_t head_rows = static_cast<int64_t>(P.T) * P.G;
    if (P.shared_len == 0) P.prefix_workers = 0;
    P.own_pitch = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(1 << P.own_rt_log2, head_rows)));
    P.prefix_pitch = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(1 << P.prefix_rt_log2, head_rows)));
    if (P.shared_len > 0)
        P.part_rows = 2 * static_cast<int64_t>(P.T) * P.Hq + static_cast<int64_t>(P.own_workers) * P.own_pitch +
                      static_cast<int64_t>(P.prefix_workers) * P.prefix_pitch;
    else
        P.part_rows = 2 * static_cast<int64_t>(P.own_workers) * P.own_pitch;
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's call that fills a tensor map in (looked up once).
static EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

template <typename E, int KT>
static cudaError_t launch_join(const AttendParams &P, cudaStream_t stream) {
    const bool shared = P.shared_len > 0;
    const int64_t blocks = shared ? (static_cast<int64_t>(P.T) * P.Hkv + kJoinWarps - 1) / kJoinWarps
                                  : static_cast<int64_t>(P.own_workers) * ((P.own_pitch + kJoinWarps - 1) / kJoinWarps);
    return launch_after(shared ? spec_attend_join_shared_kernel<E, KT> : spec_attend_join_kernel<E>,
                        dim3(static_cast<unsigned>(P.B + blocks)), dim3(kJoinThreads), 0, stream, P);
}

}  // namespace spec
