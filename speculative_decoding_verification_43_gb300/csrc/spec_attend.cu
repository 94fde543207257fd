// Attention of a round's rows over the paged cache (spec_attend). See include/spec_attend.h for the
// contract, spec_attend_plan.cuh for how the work is cut.
//
// out = sum_x softmax_x(s_x) v_x needs one pass over the keys: with a running maximum m, sum
// l = sum 2^(s_x - m) and output o = sum 2^(s_x - m) v_x, a larger maximum m' rescales l and o by
// 2^(m - m'). Parts taken over different keys join alike: with M = max m_i, out = sum o_i 2^(m_i - M) /
// sum l_i 2^(m_i - M).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "spec_attend.h"
#include "spec_attend_fma.cuh"
#include "spec_attend_pair.cuh"
#include "spec_attend_plan.cuh"
#include "spec_attend_round.cuh"
#include "spec_device.cuh"
#include "spec_paged.cuh"

namespace spec {

constexpr int kSMs = 152;

// ---------------------------------------------------------------- joining the parts

constexpr int kJoinWarps = 4, kJoinThreads = kJoinWarps * kWarp;

// Parts of one row: part x < n lies `pitch` rows after part x - 1 (part 1 after `later`, where the first
// worker's slot differs from the others').
struct PartRun {
    int n, pitch;
    int64_t base, later;
    __device__ __forceinline__ int64_t row(int x) const { return x == 0 ? base : later + static_cast<int64_t>(x) * pitch; }
};

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
        L = L * keep + warp_sum(w == 0.0f ? 0.0f : w * ml.y);
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
__global__ void __launch_bounds__(kJoinThreads) spec_attend_join_kernel(const AttendParams P) {
    griddep_launch_dependents();
    griddep_wait();
    if (blockIdx.x < static_cast<unsigned>(P.B)) return finish_request<E>(P, blockIdx.x);
    const int blk = blockIdx.x - P.B, per = (P.own_pitch + kJoinWarps - 1) / kJoinWarps;
    const int w = blk / per, r = (blk - w * per) * kJoinWarps + threadIdx.x / kWarp;
    const CutItem c = P.cut[w];
    if (r >= c.nrows || P.status[c.req] != SPEC_REQ_OK) return;
    PartRun run, none = {};
    run.n = c.parts;
    run.pitch = 2 * P.own_pitch;
    run.later = static_cast<int64_t>(2 * w) * P.own_pitch + r;
    run.base = run.later + c.slot * P.own_pitch;
    const int j = P.by_group(c.row0 + r), g = c.row0 + r - j * P.G;
    join_row<E>(P, run, none, c.t0 + j, c.head * P.G + g, threadIdx.x % kWarp);
}

// Calls with a shared prefix: every row has parts of both classes. A warp for the rows of one token that
// share a key/value head.
template <typename E, int KT>
__global__ void __launch_bounds__(kJoinThreads) spec_attend_join_shared_kernel(const AttendParams P) {
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
    P.scale_log2 = a->scale * 1.4426950408889634f;

    return SPEC_OK;
}

// Rows of an item (as a power of two) and workers for `rows` packed rows of a head over `groups` requests
// on the tensor cores: the round kernel's items of 32 or 64 rows while they hold most requests, else the pair
// kernel's of 256. In us, 64 requests of 2000 to 4000 positions, all with this many rows:
//     rows      16   24   32   40   48   64   80
//     32       139  145  148  263  265  272  391
//     64       146  154  159  175  184  208  316
//     256      176  183  191  191  192  193  194
// The first limit is below 32 because the average is all that is known here (lengths are on the device), and a
// request of n packed rows reads its keys once for each item, n / RT times rounded up. Batches of unlike
// requests pay for that: 63 of 5 rows after 8000 positions with one prompt of 2000 rows take 471 us, the two
// parts by themselves 333 and 69; 512 single tokens after 1000 with that prompt 590, by themselves 355 and 69.
static void tensor_class(int64_t rows, int64_t groups, int32_t &rt_log2, int32_t &workers) {
    rt_log2 = rows <= 24 * groups ? 5 : rows <= 48 * groups ? 6 : pair::kRTLog2;
    workers = rt_log2 == pair::kRTLog2 ? kSMs : kSMs * round_::kPerSM;
}

// Time of an item beside its tiles, in tiles: what makes the workers end together. Pair kernel, 4 prompts, at
// 4, 6, 8: 390, 369, 378 us; round kernel, 64 windowed requests, at 2, 3, 4, 5: 84, 81, 81, 80 us. (One batch
// each. The fp32 units' kernel, where 2 is taken: attend_work.)
static int own_extra_units(int rt_log2) { return rt_log2 == pair::kRTLog2 ? 6 : 4; }

// Workers and parts of the kernels that serve the call.
static void attend_work(AttendParams &P, bool tensor) {
    const int64_t head_rows = static_cast<int64_t>(P.T) * P.G;
    if (tensor) {
        tensor_class(head_rows, P.B, P.own_rt_log2, P.own_workers);
        tensor_class(head_rows, 1, P.prefix_rt_log2, P.prefix_workers);
        // an item's beginning and end take the time of some tiles
        P.own_extra = own_extra_units(P.own_rt_log2);
        P.prefix_extra = own_extra_units(P.prefix_rt_log2);
        // boxes of slots: the largest power of two that divides the page, from 8 to a tile
        P.box_log2 = 0;
        for (int b = 3; b <= 7; ++b)
            if (P.page_size % (1 << b) == 0) P.box_log2 = b;
    } else {
        P.own_rt_log2 = P.prefix_rt_log2 = fma::kRTLog2;
        P.own_workers = P.prefix_workers = kSMs * fma::ctas_per_sm(P.D);
        P.box_log2 = 0;
        // at 0, 1, 2, 4, 8: 250, 248, 248, 252, 256 us (256 fp32 requests under a window), 411, 408, 412, 417, 427
        // (64 fp32 requests of up to 8000 positions), 894, 875, 888, 912, 956 (an fp32 prompt of 2000 rows)
        P.own_extra = P.prefix_extra = 2;
    }
    if (P.shared_len == 0) P.prefix_workers = 0;
    P.own_pitch = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(1 << P.own_rt_log2, head_rows)));
    P.prefix_pitch = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(1 << P.prefix_rt_log2, head_rows)));
    if (P.shared_len > 0)
        P.part_rows = 2 * static_cast<int64_t>(P.T) * P.Hq + static_cast<int64_t>(P.own_workers) * P.own_pitch +
                      static_cast<int64_t>(P.prefix_workers) * P.prefix_pitch;
    else
        P.part_rows = 2 * static_cast<int64_t>(P.own_workers) * P.own_pitch;
}

// The cache as two-dimensional tensor maps of slots, where its strides allow it: pages a whole number of
// slots apart, heads inside a slot or a whole number of slots apart. bf16, head sizes the matrix
// instructions take.
static bool cache_map(const spec_attend_args *a, tiles::CacheMap &M, int64_t &rows, int64_t &cols) {
    if (a->dtype != SPEC_BF16 || a->head_dim % 16 != 0 || a->head_dim > 128) return false;
    const int64_t slot = a->slot_stride, D = a->head_dim, heads = a->n_kv_heads;
    if (slot <= 0 || (a->n_pages > 1 && a->page_stride % slot != 0)) return false;
    const int64_t page_rows = a->n_pages > 1 ? a->page_stride / slot : 0;
    int64_t head_rows = 0, head_cols = 0;
    cols = D;
    if ((heads - 1) * a->head_stride + D <= slot) {
        head_cols = heads > 1 ? a->head_stride : 0;
        cols = (heads - 1) * a->head_stride + D;
    } else if (a->head_stride % slot == 0 && D <= slot) {
        head_rows = a->head_stride / slot;
    } else {
        return false;
    }
    rows = (a->n_pages - 1) * page_rows + (heads - 1) * head_rows + a->page_size;
    if (rows > INT_MAX / 2 || cols > INT_MAX / 2 || slot * 2 >= (1ll << 40)) return false;
    M.page_rows = static_cast<int32_t>(page_rows);
    M.head_rows = static_cast<int32_t>(head_rows);
    M.head_cols = static_cast<int32_t>(head_cols);
    return true;
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

// box_rows: slots of a copied box (1 for gathering copies).
static bool encode_map(CUtensorMap &map, const void *cache, int64_t rows, int64_t cols, int64_t slot_stride, int box_rows) {
    const EncodeTiled encode = encode_tiled();
    if (!encode) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(slot_stride) * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)}, step[2] = {1, 1};
    return encode(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(cache), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct CacheMaps {
    tiles::CacheMap where;
    CUtensorMap k, v;
};

template <typename Kernel>
static cudaError_t launch_tensor(Kernel *kernel, int ctas, int threads, int smem, int stages, const AttendParams &P,
                                 const CacheMaps &M, cudaStream_t stream) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_after(kernel, dim3(static_cast<unsigned>(ctas)), dim3(static_cast<unsigned>(threads)),
                        static_cast<size_t>(smem), stream, P, M.where, M.k, M.v, stages);
}

// One class of items on the tensor cores.
template <bool PREFIX>
static cudaError_t launch_class(const AttendParams &P, const CacheMaps &M, cudaStream_t stream) {
    const int rt_log2 = PREFIX ? P.prefix_rt_log2 : P.own_rt_log2, workers = PREFIX ? P.prefix_workers : P.own_workers;
    if (rt_log2 == 5)
        return launch_tensor(round_::spec_attend_round_kernel<32, PREFIX>, workers, round_::kThreads,
                             round_::smem_bytes<32>(P.D), round_::stages<32>(P.D), P, M, stream);
    if (rt_log2 == 6)
        return launch_tensor(round_::spec_attend_round_kernel<64, PREFIX>, workers, round_::kThreads,
                             round_::smem_bytes<64>(P.D), round_::stages<64>(P.D), P, M, stream);
    return launch_tensor(pair::spec_attend_pair_kernel<PREFIX>, workers, pair::kThreads, pair::smem_bytes(P.D),
                         pair::stages(P.D), P, M, stream);
}

template <typename E, int NC, bool PREFIX>
static cudaError_t launch_fma(const AttendParams &P, cudaStream_t stream) {
    const int smem = fma::smem_floats(P.D) * 4;
    const cudaError_t e = cudaFuncSetAttribute(fma::spec_attend_fma_kernel<E, NC, PREFIX>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_after(fma::spec_attend_fma_kernel<E, NC, PREFIX>,
                        dim3(static_cast<unsigned>(PREFIX ? P.prefix_workers : P.own_workers)), dim3(fma::kThreads),
                        static_cast<size_t>(smem), stream, P);
}

template <typename E, int KT>
static cudaError_t launch_join(const AttendParams &P, cudaStream_t stream) {
    const bool shared = P.shared_len > 0;
    const int64_t blocks = shared ? (static_cast<int64_t>(P.T) * P.Hkv + kJoinWarps - 1) / kJoinWarps
                                  : static_cast<int64_t>(P.own_workers) * ((P.own_pitch + kJoinWarps - 1) / kJoinWarps);
    return launch_after(shared ? spec_attend_join_shared_kernel<E, KT> : spec_attend_join_kernel<E>,
                        dim3(static_cast<unsigned>(P.B + blocks)), dim3(kJoinThreads), 0, stream, P);
}

static cudaError_t enqueue_tensor(const AttendParams &P, const CacheMaps &M, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    if (P.shared_len > 0) e = launch_class<true>(P, M, stream);
    if (e == cudaSuccess) e = launch_class<false>(P, M, stream);
    if (e == cudaSuccess) e = launch_join<__nv_bfloat16, tiles::kKT>(P, stream);
    return e;
}

template <typename E>
static cudaError_t enqueue_fma(const AttendParams &P, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    const bool wide = P.D > 128;
    if (P.shared_len > 0) e = wide ? launch_fma<E, 2, true>(P, stream) : launch_fma<E, 1, true>(P, stream);
    if (e == cudaSuccess) e = wide ? launch_fma<E, 2, false>(P, stream) : launch_fma<E, 1, false>(P, stream);
    if (e == cudaSuccess) e = launch_join<E, fma::kKT>(P, stream);
    return e;
}

}  // namespace spec

using namespace spec;

extern "C" size_t spec_attend_workspace_size(const spec_attend_args *a) {
    AttendParams P = {};
    if (attend_sizes(a, P) != SPEC_OK) return 0;
    // either kernel may serve the call: which one follows from the strides
    attend_work(P, false);
    const size_t fma_bytes = attend_layout(P).total;
    if (a->dtype != SPEC_BF16) return fma_bytes;
    attend_work(P, true);
    return std::max(fma_bytes, attend_layout(P).total);
}

extern "C" const char *spec_attend_plan(const spec_attend_args *a) {
    AttendParams P = {};
    if (attend_sizes(a, P) != SPEC_OK) return nullptr;
    tiles::CacheMap M = {};
    int64_t rows = 0, cols = 0;
    if (!cache_map(a, M, rows, cols)) return "spec_attend_fma_kernel";
    attend_work(P, true);
    return P.own_rt_log2 == pair::kRTLog2 ? "spec_attend_pair_kernel" : "spec_attend_round_kernel";
}

extern "C" spec_status spec_attend(const spec_attend_args *a, void *workspace, size_t workspace_bytes,
                                   cudaStream_t stream) {
    AttendParams P = {};
    const spec_status st = attend_sizes(a, P);
    if (st != SPEC_OK) return st;
    if (!a->row_off || !a->kv_len || !a->block_table || !a->k_cache || !a->v_cache) return SPEC_ERR_INVALID_ARG;
    if (P.T > 0 && (!a->q || !a->out)) return SPEC_ERR_INVALID_ARG;
    if (P.shared_len > 0 && !a->shared_table) return SPEC_ERR_INVALID_ARG;
    const int64_t width = static_cast<int64_t>(P.Hq) * P.D;
    if (P.T > 1 && (a->q_stride < width || a->out_stride < width)) return SPEC_ERR_INVALID_ARG;
    if (a->page_stride < 0 || a->slot_stride < 0 || a->head_stride < 0) return SPEC_ERR_INVALID_ARG;
    const int vec = a->dtype == SPEC_BF16 ? 8 : 4;
    auto aligned = [](const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    if ((a->q_stride | a->out_stride | a->page_stride | a->slot_stride | a->head_stride) % vec != 0 || !aligned(a->q) ||
        !aligned(a->out) || !aligned(a->k_cache) || !aligned(a->v_cache))
        return SPEC_ERR_UNSUPPORTED;
    CacheMaps M = {};
    int64_t map_rows = 0, map_cols = 0;
    const bool tensor = cache_map(a, M.where, map_rows, map_cols);
    attend_work(P, tensor);
    const AttendLayout L = attend_layout(P);
    if (!workspace || workspace_bytes < spec_attend_workspace_size(a) || reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
        return SPEC_ERR_WORKSPACE;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
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
    P.status = reinterpret_cast<int32_t *>(ws + L.status);
    P.unit_prefix = reinterpret_cast<int32_t *>(ws + L.unit_prefix);
    P.cut = reinterpret_cast<CutItem *>(ws + L.cut);
    P.prefix_units = reinterpret_cast<int32_t *>(ws + L.prefix_units);
    P.broken = reinterpret_cast<int32_t *>(ws + L.broken);
    P.err = reinterpret_cast<int32_t *>(ws + L.err);
    P.part_ml = reinterpret_cast<float2 *>(ws + L.ml);
    P.part_o = reinterpret_cast<float *>(ws + L.o);
    if (tensor) {
        const int box = 1 << P.box_log2;
        if (!encode_map(M.k, a->k_cache, map_rows, map_cols, a->slot_stride, box) ||
            !encode_map(M.v, a->v_cache, map_rows, map_cols, a->slot_stride, box))
            return SPEC_ERR_CUDA;
        return enqueue_tensor(P, M, stream) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
    }
    const cudaError_t e =
        a->dtype == SPEC_BF16 ? enqueue_fma<__nv_bfloat16>(P, stream) : enqueue_fma<float>(P, stream);
    return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

#ifdef SPEC_DEBUG
namespace spec {
// The debug words of this translation unit's kernels.
cudaError_t debug_take_attend(unsigned int out[4]) { return spec_dbg_take(out); }
}  // namespace spec
#endif
