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
#include "spec_attend_host.cuh"
#include "spec_attend_pair.cuh"
#include "spec_attend_plan.cuh"
#include "spec_attend_round.cuh"
#include "spec_device.cuh"
#include "spec_paged.cuh"

namespace spec {

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
        P.box_log2 = box_log2_of(P.page_size);
    } else {
        attend_fma_work(P);
    }
    attend_parts(P);
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
    const cudaError_t e = cudaFuncSetAttribute(fma::spec_attend_fma_kernel<E, E, NC, PREFIX>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_after(fma::spec_attend_fma_kernel<E, E, NC, PREFIX>,
                        dim3(static_cast<unsigned>(PREFIX ? P.prefix_workers : P.own_workers)), dim3(fma::kThreads),
                        static_cast<size_t>(smem), stream, P);
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
    const int vec = a->dtype == SPEC_BF16 ? 8 : 4;
    const spec_status ptrs = attend_pointers(a, P, vec, vec);
    if (ptrs != SPEC_OK) return ptrs;
    CacheMaps M = {};
    int64_t map_rows = 0, map_cols = 0;
    const bool tensor = cache_map(a, M.where, map_rows, map_cols);
    attend_work(P, tensor);
    if (!workspace || workspace_bytes < spec_attend_workspace_size(a) || reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
        return SPEC_ERR_WORKSPACE;
    attend_place(P, workspace);
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
