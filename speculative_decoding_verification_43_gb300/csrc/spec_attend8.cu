// Attention of a round's rows over the paged cache in 8 bits (spec_attend8). See include/spec_cache8.h for the
// contract, spec_attend_plan.cuh for how the work is cut, spec_attend.cu for the passes' mathematics.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "spec_attend8_pair.cuh"
#include "spec_attend8_round.cuh"
#include "spec_attend8_tiles.cuh"
#include "spec_attend_fma.cuh"
#include "spec_attend_host.cuh"
#include "spec_attend_plan.cuh"
#include "spec_cache8.h"
#include "spec_device.cuh"

namespace spec {

// Sizes that spec_attend8 takes beside spec_attend's.
static spec_status attend8_sizes(const spec_attend8_args *a, AttendParams &P) {
    if (!a) return SPEC_ERR_INVALID_ARG;
    const spec_status st = attend_sizes(&a->attend, P);
    if (st != SPEC_OK) return st;
    return a->attend.head_dim % 16 == 0 ? SPEC_OK : SPEC_ERR_UNSUPPORTED;
}

// Rows of an item (as a power of two) and workers for `rows` packed rows of a head over `groups` requests on the
// tensor cores. By the average, because lengths are known on the device alone. Measured with 64 requests of 32 / 8 heads
// of 128 (us with items of 32, 64 and 256 rows):
//   packed rows of each request   32            48            64            96             128
//   up to 2000 positions          69 89 128     104 101 128   111 114 129   155 175 132    200 195 129
//   up to 8000                    169 201 279   289 236 283   308 275 284   449 463 302    591 523 305
//   rows that differ, average     30            34            53            66             93
//   up to 2000                    86 97 127     88 107 128    114 139 127   132 149 130    169 189 151
//   up to 8000                    226 240 280   238 266 282   324 356 301   378 388 302    500 511 411
// Between 32 and 48 the 64 rows win where the requests are alike and texts are long (a fifth) and lose where requests differ
// (a tenth, a fifth on short texts). The rule goes by rows alone: on texts to 2000 positions it gives up 16 % with 64 rows
// alike and 22 % with 34 that differ. All at one shape; heads of 64, whose products take half and whose weights do not, were
// not measured. fp32 rows need the room of 64 rows for their further parts.
static void tensor8_class(bool wide, int64_t rows, int64_t groups, int32_t &rt_log2, int32_t &workers) {
    rt_log2 = wide || rows <= 32 * groups ? 5 : rows <= 48 * groups ? 6 : pair8::kRTLog2;
    workers = rt_log2 == pair8::kRTLog2 ? kSMs : kSMs * round8::kPerSM;
}

// Time of an item beside its tiles, in tiles. (Flat: 64 round items of up to 4000 positions take 95 us with 0, 96 with 4,
// 103 with 16; prompts of 1000-2500 rows 460 us with 3, 456 with 4, 457 with 6, 474 with 8.)
constexpr int kExtra8 = 4;

// Workers and parts of the kernels that serve the call.
static void attend8_work(AttendParams &P, bool tensor, bool wide) {
    const int64_t head_rows = static_cast<int64_t>(P.T) * P.G;
    if (tensor) {
        tensor8_class(wide, head_rows, P.B, P.own_rt_log2, P.own_workers);
        tensor8_class(wide, head_rows, 1, P.prefix_rt_log2, P.prefix_workers);
        P.own_extra = P.prefix_extra = kExtra8;
        P.box_log2 = box_log2_of(P.page_size);
        // A slot's heads lie side by side, 128 bytes each: read at different times they cost DRAM more than their
        // bytes. So up to eight heads of the same positions are read in step, by workers that begin together: 16 requests
        // of up to 16000 positions take 106 us with heads apart, 98 with two, 96 with eight in step.
        if (P.shared_len == 0 && P.own_rt_log2 != pair8::kRTLog2)
            while (P.head_step < 8 && P.Hkv % (2 * P.head_step) == 0) P.head_step *= 2;
        P.own_workers -= P.own_workers % P.head_step;
    } else {
        attend_fma_work(P);
    }
    attend_parts(P);
}

// Whether the tensor cores may serve a call of these sizes; strides apart.
static bool tensor8_sizes(const spec_attend8_args *a) {
    return a->attend.head_dim <= 128 && box_log2_of(a->attend.page_size) > 0;
}

// The cache as three-dimensional tensor maps (head_dim x heads x slots), where its strides allow it: pages a whole
// number of slots apart, heads inside a slot or a whole number of slots apart. What a tile's rows have beyond
// head_dim comes as zeros, not as the next head's elements.
struct CacheShape {
    int64_t heads, head_stride, rows;
};
static bool cache_map8(const spec_attend8_args *args, tiles8::CacheMap &M, CacheShape &shape) {
    const spec_attend_args *a = &args->attend;
    if (!tensor8_sizes(args)) return false;
    const int64_t slot = a->slot_stride, D = a->head_dim, heads = a->n_kv_heads;
    if (slot <= 0 || (a->n_pages > 1 && a->page_stride % slot != 0)) return false;
    const int64_t page_rows = a->n_pages > 1 ? a->page_stride / slot : 0;
    int64_t head_rows = 0;
    shape = {1, slot, 0};
    M.head_step = 0;
    if (heads > 1 && a->head_stride >= D && (heads - 1) * a->head_stride + D <= slot) {
        shape.heads = heads;
        shape.head_stride = a->head_stride;
        M.head_step = 1;
    } else if (D <= slot && (heads == 1 || (a->head_stride > 0 && a->head_stride % slot == 0))) {
        head_rows = heads > 1 ? a->head_stride / slot : 0;
    } else {
        return false;
    }
    shape.rows = (a->n_pages - 1) * page_rows + (heads - 1) * head_rows + a->page_size;
    if (shape.rows > INT_MAX / 2 || slot >= (1ll << 40) || shape.head_stride >= (1ll << 40)) return false;
    M.page_rows = static_cast<int32_t>(page_rows);
    M.head_rows = static_cast<int32_t>(head_rows);
    return page_rows <= INT_MAX / 2 && head_rows <= INT_MAX / 2;
}
static bool encode_map8(CUtensorMap &map, const void *cache, const CacheShape &shape, const spec_attend_args *a, int box_rows) {
    const EncodeTiled encode = encode_tiled();
    if (!encode) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a->head_dim), static_cast<cuuint64_t>(shape.heads),
                                static_cast<cuuint64_t>(shape.rows)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(shape.head_stride), static_cast<cuuint64_t>(a->slot_stride)};
    const cuuint32_t box[3] = {128, 1, static_cast<cuuint32_t>(box_rows)}, step[3] = {1, 1, 1};
    // no more than the head's own bytes: promoted to 256, a read brought the next head's too, 1.4 times the bytes
    const CUtensorMapL2promotion promotion =
        a->head_dim > 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
    return encode(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(cache), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, promotion,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct CacheMaps8 {
    tiles8::CacheMap where;
    CUtensorMap k, v;
};

template <typename Kernel>
static cudaError_t launch_tensor8(Kernel *kernel, int ctas, int threads, int smem, const AttendParams &P, const CacheMaps8 &M,
                                  cudaStream_t stream) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_after(kernel, dim3(static_cast<unsigned>(ctas)), dim3(static_cast<unsigned>(threads)),
                        static_cast<size_t>(smem), stream, P, M.where, M.k, M.v);
}

template <int RT, bool PREFIX, bool WIDE>
static cudaError_t launch_round8(int workers, const AttendParams &P, const CacheMaps8 &M, cudaStream_t stream) {
    return launch_tensor8(round8::spec_attend8_round_kernel<RT, PREFIX, WIDE>, workers, round8::kThreads,
                          round8::smem_bytes<RT, WIDE>(), P, M, stream);
}
// One class of items on the tensor cores.
template <bool PREFIX>
static cudaError_t launch_class8(bool wide, const AttendParams &P, const CacheMaps8 &M, cudaStream_t stream) {
    const int rt_log2 = PREFIX ? P.prefix_rt_log2 : P.own_rt_log2, workers = PREFIX ? P.prefix_workers : P.own_workers;
    if (wide) return launch_round8<32, PREFIX, true>(workers, P, M, stream);
    if (rt_log2 == 5) return launch_round8<32, PREFIX, false>(workers, P, M, stream);
    if (rt_log2 == 6) return launch_round8<64, PREFIX, false>(workers, P, M, stream);
    return launch_tensor8(pair8::spec_attend8_pair_kernel<PREFIX>, workers, pair8::kThreads, pair8::kSmem, P, M, stream);
}

static cudaError_t enqueue_tensor8(bool wide, const AttendParams &P, const CacheMaps8 &M, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    if (P.shared_len > 0) e = launch_class8<true>(wide, P, M, stream);
    if (e == cudaSuccess) e = launch_class8<false>(wide, P, M, stream);
    if (e == cudaSuccess)
        e = wide ? launch_join<float, tiles8::kKT>(P, stream) : launch_join<__nv_bfloat16, tiles8::kKT>(P, stream);
    return e;
}

template <typename E, int NC, bool PREFIX>
static cudaError_t launch_fma8(const AttendParams &P, cudaStream_t stream) {
    const int smem = fma::smem_floats(P.D) * 4;
    const auto kernel = fma::spec_attend_fma_kernel<E, __nv_fp8_e4m3, NC, PREFIX>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_after(kernel, dim3(static_cast<unsigned>(PREFIX ? P.prefix_workers : P.own_workers)), dim3(fma::kThreads),
                        static_cast<size_t>(smem), stream, P);
}

template <typename E>
static cudaError_t enqueue_fma8(const AttendParams &P, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    const bool wide = P.D > 128;
    if (P.shared_len > 0) e = wide ? launch_fma8<E, 2, true>(P, stream) : launch_fma8<E, 1, true>(P, stream);
    if (e == cudaSuccess) e = wide ? launch_fma8<E, 2, false>(P, stream) : launch_fma8<E, 1, false>(P, stream);
    if (e == cudaSuccess) e = launch_join<E, fma::kKT>(P, stream);
    return e;
}

}  // namespace spec

using namespace spec;

extern "C" size_t spec_attend8_workspace_size(const spec_attend8_args *a) {
    AttendParams P = {};
    if (attend8_sizes(a, P) != SPEC_OK) return 0;
    // either kernel may serve the call: which one follows from the strides
    const bool wide = a->attend.dtype == SPEC_F32;
    attend8_work(P, false, wide);
    const size_t fma_bytes = attend_layout(P).total;
    if (!tensor8_sizes(a)) return fma_bytes;
    attend8_work(P, true, wide);
    return std::max(fma_bytes, attend_layout(P).total);
}

extern "C" const char *spec_attend8_plan(const spec_attend8_args *a) {
    AttendParams P = {};
    if (attend8_sizes(a, P) != SPEC_OK) return nullptr;
    tiles8::CacheMap M = {};
    CacheShape shape = {};
    if (!cache_map8(a, M, shape)) return "spec_attend_fma_kernel";
    attend8_work(P, true, a->attend.dtype == SPEC_F32);
    return P.own_rt_log2 == pair8::kRTLog2 ? "spec_attend8_pair_kernel" : "spec_attend8_round_kernel";
}

extern "C" spec_status spec_attend8(const spec_attend8_args *a, void *workspace, size_t workspace_bytes,
                                    cudaStream_t stream) {
    AttendParams P = {};
    spec_status st = attend8_sizes(a, P);
    if (st != SPEC_OK) return st;
    if (!a->k_scale || !a->v_scale) return SPEC_ERR_INVALID_ARG;
    st = attend_pointers(&a->attend, P, a->attend.dtype == SPEC_BF16 ? 8 : 4, 16);
    if (st != SPEC_OK) return st;
    P.k_scale = a->k_scale;
    P.v_scale = a->v_scale;
    CacheMaps8 M = {};
    CacheShape shape = {};
    const bool tensor = cache_map8(a, M.where, shape);
    const bool wide = a->attend.dtype == SPEC_F32;
    attend8_work(P, tensor, wide);
    if (!workspace || workspace_bytes < spec_attend8_workspace_size(a) || reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
        return SPEC_ERR_WORKSPACE;
    attend_place(P, workspace);
    if (tensor) {
        const int box = 1 << P.box_log2;
        if (!encode_map8(M.k, a->attend.k_cache, shape, &a->attend, box) ||
            !encode_map8(M.v, a->attend.v_cache, shape, &a->attend, box))
            return SPEC_ERR_CUDA;
        return enqueue_tensor8(wide, P, M, stream) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
    }
    const cudaError_t e =
        wide ? enqueue_fma8<float>(P, stream) : enqueue_fma8<__nv_bfloat16>(P, stream);
    return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

#ifdef SPEC_DEBUG
namespace spec {
// The debug words of this translation unit's kernels.
cudaError_t debug_take_attend8(unsigned int out[4]) { return spec_dbg_take(out); }
}  // namespace spec
#endif
