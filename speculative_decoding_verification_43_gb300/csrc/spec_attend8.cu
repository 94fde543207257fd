// Attention of a round's rows over the paged cache in 8 bits (spec_attend8). See include/spec_cache8.h for the
// contract, spec_attend_plan.cuh for how the work is cut, spec_attend.cu for the passes' mathematics.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

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

// Workers and parts of the kernels that serve the call.
static void attend8_work(AttendParams &P, bool tensor) {
    attend_fma_work(P);
    attend_parts(P);
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
    attend8_work(P, false);
    return attend_layout(P).total;
}

extern "C" const char *spec_attend8_plan(const spec_attend8_args *a) {
    AttendParams P = {};
    if (attend8_sizes(a, P) != SPEC_OK) return nullptr;
    return "spec_attend_fma_kernel";
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
    attend8_work(P, false);
    if (!workspace || workspace_bytes < spec_attend8_workspace_size(a) || reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
        return SPEC_ERR_WORKSPACE;
    attend_place(P, workspace);
    const cudaError_t e =
        a->attend.dtype == SPEC_BF16 ? enqueue_fma8<__nv_bfloat16>(P, stream) : enqueue_fma8<float>(P, stream);
    return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

#ifdef SPEC_DEBUG
namespace spec {
// The debug words of this translation unit's kernels.
cudaError_t debug_take_attend8(unsigned int out[4]) { return spec_dbg_take(out); }
}  // namespace spec
#endif
