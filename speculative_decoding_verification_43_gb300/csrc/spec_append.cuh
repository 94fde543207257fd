// What appending to the paged cache shares, whatever type the cache has: the call's parameters, rows in pieces of
// 16 bytes, and the requests' status.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

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

// V consecutive elements of E as they lie in memory: 16 bytes, or one element.
template <typename E, int V>
struct Piece {
    uint4 w;
};
template <typename E>
struct Piece<E, 1> {
    E w;
};
__device__ __forceinline__ void unpack(const Piece<__nv_bfloat16, 8> &p, float (&f)[8]) {
    const uint32_t w[4] = {p.w.x, p.w.y, p.w.z, p.w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack(const Piece<float, 4> &p, float (&f)[4]) {
    f[0] = __uint_as_float(p.w.x);
    f[1] = __uint_as_float(p.w.y);
    f[2] = __uint_as_float(p.w.z);
    f[3] = __uint_as_float(p.w.w);
}
__device__ __forceinline__ void unpack(const Piece<__nv_bfloat16, 1> &p, float (&f)[1]) { f[0] = __bfloat162float(p.w); }
__device__ __forceinline__ void unpack(const Piece<float, 1> &p, float (&f)[1]) { f[0] = p.w; }
__device__ __forceinline__ void pack(Piece<__nv_bfloat16, 8> &p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    p.w = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void pack(Piece<float, 4> &p, const float (&f)[4]) {
    p.w = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ void pack(Piece<__nv_bfloat16, 1> &p, const float (&f)[1]) { p.w = __float2bfloat16_rn(f[0]); }
__device__ __forceinline__ void pack(Piece<float, 1> &p, const float (&f)[1]) { p.w = f[0]; }

// Floats of the cos_sin table, as wide as their alignment allows.
template <int N>
__device__ __forceinline__ void load_floats(float (&out)[N], const float *p) {
#pragma unroll
    for (int i = 0; i < N; i += (N % 4 == 0 ? 4 : N % 2 == 0 ? 2 : 1)) {
        if constexpr (N % 4 == 0) {
            const float4 x = *reinterpret_cast<const float4 *>(p + i);
            out[i] = x.x;
            out[i + 1] = x.y;
            out[i + 2] = x.z;
            out[i + 3] = x.w;
        } else if constexpr (N % 2 == 0) {
            const float2 x = *reinterpret_cast<const float2 *>(p + i);
            out[i] = x.x;
            out[i + 1] = x.y;
        } else {
            out[i] = p[i];
        }
    }
}

// Status of request i of an append, by one warp. in_doubt: rows that other offsets leave in doubt.
template <typename Doubt>
__device__ __forceinline__ int append_status(const AppendParams &P, int i, int lane, const Doubt &in_doubt) {
    const int r0 = P.row_off[i], r1 = P.row_off[i + 1], kv = P.kv_len[i];
    if (!offsets_right(r0, r1, P.T) || kv < 0 || in_doubt(i)) return SPEC_REQ_BAD_SHAPE;
    if (r1 == r0 || kv == 0) return SPEC_REQ_OK;
    int st = kv > P.n_pos ? SPEC_REQ_BAD_SHAPE : SPEC_REQ_OK;
    const int b1 = (kv - 1) / P.page_size;
    if (b1 >= P.max_blocks) st |= SPEC_REQ_BAD_BLOCKS;
    bool bad = false;
    for (int b = max(0, kv - (r1 - r0)) / P.page_size + lane; b <= min(b1, P.max_blocks - 1); b += kWarp) {
        const int page = P.block_table[static_cast<int64_t>(i) * P.max_blocks + b];
        bad |= page < 0 || page >= P.n_pages;
    }
    if (__any_sync(0xffffffffu, bad)) st |= SPEC_REQ_BAD_BLOCKS;
    return st;
}

// The arguments checked and taken over, all but the alignments.
static spec_status append_params(const spec_kv_append_args *a, AppendParams &P) {
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
    return SPEC_OK;
}

}  // namespace spec
