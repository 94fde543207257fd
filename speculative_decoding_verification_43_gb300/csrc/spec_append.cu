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

#include "spec_append.cuh"
#include "spec_attend.h"
#include "spec_device.cuh"
#include "spec_paged.cuh"

namespace spec {

constexpr int kAppendThreads = 256, kAppendWarps = kAppendThreads / kWarp, kAppendPerSM = 4;

// One thread moves the same part of a row (its task) for every row of its column of blocks: a pair
// of pieces c and c + rot/2 that turn together, a piece of interleaved pairs, or a piece that is
// copied. V: elements per piece (16 bytes, or 1 when something is not on 16-byte boundaries).
//
// Bound by latency when there are few rows (offsets -> length -> page -> store is a chain of
// dependent loads; a row's own values are requested before it): 2.5 us for 5 rows, 4.6 us for 290 rows of
// 32 + 2 x 8 heads of 128 in bf16. By DRAM when there are many: 12935 rows of 48 heads of 64, 153 MB, in 29.7
// us, 0.77 of the measured copy rate. One element at a time (V = 1) 288 rows of 32 + 2 x 8 heads of 80, 40
// columns turned, take 6.1 us; 4.6 with all 80 turned, in pieces of 16 bytes. Four blocks an SM leave a thread 64 registers; six (40) spilled, and
// finding every row's slot in turn, without the next row's values under way, took 39 us.
template <typename E, int V, bool INTER>
__global__ void __launch_bounds__(kAppendThreads, kAppendPerSM) spec_append_kernel(const AppendParams P) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x % kWarp;
    // Whether some request's offsets are wrong: the first ones are asked for here and looked at where the block
    // has other reads to wait for.
    int off0 = 0, off1 = 0;
    if (static_cast<int>(threadIdx.x) < P.B) {
        off0 = P.row_off[threadIdx.x];
        off1 = P.row_off[threadIdx.x + 1];
    }
    auto some_wrong = [&]() -> bool {
        bool wrong = !offsets_right(off0, off1, P.T);
#pragma unroll 4
        for (int i = threadIdx.x + kAppendThreads; i < P.B; i += kAppendThreads)
            wrong |= !offsets_right(P.row_off[i], P.row_off[i + 1], P.T);
        return __syncthreads_or(wrong) != 0;
    };
    // by a warp, where some are
    auto in_doubt = [&](int i) -> bool {
        return __any_sync(0xffffffffu, offsets_contradict(P.row_off, P.B, P.T, i, P.row_off[i], P.row_off[i + 1], lane,
                                                          kWarp)) != 0;
    };
    if (blockIdx.x == static_cast<unsigned>(P.copy_blocks)) {
        const bool broken = some_wrong();
        // the requests' status, a warp each
        for (int i = blockIdx.y * kAppendWarps + threadIdx.x / kWarp; i < P.B; i += gridDim.y * kAppendWarps) {
            const int st = append_status(P, i, lane, [&](int r) { return broken && in_doubt(r); });
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
    using Vec = Piece<E, V>;

    // Rows in batches of as many as there are warps: each warp finds one row's position and slot (a chain of
    // dependent reads: offsets, length, page), then all threads move the rows, the next row's values under
    // way while one is turned and stored. A block with a single row has every warp find it, without meeting.
    __shared__ int64_t slot_of[kAppendWarps];  // element offset of the row's slot, -1: not written
    __shared__ int pos_of[kAppendWarps];
    const int step = gridDim.y, warp = threadIdx.x / kWarp;
    const bool single = step >= P.T;
    bool broken = false;
    for (int first = blockIdx.y; first < P.T; first += kAppendWarps * step) {
        Vec a = {}, b = {};
        auto fetch = [&](int r) {
            if (!have || r >= P.T) return;
            a = *reinterpret_cast<const Vec *>(src + r * src_stride + d0);
            if (two) b = *reinterpret_cast<const Vec *>(src + r * src_stride + d1);
        };
        fetch(first);
        const int mine = single ? first : first + warp * step;
        int64_t my_slot = -1;
        int my_pos = 0;
        if (mine < P.T) {
            const int i = find_request(P.row_off, P.B, P.T, mine, lane);
            const int r0 = P.row_off[i], r1 = P.row_off[i + 1], kv = P.kv_len[i];
            const int pos = kv - (r1 - r0) + (mine - r0);
            if (offsets_right(r0, r1, P.T) && mine >= r0 && mine < r1 && kv >= 0 && pos >= 0 && pos < P.n_pos) {
                const int blk = pos / P.page_size;
                if (blk < P.max_blocks) {
                    const int page = P.block_table[static_cast<int64_t>(i) * P.max_blocks + blk];
                    if (page >= 0 && page < P.n_pages)
                        my_slot = page * P.page_stride + (pos - blk * P.page_size) * P.slot_stride;
                }
            }
            my_pos = pos;
            if (lane == 0 && !single) {
                slot_of[warp] = my_slot;
                pos_of[warp] = my_pos;
            }
        }
        if (first == static_cast<int>(blockIdx.y))
            broken = some_wrong();
        else
            __syncthreads();
        if (broken) {
            if (my_slot >= 0 && in_doubt(find_request(P.row_off, P.B, P.T, mine, lane))) {
                my_slot = -1;
                if (lane == 0) slot_of[warp] = -1;
            }
            __syncthreads();
        }
#pragma unroll 1
        for (int j = 0; j < kAppendWarps; ++j) {
            const int r = first + j * step;
            if (r >= P.T) break;
            Vec x = a, y = b;
            if (j + 1 < kAppendWarps) fetch(r + step);
            const int64_t slot = single ? my_slot : slot_of[j];
            if (!have || slot < 0) continue;
            if (rotates && SPEC_IN(single ? my_pos : pos_of[j], P.n_pos, DBG_CACHE)) {
                constexpr int NC = kPairs ? V : (V + 1) / 2;
                float c[NC], s[NC];
                const float *cs = P.cos_sin + static_cast<int64_t>(single ? my_pos : pos_of[j]) * P.rot + c0;
                load_floats(c, cs);
                load_floats(s, cs + P.rot / 2);
                float u[V];
                unpack(x, u);
                if constexpr (kPairs) {
                    float w[V];
                    unpack(y, w);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float t = u[e];
                        u[e] = t * c[e] - w[e] * s[e];
                        w[e] = w[e] * c[e] + t * s[e];
                    }
                    pack(y, w);
                } else {
#pragma unroll
                    for (int e = 0; e < NC; ++e) {
                        const float t = u[2 * e];
                        u[2 * e] = t * c[e] - u[2 * e + 1] * s[e];
                        u[2 * e + 1] = u[2 * e + 1] * c[e] + t * s[e];
                    }
                }
                pack(x, u);
            }
            E *base = what == Q ? static_cast<E *>(P.q_out) : cache;
            const int64_t at =
                what == Q ? r * P.q_out_stride + static_cast<int64_t>(head) * P.D : slot + head * P.head_stride;
            auto inside = [&](int d) -> bool {
                return SPEC_IN(d + V - 1, P.D, DBG_CACHE) &&
                       (what == Q ? SPEC_IN(r, P.T, DBG_OUT_ROWS) && SPEC_IN(head, P.Hq, DBG_OUT_ROWS)
                                  : SPEC_IN(at, cache_extent(P), DBG_CACHE) &&
                                        SPEC_IN(at + d + V - 1, cache_extent(P), DBG_CACHE));
            };
            if (inside(d0)) *reinterpret_cast<Vec *>(base + at + d0) = x;
            if (two && inside(d1)) *reinterpret_cast<Vec *>(base + at + d1) = y;
        }
        if (!single) __syncthreads();  // the batch's slots have been read
    }
}

template <typename E, int V, bool INTER>
static spec_status launch_append(AppendParams &P, cudaStream_t stream) {
    constexpr bool kPairs = !INTER || V == 1;
    const int turn = kPairs ? P.rot / 2 / V : P.rot / V;
    const int tasks = (P.Hq + P.Hkv) * (turn + (P.D - P.rot) / V) + P.Hkv * (P.D / V);
    P.copy_blocks = (tasks + kAppendThreads - 1) / kAppendThreads;
    // a block a row until the device is full (152 SMs), then blocks walk rows, all about as many
    const int most = std::max(1, 152 * kAppendPerSM / P.copy_blocks), turns = std::max(1, (P.T + most - 1) / most);
    const int rows = std::max(1, (P.T + turns - 1) / turns);
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
    AppendParams P = {};
    const spec_status st = append_params(a, P);
    if (st != SPEC_OK) return st;
    return a->dtype == SPEC_BF16 ? dispatch_append<__nv_bfloat16>(P, a->interleaved != 0, stream)
                                 : dispatch_append<float>(P, a->interleaved != 0, stream);
}

#ifdef SPEC_DEBUG
namespace spec {
// The debug words of this translation unit's kernel.
cudaError_t debug_take_append(unsigned int out[4]) { return spec_dbg_take(out); }
}  // namespace spec
#endif
