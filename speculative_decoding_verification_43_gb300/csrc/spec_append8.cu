// Appending a round's keys and values to the paged cache in 8 bits (spec_kv_append8). See include/spec_cache8.h
// for the contract, spec_append.cu for the rotation.
//
// A page's values of one head share a scale s, the least power of two with |x| <= 448 s. A power of two loses
// nothing against any other scale: e4m3 has an exponent of its own, so only the values below s / 64, which it
// holds with fewer bits, depend on s at all. And it keeps what is in a page exact when a later token needs a
// larger scale: c s = (c s / s') s', and dividing by a power of two changes the exponent alone (down to
// 2^-6; below that the value is rounded again).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "spec_append.cuh"
#include "spec_cache8.h"
#include "spec_device.cuh"
#include "spec_fp8.cuh"
#include "spec_paged.cuh"

namespace spec {

struct Append8Params : AppendParams {
    float *k_scale, *v_scale;   // [n_pages][Hkv]
    FastDiv by_page, by_k, by_v;  // by page_size; by the tasks of a head's row, keys (or queries) and values
    int32_t page_units, q_units;  // warps of pages and of query rows; the requests' status after them
};

constexpr int kAppend8Threads = 256, kAppend8Warps = kAppend8Threads / kWarp, kLookAlone = 256;

// Pages that a call touches, as candidates: request i's page number k is candidate
//     2 i + row_off[i] / page_size + k.
// n rows touch n / page_size + 2 pages at most (rounded down), and the next request's candidates begin
// 2 + floor(r1 / page_size) - floor(r0 / page_size) >= 2 + floor(n / page_size) further on. The request of
// candidate c is the last one whose first candidate is not above c; what find_request says of offsets out of
// order holds here too, as the candidates' order follows the offsets'.
__device__ __forceinline__ int64_t first_candidate(const Append8Params &P, int i) {
    return 2ll * i + P.by_page(offset_from(P.row_off, P.B, P.T, i));
}
__device__ __forceinline__ int find_candidate(const Append8Params &P, int c, int lane) {
    int lo = 0, n = P.B;
#pragma unroll 1
    while (n > 1) {
        const int step = (n + kWarp - 1) / kWarp;
        const int x = lane * step;
        const bool le = x < n && first_candidate(P, lo + x) <= c;
        const int k = max(__popc(__ballot_sync(0xffffffffu, le)) - 1, 0);
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}

// Part of a head's row: a pair of pieces that turn together, a piece of interleaved pairs, or a piece as it is.
template <int V, bool INTER>
struct Task {
    static constexpr bool kPairs = !INTER || V == 1;
    int d0, d1, c0;
    bool rotates, two;
    __device__ __forceinline__ Task(const AppendParams &P, int x, bool turned) {
        const int turn = turned ? (kPairs ? P.rot / 2 / V : P.rot / V) : 0;
        rotates = x < turn;
        two = kPairs && rotates;
        d1 = c0 = 0;
        if (!rotates) {
            d0 = (turned ? P.rot : 0) + (x - turn) * V;
        } else if (!INTER) {
            d0 = c0 = x * V;
            d1 = d0 + P.rot / 2;
        } else {
            d0 = V == 1 ? 2 * x : x * V;
            d1 = d0 + 1;
            c0 = d0 / 2;
        }
    }
};
// Turns the values of a task by position pos: u (and w, with two pieces).
template <int V, bool INTER>
__device__ __forceinline__ void turn(const AppendParams &P, const Task<V, INTER> &t, int pos, float (&u)[V], float (&w)[V]) {
    if (!t.rotates || !SPEC_IN(pos, P.n_pos, DBG_CACHE)) return;
    constexpr bool kPairs = Task<V, INTER>::kPairs;
    constexpr int NC = kPairs ? V : (V + 1) / 2;
    float c[NC], s[NC];
    const float *cs = P.cos_sin + static_cast<int64_t>(pos) * P.rot + t.c0;
    load_floats(c, cs);
    load_floats(s, cs + P.rot / 2);
    if constexpr (kPairs) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float x = u[e];
            u[e] = x * c[e] - w[e] * s[e];
            w[e] = w[e] * c[e] + x * s[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < NC; ++e) {
            const float x = u[2 * e];
            u[2 * e] = x * c[e] - u[2 * e + 1] * s[e];
            u[2 * e + 1] = u[2 * e + 1] * c[e] + x * s[e];
        }
    }
}

// V values to e4m3 at p. strange: there is an infinity among the unit's values, which must become NaN as well (x + 0 x
// is x, and not a number where x is not finite).
template <int V>
__device__ __forceinline__ void store8(unsigned char *p, const float (&x)[V], float scale, float inv, bool strange) {
    float y[V];
#pragma unroll
    for (int e = 0; e < V; ++e) y[e] = x[e] * inv;
    if (inv == 0.0f)  // (no power of two: the product would not be the quotient)
#pragma unroll
        for (int e = 0; e < V; ++e) y[e] = __fdiv_rn(x[e], scale);
    if (strange)
#pragma unroll
        for (int e = 0; e < V; ++e) y[e] = fmaf(x[e], 0.0f, y[e]);
    if constexpr (V == 1) {
        *p = static_cast<unsigned char>(to_e4m3(y[0], 0.0f));
    } else {
        uint32_t w[V / 4];
#pragma unroll
        for (int e = 0; e < V; e += 4)
            w[e / 4] = to_e4m3(y[e], y[e + 1]) | static_cast<uint32_t>(to_e4m3(y[e + 2], y[e + 3])) << 16;
        if constexpr (V == 8)
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint32_t *>(p) = w[0];
    }
}
// The scale's reciprocal where it is a power of two whose reciprocal is a normal number, else 0.
__device__ __forceinline__ float exact_reciprocal(float s) {
    const uint32_t b = __float_as_uint(s), e = b >> 23;
    return (b & 0x7fffffu) == 0 && e >= 1 && e <= 253 ? __uint_as_float((254u - e) << 23) : 0.0f;
}
// The largest magnitude, NaN aside. finite: infinities aside too.
template <int V>
__device__ __forceinline__ float top_of(const float (&x)[V], float top, bool finite) {
    if (!finite) {
#pragma unroll
        for (int e = 0; e < V; ++e) top = fmaxf(top, fabsf(x[e]));
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) top = isfinite(x[e]) ? fmaxf(top, fabsf(x[e])) : top;
    }
    return top;
}
// The values of one head in one page, by a warp: rows [row, row + n) at positions x0 .., `kept` earlier slots of the
// page. KEYS: turned on the way. A lane has one part of the head's row (or one after the other) for every r_step-th
// row. The first kHold rows' loads are under way together, and their values stay in registers until the scale is known;
// more are read and turned again (from L1 or L2).
template <typename E, int V, bool INTER, bool KEYS>
__device__ __forceinline__ void append_page(const Append8Params &P, int head, int row, int n, int x0, int kept, int page,
                                            int lane) {
    using Vec = Piece<E, V>;
    constexpr bool kTwo = KEYS && Task<V, INTER>::kPairs;
    constexpr int kHold = V == 1 ? 2 : 16 / (kTwo ? 2 * V : V);
    const int per = KEYS && Task<V, INTER>::kPairs ? P.D / V - P.rot / 2 / V : P.D / V;
    const int cols = min(per, kWarp), r_first = lane / cols, r_step = kWarp / cols, x_first = lane - r_first * cols;
    const int rows = r_first < r_step ? n : 0;  // (lanes that are left over have none)
    const int64_t stride = KEYS ? P.k_stride : P.v_stride;
    const E *src = static_cast<const E *>(KEYS ? P.k : P.v) + row * stride + static_cast<int64_t>(head) * P.D;

    auto fetch = [&](const Task<V, INTER> &t, int r, Vec &a, Vec &b) {
        const E *p = src + r * stride;
        a = *reinterpret_cast<const Vec *>(p + t.d0);
        if (kTwo && t.two) b = *reinterpret_cast<const Vec *>(p + t.d1);
    };
    auto values = [&](const Task<V, INTER> &t, int r, const Vec &a, const Vec &b, float (&u)[V], float (&w)[V]) {
        unpack(a, u);
        if constexpr (kTwo) unpack(b, w);  // (zeros with a single piece)
        if constexpr (KEYS) turn<V, INTER>(P, t, x0 + r, u, w);
    };
    Task<V, INTER> first(P, x_first, KEYS);
    Vec a[kHold], b[kTwo ? kHold : 1];
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
        a[i] = {};
        b[kTwo ? i : 0] = {};
        if (r_first + i * r_step < rows) fetch(first, r_first + i * r_step, a[i], b[kTwo ? i : 0]);
    }
    if (page < 0) return;  // (its number has been on its way with the values)
    const int64_t slot = page * P.page_stride;
    unsigned char *cache = static_cast<unsigned char *>(KEYS ? P.k_cache : P.v_cache) + slot + head * P.head_stride;
    float *scale_at = (KEYS ? P.k_scale : P.v_scale) + static_cast<int64_t>(page) * P.Hkv + head;
    const float old = kept > 0 ? *scale_at : 0.0f;

    float u[kHold][V], w[kTwo ? kHold : 1][V];
#pragma unroll
    for (int i = 0; i < kHold; ++i)
        if (i * r_step < n) values(first, min(r_first + i * r_step, n - 1), a[i], b[kTwo ? i : 0], u[i], w[kTwo ? i : 0]);
    // calls f(task, row, values) for all of the lane's
    auto all = [&](auto &&f) {
#pragma unroll
        for (int i = 0; i < kHold; ++i)
            if (r_first + i * r_step < rows) f(first, r_first + i * r_step, u[i], w[kTwo ? i : 0]);
        if (kHold * r_step < n || per > kWarp) {
#pragma unroll 1
            for (int x = x_first; x < per; x += kWarp) {
                const Task<V, INTER> t(P, x, KEYS);
#pragma unroll 2
                for (int r = r_first + (x == x_first ? kHold * r_step : 0); r < rows; r += r_step) {
                    Vec c = {}, d = {};
                    float y[V], z[V];
                    fetch(t, r, c, d);
                    values(t, r, c, d, y, z);
                    f(t, r, y, z);
                }
            }
        }
    };
    float top = 0.0f;
    bool strange = false;
#pragma unroll 1
    for (;;) {  // once; twice with an infinity
        top = 0.0f;
        all([&](const Task<V, INTER> &t, int, const float (&y)[V], const float (&z)[V]) {
            top = top_of<V>(y, top, strange);
            if (kTwo && t.two) top = top_of<V>(z, top, strange);
        });
        top = warp_max(top);
        if (top < INFINITY) break;
        strange = true;
    }
    const float scale = fmaxf(e4m3_scale(top), old), inv = exact_reciprocal(scale);
    if (lane == 0 && scale != old) *scale_at = scale;
    all([&](const Task<V, INTER> &t, int r, const float (&u)[V], const float (&w)[V]) {
        unsigned char *p = cache + (kept + r) * P.slot_stride;
        auto inside = [&](int d) -> bool {
            return SPEC_IN(d + V - 1, P.D, DBG_CACHE) &&
                   SPEC_IN(slot + (kept + r) * P.slot_stride + head * P.head_stride + d + V - 1, cache_extent(P), DBG_CACHE);
        };
        if (inside(t.d0)) store8<V>(p + t.d0, u, scale, inv, strange);
        if (kTwo && t.two && inside(t.d1)) store8<V>(p + t.d1, w, scale, inv, strange);
    });
    if (kept > 0 && scale != old) {
        // the earlier tokens' values under the new scale
        const float by_old = __fdiv_rn(old, scale);
        const int pieces = P.D / V;
#pragma unroll 1
        for (int idx = lane; idx < kept * pieces; idx += kWarp) {
            const int r = P.by_v(idx), d = (idx - r * pieces) * V;
            if (!SPEC_IN(slot + r * P.slot_stride + head * P.head_stride + d + V - 1, cache_extent(P), DBG_CACHE)) continue;
            unsigned char *p = cache + r * P.slot_stride + d;
            float x[V];
            if constexpr (V == 1) {
                x[0] = e4m3_to_float2(*p).x;
            } else {
#pragma unroll
                for (int e = 0; e < V; e += 4) {
                    const float4 f = e4m3_to_float4(*reinterpret_cast<const uint32_t *>(p + e));
                    x[e] = f.x;
                    x[e + 1] = f.y;
                    x[e + 2] = f.z;
                    x[e + 3] = f.w;
                }
            }
#pragma unroll
            for (int e = 0; e < V; ++e) x[e] *= by_old;
            store8<V>(p, x, 1.0f, 1.0f, false);
        }
    }
}

// A warp's work is a page's keys or values of one head (a candidate page that is none ends at once), a row's queries, or
// a request's status. Between the search for the largest and the rounding 16 values a lane stay in registers: in bf16 the first
// 4 of a page's 16 rows with heads of 128, 8 of 64 with heads of 64. The other rows are read twice (from L1 or L2 the second
// time), and keys turned twice, angles included.
// Pages of one head each, because a scale is one head's, and a warp each, because a round touches a page or two of
// each request (a CTA of eight warps a page was slower, for prompts as well).
// Measured (us a call, back to back): 5 rows of 32 / 8 heads of 128 6.3 (the host's call; 4.2 in a graph of calls), 64 requests
// of 1-8 rows 6.8-7.4 (7.7 MB; the chain offsets -> candidate -> page -> values -> scale -> stores, launch included), 6
// prompts of 500-4000 rows, 12 heads of 64, 30 (97 MB, 3.3 TB/s, 0.49 of the copy rate): there the warps wait for their
// loads, the second ones among them, so that it counts how many warps there are (CTAS an SM): 38 us with two (117
// registers), 36 with three, 30 with four (64). Rounds have few, and four's spills cost them more than they bring: 7.9, 6.8,
// 7.8; 256 requests of 4 fp32 rows 8.5, 8.1, 8.6.
template <typename E, int V, bool INTER, int CTAS>
__global__ void __launch_bounds__(kAppend8Threads, CTAS) spec_append8_kernel(const __grid_constant__ Append8Params P) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x % kWarp;
    // whether some request's offsets are wrong: each warp looks for itself where there are few, so that none waits
    bool broken = false;
    if (P.B <= kLookAlone) {
#pragma unroll 4
        for (int i = lane; i < P.B; i += kWarp) broken |= !offsets_right(P.row_off[i], P.row_off[i + 1], P.T);
        broken = __any_sync(0xffffffffu, broken) != 0;
    } else {
#pragma unroll 4
        for (int i = threadIdx.x; i < P.B; i += kAppend8Threads) broken |= !offsets_right(P.row_off[i], P.row_off[i + 1], P.T);
        broken = __syncthreads_or(broken) != 0;
    }
    auto in_doubt = [&](int i) -> bool {
        return broken && __any_sync(0xffffffffu, offsets_contradict(P.row_off, P.B, P.T, i, P.row_off[i], P.row_off[i + 1],
                                                                    lane, kWarp)) != 0;
    };
    // request i's first position, or -1 where it has no rows that are its own
    struct Request {
        int r0, n, kv, base;
    };
    auto request = [&](int i) -> Request {
        const int r0 = P.row_off[i], r1 = P.row_off[i + 1], kv = P.kv_len[i];
        if (!offsets_right(r0, r1, P.T) || kv < 0 || in_doubt(i)) return {0, 0, 0, 0};
        return {r0, r1 - r0, kv, kv - (r1 - r0)};
    };
    auto page_of = [&](int i, int blk) -> int {
        if (blk >= P.max_blocks) return -1;
        const int page = P.block_table[static_cast<int64_t>(i) * P.max_blocks + blk];
        return page < P.n_pages ? page : -1;
    };
    int unit = blockIdx.x * kAppend8Warps + threadIdx.x / kWarp;
    if (unit < P.page_units) {
        const int c = unit / (2 * P.Hkv), which = unit - c * 2 * P.Hkv, head = which >> 1;
        const int i = find_candidate(P, c, lane);
        const Request q = request(i);
        const int64_t k = c - (2ll * i + P.by_page(q.r0));
        if (q.n == 0 || q.kv == 0 || k < 0) return;
        const int from = max(q.base, 0), blk = P.by_page(from) + static_cast<int>(k);
        const int64_t begin = static_cast<int64_t>(blk) * P.page_size;
        const int x0 = static_cast<int>(max(begin, static_cast<int64_t>(from)));
        const int x1 = static_cast<int>(min(begin + P.page_size, static_cast<int64_t>(min(q.kv, P.n_pos))));
        if (begin >= q.kv || x0 >= x1) return;
        const int page = page_of(i, blk);
        const int kept = static_cast<int>(x0 - begin), row = q.r0 + (x0 - q.base);
        if (which & 1)
            append_page<E, V, INTER, false>(P, head, row, x1 - x0, x0, kept, page, lane);
        else
            append_page<E, V, INTER, true>(P, head, row, x1 - x0, x0, kept, page, lane);
        return;
    }
    unit -= P.page_units;
    if (unit < P.q_units) {
        using Vec = Piece<E, V>;
        constexpr int kAtOnce = 4;
        const int r = unit;
        const int per = Task<V, INTER>::kPairs ? P.D / V - P.rot / 2 / V : P.D / V, total = P.Hq * per;
        const E *src = static_cast<const E *>(P.q) + r * P.q_stride;
        E *dst = static_cast<E *>(P.q_out) + r * P.q_out_stride;
        int pos = -1;
#pragma unroll 1
        for (int first = lane; first - lane < total; first += kAtOnce * kWarp) {
            Vec a[kAtOnce] = {}, b[kAtOnce] = {};
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const int idx = first + j * kWarp, h = P.by_k(idx);
                const Task<V, INTER> t(P, idx - h * per, true);
                if (idx >= total) continue;
                a[j] = *reinterpret_cast<const Vec *>(src + h * P.D + t.d0);
                if (t.two) b[j] = *reinterpret_cast<const Vec *>(src + h * P.D + t.d1);
            }
            if (first == lane) {  // the row's position, while its values are under way
                const int i = find_request(P.row_off, P.B, P.T, r, lane);
                const Request q = request(i);
                if (r < q.r0 || r >= q.r0 + q.n) return;
                pos = q.base + (r - q.r0);
                if (pos < 0 || pos >= P.n_pos || page_of(i, P.by_page(pos)) < 0) return;
            }
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const int idx = first + j * kWarp, h = P.by_k(idx);
                const Task<V, INTER> t(P, idx - h * per, true);
                if (idx >= total || !SPEC_IN(r, P.T, DBG_OUT_ROWS) || !SPEC_IN(h, P.Hq, DBG_OUT_ROWS)) continue;
                float u[V], w[V];
                unpack(a[j], u);
                unpack(b[j], w);
                turn<V, INTER>(P, t, pos, u, w);
                // (what does not turn keeps its bits)
                if (t.rotates) pack(a[j], u);
                if (t.two) pack(b[j], w);
                if (SPEC_IN(t.d0 + V - 1, P.D, DBG_CACHE)) *reinterpret_cast<Vec *>(dst + h * P.D + t.d0) = a[j];
                if (t.two && SPEC_IN(t.d1 + V - 1, P.D, DBG_CACHE)) *reinterpret_cast<Vec *>(dst + h * P.D + t.d1) = b[j];
            }
        }
        return;
    }
    const int i = unit - P.q_units;
    if (i >= P.B || !P.req_status) return;
    const int st = append_status(P, i, lane, in_doubt);
    if (lane == 0 && SPEC_IN(i, P.B, DBG_OUT_REQS)) P.req_status[i] = st;
}

template <typename E, int V, bool INTER>
static spec_status launch_append8(Append8Params &P, cudaStream_t stream) {
    P.by_k = FastDiv(Task<V, INTER>::kPairs ? P.D / V - P.rot / 2 / V : P.D / V);
    P.by_v = FastDiv(P.D / V);
    const int64_t units = static_cast<int64_t>(P.page_units) + P.q_units + P.B;
    const int64_t blocks = (units + kAppend8Warps - 1) / kAppend8Warps;
    const dim3 grid(static_cast<unsigned>(blocks)), block(kAppend8Threads);
    // four CTAs an SM for prompts: more rows a request than a page has slots
    const bool prompts = P.T > static_cast<int64_t>(P.B) * P.page_size;
    const cudaError_t e = prompts ? launch_after(spec_append8_kernel<E, V, INTER, 4>, grid, block, 0, stream, P)
                                  : launch_after(spec_append8_kernel<E, V, INTER, 3>, grid, block, 0, stream, P);
    return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

template <typename E>
static spec_status dispatch_append8(Append8Params &P, bool inter, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(E);
    auto aligned = [](const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    const int64_t rows = P.k_stride | P.v_stride | (P.Hq ? P.q_stride | P.q_out_stride : 0);
    const int64_t cache = P.page_stride | P.slot_stride | P.head_stride;
    const bool vec = rows % V == 0 && cache % V == 0 && P.D % V == 0 && P.rot % (inter ? V : 2 * V) == 0 && aligned(P.k) &&
                     aligned(P.v) && aligned(P.k_cache) && aligned(P.v_cache) && (!P.rot || aligned(P.cos_sin)) &&
                     (!P.Hq || (aligned(P.q) && aligned(P.q_out)));
    if (inter) return vec ? launch_append8<E, V, true>(P, stream) : launch_append8<E, 1, true>(P, stream);
    return vec ? launch_append8<E, V, false>(P, stream) : launch_append8<E, 1, false>(P, stream);
}

}  // namespace spec

using namespace spec;

extern "C" spec_status spec_kv_append8(const spec_kv_append8_args *a, cudaStream_t stream) {
    if (!a) return SPEC_ERR_INVALID_ARG;
    Append8Params P = {};
    const spec_status st = append_params(&a->append, P);
    if (st != SPEC_OK) return st;
    if (!a->k_scale || !a->v_scale) return SPEC_ERR_INVALID_ARG;
    P.k_scale = a->k_scale;
    P.v_scale = a->v_scale;
    // a page's tasks and the warps are counted in 32 bits
    if (P.T > (1 << 20) || P.page_size > (1 << 16)) return SPEC_ERR_UNSUPPORTED;
    const int64_t pages = (2ll * P.B + P.T / P.page_size) * 2 * P.Hkv;
    if (pages + P.T + P.B > INT32_MAX / 2) return SPEC_ERR_UNSUPPORTED;
    P.by_page = FastDiv(P.page_size);
    P.page_units = P.T > 0 ? static_cast<int32_t>(pages) : 0;
    P.q_units = P.Hq > 0 ? P.T : 0;
    return a->append.dtype == SPEC_BF16 ? dispatch_append8<__nv_bfloat16>(P, a->append.interleaved != 0, stream)
                                        : dispatch_append8<float>(P, a->append.interleaved != 0, stream);
}

#ifdef SPEC_DEBUG
namespace spec {
// The debug words of this translation unit's kernel.
cudaError_t debug_take_append8(unsigned int out[4]) { return spec_dbg_take(out); }
}  // namespace spec
#endif
