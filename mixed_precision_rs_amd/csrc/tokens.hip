// Tokens sorted by expert and back (tide_route_tokens, tide_dispatch_tokens,
// tide_combine_tokens, tide_combine_tokens_grad) for gfx950.
//
// The sort is a stable counting sort of the T * k (expert, flat index) pairs;
// moving the rows is a copy, and the way back a sum of k rows a token in
// fixed order, so both are HBM streams: each row of a sorted buffer is
// touched once, in 16-byte vectors, by the lanes of its token. A row's last
// vector ends at its end: the elements that it shares with the one before are
// written twice, with the same value. (Element by element, each of a token's
// rows waited for the one before: gradients of 16384 x 2047 bf16, k = 8, 401 us
// instead of 240, combined 152 instead of 112.)
#include <climits>

#include "device.hpp"
#include "host.hpp"

using namespace tide;

namespace {

constexpr int kMaxExperts = 512;     // LDS of the placing kernel: 16 wave histograms of 4 bytes each
constexpr int kRouteThreads = 1024;
constexpr int kRouteWaves = kRouteThreads / 64;
// Pairs that one workgroup sorts alone, in one launch: 4096 pairs take 7.9 us
// so, as 4800 do in two launches; 8192 would take 12.2 alone and 7.9 in two.
constexpr int64_t kRouteAlone = 4096;
// Pairs a workgroup sorts when there are several: 131072 pairs in 10.9 us with
// 2048, 13.0 with 1024, 12.0 with 4096.
constexpr int64_t kRouteChunk = 2048;
constexpr int64_t kRouteMaxBlocks = 128;

// Pairs a workgroup sorts: a multiple of 64 a wave.
int64_t route_chunk(int64_t n) {
    const int64_t step = kRouteThreads;
    int64_t c = n <= kRouteAlone ? n : kRouteChunk;
    if (n > c * kRouteMaxBlocks) c = (n + kRouteMaxBlocks - 1) / kRouteMaxBlocks;
    return (c + step - 1) / step * step;
}
int64_t route_blocks(int64_t n) {
    const int64_t c = route_chunk(n);
    return n <= c ? 1 : (n + c - 1) / c;
}

template <class Id>
__device__ __forceinline__ int32_t expert_of(const Id* ids, int64_t i, int64_t n, int32_t E) {
    if (i >= n) return -1;
    const Id id = *gbl<Id>(ids + i);
    return id >= 0 && id < (Id)E ? (int32_t)id : -1;
}

// Pairs of each expert in one workgroup's chunk: counts[block * E + e].
template <class Id>
__global__ __launch_bounds__(kRouteThreads) void route_count(const Id* ids, int64_t n, int32_t E,
                                                             int64_t chunk, int32_t* counts) {
    __shared__ int32_t hist[kMaxExperts];
    for (int e = threadIdx.x; e < E; e += kRouteThreads) hist[e] = 0;
    __syncthreads();
    const int64_t lo = blockIdx.x * chunk;
    for (int64_t i = threadIdx.x; i < chunk; i += kRouteThreads) {
        const int32_t e = expert_of(ids, lo + i, n, E);
        if (e >= 0) atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kRouteThreads)
        *gbl_mut<int32_t>(counts + (int64_t)blockIdx.x * E + e) = hist[e];
}

// Position of every pair. A wave owns a contiguous run of its workgroup's
// chunk, so (workgroup, wave, step, lane) is the flat order and the sort is
// stable: position = pairs of smaller experts + this expert's pairs in
// earlier workgroups + in earlier waves + in earlier steps + in lower lanes.
// The counts are integers, so the order of the LDS additions does not matter.
template <class Id>
__global__ __launch_bounds__(kRouteThreads) void route_place(const Id* ids, int64_t n, int32_t k,
                                                             int32_t E, int64_t chunk,
                                                             const int32_t* counts,
                                                             int32_t* offsets, int32_t* tokens,
                                                             int32_t* slots) {
    extern __shared__ int32_t wave_at[];           // [kRouteWaves][E]
    __shared__ int32_t total[kMaxExperts], before[kMaxExperts];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int nb = gridDim.x, me = blockIdx.x;
    for (int i = tid; i < kRouteWaves * E; i += kRouteThreads) wave_at[i] = 0;
    for (int i = tid; i < E; i += kRouteThreads) total[i] = before[i] = 0;
    __syncthreads();
    const int64_t run = chunk / kRouteWaves;       // a multiple of 64
    const int64_t lo = me * chunk + wave * run;
    int32_t* mine = wave_at + wave * E;
    for (int64_t i = lane; i < run; i += 64) {
        const int32_t e = expert_of(ids, lo + i, n, E);
        if (e >= 0) atomicAdd(&mine[e], 1);
    }
    if (nb > 1) {
        for (int i = tid; i < nb * E; i += kRouteThreads) {
            const int b = i / E, e = i - b * E;
            const int32_t c = *gbl<int32_t>(counts + i);
            if (c) {
                atomicAdd(&total[e], c);
                if (b < me) atomicAdd(&before[e], c);
            }
        }
        __syncthreads();
    } else {
        __syncthreads();
        for (int e = tid; e < E; e += kRouteThreads) {
            int32_t t = 0;
            for (int w = 0; w < kRouteWaves; ++w) t += wave_at[w * E + e];
            total[e] = t;
        }
        __syncthreads();
    }
    if (wave == 0) {                               // exclusive scan of total[], in place
        constexpr int kPer = kMaxExperts / 64;
        int32_t v[kPer], sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = lane * kPer + i;
            v[i] = e < E ? total[e] : 0;
            sum += v[i];
        }
        int32_t inc = sum;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int32_t up = __shfl_up(inc, d);
            if (lane >= d) inc += up;
        }
        int32_t at = inc - sum;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = lane * kPer + i;
            if (e < E) total[e] = at;
            at += v[i];
            if (me == 0 && e < E) {
                if (e == 0) *gbl_mut<int32_t>(offsets) = 0;
                *gbl_mut<int32_t>(offsets + e + 1) = at;
            }
        }
    }
    __syncthreads();
    for (int e = tid; e < E; e += kRouteThreads) {
        int32_t at = total[e] + before[e];
        for (int w = 0; w < kRouteWaves; ++w) {
            const int32_t c = wave_at[w * E + e];
            wave_at[w * E + e] = at;
            at += c;
        }
    }
    __syncthreads();
    const int bits = 32 - __builtin_clz(E);
    for (int64_t i0 = 0; i0 < run; i0 += 64) {
        const int64_t i = lo + i0 + lane;
        if (lo + i0 >= n) break;
        const int32_t e = expert_of(ids, i, n, E);
        uint64_t same = ~0ull;                     // lanes with this lane's expert
        for (int b = 0; b < bits; ++b) {
            const uint64_t ones = __ballot((e >> b) & 1);
            same &= (e >> b) & 1 ? ones : ~ones;
        }
        same &= __ballot(e >= 0);
        int32_t at = -1;
        if (e >= 0) {
            const int below = __popcll(same & ((1ull << lane) - 1));
            const int32_t base = mine[e];
            at = base + below;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (below == 0) mine[e] = base + __popcll(same);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (i < n) {
            *gbl_mut<int32_t>(slots + i) = at;
            if (at >= 0) *gbl_mut<int32_t>(tokens + at) = (int32_t)((uint32_t)i / (uint32_t)k);
        }
    }
}

// First element of vector u of a row.
template <int V>
__device__ __forceinline__ int64_t at_vector(int64_t u, int64_t width) {
    return u > 0 && u * V > width - V ? width - V : u * V;
}

// rows[slots[t, j]] = x[t]: a token's lanes read its row once and write it to
// each of its slots. Elements are moved as 2-byte units (an fp32 is two).
__global__ __launch_bounds__(kRowThreads) void dispatch_rows(
    const uint16_t* x, int64_t x_stride, int64_t T, int64_t width, int32_t k,
    const int32_t* slots, uint16_t* rows, int64_t rows_stride, uint32_t nrows, int lane_log2) {
    const int lanes = 1 << lane_log2;
    const int64_t units = (width + 7) / 8;
    for (int64_t t = (int64_t)blockIdx.x * (kRowThreads >> lane_log2) + (threadIdx.x >> lane_log2);
         t < T; t += (int64_t)gridDim.x * (kRowThreads >> lane_log2)) {
        for (int64_t u = (int64_t)blockIdx.y * lanes + (threadIdx.x & (lanes - 1)); u < units;
             u += (int64_t)gridDim.y * lanes) {
            const int64_t at = at_vector<8>(u, width);
            const int some = width < 8 ? (int)width : 8;
            const u32x4 v = load_row(x + t * x_stride + at, some);
            for (int32_t j = 0; j < k; ++j) {
                const int32_t s = *gbl<int32_t>(slots + t * k + j);
                if ((uint32_t)s < nrows) store_row(rows + (int64_t)s * rows_stride + at, some, v);
            }
        }
    }
}

// out[t] = sum over j of weights[t, j] * rows[slots[t, j]], j ascending, fp32,
// rounded once. KU rows' loads are in flight before the first addition.
template <class T, int KU>
__global__ __launch_bounds__(kRowThreads) void combine_rows(
    const T* rows, int64_t rows_stride, uint32_t nrows, int64_t width, const int32_t* slots,
    const float* weights, int64_t tokens, int32_t k, T* out, int64_t out_stride, int lane_log2) {
    constexpr int V = kVecOf<T>;
    const int lanes = 1 << lane_log2;
    const int64_t units = (width + V - 1) / V;
    for (int64_t t = (int64_t)blockIdx.x * (kRowThreads >> lane_log2) + (threadIdx.x >> lane_log2);
         t < tokens; t += (int64_t)gridDim.x * (kRowThreads >> lane_log2)) {
        for (int64_t u = (int64_t)blockIdx.y * lanes + (threadIdx.x & (lanes - 1)); u < units;
             u += (int64_t)gridDim.y * lanes) {
            const int64_t at = at_vector<V>(u, width);
            const int some = width < V ? (int)width : V;
            float acc[V] = {};
            for (int32_t j0 = 0; j0 < k; j0 += KU) {
                u32x4 raw[KU];
                float w[KU];
#pragma unroll
                for (int i = 0; i < KU; ++i) {
                    const int32_t s = j0 + i < k ? *gbl<int32_t>(slots + t * k + j0 + i) : -1;
                    raw[i] = u32x4{};
                    w[i] = 0.0f;
                    if ((uint32_t)s < nrows) {
                        raw[i] = load_row<true>(rows + (int64_t)s * rows_stride + at, some);
                        w[i] = weights ? *gbl<float>(weights + t * k + j0 + i) : 1.0f;
                    }
                }
#pragma unroll
                for (int i = 0; i < KU; ++i) {
                    float v[V];
                    widen(raw[i], v);
#pragma unroll
                    for (int c = 0; c < V; ++c) acc[c] = __builtin_fmaf(w[i], v[c], acc[c]);
                }
            }
            store_row(out + t * out_stride + at, some, narrow(acc));
        }
    }
}

// drows[slots[t, j]] = weights[t, j] * dout[t] and dweights[t, j] = dout[t] .
// rows[slots[t, j]], KU rows at a time. A token has 64 to 256 lanes, enough
// for a row of 2048 bf16 in one pass: a wave's later loads wait for its
// earlier stores, so a token's loads all come first. Each lane sums its
// vectors in order, a fixed tree joins a wave's lanes and LDS the waves.
template <class T, int KU>
__global__ __launch_bounds__(kRowThreads) void combine_rows_grad(
    const T* dout, int64_t dout_stride, const T* rows, int64_t rows_stride, uint32_t nrows,
    int64_t width, const int32_t* slots, const float* weights, int64_t tokens, int32_t k,
    T* drows, int64_t drows_stride, float* dweights, int lane_log2) {
    constexpr int V = kVecOf<T>;
    __shared__ float dots[kRowThreads / 64][KU];
    const int lanes = 1 << lane_log2, lane = threadIdx.x & (lanes - 1);
    const int64_t units = (width + V - 1) / V;
    const int64_t per = kRowThreads >> lane_log2;
    for (int64_t t0 = (int64_t)blockIdx.x * per; t0 < tokens; t0 += (int64_t)gridDim.x * per) {
        const int64_t t = t0 + (threadIdx.x >> lane_log2);
        for (int32_t j0 = 0; j0 < k; j0 += KU) {
            int32_t s[KU];
            float w[KU], dot[KU] = {};
#pragma unroll
            for (int i = 0; i < KU; ++i) {
                s[i] = t < tokens && j0 + i < k ? *gbl<int32_t>(slots + t * k + j0 + i) : -1;
                if ((uint32_t)s[i] >= nrows) s[i] = -1;
                w[i] = s[i] >= 0 && weights ? *gbl<float>(weights + t * k + j0 + i) : 1.0f;
            }
            for (int64_t u = lane; t < tokens && u < units; u += lanes) {
                const int64_t at = at_vector<V>(u, width);
                const int some = width < V ? (int)width : V, seen = width < V ? 0 : (int)(u * V - at);
                float d[V];
                widen(load_row(dout + t * dout_stride + at, some), d);
                u32x4 raw[KU];
#pragma unroll
                for (int i = 0; i < KU; ++i) {
                    raw[i] = u32x4{};
                    if (s[i] >= 0 && dweights)
                        raw[i] = load_row<true>(rows + (int64_t)s[i] * rows_stride + at, some);
                }
#pragma unroll
                for (int i = 0; i < KU; ++i) {
                    float v[V];
                    widen(raw[i], v);
#pragma unroll
                    for (int c = 0; c < V; ++c) dot[i] = c < seen ? dot[i] : __builtin_fmaf(d[c], v[c], dot[i]);
                }
#pragma unroll
                for (int i = 0; i < KU; ++i) {
                    if (s[i] < 0) continue;
                    float v[V];
#pragma unroll
                    for (int c = 0; c < V; ++c) v[c] = w[i] * d[c];
                    store_row(drows + (int64_t)s[i] * drows_stride + at, some, narrow(v));
                }
            }
            if (!dweights) continue;
#pragma unroll
            for (int i = 0; i < KU; ++i) {
#pragma unroll
                for (int m = 32; m > 0; m >>= 1) dot[i] += __shfl_xor(dot[i], m);
                if ((threadIdx.x & 63) == 0) dots[threadIdx.x / 64][i] = s[i] >= 0 ? dot[i] : 0.0f;
            }
            __syncthreads();
            if (lane < KU && t < tokens && j0 + lane < k) {
                float v = 0.0f;
                for (int i = 0; i < lanes / 64; ++i) v += dots[threadIdx.x / 64 + i][lane];
                *gbl_mut<float>(dweights + t * k + j0 + lane) = v;
            }
            __syncthreads();
        }
    }
}

template <class F>
hipError_t with_ku(int32_t k, F&& f) {
    if (k == 1) return f(std::integral_constant<int, 1>{});
    if (k == 2) return f(std::integral_constant<int, 2>{});
    if (k <= 4) return f(std::integral_constant<int, 4>{});
    return f(std::integral_constant<int, 8>{});
}

template <class Id>
hipError_t launch_route(const void* ids, int64_t n, int32_t k, int32_t E, int32_t* offsets,
                        int32_t* tokens, int32_t* slots, int32_t* counts, hipStream_t stream) {
    const int64_t chunk = route_chunk(n), nb = route_blocks(n);
    if (nb > 1) {
        const hipError_t e = enqueue(route_count<Id>, dim3((uint32_t)nb), kRouteThreads, 0, stream,
            (const Id*)ids, n, E, chunk, counts);
        if (e != hipSuccess) return e;
    }
    return enqueue(route_place<Id>, dim3((uint32_t)nb), kRouteThreads, (size_t)kRouteWaves * E * 4, stream,
        (const Id*)ids, n, k, E, chunk, counts, offsets, tokens, slots);
}

tide_status check_sort(int32_t dtype, int64_t T, int32_t k, int64_t nrows) {
    if (dtype != TIDE_DTYPE_BF16 && dtype != TIDE_DTYPE_FP32)
        return fail(TIDE_ERR_INVALID_ARG, "dtype %d is not BF16 (0) or FP32 (1)", dtype);
    if (T < 0 || k < 1) return fail(TIDE_ERR_INVALID_ARG, "need tokens >= 0 and k >= 1");
    if (nrows < 0) return fail(TIDE_ERR_INVALID_ARG, "negative row count");
    if (T > INT32_MAX / k || nrows > INT32_MAX)
        return fail(TIDE_ERR_UNSUPPORTED, "tokens * k and the rows must be below 2^31");
    return TIDE_OK;
}

}  // namespace

extern "C" {

tide_status tide_route_workspace(int64_t tokens, int32_t k, int32_t experts, int64_t* bytes) {
    return guarded([&]() -> tide_status {
        if (!bytes) return fail(TIDE_ERR_INVALID_ARG, "bytes is NULL");
        TIDE_TRY(check_sort(TIDE_DTYPE_BF16, tokens, k, 0));
        if (experts < 1) return fail(TIDE_ERR_INVALID_ARG, "need experts >= 1");
        if (experts > kMaxExperts)
            return fail(TIDE_ERR_UNSUPPORTED, "%d experts: at most %d", experts, kMaxExperts);
        const int64_t nb = route_blocks(tokens * k);
        *bytes = nb > 1 ? nb * experts * 4 : 0;
        return TIDE_OK;
    });
}

tide_status tide_route_tokens(const void* experts_of, int32_t id_bytes, int64_t tokens, int32_t k,
                              int32_t experts, int32_t* offsets, int32_t* token_of_row,
                              int32_t* slots, void* workspace, int64_t workspace_bytes,
                              void* stream) {
    return guarded([&]() -> tide_status {
        int64_t need = 0;
        TIDE_TRY(tide_route_workspace(tokens, k, experts, &need));
        if (id_bytes != 4 && id_bytes != 8)
            return fail(TIDE_ERR_INVALID_ARG, "expert ids have 4 or 8 bytes, not %d", id_bytes);
        if (need > 0 && (!workspace || workspace_bytes < need))
            return fail(TIDE_ERR_INVALID_ARG, "workspace holds %lld bytes, %lld needed",
                        (long long)(workspace ? workspace_bytes : 0), (long long)need);
        const int64_t n = tokens * k;
        Mat in, wr[4];
        TIDE_TRY(matrix("experts_of", experts_of, 1, n, n, id_bytes, &in));
        TIDE_TRY(matrix("offsets", offsets, 1, experts + 1, experts + 1, 4, &wr[0]));
        TIDE_TRY(matrix("token_of_row", token_of_row, 1, n, n, 4, &wr[1]));
        TIDE_TRY(matrix("slots", slots, 1, n, n, 4, &wr[2]));
        TIDE_TRY(matrix("workspace", workspace, 1, need / 4, need / 4, 4, &wr[3]));
        TIDE_TRY(no_overlap(wr, 4, &in, 1));
        return on_stream(stream, [&](hipStream_t s) {
            return id_bytes == 4 ? launch_route<int32_t>(experts_of, n, k, experts, offsets,
                                                         token_of_row, slots, (int32_t*)workspace, s)
                                 : launch_route<int64_t>(experts_of, n, k, experts, offsets,
                                                         token_of_row, slots, (int32_t*)workspace, s);
        });
    });
}

tide_status tide_dispatch_tokens(int32_t dtype, const void* x, int64_t x_stride, int64_t tokens,
                                 int64_t width, const int32_t* slots, int32_t k, void* rows,
                                 int64_t rows_stride, int64_t nrows, void* stream) {
    return guarded([&]() -> tide_status {
        TIDE_TRY(check_sort(dtype, tokens, k, nrows));
        const int32_t size = dtype == TIDE_DTYPE_FP32 ? 4 : 2;
        Mat rd[2], wr;
        TIDE_TRY(matrix("x", x, tokens, width, x_stride, size, &rd[0]));
        TIDE_TRY(matrix("slots", slots, width ? tokens : 0, k, k, 4, &rd[1]));
        TIDE_TRY(matrix("rows", rows, nrows, width, rows_stride, size, &wr));
        TIDE_TRY(no_overlap(&wr, 1, rd, 2));
        if (tokens == 0 || width == 0 || nrows == 0) return TIDE_OK;
        return on_stream(stream, [&](hipStream_t s) {
            const int64_t per = size / 2, units = (width * per + 7) / 8;
            const RowGrid g = row_grid(tokens, units);
            return enqueue(dispatch_rows, g.grid, kRowThreads, 0, s,
                (const uint16_t*)x, x_stride * per, tokens, width * per, k, slots, (uint16_t*)rows,
                rows_stride * per, (uint32_t)nrows, g.lane_log2);
        });
    });
}

tide_status tide_combine_tokens(int32_t dtype, const void* rows, int64_t rows_stride,
                                int64_t nrows, int64_t width, const int32_t* slots,
                                const float* weights, int64_t tokens, int32_t k, void* out,
                                int64_t out_stride, void* stream) {
    return guarded([&]() -> tide_status {
        TIDE_TRY(check_sort(dtype, tokens, k, nrows));
        const int32_t size = dtype == TIDE_DTYPE_FP32 ? 4 : 2;
        Mat rd[3], wr;
        TIDE_TRY(matrix("rows", rows, nrows, width, rows_stride, size, &rd[0]));
        TIDE_TRY(matrix("slots", slots, width ? tokens : 0, k, k, 4, &rd[1]));
        TIDE_TRY(matrix("weights", weights, weights && width ? tokens : 0, k, k, 4, &rd[2]));
        TIDE_TRY(matrix("out", out, tokens, width, out_stride, size, &wr));
        TIDE_TRY(no_overlap(&wr, 1, rd, 3));
        if (tokens == 0 || width == 0) return TIDE_OK;
        return on_stream(stream, [&](hipStream_t s) {
            const RowGrid g = row_grid(tokens, (width * size + 15) / 16);
            return with_ku(k, [&](auto ku) {
                if (size == 2)
                    return enqueue(combine_rows<uint16_t, ku.value>, g.grid, kRowThreads, 0, s,
                        (const uint16_t*)rows, rows_stride, (uint32_t)nrows, width, slots, weights,
                        tokens, k, (uint16_t*)out, out_stride, g.lane_log2);
                else
                    return enqueue(combine_rows<float, ku.value>, g.grid, kRowThreads, 0, s,
                        (const float*)rows, rows_stride, (uint32_t)nrows, width, slots, weights,
                        tokens, k, (float*)out, out_stride, g.lane_log2);
            });
        });
    });
}

tide_status tide_combine_tokens_grad(int32_t dtype, const void* dout, int64_t dout_stride,
                                     const void* rows, int64_t rows_stride, int64_t nrows,
                                     int64_t width, const int32_t* slots, const float* weights,
                                     int64_t tokens, int32_t k, void* drows,
                                     int64_t drows_stride, float* dweights, void* stream) {
    return guarded([&]() -> tide_status {
        TIDE_TRY(check_sort(dtype, tokens, k, nrows));
        const int32_t size = dtype == TIDE_DTYPE_FP32 ? 4 : 2;
        Mat rd[4], wr[2];
        TIDE_TRY(matrix("dout", dout, tokens, width, dout_stride, size, &rd[0]));
        TIDE_TRY(matrix("rows", rows, dweights ? nrows : 0, width, rows_stride, size, &rd[1]));
        TIDE_TRY(matrix("slots", slots, tokens, k, k, 4, &rd[2]));
        TIDE_TRY(matrix("weights", weights, weights ? tokens : 0, k, k, 4, &rd[3]));
        TIDE_TRY(matrix("drows", drows, nrows, width, drows_stride, size, &wr[0]));
        TIDE_TRY(matrix("dweights", dweights, dweights ? tokens : 0, k, k, 4, &wr[1]));
        TIDE_TRY(no_overlap(wr, 2, rd, 4));
        if (tokens == 0 || (width == 0 && !dweights)) return TIDE_OK;
        return on_stream(stream, [&](hipStream_t s) {
            const RowGrid g = row_grid(tokens, (width * size + 15) / 16, 6);
            const dim3 grid(g.grid.x);
            return with_ku(k, [&](auto ku) {
                if (size == 2)
                    return enqueue(combine_rows_grad<uint16_t, ku.value>, grid, kRowThreads, 0, s,
                        (const uint16_t*)dout, dout_stride, (const uint16_t*)rows, rows_stride,
                        (uint32_t)nrows, width, slots, weights, tokens, k, (uint16_t*)drows,
                        drows_stride, dweights, g.lane_log2);
                else
                    return enqueue(combine_rows_grad<float, ku.value>, grid, kRowThreads, 0, s,
                        (const float*)dout, dout_stride, (const float*)rows, rows_stride,
                        (uint32_t)nrows, width, slots, weights, tokens, k, (float*)drows,
                        drows_stride, dweights, g.lane_log2);
            });
        });
    });
}

}  // extern "C"
