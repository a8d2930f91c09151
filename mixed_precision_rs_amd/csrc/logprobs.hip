// Log probabilities of given tokens, entropy and the most probable
// alternatives (tide_token_logprobs), and the gradient to the logits
// (tide_token_logprobs_grad), for gfx950.
//
// A row's maximum m, s = sum exp(x - m) and t = sum exp(x - m) (x - m) come from
// one pass: each lane keeps the three over its own logits, t and s brought to the
// new maximum when it rises, and a fixed tree joins the lanes.
#include <climits>
#include <cmath>

#include "device.hpp"
#include "host.hpp"

using namespace tide;

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMostTop = 32;
constexpr float kLog2e = 0x1.715476p+0f;
constexpr float kNegInf = -__builtin_inff();
// A lane's maximum starts here, not at -infinity: x - m is then never
// -infinity - -infinity, and logits of -infinity have exp 0.
constexpr float kLowest = -__FLT_MAX__;
// exp(-200) is 0 in fp32: differences are held above it where they are
// factors, so that 0 * -infinity does not arise.
constexpr float kFar = -200.0f;

// exp(z) for z <= 0; a NaN or +infinity - +infinity stays NaN.
__device__ __forceinline__ float exp_of(float z) { return __builtin_amdgcn_exp2f(z * kLog2e); }

struct Sums {
    float m, s, t;
};
// t of a sum whose maximum rises by -d: sum e (z + d) = t + s d.
__device__ __forceinline__ void rise(Sums& a, float m) {
    const float d = fmaxf(a.m - m, kFar), f = exp_of(d);
    a.t = __builtin_fmaf(a.s, d, a.t) * f;
    a.s *= f;
    a.m = m;
}
__device__ __forceinline__ Sums join(Sums a, Sums b) {
    const float m = fmaxf(a.m, b.m);
    rise(a, m);
    rise(b, m);
    return Sums{m, a.s + b.s, a.t + b.t};
}

// Alternatives are ordered by (larger logit, lower id).
struct Best {
    float v;
    int32_t id;      // -1: none
};
__device__ __forceinline__ bool ahead(Best a, Best b) {
    return b.id < 0 ? a.id >= 0 : a.id >= 0 && (a.v > b.v || (a.v == b.v && a.id < b.id));
}
__device__ __forceinline__ Best wave_best(Best b) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        const Best o{__shfl_xor(b.v, d), __shfl_xor(b.id, d)};
        if (ahead(o, b)) b = o;
    }
    return b;
}

// The best of a lane's logits that comes after `last` (id -1: of all), looked
// for by its whole wave: lane l of 64 takes the vectors l, l + 64, ... of it.
template <class T>
__device__ __forceinline__ Best best_after(const T* row, int64_t V, int owner, Best last) {
    constexpr int N = kVecOf<T>;
    const int64_t units = (V + N - 1) / N;
    Best b{kNegInf, -1};
    for (int64_t u = owner + (int64_t)(threadIdx.x & 63) * kThreads; u < units; u += 64 * kThreads) {
        const int n = V - u * N < N ? (int)(V - u * N) : N;
        float v[N];
        widen(load_row(row + u * N, n), v);
#pragma unroll
        for (int c = 0; c < N; ++c) {
            const Best x{v[c], (int32_t)(u * N + c)};
            if (c < n && v[c] > kNegInf && (last.id < 0 || ahead(last, x)) && ahead(x, b)) b = x;
        }
    }
    return wave_best(b);
}

template <class T, class Id>
__global__ __launch_bounds__(kThreads) void row_logprobs(
    const T* logits, int64_t stride, int64_t tokens, int64_t V, const Id* targets, float* logprob,
    float* stats, float* entropy, int32_t top, int32_t* top_ids, float* top_logprobs) {
    constexpr int N = kVecOf<T>, KU = 4;
    __shared__ Sums part[kWaves];
    __shared__ Best found[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t units = (V + N - 1) / N;
    for (int64_t r = blockIdx.x; r < tokens; r += gridDim.x) {
        const T* row = logits + r * stride;
        Sums a{kLowest, 0.0f, 0.0f};
        for (int64_t u0 = tid; u0 < units; u0 += KU * kThreads) {
            float v[KU][N];
            float m = a.m;
#pragma unroll
            for (int j = 0; j < KU; ++j) {
                const int64_t u = u0 + j * kThreads, left = V - u * N;
#pragma unroll
                for (int c = 0; c < N; ++c) v[j][c] = kNegInf;
                if (left > 0) {
                    widen(load_row(row + u * N, left < N ? (int)left : N), v[j]);
#pragma unroll
                    for (int c = 0; c < N; ++c)
                        if (c >= left) v[j][c] = kNegInf;
                }
#pragma unroll
                for (int c = 0; c < N; ++c) m = fmaxf(m, v[j][c]);
            }
            rise(a, m);
#pragma unroll
            for (int j = 0; j < KU; ++j) {
#pragma unroll
                for (int c = 0; c < N; ++c) {
                    const float z = v[j][c] - m, e = exp_of(z);
                    a.s += e;
                    a.t = __builtin_fmaf(e, fmaxf(z, kFar), a.t);
                }
            }
        }
#pragma unroll
        for (int d = 32; d > 0; d >>= 1)
            a = join(a, Sums{__shfl_xor(a.m, d), __shfl_xor(a.s, d), __shfl_xor(a.t, d)});
        if (lane == 0) part[wave] = a;
        __syncthreads();
        a = part[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) a = join(a, part[w]);
        const bool none = a.s == 0.0f;             // no logit above -infinity
        const float log_s = none ? kNegInf : logf(a.s);
        if (tid == 0) {
            const Id at = *gbl<Id>(targets + r);
            float lp = 0.0f;
            if (at >= 0 && (int64_t)at < V) {
                float x;
                if constexpr (sizeof(T) == 2) x = lo_bf16(*gbl<T>(row + at));
                else x = *gbl<float>(row + at);
                lp = none ? kNegInf : (x - a.m) - log_s;
            }
            *gbl_mut<float>(logprob + r) = lp;
            if (stats) {
                *gbl_mut<float>(stats + 2 * r) = none ? kNegInf : a.m;
                *gbl_mut<float>(stats + 2 * r + 1) = log_s;
            }
            if (entropy) *gbl_mut<float>(entropy + r) = none ? 0.0f : log_s - a.t / a.s;
        }
        if (top > 0) {
            Best mine{kNegInf, -1};
            for (int64_t u = tid; u < units; u += kThreads) {
                const int n = V - u * N < N ? (int)(V - u * N) : N;
                float v[N];
                widen(load_row(row + u * N, n), v);
#pragma unroll
                for (int c = 0; c < N; ++c)
                    if (c < n && v[c] > mine.v) mine = Best{v[c], (int32_t)(u * N + c)};
            }
            for (int32_t j = 0; j < top; ++j) {
                const Best w = wave_best(mine);
                __syncthreads();
                if (lane == 0) found[wave] = w;
                __syncthreads();
                Best b = found[0];
#pragma unroll
                for (int i = 1; i < kWaves; ++i)
                    if (ahead(found[i], b)) b = found[i];
                if (tid == 0) {
                    *gbl_mut<int32_t>(top_ids + r * top + j) = b.id;
                    *gbl_mut<float>(top_logprobs + r * top + j) = b.id < 0 ? kNegInf : (b.v - a.m) - log_s;
                }
                const int owner = (int)(b.id / N % kThreads);
                if (b.id >= 0 && owner >> 6 == wave) {
                    const Best next = best_after(row, V, owner, b);
                    if (tid == owner) mine = next;
                }
            }
        }
        __syncthreads();
    }
}

template <class T, class Id>
__global__ __launch_bounds__(kThreads) void row_logprobs_grad(
    const T* logits, int64_t stride, int64_t tokens, int64_t V, const Id* targets, const float* stats,
    const float* dlogprob, const float* entropy, const float* dentropy, T* dlogits, int64_t dstride) {
    constexpr int N = kVecOf<T>;
    const int64_t units = (V + N - 1) / N;
    for (int64_t r = blockIdx.x; r < tokens; r += gridDim.x) {
        const Id id = *gbl<Id>(targets + r);
        const int64_t at = id >= 0 && (int64_t)id < V ? (int64_t)id : -1;
        const float m = *gbl<float>(stats + 2 * r), log_s = *gbl<float>(stats + 2 * r + 1);
        const float d = at >= 0 ? *gbl<float>(dlogprob + r) : 0.0f;
        const float h = dentropy ? *gbl<float>(dentropy + r) : 0.0f, H = dentropy ? *gbl<float>(entropy + r) : 0.0f;
        const bool zero = (at < 0 && !dentropy) || m == kNegInf;
        for (int64_t u = (int64_t)blockIdx.y * kThreads + threadIdx.x; u < units; u += (int64_t)gridDim.y * kThreads) {
            const int n = V - u * N < N ? (int)(V - u * N) : N;
            float v[N] = {};
            if (!zero) {
                widen(load_row(logits + r * stride + u * N, n), v);
#pragma unroll
                for (int c = 0; c < N; ++c) {
                    const float lp = (v[c] - m) - log_s, p = exp_of(lp);
                    float g = u * N + c == at ? d : 0.0f;
                    g = __builtin_fmaf(-d, p, g);
                    if (dentropy) g = __builtin_fmaf(-h, p * (fmaxf(lp, kFar) + H), g);
                    v[c] = g;
                }
            }
            store_row(dlogits + r * dstride + u * N, n, narrow(v));
        }
    }
}

tide_status check(int32_t dtype, int64_t tokens, int64_t vocab, int32_t id_bytes) {
    if (dtype != TIDE_DTYPE_BF16 && dtype != TIDE_DTYPE_FP32)
        return fail(TIDE_ERR_INVALID_ARG, "dtype %d is not BF16 (0) or FP32 (1)", dtype);
    if (id_bytes != 4 && id_bytes != 8)
        return fail(TIDE_ERR_INVALID_ARG, "ids have 4 or 8 bytes, not %d", id_bytes);
    if (tokens < 0 || vocab < 0) return fail(TIDE_ERR_INVALID_ARG, "need tokens and vocab >= 0");
    if (vocab > INT32_MAX) return fail(TIDE_ERR_UNSUPPORTED, "vocab must be below 2^31");
    return TIDE_OK;
}

template <class F>
hipError_t with_types(int32_t dtype, int32_t id_bytes, F&& go) {
    if (dtype == TIDE_DTYPE_BF16) return id_bytes == 4 ? go(uint16_t{}, int32_t{}) : go(uint16_t{}, int64_t{});
    return id_bytes == 4 ? go(float{}, int32_t{}) : go(float{}, int64_t{});
}

}  // namespace

extern "C" {

tide_status tide_token_logprobs(int32_t dtype, const void* logits, int64_t logits_stride,
                                int64_t tokens, int64_t vocab, const void* targets,
                                int32_t id_bytes, float* logprob, float* stats, float* entropy,
                                int32_t top, int32_t* top_ids, float* top_logprobs, void* stream) {
    return guarded([&]() -> tide_status {
        TIDE_TRY(check(dtype, tokens, vocab, id_bytes));
        if (top < 0) return fail(TIDE_ERR_INVALID_ARG, "negative top");
        if (top > kMostTop) return fail(TIDE_ERR_UNSUPPORTED, "%d alternatives: at most %d", top, kMostTop);
        const int32_t size = dtype == TIDE_DTYPE_FP32 ? 4 : 2;
        Mat rd[2], wr[5];
        TIDE_TRY(matrix("logits", logits, tokens, vocab, logits_stride, size, &rd[0]));
        TIDE_TRY(matrix("targets", targets, 1, tokens, tokens, id_bytes, &rd[1]));
        TIDE_TRY(matrix("logprob", logprob, 1, tokens, tokens, 4, &wr[0]));
        TIDE_TRY(matrix("stats", stats, stats ? tokens : 0, 2, 2, 4, &wr[1]));
        TIDE_TRY(matrix("entropy", entropy, entropy ? 1 : 0, tokens, tokens, 4, &wr[2]));
        TIDE_TRY(matrix("top_ids", top_ids, tokens, top, top, 4, &wr[3]));
        TIDE_TRY(matrix("top_logprobs", top_logprobs, tokens, top, top, 4, &wr[4]));
        TIDE_TRY(no_overlap(wr, 5, rd, 2));
        if (tokens == 0) return TIDE_OK;
        return on_stream(stream, [&](hipStream_t s) {
            const dim3 grid((uint32_t)(tokens < (1 << 20) ? tokens : (1 << 20)));
            return with_types(dtype, id_bytes, [&](auto type, auto id) {
                using T = decltype(type);
                using Id = decltype(id);
                return enqueue(row_logprobs<T, Id>, grid, kThreads, 0, s, (const T*)logits, logits_stride, tokens,
                               vocab, (const Id*)targets, logprob, stats, entropy, top, top_ids, top_logprobs);
            });
        });
    });
}

tide_status tide_token_logprobs_grad(int32_t dtype, const void* logits, int64_t logits_stride,
                                     int64_t tokens, int64_t vocab, const void* targets,
                                     int32_t id_bytes, const float* stats, const float* dlogprob,
                                     const float* entropy, const float* dentropy, void* dlogits,
                                     int64_t dlogits_stride, void* stream) {
    return guarded([&]() -> tide_status {
        TIDE_TRY(check(dtype, tokens, vocab, id_bytes));
        if (dentropy && !entropy && tokens) return fail(TIDE_ERR_INVALID_ARG, "dentropy needs entropy");
        const int32_t size = dtype == TIDE_DTYPE_FP32 ? 4 : 2;
        Mat rd[6], wr;
        TIDE_TRY(matrix("targets", targets, 1, tokens, tokens, id_bytes, &rd[0]));
        TIDE_TRY(matrix("stats", stats, tokens, 2, 2, 4, &rd[1]));
        TIDE_TRY(matrix("dlogprob", dlogprob, 1, tokens, tokens, 4, &rd[2]));
        TIDE_TRY(matrix("entropy", entropy, entropy && dentropy ? 1 : 0, tokens, tokens, 4, &rd[3]));
        TIDE_TRY(matrix("dentropy", dentropy, dentropy ? 1 : 0, tokens, tokens, 4, &rd[4]));
        TIDE_TRY(matrix("logits", logits, tokens, vocab, logits_stride, size, &rd[5]));
        TIDE_TRY(matrix("dlogits", dlogits, tokens, vocab, dlogits_stride, size, &wr));
        const bool in_place = dlogits == logits && (dlogits_stride == logits_stride || tokens <= 1);
        TIDE_TRY(no_overlap(&wr, 1, rd, in_place ? 5 : 6));
        if (tokens == 0 || vocab == 0) return TIDE_OK;
        return on_stream(stream, [&](hipStream_t s) {
            const int64_t groups = (vocab * size / 16 + kThreads) / kThreads;
            const dim3 grid((uint32_t)(tokens < (1 << 20) ? tokens : (1 << 20)),
                            (uint32_t)(groups < 32768 ? groups : 32768));
            return with_types(dtype, id_bytes, [&](auto type, auto id) {
                using T = decltype(type);
                using Id = decltype(id);
                return enqueue(row_logprobs_grad<T, Id>, grid, kThreads, 0, s, (const T*)logits, logits_stride,
                               tokens, vocab, (const Id*)targets, stats, dlogprob, entropy, dentropy, (T*)dlogits,
                               dlogits_stride);
            });
        });
    });
}

}  // extern "C"
