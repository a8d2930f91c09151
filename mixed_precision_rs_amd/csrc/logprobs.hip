// Log probabilities of given tokens, entropy and the most probable
// alternatives (tide_token_logprobs), and the gradient to the logits
// (tide_token_logprobs_grad), for gfx950.
//
// A row's maximum m, s = sum exp(x - m) and t = sum exp(x - m) (x - m) come from
// one pass: each lane keeps the three over its own logits, t and s brought to the
// new maximum when it rises, and a fixed tree joins the lanes. Logits are read
// once: 4096 x 131072 bf16 in 169 us (6.4 TB/s; a pure read of as much takes 150).
// The exponential (a quarter of the rate of other instructions) and what is around
// it, 8.6 instructions a logit, fill 158 us of the SIMDs' cycles beside the loads.
// (One maximum a wave instead of a lane's, or the next logits under way meanwhile,
// take more registers and 172 and 198 us.)
#include <climits>
#include <type_traits>

#include "device.hpp"
#include "host.hpp"

using namespace tide;

namespace {

constexpr int kMostTop = 32;
constexpr float kLog2e = 0x1.715476p+0f, kLn2 = 0x1.62e43p-1f;
constexpr float kNegInf = -__builtin_inff();
// A lane's maximum starts here, not at -infinity: x - m is then never
// -infinity - -infinity, and logits of -infinity have exp 0.
constexpr float kLowest = -__FLT_MAX__;
// Up to this magnitude what the rounding of m log2(e) takes is below 2^-8.
constexpr float kTame = 65536.0f;
// exp(-200) is 0 in fp32: differences (and exponents of 2) are held above these
// where they are factors, so that 0 * -infinity does not arise.
constexpr float kFar = -200.0f, kFar2 = -300.0f;

// exp(z) for z <= 0; a NaN or +infinity - +infinity stays NaN.
__device__ __forceinline__ float exp_of(float z) { return __builtin_amdgcn_exp2f(z * kLog2e); }

// s and t in 64 bits: a confident row has s = 1 + little, and log(s) is that little.
struct Sums {
    float m;
    double s, t;
};
// t of a sum whose maximum rises by -d: sum e (z + d) = t + s d.
__device__ __forceinline__ void rise(Sums& a, float m) {
    const float d = fmaxf(a.m - m, kFar);
    const double f = exp_of(d);
    a.t = __builtin_fma(a.s, (double)d, a.t) * f;
    a.s *= f;
    a.m = m;
}
__device__ __forceinline__ Sums join(Sums a, Sums b) {
    const float m = fmaxf(a.m, b.m);
    rise(a, m);
    rise(b, m);
    return Sums{m, a.s + b.s, a.t + b.t};
}
template <int kLanes>
__device__ __forceinline__ Sums join_lanes(Sums a) {
#pragma unroll 1
    for (int d = kLanes / 2; d > 0; d >>= 1)
        a = join(a, Sums{__shfl_xor(a.m, d), __shfl_xor(a.s, d), __shfl_xor(a.t, d)});
    return a;
}
__device__ __forceinline__ float log_of(double s) {
    return s < 2.0 ? log1pf((float)(s - 1.0)) : logf((float)s);
}

// Adds n * M logits to a lane's sums, m being the largest of them and of what the
// lane has. exp(x - m) = 2^(x log2(e) - c) 2^d with c = m log2(e) rounded and d what
// the rounding took: one fused step and the exponential a logit, and the factor
// 2^d for all of them together.
template <bool kEntropy, int M, int N>
__device__ __forceinline__ void add(Sums& a, const float (&v)[M][N], float m) {
    rise(a, m);
    float s[4] = {}, t[4] = {};
    if (__ballot(!(fabsf(m) < kTame)) == 0) {
        const float c = m * kLog2e, d = __builtin_fmaf(-m, kLog2e, c);
#pragma unroll
        for (int j = 0; j < M; ++j) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float p = __builtin_fmaf(v[j][i], kLog2e, -c), e = __builtin_amdgcn_exp2f(p);
                s[i & 3] += e;
                if (kEntropy) t[i & 3] = __builtin_fmaf(e, fmaxf(p, kFar2), t[i & 3]);
            }
        }
        const float sum = (s[0] + s[1]) + (s[2] + s[3]), f = __builtin_amdgcn_exp2f(d);
        a.s += (double)(sum * f);
        if (kEntropy) a.t += (double)(__builtin_fmaf(sum, d, (t[0] + t[1]) + (t[2] + t[3])) * (f * kLn2));
    } else {
#pragma unroll
        for (int j = 0; j < M; ++j) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float z = v[j][i] - m, e = exp_of(z);
                s[i & 3] += e;
                if (kEntropy) t[i & 3] = __builtin_fmaf(e, fmaxf(z, kFar), t[i & 3]);
            }
        }
        a.s += (double)((s[0] + s[1]) + (s[2] + s[3]));
        if (kEntropy) a.t += (double)((t[0] + t[1]) + (t[2] + t[3]));
    }
}

// Alternatives are ordered by (larger logit, lower id): as one number, 0 for none.
__device__ __forceinline__ uint64_t order_of(float v, uint32_t id) {
    const uint32_t b = __float_as_uint(v + 0.0f);                  // -0 is 0
    return (uint64_t)(b & 0x80000000u ? ~b : b | 0x80000000u) << 32 | (uint32_t)~id;
}
__device__ __forceinline__ float logit_of(uint64_t o) {
    const uint32_t b = (uint32_t)(o >> 32);
    return __uint_as_float(b & 0x80000000u ? b & 0x7FFFFFFFu : ~b);
}
__device__ __forceinline__ int32_t id_of(uint64_t o) { return (int32_t)~(uint32_t)o; }

template <int kLanes>
__device__ __forceinline__ uint64_t most_of(uint64_t v) {
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) {
        const uint64_t o = (uint64_t)__shfl_xor((unsigned long long)v, d);
        v = o > v ? o : v;
    }
    return v;
}

template <class T>
__device__ __forceinline__ int vector_of(const T* row, int64_t V, int64_t u, float (&v)[kVecOf<T>]) {
    constexpr int N = kVecOf<T>;
    const int n = V - u * N < N ? (int)(V - u * N) : N;
    widen(load_row(row + u * N, n), v);
    return n;
}

// The alternatives among the vectors begin .. end - 1 of a row, by a workgroup whose
// lane i has the vectors begin + i, begin + i + kThreads, ... and has found the
// largest logit `most` of them, in vector `unit` (-1: none above -infinity).
// emit(place, order) is called for each of the `top` places, with 0 for none.
//
// 64 groups of lanes put forward their best; the top-th of these is no better than
// the top-th of all logits, and only lanes whose own best reaches it can hold an
// alternative. Their vectors are looked through again, all at once, and what
// reaches it is ranked: usually little more than `top` logits. Where it is more
// than kFound (rows that fall or rise throughout), the lanes' bests are taken one
// by one instead.
constexpr int kFound = 512;
struct TopSpace {
    uint64_t best[64];
    uint64_t found[kFound];
    uint16_t lanes[1024];
    int lanes_count, count;
};
// Ranks w.found[0 .. count) by all threads of the workgroup.
template <class F>
__device__ __forceinline__ void rank_found(const TopSpace& w, int count, int threads, int32_t top, F&& emit) {
    for (int i = threadIdx.x; i < count; i += threads) {
        const uint64_t o = w.found[i];
        int at = 0, j = 0;
        for (; j + 16 <= count; j += 16) {         // sixteen reads under way
#pragma unroll
            for (int k = 0; k < 16; ++k) at += w.found[j + k] > o ? 1 : 0;
        }
        for (; j < count; ++j) at += w.found[j] > o ? 1 : 0;
        if (at < top) emit(at, o);
    }
    for (int i = threadIdx.x; i < top; i += threads)
        if (i >= count) emit(i, 0);
}
template <class T, int kThreads, class F>
__device__ __forceinline__ void alternatives(const T* row, int64_t V, int64_t begin, int64_t end, float most,
                                             int64_t unit, int32_t top, TopSpace& w, F&& emit) {
    constexpr int N = kVecOf<T>, kGroup = kThreads / 64;
    const int tid = threadIdx.x, lane = tid & 63;
    uint64_t mine = 0;
    if (unit >= 0) {
        float v[N];
        const int n = vector_of(row, V, unit, v);
#pragma unroll
        for (int c = N - 1; c >= 0; --c)
            if (c < n && v[c] == most) mine = order_of(most, (uint32_t)(unit * N + c));
    }
    const uint64_t group = most_of<kGroup>(mine);
    if (tid % kGroup == 0) w.best[tid / kGroup] = group;
    if (tid == 0) w.lanes_count = w.count = 0;
    __syncthreads();
    const uint64_t c = w.best[lane];
    int rank = 0;
#pragma unroll 16
    for (int i = 0; i < 64; ++i) rank += w.best[i] > c ? 1 : 0;
    const uint64_t last = __ballot(rank == top - 1 && c != 0);
    const uint64_t least = last ? (uint64_t)__shfl((unsigned long long)c, __ffsll((long long)last) - 1) : 1;
    if (mine >= least) w.lanes[atomicAdd(&w.lanes_count, 1)] = (uint16_t)tid;
    __syncthreads();
    const uint32_t per = (uint32_t)((end - begin + kThreads - 1) / kThreads);
    const int64_t items = (int64_t)w.lanes_count * per;
    for (int64_t i = tid; i < items; i += kThreads) {
        const int64_t l = items >> 32 ? i / per : (int64_t)((uint32_t)i / per);
        const int64_t u = begin + w.lanes[l] + (i - l * per) * kThreads;
        if (u >= end) continue;
        float v[N];
        const int n = vector_of(row, V, u, v);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const uint64_t o = order_of(v[k], (uint32_t)(u * N + k));
            if (k < n && v[k] > kNegInf && o >= least) {
                const int at = atomicAdd(&w.count, 1);
                if (at < kFound) w.found[at] = o;
            }
        }
    }
    __syncthreads();
    const int count = w.count;
    if (count <= kFound) {
        rank_found(w, count, kThreads, top, emit);
        return;
    }
    for (int32_t j = 0; j < top; ++j) {
        const uint64_t wave = most_of<64>(mine);
        __syncthreads();
        if (lane == 0) w.best[tid >> 6] = wave;
        __syncthreads();
        uint64_t b = w.best[0];
#pragma unroll
        for (int i = 1; i < kGroup; ++i) b = w.best[i] > b ? w.best[i] : b;
        if (tid == 0) emit(j, b);
        // The owner's next, looked for by its whole wave.
        const int owner = (int)((id_of(b) / N - begin) % kThreads);
        if (b == 0 || owner >> 6 != tid >> 6) continue;
        uint64_t next = 0;
        for (int64_t u = begin + owner + (int64_t)lane * kThreads; u < end; u += 64 * kThreads) {
            float v[N];
            const int n = vector_of(row, V, u, v);
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const uint64_t o = order_of(v[k], (uint32_t)(u * N + k));
                if (k < n && v[k] > kNegInf && o < b && o > next) next = o;
            }
        }
        next = most_of<64>(next);
        if (tid == owner) mine = next;
    }
}

// A lane's largest logit and its vector by comparisons, for a row whose sum is NaN: the
// maximum of a signalling NaN and a number is NaN, and hides that number.
template <class T, int kThreads>
__device__ __forceinline__ void largest_of(const T* row, int64_t V, int64_t begin, int64_t end, float& most, int64_t& unit) {
    constexpr int N = kVecOf<T>;
    most = kNegInf;
    unit = -1;
#pragma unroll 1
    for (int32_t u = (int32_t)begin + threadIdx.x; u < (int32_t)end; u += kThreads) {
        float v[N], b = kNegInf;
        const int n = vector_of(row, V, u, v);
#pragma unroll
        for (int c = 0; c < N; ++c) b = c < n && v[c] > b ? v[c] : b;
        unit = b > most ? u : unit;
        most = b > most ? b : most;
    }
}

// A row's results from its sums, by thread 0.
struct Outputs {
    float *logprob, *stats, *entropy;
    int32_t* top_ids;
    float* top_logprobs;
    int32_t top;
};
template <class T, class Id>
__device__ __forceinline__ void put_row(const Outputs& to, const T* row, int64_t r, int64_t V, const Id* targets,
                                        const Sums& a, float log_s) {
    const bool none = a.s == 0.0;                  // no logit above -infinity
    const Id at = *gbl<Id>(targets + r);
    float lp = 0.0f;
    if (at >= 0 && (int64_t)at < V) {
        float x;
        if constexpr (sizeof(T) == 2) x = lo_bf16(*gbl<T>(row + at));
        else x = *gbl<float>(row + at);
        lp = none ? kNegInf : (x - a.m) - log_s;
    }
    *gbl_mut<float>(to.logprob + r) = lp;
    if (to.stats) {
        *gbl_mut<float>(to.stats + 2 * r) = none ? kNegInf : a.m;
        *gbl_mut<float>(to.stats + 2 * r + 1) = log_s;
    }
    if (to.entropy) *gbl_mut<float>(to.entropy + r) = none ? 0.0f : log_s - (float)(a.t / a.s);
}
__device__ __forceinline__ void put_alternative(const Outputs& to, int64_t r, int at, uint64_t o, float m, float log_s) {
    *gbl_mut<int32_t>(to.top_ids + r * to.top + at) = o ? id_of(o) : -1;
    *gbl_mut<float>(to.top_logprobs + r * to.top + at) = o ? (logit_of(o) - m) - log_s : kNegInf;
}

// One workgroup a row, or, with kPart, a part of one, whose sums and best logits go
// to the workspace. A lane has 32 logits in hand at a time; four waves a SIMD have to
// fit (with 130 registers 257 rows of 50001 fp32 with 20 alternatives took 31 us, not 25).
struct Parts {
    Sums* sums;            // [row][parts]
    uint64_t* found;       // [row][parts][top]
    int64_t units;         // vectors of a part
    int32_t parts;
};
template <class T, class Id, int kThreads, bool kEntropy, bool kTop, bool kPart>
__global__ __launch_bounds__(kThreads, 4) void row_logprobs(const T* logits, int64_t stride, int64_t tokens, int64_t V,
                                                         const Id* targets, Outputs to, Parts parts) {
    constexpr int N = kVecOf<T>, KU = 32 / N, kWaves = kThreads / 64;
    __shared__ Sums part[kWaves];
    __shared__ std::conditional_t<kTop, TopSpace, int> space;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t units = (V + N - 1) / N;
    for (int64_t r = blockIdx.x; r < tokens; r += gridDim.x) {
        const T* row = logits + r * stride;
        const int64_t begin = kPart ? blockIdx.y * parts.units : 0;
        const int64_t end = kPart && begin + parts.units < units ? begin + parts.units : units;
        const int64_t whole = end < V / N ? end : V / N;
        Sums a{kLowest, 0.0, 0.0};
        float most = kNegInf;
        int64_t unit = -1;
        for (int64_t u0 = begin; u0 < end; u0 += KU * kThreads) {
            float v[KU][N];
            float m = a.m;
            if (u0 + KU * kThreads <= whole) {
                u32x4 raw[KU];
#pragma unroll
                for (int j = 0; j < KU; ++j) raw[j] = load16_once(row + (u0 + j * kThreads + tid) * N);
#pragma unroll
                for (int j = 0; j < KU; ++j) widen(raw[j], v[j]);
            } else {
#pragma unroll
                for (int j = 0; j < KU; ++j) {
                    const int64_t u = u0 + j * kThreads + tid, left = u < end ? V - u * N : 0;
#pragma unroll
                    for (int c = 0; c < N; ++c) v[j][c] = kNegInf;
                    if (left <= 0) continue;
                    widen(load_row(row + u * N, left < N ? (int)left : N), v[j]);
#pragma unroll
                    for (int c = 0; c < N; ++c)
                        if (c >= left) v[j][c] = kNegInf;
                }
            }
#pragma unroll
            for (int j = 0; j < KU; ++j) {
                float b = v[j][0];
#pragma unroll
                for (int c = 1; c < N; ++c) b = fmaxf(b, v[j][c]);
                if (kTop && b > most) {
                    most = b;
                    unit = u0 + j * kThreads + tid;
                }
                m = fmaxf(m, b);
            }
            add<kEntropy>(a, v, m);
        }
        a = join_lanes<64>(a);
        if (kWaves > 1) {
            if (lane == 0) part[wave] = a;
            __syncthreads();
            a = join_lanes<kWaves>(part[lane % kWaves]);
        }
        if constexpr (kTop)
            if (a.s != a.s) largest_of<T, kThreads>(row, V, begin, end, most, unit);
        if constexpr (kPart) {
            const int64_t p = r * parts.parts + blockIdx.y;
            if (tid == 0) parts.sums[p] = a;
            if constexpr (kTop)
                alternatives<T, kThreads>(row, V, begin, end, most, unit, to.top, space,
                                          [&](int at, uint64_t o) { parts.found[p * to.top + at] = o; });
        } else {
            const float log_s = a.s == 0.0 ? kNegInf : log_of(a.s);
            if (tid == 0) put_row(to, row, r, V, targets, a, log_s);
            if constexpr (kTop)
                alternatives<T, kThreads>(row, V, begin, end, most, unit, to.top, space,
                                          [&](int at, uint64_t o) { put_alternative(to, r, at, o, a.m, log_s); });
        }
        __syncthreads();
    }
}

// A row's parts joined, by one workgroup; the alternatives of the parts are ranked
// as those of a row's lanes are.
constexpr int kMostParts = 16, kJoinThreads = 256;
template <class T, class Id>
__global__ __launch_bounds__(kJoinThreads) void join_parts(const T* logits, int64_t stride, int64_t tokens, int64_t V,
                                                           const Id* targets, Outputs to, Parts parts) {
    __shared__ TopSpace space;
    const int lane = threadIdx.x & 63;
    for (int64_t r = blockIdx.x; r < tokens; r += gridDim.x) {
        Sums a{kLowest, 0.0, 0.0};
        if (lane % kMostParts < parts.parts) a = parts.sums[r * parts.parts + lane % kMostParts];
        a = join_lanes<kMostParts>(a);
        const float log_s = a.s == 0.0 ? kNegInf : log_of(a.s);
        if (threadIdx.x == 0) put_row(to, logits + r * stride, r, V, targets, a, log_s);
        if (to.top == 0) continue;
        const int all = parts.parts * to.top;      // at most kFound
        if (threadIdx.x == 0) space.count = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < all; i += kJoinThreads) {
            const uint64_t o = parts.found[r * all + i];
            if (o) space.found[atomicAdd(&space.count, 1)] = o;
        }
        __syncthreads();
        rank_found(space, space.count, kJoinThreads, to.top,
                   [&](int at, uint64_t o) { put_alternative(to, r, at, o, a.m, log_s); });
        __syncthreads();
    }
}

// p = exp(x - m - log s) = 2^(x log2(e) - c) 2^d, as in the forward pass; the
// factor 2^d goes to the row's factors. c has to come from the same fp32 log2(e) that x
// is multiplied by: then its error (1.3e-8 of it) is one of x - m - log s, with another
// constant one of x, which a row far from zero makes as large as it likes. A stream of
// reads and writes: 4096 x 131072 bf16 in 361 us (5.6 TB/s). A lane has KU vectors in
// hand at a time (one: 497 us).
constexpr int kGradVectors = 4;
template <class T, class Id, int kThreads, bool kEntropy>
__global__ __launch_bounds__(kThreads) void row_logprobs_grad(
    const T* logits, int64_t stride, int64_t tokens, int64_t V, const Id* targets, const float* stats,
    const float* dlogprob, const float* entropy, const float* dentropy, T* dlogits, int64_t dstride) {
    constexpr int N = kVecOf<T>, KU = kGradVectors;
    const int64_t units = (V + N - 1) / N;
    for (int64_t r = blockIdx.x; r < tokens; r += gridDim.x) {
        const Id id = *gbl<Id>(targets + r);
        const int64_t at = id >= 0 && (int64_t)id < V ? (int64_t)id : -1;
        const float m = *gbl<float>(stats + 2 * r), log_s = *gbl<float>(stats + 2 * r + 1);
        const float d = at >= 0 ? *gbl<float>(dlogprob + r) : 0.0f;
        const float h = kEntropy ? *gbl<float>(dentropy + r) : 0.0f, H = kEntropy ? *gbl<float>(entropy + r) : 0.0f;
        const bool zero = (at < 0 && !kEntropy) || m == kNegInf, tame = fabsf(m) < kTame;
        const double exact = ((double)m + (double)log_s) * (double)kLog2e;
        const float c0 = (float)exact, rest = (float)((double)c0 - exact), f = __builtin_amdgcn_exp2f(rest);
        for (int64_t u0 = (int64_t)blockIdx.y * KU * kThreads; u0 < units; u0 += (int64_t)gridDim.y * KU * kThreads) {
            float v[KU][N];
            if (!zero) {
                u32x4 raw[KU];
#pragma unroll
                for (int j = 0; j < KU; ++j) {
                    const int64_t u = u0 + j * kThreads + threadIdx.x, left = V - u * N;
                    raw[j] = u32x4{};
                    if (left > 0) raw[j] = load_row<true>(logits + r * stride + u * N, left < N ? (int)left : N);
                }
#pragma unroll
                for (int j = 0; j < KU; ++j) widen(raw[j], v[j]);
#pragma unroll
                for (int j = 0; j < KU; ++j) {
                    const int64_t first = (u0 + j * kThreads + threadIdx.x) * N;
#pragma unroll
                    for (int c = 0; c < N; ++c) {
                        float p, lp;
                        if (tame) {
                            const float q = __builtin_fmaf(v[j][c], kLog2e, -c0);
                            p = __builtin_amdgcn_exp2f(q) * f;
                            lp = (fmaxf(q, kFar2) + rest) * kLn2;
                        } else {
                            lp = (v[j][c] - m) - log_s;
                            p = exp_of(lp);
                            lp = fmaxf(lp, kFar);
                        }
                        float g = first + c == at ? d : 0.0f;
                        g = __builtin_fmaf(-d, p, g);
                        if (kEntropy) g = __builtin_fmaf(-h, p * (lp + H), g);
                        v[j][c] = g;
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < KU; ++j)
#pragma unroll
                    for (int c = 0; c < N; ++c) v[j][c] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < KU; ++j) {
                const int64_t u = u0 + j * kThreads + threadIdx.x, left = V - u * N;
                if (left > 0) store_row(dlogits + r * dstride + u * N, left < N ? (int)left : N, narrow(v[j]));
            }
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

// Threads of a row's workgroup: as many as give 4096 waves with the rows there are
// (four a SIMD, what fits with alternatives), two vectors each at least, and four
// waves for rows over 128 KiB. us with 64 / 256 threads: 4096 rows of 4000 bf16
// 12 / 22, of 8000 18 / 25 (with 8 alternatives 27 / 44), of 32000 48 / 54, of 131072
// 194 / 183; 200 rows of 16000 10 / 6. 257 rows of 50001 fp32 with 20 alternatives: 24
// with 512, 33 with 1024; 700 rows 40 with 256, 42 with 512, 56 with 1024.
int threads_of(int64_t tokens, int64_t units) {
    int waves = units > 8192 ? 4 : 1;
    while (waves < 16 && 2 * waves * tokens <= 4096) waves *= 2;
    while (waves > 1 && waves * 128 > units) waves /= 2;
    return 64 * waves;
}
// Parts of a row, of 16 KiB at least, for few tokens. One row of 131072 bf16 with 8
// alternatives: 12.3 us in 16 parts and their join, 17.2 in one workgroup; 32 rows
// 14.4 and 18.3; 128 rows 21.6 and 21.0.
int32_t parts_of(int64_t tokens, int64_t units) {
    if (tokens < 1 || tokens > 64) return 1;
    const int64_t p = units / 1024 < kMostParts ? units / 1024 : kMostParts;
    return p < 2 ? 1 : (int32_t)p;
}

int64_t units_of(int32_t dtype, int64_t vocab) {
    const int64_t n = dtype == TIDE_DTYPE_FP32 ? 4 : 8;
    return (vocab + n - 1) / n;
}

template <class F>
hipError_t with_types(int32_t dtype, int32_t id_bytes, F&& go) {
    if (dtype == TIDE_DTYPE_BF16) return id_bytes == 4 ? go(uint16_t{}, int32_t{}) : go(uint16_t{}, int64_t{});
    return id_bytes == 4 ? go(float{}, int32_t{}) : go(float{}, int64_t{});
}

}  // namespace

extern "C" {

tide_status tide_token_logprobs_workspace(int32_t dtype, int64_t tokens, int64_t vocab, int32_t top,
                                          int64_t* bytes) {
    return guarded([&]() -> tide_status {
        if (!bytes) return fail(TIDE_ERR_INVALID_ARG, "bytes is NULL");
        TIDE_TRY(check(dtype, tokens, vocab, 4));
        if (top < 0) return fail(TIDE_ERR_INVALID_ARG, "negative top");
        if (top > kMostTop) return fail(TIDE_ERR_UNSUPPORTED, "%d alternatives: at most %d", top, kMostTop);
        const int64_t parts = parts_of(tokens, units_of(dtype, vocab));
        *bytes = parts > 1 ? tokens * parts * ((int64_t)sizeof(Sums) + 8 * top) : 0;
        return TIDE_OK;
    });
}

tide_status tide_token_logprobs(int32_t dtype, const void* logits, int64_t logits_stride,
                                int64_t tokens, int64_t vocab, const void* targets,
                                int32_t id_bytes, float* logprob, float* stats, float* entropy,
                                int32_t top, int32_t* top_ids, float* top_logprobs, void* workspace,
                                int64_t workspace_bytes, void* stream) {
    return guarded([&]() -> tide_status {
        TIDE_TRY(check(dtype, tokens, vocab, id_bytes));
        int64_t need = 0;
        TIDE_TRY(tide_token_logprobs_workspace(dtype, tokens, vocab, top, &need));
        if (need > 0 && (!workspace || workspace_bytes < need))
            return fail(TIDE_ERR_INVALID_ARG, "workspace holds %lld bytes, %lld needed",
                        (long long)(workspace ? workspace_bytes : 0), (long long)need);
        const int32_t size = dtype == TIDE_DTYPE_FP32 ? 4 : 2;
        Mat rd[2], wr[6];
        TIDE_TRY(matrix("logits", logits, tokens, vocab, logits_stride, size, &rd[0]));
        TIDE_TRY(matrix("targets", targets, 1, tokens, tokens, id_bytes, &rd[1]));
        TIDE_TRY(matrix("logprob", logprob, 1, tokens, tokens, 4, &wr[0]));
        TIDE_TRY(matrix("stats", stats, stats ? tokens : 0, 2, 2, 4, &wr[1]));
        TIDE_TRY(matrix("entropy", entropy, entropy ? 1 : 0, tokens, tokens, 4, &wr[2]));
        TIDE_TRY(matrix("top_ids", top_ids, tokens, top, top, 4, &wr[3]));
        TIDE_TRY(matrix("top_logprobs", top_logprobs, tokens, top, top, 4, &wr[4]));
        TIDE_TRY(matrix("workspace", workspace, 1, need / 8, need / 8, 8, &wr[5]));
        TIDE_TRY(no_overlap(wr, 6, rd, 2));
        if (tokens == 0) return TIDE_OK;
        const Outputs to{logprob, stats, entropy, top_ids, top_logprobs, top};
        const int64_t units = units_of(dtype, vocab);
        Parts parts{(Sums*)workspace, nullptr, units, parts_of(tokens, units)};
        parts.found = (uint64_t*)(parts.sums + tokens * parts.parts);
        parts.units = (units + parts.parts - 1) / parts.parts;
        return on_stream(stream, [&](hipStream_t s) {
            const int threads = threads_of(tokens, units);
            return with_types(dtype, id_bytes, [&](auto type, auto id) {
                using T = decltype(type);
                using Id = decltype(id);
                const auto go = [&](auto n, auto split, auto with_entropy, auto with_top) {
                    const dim3 grid((uint32_t)(tokens < (1 << 20) ? tokens : (1 << 20)), split.value ? parts.parts : 1);
                    return enqueue(row_logprobs<T, Id, n.value, with_entropy.value, with_top.value, split.value>, grid,
                                   n.value, 0, s, (const T*)logits, logits_stride, tokens, vocab, (const Id*)targets, to,
                                   parts);
                };
                using Yes = std::true_type;
                using No = std::false_type;
                const auto with = [&](auto n, auto split) {
                    if (entropy) return top ? go(n, split, Yes{}, Yes{}) : go(n, split, Yes{}, No{});
                    return top ? go(n, split, No{}, Yes{}) : go(n, split, No{}, No{});
                };
                if (parts.parts > 1) {
                    const hipError_t e = with(std::integral_constant<int, 256>{}, Yes{});
                    if (e != hipSuccess) return e;
                    return enqueue(join_parts<T, Id>, dim3((uint32_t)tokens), kJoinThreads, 0, s, (const T*)logits,
                                   logits_stride, tokens, vocab, (const Id*)targets, to, parts);
                }
                return threads == 64    ? with(std::integral_constant<int, 64>{}, No{})
                       : threads == 128 ? with(std::integral_constant<int, 128>{}, No{})
                       : threads == 256 ? with(std::integral_constant<int, 256>{}, No{})
                       : threads == 512 ? with(std::integral_constant<int, 512>{}, No{})
                                        : with(std::integral_constant<int, 1024>{}, No{});
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
            // A wave a row where it is short: 8192 rows of 1000 bf16 11 us, 24 with 256 threads.
            const bool small = units_of(dtype, vocab) <= 1024;
            const int64_t per = kGradVectors * (small ? 64 : 256), groups = (units_of(dtype, vocab) + per - 1) / per;
            const dim3 grid((uint32_t)(tokens < (1 << 20) ? tokens : (1 << 20)),
                            (uint32_t)(groups < 32768 ? groups : 32768));
            return with_types(dtype, id_bytes, [&](auto type, auto id) {
                using T = decltype(type);
                using Id = decltype(id);
                const auto go = [&](auto n, auto with_entropy) {
                    return enqueue(row_logprobs_grad<T, Id, n.value, with_entropy.value>, grid, n.value, 0, s,
                                   (const T*)logits, logits_stride, tokens, vocab, (const Id*)targets, stats, dlogprob,
                                   entropy, dentropy, (T*)dlogits, dlogits_stride);
                };
                using Wave = std::integral_constant<int, 64>;
                using Four = std::integral_constant<int, 256>;
                if (dentropy) return small ? go(Wave{}, std::true_type{}) : go(Four{}, std::true_type{});
                return small ? go(Wave{}, std::false_type{}) : go(Four{}, std::false_type{});
            });
        });
    });
}

}  // extern "C"
