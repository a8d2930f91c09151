// Queries and keys normalised head by head and rotated by position
// (tide_norm_rotate) and the gradient (tide_norm_rotate_grad) for gfx950.
//
// A lane holds both elements of each of its pairs, so the rotation needs no
// other lane: with halves as pairs it loads one vector from either half of the
// rotated elements, with adjacent pairs two neighbouring vectors. The lanes of a
// head join its sum of squares (and, in the gradient, one dot product) by
// exchanges. Both are HBM streams that touch each byte once; the angles' tables,
// one row a token, come from the caches.
#include <algorithm>
#include <climits>
#include <cmath>

#include "device.hpp"
#include "host.hpp"

using namespace tide;

namespace {

constexpr int kThreads = 256;
constexpr int kMostDim = 512;
constexpr int32_t kMostHeads = 1 << 24;

struct Heads {
    const void* data;
    int64_t token_stride, head_stride;
    int32_t heads;
};
struct Turn {
    const void* positions;
    const float* cos;
    const float* sin;
    int64_t rows, stride;
    int32_t id_bytes, pairs;
};

typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));

// A lane's slot of W pairs: elements first(s) + c and second(s) + c for halves,
// first(s) + 2 c and + 2 c + 1 for adjacent pairs. Elements that are not rotated
// are paired alike, (i, i + half of them).
template <class T, int W, bool kAdjacent>
struct Slot {
    static __device__ __forceinline__ void where(int s, int half, int pairs, int& a, int& b) {
        const int p = s * W;
        if (kAdjacent) {
            a = 2 * p;
            b = a + W;
        } else {
            a = p < pairs ? p : p + pairs;
            b = p < pairs ? p + pairs : p + half;
        }
    }
    // What a slot's loads give, before it is widened.
    struct Raw {
        u32x4 p, q;
    };
    template <bool kOnce = false>
    static __device__ __forceinline__ Raw load(const T* x, int a, int b) {
        Raw r{};
        if constexpr (W == 1) {
            if constexpr (sizeof(T) == 2) {
                r.p[0] = (uint32_t)*gbl<uint16_t>(x + a) << 16;
                r.q[0] = (uint32_t)*gbl<uint16_t>(x + b) << 16;
            } else {
                r.p[0] = *gbl<uint32_t>(x + a);
                r.q[0] = *gbl<uint32_t>(x + b);
            }
        } else if constexpr (W * sizeof(T) == 8) {
            const u32x2 p = *gbl<u32x2_a2>(x + a), q = *gbl<u32x2_a2>(x + b);
            r.p[0] = p[0];
            r.p[1] = p[1];
            r.q[0] = q[0];
            r.q[1] = q[1];
        } else {
            r.p = kOnce ? load16_once(x + a) : load16(x + a);
            r.q = kOnce ? load16_once(x + b) : load16(x + b);
        }
        return r;
    }
    static __device__ __forceinline__ void open(const Raw& r, float (&u)[W], float (&v)[W]) {
        if constexpr (W == 1) {
            u[0] = __uint_as_float(r.p[0]);
            v[0] = __uint_as_float(r.q[0]);
        } else {
            float p[kVecOf<T>], q[kVecOf<T>];
            widen(r.p, p);
            widen(r.q, q);
#pragma unroll
            for (int c = 0; c < W; ++c) {
                u[c] = !kAdjacent ? p[c] : 2 * c < W ? p[2 * c % W] : q[2 * c % W];
                v[c] = !kAdjacent ? q[c] : 2 * c < W ? p[(2 * c + 1) % W] : q[(2 * c + 1) % W];
            }
        }
    }
    static __device__ __forceinline__ void store(T* x, int a, int b, const float (&u)[W], const float (&v)[W]) {
        if constexpr (W == 1) {
            if constexpr (sizeof(T) == 2) {
                const uint32_t w = pack_bf16(u[0], v[0]);
                *gbl_mut<uint16_t>(x + a) = (uint16_t)w;
                *gbl_mut<uint16_t>(x + b) = (uint16_t)(w >> 16);
            } else {
                *gbl_mut<float>(x + a) = u[0];
                *gbl_mut<float>(x + b) = v[0];
            }
        } else {
            float p[kVecOf<T>] = {}, q[kVecOf<T>] = {};
#pragma unroll
            for (int c = 0; c < W; ++c) {
                p[c] = !kAdjacent ? u[c] : c & 1 ? v[c / 2] : u[c / 2];
                q[c] = !kAdjacent ? v[c] : c & 1 ? v[W / 2 + c / 2] : u[W / 2 + c / 2];
            }
            const u32x4 lo = narrow(p), hi = narrow(q);
            if constexpr (W * sizeof(T) == 8) {
                *gbl_mut<u32x2_a2>(x + a) = u32x2{lo[0], lo[1]};
                *gbl_mut<u32x2_a2>(x + b) = u32x2{hi[0], hi[1]};
            } else {
                store16(x + a, lo);
                store16(x + b, hi);
            }
        }
    }
};

// Row of the rotation's tables for token t, -1 where it is not rotated.
__device__ __forceinline__ int64_t table_row(const Turn& turn, int64_t t) {
    if (turn.pairs == 0) return -1;
    int64_t p = t;
    if (turn.positions)
        p = turn.id_bytes == 4 ? *gbl<int32_t>((const int32_t*)turn.positions + t)
                               : *gbl<int64_t>((const int64_t*)turn.positions + t);
    return p >= 0 && p < turn.rows ? p : -1;
}
// cos and sin of a slot's pairs; 1 and 0 where they are not rotated.
template <int W>
__device__ __forceinline__ void angles(const Turn& turn, int64_t row, int s, float (&c)[W], float (&n)[W]) {
    if (row >= 0 && s * W < turn.pairs) {
        const int64_t at = row * turn.stride + s * W;
        if constexpr (W == 1) {
            c[0] = *gbl<float>(turn.cos + at);
            n[0] = *gbl<float>(turn.sin + at);
        } else {
#pragma unroll
            for (int i = 0; i < W / 4; ++i) {
                const u32x4 x = load16(turn.cos + at + 4 * i), y = load16(turn.sin + at + 4 * i);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    c[4 * i + j] = __uint_as_float(x[j]);
                    n[4 * i + j] = __uint_as_float(y[j]);
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            c[i] = 1.0f;
            n[i] = 0.0f;
        }
    }
}

__device__ __forceinline__ float head_sum(float v, int lanes) {
    for (int d = lanes >> 1; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}
// 1 / sqrt(v); the instruction takes no subnormals.
__device__ __forceinline__ float inverse_root(float v) {
    const bool low = v < 0x1p-100f;
    const float r = __builtin_amdgcn_rsqf(low ? v * 0x1p+96f : v);
    return low ? r * 0x1p+48f : r;
}

// A slot's weights, 1 where there are none.
template <class T, int W, bool kAdjacent>
__device__ __forceinline__ void weights(const void* w, int a, int b, float (&u)[W], float (&v)[W]) {
    using S = Slot<T, W, kAdjacent>;
    constexpr uint32_t kOne = sizeof(T) == 2 && W > 1 ? 0x3F803F80u : 0x3F800000u;
    typename S::Raw r{{kOne, kOne, kOne, kOne}, {kOne, kOne, kOne, kOne}};
    if (w) r = S::load((const T*)w, a, b);
    S::open(r, u, v);
}

// W pairs a slot, NS slots a lane, 2^lane_log2 lanes a head, 64 >> lane_log2 heads a
// wave at once and KH times that in all, of one token: its angles are loaded once
// for them, and all their loads are under way before the first is used. 8192 tokens
// of 72 heads of 128: 62 us with KH 1, 55 with 2, 56 with 3, 59 with 4 (302 MB moved:
// 5.5 TB/s). A few tokens take KH 1, for more waves.
template <class T, int W, int NS, int KH, bool kAdjacent>
__global__ __launch_bounds__(kThreads) void rotate_heads(Heads q, Heads k, Heads qo, Heads ko,
                                                         const void* qw, const void* kw, Turn turn,
                                                         int64_t waves, int32_t parts, int dim,
                                                         float eps, int lane_log2) {
    using S = Slot<T, W, kAdjacent>;
    const int lanes = 1 << lane_log2, lane = threadIdx.x & (lanes - 1), at_once = 64 >> lane_log2;
    const int half = dim / 2, slots = half / W, all = q.heads + k.heads;
    const float per_element = 1.0f / (float)dim;
    int a[NS], b[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) S::where(lane + i * lanes, half, turn.pairs, a[i], b[i]);
    for (int64_t w = (int64_t)blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); w < waves;
         w += (int64_t)gridDim.x * (kThreads / 64)) {
        const int64_t t = w / parts;
        const int first = (int)(w - t * parts) * KH * at_once + ((threadIdx.x & 63) >> lane_log2);
        typename S::Raw raw[KH][NS];
#pragma unroll
        for (int j = 0; j < KH; ++j) {
            const int h = first + j * at_once;
            const T* x = h < q.heads ? (const T*)q.data + t * q.token_stride + h * q.head_stride
                                     : (const T*)k.data + t * k.token_stride + (h - q.heads) * k.head_stride;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                raw[j][i] = typename S::Raw{};
                if (h < all && lane + i * lanes < slots) raw[j][i] = S::template load<true>(x, a[i], b[i]);
            }
        }
        const int64_t row = table_row(turn, t);
        float c[NS][W], n[NS][W];
#pragma unroll
        for (int i = 0; i < NS; ++i) angles<W>(turn, lane + i * lanes < slots ? row : -1, lane + i * lanes, c[i], n[i]);
#pragma unroll
        for (int j = 0; j < KH; ++j) {
            const int h = first + j * at_once;
            float u[NS][W], v[NS][W], sum = 0.0f;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                S::open(raw[j][i], u[i], v[i]);
#pragma unroll
                for (int e = 0; e < W; ++e) sum = __builtin_fmaf(u[i][e], u[i][e], __builtin_fmaf(v[i][e], v[i][e], sum));
            }
            const float scale = inverse_root(__builtin_fmaf(head_sum(sum, lanes), per_element, eps));
            T* y = h < q.heads ? (T*)qo.data + t * qo.token_stride + h * qo.head_stride
                               : (T*)ko.data + t * ko.token_stride + (h - q.heads) * ko.head_stride;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                if (h >= all || lane + i * lanes >= slots) continue;
                float wu[W], wv[W];
                weights<T, W, kAdjacent>(h < q.heads ? qw : kw, a[i], b[i], wu, wv);
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    const float p = u[i][e] * scale * wu[e], o = v[i][e] * scale * wv[e];
                    u[i][e] = __builtin_fmaf(p, c[i][e], -(o * n[i][e]));
                    v[i][e] = __builtin_fmaf(p, n[i][e], o * c[i][e]);
                }
                S::store(y, a[i], b[i], u[i], v[i]);
            }
        }
    }
}

// The gradient of one set of heads; partial (when not NULL) gets this
// workgroup's sum of g * n, dim fp32 in element order. A wave takes 64 >> lane_log2
// heads of a token at a time, then those some waves further on. Bound by HBM and by
// the waves that 104 registers leave (four a SIMD): 8191 tokens of 36 heads of 128 in
// 46 us, 231 MB. (The next ones' loads under way meanwhile were 4% slower, 512 or 2048
// workgroups instead of 1024 26 and 16%, queries and then keys by the same workgroups
// 9%.)
struct Steps {
    int64_t t;             // the step between a wave's turns: tokens, and sets of heads
    int32_t part, parts;   // sets of heads of a token
};
template <class T, int W, int NS, bool kAdjacent>
__device__ __forceinline__ void grad_of(const Heads& x, const Heads& dy, const Heads& dx, const void* w,
                                        const Turn& turn, int64_t tokens, int dim, float eps, int lane_log2,
                                        Steps step, int64_t group0, float* partial, float* joint) {
    using S = Slot<T, W, kAdjacent>;
    const int lanes = 1 << lane_log2, lane = threadIdx.x & (lanes - 1), group = threadIdx.x >> lane_log2;
    const int half = dim / 2, slots = half / W, at_once = 64 >> lane_log2;
    const float per_element = 1.0f / (float)dim;
    float wu[NS][W], wv[NS][W], au[NS][W] = {}, av[NS][W] = {};
    int a[NS], b[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int s = lane + i * lanes;
        S::where(s, half, turn.pairs, a[i], b[i]);
        if (s < slots) weights<T, W, kAdjacent>(w, a[i], b[i], wu[i], wv[i]);
    }
    const int64_t w0 = ((int64_t)blockIdx.x - group0) * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int64_t t = step.parts ? w0 / step.parts : tokens;
    int32_t part = (int32_t)(w0 - t * step.parts);
    while (t < tokens) {
        const int h = part * at_once + ((threadIdx.x & 63) >> lane_log2);
        const bool mine = h < x.heads;
        const T* px = (const T*)x.data + t * x.token_stride + h * x.head_stride;
        const T* py = (const T*)dy.data + t * dy.token_stride + h * dy.head_stride;
        typename S::Raw rx[NS] = {}, ry[NS] = {};
#pragma unroll
        for (int i = 0; i < NS; ++i)
            if (mine && lane + i * lanes < slots) {
                rx[i] = S::load(px, a[i], b[i]);
                ry[i] = S::load(py, a[i], b[i]);
            }
        const int64_t row = table_row(turn, t);
        float u[NS][W], v[NS][W], gu[NS][W], gv[NS][W], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int s = lane + i * lanes;
            float c[W], n[W];
            S::open(rx[i], u[i], v[i]);
            S::open(ry[i], gu[i], gv[i]);
            angles<W>(turn, s < slots ? row : -1, s, c, n);
#pragma unroll
            for (int j = 0; j < W; ++j) {
                sum = __builtin_fmaf(u[i][j], u[i][j], __builtin_fmaf(v[i][j], v[i][j], sum));
                const float p = gu[i][j], o = gv[i][j];
                gu[i][j] = __builtin_fmaf(p, c[j], o * n[j]);
                gv[i][j] = __builtin_fmaf(o, c[j], -(p * n[j]));
            }
        }
        const float scale = inverse_root(__builtin_fmaf(head_sum(sum, lanes), per_element, eps));
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            if (!mine || lane + i * lanes >= slots) continue;
#pragma unroll
            for (int j = 0; j < W; ++j) {
                u[i][j] *= scale;
                v[i][j] *= scale;
                au[i][j] = __builtin_fmaf(gu[i][j], u[i][j], au[i][j]);
                av[i][j] = __builtin_fmaf(gv[i][j], v[i][j], av[i][j]);
                gu[i][j] *= wu[i][j];
                gv[i][j] *= wv[i][j];
                dot = __builtin_fmaf(gu[i][j], u[i][j], __builtin_fmaf(gv[i][j], v[i][j], dot));
            }
        }
        dot = head_sum(dot, lanes) * per_element;
        T* pd = (T*)dx.data + t * dx.token_stride + h * dx.head_stride;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            if (!mine || lane + i * lanes >= slots) continue;
#pragma unroll
            for (int j = 0; j < W; ++j) {
                u[i][j] = scale * __builtin_fmaf(-u[i][j], dot, gu[i][j]);
                v[i][j] = scale * __builtin_fmaf(-v[i][j], dot, gv[i][j]);
            }
            S::store(pd, a[i], b[i], u[i], v[i]);
        }
        t += step.t;
        part += step.part;
        if (part >= step.parts) {
            part -= step.parts;
            ++t;
        }
    }
    if (!partial) return;
    // The workgroup's heads in LDS, [group][pair][2], joined in order.
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int s = lane + i * lanes;
        if (s >= slots) continue;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            joint[group * dim + 2 * (s * W + j)] = au[i][j];
            joint[group * dim + 2 * (s * W + j) + 1] = av[i][j];
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < dim; e += kThreads) {
        float sum = 0.0f;
        for (int g = 0; g < kThreads >> lane_log2; ++g) sum += joint[g * dim + e];
        const int p = e / 2;
        int at = e;
        if (!kAdjacent) at = p < turn.pairs ? p + (e & 1) * turn.pairs : p + (e & 1 ? half : turn.pairs);
        *gbl_mut<float>(partial + at) = sum;
    }
}

// The first workgroups take the queries, the others the keys.
template <class T, int W, int NS, bool kAdjacent>
__global__ __launch_bounds__(kThreads) void rotate_heads_grad(Heads q, Heads k, Heads dqo, Heads dko,
                                                              Heads dq, Heads dk, const void* qw,
                                                              const void* kw, Turn turn, int64_t tokens,
                                                              int dim, float eps, int lane_log2, Steps of_q,
                                                              Steps of_k, int64_t of_queries, float* partial,
                                                              int want_q, int want_k) {
    __shared__ float joint[kThreads * 2 * W * NS];
    float* mine = partial + (int64_t)blockIdx.x * dim;
    if (blockIdx.x < of_queries)
        grad_of<T, W, NS, kAdjacent>(q, dqo, dq, qw, turn, tokens, dim, eps, lane_log2, of_q, 0, want_q ? mine : nullptr,
                                     joint);
    else
        grad_of<T, W, NS, kAdjacent>(k, dko, dk, kw, turn, tokens, dim, eps, lane_log2, of_k, of_queries,
                                     want_k ? mine : nullptr, joint);
}

// Weights' gradients: the workgroups' sums in order, 64 runs of them at once, 16
// elements a workgroup (819 and 205 sums of 128: 4.6 us; 64 elements in 16 runs 6).
constexpr int kRuns = 64, kColumns = 16;
template <class T>
__global__ __launch_bounds__(kRuns * kColumns) void join_weights(const float* partial, int64_t of_queries,
                                                                 int64_t of_keys, int dim, T* dqw, T* dkw,
                                                                 int accumulate) {
    __shared__ float part[kRuns][kColumns];
    const int c = threadIdx.x % kColumns, e = blockIdx.x * kColumns + c, run = threadIdx.x / kColumns;
    T* to = blockIdx.y ? dkw : dqw;
    if (!to) return;
    const int64_t first = blockIdx.y ? of_queries : 0, groups = blockIdx.y ? of_keys : of_queries;
    const int64_t per = (groups + kRuns - 1) / kRuns;
    const int64_t end = (run + 1) * per < groups ? (run + 1) * per : groups;
    float sum = 0.0f;
    if (e < dim)
        for (int64_t g = run * per; g < end; g += 16) {
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = g + i < end ? *gbl<float>(partial + (first + g + i) * dim + e) : 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) sum += v[i];
        }
    part[run][c] = sum;
    __syncthreads();
    if (run < 8) {
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += part[8 * run + i][c];
    }
    __syncthreads();
    if (run < 8) part[run][c] = sum;
    __syncthreads();
    if (run || e >= dim) return;
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += part[i][c];
    if constexpr (sizeof(T) == 2) {
        if (accumulate) sum += lo_bf16(*gbl<T>(to + e));
        *gbl_mut<T>(to + e) = (T)pack_bf16(sum, 0.0f);
    } else {
        if (accumulate) sum += *gbl<float>(to + e);
        *gbl_mut<float>(to + e) = sum;
    }
}

// Workgroups of the gradient: each leaves a partial sum of the weights' gradients.
constexpr int64_t kMostGroups = 1024;
int64_t grad_groups(int64_t tokens, int64_t heads, int dim) {
    const int64_t rows = tokens * heads, per = dim <= 64 ? 16 : 8;
    const int64_t g = (rows + per - 1) / per;
    return g < 1 ? 1 : g < kMostGroups ? g : kMostGroups;
}

tide_status check_dims(int64_t tokens, int32_t dim) {
    if (tokens < 0 || dim < 0) return fail(TIDE_ERR_INVALID_ARG, "need tokens and head_dim >= 0");
    if (dim % 2 || dim > kMostDim)
        return fail(TIDE_ERR_UNSUPPORTED, "head_dim %d: even and at most %d", dim, kMostDim);
    if (tokens > INT32_MAX) return fail(TIDE_ERR_UNSUPPORTED, "tokens must be below 2^31");
    return TIDE_OK;
}

// The heads as a matrix of rows (t, h); with several heads the strides have to
// keep heads apart: either a token's heads lie between two tokens, or the
// tokens of a head between two heads.
tide_status check_heads(const char* name, const tide_heads* h, int64_t tokens, int32_t dim, int32_t size,
                        const tide_heads* like, Heads* out, Mat* m) {
    *out = Heads{};
    *m = Mat{name, 0, 0, 0, 0};
    if (!h) {
        if (like) return fail(TIDE_ERR_INVALID_ARG, "%s is NULL", name);
        return TIDE_OK;
    }
    if (h->heads < 0 || h->reserved) return fail(TIDE_ERR_INVALID_ARG, "%s: negative heads or reserved not 0", name);
    if (like && like->heads != h->heads)
        return fail(TIDE_ERR_INVALID_ARG, "%s has %d heads, expected %d", name, h->heads, like->heads);
    *out = Heads{h->data, h->token_stride, h->head_stride, h->heads};
    if (tokens == 0 || h->heads == 0 || dim == 0) {
        out->heads = tokens && dim ? h->heads : 0;
        return TIDE_OK;
    }
    if ((tokens > 1 && h->token_stride < dim) || (h->heads > 1 && h->head_stride < dim))
        return fail(TIDE_ERR_INVALID_ARG, "%s: a stride is below head_dim", name);
    int64_t a = 0, b = 0, span;
    if (__builtin_mul_overflow(tokens - 1, tokens > 1 ? h->token_stride : 0, &a) ||
        __builtin_mul_overflow((int64_t)h->heads - 1, h->heads > 1 ? h->head_stride : 0, &b) ||
        __builtin_add_overflow(a, b, &span) || __builtin_add_overflow(span, (int64_t)dim, &span) ||
        span > INT64_MAX / 8)
        return fail(TIDE_ERR_OVERFLOW, "%s: its extent overflows int64", name);
    if (tokens > 1 && h->heads > 1 && b + dim > h->token_stride && a + dim > h->head_stride)
        return fail(TIDE_ERR_INVALID_ARG, "%s: its heads overlap", name);
    // A token's heads as one row where they lie together, else the whole span.
    const bool rows = tokens > 1 && b + dim <= h->token_stride;
    return rows ? matrix(name, h->data, tokens, b + dim, h->token_stride, size, m)
                : matrix(name, h->data, 1, span, span, size, m);
}

tide_status check_turn(const tide_rotation* r, int64_t tokens, int32_t dim, Turn* out, Mat* m) {
    *out = Turn{};
    m[0] = m[1] = m[2] = Mat{"rotation", 0, 0, 0, 0};
    if (!r) return TIDE_OK;
    if (r->reserved) return fail(TIDE_ERR_INVALID_ARG, "rotation: reserved is not 0");
    if (r->pairs < 0 || 2 * (int64_t)r->pairs > dim)
        return fail(TIDE_ERR_INVALID_ARG, "%d pairs in heads of %d", r->pairs, dim);
    if (r->pairs == 0) return TIDE_OK;
    if (r->positions && r->id_bytes != 4 && r->id_bytes != 8)
        return fail(TIDE_ERR_INVALID_ARG, "positions have 4 or 8 bytes, not %d", r->id_bytes);
    TIDE_TRY(matrix("positions", r->positions, r->positions ? 1 : 0, tokens, tokens, r->id_bytes, &m[0]));
    TIDE_TRY(matrix("cos", r->cos, r->table_rows, r->pairs, r->table_stride, 4, &m[1]));
    TIDE_TRY(matrix("sin", r->sin, r->table_rows, r->pairs, r->table_stride, 4, &m[2]));
    if (!r->positions && r->table_rows < tokens)
        return fail(TIDE_ERR_INVALID_ARG, "the tables have %lld rows for %lld tokens", (long long)r->table_rows,
                    (long long)tokens);
    *out = Turn{r->positions, r->cos, r->sin, r->table_rows, r->table_stride, r->id_bytes, r->pairs};
    return TIDE_OK;
}

// Pairs of a slot: the widest slots that lie on one side of the rotated elements'
// end each: whole vectors, half ones of bf16, or single pairs.
int slot_pairs(int32_t size, int dim, int pairs) {
    const auto fits = [&](int w) { return dim / 2 % w == 0 && pairs % w == 0; };
    return size == 2 && fits(8) ? 8 : fits(4) ? 4 : 1;
}
int lanes_log2(int32_t size, int dim, int pairs) {
    const int slots = dim / 2 / slot_pairs(size, dim, pairs);
    int lg = 0;
    while (lg < 6 && (1 << lg) < slots) ++lg;
    return lg;
}
// Calls go(T, W, NS, adjacent).
template <class F>
hipError_t with_slots(int32_t size, int dim, int pairs, bool adjacent, F&& go) {
    const auto with = [&](auto type, auto w, auto ns) {
        return adjacent ? go(type, w, ns, std::true_type{}) : go(type, w, ns, std::false_type{});
    };
    using One = std::integral_constant<int, 1>;
    using Four = std::integral_constant<int, 4>;
    using Eight = std::integral_constant<int, 8>;
    using Most = std::integral_constant<int, kMostDim / 128>;
    const int w = slot_pairs(size, dim, pairs);
    if (size == 2)
        return w == 8 ? with(uint16_t{}, Eight{}, One{}) : w == 4 ? with(uint16_t{}, Four{}, One{}) : with(uint16_t{}, One{}, Most{});
    return w == 4 ? with(float{}, Four{}, One{}) : with(float{}, One{}, Most{});
}

tide_status check_type(int32_t dtype) {
    if (dtype != TIDE_DTYPE_BF16 && dtype != TIDE_DTYPE_FP32)
        return fail(TIDE_ERR_INVALID_ARG, "dtype %d is not BF16 (0) or FP32 (1)", dtype);
    return TIDE_OK;
}
tide_status check_eps(float eps) {
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(TIDE_ERR_INVALID_ARG, "eps has to be 0 or more and finite");
    return TIDE_OK;
}

}  // namespace

extern "C" {

tide_status tide_norm_rotate(int32_t dtype, int64_t tokens, int32_t head_dim,
                             const tide_heads* q, const tide_heads* k, const void* q_weight,
                             const void* k_weight, float eps, const tide_rotation* rotation,
                             const tide_heads* q_out, const tide_heads* k_out, void* stream) {
    return guarded([&]() -> tide_status {
        TIDE_TRY(check_type(dtype));
        TIDE_TRY(check_dims(tokens, head_dim));
        TIDE_TRY(check_eps(eps));
        if (!q) return fail(TIDE_ERR_INVALID_ARG, "q is NULL");
        if (!k && k_out) return fail(TIDE_ERR_INVALID_ARG, "k_out without k");
        const int32_t size = dtype == TIDE_DTYPE_FP32 ? 4 : 2;
        Heads hq, hk, oq, ok;
        Turn turn;
        Mat rd[7], wr[2];
        TIDE_TRY(check_heads("q", q, tokens, head_dim, size, nullptr, &hq, &rd[0]));
        TIDE_TRY(check_heads("k", k, tokens, head_dim, size, nullptr, &hk, &rd[1]));
        TIDE_TRY(check_heads("q_out", q_out, tokens, head_dim, size, q, &oq, &wr[0]));
        TIDE_TRY(check_heads("k_out", k_out, tokens, head_dim, size, k, &ok, &wr[1]));
        TIDE_TRY(matrix("q_weight", q_weight, q_weight ? 1 : 0, head_dim, head_dim, size, &rd[2]));
        TIDE_TRY(matrix("k_weight", k_weight, k_weight ? 1 : 0, head_dim, head_dim, size, &rd[3]));
        TIDE_TRY(check_turn(rotation, tokens, head_dim, &turn, &rd[4]));
        TIDE_TRY(no_overlap(wr, 2, rd, 7));
        const int64_t all = (int64_t)hq.heads + hk.heads;
        if (all > kMostHeads) return fail(TIDE_ERR_UNSUPPORTED, "q and k have over %d heads", kMostHeads);
        if (all == 0) return TIDE_OK;
        const int lg = lanes_log2(size, head_dim, turn.pairs);
        return on_stream(stream, [&](hipStream_t s) {
            return with_slots(size, head_dim, turn.pairs, rotation && rotation->adjacent,
                              [&](auto type, auto w, auto ns, auto adjacent) {
                const auto go = [&](auto kh) {
                    const int64_t at_once = 64 >> lg, sets = (all + at_once - 1) / at_once;
                    const int64_t parts = (sets + kh.value - 1) / kh.value, waves = tokens * parts;
                    const int64_t groups = (waves + 3) / 4;
                    return enqueue(rotate_heads<decltype(type), w.value, ns.value, kh.value, adjacent.value>,
                                   dim3((uint32_t)(groups < (1 << 22) ? groups : (1 << 22))), kThreads, 0, s, hq, hk, oq,
                                   ok, q_weight, k_weight, turn, waves, (int32_t)parts, (int)head_dim, eps, lg);
                };
                if constexpr (ns.value > 1) return go(std::integral_constant<int, 1>{});
                else return tokens * all < 16384 ? go(std::integral_constant<int, 1>{}) : go(std::integral_constant<int, 2>{});
            });
        });
    });
}

tide_status tide_norm_rotate_grad_workspace(int64_t tokens, int32_t heads, int32_t head_dim,
                                            int64_t* bytes) {
    return guarded([&]() -> tide_status {
        if (!bytes) return fail(TIDE_ERR_INVALID_ARG, "bytes is NULL");
        TIDE_TRY(check_dims(tokens, head_dim));
        if (heads < 0) return fail(TIDE_ERR_INVALID_ARG, "negative heads");
        if (heads > kMostHeads) return fail(TIDE_ERR_UNSUPPORTED, "over %d heads", kMostHeads);
        *bytes = grad_groups(tokens, heads, head_dim) * 2 * head_dim * 4;
        return TIDE_OK;
    });
}

tide_status tide_norm_rotate_grad(int32_t dtype, int64_t tokens, int32_t head_dim,
                                  const tide_heads* dq_out, const tide_heads* dk_out,
                                  const tide_heads* q, const tide_heads* k, const void* q_weight,
                                  const void* k_weight, float eps, const tide_rotation* rotation,
                                  const tide_heads* dq, const tide_heads* dk, void* dq_weight,
                                  void* dk_weight, int32_t accumulate, void* workspace,
                                  int64_t workspace_bytes, void* stream) {
    return guarded([&]() -> tide_status {
        TIDE_TRY(check_type(dtype));
        TIDE_TRY(check_dims(tokens, head_dim));
        TIDE_TRY(check_eps(eps));
        if (!q) return fail(TIDE_ERR_INVALID_ARG, "q is NULL");
        if (!k && (dk_out || dk || dk_weight)) return fail(TIDE_ERR_INVALID_ARG, "gradients of k without k");
        const int32_t size = dtype == TIDE_DTYPE_FP32 ? 4 : 2;
        Heads hq, hk, gq, gk, xq, xk;
        Turn turn;
        Mat rd[9], wr[5];
        TIDE_TRY(check_heads("q", q, tokens, head_dim, size, nullptr, &hq, &rd[0]));
        TIDE_TRY(check_heads("k", k, tokens, head_dim, size, nullptr, &hk, &rd[1]));
        TIDE_TRY(check_heads("dq_out", dq_out, tokens, head_dim, size, q, &gq, &rd[7]));
        TIDE_TRY(check_heads("dk_out", dk_out, tokens, head_dim, size, k, &gk, &rd[8]));
        TIDE_TRY(check_heads("dq", dq, tokens, head_dim, size, q, &xq, &wr[0]));
        TIDE_TRY(check_heads("dk", dk, tokens, head_dim, size, k, &xk, &wr[1]));
        TIDE_TRY(matrix("q_weight", q_weight, q_weight ? 1 : 0, head_dim, head_dim, size, &rd[2]));
        TIDE_TRY(matrix("k_weight", k_weight, k_weight ? 1 : 0, head_dim, head_dim, size, &rd[3]));
        TIDE_TRY(check_turn(rotation, tokens, head_dim, &turn, &rd[4]));
        TIDE_TRY(matrix("dq_weight", dq_weight, dq_weight ? 1 : 0, head_dim, head_dim, size, &wr[2]));
        TIDE_TRY(matrix("dk_weight", dk_weight, dk_weight ? 1 : 0, head_dim, head_dim, size, &wr[3]));
        const int64_t all = (int64_t)hq.heads + hk.heads;
        if (all > kMostHeads) return fail(TIDE_ERR_UNSUPPORTED, "q and k have over %d heads", kMostHeads);
        int64_t need = 0;
        if (dq_weight || dk_weight) TIDE_TRY(tide_norm_rotate_grad_workspace(tokens, (int32_t)all, head_dim, &need));
        if (need > 0 && (!workspace || workspace_bytes < need))
            return fail(TIDE_ERR_INVALID_ARG, "workspace holds %lld bytes, %lld needed",
                        (long long)(workspace ? workspace_bytes : 0), (long long)need);
        TIDE_TRY(matrix("workspace", workspace, 1, need / 4, need / 4, 4, &wr[4]));
        if (need > 0 && (wr[4].base & 15))
            return fail(TIDE_ERR_ALIGNMENT, "workspace is not 16-byte aligned");
        TIDE_TRY(no_overlap(wr, 5, rd, 9));
        if (head_dim == 0 || (all == 0 && need == 0)) return TIDE_OK;
        // The workgroups, shared by queries and keys as their waves' turns are.
        const int lg = lanes_log2(size, head_dim, turn.pairs);
        const int64_t at_once = 64 >> lg, groups = grad_groups(tokens, all, head_dim);
        const int64_t turns_q = (hq.heads + at_once - 1) / at_once, turns_k = (hk.heads + at_once - 1) / at_once;
        const int64_t of_queries = turns_q ? std::max<int64_t>(groups * turns_q / (turns_q + turns_k), 1) : dq_weight ? 1 : 0;
        const int64_t of_keys = turns_k ? std::max<int64_t>(groups - of_queries, 1) : dk_weight ? 1 : 0;
        const auto steps = [](int64_t turns, int64_t of) {
            const int64_t waves = of * (kThreads / 64);
            return turns ? Steps{waves / turns, (int32_t)(waves % turns), (int32_t)turns} : Steps{};
        };
        return on_stream(stream, [&](hipStream_t s) {
            const hipError_t e = with_slots(size, head_dim, turn.pairs, rotation && rotation->adjacent,
                                            [&](auto type, auto w, auto ns, auto adjacent) {
                return enqueue(rotate_heads_grad<decltype(type), w.value, ns.value, adjacent.value>,
                               dim3((uint32_t)(of_queries + of_keys)), kThreads, 0, s, hq, hk, gq, gk, xq, xk, q_weight,
                               k_weight, turn, tokens, (int)head_dim, eps, lg, steps(turns_q, of_queries),
                               steps(turns_k, of_keys), of_queries, (float*)workspace, dq_weight ? 1 : 0,
                               dk_weight ? 1 : 0);
            });
            if (e != hipSuccess || need == 0) return e;
            const dim3 grid((uint32_t)((head_dim + kColumns - 1) / kColumns), 2);
            const auto join = [&](auto type) {
                using T = decltype(type);
                return enqueue(join_weights<T>, grid, kRuns * kColumns, 0, s, (const float*)workspace, of_queries, of_keys,
                               (int)head_dim, (T*)dq_weight, (T*)dk_weight, accumulate ? 1 : 0);
            };
            return size == 2 ? join(uint16_t{}) : join(float{});
        });
    });
}

}  // extern "C"
