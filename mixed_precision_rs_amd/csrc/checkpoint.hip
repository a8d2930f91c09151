// Activation checkpoints in 8 bits (tide_checkpoint_pack, tide_checkpoint_unpack)
// and the gated activation that writes them in its forward pass and reads them
// in its backward pass (tide_gated_silu, tide_gated_silu_grad), for gfx950.
//
// A checkpoint holds one e4m3 code an element and one scale byte for each 32
// consecutive elements of a row. The scale is a power of two, so neither the
// division before the rounding nor the product after it rounds: a code is off
// by half a step of e4m3 (2^-4 of its value) and nothing else, and decoding
// to bf16 is exact. Four lanes (bf16, eight with fp32) share a block and join its
// maximum with DPP steps. All four kernels are HBM streams that touch each byte once.
#include "device.hpp"
#include "host.hpp"

using namespace tide;

namespace {

typedef uint32_t u32_a1 __attribute__((aligned(1)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// The largest of the kLanes (4 or 8) lanes that share a scale.
template <int kLanes>
__device__ __forceinline__ uint32_t block_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));       // lane ^ 1
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));       // lane ^ 2
    if (kLanes == 8) v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));  // lane ^ 7
    return v;
}
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
constexpr uint32_t kInfinity = 0x7F800000u, kLargest = 0x7F600000u;   // 448 * 2^119

// The scale byte (exponent + 127) of a block: the least 2^e with amax <= 448 *
// 2^e. 448 = 1.75 * 2^8, so e is amax's exponent - 8, one more where its
// mantissa passes 1.75. Bytes stop at 10 (the smallest code, 2^-9, then
// stands for 2^-126, the smallest normal bf16) and at 246 (448 * 2^119 is the
// largest value that does not pass bf16's range after rounding).
__device__ __forceinline__ uint32_t scale_byte(uint32_t b) {
    const int e = (int)(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return (uint32_t)(e < 10 ? 10 : e > 246 ? 246 : e);
}
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// Four values within 448 (or NaN) as codes.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}
__device__ __forceinline__ void decode4(uint32_t c, uint32_t byte, float* v) {
    const float s = scale_of(byte);
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false);
    const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
    v[0] = lo[0] * s;
    v[1] = lo[1] * s;
    v[2] = hi[0] * s;
    v[3] = hi[1] * s;
}

struct Saved {
    uint8_t* codes;
    uint8_t* scales;
    int64_t codes_stride, scales_stride;
};

// A lane's V codes, n of them in the row.
template <int V>
struct Codes {
    uint32_t w[V / 4];
};
template <int V>
__device__ __forceinline__ Codes<V> load_codes(const uint8_t* p, int n) {
    Codes<V> c{};
    if (n >= V) {
        if constexpr (V == 8) {
            const u32x2 v = *gbl<u32x2_a1>(p);
            c.w[0] = v[0];
            c.w[1] = v[1];
        } else {
            c.w[0] = *gbl<u32_a1>(p);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V - 1; ++i)
            if (i < n) c.w[i / 4] |= (uint32_t)*gbl<uint8_t>(p + i) << (8 * (i & 3));
    }
    return c;
}
template <int V>
__device__ __forceinline__ void store_codes(uint8_t* p, int n, const Codes<V>& c) {
    if (n >= V) {
        if constexpr (V == 8) {
            const u32x2 v = {c.w[0], c.w[1]};
            __builtin_nontemporal_store(v, gbl_mut<u32x2_a1>(p));
        } else {
            __builtin_nontemporal_store(c.w[0], gbl_mut<u32_a1>(p));
        }
    } else {
#pragma unroll
        for (int i = 0; i < V - 1; ++i)
            if (i < n) *gbl_mut<uint8_t>(p + i) = (uint8_t)(c.w[i / 4] >> (8 * (i & 3)));
    }
}

// Largest magnitude of a lane's vector, as fp32 bits.
__device__ __forceinline__ uint32_t largest(u32x4 raw, const uint16_t*) {
    u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, raw[i] & 0x7FFF7FFFu));
    return (uint32_t)max(m[0], m[1]) << 16;
}
__device__ __forceinline__ uint32_t largest(u32x4 raw, const float*) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, raw[i] & 0x7FFFFFFFu);
    return m;
}

// A lane's vector as codes: x / 2^e to nearest even; the division is exact.
template <int V>
__device__ __forceinline__ Codes<V> encode(const float (&v)[V], uint32_t byte) {
    const float inv = scale_of(254 - byte);
    Codes<V> c;
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
        c.w[i] = encode4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
    return c;
}

// Packs this lane's vector (n elements of it in the row; lanes past the row
// have n <= 0 and zeros, and take part in the maximum all the same).
// Magnitudes are compared as integers, in which infinities and NaN are the
// largest: only a block with one of them, or with a value past the largest
// scale, takes a second look at each element.
template <class T>
__device__ __forceinline__ void pack_row(const Saved& s, int64_t r, int64_t u, int n, u32x4 raw) {
    constexpr int V = kVecOf<T>, kLanes = kScaleBlock / V;
    uint32_t m = block_max<kLanes>(largest(raw, (const T*)nullptr));
    float v[V];
    widen(raw, v);
    if (m > kLargest) {
        m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) m = max(m, magnitude(v[i]) < kInfinity ? magnitude(v[i]) : 0u);
        m = block_max<kLanes>(m);
        const float most = 448.0f * scale_of(scale_byte(m));
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] = magnitude(v[i]) < kInfinity ? fminf(fmaxf(v[i], -most), most) : __builtin_nanf("");
    }
    const uint32_t byte = scale_byte(m);
    if (n <= 0) return;
    store_codes<V>(s.codes + r * s.codes_stride + u * V, n, encode<V>(v, byte));
    if ((u & (kLanes - 1)) == 0)
        *gbl_mut<uint8_t>(s.scales + r * s.scales_stride + u / kLanes) = (uint8_t)byte;
}
template <int V>
__device__ __forceinline__ void unpack_row(const Saved& s, int64_t r, int64_t u, int n, float (&v)[V]) {
    const Codes<V> c = load_codes<V>(s.codes + r * s.codes_stride + u * V, n);
    const uint32_t byte = *gbl<uint8_t>(s.scales + r * s.scales_stride + u / (kScaleBlock / V));
#pragma unroll
    for (int i = 0; i < V / 4; ++i) decode4(c.w[i], byte, v + 4 * i);
}

// Calls f(row, vector, elements left) for this lane's share; with kWhole the
// lanes of a block always run together, some of them with nothing left.
template <int V, bool kWhole, class F>
__device__ __forceinline__ void each_vector(int64_t n, int64_t width, int lane_log2, F&& f) {
    const int lanes = 1 << lane_log2;
    int64_t units = (width + V - 1) / V;
    if (kWhole) units = (width + kScaleBlock - 1) / kScaleBlock * (kScaleBlock / V);
    for (int64_t r = (int64_t)blockIdx.x * (kRowThreads >> lane_log2) + (threadIdx.x >> lane_log2);
         r < n; r += (int64_t)gridDim.x * (kRowThreads >> lane_log2)) {
        for (int64_t u = (int64_t)blockIdx.y * lanes + (threadIdx.x & (lanes - 1)); u < units;
             u += (int64_t)gridDim.y * lanes) {
            const int64_t left = width - u * V;
            f(r, u, (int)(left > V ? V : left));
        }
    }
}

template <class T>
__global__ __launch_bounds__(kRowThreads) void pack_rows(const T* x, int64_t x_stride, int64_t n,
                                                         int64_t width, Saved to, int lane_log2) {
    constexpr int V = kVecOf<T>;
    each_vector<V, true>(n, width, lane_log2, [&](int64_t r, int64_t u, int left) {
        u32x4 v{};
        if (left > 0) v = load_row(x + r * x_stride + u * V, left);
        pack_row<T>(to, r, u, left, v);
    });
}

template <class T>
__global__ __launch_bounds__(kRowThreads) void unpack_rows(Saved from, int64_t n, int64_t width,
                                                           T* out, int64_t out_stride,
                                                           int lane_log2) {
    constexpr int V = kVecOf<T>;
    each_vector<V, false>(n, width, lane_log2, [&](int64_t r, int64_t u, int left) {
        float v[V];
        unpack_row<V>(from, r, u, left, v);
        store_row(out + r * out_stride + u * V, left, narrow(v));
    });
}

// sigmoid(g) and sigmoid(-g), neither by a difference that cancels: with e =
// exp(-|g|) they are 1 / (1 + e) and e / (1 + e). e = 2^p, p = -|g| log2(e),
// past the range of normal results taken 2^64 too large and brought back. For
// fp32 results p has a second float (one alone is off by |g| 2^-24 of e) and
// the reciprocal is refined once; a bf16 result hides both. 14 and 20
// instructions instead of 45 of the library's expf and division, which bounded
// the forward pass.
template <class T>
__device__ __forceinline__ void sigmoids(float g, float& s, float& c) {
    constexpr bool kFull = sizeof(T) == 4;
    const float a = fmaxf(-fabsf(g), -200.0f);     // exp(-200) is 0; a NaN comes back with the factor g
    const float kLog2e = 0x1.715476p+0f, kRest = 0x1.4ae0cp-26f;
    float p = a * kLog2e;
    const float rest = __builtin_fmaf(a, kRest, __builtin_fmaf(a, kLog2e, -p));
    const bool far = p < -120.0f;
    p = far ? p + 64.0f : p;
    float e = __builtin_amdgcn_exp2f(p);
    if (kFull) e = __builtin_fmaf(e, rest * 0x1.62e43p-1f, e);
    e = far ? e * 0x1p-64f : e;
    const float d = 1.0f + e;
    float big = __builtin_amdgcn_rcpf(d);
    if (kFull) big = __builtin_fmaf(__builtin_fmaf(-d, big, 1.0f), big, big);
    const float small = e * big;
    s = g >= 0.0f ? big : small;
    c = g >= 0.0f ? small : big;
}

template <class T>
__global__ __launch_bounds__(kRowThreads) void gated_rows(const T* gate, int64_t gate_stride,
                                                          const T* up, int64_t up_stride,
                                                          int64_t n, int64_t width, T* out,
                                                          int64_t out_stride, Saved gate_to,
                                                          Saved up_to, int lane_log2) {
    constexpr int V = kVecOf<T>;
    each_vector<V, true>(n, width, lane_log2, [&](int64_t r, int64_t u, int left) {
        u32x4 a{}, b{};
        if (left > 0) {
            a = load_row(gate + r * gate_stride + u * V, left);
            b = load_row(up + r * up_stride + u * V, left);
            float g[V], v[V], h[V];
            widen(a, g);
            widen(b, v);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float s, c;
                sigmoids<T>(g[i], s, c);
                h[i] = g[i] * s * v[i];
            }
            store_row(out + r * out_stride + u * V, left, narrow(h));
        }
        if (gate_to.codes) pack_row<T>(gate_to, r, u, left, a);
        if (up_to.codes) pack_row<T>(up_to, r, u, left, b);
    });
}

template <class T>
__global__ __launch_bounds__(kRowThreads) void gated_rows_grad(const T* dout, int64_t dout_stride,
                                                               Saved gate, Saved up, int64_t n,
                                                               int64_t width, T* dgate,
                                                               int64_t dgate_stride, T* dup,
                                                               int64_t dup_stride, T* out,
                                                               int64_t out_stride, int lane_log2) {
    constexpr int V = kVecOf<T>;
    each_vector<V, false>(n, width, lane_log2, [&](int64_t r, int64_t u, int left) {
        float d[V], g[V], v[V], dg[V], du[V], h[V];
        widen(load_row(dout + r * dout_stride + u * V, left), d);
        unpack_row<V>(gate, r, u, left, g);
        unpack_row<V>(up, r, u, left, v);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float s, c;
            sigmoids<T>(g[i], s, c);
            const float t = g[i] * s;
            dg[i] = d[i] * v[i] * __builtin_fmaf(t, c, s);
            du[i] = d[i] * t;
            h[i] = t * v[i];
        }
        store_row(dgate + r * dgate_stride + u * V, left, narrow(dg));
        store_row(dup + r * dup_stride + u * V, left, narrow(du));
        if (out) store_row(out + r * out_stride + u * V, left, narrow(h));
    });
}

struct Check {
    Mat rd[8], wr[8];
    int nr = 0, nw = 0;
    tide_status read(const char* name, const void* p, int64_t r, int64_t c, int64_t s, int32_t size) {
        return matrix(name, p, r, c, s, size, &rd[nr++]);
    }
    tide_status write(const char* name, const void* p, int64_t r, int64_t c, int64_t s, int32_t size) {
        return matrix(name, p, r, c, s, size, &wr[nw++]);
    }
    tide_status read(const char* name, const tide_saved* s, int64_t r, int64_t c) {
        if (!s) return fail(TIDE_ERR_INVALID_ARG, "%s is NULL", name);
        const tide_status st = read(name, s->codes, r, c, s->codes_stride, 1);
        if (st != TIDE_OK) return st;
        return read(name, s->scales, r, (c + kScaleBlock - 1) / kScaleBlock, s->scales_stride, 1);
    }
    tide_status write(const char* name, const tide_saved* s, int64_t r, int64_t c) {
        if (!s) return fail(TIDE_ERR_INVALID_ARG, "%s is NULL", name);
        const tide_status st = write(name, s->codes, r, c, s->codes_stride, 1);
        if (st != TIDE_OK) return st;
        return write(name, s->scales, r, (c + kScaleBlock - 1) / kScaleBlock, s->scales_stride, 1);
    }
    tide_status done() { return no_overlap(wr, nw, rd, nr); }
};

tide_status check_type(int32_t dtype, int64_t n, int64_t width) {
    if (dtype != TIDE_DTYPE_BF16 && dtype != TIDE_DTYPE_FP32)
        return fail(TIDE_ERR_INVALID_ARG, "dtype %d is not BF16 (0) or FP32 (1)", dtype);
    if (n < 0 || width < 0) return fail(TIDE_ERR_INVALID_ARG, "negative size");
    return TIDE_OK;
}

Saved device_of(const tide_saved* s) {
    return s ? Saved{s->codes, s->scales, s->codes_stride, s->scales_stride} : Saved{};
}

// Runs launch(grid, stream), which returns a hipError_t, over the vectors of `rows` x `width` elements.
template <class F>
tide_status over_rows(int64_t rows, int64_t width, int32_t size, void* stream, F&& launch) {
    if (rows == 0 || width == 0) return TIDE_OK;
    return on_stream(stream, [&](hipStream_t s) {
        return launch(row_grid(rows, (width * size + 15) / 16, size == 2 ? 2 : 3), s);
    });
}

}  // namespace

extern "C" {

tide_status tide_checkpoint_pack(int32_t dtype, const void* x, int64_t x_stride, int64_t rows,
                                 int64_t width, const tide_saved* saved, void* stream) {
    return guarded([&]() -> tide_status {
        TIDE_TRY(check_type(dtype, rows, width));
        const int32_t size = dtype == TIDE_DTYPE_FP32 ? 4 : 2;
        Check c;
        TIDE_TRY(c.read("x", x, rows, width, x_stride, size));
        TIDE_TRY(c.write("saved", saved, rows, width));
        TIDE_TRY(c.done());
        return over_rows(rows, width, size, stream, [&](RowGrid g, hipStream_t s) {
            if (size == 2)
                return enqueue(pack_rows<uint16_t>, g.grid, kRowThreads, 0, s,
                    (const uint16_t*)x, x_stride, rows, width, device_of(saved), g.lane_log2);
            else
                return enqueue(pack_rows<float>, g.grid, kRowThreads, 0, s,
                    (const float*)x, x_stride, rows, width, device_of(saved), g.lane_log2);
        });
    });
}

tide_status tide_checkpoint_unpack(int32_t dtype, const tide_saved* saved, int64_t rows,
                                   int64_t width, void* out, int64_t out_stride, void* stream) {
    return guarded([&]() -> tide_status {
        TIDE_TRY(check_type(dtype, rows, width));
        const int32_t size = dtype == TIDE_DTYPE_FP32 ? 4 : 2;
        Check c;
        TIDE_TRY(c.read("saved", saved, rows, width));
        TIDE_TRY(c.write("out", out, rows, width, out_stride, size));
        TIDE_TRY(c.done());
        return over_rows(rows, width, size, stream, [&](RowGrid g, hipStream_t s) {
            if (size == 2)
                return enqueue(unpack_rows<uint16_t>, g.grid, kRowThreads, 0, s,
                    device_of(saved), rows, width, (uint16_t*)out, out_stride, g.lane_log2);
            else
                return enqueue(unpack_rows<float>, g.grid, kRowThreads, 0, s,
                    device_of(saved), rows, width, (float*)out, out_stride, g.lane_log2);
        });
    });
}

tide_status tide_gated_silu(int32_t dtype, const void* gate, int64_t gate_stride, const void* up,
                            int64_t up_stride, int64_t rows, int64_t width, void* out,
                            int64_t out_stride, const tide_saved* gate_saved,
                            const tide_saved* up_saved, void* stream) {
    return guarded([&]() -> tide_status {
        TIDE_TRY(check_type(dtype, rows, width));
        const int32_t size = dtype == TIDE_DTYPE_FP32 ? 4 : 2;
        Check c;
        TIDE_TRY(c.read("gate", gate, rows, width, gate_stride, size));
        TIDE_TRY(c.read("up", up, rows, width, up_stride, size));
        TIDE_TRY(c.write("out", out, rows, width, out_stride, size));
        if (gate_saved) TIDE_TRY(c.write("gate_saved", gate_saved, rows, width));
        if (up_saved) TIDE_TRY(c.write("up_saved", up_saved, rows, width));
        TIDE_TRY(c.done());
        return over_rows(rows, width, size, stream, [&](RowGrid g, hipStream_t s) {
            if (size == 2)
                return enqueue(gated_rows<uint16_t>, g.grid, kRowThreads, 0, s,
                    (const uint16_t*)gate, gate_stride, (const uint16_t*)up, up_stride, rows, width,
                    (uint16_t*)out, out_stride, device_of(gate_saved), device_of(up_saved),
                    g.lane_log2);
            else
                return enqueue(gated_rows<float>, g.grid, kRowThreads, 0, s,
                    (const float*)gate, gate_stride, (const float*)up, up_stride, rows, width,
                    (float*)out, out_stride, device_of(gate_saved), device_of(up_saved), g.lane_log2);
        });
    });
}

tide_status tide_gated_silu_grad(int32_t dtype, const void* dout, int64_t dout_stride,
                                 const tide_saved* gate_saved, const tide_saved* up_saved,
                                 int64_t rows, int64_t width, void* dgate, int64_t dgate_stride,
                                 void* dup, int64_t dup_stride, void* out, int64_t out_stride,
                                 void* stream) {
    return guarded([&]() -> tide_status {
        TIDE_TRY(check_type(dtype, rows, width));
        const int32_t size = dtype == TIDE_DTYPE_FP32 ? 4 : 2;
        Check c;
        TIDE_TRY(c.read("dout", dout, rows, width, dout_stride, size));
        TIDE_TRY(c.read("gate_saved", gate_saved, rows, width));
        TIDE_TRY(c.read("up_saved", up_saved, rows, width));
        TIDE_TRY(c.write("dgate", dgate, rows, width, dgate_stride, size));
        TIDE_TRY(c.write("dup", dup, rows, width, dup_stride, size));
        TIDE_TRY(c.write("out", out, out ? rows : 0, width, out_stride, size));
        TIDE_TRY(c.done());
        return over_rows(rows, width, size, stream, [&](RowGrid g, hipStream_t s) {
            if (size == 2)
                return enqueue(gated_rows_grad<uint16_t>, g.grid, kRowThreads, 0, s,
                    (const uint16_t*)dout, dout_stride, device_of(gate_saved), device_of(up_saved),
                    rows, width, (uint16_t*)dgate, dgate_stride, (uint16_t*)dup, dup_stride,
                    (uint16_t*)out, out_stride, g.lane_log2);
            else
                return enqueue(gated_rows_grad<float>, g.grid, kRowThreads, 0, s,
                    (const float*)dout, dout_stride, device_of(gate_saved), device_of(up_saved),
                    rows,
                    width, (float*)dgate, dgate_stride, (float*)dup, dup_stride, (float*)out,
                    out_stride, g.lane_log2);
        });
    });
}

}  // extern "C"
