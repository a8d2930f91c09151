// Activation checkpoints in 8 bits (tide_checkpoint_pack, tide_checkpoint_unpack)
// and the gated activation that writes them in its forward pass and reads them
// in its backward pass (tide_gated_silu, tide_gated_silu_grad), for gfx950.
//
// A checkpoint holds one e4m3 code an element and one scale byte for each 32
// consecutive elements of a row. The scale is a power of two, so neither the
// division before the rounding nor the product after it rounds: a code is off
// by half a step of e4m3 (2^-4 of its value) and nothing else, and decoding
// to bf16 is exact. Four lanes share a block and join its maximum with two
// DPP steps. All four kernels are HBM streams that touch each byte once.
#include "device.hpp"
#include "host.hpp"

using namespace tide;

namespace {

constexpr int kBlock = 32;
constexpr int kQuad = kBlock / 8;    // lanes that share a scale

__device__ __forceinline__ float quad_max(float v) {
    const int x1 = __builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xF, 0xF, true);  // lane ^ 1
    v = fmaxf(v, __int_as_float(x1));
    const int x2 = __builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xF, 0xF, true);  // lane ^ 2
    return fmaxf(v, __int_as_float(x2));
}

__device__ __forceinline__ bool finite(float v) { return fabsf(v) < __builtin_inff(); }

// The scale byte (exponent + 127) of a block: the least 2^e with amax <= 448 *
// 2^e. 448 = 1.75 * 2^8, so e is amax's exponent - 8, one more where its
// mantissa passes 1.75. Bytes stop at 10 (the smallest code, 2^-9, then
// stands for 2^-126, the smallest normal bf16) and at 246 (448 * 2^119 is the
// largest value that does not pass bf16's range after rounding).
__device__ __forceinline__ uint32_t scale_byte(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = (int)(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return (uint32_t)(e < 10 ? 10 : e > 246 ? 246 : e);
}
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// Eight values of a block with scale byte `byte` as codes; what is not finite
// becomes the NaN code.
__device__ __forceinline__ u32x2 encode8(const float v[8], uint32_t byte) {
    const float inv = scale_of(254 - byte);
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        q[i] = finite(v[i]) ? fminf(fmaxf(v[i] * inv, -448.0f), 448.0f) : __builtin_nanf("");
    u32x2 c;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], 0, false);
        c[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], w, true);
    }
    return c;
}

__device__ __forceinline__ void decode8(u32x2 c, uint32_t byte, float v[8]) {
    const float s = scale_of(byte);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], false);
        const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], true);
        v[4 * i] = lo[0] * s;
        v[4 * i + 1] = lo[1] * s;
        v[4 * i + 2] = hi[0] * s;
        v[4 * i + 3] = hi[1] * s;
    }
}

__device__ __forceinline__ u32x2 load_codes(const uint8_t* p, int n) {
    if (n >= 8) return *gbl<u32x2_a1>(p);
    u32x2 c = {0, 0};
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < n) c[i / 4] |= (uint32_t)*gbl<uint8_t>(p + i) << (8 * (i & 3));
    return c;
}
__device__ __forceinline__ void store_codes(uint8_t* p, int n, u32x2 c) {
    if (n >= 8) {
        *gbl_mut<u32x2_a1>(p) = c;
    } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < n) *gbl_mut<uint8_t>(p + i) = (uint8_t)(c[i / 4] >> (8 * (i & 3)));
    }
}

struct Saved {
    uint8_t* codes;
    uint8_t* scales;
    int64_t codes_stride, scales_stride;
};

// Packs this lane's eight values (n of them in the row; lanes past the row
// have n <= 0 and zeros, and take part in the maximum all the same).
__device__ __forceinline__ void pack8(const Saved& s, int64_t r, int64_t u, int n,
                                      const float v[8]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, finite(v[i]) ? fabsf(v[i]) : 0.0f);
    const uint32_t byte = scale_byte(quad_max(m));
    if (n <= 0) return;
    store_codes(s.codes + r * s.codes_stride + u * 8, n, encode8(v, byte));
    if ((u & (kQuad - 1)) == 0)
        *gbl_mut<uint8_t>(s.scales + r * s.scales_stride + u / kQuad) = (uint8_t)byte;
}
__device__ __forceinline__ void unpack8(const Saved& s, int64_t r, int64_t u, int n, float v[8]) {
    const u32x2 c = load_codes(s.codes + r * s.codes_stride + u * 8, n);
    decode8(c, *gbl<uint8_t>(s.scales + r * s.scales_stride + u / kQuad), v);
}

// Calls f(row, vector, elements left) for this lane's share; with kWhole the
// four lanes of a block always run together, some of them with nothing left.
template <bool kWhole, class F>
__device__ __forceinline__ void each_vector(int64_t n, int64_t width, int lane_log2, F&& f) {
    const int lanes = 1 << lane_log2;
    int64_t units = (width + 7) / 8;
    if (kWhole) units = (units + kQuad - 1) / kQuad * kQuad;
    for (int64_t r = (int64_t)blockIdx.x * (kRowThreads >> lane_log2) + (threadIdx.x >> lane_log2);
         r < n; r += (int64_t)gridDim.x * (kRowThreads >> lane_log2)) {
        for (int64_t u = (int64_t)blockIdx.y * lanes + (threadIdx.x & (lanes - 1)); u < units;
             u += (int64_t)gridDim.y * lanes) {
            const int64_t left = width - u * 8;
            f(r, u, (int)(left > 8 ? 8 : left));
        }
    }
}

template <class T>
__global__ __launch_bounds__(kRowThreads) void pack_rows(const T* x, int64_t x_stride, int64_t n,
                                                         int64_t width, Saved to, int lane_log2) {
    each_vector<true>(n, width, lane_log2, [&](int64_t r, int64_t u, int left) {
        float v[8] = {};
        if (left > 0) widen8(load8(x + r * x_stride + u * 8, left), v);
        pack8(to, r, u, left, v);
    });
}

template <class T>
__global__ __launch_bounds__(kRowThreads) void unpack_rows(Saved from, int64_t n, int64_t width,
                                                           T* out, int64_t out_stride,
                                                           int lane_log2) {
    each_vector<false>(n, width, lane_log2, [&](int64_t r, int64_t u, int left) {
        float v[8];
        unpack8(from, r, u, left, v);
        store8(out + r * out_stride + u * 8, left, v);
    });
}

// sigmoid(g) and sigmoid(-g), neither by a difference that cancels.
__device__ __forceinline__ void sigmoids(float g, float& s, float& c) {
    const float e = expf(-fabsf(g));
    const float big = 1.0f / (1.0f + e), small = e * big;
    s = g >= 0.0f ? big : g < 0.0f ? small : g;      // NaN stays
    c = g >= 0.0f ? small : g < 0.0f ? big : g;
}

template <class T>
__global__ __launch_bounds__(kRowThreads) void gated_rows(const T* gate, int64_t gate_stride,
                                                          const T* up, int64_t up_stride,
                                                          int64_t n, int64_t width, T* out,
                                                          int64_t out_stride, Saved gate_to,
                                                          Saved up_to, int lane_log2) {
    each_vector<true>(n, width, lane_log2, [&](int64_t r, int64_t u, int left) {
        float g[8] = {}, v[8] = {}, h[8];
        if (left > 0) {
            const Raw8<T> a = load8(gate + r * gate_stride + u * 8, left);
            const Raw8<T> b = load8(up + r * up_stride + u * 8, left);
            widen8(a, g);
            widen8(b, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float s, c;
                sigmoids(g[i], s, c);
                h[i] = g[i] * s * v[i];
            }
            store8(out + r * out_stride + u * 8, left, h);
        }
        if (gate_to.codes) pack8(gate_to, r, u, left, g);
        if (up_to.codes) pack8(up_to, r, u, left, v);
    });
}

template <class T>
__global__ __launch_bounds__(kRowThreads) void gated_rows_grad(const T* dout, int64_t dout_stride,
                                                               Saved gate, Saved up, int64_t n,
                                                               int64_t width, T* dgate,
                                                               int64_t dgate_stride, T* dup,
                                                               int64_t dup_stride, T* out,
                                                               int64_t out_stride, int lane_log2) {
    each_vector<false>(n, width, lane_log2, [&](int64_t r, int64_t u, int left) {
        float d[8], g[8], v[8], dg[8], du[8], h[8];
        widen8(load8(dout + r * dout_stride + u * 8, left), d);
        unpack8(gate, r, u, left, g);
        unpack8(up, r, u, left, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float s, c;
            sigmoids(g[i], s, c);
            const float t = g[i] * s;
            dg[i] = d[i] * v[i] * __builtin_fmaf(t, c, s);
            du[i] = d[i] * t;
            h[i] = t * v[i];
        }
        store8(dgate + r * dgate_stride + u * 8, left, dg);
        store8(dup + r * dup_stride + u * 8, left, du);
        if (out) store8(out + r * out_stride + u * 8, left, h);
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
        return read(name, s->scales, r, (c + kBlock - 1) / kBlock, s->scales_stride, 1);
    }
    tide_status write(const char* name, const tide_saved* s, int64_t r, int64_t c) {
        if (!s) return fail(TIDE_ERR_INVALID_ARG, "%s is NULL", name);
        const tide_status st = write(name, s->codes, r, c, s->codes_stride, 1);
        if (st != TIDE_OK) return st;
        return write(name, s->scales, r, (c + kBlock - 1) / kBlock, s->scales_stride, 1);
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

#define TIDE_TRY(expr)                        \
    do {                                      \
        tide_status s_ = (expr);              \
        if (s_ != TIDE_OK) return s_;         \
    } while (0)

// Runs `launch` (grid, stream) with the stream's device current.
template <class F>
tide_status over_rows(int64_t n, int64_t width, void* stream_v, F&& launch) {
    if (n == 0 || width == 0) return TIDE_OK;
    hipStream_t stream = reinterpret_cast<hipStream_t>(stream_v);
    int dev = 0;
    TIDE_TRY(stream_device(stream, &dev));
    DeviceGuard guard(dev);
    if (guard.status() != hipSuccess) return hip_fail(guard.status(), "hipSetDevice");
    launch(row_grid(n, (width + 7) / 8, 2), stream);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? TIDE_OK : hip_fail(e, "kernel launch");
}

}  // namespace

extern "C" {

tide_status tide_checkpoint_pack(int32_t dtype, const void* x, int64_t x_stride, int64_t rows,
                                 int64_t width, const tide_saved* saved, void* stream) {
    TIDE_TRY(check_type(dtype, rows, width));
    const int32_t size = dtype == TIDE_DTYPE_FP32 ? 4 : 2;
    Check c;
    TIDE_TRY(c.read("x", x, rows, width, x_stride, size));
    TIDE_TRY(c.write("saved", saved, rows, width));
    TIDE_TRY(c.done());
    return over_rows(rows, width, stream, [&](RowGrid g, hipStream_t s) {
        if (size == 2)
            pack_rows<uint16_t><<<g.grid, dim3(kRowThreads), 0, s>>>(
                (const uint16_t*)x, x_stride, rows, width, device_of(saved), g.lane_log2);
        else
            pack_rows<float><<<g.grid, dim3(kRowThreads), 0, s>>>(
                (const float*)x, x_stride, rows, width, device_of(saved), g.lane_log2);
    });
}

tide_status tide_checkpoint_unpack(int32_t dtype, const tide_saved* saved, int64_t rows,
                                   int64_t width, void* out, int64_t out_stride, void* stream) {
    TIDE_TRY(check_type(dtype, rows, width));
    const int32_t size = dtype == TIDE_DTYPE_FP32 ? 4 : 2;
    Check c;
    TIDE_TRY(c.read("saved", saved, rows, width));
    TIDE_TRY(c.write("out", out, rows, width, out_stride, size));
    TIDE_TRY(c.done());
    return over_rows(rows, width, stream, [&](RowGrid g, hipStream_t s) {
        if (size == 2)
            unpack_rows<uint16_t><<<g.grid, dim3(kRowThreads), 0, s>>>(
                device_of(saved), rows, width, (uint16_t*)out, out_stride, g.lane_log2);
        else
            unpack_rows<float><<<g.grid, dim3(kRowThreads), 0, s>>>(
                device_of(saved), rows, width, (float*)out, out_stride, g.lane_log2);
    });
}

tide_status tide_gated_silu(int32_t dtype, const void* gate, int64_t gate_stride, const void* up,
                            int64_t up_stride, int64_t rows, int64_t width, void* out,
                            int64_t out_stride, const tide_saved* gate_saved,
                            const tide_saved* up_saved, void* stream) {
    TIDE_TRY(check_type(dtype, rows, width));
    const int32_t size = dtype == TIDE_DTYPE_FP32 ? 4 : 2;
    Check c;
    TIDE_TRY(c.read("gate", gate, rows, width, gate_stride, size));
    TIDE_TRY(c.read("up", up, rows, width, up_stride, size));
    TIDE_TRY(c.write("out", out, rows, width, out_stride, size));
    if (gate_saved) TIDE_TRY(c.write("gate_saved", gate_saved, rows, width));
    if (up_saved) TIDE_TRY(c.write("up_saved", up_saved, rows, width));
    TIDE_TRY(c.done());
    return over_rows(rows, width, stream, [&](RowGrid g, hipStream_t s) {
        if (size == 2)
            gated_rows<uint16_t><<<g.grid, dim3(kRowThreads), 0, s>>>(
                (const uint16_t*)gate, gate_stride, (const uint16_t*)up, up_stride, rows, width,
                (uint16_t*)out, out_stride, device_of(gate_saved), device_of(up_saved),
                g.lane_log2);
        else
            gated_rows<float><<<g.grid, dim3(kRowThreads), 0, s>>>(
                (const float*)gate, gate_stride, (const float*)up, up_stride, rows, width,
                (float*)out, out_stride, device_of(gate_saved), device_of(up_saved), g.lane_log2);
    });
}

tide_status tide_gated_silu_grad(int32_t dtype, const void* dout, int64_t dout_stride,
                                 const tide_saved* gate_saved, const tide_saved* up_saved,
                                 int64_t rows, int64_t width, void* dgate, int64_t dgate_stride,
                                 void* dup, int64_t dup_stride, void* out, int64_t out_stride,
                                 void* stream) {
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
    return over_rows(rows, width, stream, [&](RowGrid g, hipStream_t s) {
        if (size == 2)
            gated_rows_grad<uint16_t><<<g.grid, dim3(kRowThreads), 0, s>>>(
                (const uint16_t*)dout, dout_stride, device_of(gate_saved), device_of(up_saved),
                rows, width, (uint16_t*)dgate, dgate_stride, (uint16_t*)dup, dup_stride,
                (uint16_t*)out, out_stride, g.lane_log2);
        else
            gated_rows_grad<float><<<g.grid, dim3(kRowThreads), 0, s>>>(
                (const float*)dout, dout_stride, device_of(gate_saved), device_of(up_saved), rows,
                width, (float*)dgate, dgate_stride, (float*)dup, dup_stride, (float*)out,
                out_stride, g.lane_log2);
    });
}

}  // extern "C"
