// Device helpers shared by the training-layer kernels (tokens.hip,
// checkpoint.hip, weight_grads.hip): 8-element row vectors of bf16 or fp32 at
// any element alignment, exact widening, rounding to nearest even.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tide {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// A 16-byte access at 2- or 4-byte alignment is one dwordx4 instruction on
// gfx950 (unaligned access mode), so a row of any stride takes the same path.
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_a1 __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_a1 __attribute__((ext_vector_type(2), aligned(1)));

#define TIDE_GLOBAL __attribute__((address_space(1)))
template <class T>
__device__ __forceinline__ const TIDE_GLOBAL T* gbl(const void* p) {
    return (const TIDE_GLOBAL T*)(p);
}
template <class T>
__device__ __forceinline__ TIDE_GLOBAL T* gbl_mut(void* p) {
    return (TIDE_GLOBAL T*)(p);
}

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two fp32 rounded to nearest even into one dword of bf16 (a in the low half).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// Eight consecutive elements as they lie in memory, and as fp32.
template <class T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
    u32x4 a;
};
template <>
struct Raw8<float> {
    u32x4 a, b;
};

// n = elements left in the row, at least 1; a row's last vector goes element
// by element so that nothing past the row is touched. Elements past n read 0.
__device__ __forceinline__ Raw8<uint16_t> load8(const uint16_t* p, int n) {
    Raw8<uint16_t> r;
    if (n >= 8) {
        r.a = *gbl<u32x4_a2>(p);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t lo = 2 * i < n ? *gbl<uint16_t>(p + 2 * i) : 0;
            uint32_t hi = 2 * i + 1 < n ? *gbl<uint16_t>(p + 2 * i + 1) : 0;
            r.a[i] = lo | (hi << 16);
        }
    }
    return r;
}
__device__ __forceinline__ Raw8<float> load8(const float* p, int n) {
    Raw8<float> r;
    if (n >= 8) {
        r.a = *gbl<u32x4_a4>(p);
        r.b = *gbl<u32x4_a4>(p + 4);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r.a[i] = i < n ? *gbl<uint32_t>(p + i) : 0;
            r.b[i] = i + 4 < n ? *gbl<uint32_t>(p + i + 4) : 0;
        }
    }
    return r;
}

__device__ __forceinline__ void widen8(const Raw8<uint16_t>& r, float v[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = lo_bf16(r.a[i]);
        v[2 * i + 1] = hi_bf16(r.a[i]);
    }
}
__device__ __forceinline__ void widen8(const Raw8<float>& r, float v[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = __uint_as_float(r.a[i]);
        v[i + 4] = __uint_as_float(r.b[i]);
    }
}

__device__ __forceinline__ void store8(uint16_t* p, int n, const float v[8]) {
    u32x4 a;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    if (n >= 8) {
        *gbl_mut<u32x4_a2>(p) = a;
    } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < n) *gbl_mut<uint16_t>(p + i) = (uint16_t)(a[i / 2] >> (16 * (i & 1)));
    }
}
__device__ __forceinline__ void store8(float* p, int n, const float v[8]) {
    if (n >= 8) {
        u32x4 a, b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = __float_as_uint(v[i]);
            b[i] = __float_as_uint(v[i + 4]);
        }
        *gbl_mut<u32x4_a4>(p) = a;
        *gbl_mut<u32x4_a4>(p + 4) = b;
    } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < n) *gbl_mut<float>(p + i) = v[i];
    }
}

// Lanes of a 256-thread workgroup over rows of `units` vectors: 2^lane_log2
// lanes a row, the rest of the workgroup on further rows. The grid's y
// dimension covers a row that is wider than its lanes; both dimensions are
// capped and the kernels stride over what is left, so no dispatch dimension
// passes 2^32 work-items.
constexpr int kRowThreads = 256;
struct RowGrid {
    dim3 grid;
    int32_t lane_log2;
};
inline RowGrid row_grid(int64_t rows, int64_t units, int min_log2 = 0) {
    int lg = min_log2;
    while (lg < 8 && ((int64_t)1 << lg) < units) ++lg;
    const int64_t per = kRowThreads >> lg;
    const int64_t gx = (rows + per - 1) / per, gy = (units + (1 << lg) - 1) >> lg;
    return RowGrid{dim3((uint32_t)(gx < (1 << 23) ? gx : (1 << 23)),
                        (uint32_t)(gy < 32768 ? gy : 32768)),
                   lg};
}

}  // namespace tide
