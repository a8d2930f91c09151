// Device helpers shared by the training layer's kernels (tokens.hip, checkpoint.hip,
// weight_grads.hip) and those at a step's ends (embedding.hip, logprobs.hip, heads.hip,
// grad_norm.hip): 16-byte row vectors of bf16 or fp32 at any element alignment, exact
// widening, rounding to nearest even.
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

// A lane's vector: 16 bytes of a row, 8 bf16 or 4 fp32, so that every load and
// store of a wave covers 1 KiB without gaps (8 fp32 a lane in two stores of
// half-covered lines wrote 40% slower once the stores were non-temporal).
template <class T>
constexpr int kVecOf = 16 / sizeof(T);

// 16 bytes of elements of type T, at their alignment; the stores are
// non-temporal, since no kernel here reads what it wrote (dispatch 123 -> 110
// us, unpacking to bf16 40 -> 30 at 16384 tokens and 8192 x 8192).
__device__ __forceinline__ u32x4 load16(const uint16_t* p) { return *gbl<u32x4_a2>(p); }
__device__ __forceinline__ u32x4 load16(const float* p) { return *gbl<u32x4_a4>(p); }
__device__ __forceinline__ u32x4 load16_once(const uint16_t* p) {
    return __builtin_nontemporal_load(gbl<u32x4_a2>(p));
}
__device__ __forceinline__ u32x4 load16_once(const float* p) {
    return __builtin_nontemporal_load(gbl<u32x4_a4>(p));
}
__device__ __forceinline__ void store16(uint16_t* p, u32x4 v) {
    __builtin_nontemporal_store(v, gbl_mut<u32x4_a2>(p));
}
__device__ __forceinline__ void store16(float* p, u32x4 v) {
    __builtin_nontemporal_store(v, gbl_mut<u32x4_a4>(p));
}

// A vector of a row with n >= 1 elements left: a row's last vector goes element
// by element, so that nothing past the row is touched; elements past n read 0.
template <bool kOnce = false>
__device__ __forceinline__ u32x4 load_row(const uint16_t* p, int n) {
    if (n >= 8) return kOnce ? load16_once(p) : load16(p);
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = 2 * i < n ? *gbl<uint16_t>(p + 2 * i) : 0;
        const uint32_t hi = 2 * i + 1 < n ? *gbl<uint16_t>(p + 2 * i + 1) : 0;
        r[i] = lo | (hi << 16);
    }
    return r;
}
template <bool kOnce = false>
__device__ __forceinline__ u32x4 load_row(const float* p, int n) {
    if (n >= 4) return kOnce ? load16_once(p) : load16(p);
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = i < n ? *gbl<uint32_t>(p + i) : 0;
    return r;
}
__device__ __forceinline__ void store_row(uint16_t* p, int n, u32x4 v) {
    if (n >= 8) {
        store16(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < n) *gbl_mut<uint16_t>(p + i) = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
    }
}
__device__ __forceinline__ void store_row(float* p, int n, u32x4 v) {
    if (n >= 4) {
        store16(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < n) *gbl_mut<uint32_t>(p + i) = v[i];
    }
}

__device__ __forceinline__ void widen(u32x4 r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = lo_bf16(r[i]);
        v[2 * i + 1] = hi_bf16(r[i]);
    }
}
__device__ __forceinline__ void widen(u32x4 r, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ u32x4 narrow(const float (&v)[8]) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    return r;
}
__device__ __forceinline__ u32x4 narrow(const float (&v)[4]) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __float_as_uint(v[i]);
    return r;
}

constexpr int kScaleBlock = 32;        // consecutive elements of a row that share a checkpoint scale

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
