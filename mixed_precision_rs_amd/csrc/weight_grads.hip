// Weight gradients from saved activations (tide_weight_grads_bf16) for gfx950:
// for each expert e, dW_e = dy_e^T x_e over the rows of e, written in bf16
// straight into the parameter's gradient tensor.
#include <algorithm>
#include <climits>
#include <new>
#include <vector>

#include "device.hpp"
#include "host.hpp"

using namespace tide;

namespace {

constexpr int kBlock = 32;             // elements that share a scale
constexpr int kMaxGrads = 256;         // gradient pointers in one launch's arguments
constexpr int64_t kMaxGroups = 1 << 23;   // workgroups of a launch (2^32 work-items a dimension)
struct GradPtrs {
    uint16_t* p[kMaxGrads];
};

struct Args {
    const uint16_t* dy;
    const uint16_t* x;                 // bf16 rows, or NULL: the checkpoint
    const uint8_t* codes;
    const uint8_t* scales;
    const int32_t* offsets;            // E + 1, or NULL: one expert with all n rows
    const int32_t* tokens;             // row of x of each row of dy, or NULL: its own
    int64_t dy_stride, x_stride, codes_stride, scales_stride;
    int64_t n, x_rows, O, I;
    int32_t accumulate, tiles_o, tiles_i, first;
};

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
constexpr int kTile = 64, kDepth = 16, kPitch = kTile + 2;

__global__ __launch_bounds__(256) void weight_grads(Args a, GradPtrs g) {
    __shared__ uint16_t A[kDepth * kPitch], B[kDepth * kPitch];
    const int tiles = a.tiles_o * a.tiles_i;
    const int e = blockIdx.x / tiles, tile = blockIdx.x - e * tiles;
    const int64_t o0 = (int64_t)(tile / a.tiles_i) * kTile, i0 = (int64_t)(tile % a.tiles_i) * kTile;
    int64_t lo = 0, hi = a.n;
    if (a.offsets) {
        lo = a.offsets[a.first + e];
        hi = a.offsets[a.first + e + 1];
        lo = lo < 0 ? 0 : lo > a.n ? a.n : lo;
        hi = hi < lo ? lo : hi > a.n ? a.n : hi;
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int m0 = (wave >> 1) * 32, n0 = (wave & 1) * 32;
    f32x16 acc = {};
    for (int64_t t0 = lo; t0 < hi; t0 += kDepth) {
        for (int i = threadIdx.x; i < kDepth * kTile; i += 256) {
            const int t = i / kTile, c = i % kTile;
            const int64_t row = t0 + t;
            uint16_t va = 0, vb = 0;
            if (row < hi) {
                if (o0 + c < a.O) va = a.dy[row * a.dy_stride + o0 + c];
                const int64_t xr = a.tokens ? a.tokens[row] : row;
                if (i0 + c < a.I && xr >= 0 && xr < a.x_rows) {
                    if (a.x) {
                        vb = a.x[xr * a.x_stride + i0 + c];
                    } else {
                        const float v = __builtin_amdgcn_cvt_f32_fp8(
                            a.codes[xr * a.codes_stride + i0 + c], 0);
                        const float s = __uint_as_float(
                            (uint32_t)a.scales[xr * a.scales_stride + (i0 + c) / kBlock] << 23);
                        vb = (uint16_t)pack_bf16(v * s, 0.0f);
                    }
                }
            }
            A[t * kPitch + c] = va;
            B[t * kPitch + c] = vb;
        }
        __syncthreads();
        bf16x8 fa, fb;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int t = (lane >> 5) * 8 + j;
            fa[j] = __builtin_bit_cast(__bf16, A[t * kPitch + m0 + (lane & 31)]);
            fb[j] = __builtin_bit_cast(__bf16, B[t * kPitch + n0 + (lane & 31)]);
        }
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa, fb, acc, 0, 0, 0);
        __syncthreads();
    }
    uint16_t* out = g.p[e];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int64_t o = o0 + m0 + (r & 3) + 8 * (r >> 2) + 4 * (lane >> 5);
        const int64_t i = i0 + n0 + (lane & 31);
        if (o < a.O && i < a.I) {
            float v = acc[r];
            if (a.accumulate) v += lo_bf16(out[o * a.I + i]);
            out[o * a.I + i] = (uint16_t)pack_bf16(v, 0.0f);
        }
    }
}

#define TIDE_TRY(expr)                        \
    do {                                      \
        tide_status s_ = (expr);              \
        if (s_ != TIDE_OK) return s_;         \
    } while (0)

tide_status check_sizes(int64_t n, int64_t O, int64_t I, int32_t experts) {
    if (n < 0 || O < 0 || I < 0 || experts < 1)
        return fail(TIDE_ERR_INVALID_ARG, "need rows, out and in >= 0 and experts >= 1");
    if (n > INT32_MAX || O > INT32_MAX || I > INT32_MAX)
        return fail(TIDE_ERR_UNSUPPORTED, "rows, out and in must be below 2^31");
    int64_t elems;
    if (__builtin_mul_overflow(O, I, &elems) || elems > INT64_MAX / 8 / experts)
        return fail(TIDE_ERR_OVERFLOW, "the gradients' size overflows int64");
    return TIDE_OK;
}

}  // namespace

extern "C" {

tide_status tide_weight_grads_workspace(int64_t rows, int64_t out, int64_t in, int32_t experts,
                                        int64_t* bytes) {
    if (!bytes) return fail(TIDE_ERR_INVALID_ARG, "bytes is NULL");
    TIDE_TRY(check_sizes(rows, out, in, experts));
    *bytes = 0;
    return TIDE_OK;
}

tide_status tide_weight_grads_bf16(const uint16_t* dy, int64_t dy_stride, int64_t rows,
                                   int64_t out, const uint16_t* x, int64_t x_stride,
                                   const tide_saved* saved, int64_t x_rows, int64_t in,
                                   const int32_t* offsets, const int32_t* token_of_row,
                                   int32_t experts, uint16_t* const* grads, int32_t accumulate,
                                   void* workspace, int64_t workspace_bytes, void* stream_v) {
    try {
        int64_t need = 0;
        TIDE_TRY(tide_weight_grads_workspace(rows, out, in, experts, &need));
        if (need > 0 && (!workspace || workspace_bytes < need))
            return fail(TIDE_ERR_INVALID_ARG, "workspace holds %lld bytes, %lld needed",
                        (long long)(workspace ? workspace_bytes : 0), (long long)need);
        if (x_rows < 0) return fail(TIDE_ERR_INVALID_ARG, "negative x_rows");
        if (x_rows > INT32_MAX) return fail(TIDE_ERR_UNSUPPORTED, "x_rows must be below 2^31");
        if (experts > 1 && !offsets)
            return fail(TIDE_ERR_INVALID_ARG, "%d experts need offsets", experts);
        if (!token_of_row && x_rows < rows)
            return fail(TIDE_ERR_INVALID_ARG, "x has %lld rows, dy %lld", (long long)x_rows,
                        (long long)rows);
        if ((x != nullptr) == (saved != nullptr) && rows > 0 && in > 0)
            return fail(TIDE_ERR_INVALID_ARG, "need either x or saved");
        Mat rd[5], wr;
        TIDE_TRY(matrix("dy", dy, rows, out, dy_stride, 2, &rd[0]));
        if (saved) {
            TIDE_TRY(matrix("saved", saved->codes, x_rows, in, saved->codes_stride, 1, &rd[1]));
            TIDE_TRY(matrix("saved", saved->scales, x_rows, (in + kBlock - 1) / kBlock,
                            saved->scales_stride, 1, &rd[2]));
        } else {
            TIDE_TRY(matrix("x", x, x_rows, in, x_stride, 2, &rd[1]));
            rd[2] = Mat{};
        }
        TIDE_TRY(matrix("offsets", offsets, offsets ? 1 : 0, (int64_t)experts + 1,
                        (int64_t)experts + 1, 4, &rd[3]));
        TIDE_TRY(matrix("token_of_row", token_of_row, token_of_row ? 1 : 0, rows, rows, 4, &rd[4]));
        if (out == 0 || in == 0) return TIDE_OK;
        if (!grads) return fail(TIDE_ERR_INVALID_ARG, "grads is NULL");
        std::vector<uintptr_t> at(experts);
        for (int32_t e = 0; e < experts; ++e) {
            char name[32];
            snprintf(name, sizeof name, "grads[%d]", e);
            TIDE_TRY(matrix(name, grads[e], 1, out * in, out * in, 2, &wr));
            TIDE_TRY(no_overlap(&wr, 1, rd, 5));
            at[e] = wr.base;
        }
        if (!std::is_sorted(at.begin(), at.end())) std::sort(at.begin(), at.end());
        for (int32_t e = 1; e < experts; ++e)
            if (at[e] - at[e - 1] < (uintptr_t)(out * in) * 2)
                return fail(TIDE_ERR_INVALID_ARG, "two of the grads overlap");
        hipStream_t stream = reinterpret_cast<hipStream_t>(stream_v);
        int dev = 0;
        TIDE_TRY(stream_device(stream, &dev));
        DeviceGuard guard(dev);
        if (guard.status() != hipSuccess) return hip_fail(guard.status(), "hipSetDevice");
        Args a{};
        a.dy = dy;
        a.x = x;
        if (saved) {
            a.codes = saved->codes;
            a.scales = saved->scales;
            a.codes_stride = saved->codes_stride;
            a.scales_stride = saved->scales_stride;
        }
        a.offsets = offsets;
        a.tokens = token_of_row;
        a.dy_stride = dy_stride;
        a.x_stride = x_stride;
        a.n = rows;
        a.x_rows = x_rows;
        a.O = out;
        a.I = in;
        a.accumulate = accumulate ? 1 : 0;
        const int64_t to = (out + kTile - 1) / kTile, ti = (in + kTile - 1) / kTile;
        if (to > kMaxGroups / ti)
            return fail(TIDE_ERR_UNSUPPORTED, "gradients of %lld x %lld", (long long)out, (long long)in);
        a.tiles_o = (int32_t)to;
        a.tiles_i = (int32_t)ti;
        const int32_t most = (int32_t)std::min<int64_t>(kMaxGrads, kMaxGroups / (to * ti));
        for (int32_t e0 = 0; e0 < experts; e0 += most) {
            const int32_t ne = std::min(experts - e0, most);
            GradPtrs g{};
            for (int32_t e = 0; e < ne; ++e) g.p[e] = grads[e0 + e];
            a.first = e0;
            weight_grads<<<dim3((uint32_t)(ne * to * ti)), dim3(256), 0, stream>>>(a, g);
            TIDE_HIP_TRY(hipGetLastError());
        }
        return TIDE_OK;
    } catch (const std::bad_alloc&) {
        return fail(TIDE_ERR_NO_MEMORY, "host allocation failed");
    } catch (...) {
        return fail(TIDE_ERR_INVALID_ARG, "unexpected exception");
    }
}

}  // extern "C"
