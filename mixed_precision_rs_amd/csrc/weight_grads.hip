// Weight gradients from saved activations (tide_weight_grads_bf16) for gfx950:
// for each expert e, dW_e = dy_e^T x_e over the rows of e, written in bf16
// straight into the parameter's gradient tensor.
#include <algorithm>
#include <climits>
#include <cstdio>
#include <vector>

#include "device.hpp"
#include "host.hpp"

using namespace tide;

namespace {

typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
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
    float* partial;                    // with splits > 1: the sums of each split of each tile
    int32_t accumulate, tiles_o, tiles_i, first, count, splits;
    int32_t past_caches;               // how gradients are stored
};

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
#define TIDE_LDS __attribute__((address_space(3)))

constexpr int kMostDepth = 64;         // rows (tokens) of one stage, at most
// How rows are read. Buffers: rows of any alignment and of one 16-byte load or
// more, by buffer loads. Wide: as Buffers, but through 64-bit addresses, for
// token indices into more than 2 GiB and for strides of 32 MiB. Elements: rows
// shorter than a load.
enum Access { kBuffers, kWide, kElements };
constexpr uint32_t kBufferWord = 0x00020000;      // raw buffer, bounds checked in bytes
constexpr uint32_t kOutside = 0x80000000u;        // past every buffer: loads read 0
constexpr int64_t kMostBytes = 0x7F000000;        // of a buffer

// Position of 16-byte chunk c (8 elements) of row t in a staged row of kWidth
// elements: rows t, t + 1, t + 2, t + 3 place one column 64 bytes apart (modulo
// the 256 bytes of all banks), so the four rows that a transposing read takes
// at once come from different banks.
template <int kWidth>
__device__ __forceinline__ int chunk_at(int t, int c) {
    static_assert(kWidth == 64 || kWidth % 128 == 0, "bank pattern of a row");
    return kWidth == 64 ? c ^ ((t & 2) << 1) : c ^ ((t & 3) << 2);
}

__device__ __forceinline__ u32x4 buffer16(__amdgpu_buffer_rsrc_t r, uint32_t at) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)at, 0, 0));
}

// A buffer that ends with the last of `rows` rows.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, uint32_t rows, uint32_t stride,
                                                         uint32_t length) {
    const int bytes = (int)(rows * stride) - (int)(stride - length);
    return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, max(bytes, 0), (int)kBufferWord);
}

// The scale block of column c of a row; of the row's last column for loads past
// its end, whose values are not stored: no byte behind a row's scales is read.
__host__ __device__ constexpr int64_t scale_block(int64_t c, int64_t width) {
    return (c < width ? c : width - 1) / kScaleBlock;
}
static_assert(scale_block(0, 1) == 0 && scale_block(31, 33) == 0 && scale_block(32, 33) == 1 &&
                  scale_block(48, 33) == 1 && scale_block(240, 33) == 1 && scale_block(240, 241) == 7,
              "within the row's scales");

// Sixteen e4m3 codes with one scale as two chunks of bf16 (exact).
__device__ __forceinline__ void decode16(u32x4 c, float scale, u32x4& lo, u32x4& hi) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = __builtin_bit_cast(
            uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)c[i], scale, false));
        const uint32_t b = __builtin_bit_cast(
            uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)c[i], scale, true));
        u32x4& d = i < 2 ? lo : hi;
        d[2 * (i & 1)] = a;
        d[2 * (i & 1) + 1] = b;
    }
}

__device__ __forceinline__ u32x4 codes16(const uint8_t* p, int n) {
    if (n >= 16) return *gbl<u32x4_a1>(p);
    u32x4 c = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 15; ++i)
        if (i < n) c[i / 4] |= (uint32_t)*gbl<uint8_t>(p + i) << (8 * (i & 3));
    return c;
}

// Four columns of a gradient from column i of row o on, as far as they are in it.
__device__ __forceinline__ void store4(const Args& a, uint16_t* out, int64_t o, int64_t i, float v[4]) {
    if (o >= a.O || i >= a.I) return;
    out += o * a.I + i;
    if (a.accumulate) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (i + q < a.I) v[q] += lo_bf16(*gbl<uint16_t>(out + q));
    }
    const u32x2 p = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    if (i + 4 <= a.I) {
        *gbl_mut<u32x2_a2>(out) = p;
    } else {
#pragma unroll
        for (int q = 0; q < 3; ++q)
            if (i + q < a.I) *gbl_mut<uint16_t>(out + q) = (uint16_t)(p[q / 2] >> (16 * (q & 1)));
    }
}

// Eight columns of a gradient. The empty statements keep the two stores from
// being merged into one without the hint (128 experts of 768 x 2048: 216 us instead of 166).
template <bool kPastCaches>
__device__ __forceinline__ void store_chunk(uint16_t* out, u32x4 v) {
    if constexpr (kPastCaches) {
        __builtin_nontemporal_store(v, gbl_mut<u32x4_a2>(out));
    } else {
        asm volatile("");
        *gbl_mut<u32x4_a2>(out) = v;
        asm volatile("");
    }
}

// A TO x TI tile of one expert's gradient. Rows of dy and x are staged in
// LDS as bf16, 64 or 32 at a time, and read back transposed
// (ds_read_b64_tr_b16), since the matrix instruction wants the summed index
// (the row) inside a lane; products are 32x32x16 bf16 with fp32 sums. The 256
// tile has 8 waves of 128 x 64 (128 sums a lane, two waves a SIMD): 1300
// TFLOP/s on 8192 x 8192 x 8192, where 4 waves of 128 x 128, which leave every
// wait exposed, had 1060. The 128 tile has 4 of 64 x 64. The 256 x 128 tile has 4
// waves of 128 x 64 and stages of 32 rows, so that two workgroups fit a CU: one
// stores its tile while the other sums (128 experts of 768 x 2048, 32 rows
// each: 67 us against 91 in tiles of 256). The 64 tile is for few
// tiles: its 4 waves are teams of one, each with the whole tile, stages of its
// own and a quarter of the rows, joined at the end through LDS; nothing but
// that join waits on another wave. Stages of 32 rows let two workgroups fit a
// CU (576 x 2080 from 2067 rows: 26 us in stages of 64, 19 so).
// kSaved: x is a checkpoint, decoded on its way into LDS (exact, and free: 826
// us on 8192 x 8192 x 8192, from bf16 841-849). The two chunks that a lane
// decodes go to every other chunk of a row, which the counters show as bank
// conflicts (17% of the LDS cycles of the 256 tile, 1% in its bf16 form).
// kTokens: there are token indices (with kElements: there may be).
template <int TO, int TI, bool kSaved, int kAccess, bool kTokens>
struct Tile {
    static constexpr int kTeams = TO == 64 ? 4 : 1;
    static constexpr int kThreads = (TI == 256 ? 512 : 256) / kTeams;          // of a team
    static constexpr int kDepth = TO == TI && TO > 64 ? kMostDepth : kMostDepth / 2;      // rows of a stage
    static constexpr int WO = TO == 64 ? 1 : 2, WI = kThreads / 64 / WO;       // waves over the tile
    static constexpr int FO = TO / WO / 32, FI = TI / WI / 32;  // 32 x 32 blocks of a wave
    static constexpr int kSteps = kDepth / 16;                 // matrix steps of a stage
    static constexpr int kParts = kSteps / 2;                  // steps that move a stage's chunks
    static constexpr int CO = TO / 8;                          // chunks of a staged row of dy
    static constexpr int NO = kDepth * CO / kThreads;          // chunks of dy a thread stages
    static constexpr int CI = TI / (kSaved ? 16 : 8);          // 16-byte loads of a row of x
    static constexpr int NI = kDepth * CI / kThreads;
    static_assert(kSteps == 2 || kSteps == 4, "the steps of sum()");
    static_assert(NO <= 16 && NI <= 16, "the bits of Moving::none");
    static constexpr int kStage = kDepth * (TO + TI);          // elements of one stage
    static constexpr int kLds = 2 * kStage * 2 > TO * TI * 2 ? 2 * kStage * 2 : TO * TI * 2;

    const Args& a;
    uint16_t* lds;
    int64_t lo, hi, o0, i0;
    int tid, lane, wave;
    // A stage on its way into LDS.
    struct Moving {
        u32x4 o[NO], i[NI];
        uint32_t s[kSaved ? NI : 1];
        uint32_t none;                 // Wide: bit j: o[j], bit 16 + j: i[j] is of no row
        int32_t tok[NI];               // the next one's rows of x
        uint64_t dropped;              // the next one's rows without a token, a bit each
        int32_t of_lane;               // the token of row `lane` of the one after it
    };

    // A team of one wave needs no barrier: its LDS accesses run in order.
    __device__ __forceinline__ void sync() {
        if constexpr (kThreads == 64) __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        else __syncthreads();
    }
    __device__ __forceinline__ uint16_t* stage_o(int b) { return lds + b * kStage; }
    __device__ __forceinline__ uint16_t* stage_i(int b) { return lds + b * kStage + kDepth * TO; }

    // Columns that this thread loads. A load that would cross the row's end
    // ends there, so its columns lie behind their places by as much as the row
    // is short of whole loads; place_o and place_i say where they belong. Loads
    // wholly past the end fill columns that are not stored, with anything: a
    // column of dy or x reaches only its own row or column of the gradient.
    __device__ __forceinline__ int64_t column_o() const { return min(o0 + tid % CO * 8, a.O - 8); }
    __device__ __forceinline__ int64_t column_i() const {
        constexpr int kLoad = kSaved ? 16 : 8;
        return min(i0 + tid % CI * kLoad, a.I - kLoad);
    }
    // The place in the tile of its row or column r: within the load that the
    // end crosses, the elements past those that belong to the load before it.
    template <int kLoad>
    static __device__ __forceinline__ int place(int r, int64_t left) {
        const int n = kAccess == kElements || left > 256 ? 256 : (int)left;
        return (r ^ n) & -kLoad ? r : (r & -kLoad) | ((r + n) & (kLoad - 1));
    }
    __device__ __forceinline__ int place_o(int r) const { return place<8>(r, a.O - o0); }
    __device__ __forceinline__ int place_i(int r) const { return place<kSaved ? 16 : 8>(r, a.I - i0); }

    __device__ __forceinline__ bool indexed() const { return kTokens && (kAccess != kElements || a.tokens); }

    // The tokens of the stage at t0, a row a lane (0 past the last row and
    // without token indices: no load uses those).
    __device__ __forceinline__ int32_t lane_token(int64_t t0) const {
        const int64_t left = hi - t0 < 0 ? 0 : hi - t0;
        const int rows = left < kDepth ? (int)left : kDepth;
        return __builtin_amdgcn_raw_buffer_load_b32(
            __builtin_amdgcn_make_buffer_rsrc((void*)(a.tokens + t0), (short)0, indexed() ? rows * 4 : 0,
                                              (int)kBufferWord), lane * 4, 0, 0);
    }
    // What a stage's loads need of its tokens: this thread's rows of x, and which
    // rows have none in x. Those add nothing, whatever dy holds there (zeros for
    // their x alone would not do against NaN and infinities).
    __device__ __forceinline__ void use_tokens(Moving& m, int32_t of_lane) {
#pragma unroll
        for (int j = 0; j < NI; ++j)
            m.tok[j] = __builtin_amdgcn_ds_bpermute((j * (kThreads / CI) + tid / CI) * 4, of_lane);
        m.dropped = __ballot((uint32_t)of_lane >= (uint32_t)a.x_rows);
    }
    // kOutside where the row of dy in chunk j of this thread is one of `rows`, else 0.
    __device__ __forceinline__ uint32_t is_of(uint64_t rows, int j) const {
        constexpr int R = kThreads / CO;
        static_assert(R <= 32 && 32 % R == 0 && kDepth <= 64, "the rows of a chunk are in one word");
        const uint32_t w = (uint32_t)(rows >> (j * R / 32 * 32));
        return (w << (32 - R - j * R % 32) << (R - 1 - tid / CO)) & kOutside;
    }

    // Part kPart of kOf of the loads of dy for the stage at t0. With kDrop, rows
    // without a token are not loaded.
    template <int kPart, int kOf, bool kDrop = kTokens>
    __device__ __forceinline__ void load_o(Moving& m, int64_t t0) {
        const int64_t left = hi - t0 < 0 ? 0 : hi - t0;
        const int rows = left < kDepth ? (int)left : kDepth;
        if constexpr (kAccess == kBuffers) {
            // rows past the last lie past the buffer by themselves
            const __amdgpu_buffer_rsrc_t d =
                buffer(a.dy + t0 * a.dy_stride, rows, (uint32_t)a.dy_stride * 2, (uint32_t)a.O * 2);
            const uint32_t at = (uint32_t)(tid / CO) * (uint32_t)a.dy_stride * 2 + (uint32_t)column_o() * 2;
#pragma unroll
            for (int j = kPart * NO / kOf; j < (kPart + 1) * NO / kOf; ++j)
                m.o[j] = buffer16(d, (at + (uint32_t)(j * (kThreads / CO)) * (uint32_t)a.dy_stride * 2) |
                                         (kDrop ? is_of(m.dropped, j) : 0));
        } else if constexpr (kAccess == kWide) {
            const uint64_t gone = (kDrop ? m.dropped : 0) | (rows < 64 ? ~0ull << rows : 0);
#pragma unroll
            for (int j = kPart * NO / kOf; j < (kPart + 1) * NO / kOf; ++j) {
                const int t = j * (kThreads / CO) + tid / CO;
                m.none = (m.none & ~(1u << j)) | is_of(gone, j) >> (31 - j);
                m.o[j] = *gbl<u32x4_a2>(a.dy + min(t0 + t, hi - 1) * a.dy_stride + column_o());
            }
        } else {
#pragma unroll
            for (int j = kPart * NO / kOf; j < (kPart + 1) * NO / kOf; ++j) {
                const int t = j * (kThreads / CO) + tid / CO, c = tid % CO;
                const int64_t n = a.O - o0 - c * 8;
                m.o[j] = u32x4{};
                if (n > 0 && t < rows && !(kDrop && is_of(m.dropped, j)))
                    m.o[j] = load_row(a.dy + (t0 + t) * a.dy_stride + o0 + c * 8, (int)(n < 8 ? n : 8));
            }
        }
    }

    // The same of x.
    template <int kPart, int kOf>
    __device__ __forceinline__ void load_i(Moving& m, int64_t t0) {
        const int64_t left = hi - t0 < 0 ? 0 : hi - t0;
        const int rows = left < kDepth ? (int)left : kDepth;
        if constexpr (kAccess == kBuffers) {
            // with token indices the whole of x is one buffer, without the stage's rows are
            const uint32_t stride = (uint32_t)(kSaved ? a.codes_stride : a.x_stride * 2);
            const uint32_t length = (uint32_t)a.I * (kSaved ? 1 : 2);
            const uint8_t* base = kSaved ? a.codes : (const uint8_t*)a.x;
            const uint32_t span = kTokens ? (uint32_t)a.x_rows : (uint32_t)rows;
            const int64_t first = kTokens ? 0 : t0;
            const __amdgpu_buffer_rsrc_t x = buffer(base + first * stride, span, stride, length);
            __amdgpu_buffer_rsrc_t s = x;
            if constexpr (kSaved)
                s = buffer(a.scales + first * a.scales_stride, span, (uint32_t)a.scales_stride,
                           (uint32_t)(a.I + kScaleBlock - 1) / kScaleBlock);
            const uint32_t col = (uint32_t)column_i() * (kSaved ? 1 : 2);
            const uint32_t block = (uint32_t)scale_block(i0 + tid % CI * 16, a.I);
#pragma unroll
            for (int j = kPart * NI / kOf; j < (kPart + 1) * NI / kOf; ++j) {
                const int t = j * (kThreads / CI) + tid / CI;
                const uint32_t row = kTokens ? (uint32_t)m.tok[j] : (uint32_t)t;
                // or'ed in rather than selected, so that no branch guards the products
                const uint32_t out = row < span && t < rows ? 0 : kOutside;
                m.i[j] = buffer16(x, min(out | (row * stride + col), kOutside));
                if constexpr (kSaved)
                    m.s[j] = __builtin_amdgcn_raw_buffer_load_b8(
                        s, (int)min(out | (row * (uint32_t)a.scales_stride + block), kOutside), 0, 0);
            }
        } else if constexpr (kAccess == kWide) {
            const int64_t block = scale_block(i0 + tid % CI * 16, a.I);
#pragma unroll
            for (int j = kPart * NI / kOf; j < (kPart + 1) * NI / kOf; ++j) {
                const int t = j * (kThreads / CI) + tid / CI;
                int64_t row = indexed() ? m.tok[j] : t0 + t;
                const bool in = t < rows && (uint64_t)row < (uint64_t)a.x_rows;
                m.none = (m.none & ~(0x10000u << j)) | (in ? 0 : 0x10000u << j);
                row = in ? row : 0;
                if constexpr (kSaved) {
                    m.i[j] = *gbl<u32x4_a1>(a.codes + row * a.codes_stride + column_i());
                    m.s[j] = *gbl<uint8_t>(a.scales + row * a.scales_stride + block);
                } else {
                    m.i[j] = *gbl<u32x4_a2>(a.x + row * a.x_stride + column_i());
                }
            }
        } else {
#pragma unroll
            for (int j = kPart * NI / kOf; j < (kPart + 1) * NI / kOf; ++j) {
                const int t = j * (kThreads / CI) + tid / CI, c = tid % CI;
                const int64_t row = t >= rows ? -1 : indexed() ? m.tok[j] : t0 + t;
                const int64_t col = i0 + c * (kSaved ? 16 : 8), n = a.I - col;
                m.i[j] = u32x4{};
                if constexpr (kSaved) m.s[j] = 0;
                if (n > 0 && row >= 0 && row < a.x_rows) {
                    if constexpr (kSaved) {
                        m.i[j] = codes16(a.codes + row * a.codes_stride + col, (int)(n < 16 ? n : 16));
                        m.s[j] = *gbl<uint8_t>(a.scales + row * a.scales_stride + col / kScaleBlock);
                    } else {
                        m.i[j] = load_row(a.x + row * a.x_stride + col, (int)(n < 8 ? n : 8));
                    }
                }
            }
        }
    }

    // Part of the loaded chunks into LDS buffer b.
    template <int kPart, int kOf>
    __device__ __forceinline__ void store(Moving& m, int b) {
#pragma unroll
        for (int j = kPart * NO / kOf; j < (kPart + 1) * NO / kOf; ++j) {
            const int t = j * (kThreads / CO) + tid / CO, c = tid % CO;
            if constexpr (kAccess == kWide) m.o[j] = m.none >> j & 1 ? u32x4{} : m.o[j];
            *(u32x4*)(stage_o(b) + t * TO + chunk_at<TO>(t, c) * 8) = m.o[j];
        }
#pragma unroll
        for (int j = kPart * NI / kOf; j < (kPart + 1) * NI / kOf; ++j) {
            const int t = j * (kThreads / CI) + tid / CI, c = tid % CI;
            if constexpr (kAccess == kWide) m.i[j] = m.none >> (16 + j) & 1 ? u32x4{} : m.i[j];
            if constexpr (kSaved) {
                u32x4 p, q;
                decode16(m.i[j], __uint_as_float(m.s[j] << 23), p, q);
                u32x4* d = (u32x4*)(stage_i(b) + t * TI + chunk_at<TI>(t, 2 * c) * 8);
                d[0] = p;
                d[1] = q;
            } else {
                *(u32x4*)(stage_i(b) + t * TI + chunk_at<TI>(t, c) * 8) = m.i[j];
            }
        }
    }

    // A 32-column block of 16 staged rows as a matrix operand: lane l holds
    // column l % 32, rows (l / 32) * 8 + 0 .. 7. Each transposing read gives a
    // lane four rows of one column out of the 4 x 16 blocks that 16 lanes name.
    template <int kWidth>
    __device__ __forceinline__ bf16x8 operand(const uint16_t* rows, int step, int col) {
        const int t = step * 16 + (lane >> 5) * 8 + ((lane & 15) >> 2);
        const int c = (col >> 3) + ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
        const uint16_t* p = rows + t * kWidth + chunk_at<kWidth>(t, c) * 8 + (lane & 1) * 4;
        const s16x4 u = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TIDE_LDS s16x4*)p);
        const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TIDE_LDS s16x4*)(p + 4 * kWidth));
        const bf16x4 x = __builtin_bit_cast(bf16x4, u), y = __builtin_bit_cast(bf16x4, v);
        return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    __device__ __forceinline__ void operands(int b, int step, bf16x8 (&fo)[FO], bf16x8 (&fi)[FI]) {
#pragma unroll
        for (int f = 0; f < FO; ++f) fo[f] = operand<TO>(stage_o(b), step, (wave / WI) * (TO / WO) + f * 32);
#pragma unroll
        for (int f = 0; f < FI; ++f) fi[f] = operand<TI>(stage_i(b), step, (wave % WI) * (TI / WI) + f * 32);
    }

    // Asks the scheduler to spread a step's LDS and memory instructions over
    // its matrix instructions, each of which leaves 32 cycles to issue others.
    template <int kStep, int kAt = 0>
    __device__ __forceinline__ void interleave() {
        constexpr int kMatrix = 0x8, kRead = 0x100, kWrite = 0x200, kLoad = 0x20;
        constexpr int M = FO * FI, R = 2 * (FO + FI);
        constexpr bool moves = kStep < kParts;
        constexpr int W = moves ? (NO + (kSaved ? 2 : 1) * NI) / kParts : 0;
        constexpr int L = moves ? (NO + (kSaved ? 2 : 1) * NI) / kParts : kStep == kParts && kTokens ? 1 : 0;
        if constexpr (kAt < M) {
            constexpr int r = (kAt + 1) * R / M - kAt * R / M, w = (kAt + 1) * W / M - kAt * W / M;
            constexpr int l = (kAt + 1) * L / M - kAt * L / M;
            __builtin_amdgcn_sched_group_barrier(kMatrix, 1, 0);
            if constexpr (r > 0) __builtin_amdgcn_sched_group_barrier(kRead, r, 0);
            if constexpr (w > 0) __builtin_amdgcn_sched_group_barrier(kWrite, w, 0);
            if constexpr (l > 0) __builtin_amdgcn_sched_group_barrier(kLoad, l, 0);
            interleave<kStep, kAt + 1>();
        }
    }

    template <int kStep>
    __device__ __forceinline__ void step(int64_t t0, int b, Moving& m, bf16x8 (&fo)[2][FO], bf16x8 (&fi)[2][FI],
                                         f32x16 (&acc)[FO][FI]) {
        constexpr int now = kStep & 1, next = now ^ 1;
        if constexpr (kStep < kSteps - 1) {
            operands(b, kStep + 1, fo[next], fi[next]);
        } else {
            sync();
            operands(b ^ 1, 0, fo[next], fi[next]);
        }
        if constexpr (kStep < kParts) {
            store<kStep, kParts>(m, b ^ 1);
            load_o<kStep, kParts>(m, t0 + 2 * kDepth);
            load_i<kStep, kParts>(m, t0 + 2 * kDepth);
        }
        if constexpr (kStep == kParts && kTokens) {
            use_tokens(m, m.of_lane);
            m.of_lane = lane_token(t0 + 4 * kDepth);
        }
#pragma unroll
        for (int x = 0; x < FO; ++x)
#pragma unroll
            for (int y = 0; y < FI; ++y)
                acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fi[now][y], fo[now][x], acc[x][y], 0, 0, 0);
        if constexpr (kAccess != kElements) interleave<kStep>();
    }

    // The sum over rows [lo, hi). A step's operands are read while the step
    // before is multiplied; a stage is loaded two stages before it is multiplied
    // and written to LDS one before, in the shadow of the matrix instructions;
    // one barrier a stage, before its last step, by when nothing of it is left
    // to read.
    __device__ __forceinline__ void sum(f32x16 (&acc)[FO][FI]) {
        if (lo >= hi) return;
        Moving first, m;
        // The first rows of dy do not wait for their tokens; those without one are
        // dropped when they are there, by a mask (a select became a branch around
        // the load and a wait for everything). All other stages' tokens are loaded
        // a stage before their rows, which then wait for no newer load. 128 experts
        // of 767 x 2047 with 32 rows each take 114 us, as without the dropping,
        // and 127 where the first rows do wait.
        if constexpr (kTokens) {
            const int32_t first_of = lane_token(lo), next_of = lane_token(lo + kDepth);
            const int32_t third_of = lane_token(lo + 2 * kDepth);
            m.of_lane = lane_token(lo + 3 * kDepth);
            load_o<0, 1, false>(first, lo);
            __builtin_amdgcn_sched_barrier(0);
            use_tokens(first, first_of);
            load_i<0, 1>(first, lo);
            use_tokens(m, next_of);
            load_o<0, 1>(m, lo + kDepth);
            load_i<0, 1>(m, lo + kDepth);
            use_tokens(m, third_of);
#pragma unroll
            for (int j = 0; j < NO; ++j) first.o[j] &= (is_of(first.dropped, j) >> 31) - 1;
        } else {
            load_o<0, 1>(first, lo);
            load_i<0, 1>(first, lo);
            load_o<0, 1>(m, lo + kDepth);
            load_i<0, 1>(m, lo + kDepth);
        }
        store<0, 1>(first, 0);
        sync();
        bf16x8 fo[2][FO], fi[2][FI];
        operands(0, 0, fo[0], fi[0]);
        // two stages a turn, so that the buffer is known when compiling (4% faster)
        for (int64_t t0 = lo; t0 < hi; t0 += 2 * kDepth) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int64_t t = t0 + b * kDepth;
                if (b > 0 && t >= hi) break;
                step<0>(t, b, m, fo, fi, acc);
                step<1>(t, b, m, fo, fi, acc);
                if constexpr (kSteps == 4) {
                    step<2>(t, b, m, fo, fi, acc);
                    step<3>(t, b, m, fo, fi, acc);
                }
            }
        }
        sync();
    }

    // acc[x][y]: lane l holds out row (o) l % 32 of the block, and for each
    // group of four registers four consecutive in columns (i).
    static __device__ __forceinline__ int row_of(int wave, int lane, int x) {
        return wave / WI * (TO / WO) + x * 32 + (lane & 31);
    }
    static __device__ __forceinline__ int column_of(int wave, int lane, int y, int r) {
        return wave % WI * (TI / WI) + y * 32 + r * 8 + (lane >> 5) * 4;
    }

    // Whether columns y, r of a wave are of the load that the row's end crosses.
    __device__ __forceinline__ bool crossed(int y, int r) const {
        const int i = __builtin_amdgcn_readfirstlane(wave) % WI * (TI / WI) + y * 32 + r * 8;
        return place_i(i) != i;
    }

    // The 64 tile: each team's sums go to LDS, four columns a 16-byte chunk,
    // placed by row for the banks, and are added in the teams' order; the whole
    // workgroup stores them, or keeps them in fp32 for join_splits.
    __device__ __forceinline__ void finish_teams(f32x16 (&acc)[FO][FI], uint16_t* all, int team, uint16_t* out,
                                                 float* partial) {
        constexpr int C = TI / 4;
        __syncthreads();
        float* mine = (float*)all + team * TO * TI;
#pragma unroll
        for (int x = 0; x < FO; ++x)
#pragma unroll
            for (int y = 0; y < FI; ++y)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int o = place_o(row_of(wave, lane, x)), i = column_of(wave, lane, y, r);
                    u32x4 v;
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = __float_as_uint(acc[x][y][r * 4 + q]);
                    if (!crossed(y, r)) {
                        *(u32x4*)(mine + o * TI + ((i >> 2) ^ (o & (C - 1))) * 4) = v;
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int at = place_i(i + q);
                            mine[o * TI + ((at >> 2) ^ (o & (C - 1))) * 4 + (at & 3)] = __uint_as_float(v[q]);
                        }
                    }
                }
        __syncthreads();
        for (int j = threadIdx.x; j < TO * C; j += kThreads * kTeams) {
            const int o = j / C, c = j % C;
            float v[4] = {};
            for (int k = 0; k < kTeams; ++k) {
                const u32x4 w = *(const u32x4*)((const float*)all + k * TO * TI + o * TI + (c ^ (o & (C - 1))) * 4);
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] += __uint_as_float(w[q]);
            }
            if (partial) {
                *gbl_mut<u32x4>(partial + j * 4) = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]),
                                                         __float_as_uint(v[2]), __float_as_uint(v[3])};
            } else {
                store4(a, out, o0 + o, i0 + c * 4, v);
            }
        }
    }

    // The sums start with what the gradient holds.
    __device__ __forceinline__ void add_to(f32x16 (&acc)[FO][FI], const uint16_t* out) {
#pragma unroll
        for (int x = 0; x < FO; ++x) {
            const int64_t o = o0 + place_o(row_of(wave, lane, x));
#pragma unroll
            for (int y = 0; y < FI; ++y)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int64_t i = i0 + place_i(column_of(wave, lane, y, r / 4) + r % 4);
                    if (o < a.O && i < a.I) acc[x][y][r] = lo_bf16(*gbl<uint16_t>(out + o * a.I + i));
                }
        }
    }

    // The tile goes through LDS so that whole rows are stored: row o's 16-byte
    // chunk c lies at c ^ o, its halves swapped in every other 16 rows, so that,
    // by their addresses, neither the 8-byte writes nor the reads meet a bank twice.
    __device__ __forceinline__ void finish(f32x16 (&acc)[FO][FI], uint16_t* out) {
        const bool whole = o0 + TO <= a.O && i0 + TI <= a.I;
        if (whole) {
            into_lds<true>(acc);
            __syncthreads();
            if (a.past_caches) store_tile<true, true>(out);
            else store_tile<true, false>(out);
        } else {
            into_lds<false>(acc);
            __syncthreads();
            if (a.past_caches) store_tile<false, true>(out);
            else store_tile<false, false>(out);
        }
    }
    template <bool kWhole>
    __device__ __forceinline__ void into_lds(f32x16 (&acc)[FO][FI]) {
        constexpr int C = TI / 8;
#pragma unroll
        for (int x = 0; x < FO; ++x) {
            const int o = kWhole ? row_of(wave, lane, x) : place_o(row_of(wave, lane, x));
#pragma unroll
            for (int y = 0; y < FI; ++y) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = column_of(wave, lane, y, r);
                    const u32x2 p = {pack_bf16(acc[x][y][r * 4], acc[x][y][r * 4 + 1]),
                                     pack_bf16(acc[x][y][r * 4 + 2], acc[x][y][r * 4 + 3])};
                    if (kWhole || !crossed(y, r)) {
                        *(u32x2*)(lds + o * TI + ((i >> 3) ^ (o & (C - 1))) * 8 + ((i & 4) ^ ((o >> 2) & 4))) = p;
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int at = place_i(i + q);
                            lds[o * TI + ((at >> 3) ^ (o & (C - 1))) * 8 + ((at & 7) ^ ((o >> 2) & 4))] =
                                (uint16_t)(p[q / 2] >> (16 * (q & 1)));
                        }
                    }
                }
            }
        }
    }
    template <bool kWhole, bool kPastCaches>
    __device__ __forceinline__ void store_tile(uint16_t* out) {
        constexpr int C = TI / 8, N = TO * C / kThreads;
#pragma unroll
        for (int j0 = 0; j0 < N; j0 += 4) {
            u32x4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = *(const u32x4*)(lds + (tid + (j0 + j) * kThreads) * 8);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at = tid + (j0 + j) * kThreads, o = at / C, c = (at % C) ^ (o & (C - 1));
                if (o & 16) v[j] = u32x4{v[j][2], v[j][3], v[j][0], v[j][1]};
                uint16_t* d = out + (o0 + o) * a.I + i0 + c * 8;
                const int64_t n = kWhole ? 8 : o0 + o < a.O ? a.I - i0 - c * 8 : 0;
                if (n >= 8) {
                    store_chunk<kPastCaches>(d, v[j]);
                } else {
#pragma unroll
                    for (int q = 0; q < 7; ++q)
                        if (q < n) *gbl_mut<uint16_t>(d + q) = (uint16_t)(v[j][q / 2] >> (16 * (q & 1)));
                }
            }
        }
    }
};

template <int TO, int TI, bool kSaved, int kAccess, bool kTokens>
__global__ __launch_bounds__(TI == 256 ? 512 : 256, 2) void weight_grads(Args a, GradPtrs g) {
    using K = Tile<TO, TI, kSaved, kAccess, kTokens>;
    constexpr bool kInTeams = K::kTeams > 1;
    __shared__ __attribute__((aligned(1024))) uint16_t lds[K::kTeams * K::kLds / 2];
    // Workgroups go round robin over the XCDs: each XCD gets one run of tiles,
    // so that tiles that share rows share an L2.
    const int per = gridDim.x / 8, at = (int)(blockIdx.x % 8) * per + (int)(blockIdx.x / 8);
    const int tiles = a.tiles_o * a.tiles_i;
    if (at >= a.count * a.splits * tiles) return;
    const int part = at / tiles, e = part / a.splits, split = part - e * a.splits;
    int tile = at - part * tiles;
    // within an expert, bands of 8 tile rows, walked column by column
    const int band = tile / (8 * a.tiles_i), high = min(8, a.tiles_o - band * 8);
    tile -= band * 8 * a.tiles_i;
    const int to = band * 8 + tile % high, ti = tile / high;
    int64_t lo = 0, hi = a.n;
    if (a.offsets) {
        lo = a.offsets[a.first + e];
        hi = a.offsets[a.first + e + 1];
        lo = lo < 0 ? 0 : lo > a.n ? a.n : lo;
        hi = hi < lo ? lo : hi > a.n ? a.n : hi;
    }
    const int team = kInTeams ? __builtin_amdgcn_readfirstlane(threadIdx.x / K::kThreads) : 0;
    if (kInTeams) {                    // whole stages to each team of each split
        const int64_t parts = a.splits * K::kTeams, stages = (hi - lo + K::kDepth - 1) / K::kDepth;
        const int64_t each = (stages + parts - 1) / parts * K::kDepth;
        lo = min(lo + (split * K::kTeams + team) * each, hi);
        hi = min(lo + each, hi);
    }
    const int tid = threadIdx.x % K::kThreads;
    K k{a, lds + team * (K::kLds / 2), lo, hi, (int64_t)to * TO, (int64_t)ti * TI, tid, tid & 63, tid >> 6};
    f32x16 acc[K::FO][K::FI] = {};
    if (!kInTeams && a.accumulate) k.add_to(acc, g.p[e]);
    k.sum(acc);
    if constexpr (kInTeams)
        k.finish_teams(acc, lds, team, g.p[e],
                       a.splits > 1 ? a.partial + ((int64_t)part * tiles + to * a.tiles_i + ti) * (TO * TI)
                                    : nullptr);
    else
        k.finish(acc, g.p[e]);
}

// Joins the splits of 64 tiles, in order: four columns a lane.
__global__ __launch_bounds__(256) void join_splits(Args a, GradPtrs g) {
    constexpr int kTile = 64, kPer = kTile * kTile / 4 / 256;      // workgroups for a tile
    const int tiles = a.tiles_o * a.tiles_i;
    const int j = blockIdx.x % kPer * 256 + threadIdx.x, tile = blockIdx.x / kPer % tiles;
    const int e = blockIdx.x / kPer / tiles;
    const int64_t apart = (int64_t)tiles * (kTile * kTile);
    const float* p = a.partial + (int64_t)e * a.splits * apart + (int64_t)tile * (kTile * kTile) + j * 4;
    float v[4] = {};
    for (int s = 0; s < a.splits; s += 8) {
        u32x4 w[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) w[c] = *gbl<u32x4>(p + min(s + c, a.splits - 1) * apart);
#pragma unroll
        for (int c = 0; c < 8; ++c)
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] += s + c < a.splits ? __uint_as_float(w[c][q]) : 0.0f;
    }
    store4(a, g.p[e], (int64_t)(tile / a.tiles_i) * kTile + j / (kTile / 4),
           (int64_t)(tile % a.tiles_i) * kTile + j % (kTile / 4) * 4, v);
}

template <int TO, int TI>
hipError_t launch_tiles(const Args& a, const GradPtrs& g, Access how, hipStream_t stream) {
    const int64_t groups = (int64_t)a.count * a.splits * a.tiles_o * a.tiles_i;
    const dim3 grid((uint32_t)((groups + 7) / 8 * 8));
    constexpr uint32_t threads = TI == 256 ? 512 : 256;
    const auto start = [&](auto kernel) { return enqueue(kernel, grid, threads, 0, stream, a, g); };
    const auto run = [&](auto saved) {
        constexpr bool kSaved = saved.value;
        if (how == kBuffers && a.tokens) return start(weight_grads<TO, TI, kSaved, kBuffers, true>);
        if (how == kBuffers) return start(weight_grads<TO, TI, kSaved, kBuffers, false>);
        if (how == kWide && a.tokens) return start(weight_grads<TO, TI, kSaved, kWide, true>);
        if (how == kWide) return start(weight_grads<TO, TI, kSaved, kWide, false>);
        if constexpr (TO == 64)
            if (how == kElements) return start(weight_grads<TO, TI, kSaved, kElements, true>);
        return hipErrorInvalidConfiguration;           // plan_tiles and how_to_read disagree
    };
    const hipError_t e = a.codes ? run(std::true_type{}) : run(std::false_type{});
    if (e != hipSuccess || a.splits == 1) return e;
    const int64_t blocks = (int64_t)a.count * a.tiles_o * a.tiles_i * (64 * 64 / 4 / 256);
    return enqueue(join_splits, dim3((uint32_t)blocks), 256, 0, stream, a, g);
}

// The buffers' 32-bit byte offsets have to reach a stage of dy and, with token
// indices, all of x. Alignment does not matter to them: from 4096 rows, 4096 x
// 4096 takes 112-117 us and 4095 x 4095, rows end to end, 125.
Access how_to_read(const Args& a) {
    const int64_t step = a.codes ? 16 : 8, xs = a.codes ? a.codes_stride : a.x_stride * 2;
    const int64_t lim = kMostBytes, rows = a.tokens ? a.x_rows : kMostDepth;
    if (a.O < 8 || a.I < step) return kElements;       // plan_tiles gives these tiles of 64
    if (a.dy_stride > lim / 2 / kMostDepth || (rows > 0 && (xs > lim / rows || a.scales_stride > lim / rows)))
        return kWide;
    return kBuffers;
}

// Whether the gradients are stored past the caches. It leaves those to dy and x
// (128 experts of 767 x 2047, 128 rows each, 164 us against 178-180), but the
// lines that two tiles share, where rows of the gradient do not start on lines,
// are written twice. With few rows nothing is there to be left in: the same with
// 64 rows each 166 us past the caches and 140-146 through them; 128 experts of
// 512 x 1001 with 5 rows each 56 and 36-38, with 128 62 and 47-63, with 192 64
// and 55-72; 8192 x 8191 from 64 rows 59 and 39.
bool stores_past_caches(int64_t n, int64_t I, int32_t experts) {
    return I % 64 == 0 || n / experts > kMostDepth;
}

// Tile and splits. A large tile reuses each staged element more (1300, 1150,
// 990 and 480 TFLOP/s on long sums, in tiles of 256 x 256, 256 x 128, 128 x 128
// and 64 x 64), a small one leaves fewer CUs idle and, with its teams, waits
// less. The costs below, in us, were fitted to measured times: a round of
// workgroups has a part that does not depend on the rows, and each stage of 64
// rows adds to it. Both sides where the choice turns: 128 experts of 768 x 2048
// with 512 rows each 276-280 us in 256 x 256 and 276-297 in 256 x 128, with 64
// rows 93 and 77; 1024 x 8192 from 8192 rows 152-154 us (128 tiles of 256 x 256),
// 138-145 (256 of 256 x 128) and 147-151 (512 of 128 x 128); 8 experts of 384 x
// 700, 512 rows each, 17 us (96 of 256 x 128) and 13 (144 of 128 x 128); 2048 x
// 2048 from 2000 rows 35-37 us (1024 of 64 x 64) and 25-28 (256 of 128 x 128);
// 576 x 2080 from 2067 rows 24 us (85 of 128 x 128) and 19 (297 of 64 x 64).
// Splits: where even tiles of 64 leave CUs idle, the rows of each are divided
// among several workgroups, whose fp32 sums a second kernel adds in order:
// 128 x 2048 from 8192 rows 29 us with one, 21 with two, 17 with four, 19 with
// eight. The rows are taken as evenly spread over the experts: how many each
// has is known on the device only.
struct Plan {
    int64_t tiles_o, tiles_i;
    int tile_o, tile_i, splits;
};
Plan plan_tiles(int64_t n, int64_t O, int64_t I, int32_t experts) {
    const int64_t cap = 1 << 20, stages = (n / experts + kMostDepth - 1) / kMostDepth;
    const auto tiles = [&](int64_t o, int64_t i) {
        return std::min((O + o - 1) / o, cap) * std::min((I + i - 1) / i, cap) * experts;
    };
    const auto rounds = [](int64_t groups, int64_t at_once) { return (double)((groups + at_once - 1) / at_once); };
    const double s = (double)stages;
    const int64_t small = tiles(64, 64);
    Plan p{0, 0, 64, 64, 1};
    double best = 0;
    for (int64_t k = 1; k == 1 || (k * small <= 512 && k * 4 <= stages); k *= 2) {
        const double each = (double)((stages + 4 * k - 1) / (4 * k));      // stages of a wave
        const double us = (k * small <= 256 ? 6 + each : rounds(k * small, 512) * (6 + 1.55 * each)) +
                          (k > 1 ? 5 + 0.01 * (double)(k * small) : 0);
        if (k == 1 || us < best) {
            best = us;
            p.splits = (int)k;
        }
    }
    if (O >= 16 && I >= 16) {
        const int64_t mid = tiles(128, 128), tall = tiles(256, 128), big = tiles(256, 256);
        const auto offer = [&](double us, int o, int i) {
            if (us < best) p = Plan{0, 0, o, i, 1}, best = us;
        };
        offer(mid <= 256 ? 6 + 0.75 * s : rounds(mid, 512) * (7 + 1.35 * s), 128, 128);
        offer(tall <= 256 ? 8 + 1.15 * s : rounds(tall, 512) * (5.5 + 1.95 * s), 256, 128);
        offer(rounds(big, 256) * (7.5 + 1.65 * s), 256, 256);
    }
    p.tiles_o = (O + p.tile_o - 1) / p.tile_o;
    p.tiles_i = (I + p.tile_i - 1) / p.tile_i;
    return p;
}

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
    return guarded([&]() -> tide_status {
        if (!bytes) return fail(TIDE_ERR_INVALID_ARG, "bytes is NULL");
        TIDE_TRY(check_sizes(rows, out, in, experts));
        const Plan p = plan_tiles(rows, out, in, experts);
        *bytes = p.splits > 1 ? p.splits * experts * p.tiles_o * p.tiles_i * p.tile_o * p.tile_i * 4 : 0;
        return TIDE_OK;
    });
}

tide_status tide_weight_grads_bf16(const uint16_t* dy, int64_t dy_stride, int64_t rows,
                                   int64_t out, const uint16_t* x, int64_t x_stride,
                                   const tide_saved* saved, int64_t x_rows, int64_t in,
                                   const int32_t* offsets, const int32_t* token_of_row,
                                   int32_t experts, uint16_t* const* grads, int32_t accumulate,
                                   void* workspace, int64_t workspace_bytes, void* stream) {
    return guarded([&]() -> tide_status {
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
        if (x && saved) return fail(TIDE_ERR_INVALID_ARG, "x and saved are both given");
        Mat rd[6];                     // dy, x or codes, scales, offsets, token_of_row, workspace
        TIDE_TRY(matrix("dy", dy, rows, out, dy_stride, 2, &rd[0]));
        if (saved) {
            TIDE_TRY(matrix("saved", saved->codes, x_rows, in, saved->codes_stride, 1, &rd[1]));
            TIDE_TRY(matrix("saved", saved->scales, x_rows, (in + kScaleBlock - 1) / kScaleBlock,
                            saved->scales_stride, 1, &rd[2]));
        } else {
            TIDE_TRY(matrix("x", x, x_rows, in, x_stride, 2, &rd[1]));
            rd[2] = Mat{};
        }
        TIDE_TRY(matrix("offsets", offsets, offsets ? 1 : 0, (int64_t)experts + 1,
                        (int64_t)experts + 1, 4, &rd[3]));
        TIDE_TRY(matrix("token_of_row", token_of_row, token_of_row ? 1 : 0, rows, rows, 4, &rd[4]));
        TIDE_TRY(matrix("workspace", workspace, 1, need / 4, need / 4, 4, &rd[5]));
        if (need > 0 && (rd[5].base & 15))
            return fail(TIDE_ERR_ALIGNMENT, "workspace is not 16-byte aligned");
        TIDE_TRY(no_overlap(&rd[5], 1, rd, 5));
        if (out == 0 || in == 0) return TIDE_OK;
        if (!grads) return fail(TIDE_ERR_INVALID_ARG, "grads is NULL");
        std::vector<uintptr_t> at(experts);
        const uintptr_t bytes = (uintptr_t)(out * in) * 2;
        for (int32_t e = 0; e < experts; ++e) {
            at[e] = (uintptr_t)grads[e];
            if (!at[e]) return fail(TIDE_ERR_INVALID_ARG, "grads[%d] is NULL", e);
            if (at[e] & 1) return fail(TIDE_ERR_ALIGNMENT, "grads[%d] is not 2-byte aligned", e);
            const Mat m{"one of the grads", at[e], 1, (int64_t)bytes, (int64_t)bytes};
            TIDE_TRY(no_overlap(&m, 1, rd, 6));
        }
        if (!std::is_sorted(at.begin(), at.end())) std::sort(at.begin(), at.end());
        for (int32_t e = 1; e < experts; ++e)
            if (at[e] - at[e - 1] < bytes)
                return fail(TIDE_ERR_INVALID_ARG, "two of the grads overlap");
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
        if (x_rows == 0) a.n = 0;              // no row of x to add
        const Access how = how_to_read(a);
        const Plan p = plan_tiles(rows, out, in, experts);
        a.past_caches = stores_past_caches(rows, in, experts);
        if (p.tiles_o > kMaxGroups / p.tiles_i)
            return fail(TIDE_ERR_UNSUPPORTED, "gradients of %lld x %lld", (long long)out, (long long)in);
        const int64_t tiles = p.tiles_o * p.tiles_i;
        a.tiles_o = (int32_t)p.tiles_o;
        a.tiles_i = (int32_t)p.tiles_i;
        a.splits = p.splits;
        const int32_t most = (int32_t)std::min<int64_t>(kMaxGrads, kMaxGroups / (tiles * p.splits));
        return on_stream(stream, [&](hipStream_t s) {
            for (int32_t e0 = 0; e0 < experts; e0 += most) {
                const int32_t ne = std::min(experts - e0, most);
                GradPtrs g{};
                for (int32_t e = 0; e < ne; ++e) g.p[e] = grads[e0 + e];
                a.first = e0;
                a.count = ne;
                a.partial = (float*)workspace + (int64_t)e0 * p.splits * tiles * p.tile_o * p.tile_i;
                const hipError_t launched = p.tile_i == 256   ? launch_tiles<256, 256>(a, g, how, s)
                                            : p.tile_o == 256 ? launch_tiles<256, 128>(a, g, how, s)
                                            : p.tile_o == 128 ? launch_tiles<128, 128>(a, g, how, s)
                                                              : launch_tiles<64, 64>(a, g, how, s);
                if (launched != hipSuccess) return launched;
            }
            return hipSuccess;
        });
    });
}

}  // extern "C"
