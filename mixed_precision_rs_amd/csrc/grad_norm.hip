// The square of the gradient norm over many tensors (tide_grad_squares) and
// clipping by it (tide_clip_grads) for gfx950.
//
// Tensors are cut into tiles of 16 KiB, and the workgroups walk the
// tiles; which workgroup has which tile follows from the sizes alone, so the
// sum does not depend on when they run. Squares and sums are fp64: a square of
// an fp32 number is exact in it, and neither overflows nor vanishes.
#include <algorithm>
#include <climits>
#include <type_traits>
#include <vector>

#include "device.hpp"
#include "host.hpp"

using namespace tide;

namespace {

constexpr int kThreads = 256;
// Each changed alone, over 1.2 GB of bf16 in 391 tensors, the median launch of the two
// that the squares take and of the three that clipping takes: as it is 100 and 174 us;
// tiles of 8 KiB 112 and 168, of 32 98 and 172, of 64 104 and 182; 2048 workgroups 106
// and 177, 16384 100 and 170, with 2 us more for joining their sums.
constexpr int kTileBytes = 16384;
template <class T>
constexpr int kTileOf = kTileBytes / (int)sizeof(T);
constexpr int64_t kMostGroups = 8192;
// Tiles that one workgroup sums alone, in one launch.
constexpr int64_t kAlone = 8;
// Tensors that together pass the memory-side cache (256 MiB) are read past the
// caches (the same launches: 100 us instead of 106, clipping 174 instead of 179);
// smaller ones by ordinary loads, so that clipping finds there what the squares
// have read (53 MB: 18.4 us instead of 20.7).
constexpr int64_t kPastCaches = (int64_t)192 << 20;

// The tensors of one launch, in its arguments (below 4 KiB). Tensor i has the tiles
// first[i] .. first[i + 1] - 1, the last of them with last[i] elements.
template <bool kOut>
struct Tensors {
    static constexpr int kMost = kOut ? 160 : 256;
    const void* in[kMost];
    void* out[kOut ? kMost : 1];
    int32_t first[kMost + 1];
    uint16_t last[kMost];
    int32_t count;
};
static_assert(sizeof(Tensors<true>) < 4000 && sizeof(Tensors<false>) < 4000, "launch arguments");

template <bool kOut>
__device__ __forceinline__ int tensor_of(const Tensors<kOut>& a, int tile) {
    int lo = 0, hi = a.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (a.first[mid] <= tile) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <int kAll>
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double part[kAll / 64];
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x / 64] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < kAll / 64; ++w) v += part[w];
    return v;
}

// Calls f(tensor, element, elements left in the tile) for this thread's vectors of a tile.
template <class T, bool kOut, class F>
__device__ __forceinline__ void each_vector(const Tensors<kOut>& a, int tile, F&& f) {
    constexpr int N = kVecOf<T>;
    const int i = tensor_of(a, tile);
    const int64_t lo = (int64_t)(tile - a.first[i]) * kTileOf<T>;
    const int n = tile + 1 == a.first[i + 1] ? a.last[i] : kTileOf<T>;
#pragma unroll 4
    for (int e = threadIdx.x * N; e < n; e += kThreads * N) f(i, lo + e, n - e < N ? n - e : N);
}

// Each workgroup's sum into partial; one workgroup alone writes the total.
template <class T, bool kOnce>
__global__ __launch_bounds__(kThreads) void sum_squares(Tensors<false> a, double* partial, double* total, int accumulate) {
    constexpr int N = kVecOf<T>;
    double sum = 0.0;
    for (int tile = blockIdx.x; tile < a.first[a.count]; tile += gridDim.x)
        each_vector<T>(a, tile, [&](int i, int64_t e, int n) {
            float v[N];
            widen(load_row<kOnce>((const T*)a.in[i] + e, n), v);
#pragma unroll
            for (int c = 0; c < N; ++c) sum = __builtin_fma((double)v[c], (double)v[c], sum);
        });
    sum = block_sum<kThreads>(sum);
    if (threadIdx.x) return;
    if (total) *gbl_mut<double>(total) = accumulate ? *gbl<double>(total) + sum : sum;
    else *gbl_mut<double>(partial + blockIdx.x) = sum;
}

constexpr int kSumThreads = 1024;
__global__ __launch_bounds__(kSumThreads) void sum_partials(const double* partial, int64_t n,
                                                            double* total, int accumulate) {
    double sum = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += 8 * kSumThreads) {
        double v[8];                   // loads that are under way together
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = i + j * kSumThreads < n ? *gbl<double>(partial + i + j * kSumThreads) : 0.0;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += v[j];
    }
    sum = block_sum<kSumThreads>(sum);
    if (threadIdx.x == 0) *gbl_mut<double>(total) = accumulate ? *gbl<double>(total) + sum : sum;
}

// Without kOut every tensor is clipped in place.
template <class T, bool kOnce, bool kOut>
__global__ __launch_bounds__(kThreads) void clip(Tensors<kOut> a, const double* total, double most, float* norm_to) {
    constexpr int N = kVecOf<T>;
    const double norm = sqrt(*gbl<double>(total));
    if (norm_to && blockIdx.x == 0 && threadIdx.x == 0) *gbl_mut<float>(norm_to) = (float)norm;
    const bool scaled = norm > most && norm < __builtin_inf();
    if (!kOut && !scaled) return;
    const double factor = most / norm;
    for (int tile = blockIdx.x; tile < a.first[a.count]; tile += gridDim.x)
        each_vector<T>(a, tile, [&](int i, int64_t e, int n) {
            T* to = (T*)(kOut ? a.out[i] : a.in[i]);
            if (!scaled && to == a.in[i]) return;
            u32x4 raw = load_row<kOnce>((const T*)a.in[i] + e, n);
            if (scaled) {
                float v[N];
                widen(raw, v);
#pragma unroll
                for (int c = 0; c < N; ++c) v[c] = (float)((double)v[c] * factor);
                raw = narrow(v);
            }
            store_row(to + e, n, raw);
        });
}

tide_status check_sizes(int32_t dtype, const int64_t* elems, int32_t tensors) {
    if (dtype != TIDE_DTYPE_BF16 && dtype != TIDE_DTYPE_FP32)
        return fail(TIDE_ERR_INVALID_ARG, "dtype %d is not BF16 (0) or FP32 (1)", dtype);
    if (tensors < 0) return fail(TIDE_ERR_INVALID_ARG, "negative tensor count");
    if (tensors && !elems) return fail(TIDE_ERR_INVALID_ARG, "elems is NULL");
    int64_t all = 0;
    for (int32_t i = 0; i < tensors; ++i) {
        if (elems[i] < 0) return fail(TIDE_ERR_INVALID_ARG, "elems[%d] is negative", i);
        if (__builtin_add_overflow(all, elems[i], &all) || all > INT64_MAX / 8)
            return fail(TIDE_ERR_OVERFLOW, "the tensors' sizes overflow int64");
    }
    return TIDE_OK;
}

bool past_caches(const int64_t* elems, int32_t tensors, int32_t size) {
    int64_t all = 0;
    for (int32_t i = 0; i < tensors; ++i) all += elems[i];
    return all > kPastCaches / size;
}

// Calls go(Tensors, workgroups, workgroups before) for each launch: up to kMost
// tensors and 2^30 tiles (a larger tensor is cut).
template <bool kOut, class F>
hipError_t each_launch(const void* const* in, void* const* out, const int64_t* elems, int32_t tensors,
                       int32_t size, F&& go) {
    const int64_t kMostTiles = (int64_t)1 << 30, tile = kTileBytes / size;
    Tensors<kOut> a{};
    int64_t tiles = 0, groups = 0;
    const auto flush = [&]() -> hipError_t {
        if (a.count == 0) return hipSuccess;
        a.first[a.count] = (int32_t)tiles;
        const int64_t g = tiles < kMostGroups ? tiles : kMostGroups;
        const hipError_t e = go(a, g, groups);
        groups += g;
        a.count = 0;
        tiles = 0;
        return e;
    };
    for (int32_t i = 0; i < tensors; ++i) {
        for (int64_t at = 0; at < elems[i];) {
            const int64_t left = elems[i] - at;
            const int64_t n = left < kMostTiles * tile ? left : kMostTiles * tile;
            const int64_t t = (n + tile - 1) / tile;
            if (a.count == Tensors<kOut>::kMost || tiles + t > kMostTiles) {
                const hipError_t e = flush();
                if (e != hipSuccess) return e;
            }
            a.in[a.count] = in ? (const char*)in[i] + at * size : nullptr;
            if (kOut) a.out[a.count] = (char*)out[i] + at * size;
            a.first[a.count] = (int32_t)tiles;
            a.last[a.count] = (uint16_t)(n - (t - 1) * tile);
            ++a.count;
            tiles += t;
            at += n;
        }
    }
    return flush();
}

// A range of addresses that is read or written.
struct Range {
    uintptr_t lo, hi;
};
void in_order(std::vector<Range>& r) {
    const auto less = [](const Range& a, const Range& b) { return a.lo < b.lo; };
    if (!std::is_sorted(r.begin(), r.end(), less)) std::sort(r.begin(), r.end(), less);
}
// INVALID_ARG where a range that is written shares a byte with another one that is
// written, or with one that is read.
tide_status check_ranges(std::vector<Range>& written, std::vector<Range>& read) {
    in_order(written);
    in_order(read);
    const char* what = "a tensor that is written overlaps another one";
    for (size_t i = 1; i < written.size(); ++i)
        if (written[i].lo < written[i - 1].hi) return fail(TIDE_ERR_INVALID_ARG, "%s", what);
    size_t w = 0;
    uintptr_t end = 0;                             // of what is read so far
    for (const Range& r : read) {
        for (; w < written.size() && written[w].lo < r.lo; ++w)
            if (written[w].lo < end) return fail(TIDE_ERR_INVALID_ARG, "%s", what);
        if (w > 0 && written[w - 1].hi > r.lo) return fail(TIDE_ERR_INVALID_ARG, "%s", what);
        end = std::max(end, r.hi);
    }
    for (; w < written.size(); ++w)
        if (written[w].lo < end) return fail(TIDE_ERR_INVALID_ARG, "%s", what);
    return TIDE_OK;
}

}  // namespace

extern "C" {

tide_status tide_grad_squares_workspace(int32_t dtype, const int64_t* elems, int32_t tensors,
                                        int64_t* bytes) {
    return guarded([&]() -> tide_status {
        if (!bytes) return fail(TIDE_ERR_INVALID_ARG, "bytes is NULL");
        TIDE_TRY(check_sizes(dtype, elems, tensors));
        int64_t groups = 0;
        (void)each_launch<false>(nullptr, nullptr, elems, tensors, dtype == TIDE_DTYPE_FP32 ? 4 : 2,
                                 [&](const Tensors<false>&, int64_t g, int64_t) {
            groups += g;
            return hipSuccess;
        });
        *bytes = groups <= kAlone ? 0 : groups * 8;
        return TIDE_OK;
    });
}

tide_status tide_grad_squares(int32_t dtype, const void* const* grads, const int64_t* elems,
                              int32_t tensors, double* total, int32_t accumulate, void* workspace,
                              int64_t workspace_bytes, void* stream) {
    return guarded([&]() -> tide_status {
        int64_t need = 0;
        TIDE_TRY(tide_grad_squares_workspace(dtype, elems, tensors, &need));
        if (need > 0 && (!workspace || workspace_bytes < need))
            return fail(TIDE_ERR_INVALID_ARG, "workspace holds %lld bytes, %lld needed",
                        (long long)(workspace ? workspace_bytes : 0), (long long)need);
        if (tensors && !grads) return fail(TIDE_ERR_INVALID_ARG, "grads is NULL");
        const int32_t size = dtype == TIDE_DTYPE_FP32 ? 4 : 2;
        Mat wr[2];
        TIDE_TRY(matrix("total", total, 1, 1, 1, 8, &wr[0]));
        TIDE_TRY(matrix("workspace", workspace, 1, need / 8, need / 8, 8, &wr[1]));
        TIDE_TRY(no_overlap(wr, 2, nullptr, 0));
        for (int32_t i = 0; i < tensors; ++i) {
            Mat rd;
            TIDE_TRY(matrix("one of the grads", grads[i], 1, elems[i], elems[i], size, &rd));
            TIDE_TRY(no_overlap(wr, 2, &rd, 1));
        }
        const bool once = past_caches(elems, tensors, size);
        return on_stream(stream, [&](hipStream_t s) {
            const bool alone = need == 0;          // no tile, or one launch of kAlone at most
            bool none = true;
            const hipError_t e = each_launch<false>(grads, nullptr, elems, tensors, size,
                                                    [&](const Tensors<false>& a, int64_t groups, int64_t before) {
                none = false;
                const auto kernel = once ? (size == 2 ? sum_squares<uint16_t, true> : sum_squares<float, true>)
                                         : (size == 2 ? sum_squares<uint16_t, false> : sum_squares<float, false>);
                return enqueue(kernel, dim3(alone ? 1 : (uint32_t)groups), kThreads, 0, s, a,
                               alone ? nullptr : (double*)workspace + before, alone ? total : nullptr,
                               accumulate ? 1 : 0);
            });
            if (e != hipSuccess || (alone && !none)) return e;
            return enqueue(sum_partials, dim3(1), kSumThreads, 0, s, (const double*)workspace, need / 8, total,
                           accumulate ? 1 : 0);
        });
    });
}

tide_status tide_clip_grads(int32_t dtype, const void* const* grads, const int64_t* elems,
                            int32_t tensors, const double* total, double max_norm,
                            void* const* out, float* norm, void* stream) {
    return guarded([&]() -> tide_status {
        TIDE_TRY(check_sizes(dtype, elems, tensors));
        if (!(max_norm >= 0.0)) return fail(TIDE_ERR_INVALID_ARG, "max_norm has to be 0 or more");
        if (tensors && !grads) return fail(TIDE_ERR_INVALID_ARG, "grads is NULL");
        const int32_t size = dtype == TIDE_DTYPE_FP32 ? 4 : 2;
        Mat rd[1], small[1];
        TIDE_TRY(matrix("total", total, 1, 1, 1, 8, &rd[0]));
        TIDE_TRY(matrix("norm", norm, norm ? 1 : 0, 1, 1, 4, &small[0]));
        TIDE_TRY(no_overlap(small, 1, rd, 1));
        std::vector<Range> read{Range{rd[0].base, rd[0].base + 8}}, written;
        read.reserve((size_t)tensors + 1);
        written.reserve((size_t)tensors + 1);
        if (norm) written.push_back(Range{small[0].base, small[0].base + 4});
        bool elsewhere = false;
        for (int32_t i = 0; i < tensors; ++i) {
            Mat a, b;
            TIDE_TRY(matrix("one of the grads", grads[i], 1, elems[i], elems[i], size, &a));
            TIDE_TRY(matrix("one of the outputs", out ? out[i] : grads[i], 1, elems[i], elems[i], size, &b));
            if (a.rows == 0) continue;
            if (a.base != b.base) {
                read.push_back(Range{a.base, a.base + (uintptr_t)a.width});
                elsewhere = true;
            }
            written.push_back(Range{b.base, b.base + (uintptr_t)b.width});
        }
        TIDE_TRY(check_ranges(written, read));
        const bool once = past_caches(elems, tensors, size);
        return on_stream(stream, [&](hipStream_t s) {
            bool first = true;
            const auto go = [&](const auto& a, int64_t groups, int64_t) {
                constexpr bool kOut = std::is_same_v<std::decay_t<decltype(a)>, Tensors<true>>;
                float* to = first ? norm : nullptr;
                first = false;
                const dim3 grid((uint32_t)groups);
                const auto kernel = once ? (size == 2 ? clip<uint16_t, true, kOut> : clip<float, true, kOut>)
                                         : (size == 2 ? clip<uint16_t, false, kOut> : clip<float, false, kOut>);
                return enqueue(kernel, grid, kThreads, 0, s, a, total, max_norm, to);
            };
            const hipError_t e = elsewhere ? each_launch<true>(grads, out, elems, tensors, size, go)
                                           : each_launch<false>(grads, nullptr, elems, tensors, size, go);
            if (e != hipSuccess || !first || !norm) return e;
            return enqueue(clip<float, false, false>, dim3(1), kThreads, 0, s, Tensors<false>{}, total, max_norm, norm);
        });
    });
}

}  // extern "C"
