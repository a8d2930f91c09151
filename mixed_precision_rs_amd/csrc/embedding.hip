// Token ids sorted by id (tide_sort_ids), rows of the embedding table
// (tide_embed_tokens) and the table's gradient (tide_embed_tokens_grad) for
// gfx950.
#include <climits>

#include "device.hpp"
#include "host.hpp"

using namespace tide;

namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kDigits = 512;           // a pass sorts by up to 9 bits of the id
constexpr int64_t kSortAlone = 4096;   // tokens that one workgroup sorts alone, in LDS
constexpr int64_t kSortChunk = 2048;   // tokens of a workgroup otherwise, while that makes at most kSortBlocks
constexpr int64_t kSortBlocks = 128;

// The least-significant-digit-first radix sort of the valid ids. Every pass is
// stable: a wave owns a contiguous run of its workgroup's chunk, so
// (workgroup, wave, step, lane) is the order of the pass before.
struct Digits {
    int passes, bits;
};
Digits digits_of(int64_t vocab) {
    int need = 1;
    while (need < 31 && ((int64_t)1 << need) < vocab) ++need;
    const int passes = (need + 8) / 9;
    return Digits{passes, (need + passes - 1) / passes};
}
int64_t sort_chunk(int64_t n) {
    int64_t c = kSortChunk;
    if (n > c * kSortBlocks) c = (n + kSortBlocks - 1) / kSortBlocks;
    return (c + kSortThreads - 1) / kSortThreads * kSortThreads;
}

// Workspace, in int32: the number of valid ids, two pairs of (id, token)
// arrays, and each workgroup's counts.
struct SortSpace {
    int32_t* valid;
    int32_t* key[2];
    int32_t* token[2];
    int32_t* counts;
};
int64_t sort_words(int64_t n) {
    return n <= kSortAlone ? 4 + n : 4 + 4 * n + ((n + sort_chunk(n) - 1) / sort_chunk(n)) * kDigits;
}
SortSpace sort_space(void* workspace, int64_t n) {
    int32_t* w = (int32_t*)workspace;
    return SortSpace{w, {w + 4, w + 4 + n}, {w + 4 + 2 * n, w + 4 + 3 * n}, w + 4 + 4 * n};
}

template <class Id>
__device__ __forceinline__ int32_t key_of(const Id* ids, int64_t i, int64_t n, int64_t vocab) {
    if (i >= n) return -1;
    const Id id = *gbl<Id>(ids + i);
    return id >= 0 && (int64_t)id < vocab ? (int32_t)id : -1;
}

// Place of this lane's digit (-1: none): the wave's next place for it, and the
// lanes below that have it too.
__device__ __forceinline__ int32_t place_digit(int32_t d, int bits, int32_t* next) {
    const int lane = threadIdx.x & 63;
    uint64_t same = __ballot(d >= 0);
    for (int b = 0; b < bits; ++b) {
        const uint64_t ones = __ballot((d >> b) & 1);
        same &= (d >> b) & 1 ? ones : ~ones;
    }
    int32_t at = -1;
    if (d >= 0) {
        const int below = __popcll(same & ((1ull << lane) - 1));
        const int32_t base = next[d];
        at = base + below;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (below == 0) next[d] = base + __popcll(same);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    return at;
}

// Exclusive scan of v[kDigits] in LDS by one wave; the sum of all.
__device__ __forceinline__ int32_t scan_digits(int32_t* v) {
    constexpr int kPer = kDigits / 64;
    const int lane = threadIdx.x & 63;
    int32_t own[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        own[i] = v[lane * kPer + i];
        sum += own[i];
    }
    int32_t inc = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t up = __shfl_up(inc, d);
        if (lane >= d) inc += up;
    }
    int32_t at = inc - sum;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        v[lane * kPer + i] = at;
        at += own[i];
    }
    return __shfl(inc, 63);
}

// All passes by one workgroup, the pairs in LDS between them.
template <class Id>
__global__ __launch_bounds__(kSortThreads) void sort_alone(const Id* ids, int n, int64_t vocab,
                                                           Digits digits, int32_t* order,
                                                           int32_t* keys, int32_t* valid) {
    constexpr int kSteps = (int)(kSortAlone / kSortThreads);
    __shared__ int32_t key_at[kSortAlone];
    __shared__ uint16_t token_at[kSortAlone];
    __shared__ int32_t wave_at[kSortWaves][kDigits];
    __shared__ int32_t total[kDigits];
    __shared__ int32_t count;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int lo = wave * kSteps * 64;
    int32_t key[kSteps], token[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        token[i] = lo + i * 64 + lane;
        key[i] = key_of(ids, token[i], n, vocab);
    }
    for (int pass = 0; pass < digits.passes; ++pass) {
        const int shift = pass * digits.bits, mask = (1 << digits.bits) - 1;
        for (int i = tid; i < kSortWaves * kDigits; i += kSortThreads) (&wave_at[0][0])[i] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
            if (key[i] >= 0) atomicAdd(&wave_at[wave][(key[i] >> shift) & mask], 1);
        __syncthreads();
        if (tid < kDigits) {
            int32_t sum = 0;
            for (int w = 0; w < kSortWaves; ++w) sum += wave_at[w][tid];
            total[tid] = sum;
        }
        __syncthreads();
        if (wave == 0) {
            const int32_t all = scan_digits(total);
            if (lane == 0) count = all;
        }
        __syncthreads();
        if (tid < kDigits) {
            int32_t at = total[tid];
            for (int w = 0; w < kSortWaves; ++w) {
                const int32_t c = wave_at[w][tid];
                wave_at[w][tid] = at;
                at += c;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int32_t at = place_digit(key[i] < 0 ? -1 : (key[i] >> shift) & mask, digits.bits, wave_at[wave]);
            if (at >= 0) {
                key_at[at] = key[i];
                token_at[at] = (uint16_t)token[i];
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int at = lo + i * 64 + lane;
            key[i] = at < count ? key_at[at] : -1;
            token[i] = at < count ? token_at[at] : 0;
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int at = lo + i * 64 + lane;
        if (key[i] >= 0) {
            *gbl_mut<int32_t>(order + at) = token[i];
            *gbl_mut<int32_t>(keys + at) = key[i];
        }
    }
    if (tid == 0) *gbl_mut<int32_t>(valid) = count;
}

// The pairs that a pass reads: the caller's ids in the first, then what the
// pass before wrote.
template <class Id>
struct FromIds {
    const Id* ids;
    int64_t n, vocab;
    __device__ int64_t count() const { return n; }
    __device__ int32_t key(int64_t i) const { return key_of(ids, i, n, vocab); }
    __device__ int32_t token(int64_t i) const { return (int32_t)i; }
};
struct FromPairs {
    const int32_t* keys;
    const int32_t* tokens;
    const int32_t* valid;
    __device__ int64_t count() const { return *gbl<int32_t>(valid); }
    __device__ int32_t key(int64_t i) const { return *gbl<int32_t>(keys + i); }
    __device__ int32_t token(int64_t i) const { return *gbl<int32_t>(tokens + i); }
};

// Counts of a pass's digits in one workgroup's chunk. (Added up by the pass before
// as it places its pairs, in global memory, they would save a launch of 4.6 us, and
// cost 20 where half of the ids share a digit.)
template <class From>
__global__ __launch_bounds__(kSortThreads) void digit_count(From from, int64_t chunk, int shift,
                                                            int bits, int32_t* counts) {
    __shared__ int32_t hist[kDigits];
    const int64_t n = from.count(), lo = blockIdx.x * chunk;
    if (threadIdx.x < kDigits) hist[threadIdx.x] = 0;
    __syncthreads();
    for (int64_t i = lo + threadIdx.x; i < lo + chunk && i < n; i += kSortThreads) {
        const int32_t k = from.key(i);
        if (k >= 0) atomicAdd(&hist[(k >> shift) & ((1 << bits) - 1)], 1);
    }
    __syncthreads();
    if (threadIdx.x < kDigits)
        *gbl_mut<int32_t>(counts + (int64_t)blockIdx.x * kDigits + threadIdx.x) = hist[threadIdx.x];
}

// One pass. A wave's run of two steps (chunks of kSortChunk) stays in registers
// between counting and placing.
template <class From, bool kTwo>
__global__ __launch_bounds__(kSortThreads) void digit_place(From from, int64_t chunk, int shift,
                                                            int bits, const int32_t* counts,
                                                            int32_t* keys, int32_t* tokens,
                                                            int32_t* valid) {
    __shared__ int32_t wave_at[kSortWaves][kDigits];
    __shared__ int32_t total[kDigits], before[kDigits];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int nb = gridDim.x, me = blockIdx.x, mask = (1 << bits) - 1;
    const int64_t n = from.count();
    const int64_t run = chunk / kSortWaves, lo = me * chunk + wave * run;      // a multiple of 64
    int32_t held[2] = {-1, -1}, whose[2] = {};
    if (kTwo) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (lo + i * 64 + lane < n) {
                held[i] = from.key(lo + i * 64 + lane);
                whose[i] = from.token(lo + i * 64 + lane);
            }
    }
    for (int i = tid; i < kSortWaves * kDigits; i += kSortThreads) (&wave_at[0][0])[i] = 0;
    if (tid < kDigits) {
        int32_t all = 0, less = 0;
#pragma unroll 8
        for (int b = 0; b < nb; ++b) {
            const int32_t c = *gbl<int32_t>(counts + (int64_t)b * kDigits + tid);
            all += c;
            less += b < me ? c : 0;
        }
        total[tid] = all;
        before[tid] = less;
    }
    __syncthreads();
    if (kTwo) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (held[i] >= 0) atomicAdd(&wave_at[wave][(held[i] >> shift) & mask], 1);
    } else {
        for (int64_t i = lo + lane; i < lo + run && i < n; i += 64) {
            const int32_t k = from.key(i);
            if (k >= 0) atomicAdd(&wave_at[wave][(k >> shift) & mask], 1);
        }
    }
    if (wave == 0) {
        const int32_t all = scan_digits(total);
        if (me == 0 && lane == 0 && valid) *gbl_mut<int32_t>(valid) = all;
    }
    __syncthreads();
    if (tid < kDigits) {
        int32_t at = total[tid] + before[tid], c[kSortWaves];
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) c[w] = wave_at[w][tid];
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            wave_at[w][tid] = at;
            at += c[w];
        }
    }
    __syncthreads();
    const auto place = [&](int32_t k, int32_t token) {
        const int32_t at = place_digit(k < 0 ? -1 : (k >> shift) & mask, bits, wave_at[wave]);
        if (at < 0) return;
        *gbl_mut<int32_t>(keys + at) = k;
        *gbl_mut<int32_t>(tokens + at) = token;
    };
    if (kTwo) {
        place(held[0], whose[0]);
        place(held[1], whose[1]);
    } else {
        for (int64_t i0 = lo; i0 < lo + run && i0 < n; i0 += 64) {
            const int64_t i = i0 + lane;
            place(i < n ? from.key(i) : -1, i < n ? from.token(i) : 0);
        }
    }
}

// offsets[v]: the first place whose id is not below v, for v up to vocab.
__global__ __launch_bounds__(256) void find_offsets(const int32_t* keys, const int32_t* valid,
                                                    int64_t vocab, int32_t* offsets) {
    const int32_t n = *gbl<int32_t>(valid);
    for (int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x; v <= vocab; v += (int64_t)gridDim.x * 256) {
        int32_t lo = 0, hi = n;
        while (lo < hi) {
            const int32_t mid = lo + (hi - lo) / 2;
            if (*gbl<int32_t>(keys + mid) < v) lo = mid + 1;
            else hi = mid;
        }
        *gbl_mut<int32_t>(offsets + v) = lo;
    }
}

template <class From>
hipError_t sort_pass(const From& from, int64_t n, int shift, int bits, int32_t* counts, int32_t* keys,
                     int32_t* tokens, int32_t* valid, hipStream_t s) {
    const int64_t chunk = sort_chunk(n);
    const dim3 grid((uint32_t)((n + chunk - 1) / chunk));
    const hipError_t e = enqueue(digit_count<From>, grid, kSortThreads, 0, s, from, chunk, shift, bits, counts);
    if (e != hipSuccess) return e;
    const auto place = chunk == 2 * kSortThreads ? digit_place<From, true> : digit_place<From, false>;
    return enqueue(place, grid, kSortThreads, 0, s, from, chunk, shift, bits, (const int32_t*)counts, keys, tokens,
                   valid);
}

template <class Id>
hipError_t launch_sort(const Id* ids, int64_t n, int64_t vocab, int32_t* offsets, int32_t* order,
                       void* workspace, hipStream_t s) {
    const Digits d = digits_of(vocab);
    const SortSpace w = sort_space(workspace, n);
    const int32_t* sorted = w.key[0];
    if (n <= kSortAlone) {
        const hipError_t e = enqueue(sort_alone<Id>, dim3(1), kSortThreads, 0, s, ids, (int)n, vocab, d, order,
                                     w.key[0], w.valid);
        if (e != hipSuccess) return e;
    } else {
        for (int p = 0; p < d.passes; ++p) {
            int32_t* tokens = p == d.passes - 1 ? order : w.token[p & 1];
            const hipError_t e =
                p == 0 ? sort_pass(FromIds<Id>{ids, n, vocab}, n, 0, d.bits, w.counts, w.key[0], tokens, w.valid, s)
                       : sort_pass(FromPairs{w.key[(p - 1) & 1], w.token[(p - 1) & 1], w.valid}, n, p * d.bits,
                                   d.bits, w.counts, w.key[p & 1], tokens, (int32_t*)nullptr, s);
            if (e != hipSuccess) return e;
            sorted = w.key[p & 1];
        }
    }
    const int64_t groups = (vocab + 256) / 256;
    return enqueue(find_offsets, dim3((uint32_t)(groups < (1 << 20) ? groups : (1 << 20))), 256, 0, s, sorted,
                   (const int32_t*)w.valid, vocab, offsets);
}

// First element of vector u of a row: the last vector ends at the row's end.
template <int V>
__device__ __forceinline__ int64_t at_vector(int64_t u, int64_t width) {
    return u > 0 && u * V > width - V ? width - V : u * V;
}

template <class T, class Id>
__global__ __launch_bounds__(kRowThreads) void embed_rows(const Id* ids, int64_t tokens,
                                                          const T* table, int64_t table_stride,
                                                          int64_t vocab, int64_t width, float scale,
                                                          T* out, int64_t out_stride, int lane_log2) {
    constexpr int V = kVecOf<T>;
    const int lanes = 1 << lane_log2;
    const int64_t units = (width + V - 1) / V;
    for (int64_t t = (int64_t)blockIdx.x * (kRowThreads >> lane_log2) + (threadIdx.x >> lane_log2);
         t < tokens; t += (int64_t)gridDim.x * (kRowThreads >> lane_log2)) {
        const Id id = *gbl<Id>(ids + t);
        const bool there = id >= 0 && (int64_t)id < vocab;
        for (int64_t u = (int64_t)blockIdx.y * lanes + (threadIdx.x & (lanes - 1)); u < units;
             u += (int64_t)gridDim.y * lanes) {
            const int64_t at = at_vector<V>(u, width);
            const int some = width < V ? (int)width : V;
            u32x4 raw{};
            if (there) raw = load_row(table + (int64_t)id * table_stride + at, some);
            if (scale != 1.0f && there) {
                float v[V];
                widen(raw, v);
#pragma unroll
                for (int c = 0; c < V; ++c) v[c] *= scale;
                raw = narrow(v);
            }
            store_row(out + t * out_stride + at, some, raw);
        }
    }
}

// ---- The table's gradient --------------------------------------------------------
//
// A row of the table with up to `chunk` tokens is summed by its own lanes. One with
// more (the words that a text is full of) would keep them busy long after the
// others: its tokens are summed chunk by chunk, at multiples of `chunk` places of
// the order, by the waves of a kernel before, and its lanes add up those sums.
// A chunk of places can hold pieces of two such rows: one that it begins inside
// (or with), and one that begins in it and goes on behind it. row_of says whose
// pieces they are, -1 where there is none.
struct Sorted {
    const int32_t* offsets;
    const int32_t* order;
    int64_t tokens, vocab;
};
struct Pieces {
    float* sums;           // [chunk of places][2][padded]
    int32_t* row_of;       // [chunk of places][2]
    int64_t padded;        // elements of a sum
    int32_t chunk;
};
// Chunks: the row of the most tokens then has at most 256 sums up to 16384
// tokens and 1024 up to 131072.
int64_t chunk_of(int64_t tokens) { return tokens <= 16384 ? 64 : tokens <= 131072 ? 128 : 512; }
int64_t chunks_of(int64_t tokens) {
    const int64_t c = chunk_of(tokens);
    return tokens <= c ? 0 : (tokens + c - 1) / c;
}
int64_t padded_width(int64_t width) { return (width + 7) / 8 * 8; }

__device__ __forceinline__ void row_range(const Sorted& s, int64_t v, int64_t& lo, int64_t& hi) {
    lo = *gbl<int32_t>(s.offsets + v);
    hi = *gbl<int32_t>(s.offsets + v + 1);
    lo = lo < 0 ? 0 : lo;
    hi = hi > s.tokens ? s.tokens : hi;
}

// acc += the vectors at column `at` of the tokens order[lo .. hi), in order, KU
// loads in flight. With kWave all lanes of the wave have the same lo and hi (some
// may have no column: some <= 0): 64 entries of the order come by one load, a lane
// each, so that no load of a token waits for another one.
template <class T, int V, bool kWave, int KU>
__device__ __forceinline__ void add_tokens(const Sorted& s, const T* dout, int64_t stride, int64_t lo, int64_t hi,
                                           int64_t at, int some, float (&acc)[V]) {
    constexpr int kRun = kWave ? 64 : KU;
    for (int64_t i0 = lo; i0 < hi; i0 += kRun) {
        const int n = hi - i0 < kRun ? (int)(hi - i0) : kRun;
        uint32_t mine = ~0u;
        if (kWave && (int)(threadIdx.x & 63) < n) mine = *gbl<uint32_t>(s.order + i0 + (threadIdx.x & 63));
        for (int i = 0; i < n; i += KU) {
            u32x4 raw[KU];
#pragma unroll
            for (int j = 0; j < KU; ++j) {
                uint32_t t = ~0u;
                if (kWave) t = __builtin_amdgcn_readlane(mine, (i + j) & 63);
                else if (i + j < n) t = *gbl<uint32_t>(s.order + i0 + i + j);
                raw[j] = u32x4{};
                if (i + j < n && t < s.tokens && some > 0) raw[j] = load_row<true>(dout + (int64_t)t * stride + at, some);
            }
#pragma unroll
            for (int j = 0; j < KU; ++j) {
                float d[V];
                widen(raw[j], d);
#pragma unroll
                for (int c = 0; c < V; ++c) acc[c] += d[c];
            }
        }
    }
}

// The row that place p of the order belongs to, by all 64 lanes: the last one
// whose first place is not behind p.
__device__ __forceinline__ int64_t row_at(const Sorted& s, int64_t p) {
    int64_t lo = 0, hi = s.vocab;
    while (hi - lo > 1) {
        const int64_t step = (hi - lo + 63) / 64, i = lo + ((threadIdx.x & 63) + 1) * step;
        const uint64_t before = __ballot(i < hi && *gbl<int32_t>(s.offsets + (i < hi ? i : lo)) <= p);
        lo += __popcll(before) * step;
        hi = lo + step < hi ? lo + step : hi;
    }
    return lo;
}

// A wave sums one of a chunk's two pieces in 64 vectors of columns.
template <class T>
__global__ __launch_bounds__(kRowThreads) void sum_pieces(Sorted s, Pieces to, const T* dout, int64_t stride,
                                                          int64_t width, int64_t waves, int tiles) {
    constexpr int V = kVecOf<T>;
    const int64_t w = (int64_t)blockIdx.x * (kRowThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (w >= waves) return;
    const int64_t piece = w / tiles, u = (w - piece * tiles) * 64 + (threadIdx.x & 63);
    const int64_t first = (piece >> 1) * to.chunk, end = first + to.chunk < s.tokens ? first + to.chunk : s.tokens;
    const int64_t place = piece & 1 ? end - 1 : first;
    const int64_t v = row_at(s, place);
    int64_t lo, hi;
    row_range(s, v, lo, hi);
    const bool mine = hi - lo > to.chunk && lo <= place && place < hi && (!(piece & 1) || lo > first);
    if (u == 0) *gbl_mut<int32_t>(to.row_of + piece) = mine ? (int32_t)v : -1;
    if (!mine) return;
    const int64_t at = u > 0 && u * V > width - V ? width - V : u * V;
    float acc[V] = {};
    add_tokens<T, V, true, 16>(s, dout, stride, lo > first ? lo : first, hi < end ? hi : end, at,
                           u * V >= width ? 0 : width < V ? (int)width : V, acc);
    if (u * V >= width) return;
    float* sum = to.sums + piece * to.padded + u * V;
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
        *gbl_mut<u32x4>(sum + 4 * i) = u32x4{__float_as_uint(acc[4 * i]), __float_as_uint(acc[4 * i + 1]),
                                             __float_as_uint(acc[4 * i + 2]), __float_as_uint(acc[4 * i + 3])};
}

// acc += row v's pieces; false where they are not all there (offsets that do not
// rise).
template <int V>
__device__ __forceinline__ bool add_pieces(const Pieces& from, int64_t v, int64_t lo, int64_t hi, int64_t u,
                                           float (&acc)[V]) {
    constexpr int KU = 4;
    const int64_t b0 = lo / from.chunk, b1 = (hi - 1) / from.chunk;
    bool there = true;
    for (int64_t b = b0; b <= b1; ++b)
        there = there && *gbl<int32_t>(from.row_of + 2 * b + (lo <= b * from.chunk ? 0 : 1)) == v;
    if (!there) return false;
    for (int64_t b = b0; b <= b1; b += KU) {
        u32x4 raw[KU][V / 4];
#pragma unroll
        for (int j = 0; j < KU; ++j)
#pragma unroll
            for (int i = 0; i < V / 4; ++i) {
                raw[j][i] = u32x4{};
                if (b + j <= b1)
                    raw[j][i] = *gbl<u32x4>(from.sums + (2 * (b + j) + (lo <= (b + j) * from.chunk ? 0 : 1)) * from.padded +
                                            u * V + 4 * i);
            }
#pragma unroll
        for (int j = 0; j < KU; ++j)
#pragma unroll
            for (int c = 0; c < V; ++c) acc[c] += __uint_as_float(raw[j][c / 4][c % 4]);
    }
    return true;
}

// Vector u of row v of the gradient (of a wave's or a group of lanes' 64 or fewer;
// some <= 0: this lane has none).
template <class T, bool kWave>
__device__ __forceinline__ void grad_vector(const Sorted& s, const Pieces& from, const T* dout, int64_t stride,
                                            int64_t width, float scale, T* row, int accumulate, int64_t v,
                                            int64_t lo, int64_t hi, int64_t u, int64_t units) {
    constexpr int V = kVecOf<T>;
    // The last vector ends at the row's end; `seen` of its elements are the one's before.
    const int64_t at = u > 0 && u * V > width - V ? width - V : u * V;
    const int some = u >= units ? 0 : width < V ? (int)width : V, seen = (int)(u * V - at);
    float acc[V] = {};
    if (lo < hi) {
        const bool done = hi - lo > from.chunk && add_pieces<V>(from, v, lo, hi, u < units ? u : 0, acc);
        if (!done) add_tokens<T, V, kWave, 8>(s, dout, stride, lo, hi, at, some, acc);
#pragma unroll
        for (int c = 0; c < V; ++c) acc[c] *= scale;
    }
    if (some <= 0) return;
    if (!accumulate) {
        store_row(row + at, some, narrow(acc));
        return;
    }
    float old[V];
    widen(load_row(row + at, some), old);
#pragma unroll
    for (int c = 0; c < V; ++c) acc[c] += old[c];
    const u32x4 out = narrow(acc);
    if (seen == 0) {
        store_row(row + at, some, out);
    } else {
#pragma unroll
        for (int c = 1; c < V; ++c) {
            if (c < seen) continue;
            if constexpr (sizeof(T) == 2) *gbl_mut<uint16_t>(row + at + c) = (uint16_t)(out[c / 2] >> (16 * (c & 1)));
            else *gbl_mut<uint32_t>(row + at + c) = out[c];
        }
    }
}

// Narrow rows: 2^lane_log2 lanes each.
template <class T>
__global__ __launch_bounds__(kRowThreads) void table_grad_narrow(Sorted s, Pieces from, const T* dout, int64_t stride,
                                                                 int64_t width, float scale, T* grad,
                                                                 int64_t grad_stride, int accumulate, int lane_log2) {
    constexpr int V = kVecOf<T>;
    const int64_t units = (width + V - 1) / V, per = kRowThreads >> lane_log2;
    const int lane = threadIdx.x & ((1 << lane_log2) - 1);
    for (int64_t v = (int64_t)blockIdx.x * per + (threadIdx.x >> lane_log2); v < s.vocab; v += (int64_t)gridDim.x * per) {
        int64_t lo, hi;
        row_range(s, v, lo, hi);
        if (lane >= units || (accumulate && lo >= hi)) continue;
        grad_vector<T, false>(s, from, dout, stride, width, scale, grad + v * grad_stride, accumulate, v, lo, hi, lane, units);
    }
}

// Wide rows: a wave takes 64 vectors of one row, then those some waves further on.
// Most rows of a large table have no token and are stores alone (131072 x 2048 in
// 85 us, the rate of a fill); those that have wait for their loads, and stand
// together where the frequent words do. Left so they are done in 28 us before the
// others (16384 tokens: 113 us); with rows of distant stretches of the table taken
// in turn, loads and stores mix, and the whole takes 142-181. 2048 workgroups that
// stay take 145, and several rows a wave one behind the other 197 (4) to 472 (16):
// rows that are used much then wait for each other.
constexpr int64_t kGradGroups = 32768;
template <class T>
__global__ __launch_bounds__(kRowThreads) void table_grad(Sorted s, Pieces from, const T* dout, int64_t stride,
                                                          int64_t width, float scale, T* grad, int64_t grad_stride,
                                                          int accumulate, int64_t tiles, int64_t step_rows,
                                                          int64_t step_tiles) {
    constexpr int V = kVecOf<T>;
    const int64_t units = (width + V - 1) / V;
    const int64_t w = (int64_t)blockIdx.x * (kRowThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int64_t v = w / tiles, tile = w - v * tiles;
    while (v < s.vocab) {
        const int64_t u = tile * 64 + (threadIdx.x & 63);
        T* row = grad + v * grad_stride;
        int64_t lo, hi;
        row_range(s, v, lo, hi);
        if (lo < hi)
            grad_vector<T, true>(s, from, dout, stride, width, scale, row, accumulate, v, lo, hi, u, units);
        else if (!accumulate && u < units)
            store_row(row + (u > 0 && u * V > width - V ? width - V : u * V), width < V ? (int)width : V, u32x4{});
        v += step_rows;
        tile += step_tiles;
        if (tile >= tiles) {
            tile -= tiles;
            ++v;
        }
    }
}

tide_status check_ids(int32_t id_bytes, int64_t tokens, int64_t vocab) {
    if (id_bytes != 4 && id_bytes != 8)
        return fail(TIDE_ERR_INVALID_ARG, "ids have 4 or 8 bytes, not %d", id_bytes);
    if (tokens < 0 || vocab < 0) return fail(TIDE_ERR_INVALID_ARG, "need tokens and vocab >= 0");
    return TIDE_OK;
}
tide_status check_sorted(int64_t tokens, int64_t vocab) {
    if (tokens < 0 || vocab < 0) return fail(TIDE_ERR_INVALID_ARG, "need tokens and vocab >= 0");
    if (tokens > INT32_MAX || vocab >= INT32_MAX)
        return fail(TIDE_ERR_UNSUPPORTED, "tokens and vocab must be below 2^31 - 1");
    return TIDE_OK;
}
tide_status check_dtype(int32_t dtype) {
    if (dtype != TIDE_DTYPE_BF16 && dtype != TIDE_DTYPE_FP32)
        return fail(TIDE_ERR_INVALID_ARG, "dtype %d is not BF16 (0) or FP32 (1)", dtype);
    return TIDE_OK;
}

}  // namespace

extern "C" {

tide_status tide_sort_ids_workspace(int64_t tokens, int64_t vocab, int64_t* bytes) {
    return guarded([&]() -> tide_status {
        if (!bytes) return fail(TIDE_ERR_INVALID_ARG, "bytes is NULL");
        TIDE_TRY(check_sorted(tokens, vocab));
        *bytes = sort_words(tokens) * 4;
        return TIDE_OK;
    });
}

tide_status tide_sort_ids(const void* ids, int32_t id_bytes, int64_t tokens, int64_t vocab,
                          int32_t* offsets, int32_t* order, void* workspace,
                          int64_t workspace_bytes, void* stream) {
    return guarded([&]() -> tide_status {
        int64_t need = 0;
        TIDE_TRY(tide_sort_ids_workspace(tokens, vocab, &need));
        TIDE_TRY(check_ids(id_bytes, tokens, vocab));
        if (!workspace || workspace_bytes < need)
            return fail(TIDE_ERR_INVALID_ARG, "workspace holds %lld bytes, %lld needed",
                        (long long)(workspace ? workspace_bytes : 0), (long long)need);
        Mat in, wr[3];
        TIDE_TRY(matrix("ids", ids, 1, tokens, tokens, id_bytes, &in));
        TIDE_TRY(matrix("offsets", offsets, 1, vocab + 1, vocab + 1, 4, &wr[0]));
        TIDE_TRY(matrix("order", order, 1, tokens, tokens, 4, &wr[1]));
        TIDE_TRY(matrix("workspace", workspace, 1, need / 4, need / 4, 4, &wr[2]));
        TIDE_TRY(no_overlap(wr, 3, &in, 1));
        return on_stream(stream, [&](hipStream_t s) {
            return id_bytes == 4 ? launch_sort((const int32_t*)ids, tokens, vocab, offsets, order, workspace, s)
                                 : launch_sort((const int64_t*)ids, tokens, vocab, offsets, order, workspace, s);
        });
    });
}

tide_status tide_embed_tokens(int32_t dtype, const void* ids, int32_t id_bytes, int64_t tokens,
                              const void* table, int64_t table_stride, int64_t vocab,
                              int64_t width, float scale, void* out, int64_t out_stride,
                              void* stream) {
    return guarded([&]() -> tide_status {
        TIDE_TRY(check_dtype(dtype));
        TIDE_TRY(check_ids(id_bytes, tokens, vocab));
        const int32_t size = dtype == TIDE_DTYPE_FP32 ? 4 : 2;
        Mat rd[2], wr;
        TIDE_TRY(matrix("ids", ids, width ? 1 : 0, tokens, tokens, id_bytes, &rd[0]));
        TIDE_TRY(matrix("table", table, vocab, width, table_stride, size, &rd[1]));
        TIDE_TRY(matrix("out", out, tokens, width, out_stride, size, &wr));
        TIDE_TRY(no_overlap(&wr, 1, rd, 2));
        if (tokens == 0 || width == 0) return TIDE_OK;
        return on_stream(stream, [&](hipStream_t s) {
            const RowGrid g = row_grid(tokens, (width * size + 15) / 16);
            const auto go = [&](auto type, auto id) {
                using T = decltype(type);
                using Id = decltype(id);
                return enqueue(embed_rows<T, Id>, g.grid, kRowThreads, 0, s, (const Id*)ids, tokens, (const T*)table,
                               table_stride, vocab, width, scale, (T*)out, out_stride, g.lane_log2);
            };
            if (size == 2) return id_bytes == 4 ? go(uint16_t{}, int32_t{}) : go(uint16_t{}, int64_t{});
            return id_bytes == 4 ? go(float{}, int32_t{}) : go(float{}, int64_t{});
        });
    });
}

tide_status tide_embed_tokens_grad_workspace(int64_t tokens, int64_t width, int64_t* bytes) {
    return guarded([&]() -> tide_status {
        if (!bytes) return fail(TIDE_ERR_INVALID_ARG, "bytes is NULL");
        TIDE_TRY(check_sorted(tokens, 0));
        if (width < 0) return fail(TIDE_ERR_INVALID_ARG, "negative width");
        int64_t each;
        const int64_t n = chunks_of(tokens);
        *bytes = 0;
        if (n && width && (__builtin_mul_overflow(n * 2, (width + 7) / 8 * 32, &each) ||
                           __builtin_add_overflow(each, n * 8, bytes)))
            return fail(TIDE_ERR_OVERFLOW, "the workspace's size overflows int64");
        return TIDE_OK;
    });
}

tide_status tide_embed_tokens_grad(int32_t dtype, const void* dout, int64_t dout_stride,
                                   int64_t tokens, int64_t width, const int32_t* offsets,
                                   const int32_t* order, int64_t vocab, float scale, void* grad,
                                   int64_t grad_stride, int32_t accumulate, void* workspace,
                                   int64_t workspace_bytes, void* stream) {
    return guarded([&]() -> tide_status {
        TIDE_TRY(check_dtype(dtype));
        TIDE_TRY(check_sorted(tokens, vocab));
        int64_t need = 0;
        TIDE_TRY(tide_embed_tokens_grad_workspace(tokens, width, &need));
        if (need > 0 && (!workspace || workspace_bytes < need))
            return fail(TIDE_ERR_INVALID_ARG, "workspace holds %lld bytes, %lld needed",
                        (long long)(workspace ? workspace_bytes : 0), (long long)need);
        const int32_t size = dtype == TIDE_DTYPE_FP32 ? 4 : 2;
        Mat rd[3], wr[2];
        TIDE_TRY(matrix("dout", dout, tokens, width, dout_stride, size, &rd[0]));
        TIDE_TRY(matrix("offsets", offsets, width && vocab ? 1 : 0, vocab + 1, vocab + 1, 4, &rd[1]));
        TIDE_TRY(matrix("order", order, width && vocab ? 1 : 0, tokens, tokens, 4, &rd[2]));
        TIDE_TRY(matrix("grad", grad, vocab, width, grad_stride, size, &wr[0]));
        TIDE_TRY(matrix("workspace", workspace, 1, need / 4, need / 4, 4, &wr[1]));
        if (need > 0 && (wr[1].base & 15))
            return fail(TIDE_ERR_ALIGNMENT, "workspace is not 16-byte aligned");
        TIDE_TRY(no_overlap(wr, 2, rd, 3));
        if (vocab == 0 || width == 0) return TIDE_OK;
        return on_stream(stream, [&](hipStream_t s) {
            const int64_t units = (width * size + 15) / 16, padded = padded_width(width), n = need ? chunks_of(tokens) : 0;
            const Sorted sorted{offsets, order, tokens, vocab};
            const Pieces pieces{(float*)workspace, (int32_t*)((float*)workspace + 2 * n * padded), padded,
                                (int32_t)chunk_of(tokens)};
            const RowGrid g = row_grid(vocab, units < 64 ? units : 64);
            const auto go = [&](auto type) {
                using T = decltype(type);
                if (n) {
                    const int64_t tiles = (units + 63) / 64, waves = 2 * n * tiles;
                    const hipError_t e = enqueue(sum_pieces<T>, dim3((uint32_t)((waves + 3) / 4)), kRowThreads, 0, s,
                                                 sorted, pieces, (const T*)dout, dout_stride, width, waves, (int)tiles);
                    if (e != hipSuccess) return e;
                }
                if (units <= 32)
                    return enqueue(table_grad_narrow<T>, dim3(g.grid.x), kRowThreads, 0, s, sorted, pieces,
                                   (const T*)dout, dout_stride, width, scale, (T*)grad, grad_stride, accumulate ? 1 : 0,
                                   g.lane_log2);
                const int64_t tiles = (units + 63) / 64, all = (vocab * tiles + 3) / 4;
                const int64_t groups = all < kGradGroups ? all : kGradGroups, waves = 4 * groups;
                return enqueue(table_grad<T>, dim3((uint32_t)groups), kRowThreads, 0, s, sorted, pieces, (const T*)dout,
                               dout_stride, width, scale, (T*)grad, grad_stride, accumulate ? 1 : 0, tiles,
                               waves / tiles, waves % tiles);
            };
            return size == 2 ? go(uint16_t{}) : go(float{});
        });
    });
}

}  // extern "C"
