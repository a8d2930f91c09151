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

// The least-significant-digit-first radix sort of the valid ids: 16384 tokens in a
// vocabulary of 131072 take two passes of 4.7 + 6 us (count, place) and 5.7 for the
// offsets, each a launch's latency more than its work; 4096 in one workgroup 12.7 +
// 5, which 4097 exceed. Every pass is stable: a wave owns a contiguous run of its workgroup's chunk, so
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

// First element of vector u of a row: the last vector ends at the row's end (where
// the row has one at all).
template <int V>
__device__ __forceinline__ int64_t at_vector(int64_t u, int64_t width) {
    return u > 0 && u * V > width - V ? width - V : u * V;
}

// A copy of rows, scaled on the way. 16384 tokens of 8192 bf16 write 268 MB: 86 us where
// 12900 rows are read for them, 58 where ids are as unevenly used as words are (5400
// rows); 16384 of 2048 21 and 16 us, 33 of 2048 2.4.
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
// First the tokens: the places of the order are cut into chunks, and a wave adds up
// the tokens of a chunk one behind the other, in 64 vectors of columns. Where a row
// of the table ends it goes out, unless it began before the chunk or goes on behind
// it: those sums (of a frequent word, many) are left in the workspace. Then the
// table: rows without tokens become zeros, rows whose sums were left are joined.
// A kernel that reads and then one that writes: with the tokens added up among the
// waves that clear (most of a large table) 16384 tokens in 131072 x 2048 took 126 us,
// mixed through the whole of it 156-195, and so 30 and 74.
//
// Offsets that do not come from a sort may leave rows that no chunk finds whole:
// owner says for each place whether the row that begins there was written, row_of
// whose sums a chunk has left, and a row that neither names is added up by its own
// lanes.
struct Sorted {
    const int32_t* offsets;
    const int32_t* order;
    int64_t tokens, vocab;
};
struct Chunks {
    float* sums;           // [chunk][2][padded]: of a row that begins before (or with) the chunk, of one behind
    int32_t* row_of;       // [chunk][2]; -1: none
    int32_t* owner;        // [place]; -1: none
    int64_t padded;        // elements of a sum
    int32_t size;          // places of a chunk; 0: no chunks
};
template <class T>
struct Grad {
    T* data;
    int64_t stride, width;
    float scale;
    int32_t accumulate;
};
// Places of a chunk. Small ones keep the GPU busy; but a row that has all the tokens
// then has as many sums: up to kJoinTokens one wave joins them (512 at most, in 97 us),
// above join_left does, 7-25 us more whatever it finds. us of the calls on a table of
// 131072 x 2048 bf16, for even ids, ids as unevenly used as words, and one id:
//   tokens   chunks of 16   of 32         of 64         of 64, join_left  of 256, join_left
//     4096    95 100  98    106 106  98   121 121 105   124 124 110
//     4097    98 100  97    107 107  99   120 120 105   123 124 111
//     8000   102 102 142    107 105 101   121 120 105   124 124 114
//    16384   101 112 240    102 112 154   111 120 108   117 125 116
//    16385   104 113 243    102 111 154   109 120 108   115 125 118
//    32768   126 121 444    124 123 251   123 130 163   133 139 131
//   100000   211 195 1295   214 180 701   221 188 400   245 213 206
//     2^20                                              1304 1244 1247    1124 1016 899
//     2^21                                              2531 2392 2657    2027 1869 1709
// The rule bounds the worst row at the price of the others, which pay 8 us for it behind
// 4096 tokens and 13 behind 16384; its last border could stand further in.
int32_t chunk_of(int64_t tokens) { return tokens <= 4096 ? 16 : tokens <= 16384 ? 32 : tokens <= 1 << 20 ? 64 : 256; }
constexpr int64_t kJoinTokens = 16384;
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

// Vector u of row v of the gradient from its sum; old is what the row holds there
// (when it is added to).
template <class T>
__device__ __forceinline__ void put_vector(const Grad<T>& g, int64_t v, int64_t u, const float (&sum)[kVecOf<T>],
                                           u32x4 old) {
    constexpr int V = kVecOf<T>;
    if (u * V >= g.width) return;
    const int64_t at = at_vector<V>(u, g.width);
    const int some = g.width < V ? (int)g.width : V, seen = (int)(u * V - at);
    T* to = g.data + v * g.stride + at;
    float r[V];
#pragma unroll
    for (int c = 0; c < V; ++c) r[c] = sum[c] * g.scale;
    if (!g.accumulate) {
        store_row(to, some, narrow(r));
        return;
    }
    float before[V];
    widen(old, before);
#pragma unroll
    for (int c = 0; c < V; ++c) r[c] += before[c];
    const u32x4 out = narrow(r);
    if (seen == 0) {
        store_row(to, some, out);
        return;
    }
    // The first `seen` elements are those of the vector before, which adds to them.
#pragma unroll
    for (int c = 1; c < V; ++c) {
        if (c < seen) continue;
        if constexpr (sizeof(T) == 2) *gbl_mut<uint16_t>(to + c) = (uint16_t)(out[c / 2] >> (16 * (c & 1)));
        else *gbl_mut<uint32_t>(to + c) = out[c];
    }
}
template <class T>
__device__ __forceinline__ u32x4 old_vector(const Grad<T>& g, int64_t v, int64_t u) {
    constexpr int V = kVecOf<T>;
    if (!g.accumulate || u * V >= g.width) return u32x4{};
    return load_row(g.data + v * g.stride + at_vector<V>(u, g.width), g.width < V ? (int)g.width : V);
}

// The rows that two places of the order belong to, by all 64 lanes: the last one
// whose first place is not behind. Both are looked for at once.
__device__ __forceinline__ void rows_at(const Sorted& s, int64_t p0, int64_t p1, int64_t& r0, int64_t& r1) {
    int64_t end0 = s.vocab, end1 = s.vocab;
    const int64_t lane = (threadIdx.x & 63) + 1;
    r0 = r1 = 0;
    while (end0 - r0 > 1 || end1 - r1 > 1) {
        const int64_t step0 = (end0 - r0 + 63) / 64, step1 = (end1 - r1 + 63) / 64;
        const int64_t i0 = r0 + lane * step0, i1 = r1 + lane * step1;
        const int32_t o0 = *gbl<int32_t>(s.offsets + (i0 < end0 ? i0 : r0)), o1 = *gbl<int32_t>(s.offsets + (i1 < end1 ? i1 : r1));
        r0 += __popcll(__ballot(i0 < end0 && o0 <= p0)) * step0;
        r1 += __popcll(__ballot(i1 < end1 && o1 <= p1)) * step1;
        end0 = r0 + step0 < end0 ? r0 + step0 : end0;
        end1 = r1 + step1 < end1 ? r1 + step1 : end1;
    }
}

template <class T, bool kAdd>
__global__ __launch_bounds__(kRowThreads) void sum_chunks(Sorted s, Chunks to, const T* dout, int64_t stride,
                                                          Grad<T> grad, int64_t waves, int tiles) {
    constexpr int V = kVecOf<T>, KU = kAdd ? 8 : 16;
    const int lane = threadIdx.x & 63;
    const int64_t w = (int64_t)blockIdx.x * (kRowThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (w >= waves) return;
    const int64_t b = w / tiles, u = (w - b * tiles) * 64 + lane;
    const bool scribe = w == b * tiles;            // the wave that keeps the books of this chunk
    const int64_t first = b * to.size, end = first + to.size < s.tokens ? first + to.size : s.tokens;
    const int64_t at = at_vector<V>(u, grad.width);
    const int some = u * V >= grad.width ? 0 : grad.width < V ? (int)grad.width : V;
    int32_t left[2] = {-1, -1};
    // The row in hand: its places, those taken so far, and their sum.
    int32_t v = -1;
    int64_t lo = 0, hi = 0, from = 0;
    float acc[V];
    const auto finish = [&](int64_t place, u32x4 old) {
        if (v < 0) return;
        const int64_t begin = lo > first ? lo : first, stop = hi < end ? hi : end;
        const bool whole = from == begin && place == stop, inside = lo >= first && hi <= end;
        if (scribe && lane == 0 && from == lo) *gbl_mut<int32_t>(to.owner + lo) = whole && inside ? v : -1;
        if (!whole) return;
        if (inside) {
            put_vector<T>(grad, v, u, acc, old);
            return;
        }
        const int k = lo <= first ? 0 : 1;
        left[0] = k ? left[0] : v;
        left[1] = k ? v : left[1];
        if (some == 0) return;
        float* sum = to.sums + (2 * b + k) * to.padded + u * V;
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
            *gbl_mut<u32x4>(sum + 4 * i) = u32x4{__float_as_uint(acc[4 * i]), __float_as_uint(acc[4 * i + 1]),
                                                 __float_as_uint(acc[4 * i + 2]), __float_as_uint(acc[4 * i + 3])};
    };
    u32x4 old_of_last{};
    for (int64_t base = first; base < end; base += 64) {
        const int n = end - base < 64 ? (int)(end - base) : 64;
        // Lane i: the row of place base + i, its places, and the token there.
        const int64_t place = base + (lane < n ? lane : n - 1);
        uint32_t token = *gbl<uint32_t>(s.order + place);
        int64_t r0, r1;
        rows_at(s, base, base + n - 1, r0, r1);
        while (r0 < r1) {
            const int64_t mid = r0 + (r1 - r0 + 1) / 2;
            if (*gbl<int32_t>(s.offsets + mid) <= place) r0 = mid;
            else r1 = mid - 1;
        }
        int64_t own_lo, own_hi;
        row_range(s, r0, own_lo, own_hi);
        const int32_t row = own_lo <= place && place < own_hi ? (int32_t)r0 : -1;
        const int32_t row_lo = (int32_t)own_lo, row_hi = (int32_t)own_hi;
        if (row < 0) token = ~0u;                  // of no row: what the order holds there is not read
        if (scribe && lane < n && (row < 0 || row_lo != place)) *gbl_mut<int32_t>(to.owner + place) = -1;
        for (int i = 0; i < n; i += KU) {
            u32x4 raw[KU], old[kAdd ? KU : 1] = {};
#pragma unroll
            for (int j = 0; j < KU; ++j) {
                const int l = (i + j) & 63;
                const uint32_t t = __builtin_amdgcn_readlane(token, l);
                raw[j] = u32x4{};
                if (i + j < n && t < s.tokens && some) raw[j] = load_row<true>(dout + (int64_t)t * stride + at, some);
                if constexpr (kAdd) {
                    const int32_t r = __builtin_amdgcn_readlane(row, l);
                    if (i + j < n && r >= 0 && __builtin_amdgcn_readlane(row_hi, l) == base + i + j + 1)
                        old[j] = old_vector<T>(grad, r, u);
                }
            }
#pragma unroll
            for (int j = 0; j < KU; ++j) {
                if (i + j < n) {
                    const int l = (i + j) & 63;
                    const int32_t r = __builtin_amdgcn_readlane(row, l);
                    if (r != v) {
                        finish(base + i + j, old_of_last);
                        v = r;
                        lo = __builtin_amdgcn_readlane(row_lo, l);
                        hi = __builtin_amdgcn_readlane(row_hi, l);
                        from = base + i + j;
#pragma unroll
                        for (int c = 0; c < V; ++c) acc[c] = 0.0f;
                    }
                    float d[V];
                    widen(raw[j], d);
#pragma unroll
                    for (int c = 0; c < V; ++c) acc[c] += d[c];
                    if (kAdd) old_of_last = old[kAdd ? j : 0];
                }
            }
        }
    }
    finish(end, old_of_last);
    if (scribe && lane < 2) *gbl_mut<int32_t>(to.row_of + 2 * b + lane) = lane ? left[1] : left[0];
}

// sum += the sums that the chunks b0 .. b1 have left of the row that begins at lo.
template <int V>
__device__ __forceinline__ void add_sums(const Chunks& from, int64_t lo, int64_t b0, int64_t b1, int64_t u,
                                         float (&sum)[V]) {
    constexpr int KU = 4;
    for (int64_t b = b0; b <= b1; b += KU) {
        u32x4 raw[KU][V / 4];
#pragma unroll
        for (int j = 0; j < KU; ++j)
#pragma unroll
            for (int i = 0; i < V / 4; ++i) {
                raw[j][i] = u32x4{};
                if (b + j <= b1)
                    raw[j][i] = *gbl<u32x4>(from.sums + (2 * (b + j) + (lo <= (b + j) * from.size ? 0 : 1)) * from.padded +
                                            u * V + 4 * i);
            }
#pragma unroll
        for (int j = 0; j < KU; ++j)
#pragma unroll
            for (int c = 0; c < V; ++c) sum[c] += __uint_as_float(raw[j][c / 4][c % 4]);
    }
}
// The sums of row v; false where they are not all there.
template <int V>
__device__ __forceinline__ bool add_left(const Chunks& from, int64_t v, int64_t lo, int64_t hi, int64_t u,
                                         float (&sum)[V]) {
    const int64_t b0 = lo / from.size, b1 = (hi - 1) / from.size;
    int missing = 0;
#pragma unroll 8
    for (int64_t b = b0; b <= b1; ++b)
        missing |= *gbl<int32_t>(from.row_of + 2 * b + (lo <= b * from.size ? 0 : 1)) ^ (int32_t)v;
    if (missing) return false;
    add_sums<V>(from, lo, b0, b1, u, sum);
    return true;
}

// Rows of 16 chunks or more that begin in a chunk, by a workgroup for 64 vectors
// each: its waves add up a run of the sums each, and the first wave the runs, in
// order.
constexpr int kJoinWaves = 16;
constexpr int64_t kJoinGroups = (int64_t)1 << 20;
template <class T>
__global__ __launch_bounds__(64 * kJoinWaves) void join_left(Sorted s, Chunks from, Grad<T> grad, int64_t tiles,
                                                             int64_t parts) {
    constexpr int V = kVecOf<T>;
    __shared__ float runs[kJoinWaves][V][64];
    __shared__ int gone;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int64_t part = blockIdx.x; part < parts; part += gridDim.x) {
        const int64_t b = part / tiles, tile = part - b * tiles, u = tile * 64 + lane;
        int64_t v = *gbl<int32_t>(from.row_of + 2 * b + 1), lo = 0, hi = 0;
        if (v < 0) v = *gbl<int32_t>(from.row_of + 2 * b);
        if (v < 0) continue;
        row_range(s, v, lo, hi);
        const int64_t last = (hi - 1) / from.size, all = last - b + 1, per = (all + kJoinWaves - 1) / kJoinWaves;
        if (lo / from.size != b || all < kJoinWaves) continue;
        __syncthreads();                           // of the part before: runs and gone are free
        if (threadIdx.x == 0) gone = 0;
        __syncthreads();
        for (int64_t i = threadIdx.x; i < all; i += 64 * kJoinWaves)
            if (*gbl<int32_t>(from.row_of + 2 * (b + i) + (lo <= (b + i) * from.size ? 0 : 1)) != v) gone = 1;
        __syncthreads();
        if (gone) continue;
        float sum[V] = {};
        const int64_t b0 = b + wave * per, b1 = b0 + per - 1 < last ? b0 + per - 1 : last;
        if (b0 <= b1) add_sums<V>(from, lo, b0, b1, u * V < grad.width ? u : 0, sum);
#pragma unroll
        for (int c = 0; c < V; ++c) runs[wave][c][lane] = sum[c];
        __syncthreads();
        if (wave) continue;
#pragma unroll
        for (int c = 0; c < V; ++c) sum[c] = 0.0f;
#pragma unroll 1
        for (int w = 0; w < kJoinWaves; ++w)
#pragma unroll
            for (int c = 0; c < V; ++c) sum[c] += runs[w][c][lane];
        put_vector<T>(grad, v, u, sum, old_vector<T>(grad, v, u));
        if (tile == 0 && lane == 0) *gbl_mut<int32_t>(from.owner + lo) = (int32_t)v;
    }
}

// Vector u of row v, unless it has been written.
template <class T>
__device__ __forceinline__ void finish_vector(const Sorted& s, const Chunks& from, const T* dout, int64_t stride,
                                              const Grad<T>& grad, int64_t v, int64_t u) {
    constexpr int V = kVecOf<T>;
    int64_t lo, hi;
    row_range(s, v, lo, hi);
    const int some = u * V >= grad.width ? 0 : grad.width < V ? (int)grad.width : V;
    const int64_t at = at_vector<V>(u, grad.width);
    if (lo >= hi) {
        if (!grad.accumulate && some) store_row(grad.data + v * grad.stride + at, some, u32x4{});
        return;
    }
    float sum[V] = {};
    bool done = false;
    if (from.size) {
        if (*gbl<int32_t>(from.owner + lo) == v) return;
        if (lo / from.size != (hi - 1) / from.size) done = add_left<V>(from, v, lo, hi, some ? u : 0, sum);
    }
    if (!done) {
        for (int64_t i = lo; i < hi; ++i) {
            const uint32_t t = *gbl<uint32_t>(s.order + i);
            if (t >= s.tokens || !some) continue;
            float d[V];
            widen(load_row(dout + (int64_t)t * stride + at, some), d);
#pragma unroll
            for (int c = 0; c < V; ++c) sum[c] += d[c];
        }
    }
    put_vector<T>(grad, v, u, sum, old_vector<T>(grad, v, u));
}

// Wide rows: a wave takes 64 vectors of two rows, far from each other, since those
// of frequent words stand together. A lane looks up a row, so that both wait once
// before they are cleared. 131072 x 2048 bf16, 16384 tokens: 74 us, the rate of a
// fill; with one row a wave 118, with 4 94, with 8 106, in half the workgroups 89.
constexpr int kRowsAtOnce = 2;
constexpr int64_t kTableGroups = 65536, kAddedGroups = 32768;
template <class T>
__global__ __launch_bounds__(kRowThreads) void finish_table(Sorted s, Chunks from, const T* dout, int64_t stride,
                                                            Grad<T> grad, int64_t parts, int64_t tiles) {
    constexpr int V = kVecOf<T>;
    const int lane = threadIdx.x & 63;
    for (int64_t w = (int64_t)blockIdx.x * (kRowThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
         w < parts * tiles; w += (int64_t)gridDim.x * (kRowThreads / 64)) {
        const int64_t part = w / tiles, u = (w - part * tiles) * 64 + lane, v = lane * parts + part;
        int64_t lo = 0, hi = 0;
        const bool mine = lane < kRowsAtOnce && v < s.vocab;
        if (mine) row_range(s, v, lo, hi);
        const uint64_t clear = __ballot(mine && lo >= hi);
        bool open = lo < hi;
        if (open && from.size) open = *gbl<int32_t>(from.owner + lo) != v;
        if (u * V < grad.width) {
            T* to = grad.data + part * grad.stride + at_vector<V>(u, grad.width);
            const int some = grad.width < V ? (int)grad.width : V;
#pragma unroll
            for (int j = 0; j < kRowsAtOnce; ++j)
                if (clear >> j & 1) store_row(to + j * parts * grad.stride, some, u32x4{});
        }
        for (uint64_t left = __ballot(open); left; left &= left - 1)
            finish_vector<T>(s, from, dout, stride, grad, __builtin_ctzll(left) * parts + part, u);
    }
}

// A gradient that is added to: only rows that no chunk has written whole. A wave
// looks for them 64 at once, in rows far from each other, since those of frequent
// words stand together, and then takes 64 vectors of each.
template <class T>
__global__ __launch_bounds__(kRowThreads) void finish_added(Sorted s, Chunks from, const T* dout, int64_t stride,
                                                            Grad<T> grad, int64_t parts, int64_t tiles) {
    const int lane = threadIdx.x & 63;
    for (int64_t w = (int64_t)blockIdx.x * (kRowThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); w < parts * tiles;
         w += (int64_t)gridDim.x * (kRowThreads / 64)) {
        const int64_t part = w / tiles, tile = w - part * tiles, v = lane * parts + part;
        int64_t lo = 0, hi = 0;
        if (v < s.vocab) row_range(s, v, lo, hi);
        bool open = lo < hi;
        if (open && from.size) open = *gbl<int32_t>(from.owner + lo) != v;
        for (uint64_t left = __ballot(open); left; left &= left - 1)
            finish_vector<T>(s, from, dout, stride, grad, __builtin_ctzll(left) * parts + part, tile * 64 + lane);
    }
}

// Narrow rows: 2^lane_log2 lanes each.
template <class T>
__global__ __launch_bounds__(kRowThreads) void finish_narrow(Sorted s, Chunks from, const T* dout, int64_t stride,
                                                             Grad<T> grad, int lane_log2) {
    const int64_t per = kRowThreads >> lane_log2;
    for (int64_t v = (int64_t)blockIdx.x * per + (threadIdx.x >> lane_log2); v < s.vocab; v += (int64_t)gridDim.x * per)
        finish_vector<T>(s, from, dout, stride, grad, v, threadIdx.x & ((1 << lane_log2) - 1));
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
        const int64_t n = width ? chunks_of(tokens) : 0;
        *bytes = 0;
        if (n && (__builtin_mul_overflow(n * 8, padded_width(width) + 1, bytes) ||
                  __builtin_add_overflow(*bytes, tokens * 4, bytes)))
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
            const int64_t units = (width * size + 15) / 16, tiles = (units + 63) / 64;
            const int64_t padded = padded_width(width), n = need ? chunks_of(tokens) : 0;
            const Sorted sorted{offsets, order, tokens, vocab};
            Chunks chunks{(float*)workspace, nullptr, nullptr, padded, n ? chunk_of(tokens) : 0};
            chunks.row_of = (int32_t*)(chunks.sums + 2 * n * padded);
            chunks.owner = chunks.row_of + 2 * n;
            const auto go = [&](auto type) {
                using T = decltype(type);
                const Grad<T> to{(T*)grad, grad_stride, width, scale, accumulate ? 1 : 0};
                if (n) {
                    const int64_t waves = n * tiles;
                    const auto kernel = accumulate ? sum_chunks<T, true> : sum_chunks<T, false>;
                    const hipError_t e = enqueue(kernel, dim3((uint32_t)((waves + 3) / 4)), kRowThreads, 0, s, sorted,
                                                 chunks, (const T*)dout, dout_stride, to, waves, (int)tiles);
                    if (e != hipSuccess) return e;
                }
                if (n && tokens > kJoinTokens) {
                    const int64_t parts = n * tiles;
                    const hipError_t e = enqueue(join_left<T>, dim3((uint32_t)(parts < kJoinGroups ? parts : kJoinGroups)),
                                                 64 * kJoinWaves, 0, s, sorted, chunks, to, tiles, parts);
                    if (e != hipSuccess) return e;
                }
                if (accumulate) {
                    const int64_t parts = (vocab + 63) / 64, groups = (parts * tiles + 3) / 4;
                    return enqueue(finish_added<T>, dim3((uint32_t)(groups < kAddedGroups ? groups : kAddedGroups)),
                                   kRowThreads, 0, s, sorted, chunks, (const T*)dout, dout_stride, to, parts, tiles);
                }
                if (units <= 32) {
                    const RowGrid g = row_grid(vocab, units);
                    return enqueue(finish_narrow<T>, dim3(g.grid.x), kRowThreads, 0, s, sorted, chunks, (const T*)dout,
                                   dout_stride, to, g.lane_log2);
                }
                const int64_t parts = (vocab + kRowsAtOnce - 1) / kRowsAtOnce, groups = (parts * tiles + 3) / 4;
                return enqueue(finish_table<T>, dim3((uint32_t)(groups < kTableGroups ? groups : kTableGroups)), kRowThreads, 0, s,
                               sorted, chunks, (const T*)dout, dout_stride, to, parts, tiles);
            };
            return size == 2 ? go(uint16_t{}) : go(float{});
        });
    });
}

}  // extern "C"
