// Token-embedding lookup with scaling, and the gradient of its table by sorted tokens
// (sm_100a). Both move rows and compute next to nothing, so memory traffic bounds them:
// the lookup reads each row it needs and writes it once; the gradient reads each text row
// of d_out once and writes each row of the table once.
#pragma once
#include "ops_common.cuh"

namespace vlp_ops {

// ---------------------------------------------------------------- lookup
// out[r] = round(scale * table[ids[r]]). One warp per row; kWide: 8 elements a lane at a
// time (16-byte accesses, rows aligned), the N % 8 last ones singly; else singly. copy:
// one type and scale 1, the bits go through unchanged.
template <int kIn, int kOut, bool kWide>
static __global__ void __launch_bounds__(256) vlp_embed_rows_kernel(
    const int64_t* __restrict__ ids, int64_t n, int64_t token, const void* __restrict__ table, int64_t vocab,
    int64_t table_ld, void* __restrict__ out, int64_t out_ld, int N, float scale, int copy, int* status) {
    using TI = typename Elem<kIn>::T;
    using TO = typename Elem<kOut>::T;
    const int lane = threadIdx.x & 31;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (r >= n) return;
    const int64_t id = __ldg(ids + r);
    if (id == token) return;
    TO* dst = static_cast<TO*>(out) + r * out_ld;
    const bool bad = id < 0 || id >= vocab;
    if (bad) {
        if (lane == 0 && status != nullptr) atomicCAS(status, VLPROJ_OK, VLPROJ_ERR_INVALID_ARG);
        for (int c = lane; c < N; c += 32) dst[c] = Elem<kOut>::down(0.f);
        return;
    }
    const TI* src = static_cast<const TI*>(table) + id * table_ld;
    int c0 = 0;
    if constexpr (kWide) {
        c0 = N & ~7;
#pragma unroll 4
        for (int c = 8 * lane; c < c0; c += 256) {
            const Raw8<kIn> v = load8<kIn>(src + c);
            if constexpr (kIn == kOut) {
                if (copy) {
                    store8<kOut>(dst + c, v);
                    continue;
                }
            }
            float f[8];
            unpack8<kIn>(v, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= scale;
            store8<kOut>(dst + c, pack8<kOut>(f));
        }
    }
#pragma unroll 4
    for (int c = c0 + lane; c < N; c += 32) {
        const TI v = __ldg(src + c);
        if constexpr (kIn == kOut) {
            if (copy) {
                dst[c] = v;
                continue;
            }
        }
        dst[c] = Elem<kOut>::down(Elem<kIn>::up(v) * scale);
    }
}

// ---------------------------------------------------------------- sort by token
// Stable radix sort of (key, position) pairs, key = the id, or `vocab` for rows that count
// for nothing (placeholders, ids out of range), which so end up last. An element is key <<
// 32 | position. Each pass takes `bits` bits: every block counts the digits of its own
// contiguous run, then every block finds where its elements of each digit go (all smaller
// digits, then the same digit in earlier blocks, then earlier warps of its own), and each
// warp walks its part of the run in order, so equal digits keep their order.
constexpr int SORT_THREADS = 256;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_MAX_BITS = 10;
constexpr int SORT_MAX_BINS = 1 << SORT_MAX_BITS;
constexpr int SORT_MAX_BLOCKS = 128;

struct SortSource {
    const int64_t* ids;       // first pass: the ids; else null
    const uint64_t* pairs;    // later passes
    int64_t token;
    int64_t vocab;
    int* status;
};

__device__ __forceinline__ uint64_t sort_element(const SortSource& s, int64_t i, bool report) {
    if (s.ids == nullptr) return __ldg(s.pairs + i);
    const int64_t id = __ldg(s.ids + i);
    uint64_t key = static_cast<uint64_t>(id);
    if (id == s.token || id < 0 || id >= s.vocab) {
        if (report && id != s.token && s.status != nullptr) atomicCAS(s.status, VLPROJ_OK, VLPROJ_ERR_INVALID_ARG);
        key = static_cast<uint64_t>(s.vocab);
    }
    return key << 32 | static_cast<uint64_t>(i);
}

__device__ __forceinline__ int sort_digit(uint64_t e, int shift, int mask) {
    return static_cast<int>(e >> (32 + shift)) & mask;
}

// counts[block][digit] over the block's `run` elements.
static __global__ void __launch_bounds__(SORT_THREADS) vlp_sort_count_kernel(SortSource src, int64_t n, int run,
                                                                             int shift, int bins,
                                                                             uint32_t* __restrict__ counts) {
    __shared__ uint32_t hist[SORT_MAX_BINS];
    for (int d = threadIdx.x; d < bins; d += SORT_THREADS) hist[d] = 0;
    __syncthreads();
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * run;
    const int64_t i1 = i0 + run < n ? i0 + run : n;
    for (int64_t i = i0 + threadIdx.x; i < i1; i += SORT_THREADS)
        atomicAdd(&hist[sort_digit(sort_element(src, i, true), shift, bins - 1)], 1u);
    __syncthreads();
    for (int d = threadIdx.x; d < bins; d += SORT_THREADS) counts[static_cast<int64_t>(blockIdx.x) * bins + d] = hist[d];
}

static __global__ void __launch_bounds__(SORT_THREADS) vlp_sort_scatter_kernel(SortSource src, int64_t n, int run,
                                                                               int shift, int bins, int nblocks,
                                                                               const uint32_t* __restrict__ counts,
                                                                               uint64_t* __restrict__ dst) {
    __shared__ uint32_t at[SORT_WARPS][SORT_MAX_BINS];   // per warp: count, then next slot, of each digit
    __shared__ uint32_t base[SORT_MAX_BINS];
    __shared__ uint32_t before[SORT_MAX_BINS];
    __shared__ uint32_t warp_tot[SORT_WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int d = threadIdx.x; d < bins; d += SORT_THREADS)
        for (int w = 0; w < SORT_WARPS; ++w) at[w][d] = 0;
    __syncthreads();
    // the warp's part of the block's run: run is a multiple of SORT_THREADS
    const int part = run / SORT_WARPS;
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * run + static_cast<int64_t>(warp) * part;
    const int64_t i1 = i0 + part < n ? i0 + part : n;
    for (int64_t i = i0 + lane; i < i1; i += 32)
        atomicAdd(&at[warp][sort_digit(sort_element(src, i, false), shift, bins - 1)], 1u);
    // each digit's total, and its count in earlier blocks
    for (int d = threadIdx.x; d < bins; d += SORT_THREADS) {
        uint32_t total = 0, mine = 0;
#pragma unroll 8
        for (int b = 0; b < nblocks; ++b) {
            const uint32_t c = __ldg(counts + static_cast<int64_t>(b) * bins + d);
            if (b < static_cast<int>(blockIdx.x)) mine += c;
            total += c;
        }
        base[d] = total;
        before[d] = mine;
    }
    __syncthreads();
    // exclusive prefix sums of the totals over the digits: thread t owns `per` digits in a row
    const int per = (bins + SORT_THREADS - 1) / SORT_THREADS;
    const int d0 = threadIdx.x * per, d1 = d0 + per < bins ? d0 + per : bins;
    uint32_t own = 0;
    for (int d = d0; d < d1; ++d) own += base[d];
    uint32_t inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += t;
    }
    if (lane == 31) warp_tot[warp] = inc;
    __syncthreads();
    uint32_t next = inc - own;
    for (int w = 0; w < warp; ++w) next += warp_tot[w];
    for (int d = d0; d < d1; ++d) {
        const uint32_t total = base[d];
        uint32_t slot = next + before[d];
        for (int w = 0; w < SORT_WARPS; ++w) {
            const uint32_t c = at[w][d];
            at[w][d] = slot;
            slot += c;
        }
        next += total;
    }
    __syncthreads();
    for (int64_t i = i0; i < i1; i += 32) {
        const bool live = i + lane < i1;
        const unsigned act = __ballot_sync(0xffffffffu, live);
        if (live) {
            const uint64_t e = sort_element(src, i + lane, false);
            const int d = sort_digit(e, shift, bins - 1);
            const unsigned peers = __match_any_sync(act, d);
            const int rank = __popc(peers & ((1u << lane) - 1u));
            const uint32_t slot = at[warp][d];
            __syncwarp(act);
            if (rank == 0) at[warp][d] = slot + __popc(peers);
            dst[slot + rank] = e;
        }
        __syncwarp();
    }
}

// ---------------------------------------------------------------- sums over sorted rows
// The sorted rows are cut into chunks of `rows` positions, the columns into tiles of
// SUM_THREADS * kCols. A block adds one chunk's rows of one tile, each thread its own
// columns, walking the rows in order and writing a token's sum where its run ends. A run
// that began in an earlier chunk, or goes on in a later one, leaves a partial sum in the
// workspace instead: slot 0 of the chunk for the run its first row belongs to (when that
// run began earlier), slot 1 for the run its last row belongs to (when it began here).
// vlp_scatter_join_kernel adds the partial sums in order. So a token may have any number
// of rows, and the order of its sum is fixed by n and the grid alone.
constexpr int SUM_THREADS = 128;
constexpr int SUM_BATCH = 8;          // rows whose loads are in flight together
constexpr int SUM_MAX_ROWS = 128;

struct ScatterOut {
    float* d_table;
    int64_t ld;
    int N;
    float scale;
    int accumulate;
};

__device__ __forceinline__ int64_t lower_bound_key(const uint64_t* __restrict__ pairs, int64_t n, uint64_t key) {
    int64_t lo = 0, hi = n;
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if ((__ldg(pairs + mid) >> 32) < key) lo = mid + 1; else hi = mid;
    }
    return lo;
}

// Writes (or adds) kCols sums of token t at columns c ..
template <int kCols>
__device__ __forceinline__ void scatter_write(const ScatterOut& o, uint32_t t, int c, const float (&s)[kCols], bool wide) {
    float* row = o.d_table + static_cast<int64_t>(t) * o.ld + c;
    if constexpr (kCols % 4 == 0) {
        if (wide) {
#pragma unroll
            for (int q = 0; q < kCols / 4; ++q) {
                float4 v = make_float4(s[4 * q] * o.scale, s[4 * q + 1] * o.scale, s[4 * q + 2] * o.scale,
                                       s[4 * q + 3] * o.scale);
                if (o.accumulate) {
                    const float4 u = reinterpret_cast<float4*>(row)[q];
                    v = make_float4(u.x + v.x, u.y + v.y, u.z + v.z, u.w + v.w);
                }
                reinterpret_cast<float4*>(row)[q] = v;
            }
            return;
        }
    }
#pragma unroll
    for (int e = 0; e < kCols; ++e)
        if (c + e < o.N) row[e] = (o.accumulate ? row[e] : 0.f) + s[e] * o.scale;
}

// kCols 8: rows of d_out and d_table are 16-byte aligned and N % 8 == 0; kCols 1: any.
template <int kType, int kCols>
static __global__ void __launch_bounds__(SUM_THREADS) vlp_scatter_sum_kernel(
    const uint64_t* __restrict__ pairs, int64_t n, uint32_t vocab, int rows, int tiles,
    const void* __restrict__ d_out, int64_t d_out_ld, ScatterOut o, float* __restrict__ part) {
    using T = typename Elem<kType>::T;
    __shared__ uint32_t key[SUM_MAX_ROWS + 2];      // keys of rows -1 .. rows of the chunk
    __shared__ uint32_t pos[SUM_MAX_ROWS];
    const int64_t chunk = blockIdx.x / tiles;
    const int c = (static_cast<int>(blockIdx.x % tiles) * SUM_THREADS + static_cast<int>(threadIdx.x)) * kCols;
    const int64_t i0 = chunk * rows;
    const int m = static_cast<int>(i0 + rows < n ? rows : n - i0);
    for (int i = static_cast<int>(threadIdx.x) - 1; i <= m; i += SUM_THREADS) {
        const int64_t j = i0 + i;
        const uint64_t e = j >= 0 && j < n ? __ldg(pairs + j) : ~0ull;
        key[i + 1] = static_cast<uint32_t>(e >> 32);
        if (i >= 0 && i < m) pos[i] = static_cast<uint32_t>(e);
    }
    __syncthreads();
    if (c >= o.N || key[1] >= vocab) return;
    const T* src = static_cast<const T*>(d_out) + c;
    float s[kCols];
#pragma unroll
    for (int e = 0; e < kCols; ++e) s[e] = 0.f;
    bool earlier = key[0] == key[1];                // the run at hand began in an earlier chunk
    for (int i = 0; i < m; i += SUM_BATCH) {
        Raw8<kType> v[SUM_BATCH];
        T u[SUM_BATCH];
#pragma unroll
        for (int b = 0; b < SUM_BATCH; ++b) {
            if (i + b < m && key[i + b + 1] < vocab) {
                if constexpr (kCols == 8) v[b] = load8<kType>(src + pos[i + b] * d_out_ld);
                else u[b] = __ldg(src + pos[i + b] * d_out_ld);
            }
        }
#pragma unroll
        for (int b = 0; b < SUM_BATCH; ++b) {
            const int r = i + b;
            const uint32_t k = r < m ? key[r + 1] : vocab;
            if (k >= vocab) break;
            if constexpr (kCols == 8) {
                float f[8];
                unpack8<kType>(v[b], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) s[e] += f[e];
            } else {
                s[0] += Elem<kType>::up(u[b]);
            }
            const bool last = r + 1 == m;
            const bool ends = key[r + 2] != k;
            if (!ends && !last) continue;
            if (ends && !earlier) {
                scatter_write<kCols>(o, k, c, s, kCols == 8);
            } else {
                float* p = part + (2 * chunk + (earlier ? 0 : 1)) * o.N + c;
                if constexpr (kCols == 8) {
                    reinterpret_cast<float4*>(p)[0] = make_float4(s[0], s[1], s[2], s[3]);
                    reinterpret_cast<float4*>(p)[1] = make_float4(s[4], s[5], s[6], s[7]);
                } else {
                    p[0] = s[0];
                }
            }
#pragma unroll
            for (int e = 0; e < kCols; ++e) s[e] = 0.f;
            earlier = false;
        }
    }
}

// One block per chunk and column tile: the run that begins in the chunk and goes on past
// it has its first part in the chunk's slot 1 and the others in slot 0 of the following
// chunks up to the one its last row lies in; they are added in that order, in fp64.
constexpr int JOIN_THREADS = 128;
static __global__ void __launch_bounds__(JOIN_THREADS) vlp_scatter_join_kernel(const uint64_t* __restrict__ pairs,
                                                                               int64_t n, uint32_t vocab, int rows,
                                                                               int tiles,
                                                                               const float* __restrict__ part,
                                                                               ScatterOut o) {
    const int64_t chunk = blockIdx.x / tiles;
    const int c = static_cast<int>(blockIdx.x % tiles) * JOIN_THREADS + static_cast<int>(threadIdx.x);
    const int64_t i0 = chunk * rows, i1 = i0 + rows;
    if (i1 >= n) return;                                               // the last chunk: nothing follows
    const uint32_t k = static_cast<uint32_t>(__ldg(pairs + i1 - 1) >> 32);
    if (k >= vocab || static_cast<uint32_t>(__ldg(pairs + i1) >> 32) != k) return;      // ends here
    if (i0 > 0 && static_cast<uint32_t>(__ldg(pairs + i0 - 1) >> 32) == k) return;       // began earlier
    const int64_t last = (lower_bound_key(pairs, n, static_cast<uint64_t>(k) + 1) - 1) / rows;
    if (c >= o.N) return;
    double s = part[(2 * chunk + 1) * o.N + c];
#pragma unroll 8
    for (int64_t q = chunk + 1; q <= last; ++q) s += part[2 * q * o.N + c];
    float* row = o.d_table + static_cast<int64_t>(k) * o.ld + c;
    *row = (o.accumulate ? *row : 0.f) + static_cast<float>(s * o.scale);
}

// Rows of tokens that do not occur: one warp per 32 tokens, each lane looks its own up.
static __global__ void __launch_bounds__(256) vlp_scatter_zero_kernel(const uint64_t* __restrict__ pairs, int64_t n,
                                                                      int64_t vocab, ScatterOut o, int wide) {
    const int lane = threadIdx.x & 31;
    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * 32;
    if (t0 >= vocab) return;
    const int64_t t = t0 + lane;
    bool absent = false;
    if (t < vocab) {
        const int64_t j = lower_bound_key(pairs, n, static_cast<uint64_t>(t));
        absent = j >= n || static_cast<int64_t>(__ldg(pairs + j) >> 32) != t;
    }
    unsigned todo = __ballot_sync(0xffffffffu, absent);
    while (todo != 0) {
        const int b = __ffs(todo) - 1;
        todo &= todo - 1;
        float* row = o.d_table + (t0 + b) * o.ld;
        int c0 = 0;
        if (wide) {
            c0 = o.N & ~3;
            for (int c = 4 * lane; c < c0; c += 128) *reinterpret_cast<float4*>(row + c) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int c = c0 + lane; c < o.N; c += 32) row[c] = 0.f;
    }
}

}  // namespace vlp_ops
