// Token-embedding lookup with scaling, and the gradient of its table by sorted tokens
// (sm_100a). Both move rows and compute next to nothing, so memory traffic bounds them:
// the lookup reads each row it needs and writes it once; the gradient reads each text row
// of d_out once and writes each row of the table once.
#pragma once
#include "ops_common.cuh"

namespace vlp_ops {

// Whether a row holds a placeholder. Of a call without any, an id that happens to have the
// value of VLPROJ_NO_TOKEN is one outside the table, like every other negative id.
__device__ __forceinline__ bool placeholder(int64_t id, int64_t token) { return id == token && token != VLPROJ_NO_TOKEN; }

// ---------------------------------------------------------------- lookup
// out[r] = round(scale * table[ids[r]]). A warp takes one segment (blockIdx.y) of one row:
// a batch of accesses of each lane, all loads issued before the first is used, so that a
// few rows do not wait for several trips to memory and many rows keep it busy. kWide:
// 8 elements an access (rows aligned for it, the N % 8 last ones singly) and 4 accesses,
// else one element and 8 accesses. copy: one type and scale 1, the bits go through
// unchanged. All rows' first segments come before their second ones: 131072 rows of 4096
// bf16 take 196 us so (6.1 TB/s), 206 us row by row, 203 us with 8 accesses, 206 us with
// stores that stay in the caches; 65536 rows of 1001 bf16, 60 us with 8 and 86 us with 4.
template <bool kWide>
constexpr int embed_batch() { return kWide ? 4 : 8; }
template <bool kWide>
constexpr int embed_segment() { return 32 * embed_batch<kWide>() * (kWide ? 8 : 1); }      // elements

template <int kIn, int kOut, bool kWide>
static __global__ void __launch_bounds__(256) vlp_embed_rows_kernel(
    const int64_t* __restrict__ ids, int64_t n, int64_t token, const void* __restrict__ table, int64_t vocab,
    int64_t table_ld, void* __restrict__ out, int64_t out_ld, int N, float scale, int copy, int* status) {
    using TI = typename Elem<kIn>::T;
    using TO = typename Elem<kOut>::T;
    constexpr int BATCH = embed_batch<kWide>();
    const int lane = threadIdx.x & 31;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (r >= n) return;
    const int64_t id = __ldg(ids + r);
    if (placeholder(id, token)) return;
    TO* dst = static_cast<TO*>(out) + r * out_ld;
    const int c0 = static_cast<int>(blockIdx.y) * embed_segment<kWide>();
    if (id < 0 || id >= vocab) {
        if (c0 == 0 && lane == 0 && status != nullptr) atomicCAS(status, VLPROJ_OK, VLPROJ_ERR_INVALID_ARG);
        for (int c = c0 + lane; c < N && c < c0 + embed_segment<kWide>(); c += 32) dst[c] = Elem<kOut>::down(0.f);
        return;
    }
    const TI* src = static_cast<const TI*>(table) + id * table_ld;
    if constexpr (kWide) {
        const int full = N & ~7;
        if (c0 < full) {
            Raw8<kIn> v[BATCH];
#pragma unroll
            for (int q = 0; q < BATCH; ++q) {
                const int c = c0 + 8 * (lane + 32 * q);
                v[q] = load8<kIn>(src + (c < full ? c : c0));
            }
#pragma unroll
            for (int q = 0; q < BATCH; ++q) {
                const int c = c0 + 8 * (lane + 32 * q);
                if (c >= full) continue;
                if constexpr (kIn == kOut) {
                    if (copy) {
                        store8_once<kOut>(dst + c, v[q]);
                        continue;
                    }
                }
                float f[8];
                unpack8<kIn>(v[q], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] *= scale;
                store8_once<kOut>(dst + c, pack8<kOut>(f));
            }
        }
        const int c = full + lane;                     // fewer than 8 left: in the row's last segment
        if (c < N && N <= c0 + embed_segment<true>()) {
            const TI u = __ldg(src + c);
            if constexpr (kIn == kOut) {
                dst[c] = copy ? u : Elem<kOut>::down(Elem<kIn>::up(u) * scale);
            } else {
                dst[c] = Elem<kOut>::down(Elem<kIn>::up(u) * scale);
            }
        }
    } else {
        TI v[BATCH];
#pragma unroll
        for (int q = 0; q < BATCH; ++q) {
            const int c = c0 + lane + 32 * q;
            v[q] = __ldg(src + (c < N ? c : c0));
        }
#pragma unroll
        for (int q = 0; q < BATCH; ++q) {
            const int c = c0 + lane + 32 * q;
            if (c >= N) continue;
            if constexpr (kIn == kOut) {
                dst[c] = copy ? v[q] : Elem<kOut>::down(Elem<kIn>::up(v[q]) * scale);
            } else {
                dst[c] = Elem<kOut>::down(Elem<kIn>::up(v[q]) * scale);
            }
        }
    }
}

// ---------------------------------------------------------------- sort by token
// Stable radix sort of (key, position) pairs, key = the id, or `vocab` for rows that count
// for nothing (placeholders, ids out of range), which so end up last. An element is key <<
// 32 | position. Each pass takes `bits` bits: every block counts the digits of its own
// contiguous run, then every block finds where its elements of each digit go (all smaller
// digits, then the same digit in earlier blocks, then earlier warps of its own), and each
// warp ranks its elements in order, so equal digits keep their order. A block works on
// tiles of SORT_TILE elements held in registers. Both kernels wait for memory more than
// they move it (131072 ids are 1 MB), so all loads of a step are issued together.
constexpr int SORT_THREADS = 512;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_ITEMS = 4;                       // elements of a thread
constexpr int SORT_TILE = SORT_THREADS * SORT_ITEMS;
constexpr int SORT_MAX_BITS = 10;
constexpr int SORT_MAX_BINS = 1 << SORT_MAX_BITS;
constexpr int SORT_MAX_BLOCKS = 128;

struct SortSource {
    const int64_t* ids;       // first pass: the ids; else null
    const uint64_t* pairs;    // later passes
    int64_t n;
    int64_t token;
    int64_t vocab;
    int* status;
};

// The thread's elements i0 + 32 q (q < SORT_ITEMS) of [0, end); the others repeat the last one.
__device__ __forceinline__ void sort_load(const SortSource& s, int64_t i0, int64_t end, bool report,
                                          uint64_t (&e)[SORT_ITEMS]) {
    int64_t at[SORT_ITEMS];
#pragma unroll
    for (int q = 0; q < SORT_ITEMS; ++q) {
        const int64_t i = i0 + 32 * q;
        at[q] = i < end ? i : end - 1;
    }
    if (s.ids == nullptr) {
#pragma unroll
        for (int q = 0; q < SORT_ITEMS; ++q) e[q] = s.pairs[at[q]];
        return;
    }
#pragma unroll
    for (int q = 0; q < SORT_ITEMS; ++q) e[q] = static_cast<uint64_t>(s.ids[at[q]]);
#pragma unroll
    for (int q = 0; q < SORT_ITEMS; ++q) {
        const int64_t id = static_cast<int64_t>(e[q]);
        const bool in = id >= 0 && id < s.vocab;
        if (report && !in && !placeholder(id, s.token) && s.status != nullptr)
            atomicCAS(s.status, VLPROJ_OK, VLPROJ_ERR_INVALID_ARG);
        const uint64_t key = in && id != s.token ? static_cast<uint64_t>(id) : static_cast<uint64_t>(s.vocab);
        e[q] = key << 32 | static_cast<uint64_t>(at[q]);
    }
}

__device__ __forceinline__ int sort_digit(uint64_t e, int shift, int mask) {
    return static_cast<int>(e >> (32 + shift)) & mask;
}

// counts[digit][block] (pitch entries apart, a multiple of 4) of the block's `run` elements.
static __global__ void __launch_bounds__(SORT_THREADS) vlp_sort_count_kernel(SortSource src, int run, int shift,
                                                                             int bins, int pitch,
                                                                             uint32_t* counts) {
    __shared__ uint32_t hist[SORT_MAX_BINS];
    for (int d = threadIdx.x; d < bins; d += SORT_THREADS) hist[d] = 0;
    __syncthreads();
    const int64_t b0 = static_cast<int64_t>(blockIdx.x) * run;
    const int64_t b1 = b0 + run < src.n ? b0 + run : src.n;
    after_previous_kernel(src.pairs, counts);
    for (int64_t t0 = b0; t0 < b1; t0 += SORT_TILE) {
        uint64_t e[SORT_ITEMS];
        const int64_t i0 = t0 + (threadIdx.x >> 5) * (32 * SORT_ITEMS) + (threadIdx.x & 31);
        sort_load(src, i0, b1, true, e);
#pragma unroll
        for (int q = 0; q < SORT_ITEMS; ++q)
            if (i0 + 32 * q < b1) atomicAdd(&hist[sort_digit(e[q], shift, bins - 1)], 1u);
    }
    let_next_kernel_start();
    __syncthreads();
    for (int d = threadIdx.x; d < bins; d += SORT_THREADS) counts[static_cast<int64_t>(d) * pitch + blockIdx.x] = hist[d];
}

static __global__ void __launch_bounds__(SORT_THREADS) vlp_sort_scatter_kernel(SortSource src, int run, int shift,
                                                                               int bins, int nblocks, int pitch,
                                                                               const uint32_t* counts, uint64_t* dst) {
    __shared__ uint16_t at[SORT_WARPS][SORT_MAX_BINS];   // of a tile: the warp's count, then its next rank, of a digit
    __shared__ uint32_t base[SORT_MAX_BINS];             // next slot of each digit
    __shared__ uint32_t warp_tot[SORT_WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t b0 = static_cast<int64_t>(blockIdx.x) * run;
    const int64_t b1 = b0 + run < src.n ? b0 + run : src.n;
    after_previous_kernel(src.pairs, counts);
    uint64_t e[SORT_ITEMS];
    const int64_t mine = warp * (32 * SORT_ITEMS) + lane;
    sort_load(src, b0 + mine, b1, false, e);             // the first tile, on its way during what follows
    // each digit's total, and its count in earlier blocks
    uint32_t total[SORT_MAX_BINS / SORT_THREADS], own = 0;
#pragma unroll
    for (int p = 0; p < SORT_MAX_BINS / SORT_THREADS; ++p) {
        // thread t owns the digits p * SORT_THREADS + t
        const int d = p * SORT_THREADS + threadIdx.x;
        uint32_t all = 0, before = 0;
        if (d < bins) {
            const uint4* row = reinterpret_cast<const uint4*>(counts + static_cast<int64_t>(d) * pitch);
            const int mine_block = blockIdx.x;
#pragma unroll 16
            for (int b = 0; b < pitch / 4; ++b) {        // entries past nblocks are zero or not counted
                const uint4 c = row[b];                  // written by the kernel before: no read-only load
                const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int k = 4 * b + q;
                    all += k < nblocks ? w[q] : 0u;
                    before += k < mine_block ? w[q] : 0u;
                }
            }
            base[d] = before;
        }
        total[p] = all;
    }
    // exclusive prefix sums of the totals over the digits, SORT_THREADS digits at a time
#pragma unroll
    for (int p = 0; p < SORT_MAX_BINS / SORT_THREADS; ++p) {
        if (p * SORT_THREADS >= bins) break;
        uint32_t inc = total[p];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t t = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += t;
        }
        if (lane == 31) warp_tot[warp] = inc;
        __syncthreads();
        uint32_t next = own + inc - total[p];
#pragma unroll
        for (int w = 0; w < SORT_WARPS; ++w) {
            const uint32_t t = warp_tot[w];
            next += w < warp ? t : 0u;
            own += t;
        }
        const int d = p * SORT_THREADS + threadIdx.x;
        if (d < bins) base[d] += next;
        __syncthreads();
    }
    for (int64_t t0 = b0; t0 < b1; t0 += SORT_TILE) {
        for (int d = threadIdx.x; d < bins; d += SORT_THREADS)
#pragma unroll
            for (int w = 0; w < SORT_WARPS; ++w) at[w][d] = 0;
        if (t0 != b0) sort_load(src, t0 + mine, b1, false, e);
        __syncthreads();
        // the rank of each element among its warp's elements of the same digit
        int digit[SORT_ITEMS], rank[SORT_ITEMS];
#pragma unroll
        for (int q = 0; q < SORT_ITEMS; ++q) {
            const bool live = t0 + mine + 32 * q < b1;
            digit[q] = sort_digit(e[q], shift, bins - 1);
            const unsigned act = __ballot_sync(0xffffffffu, live);
            if (live) {
                const unsigned peers = __match_any_sync(act, digit[q]);
                const int below = __popc(peers & ((1u << lane) - 1u));
                const int seen = at[warp][digit[q]];
                __syncwarp(act);
                if (below == 0) at[warp][digit[q]] = static_cast<uint16_t>(seen + __popc(peers));
                rank[q] = seen + below;
            }
            __syncwarp();
        }
        __syncthreads();
        // per digit: the warps' first ranks in the tile
        for (int d = threadIdx.x; d < bins; d += SORT_THREADS) {
            uint32_t run_ = 0;
#pragma unroll
            for (int w = 0; w < SORT_WARPS; ++w) {
                const uint32_t c = at[w][d];
                at[w][d] = static_cast<uint16_t>(run_);
                run_ += c;
            }
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < SORT_ITEMS; ++q)
            if (t0 + mine + 32 * q < b1) dst[base[digit[q]] + at[warp][digit[q]] + rank[q]] = e[q];
        if (t0 + SORT_TILE >= b1) break;
        __syncthreads();
#pragma unroll
        for (int q = 0; q < SORT_ITEMS; ++q) atomicAdd(&base[digit[q]], 1u);      // a full tile: all live
        __syncthreads();
    }
}

// ---------------------------------------------------------------- sums over sorted rows
// The sorted rows are cut into chunks of `rows` positions, the columns into tiles. A group
// of a block's threads (kGroups of them, more for narrow rows) adds one chunk's rows of one
// tile, each thread its own columns, walking the rows in order with the loads of SUM_BATCH
// rows in flight, and writes a token's sum where its run ends. A run that began in an
// earlier chunk, or goes on in a later one, leaves a partial sum in the workspace instead:
// slot 0 of the chunk for the run its first row belongs to (when that run began earlier),
// slot 1 for the run its last row belongs to (when it began here). vlp_scatter_join_kernel
// adds the partial sums in order. So a token may have any number of rows, and the order of
// its sum is fixed by n and N alone. Further blocks of the same launch write the zero rows,
// ZERO_TOKENS tokens each: their writes and the chunks' reads keep the memory busy together
// (131072 x 4096 bf16 into 102400 fp32 rows: 400 us, 6.6 TB/s; in two launches 438 us).
constexpr int SUM_THREADS = 128;
constexpr int SUM_BATCH = 8;
constexpr int SUM_MAX_ROWS = 128;
constexpr int ZERO_TOKENS = 32;

struct ScatterOut {
    float* d_table;
    int64_t ld;
    int64_t vocab;
    int N;
    float scale;
    int accumulate;
};

// The columns of a thread: SUM_ACCESSES<kWidth> accesses of kWidth adjacent elements,
// `threads` * kWidth apart, from c0 on. kWidth 8: rows of d_out and d_table aligned for
// 8-element accesses and N % 8 == 0; 2: the same for 2; else 1.
template <int kWidth>
constexpr int sum_accesses() { return kWidth == 8 ? 1 : 4; }
template <int kWidth>
constexpr int sum_cols() { return kWidth * sum_accesses<kWidth>(); }

// The elements of one row at a thread's columns; accesses past N repeat the first one.
template <int kType, int kWidth>
struct SumRow;
template <int kType>
struct SumRow<kType, 8> {
    Raw8<kType> v;
    __device__ __forceinline__ void load(const typename Elem<kType>::T* row, const int (&col)[1]) { v = load8<kType>(row + col[0]); }
    __device__ __forceinline__ void add_to(float (&s)[8]) const {
        float f[8];
        unpack8<kType>(v, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] += f[e];
    }
};
template <int kType>
struct SumRow<kType, 2> {
    using T = typename Elem<kType>::T;
    using Pair = typename std::conditional<kType == VLPROJ_F32, uint2, uint32_t>::type;
    Pair v[4];
    __device__ __forceinline__ void load(const T* row, const int (&col)[4]) {
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = __ldg(reinterpret_cast<const Pair*>(row + col[q]));
    }
    __device__ __forceinline__ void add_to(float (&s)[8]) const {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if constexpr (kType == VLPROJ_F32) {
                s[2 * q] += __uint_as_float(v[q].x);
                s[2 * q + 1] += __uint_as_float(v[q].y);
            } else {
                const T* e = reinterpret_cast<const T*>(&v[q]);
                s[2 * q] += Elem<kType>::up(e[0]);
                s[2 * q + 1] += Elem<kType>::up(e[1]);
            }
        }
    }
};
template <int kType>
struct SumRow<kType, 1> {
    using T = typename Elem<kType>::T;
    T v[4];
    __device__ __forceinline__ void load(const T* row, const int (&col)[4]) {
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = __ldg(row + col[q]);
    }
    __device__ __forceinline__ void add_to(float (&s)[4]) const {
#pragma unroll
        for (int q = 0; q < 4; ++q) s[q] += Elem<kType>::up(v[q]);
    }
};

// First column of each access of thread j of a group of `threads`, the first one's where it
// lies past N; false when the thread has none.
template <int kWidth>
__device__ __forceinline__ bool sum_columns(int c0, int j, int threads, int N, int (&col)[sum_accesses<kWidth>()]) {
    const int first = c0 + j * kWidth;
#pragma unroll
    for (int q = 0; q < sum_accesses<kWidth>(); ++q) {
        const int c = first + q * threads * kWidth;
        col[q] = c < N ? c : first;
    }
    return first < N;
}

// dst[columns] = (add: itself +) s * scale.
template <int kWidth>
__device__ __forceinline__ void sum_write(float* dst, const int (&col)[sum_accesses<kWidth>()],
                                          const float (&s)[sum_cols<kWidth>()], float scale, bool add) {
    if constexpr (kWidth == 8) {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = s[e] * scale;
        if (add) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] += dst[col[0] + e];
        }
        store8<VLPROJ_F32>(dst + col[0], pack8<VLPROJ_F32>(f));
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (q > 0 && col[q] == col[0]) continue;
            if constexpr (kWidth == 2) {
                float2 v = make_float2(s[2 * q] * scale, s[2 * q + 1] * scale);
                float2* p = reinterpret_cast<float2*>(dst + col[q]);
                if (add) {
                    const float2 u = *p;
                    v = make_float2(u.x + v.x, u.y + v.y);
                }
                *p = v;
            } else {
                dst[col[q]] = (add ? dst[col[q]] : 0.f) + s[q] * scale;
            }
        }
    }
}

// First place in [lo, hi) whose key is not below `key` (hi if none).
__device__ __forceinline__ int64_t lower_bound_key(const uint64_t* pairs, int64_t lo, int64_t hi, uint64_t key) {
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if ((pairs[mid] >> 32) < key) lo = mid + 1; else hi = mid;
    }
    return lo;
}

// Zeros in row[0 .. N), by threads j < kThreads: the first elements up to a 32-byte boundary
// and the last ones singly, those between in 32-byte stores.
template <int kThreads>
__device__ __forceinline__ void zero_row(float* row, int N, int j) {
    Raw8<VLPROJ_F32> z;
    z.w[0] = z.w[1] = make_uint4(0, 0, 0, 0);
    int head = static_cast<int>((-reinterpret_cast<uintptr_t>(row) & 31) / 4);
    head = head < N ? head : N;
    const int body = head + ((N - head) & ~7);
    for (int c = head + 8 * j; c < body; c += 8 * kThreads) store8<VLPROJ_F32>(row + c, z);
    const int c = j < 8 ? j : body + j - 8;
    if (j < 8 ? c < head : c < N) row[c] = 0.f;
}

// Zero rows of the tokens t0 + b for the set bits b of `absent`, by a block of SUM_THREADS:
// narrow rows a warp each (2500 x 128 bf16 into 102400 rows: 50 us by blocks, 37 us so).
__device__ __forceinline__ void zero_rows(const ScatterOut& o, int64_t t0, unsigned absent) {
    if (o.N <= 512) {
        for (int k = threadIdx.x >> 5; absent != 0; --k) {
            const int b = __ffs(absent) - 1;
            absent &= absent - 1;
            if (k % (SUM_THREADS / 32) == 0) zero_row<32>(o.d_table + (t0 + b) * o.ld, o.N, threadIdx.x & 31);
        }
    } else {
        while (absent != 0) {
            const int b = __ffs(absent) - 1;
            absent &= absent - 1;
            zero_row<SUM_THREADS>(o.d_table + (t0 + b) * o.ld, o.N, threadIdx.x);
        }
    }
}

// Blocks 0 .. sums - 1: chunks kGroups * (b / tiles) .., column tile b % tiles; the others:
// zero rows.
template <int kType, int kWidth, int kGroups>
static __global__ void __launch_bounds__(SUM_THREADS) vlp_scatter_sum_kernel(const uint64_t* pairs, int64_t n, int rows,
                                                                             int tiles, unsigned sums,
                                                                             const void* __restrict__ d_out,
                                                                             int64_t d_out_ld, ScatterOut o,
                                                                             float* part) {
    using T = typename Elem<kType>::T;
    constexpr int THREADS = SUM_THREADS / kGroups;      // of a group
    __shared__ uint32_t keys[kGroups][SUM_MAX_ROWS + 2];      // keys of rows -1 .. rows of the chunk
    __shared__ uint32_t positions[kGroups][SUM_MAX_ROWS];
    const uint32_t vocab = static_cast<uint32_t>(o.vocab);
    after_previous_kernel(pairs);
    let_next_kernel_start();
    if (blockIdx.x >= sums) {
        const int64_t t0 = static_cast<int64_t>(blockIdx.x - sums) * ZERO_TOKENS;
        if (threadIdx.x < 32) {
            const int64_t t = t0 + threadIdx.x;
            bool absent = false;
            if (t < o.vocab) {
                const int64_t i = lower_bound_key(pairs, 0, n, static_cast<uint64_t>(t));
                absent = i >= n || static_cast<int64_t>(pairs[i] >> 32) != t;
            }
            const unsigned todo = __ballot_sync(0xffffffffu, absent);
            if (threadIdx.x == 0) keys[0][0] = todo;
        }
        __syncthreads();
        zero_rows(o, t0, keys[0][0]);
        return;
    }
    const int g = threadIdx.x / THREADS, j = threadIdx.x % THREADS;
    uint32_t* key = keys[g];
    uint32_t* pos = positions[g];
    const int64_t chunk = static_cast<int64_t>(blockIdx.x / tiles) * kGroups + g;
    const int64_t i0 = chunk * rows;
    const int m = static_cast<int>(i0 >= n ? 0 : i0 + rows < n ? rows : n - i0);
    for (int i = j - 1; i <= m; i += THREADS) {
        const int64_t at = i0 + i;
        const uint64_t e = at >= 0 && at < n ? pairs[at] : ~0ull;
        key[i + 1] = static_cast<uint32_t>(e >> 32);
        if (i >= 0 && i < m) pos[i] = static_cast<uint32_t>(e);
    }
    __syncthreads();
    int col[sum_accesses<kWidth>()];
    const int c0 = static_cast<int>(blockIdx.x % tiles) * THREADS * sum_cols<kWidth>();
    if (!sum_columns<kWidth>(c0, j, THREADS, o.N, col)) return;
    float s[sum_cols<kWidth>()];
#pragma unroll
    for (int e = 0; e < sum_cols<kWidth>(); ++e) s[e] = 0.f;
    bool earlier = key[0] == key[1];                // the run at hand began in an earlier chunk
    for (int i = 0; i < m && key[i + 1] < vocab; i += SUM_BATCH) {
        SumRow<kType, kWidth> v[SUM_BATCH];
#pragma unroll
        for (int b = 0; b < SUM_BATCH; ++b) {
            // past the chunk's last row that counts: the batch's first row again, not added
            const int r = i + b < m && key[i + b + 1] < vocab ? i + b : i;
            v[b].load(static_cast<const T*>(d_out) + pos[r] * d_out_ld, col);
        }
#pragma unroll
        for (int b = 0; b < SUM_BATCH; ++b) {
            const int r = i + b;
            const uint32_t k = r < m ? key[r + 1] : vocab;
            if (k >= vocab) break;
            v[b].add_to(s);
            const bool ends = key[r + 2] != k;
            if (!ends && r + 1 < m) continue;
            if (ends && !earlier)
                sum_write<kWidth>(o.d_table + static_cast<int64_t>(k) * o.ld, col, s, o.scale, o.accumulate);
            else
                sum_write<kWidth>(part + (2 * chunk + (earlier ? 0 : 1)) * o.N, col, s, 1.f, false);
#pragma unroll
            for (int e = 0; e < sum_cols<kWidth>(); ++e) s[e] = 0.f;
            earlier = false;
        }
    }
}

// One block per chunk and tile of columns: the run that begins in the chunk and goes on
// past it has its first part in the chunk's slot 1 and the others in slot 0 of the
// following chunks up to the one its last row lies in. kGroups groups of threads, more for
// narrow rows, each add every kGroups-th of them in order, in fp64, JOIN_BATCH loads in
// flight, and the groups' sums are added in order. Most blocks find no such run and end at
// once.
constexpr int JOIN_THREADS = 256;
constexpr int JOIN_BATCH = 8;
template <int kGroups>
static __global__ void __launch_bounds__(JOIN_THREADS) vlp_scatter_join_kernel(const uint64_t* pairs, int64_t n,
                                                                               int rows, int tiles, const float* part,
                                                                               ScatterOut o) {
    constexpr int THREADS = JOIN_THREADS / kGroups;          // of a group, 4 columns each
    __shared__ double sums[kGroups > 1 ? kGroups : 1][kGroups > 1 ? 4 * THREADS : 1];
    const int g = threadIdx.x / THREADS, j = threadIdx.x % THREADS;
    const int64_t chunk = blockIdx.x / tiles;
    const int c0 = static_cast<int>(blockIdx.x % tiles) * 4 * THREADS + j;
    const int64_t i0 = chunk * rows, i1 = i0 + rows;                   // i1 < n: the last chunk has no block
    after_previous_kernel(pairs, part);
    const uint64_t before = pairs[i0 > 0 ? i0 - 1 : 0], end = pairs[i1 - 1], next = pairs[i1];
    const uint32_t k = static_cast<uint32_t>(end >> 32);
    if (k >= o.vocab || static_cast<uint32_t>(next >> 32) != k) return;               // ends here
    if (i0 > 0 && static_cast<uint32_t>(before >> 32) == k) return;                     // began earlier
    // its last chunk: the first of the following ones whose last row has another key (or is
    // the last of all), the one before where the run ended with that chunk. The lanes of
    // every warp try the next 32, and then 32 at a time of those left, evenly spread.
    const auto past = [&](int64_t q) {
        const int64_t e = (q + 1) * rows - 1;
        return e >= n - 1 || static_cast<uint32_t>(pairs[e < n ? e : n - 1] >> 32) != k;
    };
    const int lane = threadIdx.x & 31;
    int64_t last = chunk + 1, step = 1, high = (n - 1) / rows;         // past(high) holds
    for (;;) {
        const int64_t q = last + lane * step;
        const unsigned stop = __ballot_sync(0xffffffffu, past(q < high ? q : high));
        const int f = stop != 0 ? __ffs(stop) - 1 : 32;
        if (f < 32) high = last + f * step < high ? last + f * step : high;
        if (f > 0) last += (f - 1) * step + 1;                        // the last one tried that does not hold, and one
        if (last >= high) break;
        step = (high - last) / 32 + 1;
    }
    last = high;
    if (static_cast<uint32_t>(pairs[last * rows] >> 32) != k) --last;
    int col[4];
    double s[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int c = c0 + THREADS * e;
        col[e] = c < o.N ? c : o.N - 1;
        s[e] = g == 0 ? part[(2 * chunk + 1) * o.N + col[e]] : 0.;
    }
    for (int64_t q = chunk + 1 + g; q <= last; q += JOIN_BATCH * kGroups) {
        float v[JOIN_BATCH][4];
#pragma unroll
        for (int b = 0; b < JOIN_BATCH; ++b) {
            const float* p = part + 2 * (q + b * kGroups <= last ? q + b * kGroups : q) * o.N;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[b][e] = p[col[e]];
        }
#pragma unroll
        for (int b = 0; b < JOIN_BATCH; ++b)
            if (q + b * kGroups <= last) {
#pragma unroll
                for (int e = 0; e < 4; ++e) s[e] += v[b][e];
            }
    }
    if constexpr (kGroups > 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sums[g][j + THREADS * e] = s[e];
        __syncthreads();
        if (g != 0) return;
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int h = 1; h < kGroups; ++h) s[e] += sums[h][j + THREADS * e];
    }
    float* row = o.d_table + static_cast<int64_t>(k) * o.ld;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int c = c0 + THREADS * e;
        if (c < o.N) row[c] = (o.accumulate ? row[c] : 0.f) + static_cast<float>(s[e] * o.scale);
    }
}

// ---------------------------------------------------------------- few ids
// Up to SMALL_MAX_IDS ids in one launch without sorting (200 x 128 bf16 into 1000 rows: a
// kernel of 5 us; 512 x 4096 into 1000 rows 17 us a call, floor 3 us, since 32 blocks write the
// zero rows, 512 KB each, on 148 SMs): block (i, column tile) finds the
// positions that hold id i by comparing all ids, ends when an earlier position holds it
// too, and else adds their rows in order. The n^2 comparisons are at most 16 KB of cached
// ids a block. The other blocks write the zero rows, ZERO_TOKENS tokens each.
constexpr int SMALL_MAX_IDS = 2048;
template <int kType, int kWidth>
static __global__ void __launch_bounds__(SUM_THREADS) vlp_scatter_few_kernel(const int64_t* __restrict__ ids, int n,
                                                                             int64_t token, int tiles, unsigned sums,
                                                                             const void* __restrict__ d_out,
                                                                             int64_t d_out_ld, ScatterOut o,
                                                                             int* status) {
    using T = typename Elem<kType>::T;
    constexpr int WORDS = SMALL_MAX_IDS / 32;
    __shared__ unsigned found[WORDS];               // bit i % 32 of word i / 32: position i holds the id
    __shared__ int first[WORDS];                    // found bits of earlier words
    __shared__ uint16_t list[SMALL_MAX_IDS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x >= sums) {
        const int64_t t0 = static_cast<int64_t>(blockIdx.x - sums) * ZERO_TOKENS;
        if (threadIdx.x == 0) found[0] = 0;
        __syncthreads();
        unsigned here = 0;
#pragma unroll
        for (int q = 0; q < SMALL_MAX_IDS / SUM_THREADS; ++q) {
            const int i = threadIdx.x + q * SUM_THREADS;
            const int64_t id = n > 0 ? __ldg(ids + (i < n ? i : 0)) : token;
            if (id != token && id >= t0 && id < t0 + ZERO_TOKENS) here |= 1u << static_cast<int>(id - t0);
        }
        here = __reduce_or_sync(0xffffffffu, here);
        if (lane == 0 && here != 0) atomicOr(&found[0], here);
        __syncthreads();
        const int64_t left = o.vocab - t0;
        zero_rows(o, t0, ~found[0] & (left >= 32 ? ~0u : (1u << static_cast<int>(left)) - 1u));
        return;
    }
    const int mine = static_cast<int>(blockIdx.x / tiles);
    const int tile = static_cast<int>(blockIdx.x % tiles);
    const int64_t t = __ldg(ids + mine);
    if (placeholder(t, token)) return;
    if (t < 0 || t >= o.vocab) {
        if (tile == 0 && threadIdx.x == 0 && status != nullptr) atomicCAS(status, VLPROJ_OK, VLPROJ_ERR_INVALID_ARG);
        return;
    }
#pragma unroll
    for (int q = 0; q < SMALL_MAX_IDS / SUM_THREADS; ++q) {
        const int i = threadIdx.x + q * SUM_THREADS;
        const unsigned f = __ballot_sync(0xffffffffu, __ldg(ids + (i < n ? i : 0)) == t && i < n);
        if (lane == 0) found[warp + q * (SUM_THREADS / 32)] = f;
    }
    __syncthreads();
    if (warp == 0) {                                // two words a lane
        static_assert(WORDS == 64, "two words a lane");
        const int c0 = __popc(found[2 * lane]), c1 = __popc(found[2 * lane + 1]);
        int inc = c0 + c1;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += v;
        }
        first[2 * lane] = inc - c1 - c0;
        first[2 * lane + 1] = inc - c1;
    }
    __syncthreads();
    if (first[mine / 32] != 0 || (found[mine / 32] & ((1u << (mine % 32)) - 1u)) != 0) return;      // not the first
#pragma unroll
    for (int q = 0; q < SMALL_MAX_IDS / SUM_THREADS; ++q) {
        const int w = warp + q * (SUM_THREADS / 32);
        const unsigned f = found[w];
        if ((f >> lane) & 1u) list[first[w] + __popc(f & ((1u << lane) - 1u))] = static_cast<uint16_t>(32 * w + lane);
    }
    __syncthreads();
    const int count = first[WORDS - 1] + __popc(found[WORDS - 1]);
    int col[sum_accesses<kWidth>()];
    if (!sum_columns<kWidth>(tile * SUM_THREADS * sum_cols<kWidth>(), threadIdx.x, SUM_THREADS, o.N, col)) return;
    float s[sum_cols<kWidth>()];
#pragma unroll
    for (int e = 0; e < sum_cols<kWidth>(); ++e) s[e] = 0.f;
    for (int i = 0; i < count; i += SUM_BATCH) {
        SumRow<kType, kWidth> v[SUM_BATCH];
#pragma unroll
        for (int b = 0; b < SUM_BATCH; ++b)
            v[b].load(static_cast<const T*>(d_out) + list[i + b < count ? i + b : i] * d_out_ld, col);
#pragma unroll
        for (int b = 0; b < SUM_BATCH; ++b)
            if (i + b < count) v[b].add_to(s);
    }
    sum_write<kWidth>(o.d_table + t * o.ld, col, s, o.scale, o.accumulate);
}

}  // namespace vlp_ops
