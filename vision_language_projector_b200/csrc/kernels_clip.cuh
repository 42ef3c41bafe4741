// Global norm of many gradient tensors and the gradients clipped by it (sm_100a). Memory
// traffic bounds it: every gradient is read for the norm, and read again and written for
// the clipping. 40 M fp32 gradients, 160 MB: 76 to 80 us, in which 430 MB move (5.4 TB/s): the
// L2 cache still holds about 50 MB of the second read. Tensors off a 32-byte boundary go
// element by element: the same gradients one element off 201 us, their norm alone 34 us
// (aligned 30).
#pragma once
#include <cooperative_groups.h>

#include "ops_common.cuh"

namespace vlp_ops {

constexpr int CLIP_THREADS = 256;
constexpr int CLIP_WORDS = 4;                                    // 32-byte words of a thread in a chunk
constexpr int CLIP_CHUNK = 32 * CLIP_WORDS * CLIP_THREADS;       // bytes of one tensor a block takes at a time
constexpr int CLIP_BLOCKS_PER_SM = 3;
constexpr int CLIP_MAX_BLOCKS = 148 * CLIP_BLOCKS_PER_SM;        // per table

// Tensors of one launch, passed by value as the kernel's argument, so that a call copies
// nothing to the device and can be captured. first[i]: chunks of the tensors before i.
template <int kMax>
struct ClipTable {
    const void* grad[kMax];
    void* out[kMax];
    int64_t numel[kMax];
    int32_t first[kMax + 1];
    uint8_t type[kMax];
    int32_t n;
};

// One chunk: `bytes` of it from `grad` (and to `out`), the first `words` 32-byte words of
// which are aligned; the elements behind them are taken singly.
struct ClipPiece {
    const char* grad;
    char* out;
    int bytes, words, type;
    bool skip;
};

template <int kMax>
__device__ __forceinline__ ClipPiece clip_piece(const ClipTable<kMax>& t, int chunk) {
    int lo = 0, hi = t.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= chunk) lo = mid; else hi = mid - 1;
    }
    ClipPiece p;
    p.type = t.type[lo];
    const int64_t b0 = static_cast<int64_t>(chunk - t.first[lo]) * CLIP_CHUNK;
    const int64_t left = t.numel[lo] * (p.type == VLPROJ_F32 ? 4 : 2) - b0;
    p.bytes = static_cast<int>(left < CLIP_CHUNK ? left : CLIP_CHUNK);
    p.grad = static_cast<const char*>(t.grad[lo]) + b0;
    p.out = static_cast<char*>(t.out[lo]) + b0;
    const bool aligned = ((reinterpret_cast<uintptr_t>(t.grad[lo]) | reinterpret_cast<uintptr_t>(t.out[lo])) & 31) == 0;
    p.words = aligned ? p.bytes / 32 : 0;
    p.skip = t.grad[lo] == t.out[lo];
    return p;
}

// The thread's words of a chunk, all loads issued at once; those past the chunk's words
// repeat its first one and are not used. A plain load: the same thread may write the words
// later.
struct ClipWords {
    uint32_t v[CLIP_WORDS][8];
    __device__ __forceinline__ void load(const ClipPiece& p) {
        if (p.words == 0) return;
#pragma unroll
        for (int q = 0; q < CLIP_WORDS; ++q) {
            const int w = static_cast<int>(threadIdx.x) + q * CLIP_THREADS;
            asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(v[q][0]), "=r"(v[q][1]), "=r"(v[q][2]), "=r"(v[q][3]), "=r"(v[q][4]), "=r"(v[q][5]),
                           "=r"(v[q][6]), "=r"(v[q][7])
                         : "l"(p.grad + 32 * (w < p.words ? w : 0))
                         : "memory");
        }
    }
};

// 8 elements of a word: half h (0 or 1) of a 2-byte type's 16, or all of fp32's 8.
template <int kType>
__device__ __forceinline__ void clip_unpack(const uint32_t (&v)[8], int h, float (&f)[8]) {
    Raw8<kType> r;
    if constexpr (kType == VLPROJ_F32) {
        r.w[0] = make_uint4(v[0], v[1], v[2], v[3]);
        r.w[1] = make_uint4(v[4], v[5], v[6], v[7]);
    } else {
        r.w[0] = make_uint4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
    }
    unpack8<kType>(r, f);
}

// Sum of 8 squares: in fp32 where that neither overflows nor loses what matters, else in
// fp64 (a square of an fp32 value fits there exactly).
__device__ __forceinline__ double squares8(const float (&f)[8]) {
    float q = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) q = fmaf(f[e], f[e], q);
    if (q >= 1e-30f && q <= 1e30f) return static_cast<double>(q);
    double d = 0.;
#pragma unroll
    for (int e = 0; e < 8; ++e) d = fma(static_cast<double>(f[e]), static_cast<double>(f[e]), d);
    return d;
}

template <int kType>
__device__ __forceinline__ double clip_squares(const ClipPiece& p, const ClipWords& words) {
    using T = typename Elem<kType>::T;
    constexpr int HALVES = kType == VLPROJ_F32 ? 1 : 2;
    double acc = 0.;
#pragma unroll
    for (int q = 0; q < CLIP_WORDS; ++q) {
        if (static_cast<int>(threadIdx.x) + q * CLIP_THREADS >= p.words) break;
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
            float f[8];
            clip_unpack<kType>(words.v[q], h, f);
            acc += squares8(f);
        }
    }
    const T* g = reinterpret_cast<const T*>(p.grad);
    const int n = p.bytes / static_cast<int>(sizeof(T));
    for (int e = p.words * (32 / static_cast<int>(sizeof(T))) + threadIdx.x; e < n; e += CLIP_THREADS) {
        const double v = Elem<kType>::up(g[e]);
        acc = fma(v, v, acc);
    }
    return acc;
}

// Sum over the block in a fixed order.
__device__ __forceinline__ double block_add(double v, double* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    double s = 0.;
#pragma unroll
    for (int w = 0; w < CLIP_THREADS / 32; ++w) s += red[w];
    return s;
}

// part[block] = the block's share of the sum of squares. The next chunk's words are on
// their way while one is added.
template <int kMax>
static __global__ void __launch_bounds__(CLIP_THREADS, CLIP_BLOCKS_PER_SM) vlp_clip_norm_kernel(
    const __grid_constant__ ClipTable<kMax> t, double* __restrict__ part) {
    __shared__ double red[CLIP_THREADS / 32];
    const int chunks = t.first[t.n];
    double acc = 0.;
    int k = blockIdx.x;
    if (k < chunks) {
        ClipPiece p = clip_piece(t, k);
        ClipWords words;
        words.load(p);
        for (;;) {
            ClipPiece next = p;
            ClipWords coming;
            const bool more = k + static_cast<int>(gridDim.x) < chunks;
            if (more) {
                next = clip_piece(t, k + gridDim.x);
                coming.load(next);
            }
            if (p.type == VLPROJ_F32) acc += clip_squares<VLPROJ_F32>(p, words);
            else if (p.type == VLPROJ_BF16) acc += clip_squares<VLPROJ_BF16>(p, words);
            else acc += clip_squares<VLPROJ_F16>(p, words);
            if (!more) break;
            k += gridDim.x;
            p = next;
            words = coming;
        }
    }
    let_next_kernel_start();
    const double s = block_add(acc, red);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// The coefficient in fp32, or, where it would lose bits there, in fp64.
template <bool kTiny>
__device__ __forceinline__ float clip_one(float g, double coef) {
    if constexpr (kTiny) return static_cast<float>(static_cast<double>(g) * coef);
    return g * static_cast<float>(coef);
}

template <int kType, bool kTiny>
__device__ __forceinline__ void clip_scale(const ClipPiece& p, const ClipWords& words, double coef) {
    using T = typename Elem<kType>::T;
    constexpr int HALVES = kType == VLPROJ_F32 ? 1 : 2;
#pragma unroll
    for (int q = 0; q < CLIP_WORDS; ++q) {
        const int w = static_cast<int>(threadIdx.x) + q * CLIP_THREADS;
        if (w >= p.words) break;
        Raw8<VLPROJ_F32> r;
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
            float f[8];
            clip_unpack<kType>(words.v[q], h, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = clip_one<kTiny>(f[i], coef);
            const Raw8<kType> half = pack8<kType>(f);
            r.w[h] = half.w[0];
            if constexpr (kType == VLPROJ_F32) r.w[1] = half.w[1];
        }
        store8_once<VLPROJ_F32>(p.out + 32 * w, r);                   // the word's 32 bytes
    }
    const T* g = reinterpret_cast<const T*>(p.grad);
    T* o = reinterpret_cast<T*>(p.out);
    const int n = p.bytes / static_cast<int>(sizeof(T));
    for (int e = p.words * (32 / static_cast<int>(sizeof(T))) + threadIdx.x; e < n; e += CLIP_THREADS)
        o[e] = Elem<kType>::down(clip_one<kTiny>(Elem<kType>::up(g[e]), coef));
}

template <bool kTiny>
__device__ __forceinline__ void clip_scale_typed(const ClipPiece& p, const ClipWords& words, double coef) {
    if (p.type == VLPROJ_F32) clip_scale<VLPROJ_F32, kTiny>(p, words, coef);
    else if (p.type == VLPROJ_BF16) clip_scale<VLPROJ_BF16, kTiny>(p, words, coef);
    else clip_scale<VLPROJ_F16, kTiny>(p, words, coef);
}

__device__ __forceinline__ double clip_coef(double max_norm, double norm) {
    const double coef = max_norm / (norm + 1e-6);
    return coef >= 1. ? 1. : coef;                    // a NaN stays
}

// Every block adds the nparts partial sums in the same order; block 0 writes the norm
// (when given), then all scale their chunks (when the table has outputs), the last ones
// first: of gradients larger than the L2 cache those are still there from the norm. The
// first chunk's words are loaded before the norm is known.
template <int kMax>
static __global__ void __launch_bounds__(CLIP_THREADS, CLIP_BLOCKS_PER_SM) vlp_clip_scale_kernel(
    const __grid_constant__ ClipTable<kMax> t, const double* part, int nparts, double max_norm, float* norm, int scale) {
    __shared__ double red[CLIP_THREADS / 32];
    int k = t.first[t.n] - 1 - static_cast<int>(blockIdx.x);
    ClipPiece p;
    ClipWords words;
    if (scale && k >= 0) {
        p = clip_piece(t, k);
        words.load(p);
    }
    double v = 0.;
    after_previous_kernel(part);
    for (int i = threadIdx.x; i < nparts; i += CLIP_THREADS) v += part[i];
    const double total = sqrt(block_add(v, red));
    if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(total);
    if (!scale || k < 0) return;
    const double coef = clip_coef(max_norm, total);
    for (;;) {
        ClipPiece next = p;
        ClipWords coming;
        const bool more = k - static_cast<int>(gridDim.x) >= 0;
        if (more) {
            next = clip_piece(t, k - gridDim.x);
            coming.load(next);
        }
        if (!(coef == 1. && p.skip)) {
            if (coef < 1e-30) clip_scale_typed<true>(p, words, coef);
            else clip_scale_typed<false>(p, words, coef);
        }
        if (!more) break;
        k -= gridDim.x;
        p = next;
        words = coming;
    }
}

// ---------------------------------------------------------------- few gradients
// The whole step in one launch and without a workspace: one cluster of CLIP_CLUSTER blocks,
// which read one another's share of the sum from shared memory. The last chunk of a block
// stays in its registers between the norm and the scaling. It saves a call from Python, one
// after another, the workspace and a launch: 12.5 us so and 16.0 us by the two launches for
// 262144 fp32 elements of 6 tensors, 10.2 and 11.6 us of one. On the GPU one cluster takes
// longer than the grid of the two launches: replayed in a graph 9.7 and 4.3 us, 7.8 and 4.1 us
// (1000 elements: 2.8 and 3.0 us). More elements lose from Python too.
constexpr int CLIP_CLUSTER = 8;
template <int kMax>
static __global__ void __cluster_dims__(CLIP_CLUSTER, 1, 1) __launch_bounds__(CLIP_THREADS) vlp_clip_few_kernel(
    const __grid_constant__ ClipTable<kMax> t, double max_norm, float* norm, int scale) {
    __shared__ double red[CLIP_THREADS / 32];
    __shared__ double share;
    auto cluster = cooperative_groups::this_cluster();
    const int chunks = t.first[t.n];
    int k = blockIdx.x;
    double acc = 0.;
    ClipPiece p;
    ClipWords words;
    for (; k < chunks; k += CLIP_CLUSTER) {
        p = clip_piece(t, k);
        words.load(p);
        if (p.type == VLPROJ_F32) acc += clip_squares<VLPROJ_F32>(p, words);
        else if (p.type == VLPROJ_BF16) acc += clip_squares<VLPROJ_BF16>(p, words);
        else acc += clip_squares<VLPROJ_F16>(p, words);
    }
    acc = block_add(acc, red);
    if (threadIdx.x == 0) share = acc;
    cluster.sync();
    double total = 0.;
#pragma unroll
    for (int b = 0; b < CLIP_CLUSTER; ++b) total += *cluster.map_shared_rank(&share, b);
    cluster.sync();                                  // no block ends while another reads its share
    total = sqrt(total);
    if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(total);
    if (!scale) return;
    const double coef = clip_coef(max_norm, total);
    bool held = true;                                // the last chunk's words
    for (k -= CLIP_CLUSTER; k >= 0; k -= CLIP_CLUSTER) {
        if (!held) {
            p = clip_piece(t, k);
            words.load(p);
        }
        held = false;
        if (coef == 1. && p.skip) continue;
        if (coef < 1e-30) clip_scale_typed<true>(p, words, coef);
        else clip_scale_typed<false>(p, words, coef);
    }
}

}  // namespace vlp_ops
