// Global norm of many gradient tensors and the gradients clipped by it (sm_100a). Memory
// traffic bounds it: every gradient is read for the norm, and read again and written for
// the clipping.
#pragma once
#include "ops_common.cuh"

namespace vlp_ops {

constexpr int CLIP_THREADS = 256;
constexpr int CLIP_CHUNK = 8192;          // elements of one tensor a block takes at a time
constexpr int CLIP_MAX_BLOCKS = 592;      // per table

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

template <int kMax>
__device__ __forceinline__ int clip_find(const ClipTable<kMax>& t, int chunk) {
    int lo = 0, hi = t.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= chunk) lo = mid; else hi = mid - 1;
    }
    return lo;
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
__device__ __forceinline__ double clip_chunk_squares(const void* grad, int64_t e0, int64_t e1) {
    using T = typename Elem<kType>::T;
    const T* g = static_cast<const T*>(grad);
    double acc = 0.;
    if (reinterpret_cast<uintptr_t>(g) % 16 == 0) {
        const int64_t full = e0 + ((e1 - e0) & ~int64_t(7));
#pragma unroll 4
        for (int64_t e = e0 + 8 * threadIdx.x; e < full; e += 8 * CLIP_THREADS) {
            float f[8];
            unpack8<kType>(load8<kType>(g + e), f);
            acc += squares8(f);
        }
        e0 = full;
    }
#pragma unroll 4
    for (int64_t e = e0 + threadIdx.x; e < e1; e += CLIP_THREADS) {
        const double v = Elem<kType>::up(__ldg(g + e));
        acc = fma(v, v, acc);
    }
    return acc;
}

// Sum over the block in a fixed order, given to thread 0.
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

// part[block] = the block's share of the sum of squares.
template <int kMax>
static __global__ void __launch_bounds__(CLIP_THREADS) vlp_clip_norm_kernel(const __grid_constant__ ClipTable<kMax> t,
                                                                            double* __restrict__ part) {
    __shared__ double red[CLIP_THREADS / 32];
    const int chunks = t.first[t.n];
    double acc = 0.;
    for (int k = blockIdx.x; k < chunks; k += gridDim.x) {
        const int i = clip_find(t, k);
        const int64_t e0 = static_cast<int64_t>(k - t.first[i]) * CLIP_CHUNK;
        const int64_t e1 = e0 + CLIP_CHUNK < t.numel[i] ? e0 + CLIP_CHUNK : t.numel[i];
        if (t.type[i] == VLPROJ_F32) acc += clip_chunk_squares<VLPROJ_F32>(t.grad[i], e0, e1);
        else if (t.type[i] == VLPROJ_BF16) acc += clip_chunk_squares<VLPROJ_BF16>(t.grad[i], e0, e1);
        else acc += clip_chunk_squares<VLPROJ_F16>(t.grad[i], e0, e1);
    }
    const double s = block_add(acc, red);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

struct ClipCoef {
    double exact;
    float coef;
    bool tiny;       // coef loses bits in fp32: multiply in fp64
};

__device__ __forceinline__ float clip_one(float g, const ClipCoef& c) {
    return c.tiny ? static_cast<float>(static_cast<double>(g) * c.exact) : g * c.coef;
}

template <int kType>
__device__ __forceinline__ void clip_chunk_scale(const void* grad, void* out, int64_t e0, int64_t e1,
                                                 const ClipCoef& c) {
    using T = typename Elem<kType>::T;
    const T* g = static_cast<const T*>(grad);
    T* o = static_cast<T*>(out);
    if (reinterpret_cast<uintptr_t>(g) % 16 == 0 && reinterpret_cast<uintptr_t>(o) % 16 == 0) {
        const int64_t full = e0 + ((e1 - e0) & ~int64_t(7));
#pragma unroll 4
        for (int64_t e = e0 + 8 * threadIdx.x; e < full; e += 8 * CLIP_THREADS) {
            Raw8<kType> r;
            r.w[0] = *reinterpret_cast<const uint4*>(g + e);         // may be rewritten below: a plain load
            if constexpr (kType == VLPROJ_F32) r.w[1] = *reinterpret_cast<const uint4*>(g + e + 4);
            float f[8];
            unpack8<kType>(r, f);
#pragma unroll
            for (int q = 0; q < 8; ++q) f[q] = clip_one(f[q], c);
            store8<kType>(o + e, pack8<kType>(f));
        }
        e0 = full;
    }
#pragma unroll 4
    for (int64_t e = e0 + threadIdx.x; e < e1; e += CLIP_THREADS) o[e] = Elem<kType>::down(clip_one(Elem<kType>::up(g[e]), c));
}

// Every block adds the nparts partial sums in the same order; block 0 writes the norm
// (when given), then all scale their chunks (when the table has outputs).
template <int kMax>
static __global__ void __launch_bounds__(CLIP_THREADS) vlp_clip_scale_kernel(const __grid_constant__ ClipTable<kMax> t,
                                                                             const double* __restrict__ part,
                                                                             int nparts, double max_norm, float* norm,
                                                                             int scale) {
    __shared__ double red[CLIP_THREADS / 32];
    double v = 0.;
    for (int i = threadIdx.x; i < nparts; i += CLIP_THREADS) v += part[i];
    const double total = sqrt(block_add(v, red));
    if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(total);
    if (!scale) return;
    ClipCoef c;
    c.exact = max_norm / (total + 1e-6);
    if (c.exact >= 1.) c.exact = 1.;                  // a NaN stays
    c.coef = static_cast<float>(c.exact);
    c.tiny = c.exact < 1e-30;
    const int chunks = t.first[t.n];
    for (int k = blockIdx.x; k < chunks; k += gridDim.x) {
        const int i = clip_find(t, k);
        if (c.exact == 1. && t.out[i] == t.grad[i]) continue;
        const int64_t e0 = static_cast<int64_t>(k - t.first[i]) * CLIP_CHUNK;
        const int64_t e1 = e0 + CLIP_CHUNK < t.numel[i] ? e0 + CLIP_CHUNK : t.numel[i];
        if (t.type[i] == VLPROJ_F32) clip_chunk_scale<VLPROJ_F32>(t.grad[i], t.out[i], e0, e1, c);
        else if (t.type[i] == VLPROJ_BF16) clip_chunk_scale<VLPROJ_BF16>(t.grad[i], t.out[i], e0, e1, c);
        else clip_chunk_scale<VLPROJ_F16>(t.grad[i], t.out[i], e0, e1, c);
    }
}

}  // namespace vlp_ops
