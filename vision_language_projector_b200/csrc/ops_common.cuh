// Shared pieces of the operators around the projector (embedding lookup and gradient,
// layer norm, gradient clipping): element types, 8-element loads and stores, warp sums.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>
#include <type_traits>

#include "../../include/vlproj.h"
#include "ptx.cuh"

namespace vlp_ops {

// Element types by their VLPROJ_* code: conversion to and from fp32. The conversion from
// fp32 is the one rounding (to nearest even) of every result these operators write.
template <int kType>
struct Elem;
template <>
struct Elem<VLPROJ_BF16> {
    using T = __nv_bfloat16;
    static __device__ __forceinline__ float up(T v) { return __bfloat162float(v); }
    static __device__ __forceinline__ T down(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<VLPROJ_F32> {
    using T = float;
    static __device__ __forceinline__ float up(T v) { return v; }
    static __device__ __forceinline__ T down(float v) { return v; }
};
template <>
struct Elem<VLPROJ_F16> {
    using T = __half;
    static __device__ __forceinline__ float up(T v) { return __half2float(v); }
    static __device__ __forceinline__ T down(float v) { return __float2half_rn(v); }
};

inline int64_t type_size(int t) { return t == VLPROJ_F32 ? 4 : 2; }

// The bits of 8 consecutive elements: one 16-byte word of a 2-byte type, two of fp32.
template <int kType>
struct Raw8 {
    uint4 w[kType == VLPROJ_F32 ? 2 : 1];
};

// Loads and stores of 8 elements, aligned to their 16 (fp32: 32) bytes. Each is one access:
// two 16-byte accesses of fp32, 32 bytes apart across a warp, would touch every 32-byte
// sector twice. store8_once: data not read again by the call, marked to leave the caches
// first.
template <int kType>
__device__ __forceinline__ Raw8<kType> load8(const void* p) {
    Raw8<kType> r;
    if constexpr (kType == VLPROJ_F32)
        asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
            : "=r"(r.w[0].x), "=r"(r.w[0].y), "=r"(r.w[0].z), "=r"(r.w[0].w), "=r"(r.w[1].x), "=r"(r.w[1].y),
              "=r"(r.w[1].z), "=r"(r.w[1].w)
            : "l"(p));
    else
        r.w[0] = __ldg(static_cast<const uint4*>(p));
    return r;
}
template <int kType>
__device__ __forceinline__ void store8(void* p, const Raw8<kType>& r) {
    if constexpr (kType == VLPROJ_F32)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r.w[0].x), "r"(r.w[0].y),
                     "r"(r.w[0].z), "r"(r.w[0].w), "r"(r.w[1].x), "r"(r.w[1].y), "r"(r.w[1].z), "r"(r.w[1].w)
                     : "memory");
    else
        *static_cast<uint4*>(p) = r.w[0];
}
template <int kType>
__device__ __forceinline__ void store8_once(void* p, const Raw8<kType>& r) {
    if constexpr (kType == VLPROJ_F32)
        asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r.w[0].x), "r"(r.w[0].y),
                     "r"(r.w[0].z), "r"(r.w[0].w), "r"(r.w[1].x), "r"(r.w[1].y), "r"(r.w[1].z), "r"(r.w[1].w)
                     : "memory");
    else
        __stcs(static_cast<uint4*>(p), r.w[0]);
}

template <int kType>
__device__ __forceinline__ void unpack8(const Raw8<kType>& r, float (&f)[8]) {
    if constexpr (kType == VLPROJ_F32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            f[4 * h] = __uint_as_float(r.w[h].x);
            f[4 * h + 1] = __uint_as_float(r.w[h].y);
            f[4 * h + 2] = __uint_as_float(r.w[h].z);
            f[4 * h + 3] = __uint_as_float(r.w[h].w);
        }
    } else {
        const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (kType == VLPROJ_BF16) {
                f[2 * e] = __uint_as_float(w[e] << 16);
                f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
            } else {
                const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
                f[2 * e] = t.x;
                f[2 * e + 1] = t.y;
            }
        }
    }
}

template <int kType>
__device__ __forceinline__ Raw8<kType> pack8(const float (&f)[8]) {
    Raw8<kType> r;
    if constexpr (kType == VLPROJ_F32) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            r.w[h] = make_uint4(__float_as_uint(f[4 * h]), __float_as_uint(f[4 * h + 1]),
                                __float_as_uint(f[4 * h + 2]), __float_as_uint(f[4 * h + 3]));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (kType == VLPROJ_BF16) {
                const __nv_bfloat162 t = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
                w[e] = *reinterpret_cast<const uint32_t*>(&t);
            } else {
                const __half2 t = __floats2half2_rn(f[2 * e], f[2 * e + 1]);
                w[e] = *reinterpret_cast<const uint32_t*>(&t);
            }
        }
        r.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return r;
}

// The same as 4 packed pairs (elements 2e, 2e + 1), two of which one instruction adds or
// multiplies.
template <int kType>
__device__ __forceinline__ void unpack8(const Raw8<kType>& r, uint64_t (&q)[4]) {
    float f[8];
    unpack8<kType>(r, f);
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = vlp::f2_pack(f[2 * e], f[2 * e + 1]);
}

template <int kType>
__device__ __forceinline__ Raw8<kType> pack8(const uint64_t (&q)[4]) {
    float f[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) vlp::f2_unpack(q[e], f[2 * e], f[2 * e + 1]);
    return pack8<kType>(f);
}

// Sum of a packed pair's halves.
__device__ __forceinline__ float pair_sum(uint64_t q) {
    float a, b;
    vlp::f2_unpack(q, a, b);
    return a + b;
}

__device__ __forceinline__ float warp_add(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Between two kernels of one call on a stream, the second launched by launch_after: the
// first says that its successor's blocks may take free places, and the successor waits
// until the first has ended and its writes are seen. What the successor does before the
// wait reads nothing the first writes; the pointers it reads those results through are
// passed to the wait, so that no load through them is moved ahead of it.
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <class... P>
__device__ __forceinline__ void after_previous_kernel(P*&... results) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    (..., [](P*& p) { asm volatile("" : "+l"(p)::"memory"); }(results));
}

// Launches `kernel`, which calls after_previous_kernel(), without waiting for the stream's
// previous kernel to end: its start-up then overlaps that kernel's last blocks.
template <class... Params, class... Args>
inline cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args... args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// Host: SM count of the current device, asked once per device (by any host thread).
inline int sm_count() {
    static std::atomic<int> n[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int v = n[dev].load(std::memory_order_relaxed);
    if (v == 0) {
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        n[dev].store(v, std::memory_order_relaxed);
    }
    return v;
}

inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
// A workspace: its parts begin on multiples of 256 bytes, and are written 32 bytes at a time.
inline bool workspace_ok(const void* p, int64_t bytes, int64_t need) {
    return p != nullptr && reinterpret_cast<uintptr_t>(p) % 256 == 0 && need >= 0 && bytes >= need;
}
// Whether 8-element accesses are aligned at the start of every row (and every 8 elements on).
inline bool rows_wide(const void* p, int64_t ld, int type) {
    const uintptr_t bytes = static_cast<uintptr_t>(8 * type_size(type));
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld % 8 == 0;
}

// A matrix argument: rows of n elements, ld apart, element-aligned, with addresses that fit.
inline bool matrix_ok(const void* p, int64_t rows, int64_t n, int64_t ld, int type) {
    return ld >= n && ld < (int64_t(1) << 58) / (rows > 0 ? rows : 1) && (rows == 0 || p != nullptr) &&
           reinterpret_cast<uintptr_t>(p) % type_size(type) == 0;
}

// Rows of n elements, ld apart, as the byte range they span.
struct Span {
    uintptr_t lo = 0, hi = 0;
};
inline Span span_of(const void* p, int64_t rows, int64_t n, int64_t ld, int64_t size) {
    Span s;
    s.lo = reinterpret_cast<uintptr_t>(p);
    s.hi = rows > 0 && n > 0 ? s.lo + static_cast<uintptr_t>(((rows - 1) * ld + n) * size) : s.lo;
    return s;
}
inline bool overlap(const Span& a, const Span& b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }
// Whether an output overlaps another output or an input.
inline bool any_overlap(const Span* out, int n_out, const Span* in, int n_in) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = i + 1; j < n_out; ++j)
            if (overlap(out[i], out[j])) return true;
        for (int j = 0; j < n_in; ++j)
            if (overlap(out[i], in[j])) return true;
    }
    return false;
}

inline bool known_type(int t) { return t == VLPROJ_BF16 || t == VLPROJ_F32 || t == VLPROJ_F16; }
// (input, output) pairs the operators take: one type, or fp32 in and a 2-byte type out.
inline bool known_pair(int in, int out) { return known_type(in) && known_type(out) && (in == out || in == VLPROJ_F32); }

// Calls f(type_tag<in>(), type_tag<out>()) for a known_pair.
template <int kType>
using type_tag = std::integral_constant<int, kType>;
template <class F>
inline void dispatch_pair(int in, int out, F&& f) {
    if (in == VLPROJ_BF16) f(type_tag<VLPROJ_BF16>(), type_tag<VLPROJ_BF16>());
    else if (in == VLPROJ_F16) f(type_tag<VLPROJ_F16>(), type_tag<VLPROJ_F16>());
    else if (out == VLPROJ_F32) f(type_tag<VLPROJ_F32>(), type_tag<VLPROJ_F32>());
    else if (out == VLPROJ_BF16) f(type_tag<VLPROJ_F32>(), type_tag<VLPROJ_BF16>());
    else f(type_tag<VLPROJ_F32>(), type_tag<VLPROJ_F16>());
}

}  // namespace vlp_ops
