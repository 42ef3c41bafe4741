// Layer norm over the last axis and its gradients (sm_100a). Memory traffic bounds both:
// the forward pass reads x and writes y, the backward pass reads x and d_y and writes d_x.
#pragma once
#include "ops_common.cuh"

namespace vlp_ops {

// Most row-block partial sums of d_gamma and d_beta (the workspace is sized for it).
constexpr int LN_MAX_PARTS = 592;

// Rows a block of whole-row kernels can hold in registers: 8-element vectors, kVec a thread.
constexpr int LN_MAX_THREADS = 1024;
constexpr int LN_FWD_MAX_VEC = 8;         // C up to 65536
constexpr int LN_BWD_MAX_VEC = 2;         // C up to 16384

// ---------------------------------------------------------------- rows in registers
// The threads that share a row: kLanes lanes of a warp, or (kLanes = 0) the whole block.
// Sums over them end in every thread, in a fixed order.
template <int kLanes>
struct RowGroup {
    static __device__ __forceinline__ float lanes_add(float v) {
#pragma unroll
        for (int o = (kLanes ? kLanes : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
    // Two sums at once. `red`: kLanes = 0 only, 2 x 2 x 32 floats; `turn` alternates between
    // the halves, so one barrier a call is enough.
    static __device__ __forceinline__ void add2(float& a, float& b, float* red, int turn) {
        a = lanes_add(a);
        b = lanes_add(b);
        if constexpr (kLanes == 0) {
            float2* r = reinterpret_cast<float2*>(red) + 32 * turn;
            const int warps = blockDim.x >> 5;
            if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = make_float2(a, b);
            __syncthreads();
            const int l = threadIdx.x & 31;
            const float2 v = l < warps ? r[l] : make_float2(0.f, 0.f);
            a = lanes_add(v.x);
            b = lanes_add(v.y);
        }
    }
    static __device__ __forceinline__ float add(float a, float* red, int turn) {
        float b = 0.f;
        if constexpr (kLanes == 0) {
            a = lanes_add(a);
            float* r = red + 64 * turn;
            const int warps = blockDim.x >> 5;
            if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = a;
            __syncthreads();
            const int l = threadIdx.x & 31;
            return lanes_add(l < warps ? r[l] : 0.f);
        } else {
            add2(a, b, red, turn);
            return a;
        }
    }
};

// Rows of C % 8 == 0 elements, 16-byte aligned: thread j of the row's group holds the
// vectors j, j + group, ... (kVec at most) and reads x once. kLanes as in RowGroup; with
// lanes a warp holds 32 / kLanes rows.
template <int kX, int kY, int kLanes, int kVec>
static __global__ void __launch_bounds__(kLanes ? 256 : LN_MAX_THREADS) vlp_ln_rows_kernel(
    const void* __restrict__ x, int64_t x_ld, void* __restrict__ y, int64_t y_ld, int64_t rows, int C,
    const float* __restrict__ gamma, const float* __restrict__ beta, float* __restrict__ mean_out,
    float* __restrict__ rstd_out, float eps) {
    using TX = typename Elem<kX>::T;
    using TY = typename Elem<kY>::T;
    using Group = RowGroup<kLanes>;
    __shared__ float red[kLanes ? 1 : 128];
    const int group = kLanes ? kLanes : blockDim.x;
    const int j = kLanes ? threadIdx.x % kLanes : threadIdx.x;
    const int64_t r = kLanes ? static_cast<int64_t>(blockIdx.x) * (256 / kLanes) + threadIdx.x / kLanes : blockIdx.x;
    const bool live = r < rows;              // a group past the end still takes part in the warp's sums
    const int nvec = C / 8;
    const TX* src = static_cast<const TX*>(x) + r * x_ld;
    Raw8<kX> raw[kVec];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kVec; ++i)
        if (live && j + i * group < nvec) raw[i] = load8<kX>(src + 8 * (j + i * group));
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        if (!live || j + i * group >= nvec) continue;
        float f[8];
        unpack8<kX>(raw[i], f);
        s += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
    }
    const float inv_c = 1.0f / static_cast<float>(C);
    const float mean = Group::add(s, red, 0) * inv_c;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        if (!live || j + i * group >= nvec) continue;
        float f[8];
        unpack8<kX>(raw[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = f[e] - mean;
            q = fmaf(d, d, q);
        }
    }
    const float rstd = 1.0f / sqrtf(Group::add(q, red, 1) * inv_c + eps);
    if (!live) return;
    if (j == 0) {
        if (mean_out) mean_out[r] = mean;
        if (rstd_out) rstd_out[r] = rstd;
    }
    TY* dst = static_cast<TY*>(y) + r * y_ld;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int v = j + i * group;
        if (v >= nvec) continue;
        float f[8];
        unpack8<kX>(raw[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = (f[e] - mean) * rstd;
        if (gamma) {
            float g[8];
            unpack8<VLPROJ_F32>(load8<VLPROJ_F32>(gamma + 8 * v), g);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= g[e];
        }
        if (beta) {
            float b[8];
            unpack8<VLPROJ_F32>(load8<VLPROJ_F32>(beta + 8 * v), b);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] += b[e];
        }
        store8<kY>(dst + 8 * v, pack8<kY>(f));
    }
}

__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copy_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// Gradients for rows of C % 8 == 0 elements, 16-byte aligned. A grid of resident blocks
// walks the rows; each thread keeps the column sums of its own vectors in registers over
// all its rows and copies its own vectors of the next kStages - 1 rows of x and d_y into a
// shared-memory ring that only it reads, so the copies need no barrier and the memory
// system stays busy while a row is reduced. The block's column sums are added over its
// groups in order and written to part[block][0 | 1][C]. Dynamic shared memory: the ring,
// kStages x kVec x threads x (x and d_y vectors); afterwards the column sums.
constexpr int LN_GRAD_THREADS = 128;      // of a block whose rows are held by lanes of a warp
template <int kX, int kY, int kLanes, int kVec, int kStages>
static __global__ void __launch_bounds__(kLanes ? LN_GRAD_THREADS : LN_MAX_THREADS) vlp_ln_grad_kernel(
    const void* __restrict__ x, int64_t x_ld, const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
    const void* __restrict__ dy, int64_t dy_ld, const float* __restrict__ gamma, void* __restrict__ dx, int64_t dx_ld,
    int64_t rows, int C, float* __restrict__ part) {
    using TX = typename Elem<kX>::T;
    using TY = typename Elem<kY>::T;
    using Group = RowGroup<kLanes>;
    constexpr int WX = kX == VLPROJ_F32 ? 2 : 1, WY = kY == VLPROJ_F32 ? 2 : 1;      // 16-byte words of a vector
    extern __shared__ uint4 ring[];
    __shared__ float red[kLanes ? 1 : 128];
    const int threads = kLanes ? LN_GRAD_THREADS : blockDim.x;
    const int group = kLanes ? kLanes : blockDim.x;
    const int j = kLanes ? threadIdx.x % kLanes : threadIdx.x;
    const int groups = kLanes ? LN_GRAD_THREADS / kLanes : 1;            // rows a block takes at a time
    const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * groups + (kLanes ? threadIdx.x / kLanes : 0);
    const int nvec = C / 8;
    // slot (stage, i, word) of this thread
    auto slot = [&](int stage, int i, int w) { return ring + ((stage * kVec + i) * (WX + WY) + w) * threads + threadIdx.x; };
    auto fetch = [&](int64_t r, int stage) {
        if (r < rows) {
            const TX* xs = static_cast<const TX*>(x) + r * x_ld;
            const TY* ds = static_cast<const TY*>(dy) + r * dy_ld;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int v = j + i * group;
                if (v >= nvec) continue;
#pragma unroll
                for (int w = 0; w < WX; ++w) copy_async16(slot(stage, i, w), reinterpret_cast<const uint4*>(xs + 8 * v) + w);
#pragma unroll
                for (int w = 0; w < WY; ++w) copy_async16(slot(stage, i, WX + w), reinterpret_cast<const uint4*>(ds + 8 * v) + w);
            }
        }
        copy_async_commit();
    };
    float ag[kVec][8], ab[kVec][8];
#pragma unroll
    for (int i = 0; i < kVec; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) ag[i][e] = ab[i][e] = 0.f;
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) fetch(first + k * step, k);
    const float inv_c = 1.0f / static_cast<float>(C);
    int stage = 0, turn = 0;
    // all groups of the block make the same number of turns: the sums need whole warps
    const int64_t turns = (rows - static_cast<int64_t>(blockIdx.x) * groups + step - 1) / step;
    for (int64_t k = 0; k < turns; ++k) {
        const int64_t r = first + k * step;
        const bool live = r < rows;
        fetch(r + (kStages - 1) * step, stage == 0 ? kStages - 1 : stage - 1);
        copy_async_wait<kStages - 1>();
        const float mean = live ? __ldg(mean_in + r) : 0.f, rstd = live ? __ldg(rstd_in + r) : 0.f;
        float sg = 0.f, sgx = 0.f;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int v = j + i * group;
            if (!live || v >= nvec) continue;
            Raw8<kX> rx;
            Raw8<kY> rd;
#pragma unroll
            for (int w = 0; w < WX; ++w) rx.w[w] = *slot(stage, i, w);
#pragma unroll
            for (int w = 0; w < WY; ++w) rd.w[w] = *slot(stage, i, WX + w);
            float f[8], d[8], g[8];
            unpack8<kX>(rx, f);
            unpack8<kY>(rd, d);
            if (gamma) {
                unpack8<VLPROJ_F32>(load8<VLPROJ_F32>(gamma + 8 * v), g);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) g[e] = 1.f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float xh = (f[e] - mean) * rstd;
                ag[i][e] = fmaf(d[e], xh, ag[i][e]);
                ab[i][e] += d[e];
                const float t = d[e] * g[e];
                sg += t;
                sgx = fmaf(t, xh, sgx);
            }
        }
        if (dx != nullptr) {
            Group::add2(sg, sgx, red, turn);
            turn ^= 1;
            const float mg = sg * inv_c, mgx = sgx * inv_c;
            TX* dst = static_cast<TX*>(dx) + r * dx_ld;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int v = j + i * group;
                if (!live || v >= nvec) continue;
                Raw8<kX> rx;
                Raw8<kY> rd;
#pragma unroll
                for (int w = 0; w < WX; ++w) rx.w[w] = *slot(stage, i, w);
#pragma unroll
                for (int w = 0; w < WY; ++w) rd.w[w] = *slot(stage, i, WX + w);
                float f[8], d[8], g[8];
                unpack8<kX>(rx, f);
                unpack8<kY>(rd, d);
                if (gamma) {
                    unpack8<VLPROJ_F32>(load8<VLPROJ_F32>(gamma + 8 * v), g);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) g[e] = 1.f;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float xh = (f[e] - mean) * rstd;
                    f[e] = rstd * (d[e] * g[e] - mg - xh * mgx);
                }
                store8<kX>(dst + 8 * v, pack8<kX>(f));
            }
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    if (part == nullptr) return;
    copy_async_wait<0>();
    float* row = part + static_cast<int64_t>(blockIdx.x) * 2 * C;
    if constexpr (kLanes == 0) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int v = j + i * group;
            if (v >= nvec) continue;
            store8<VLPROJ_F32>(row + 8 * v, pack8<VLPROJ_F32>(ag[i]));
            store8<VLPROJ_F32>(row + C + 8 * v, pack8<VLPROJ_F32>(ab[i]));
        }
    } else {
        // one slice of 2 C sums per warp; lanes of one warp that share columns are added first
        __syncthreads();
        float* sums = reinterpret_cast<float*>(ring);
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < kVec; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
                for (int o = kLanes; o < 32; o <<= 1) {
                    ag[i][e] += __shfl_xor_sync(0xffffffffu, ag[i][e], o);
                    ab[i][e] += __shfl_xor_sync(0xffffffffu, ab[i][e], o);
                }
        if (lane < kLanes) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int v = j + i * group;
                if (v >= nvec) continue;
                store8<VLPROJ_F32>(sums + warp * 2 * C + 8 * v, pack8<VLPROJ_F32>(ag[i]));
                store8<VLPROJ_F32>(sums + warp * 2 * C + C + 8 * v, pack8<VLPROJ_F32>(ab[i]));
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * C; c += LN_GRAD_THREADS) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < LN_GRAD_THREADS / 32; ++w) s += sums[w * 2 * C + c];
            row[c] = s;
        }
    }
}

// ---------------------------------------------------------------- any layout
// Any row length, distance and element alignment: one warp per row, the row read again
// for each of the three passes (mean, variance, output).
template <int kX, int kY>
static __global__ void __launch_bounds__(256) vlp_ln_rows_any_kernel(const void* __restrict__ x, int64_t x_ld,
                                                                     void* __restrict__ y, int64_t y_ld, int64_t rows,
                                                                     int C, const float* __restrict__ gamma,
                                                                     const float* __restrict__ beta,
                                                                     float* __restrict__ mean_out,
                                                                     float* __restrict__ rstd_out, float eps) {
    using TX = typename Elem<kX>::T;
    using TY = typename Elem<kY>::T;
    const int lane = threadIdx.x & 31;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (r >= rows) return;
    const TX* src = static_cast<const TX*>(x) + r * x_ld;
    TY* dst = static_cast<TY*>(y) + r * y_ld;
    const float inv_c = 1.0f / static_cast<float>(C);
    float s = 0.f;
#pragma unroll 4
    for (int c = lane; c < C; c += 32) s += Elem<kX>::up(__ldg(src + c));
    const float mean = warp_add(s) * inv_c;
    float q = 0.f;
#pragma unroll 4
    for (int c = lane; c < C; c += 32) {
        const float d = Elem<kX>::up(__ldg(src + c)) - mean;
        q += d * d;
    }
    const float rstd = 1.0f / sqrtf(warp_add(q) * inv_c + eps);
    if (lane == 0) {
        if (mean_out) mean_out[r] = mean;
        if (rstd_out) rstd_out[r] = rstd;
    }
#pragma unroll 4
    for (int c = lane; c < C; c += 32) {
        const float g = gamma ? __ldg(gamma + c) : 1.f, b = beta ? __ldg(beta + c) : 0.f;
        dst[c] = Elem<kY>::down((Elem<kX>::up(__ldg(src + c)) - mean) * rstd * g + b);
    }
}

// d_x of any layout: one warp per row, two passes.
template <int kX, int kY>
static __global__ void __launch_bounds__(256) vlp_ln_dx_any_kernel(const void* __restrict__ x, int64_t x_ld,
                                                                   const float* __restrict__ mean_in,
                                                                   const float* __restrict__ rstd_in,
                                                                   const void* __restrict__ dy, int64_t dy_ld,
                                                                   const float* __restrict__ gamma,
                                                                   void* __restrict__ dx, int64_t dx_ld, int64_t rows,
                                                                   int C) {
    using TX = typename Elem<kX>::T;
    using TY = typename Elem<kY>::T;
    const int lane = threadIdx.x & 31;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (r >= rows) return;
    const TX* xs = static_cast<const TX*>(x) + r * x_ld;
    const TY* ds = static_cast<const TY*>(dy) + r * dy_ld;
    TX* dst = static_cast<TX*>(dx) + r * dx_ld;
    const float mean = __ldg(mean_in + r), rstd = __ldg(rstd_in + r);
    float sg = 0.f, sgx = 0.f;
#pragma unroll 4
    for (int c = lane; c < C; c += 32) {
        const float g = Elem<kY>::up(__ldg(ds + c)) * (gamma ? __ldg(gamma + c) : 1.f);
        sg += g;
        sgx += g * ((Elem<kX>::up(__ldg(xs + c)) - mean) * rstd);
    }
    const float inv_c = 1.0f / static_cast<float>(C);
    const float mg = warp_add(sg) * inv_c, mgx = warp_add(sgx) * inv_c;
#pragma unroll 4
    for (int c = lane; c < C; c += 32) {
        const float g = Elem<kY>::up(__ldg(ds + c)) * (gamma ? __ldg(gamma + c) : 1.f);
        const float xh = (Elem<kX>::up(__ldg(xs + c)) - mean) * rstd;
        dst[c] = Elem<kX>::down(rstd * (g - mg - xh * mgx));
    }
}

// Row-block sums of d_gamma and d_beta of any layout: part[b][0 | 1][c] over the rows of
// block b, a thread per column.
template <int kX, int kY>
static __global__ void __launch_bounds__(128) vlp_ln_part_any_kernel(const void* __restrict__ x, int64_t x_ld,
                                                                     const float* __restrict__ mean_in,
                                                                     const float* __restrict__ rstd_in,
                                                                     const void* __restrict__ dy, int64_t dy_ld,
                                                                     int64_t rows, int per, int C,
                                                                     float* __restrict__ part) {
    using TX = typename Elem<kX>::T;
    using TY = typename Elem<kY>::T;
    const int c = blockIdx.y * 128 + threadIdx.x;
    if (c >= C) return;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * per;
    const int64_t r1 = r0 + per < rows ? r0 + per : rows;
    const TX* xs = static_cast<const TX*>(x) + c;
    const TY* ds = static_cast<const TY*>(dy) + c;
    float sg = 0.f, sb = 0.f;
#pragma unroll 4
    for (int64_t r = r0; r < r1; ++r) {
        const float d = Elem<kY>::up(__ldg(ds + r * dy_ld));
        sg += d * ((Elem<kX>::up(__ldg(xs + r * x_ld)) - __ldg(mean_in + r)) * __ldg(rstd_in + r));
        sb += d;
    }
    float* row = part + static_cast<int64_t>(blockIdx.x) * 2 * C;
    row[c] = sg;
    row[C + c] = sb;
}

// d_gamma[c] = sum of part[b][0][c], d_beta[c] = sum of part[b][1][c] over b < nb, in fp64:
// a block takes 32 of the 2C sums with LN_JOIN_GROUPS groups of row blocks, joined in order.
constexpr int LN_JOIN_GROUPS = 32;
static __global__ void __launch_bounds__(32 * LN_JOIN_GROUPS) vlp_ln_join_kernel(const float* __restrict__ part, int nb, int C,
                                                                 float* __restrict__ d_gamma,
                                                                 float* __restrict__ d_beta) {
    __shared__ double red[LN_JOIN_GROUPS][32];
    const int col = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + col;
    double t = 0.;
    if (c < 2 * static_cast<int64_t>(C)) {
#pragma unroll 8
        for (int b = grp; b < nb; b += LN_JOIN_GROUPS) t += __ldg(part + static_cast<int64_t>(b) * 2 * C + c);
    }
    red[grp][col] = t;
    __syncthreads();
    if (grp != 0 || c >= 2 * static_cast<int64_t>(C)) return;
    double s = 0.;
#pragma unroll
    for (int g = 0; g < LN_JOIN_GROUPS; ++g) s += red[g][col];
    if (c < C) {
        if (d_gamma) d_gamma[c] = static_cast<float>(s);
    } else if (d_beta) {
        d_beta[c - C] = static_cast<float>(s);
    }
}

}  // namespace vlp_ops
