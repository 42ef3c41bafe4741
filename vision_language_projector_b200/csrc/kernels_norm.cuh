// Layer norm over the last axis and its gradients (sm_100a). Memory traffic bounds both:
// the forward pass reads x and writes y, the backward pass reads x and d_y and writes d_x.
#pragma once
#include "ops_common.cuh"

namespace vlp_ops {

// Most row-block partial sums of d_gamma and d_beta (the workspace is sized for it).
constexpr int LN_MAX_PARTS = 592;

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
// a block takes 32 of the 2C sums with 8 groups of row blocks, joined in group order.
static __global__ void __launch_bounds__(256) vlp_ln_join_kernel(const float* __restrict__ part, int nb, int C,
                                                                 float* __restrict__ d_gamma,
                                                                 float* __restrict__ d_beta) {
    __shared__ double red[8][32];
    const int col = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + col;
    double t = 0.;
    if (c < 2 * static_cast<int64_t>(C)) {
#pragma unroll 8
        for (int b = grp; b < nb; b += 8) t += __ldg(part + static_cast<int64_t>(b) * 2 * C + c);
    }
    red[grp][col] = t;
    __syncthreads();
    if (grp != 0 || c >= 2 * static_cast<int64_t>(C)) return;
    double s = 0.;
#pragma unroll
    for (int g = 0; g < 8; ++g) s += red[g][col];
    if (c < C) {
        if (d_gamma) d_gamma[c] = static_cast<float>(s);
    } else if (d_beta) {
        d_beta[c - C] = static_cast<float>(s);
    }
}

}  // namespace vlp_ops
