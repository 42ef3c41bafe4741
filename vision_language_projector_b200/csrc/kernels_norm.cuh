// Layer norm over the last axis and its gradients (sm_100a). Memory traffic bounds both:
// the forward pass reads x and writes y, the backward pass reads x and d_y and writes d_x.
#pragma once
#include <cooperative_groups.h>

#include "ops_common.cuh"

namespace vlp_ops {

// Most row-block partial sums of d_gamma and d_beta (the workspace is sized for it):
// narrow rows need more blocks to keep the memory busy, and their sums are short.
constexpr int ln_max_parts(int64_t C) { return C <= 512 ? 1184 : 592; }

// Whether a thread's vector i (< kVec) can be a row's first or last one. The last one lies
// in the last vectors of some thread: rows of fewer vectors are held with a smaller kVec.
template <int kLanes, int kVec>
constexpr bool outer_vector(int i) {
    return i == 0 || i >= kVec - (kLanes == 0 ? 2 : kVec == 8 ? 4 : 3);
}

// Rows a block of whole-row kernels can hold in registers: 8-element vectors, kVec a thread.
constexpr int LN_MAX_THREADS = 1024;
// Their ring has to fit in shared memory too, so the forward pass holds rows of up to 57344
// two-byte or 28672 fp32 elements, the gradients 16384, or 14336 where x and d_y are fp32;
// longer rows go the way of any layout.
constexpr int LN_FWD_MAX_VEC = 8;
constexpr int LN_BWD_MAX_VEC = 2;

// A row's mean: its sum times 1 / C, the reciprocal held in two words (inv_c and what it lacks,
// inv_rest), so that the product is rounded once. With inv_c alone a row without spread keeps
// an error of the mean's last place, which 1 / sqrt(eps) enlarges: 1000 with C = 7 came out as
// 0.019 instead of 0. A division does the same and takes up to 3 % longer where a block waits
// for each row's mean (24693 x 7618 bf16: 258 us with inv_c, 260 so, 266 divided). The sum of
// an infinite row meets inv_rest as a NaN; its mean is then taken without.
__device__ __forceinline__ float ln_inverse_rest(float inv_c, int C) { return fmaf(-inv_c, static_cast<float>(C), 1.0f) * inv_c; }
__device__ __forceinline__ float ln_mean(float sum, float inv_c, float inv_rest) { return fmaf(sum, inv_c, sum * inv_rest); }

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
    // Two sums of each of kRows rows at once. `red`: kLanes = 0 only, 128 kRows floats;
    // `half` alternates between its halves, so one barrier a call is enough. With two rows a
    // block's four sums are added together: each step of the first two halves the sums a
    // lane still carries, so a warp's four take 6 exchanges, not 20, and 7 behind the barrier.
    template <int kRows>
    static __device__ __forceinline__ void add_rows(float (&a)[kRows], float (&b)[kRows], float* red, int half) {
        if constexpr (kLanes == 0 && kRows == 2) {
            add_two_rows(a, b, red, half);
        } else {
            add_each_row<kRows>(a, b, red, half);
        }
    }
    static __device__ __forceinline__ void add_two_rows(float (&a)[2], float (&b)[2], float* red, int half) {
        const int l = threadIdx.x & 31, warps = blockDim.x >> 5;
        const bool up = l & 16, odd = l & 8;
        const float u = (up ? a[1] : a[0]) + __shfl_xor_sync(0xffffffffu, up ? a[0] : a[1], 16);
        const float v = (up ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, up ? b[0] : b[1], 16);
        float s = (odd ? v : u) + __shfl_xor_sync(0xffffffffu, odd ? u : v, 8);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        // lanes 8i .. 8i + 7 hold sum i of a[0], b[0], a[1], b[1]
        float* r = red + 128 * half + 32 * (l >> 3);
        if ((l & 7) == 0) r[threadIdx.x >> 5] = s;
        __syncthreads();
        s = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) s += (l & 7) + 8 * q < warps ? r[(l & 7) + 8 * q] : 0.f;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        a[0] = __shfl_sync(0xffffffffu, s, 0);
        b[0] = __shfl_sync(0xffffffffu, s, 8);
        a[1] = __shfl_sync(0xffffffffu, s, 16);
        b[1] = __shfl_sync(0xffffffffu, s, 24);
    }
    template <int kRows>
    static __device__ __forceinline__ void add_each_row(float (&a)[kRows], float (&b)[kRows], float* red, int half) {
#pragma unroll
        for (int q = 0; q < kRows; ++q) {
            a[q] = lanes_add(a[q]);
            b[q] = lanes_add(b[q]);
        }
        if constexpr (kLanes == 0) {
            float2* r = reinterpret_cast<float2*>(red) + 32 * kRows * half;
            const int warps = blockDim.x >> 5, l = threadIdx.x & 31;
            if (l == 0)
#pragma unroll
                for (int q = 0; q < kRows; ++q) r[32 * q + (threadIdx.x >> 5)] = make_float2(a[q], b[q]);
            __syncthreads();
#pragma unroll
            for (int q = 0; q < kRows; ++q) {
                const float2 v = l < warps ? r[32 * q + l] : make_float2(0.f, 0.f);
                a[q] = lanes_add(v.x);
                b[q] = lanes_add(v.y);
            }
        }
    }
    // One sum. `red`: kLanes = 0 only, 64 floats; `half` as above.
    static __device__ __forceinline__ float add(float a, float* red, int half) {
        a = lanes_add(a);
        if constexpr (kLanes == 0) {
            float* r = red + 32 * half;
            const int warps = blockDim.x >> 5, l = threadIdx.x & 31;
            if (l == 0) r[threadIdx.x >> 5] = a;
            __syncthreads();
            a = lanes_add(l < warps ? r[l] : 0.f);
        }
        return a;
    }
};

// kShared: the other half of the 32-byte sector is copied next, so the sector is kept in L1.
template <bool kShared>
__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
    if constexpr (kShared) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                     "l"(src) : "memory");
        return;
    }
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copy_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// Which rows a block of the whole-row kernels takes, and how they are cut into vectors of 8
// elements. kShift = false: C % 8 == 0 and every row of every matrix aligned for 8-element
// accesses; a block's groups take adjacent rows. kShift = true: any C, row distance and
// element alignment for which the matrices' rows start equally far (in elements, modulo 8)
// behind an aligned vector; vector v is then the aligned one that holds the columns
// 8v - shift .. 8v - shift + 7, of which the row's first and last one may hold fewer.
// Since the shift repeats every 8 rows, a block takes rows r with one value of r % 8, so
// that its threads keep their columns. The grid is a multiple of 8.
template <bool kShift>
struct RowLayout {
    int64_t block_row;       // the block's first row
    int64_t mine;            // this group's row of a step, from there
    int64_t step;            // to the group's next row
    int64_t rows;
    int C, nvec, shift;
    __device__ __forceinline__ RowLayout(uintptr_t element, int64_t ld, int64_t rows_, int C_, int groups, int g)
        : rows(rows_), C(C_) {
        if constexpr (kShift) {
            const int rest = static_cast<int>(blockIdx.x & 7);
            const int64_t eighth = blockIdx.x >> 3;
            block_row = rest + 8 * groups * eighth;
            mine = 8 * g;
            step = 8 * static_cast<int64_t>(groups) * (gridDim.x >> 3);
            shift = static_cast<int>((element + static_cast<uintptr_t>(rest * ld)) & 7);
            nvec = (shift + C + 7) / 8;
        } else {
            block_row = static_cast<int64_t>(blockIdx.x) * groups;
            mine = g;
            step = static_cast<int64_t>(gridDim.x) * groups;
            shift = 0;
            nvec = C / 8;
        }
    }
    __device__ __forceinline__ bool edge(int v) const { return kShift && (v == 0 || v == nvec - 1); }
    __device__ __forceinline__ bool has(int c) const { return !kShift || (c >= 0 && c < C); }
    // zeros in place of the elements of vector v that lie outside the row
    __device__ __forceinline__ void mask(int v, uint64_t (&q)[4]) const {
        if constexpr (kShift) {
            if (!edge(v)) return;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float a, b;
                vlp::f2_unpack(q[e], a, b);
                const int c = 8 * v - shift + 2 * e;
                q[e] = vlp::f2_pack(has(c) ? a : 0.f, has(c + 1) ? b : 0.f);
            }
        }
    }
    // four weights of vector v from its half h on, `other` where w is null
    __device__ __forceinline__ float4 weight(const float* w, float other, int v, int h) const {
        if (w == nullptr) return make_float4(other, other, other, other);
        if constexpr (kShift) {
            const int c = 8 * v - shift + 4 * h;
            return make_float4(has(c) ? __ldg(w + c) : 0.f, has(c + 1) ? __ldg(w + c + 1) : 0.f,
                               has(c + 2) ? __ldg(w + c + 2) : 0.f, has(c + 3) ? __ldg(w + c + 3) : 0.f);
        } else {
            return __ldg(reinterpret_cast<const float4*>(w) + 2 * v + h);
        }
    }
    // Starts the copy of vector v of row r of a matrix into the words at `slot`, `pitch`
    // apart. A row's outer vector that reaches past the matrix's first or last element is
    // copied element by element, only those of the row.
    template <int kType>
    __device__ __forceinline__ void fetch(const void* m, int64_t ld, int64_t r, int v, uint4* slot, int pitch, bool outer) const {
        using T = typename Elem<kType>::T;
        constexpr int W = kType == VLPROJ_F32 ? 2 : 1;
        const int64_t first = r * ld - shift + 8 * v;          // of the vector's elements, in the matrix
        const T* src = static_cast<const T*>(m) + first;
        if (kShift && outer) {
            if (first < 0 || first + 8 > (rows - 1) * ld + C) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    reinterpret_cast<T*>(slot + (e * W / 8) * pitch)[e % (8 / W)] =
                        has(8 * v - shift + e) ? src[e] : Elem<kType>::down(0.f);
                return;
            }
        }
#pragma unroll
        for (int w = 0; w < W; ++w) copy_async16<(W > 1)>(slot + w * pitch, reinterpret_cast<const uint4*>(src) + w);
    }
    template <int kType>
    __device__ __forceinline__ void store(void* m, int64_t ld, int64_t r, int v, const uint64_t (&q)[4], bool outer) const {
        using T = typename Elem<kType>::T;
        T* dst = static_cast<T*>(m) + r * ld - shift + 8 * v;
        if (!outer || !edge(v)) {
            store8<kType>(dst, pack8<kType>(q));
            return;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float a, b;
            vlp::f2_unpack(q[e], a, b);
            const int c = 8 * v - shift + 2 * e;
            if (has(c)) dst[2 * e] = Elem<kType>::down(a);
            if (has(c + 1)) dst[2 * e + 1] = Elem<kType>::down(b);
        }
    }
};

// Thread j of a row's group holds the row's vectors j, j + group, ... (kVec at most), and x
// is read once. kLanes as in RowGroup; with
// lanes a warp holds 32 / kLanes rows and gamma and beta wait in shared memory, as arrays
// of float4 (channels 8v .. 8v+3 and 8v+4 .. 8v+7 of each) so that the lanes of a warp read
// consecutive ones (read from memory 32 bytes apart, they bound the kernel: L1 89 % busy,
// DRAM 61 %, 140 us at 163296 x 1152 bf16). The next kStages - 1 rows are on their way into
// a shared-memory ring that each thread fills and reads for itself. With a whole block per
// row each thread keeps the weights of its own channels in registers (kVec <= 2) or reads
// them again. The grid is the resident blocks, which walk the rows. 163296 x 1152 bf16, 752 MB
// to move: 121 to 129 us by the GPU one gets, 5.8 to 6.2 TB/s, with 4 stages and blocks of 128
// threads (the first measurement, in one run: 123 us; 142 us with 2 or 3 stages, 140 us with
// 6, since fewer blocks fit). A warp holds rows of up to 20 vectors a lane: joined by no
// barrier, it takes 128 to 134 us for 36000 x 5120 bf16 (5.5 to 5.8 TB/s) and 104 us for 100000
// x 1600, a block per row 153 and 156 us. Rows of a block wait at two barriers each: 25000 x 6144
// bf16 127 us and 25000 x 7168 142 us, two blocks to an SM; 24693 x 7618 262 us, floor 115 us,
// whose masked vectors take 115 registers, so that one block fits; 20000 x 9216 184 us, floor
// 113. With 8 vectors a thread the 64 registers that 1024 threads leave spill (228 bytes, 548
// when masked); it is still ahead of the kernel for any layout: 6000 x 20000 bf16 204 against
// 324 us, 2000 x 57344 221 against 790, 3000 x 28672 fp32 260 against 386.
template <int kX, int kY, bool kShift, int kLanes, int kVec, int kThreads, int kStages>
static __global__ void __launch_bounds__(kThreads) vlp_ln_rows_kernel(
    const void* __restrict__ x, int64_t x_ld, void* __restrict__ y, int64_t y_ld, int64_t rows, int C,
    const float* __restrict__ gamma, const float* __restrict__ beta, float* __restrict__ mean_out,
    float* __restrict__ rstd_out, float eps) {
    using TX = typename Elem<kX>::T;
    using Group = RowGroup<kLanes>;
    constexpr bool kKeep = kLanes == 0 && kVec <= 2;
    constexpr int WX = kX == VLPROJ_F32 ? 2 : 1;             // 16-byte words of a vector
    extern __shared__ float4 weights[];
    __shared__ float red[kLanes ? 1 : 64];
    const int threads = kLanes ? kThreads : blockDim.x;
    const int group = kLanes ? kLanes : blockDim.x;
    const int groups = kLanes ? kThreads / kLanes : 1;
    const int j = kLanes ? threadIdx.x % kLanes : threadIdx.x;
    const RowLayout<kShift> at(reinterpret_cast<uintptr_t>(x) / sizeof(TX), x_ld, rows, C, groups,
                               kLanes ? threadIdx.x / kLanes : 0);
    const int nvec = at.nvec;
    const float4 zero4 = make_float4(0.f, 0.f, 0.f, 0.f);
    // quarter q of the weights of vector v: gamma's two halves, beta's two halves
    auto weight = [&](int v, int q) { return at.weight(q < 2 ? gamma : beta, q < 2 ? 1.f : 0.f, v, q & 1); };
    float4 kept[kKeep ? kVec : 1][4];
    if constexpr (kLanes != 0) {
        for (int v = threadIdx.x; v < nvec; v += kThreads)
#pragma unroll
            for (int q = 0; q < 4; ++q) weights[q * nvec + v] = weight(v, q);
        __syncthreads();
    } else if constexpr (kKeep) {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) kept[i][q] = j + i * group < nvec ? weight(j + i * group, q) : zero4;
    }
    const float inv_c = 1.0f / static_cast<float>(C), inv_rest = ln_inverse_rest(inv_c, C);
    uint4* ring = reinterpret_cast<uint4*>(weights) + (kLanes ? 4 * nvec : 0);
    // this thread's word w of its vector i of the row in a stage
    auto slot = [&](int stage, int i, int w) { return ring + ((stage * kVec + i) * WX + w) * threads + threadIdx.x; };
    const int64_t first = at.block_row + at.mine;
    auto fetch = [&](int64_t r, int stage) {
        if (r < rows) {
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                if (j + i * group < nvec) at.template fetch<kX>(x, x_ld, r, j + i * group, slot(stage, i, 0), threads,
                                          outer_vector<kLanes, kVec>(i));
        }
        copy_async_commit();
    };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) fetch(first + k * at.step, k);
    int stage = 0;
    for (int64_t r0 = at.block_row; r0 < rows; r0 += at.step) {
        const int64_t r = r0 + at.mine;
        const bool live = r < rows;          // a group past the end still takes part in the warp's sums
        fetch(r + (kStages - 1) * at.step, stage == 0 ? kStages - 1 : stage - 1);
        copy_async_wait<kStages - 1>();
        uint64_t d[kVec][4], s = 0;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            if (!live || j + i * group >= nvec) continue;
            Raw8<kX> raw;
#pragma unroll
            for (int w = 0; w < WX; ++w) raw.w[w] = *slot(stage, i, w);
            unpack8<kX>(raw, d[i]);
            if (outer_vector<kLanes, kVec>(i)) at.mask(j + i * group, d[i]);
            s = vlp::f2_add(s, vlp::f2_add(vlp::f2_add(d[i][0], d[i][1]), vlp::f2_add(d[i][2], d[i][3])));
        }
        const float total = Group::add(pair_sum(s), red, 0), mean = ln_mean(total, inv_c, inv_rest);
        const uint64_t nm = vlp::f2_splat(-mean);
        s = 0;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            if (!live || j + i * group >= nvec) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) d[i][e] = vlp::f2_add(d[i][e], nm);
            if (outer_vector<kLanes, kVec>(i)) at.mask(j + i * group, d[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) s = vlp::f2_fma(d[i][e], d[i][e], s);
        }
        const float rstd = 1.0f / sqrtf(Group::add(pair_sum(s), red, 1) * inv_c + eps);
        if (live && j == 0) {
            if (mean_out) mean_out[r] = mean == mean ? mean : total * inv_c;
            if (rstd_out) rstd_out[r] = rstd;
        }
        const uint64_t r2 = vlp::f2_splat(rstd);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int v = j + i * group;
            if (!live || v >= nvec) continue;
            float4 w[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                if constexpr (kLanes != 0) w[h] = weights[h * nvec + v];
                else if constexpr (kKeep) w[h] = kept[i][h];
                else w[h] = weight(v, h);
            }
            const uint64_t g[4] = {vlp::f2_pack(w[0].x, w[0].y), vlp::f2_pack(w[0].z, w[0].w),
                                   vlp::f2_pack(w[1].x, w[1].y), vlp::f2_pack(w[1].z, w[1].w)};
            const uint64_t b[4] = {vlp::f2_pack(w[2].x, w[2].y), vlp::f2_pack(w[2].z, w[2].w),
                                   vlp::f2_pack(w[3].x, w[3].y), vlp::f2_pack(w[3].z, w[3].w)};
#pragma unroll
            for (int e = 0; e < 4; ++e) d[i][e] = vlp::f2_fma(vlp::f2_mul(d[i][e], r2), g[e], b[e]);
            at.template store<kY>(y, y_ld, r, v, d[i], outer_vector<kLanes, kVec>(i));
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
}

// Gradients. A grid of resident blocks walks the rows, kRows of each group at a turn; each
// thread keeps the column sums of its own vectors in registers over all its rows and copies
// its own vectors of the next kStages - 1 turns' rows of x and d_y into a shared-memory ring
// that only it reads, so the copies need no barrier and the memory system stays busy while
// rows are reduced. With t = x - mean and u = d_y * gamma a row needs sum(u) and sum(u t),
// and then
//     d_x = u rstd - rstd mean(u) - t rstd^3 mean(u t).
// 50176 x 1152 bf16, a warp a row: 55 us, 5.7 TB/s, memory-bound. 8192 x 5120, a block a row:
// 56 us, 3.9 TB/s, with neither memory nor issue slots (63 %) full: two blocks of 10 warps an
// SM, as many as their rings of 82 KB let reside, leave a barrier a turn uncovered.
// The block's column sums are added over its groups in order and written to
// part[block][0 | 1][C]. Dynamic shared memory: gamma (kLanes only, two arrays of float4 as
// in the forward pass), then the ring, kStages x kRows x kVec x (words of x and d_y) x
// threads, which holds the warps' column sums afterwards. kThreads: LN_GRAD_THREADS with
// kLanes, else the most threads of a block.
// few: the grid is one cluster of LN_FEW_BLOCKS blocks, which leave their column sums in
// shared memory (at the float few_at), read one another's and write d_gamma and d_beta
// themselves: one launch and no workspace.
constexpr int LN_GRAD_THREADS = 128;      // of a block whose rows are held by lanes of a warp
constexpr int LN_FEW_BLOCKS = 8;
template <int kX, int kY, bool kShift, int kLanes, int kVec, int kThreads, int kRows, int kStages>
static __global__ void __launch_bounds__(kThreads) vlp_ln_grad_kernel(
    const void* __restrict__ x, int64_t x_ld, const float* __restrict__ mean_in, const float* __restrict__ rstd_in,
    const void* __restrict__ dy, int64_t dy_ld, const float* __restrict__ gamma, void* __restrict__ dx, int64_t dx_ld,
    int64_t rows, int C, float* __restrict__ part, int few, int few_at, float* __restrict__ d_gamma, float* __restrict__ d_beta) {
    using TX = typename Elem<kX>::T;
    using Group = RowGroup<kLanes>;
    constexpr int WX = kX == VLPROJ_F32 ? 2 : 1, WY = kY == VLPROJ_F32 ? 2 : 1;      // 16-byte words of a vector
    extern __shared__ uint4 shared_words[];
    __shared__ float red[kLanes ? 1 : 128 * kRows];
    const int threads = kLanes ? LN_GRAD_THREADS : blockDim.x;
    const int group = kLanes ? kLanes : blockDim.x;
    const int j = kLanes ? threadIdx.x % kLanes : threadIdx.x;
    const int groups = kLanes ? LN_GRAD_THREADS / kLanes : 1;            // rows a block takes at a time
    const RowLayout<kShift> at(reinterpret_cast<uintptr_t>(x) / sizeof(TX), x_ld, rows, C, groups,
                               kLanes ? threadIdx.x / kLanes : 0);
    const int nvec = at.nvec;
    const int64_t first = at.block_row + at.mine;
    float4* weights = reinterpret_cast<float4*>(shared_words);
    uint4* ring = shared_words + (kLanes ? 2 * nvec : 0);
    float4 kept[kLanes ? 1 : kVec][2];
    if constexpr (kLanes != 0) {
        for (int v = threadIdx.x; v < nvec; v += LN_GRAD_THREADS)
#pragma unroll
            for (int h = 0; h < 2; ++h) weights[h * nvec + v] = at.weight(gamma, 1.f, v, h);
        __syncthreads();
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                kept[i][h] = j + i * group < nvec ? at.weight(gamma, 1.f, j + i * group, h) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    auto weight = [&](int i, uint64_t (&g)[4]) {
        float4 a, b;
        if constexpr (kLanes != 0) {
            a = weights[j + i * group];
            b = weights[nvec + j + i * group];
        } else {
            a = kept[i][0];
            b = kept[i][1];
        }
        g[0] = vlp::f2_pack(a.x, a.y);
        g[1] = vlp::f2_pack(a.z, a.w);
        g[2] = vlp::f2_pack(b.x, b.y);
        g[3] = vlp::f2_pack(b.z, b.w);
    };
    // this thread's word w of its vector i of row q of a stage
    auto slot = [&](int stage, int q, int i, int w) {
        return ring + (((stage * kRows + q) * kVec + i) * (WX + WY) + w) * threads + threadIdx.x;
    };
    auto fetch = [&](int64_t turn, int stage) {
#pragma unroll
        for (int q = 0; q < kRows; ++q) {
            const int64_t r = first + (turn * kRows + q) * at.step;
            if (r >= rows) continue;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int v = j + i * group;
                if (v >= nvec) continue;
                at.template fetch<kX>(x, x_ld, r, v, slot(stage, q, i, 0), threads, outer_vector<kLanes, kVec>(i));
                at.template fetch<kY>(dy, dy_ld, r, v, slot(stage, q, i, WX), threads, outer_vector<kLanes, kVec>(i));
            }
        }
        copy_async_commit();
    };
    auto take = [&](int stage, int q, int i, uint64_t (&f)[4], uint64_t (&d)[4]) {
        Raw8<kX> rx;
        Raw8<kY> rd;
#pragma unroll
        for (int w = 0; w < WX; ++w) rx.w[w] = *slot(stage, q, i, w);
#pragma unroll
        for (int w = 0; w < WY; ++w) rd.w[w] = *slot(stage, q, i, WX + w);
        unpack8<kX>(rx, f);
        unpack8<kY>(rd, d);
        if (outer_vector<kLanes, kVec>(i)) {
            at.mask(j + i * group, f);
            at.mask(j + i * group, d);
        }
    };
    uint64_t ag[kVec][4], ab[kVec][4];
#pragma unroll
    for (int i = 0; i < kVec; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) ag[i][e] = ab[i][e] = 0;
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) fetch(k, k);
    // the statistics of the next turn's rows are loaded a turn ahead
    float next_mean[kRows], next_rstd[kRows];
    auto statistics = [&](int64_t turn) {
#pragma unroll
        for (int q = 0; q < kRows; ++q) {
            const int64_t r = first + (turn * kRows + q) * at.step;
            next_mean[q] = r < rows ? __ldg(mean_in + r) : 0.f;
            next_rstd[q] = r < rows ? __ldg(rstd_in + r) : 0.f;
        }
    };
    statistics(0);
    const float inv_c = 1.0f / static_cast<float>(C);
    int stage = 0, half = 0;
    // every group of the block makes the same number of turns: the sums need whole warps
    const int64_t per_group = at.block_row < rows ? (rows - at.block_row + at.step - 1) / at.step : 0;
    const int64_t turns = (per_group + kRows - 1) / kRows;
    for (int64_t k = 0; k < turns; ++k) {
        fetch(k + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
        float mean[kRows], rstd[kRows], sg[kRows], sgx[kRows];
#pragma unroll
        for (int q = 0; q < kRows; ++q) {
            mean[q] = next_mean[q];
            rstd[q] = next_rstd[q];
        }
        statistics(k + 1);
        copy_async_wait<kStages - 1>();
#pragma unroll
        for (int q = 0; q < kRows; ++q) {
            const bool live = first + (k * kRows + q) * at.step < rows;
            const uint64_t nm = vlp::f2_splat(-mean[q]), r2 = vlp::f2_splat(rstd[q]);
            uint64_t su = 0, sut = 0;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                if (!live || j + i * group >= nvec) continue;
                uint64_t f[4], d[4], g[4];
                take(stage, q, i, f, d);
                weight(i, g);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint64_t t = vlp::f2_add(f[e], nm);
                    ag[i][e] = vlp::f2_fma(vlp::f2_mul(d[e], r2), t, ag[i][e]);
                    ab[i][e] = vlp::f2_add(ab[i][e], d[e]);
                    const uint64_t u = vlp::f2_mul(d[e], g[e]);
                    su = vlp::f2_add(su, u);
                    sut = vlp::f2_fma(u, t, sut);
                }
            }
            sg[q] = pair_sum(su);
            sgx[q] = pair_sum(sut);
        }
        if (dx != nullptr) {
            Group::template add_rows<kRows>(sg, sgx, red, half);
            half ^= 1;
#pragma unroll
            for (int q = 0; q < kRows; ++q) {
                const int64_t r = first + (k * kRows + q) * at.step;
                const uint64_t nm = vlp::f2_splat(-mean[q]), r2 = vlp::f2_splat(rstd[q]);
                const uint64_t c0 = vlp::f2_splat(-(sg[q] * inv_c) * rstd[q]);
                const uint64_t c1 = vlp::f2_splat(-sgx[q] * rstd[q] * inv_c * rstd[q] * rstd[q]);
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    const int v = j + i * group;
                    if (r >= rows || v >= nvec) continue;
                    uint64_t f[4], d[4], g[4];
                    take(stage, q, i, f, d);
                    weight(i, g);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        f[e] = vlp::f2_fma(vlp::f2_add(f[e], nm), c1, vlp::f2_fma(vlp::f2_mul(d[e], g[e]), r2, c0));
                    at.template store<kX>(dx, dx_ld, r, v, f, outer_vector<kLanes, kVec>(i));
                }
            }
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    if (part == nullptr && !few) return;
    let_next_kernel_start();
    copy_async_wait<0>();
    // the block's 2 C sums: in memory, or in one place of every block's shared memory
    float* row = few ? reinterpret_cast<float*>(shared_words) + few_at : part + static_cast<int64_t>(blockIdx.x) * 2 * C;
    if constexpr (kLanes == 0) {
        if (few) __syncthreads();                        // the place is the ring's: all have read it
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int v = j + i * group;
            if (v >= nvec) continue;
            if (kShift || few) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int c = 8 * v - at.shift + e;
                    float g[2], b[2];
                    vlp::f2_unpack(ag[i][e / 2], g[0], g[1]);
                    vlp::f2_unpack(ab[i][e / 2], b[0], b[1]);
                    if (at.has(c)) row[c] = g[e % 2], row[C + c] = b[e % 2];
                }
            } else {
                store8<VLPROJ_F32>(row + 8 * v, pack8<VLPROJ_F32>(ag[i]));
                store8<VLPROJ_F32>(row + C + 8 * v, pack8<VLPROJ_F32>(ab[i]));
            }
        }
    } else {
        // one slice of 2 x 8 nvec sums per warp; lanes of one warp that share columns are added first
        __syncthreads();
        float* sums = reinterpret_cast<float*>(ring);
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < kVec; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int o = kLanes; o < 32; o <<= 1) {
                    ag[i][e] = vlp::f2_add(ag[i][e], __shfl_xor_sync(0xffffffffu, ag[i][e], o));
                    ab[i][e] = vlp::f2_add(ab[i][e], __shfl_xor_sync(0xffffffffu, ab[i][e], o));
                }
        if (lane < kLanes) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int v = j + i * group;
                if (v >= nvec) continue;
                const Raw8<VLPROJ_F32> g = pack8<VLPROJ_F32>(ag[i]), b = pack8<VLPROJ_F32>(ab[i]);
                uint4* slice = reinterpret_cast<uint4*>(sums + warp * 16 * nvec);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    slice[2 * v + h] = g.w[h];
                    slice[2 * nvec + 2 * v + h] = b.w[h];
                }
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * C; c += LN_GRAD_THREADS) {
            const float* sum = sums + (c < C ? c : 8 * nvec + c - C) + at.shift;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < LN_GRAD_THREADS / 32; ++w) s += sum[w * 16 * nvec];
            row[c] = s;
        }
    }
    if (!few) return;
    // the grid is one cluster: every block adds its part of the columns over all blocks, in order
    auto cluster = cooperative_groups::this_cluster();
    cluster.sync();
    for (int c = static_cast<int>(blockIdx.x) * threads + static_cast<int>(threadIdx.x); c < 2 * C; c += LN_FEW_BLOCKS * threads) {
        float s = 0.f;
#pragma unroll
        for (int b = 0; b < LN_FEW_BLOCKS; ++b) s += cluster.map_shared_rank(row, b)[c];
        float* out = c < C ? d_gamma : d_beta;
        if (out != nullptr) out[c < C ? c : c - C] = s;
    }
    cluster.sync();                                      // no block ends while another reads its sums
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
    const float total = warp_add(s), mean = ln_mean(total, inv_c, ln_inverse_rest(inv_c, C));
    float q = 0.f;
#pragma unroll 4
    for (int c = lane; c < C; c += 32) {
        const float d = Elem<kX>::up(__ldg(src + c)) - mean;
        q += d * d;
    }
    const float rstd = 1.0f / sqrtf(warp_add(q) * inv_c + eps);
    if (lane == 0) {
        if (mean_out) mean_out[r] = mean == mean ? mean : total * inv_c;
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

// Row-block sums of d_gamma and d_beta of any layout, a thread per column: over the rows of
// block b, sum_g[b pitch + c] and sum_b[b pitch + c] (each unless null).
template <int kX, int kY>
static __global__ void __launch_bounds__(128) vlp_ln_part_any_kernel(const void* __restrict__ x, int64_t x_ld,
                                                                     const float* __restrict__ mean_in,
                                                                     const float* __restrict__ rstd_in,
                                                                     const void* __restrict__ dy, int64_t dy_ld,
                                                                     int64_t rows, int per, int C,
                                                                     float* __restrict__ sum_g,
                                                                     float* __restrict__ sum_b, int64_t pitch) {
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
    if (sum_g != nullptr) sum_g[blockIdx.x * pitch + c] = sg;
    if (sum_b != nullptr) sum_b[blockIdx.x * pitch + c] = sb;
}

// d_gamma[c] = sum of part[b][0][c], d_beta[c] = sum of part[b][1][c] over b < nb: a block
// takes 32 of the 2C sums with kGroups groups of row blocks (b = g, g + groups, ...),
// each added in fp32 over its at most 37 blocks, LN_JOIN_BATCH loads in flight; the groups
// are joined in order in fp64. The sums come by plain loads: the kernel may start while the
// one that writes them still runs, so they are not read-only for its whole life.
constexpr int LN_JOIN_BATCH = 8;
template <int kGroups>
static __global__ void __launch_bounds__(32 * kGroups) vlp_ln_join_kernel(const float* part, int nb,
                                                                                int C, float* __restrict__ d_gamma,
                                                                                float* __restrict__ d_beta) {
    __shared__ float red[kGroups][32];
    const int col = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const uint32_t c = blockIdx.x * 32 + col, width = 2 * static_cast<uint32_t>(C);      // all sums: below 2^31 elements
    float t = 0.f;
    after_previous_kernel(part);
    const float* column = part + (c < width ? c : 0);
    for (int b = grp; b < nb; b += kGroups * LN_JOIN_BATCH) {
        float v[LN_JOIN_BATCH];
#pragma unroll
        for (int q = 0; q < LN_JOIN_BATCH; ++q) {              // no load behind a branch: all in flight at once
            const int row = b + q * kGroups;
            v[q] = column[static_cast<uint32_t>(row < nb ? row : b) * width];
        }
#pragma unroll
        for (int q = 0; q < LN_JOIN_BATCH; ++q) t += b + q * kGroups < nb ? v[q] : 0.f;
    }
    red[grp][col] = t;
    __syncthreads();
    if (grp != 0 || c >= width) return;
    double s = 0.;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) s += red[g][col];
    if (c < static_cast<uint32_t>(C)) {
        if (d_gamma) d_gamma[c] = static_cast<float>(s);
    } else if (d_beta) {
        d_beta[c - C] = static_cast<float>(s);
    }
}

}  // namespace vlp_ops
