// Layer norm and its gradients (declared in vlproj.h as vlproj_layernorm,
// vlproj_layernorm_backward).
#include "kernels_norm.cuh"

#include <algorithm>
#include <mutex>

using namespace vlp_ops;

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 31;

bool rows_ok(const void* p, int64_t rows, int64_t C, int64_t ld, int type) {
    return ld >= C && (rows == 0 || p != nullptr) && reinterpret_cast<uintptr_t>(p) % type_size(type) == 0;
}
bool vec_ok(const float* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }
bool shape_ok(int64_t rows, int64_t C, int x_type, int y_type) {
    return rows >= 0 && rows < kMaxRows && C >= 1 && C <= VLPROJ_MAX_WIDTH && known_pair(x_type, y_type);
}

// Most row blocks of the weight gradients' partial sums, a multiple of 8.
int part_blocks(int64_t rows) { return static_cast<int>(std::min<int64_t>(LN_MAX_PARTS, std::max<int64_t>(8, (rows + 63) / 64 * 8))); }

// How the matrices' rows can be cut into aligned vectors of 8 elements: all rows aligned and
// C % 8 == 0; or all matrices' rows equally far from an aligned vector; or neither.
enum { kAligned, kShifted, kAny };
struct Rows {
    const void* p;
    int64_t ld;
    int type;
    int64_t start() const { return static_cast<int64_t>(reinterpret_cast<uintptr_t>(p) / type_size(type) % 8); }
};
int cut_of(const Rows* m, int n, int64_t C, bool weights_aligned) {
    bool aligned = C % 8 == 0 && weights_aligned, equal = true;
    for (int i = 0; i < n; ++i) {
        aligned = aligned && rows_wide(m[i].p, m[i].ld, m[i].type);
        equal = equal && m[i].start() == m[0].start() && (m[i].ld - m[0].ld) % 8 == 0;
    }
    return aligned ? kAligned : equal ? kShifted : kAny;
}

// Blocks for `rows` rows, `groups` of them a block at a time, at most `most` blocks: for
// shifted rows a multiple of 8.
int64_t row_blocks(int cut, int64_t rows, int64_t groups, int64_t most) {
    if (cut != kShifted) return std::min((rows + groups - 1) / groups, most);
    return 8 * std::min(((rows + 7) / 8 + groups - 1) / groups, std::max<int64_t>(1, most / 8));
}

constexpr int64_t kMaxDynamicSmem = 227 * 1024 - 1024;      // of a block, beside its static part

// Resident blocks per SM of one kernel, asked of the runtime once for each device and
// block shape (threads and shared memory follow from the row length alone).
struct ResidentBlocks {
    struct Entry {
        int dev, threads, smem, blocks;
    };
    std::mutex lock;
    Entry known[64];
    int n = 0;
    template <class K>
    int get(K kernel, int threads, int smem) {
        int dev = 0, blocks = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return 0;
        std::lock_guard<std::mutex> hold(lock);
        for (int i = 0; i < n; ++i)
            if (known[i].dev == dev && known[i].threads == threads && known[i].smem == smem) return known[i].blocks;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMaxDynamicSmem)) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, kernel, threads, smem) != cudaSuccess)
            return 0;
        if (n < 64) known[n++] = Entry{dev, threads, smem, blocks};
        return blocks;
    }
};

template <int kLanes, int kVec, int kThreads = LN_MAX_THREADS>
struct Shape {
    static constexpr int lanes = kLanes, vec = kVec, threads = kThreads;
};

// Calls f(Shape, threads) for the way rows of nvec vectors are held: kLanes lanes of a warp
// with up to 5 vectors each, or a whole block with up to kMaxBlockVec. False when no way
// fits.
template <int kMaxBlockVec, class F>
bool with_shape(int nvec, F&& f) {
    if (nvec <= 8) return f(Shape<8, 1>(), 256);
    if (nvec <= 16) return f(Shape<16, 1>(), 256);
    if (nvec <= 32) return f(Shape<32, 1>(), 256);
    if (nvec <= 64) return f(Shape<32, 2>(), 256);
    if (nvec <= 96) return f(Shape<32, 3>(), 256);
    if (nvec <= 128) return f(Shape<32, 4>(), 256);
    if (nvec <= 160) return f(Shape<32, 5>(), 256);
    const auto threads = [&](int vec) { return (nvec + 32 * vec - 1) / (32 * vec) * 32; };
    if constexpr (kMaxBlockVec == 2) {
        if (nvec <= 1024) return f(Shape<0, 2, 512>(), threads(2));          // 128 registers a thread
        if (nvec <= 2 * LN_MAX_THREADS) return f(Shape<0, 2>(), threads(2));
    } else {
        if (nvec <= 1024) return f(Shape<0, 2>(), threads(2));
        if (nvec <= 4 * 512) return f(Shape<0, 4>(), threads(4));
        if (nvec <= kMaxBlockVec * LN_MAX_THREADS) return f(Shape<0, kMaxBlockVec>(), threads(kMaxBlockVec));
    }
    return false;
}

}  // namespace

extern "C" {

int vlproj_layernorm(const vlproj_layernorm_args* a, void* stream) {
    if (!a || !shape_ok(a->rows, a->C, a->x_type, a->y_type)) return VLPROJ_ERR_INVALID_ARG;
    if (!rows_ok(a->x, a->rows, a->C, a->x_ld, a->x_type) || !rows_ok(a->y, a->rows, a->C, a->y_ld, a->y_type) ||
        !vec_ok(a->gamma) || !vec_ok(a->beta) || !vec_ok(a->mean) || !vec_ok(a->rstd))
        return VLPROJ_ERR_INVALID_ARG;
    const Span out[3] = {span_of(a->y, a->rows, a->C, a->y_ld, type_size(a->y_type)),
                         span_of(a->mean, a->mean ? 1 : 0, a->rows, a->rows, 4),
                         span_of(a->rstd, a->rstd ? 1 : 0, a->rows, a->rows, 4)};
    const Span in[3] = {span_of(a->x, a->rows, a->C, a->x_ld, type_size(a->x_type)),
                        span_of(a->gamma, a->gamma ? 1 : 0, a->C, a->C, 4),
                        span_of(a->beta, a->beta ? 1 : 0, a->C, a->C, 4)};
    if (any_overlap(out, 3, in, 3)) return VLPROJ_ERR_INVALID_ARG;
    if (a->rows == 0) return VLPROJ_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const float eps = a->eps > 0.f ? a->eps : 1e-5f;
    const int C = static_cast<int>(a->C);
    const Rows all[2] = {{a->x, a->x_ld, a->x_type}, {a->y, a->y_ld, a->y_type}};
    const int cut = cut_of(all, 2, a->C, aligned16(a->gamma) && aligned16(a->beta));
    const int nvec = static_cast<int>(cut == kAligned ? a->C / 8 : (a->C + 14) / 8);
    int rc = VLPROJ_OK;
    dispatch_pair(a->x_type, a->y_type, [&](auto x, auto y) {
        auto launch = [&](auto shape, int threads) {
            constexpr int lanes = decltype(shape)::lanes;
            constexpr int vec = decltype(shape)::vec, stages = vec <= 2 ? 6 : vec < 8 ? 4 : 2;
            constexpr int words = x.value == VLPROJ_F32 ? 2 : 1;
            constexpr int most = lanes ? LN_FWD_THREADS : decltype(shape)::threads;
            auto k = cut == kAligned ? vlp_ln_rows_kernel<x.value, y.value, false, lanes, vec, most, stages>
                                     : vlp_ln_rows_kernel<x.value, y.value, true, lanes, vec, most, stages>;
            if (lanes) threads = LN_FWD_THREADS;
            const int smem = (lanes ? 64 * nvec : 0) + stages * vec * words * 16 * threads;
            if (smem > kMaxDynamicSmem) return false;
            static ResidentBlocks resident[2];
            const int per_sm = resident[cut].get(k, threads, smem);
            if (per_sm < 1) {
                rc = VLPROJ_ERR_CUDA;
                return true;
            }
            const int64_t groups = lanes ? LN_FWD_THREADS / (lanes ? lanes : 1) : 1;
            const int64_t blocks = row_blocks(cut, a->rows, groups, int64_t(per_sm) * sm_count());
            k<<<static_cast<unsigned>(blocks), threads, smem, s>>>(a->x, a->x_ld, a->y, a->y_ld, a->rows, C, a->gamma,
                                                                   a->beta, a->mean, a->rstd, eps);
            return true;
        };
        if (cut != kAny && with_shape<LN_FWD_MAX_VEC>(nvec, launch)) return;
        vlp_ln_rows_any_kernel<x.value, y.value><<<static_cast<unsigned>((a->rows + 7) / 8), 256, 0, s>>>(
            a->x, a->x_ld, a->y, a->y_ld, a->rows, C, a->gamma, a->beta, a->mean, a->rstd, eps);
    });
    if (rc != VLPROJ_OK) return rc;
    return cudaGetLastError() == cudaSuccess ? VLPROJ_OK : VLPROJ_ERR_CUDA;
}

int64_t vlproj_layernorm_backward_workspace(int64_t rows, int64_t C) {
    if (rows < 0 || rows >= kMaxRows || C < 1 || C > VLPROJ_MAX_WIDTH) return VLPROJ_ERR_INVALID_ARG;
    return 8 * C * part_blocks(rows);
}

int vlproj_layernorm_backward(const vlproj_layernorm_backward_args* a, void* stream) {
    if (!a || !shape_ok(a->rows, a->C, a->x_type, a->y_type)) return VLPROJ_ERR_INVALID_ARG;
    if (!rows_ok(a->x, a->rows, a->C, a->x_ld, a->x_type) || !rows_ok(a->d_y, a->rows, a->C, a->d_y_ld, a->y_type) ||
        (a->d_x && !rows_ok(a->d_x, a->rows, a->C, a->d_x_ld, a->x_type)) || !vec_ok(a->gamma) || !vec_ok(a->mean) ||
        !vec_ok(a->rstd) || !vec_ok(a->d_gamma) || !vec_ok(a->d_beta) || (a->rows > 0 && (!a->mean || !a->rstd)))
        return VLPROJ_ERR_INVALID_ARG;
    const bool weights = a->d_gamma || a->d_beta;
    const int64_t need = weights ? vlproj_layernorm_backward_workspace(a->rows, a->C) : 0;
    if (weights && (!a->workspace || !aligned16(a->workspace) || a->workspace_bytes < need)) return VLPROJ_ERR_INVALID_ARG;
    const Span out[4] = {span_of(a->d_x, a->d_x ? a->rows : 0, a->C, a->d_x_ld, type_size(a->x_type)),
                         span_of(a->d_gamma, a->d_gamma ? 1 : 0, a->C, a->C, 4),
                         span_of(a->d_beta, a->d_beta ? 1 : 0, a->C, a->C, 4),
                         span_of(a->workspace, weights ? 1 : 0, need, need, 1)};
    const Span in[5] = {span_of(a->x, a->rows, a->C, a->x_ld, type_size(a->x_type)),
                        span_of(a->d_y, a->rows, a->C, a->d_y_ld, type_size(a->y_type)),
                        span_of(a->mean, 1, a->rows, a->rows, 4), span_of(a->rstd, 1, a->rows, a->rows, 4),
                        span_of(a->gamma, a->gamma ? 1 : 0, a->C, a->C, 4)};
    if (any_overlap(out, 4, in, 5)) return VLPROJ_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int C = static_cast<int>(a->C);
    int nb = a->rows > 0 ? part_blocks(a->rows) : 0;
    float* part = weights ? static_cast<float*>(a->workspace) : nullptr;
    const Rows all[3] = {{a->x, a->x_ld, a->x_type}, {a->d_y, a->d_y_ld, a->y_type}, {a->d_x, a->d_x_ld, a->x_type}};
    const int cut = cut_of(all, a->d_x ? 3 : 2, a->C, aligned16(a->gamma));
    const int nvec = static_cast<int>(cut == kAligned ? a->C / 8 : (a->C + 14) / 8);
    int rc = VLPROJ_OK;
    dispatch_pair(a->x_type, a->y_type, [&](auto x, auto y) {
        auto launch = [&](auto shape, int threads) {
            constexpr int lanes = decltype(shape)::lanes, vec = decltype(shape)::vec;
            constexpr int words = (x.value == VLPROJ_F32 ? 2 : 1) + (y.value == VLPROJ_F32 ? 2 : 1);
            if (lanes) threads = LN_GRAD_THREADS;
            const int64_t groups = lanes ? LN_GRAD_THREADS / (lanes ? lanes : 1) : 1;
            // Deep enough a ring that three blocks an SM, or one wide block, keep about 100 KB
            // of rows in flight; the shallow one where that does not fit.
            auto with_ring = [&](auto row_count, auto stage_count) {
                constexpr int turn = decltype(row_count)::value, stages = decltype(stage_count)::value;
                int64_t smem = int64_t(stages) * turn * vec * words * 16 * threads;
                if (lanes) smem = 32 * int64_t(nvec) + std::max<int64_t>(smem, 64 * int64_t(nvec) * (LN_GRAD_THREADS / 32));
                if (smem > kMaxDynamicSmem) return false;
                constexpr int most = lanes ? LN_GRAD_THREADS : decltype(shape)::threads;
                auto k = cut == kAligned ? vlp_ln_grad_kernel<x.value, y.value, false, lanes, vec, most, turn, stages>
                                         : vlp_ln_grad_kernel<x.value, y.value, true, lanes, vec, most, turn, stages>;
                static ResidentBlocks resident[2];
                const int per_sm = resident[cut].get(k, threads, static_cast<int>(smem));
                if (per_sm < 1) {
                    rc = VLPROJ_ERR_CUDA;
                    return true;
                }
                nb = static_cast<int>(row_blocks(cut, a->rows, groups,
                                                 std::min<int64_t>(part_blocks(a->rows), int64_t(per_sm) * sm_count())));
                k<<<nb, threads, smem, s>>>(a->x, a->x_ld, a->mean, a->rstd, a->d_y, a->d_y_ld, a->gamma, a->d_x,
                                            a->d_x_ld, a->rows, C, part);
                return true;
            };
            constexpr int turn = vec <= 2 ? 2 : 1;
            constexpr int deep = vec == 1 ? 4 : 2;
            return with_ring(type_tag<turn>(), type_tag<deep>()) || with_ring(type_tag<1>(), type_tag<2>());
        };
        if (cut != kAny && a->rows > 0 && with_shape<LN_BWD_MAX_VEC>(nvec, launch)) return;
        if (a->d_x && a->rows > 0)
            vlp_ln_dx_any_kernel<x.value, y.value><<<static_cast<unsigned>((a->rows + 7) / 8), 256, 0, s>>>(
                a->x, a->x_ld, a->mean, a->rstd, a->d_y, a->d_y_ld, a->gamma, a->d_x, a->d_x_ld, a->rows, C);
        if (weights && nb > 0)
            vlp_ln_part_any_kernel<x.value, y.value><<<dim3(nb, (C + 127) / 128), 128, 0, s>>>(
                a->x, a->x_ld, a->mean, a->rstd, a->d_y, a->d_y_ld, a->rows,
                static_cast<int>((a->rows + nb - 1) / nb), C, part);
    });
    if (rc != VLPROJ_OK) return rc;
    if (weights) {
        const unsigned blocks = static_cast<unsigned>((2 * a->C + 31) / 32);
        launch_after(vlp_ln_join_kernel, blocks, 32 * LN_JOIN_GROUPS, 0, s, part, nb, C, a->d_gamma, a->d_beta);
    }
    return cudaGetLastError() == cudaSuccess ? VLPROJ_OK : VLPROJ_ERR_CUDA;
}

}  // extern "C"
