// Gradients of layer norm (declared in vlproj.h as vlproj_layernorm_backward).
#include "norm_host.cuh"

using namespace vlp_ops;

namespace {

// Rows few enough for one cluster (or, of any layout, one row block), which writes the
// weights' gradients itself, without a workspace. It saves a call from Python, one after
// another, the workspace and a launch: 8.9 to 10.2 us so and 13.2 us by two launches (64 x
// 1152, 16 x 5120, 512 x 256, 100 x 1280 bf16). On the GPU eight blocks take longer than the
// grid of the two launches: replayed in a graph 6.2 and 5.2 us for 64 x 1152, 7.3 and 4.2 us
// for 512 x 256, and C calls one after another 8.2 and 7.1, 10.2 and 6.2 us. More elements
// lose from Python too.
bool few_rows(int64_t rows, int64_t C) { return rows <= 512 && C <= 8192 && rows * C <= 128 * 1024; }

template <class K, class... Args>
void launch_cluster(K kernel, int threads, int64_t smem, cudaStream_t s, Args... args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = LN_FEW_BLOCKS;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = LN_FEW_BLOCKS;
    cfg.blockDim = threads;
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

extern "C" {

int64_t vlproj_layernorm_backward_workspace(int64_t rows, int64_t C) {
    if (rows < 0 || rows >= kMaxRows || C < 1 || C > VLPROJ_MAX_WIDTH) return VLPROJ_ERR_INVALID_ARG;
    return few_rows(rows, C) ? 0 : 8 * C * part_blocks(rows, C);
}

int vlproj_layernorm_backward(const vlproj_layernorm_backward_args* a, void* stream) {
    if (!a || !shape_ok(a->rows, a->C, a->x_type, a->y_type)) return VLPROJ_ERR_INVALID_ARG;
    if (!matrix_ok(a->x, a->rows, a->C, a->x_ld, a->x_type) || !matrix_ok(a->d_y, a->rows, a->C, a->d_y_ld, a->y_type) ||
        (a->d_x && !matrix_ok(a->d_x, a->rows, a->C, a->d_x_ld, a->x_type)) || !vec_ok(a->gamma) || !vec_ok(a->mean) ||
        !vec_ok(a->rstd) || !vec_ok(a->d_gamma) || !vec_ok(a->d_beta) || (a->rows > 0 && (!a->mean || !a->rstd)))
        return VLPROJ_ERR_INVALID_ARG;
    const bool weights = a->d_gamma || a->d_beta;
    const int64_t need = weights ? vlproj_layernorm_backward_workspace(a->rows, a->C) : 0;
    if (need > 0 && !workspace_ok(a->workspace, a->workspace_bytes, need)) return VLPROJ_ERR_INVALID_ARG;
    const Span out[4] = {span_of(a->d_x, a->d_x ? a->rows : 0, a->C, a->d_x_ld, type_size(a->x_type)),
                         span_of(a->d_gamma, a->d_gamma ? 1 : 0, a->C, a->C, 4),
                         span_of(a->d_beta, a->d_beta ? 1 : 0, a->C, a->C, 4),
                         span_of(a->workspace, need > 0 ? 1 : 0, need, need, 1)};
    const Span in[5] = {span_of(a->x, a->rows, a->C, a->x_ld, type_size(a->x_type)),
                        span_of(a->d_y, a->rows, a->C, a->d_y_ld, type_size(a->y_type)),
                        span_of(a->mean, 1, a->rows, a->rows, 4), span_of(a->rstd, 1, a->rows, a->rows, 4),
                        span_of(a->gamma, a->gamma ? 1 : 0, a->C, a->C, 4)};
    if (any_overlap(out, 4, in, 5)) return VLPROJ_ERR_INVALID_ARG;
    if (!weights && !a->d_x) return VLPROJ_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int C = static_cast<int>(a->C);
    int nb = a->rows > 0 ? part_blocks(a->rows, a->C) : 0;
    float* part = need > 0 ? static_cast<float*>(a->workspace) : nullptr;
    const bool few = weights && a->rows > 0 && few_rows(a->rows, a->C);
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
            // A turn of two rows where a row is short, or where a whole block holds it and its two
            // barriers are worth sharing (8192 x 5120 bf16: 64 us with two rows, 70 us with one;
            // 50176 x 1152 in warps: 69 and 63 us), and a ring that keeps about 100 KB of rows on
            // their way to an SM.
            constexpr int most = lanes ? LN_GRAD_THREADS : decltype(shape)::threads;
            constexpr int turn = lanes ? (vec <= 2 ? 2 : 1) : (most <= 512 && words <= 3 ? 2 : 1);
            constexpr int stages = 2;
            int64_t smem = int64_t(stages) * turn * vec * words * 16 * threads;
            int few_at = 0;
            if (lanes) {
                const int64_t slices = 64 * int64_t(nvec) * (LN_GRAD_THREADS / 32);
                few_at = static_cast<int>((32 * int64_t(nvec) + slices) / 4);
                smem = 32 * int64_t(nvec) + std::max<int64_t>(smem, slices + (few ? 64 * int64_t(nvec) : 0));
            } else if (few) {
                smem = std::max<int64_t>(smem, 64 * int64_t(nvec));
            }
            if (smem > kMaxDynamicSmem) return false;
            auto k = cut == kAligned ? vlp_ln_grad_kernel<x.value, y.value, false, lanes, vec, most, turn, stages>
                                     : vlp_ln_grad_kernel<x.value, y.value, true, lanes, vec, most, turn, stages>;
            static ResidentBlocks resident[2];
            const int per_sm = resident[cut].get(k, threads, static_cast<int>(smem));
            if (per_sm < 1) {
                rc = VLPROJ_ERR_CUDA;
                return true;
            }
            if (few) {
                launch_cluster(k, threads, smem, s, a->x, a->x_ld, a->mean, a->rstd, a->d_y, a->d_y_ld, a->gamma, a->d_x,
                               a->d_x_ld, a->rows, C, nullptr, 1, few_at, a->d_gamma, a->d_beta);
                return true;
            }
            nb = static_cast<int>(row_blocks(cut, a->rows, groups,
                                             std::min<int64_t>(part_blocks(a->rows, a->C), int64_t(per_sm) * sm_count())));
            k<<<nb, threads, smem, s>>>(a->x, a->x_ld, a->mean, a->rstd, a->d_y, a->d_y_ld, a->gamma, a->d_x, a->d_x_ld,
                                        a->rows, C, part, 0, 0, nullptr, nullptr);
            return true;
        };
        if (cut != kAny && a->rows > 0 && with_shape<5, LN_BWD_MAX_VEC>(nvec, launch)) return;
        if (a->d_x && a->rows > 0)
            vlp_ln_dx_any_kernel<x.value, y.value><<<static_cast<unsigned>((a->rows + 7) / 8), 256, 0, s>>>(
                a->x, a->x_ld, a->mean, a->rstd, a->d_y, a->d_y_ld, a->gamma, a->d_x, a->d_x_ld, a->rows, C);
        if (few) nb = 1;
        if (weights && nb > 0)
            vlp_ln_part_any_kernel<x.value, y.value><<<dim3(nb, (C + 127) / 128), 128, 0, s>>>(
                a->x, a->x_ld, a->mean, a->rstd, a->d_y, a->d_y_ld, a->rows, static_cast<int>((a->rows + nb - 1) / nb), C,
                few ? a->d_gamma : part, few ? a->d_beta : part + C, few ? 0 : 2 * int64_t(C));
    });
    if (rc != VLPROJ_OK) return rc;
    if (weights && !few) {
        const unsigned blocks = static_cast<unsigned>((2 * a->C + 31) / 32);
        const int groups = blocks <= 148 ? 32 : 16;              // one wave of blocks either way
        launch_after(groups == 32 ? vlp_ln_join_kernel<32> : vlp_ln_join_kernel<16>, blocks, 32 * groups, 0, s, part, nb, C,
                     a->d_gamma, a->d_beta);
    }
    return cudaGetLastError() == cudaSuccess ? VLPROJ_OK : VLPROJ_ERR_CUDA;
}

}  // extern "C"
