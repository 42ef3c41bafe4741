// Layer norm and its gradients (declared in vlproj.h as vlproj_layernorm,
// vlproj_layernorm_backward).
#include "kernels_norm.cuh"

#include <algorithm>

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

// Row blocks of the weight gradients' partial sums.
int part_blocks(int64_t rows) {
    return static_cast<int>(std::min<int64_t>(LN_MAX_PARTS, std::max<int64_t>(1, (rows + 31) / 32)));
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
    dispatch_pair(a->x_type, a->y_type, [&](auto x, auto y) {
        vlp_ln_rows_any_kernel<x.value, y.value><<<static_cast<unsigned>((a->rows + 7) / 8), 256, 0, s>>>(
            a->x, a->x_ld, a->y, a->y_ld, a->rows, C, a->gamma, a->beta, a->mean, a->rstd, eps);
    });
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
    const int nb = a->rows > 0 ? part_blocks(a->rows) : 0;
    float* part = static_cast<float*>(a->workspace);
    dispatch_pair(a->x_type, a->y_type, [&](auto x, auto y) {
        if (a->d_x && a->rows > 0)
            vlp_ln_dx_any_kernel<x.value, y.value><<<static_cast<unsigned>((a->rows + 7) / 8), 256, 0, s>>>(
                a->x, a->x_ld, a->mean, a->rstd, a->d_y, a->d_y_ld, a->gamma, a->d_x, a->d_x_ld, a->rows, C);
        if (weights && nb > 0)
            vlp_ln_part_any_kernel<x.value, y.value><<<dim3(nb, (C + 127) / 128), 128, 0, s>>>(
                a->x, a->x_ld, a->mean, a->rstd, a->d_y, a->d_y_ld, a->rows,
                static_cast<int>((a->rows + nb - 1) / nb), C, part);
    });
    if (weights)
        vlp_ln_join_kernel<<<static_cast<unsigned>((2 * a->C + 31) / 32), 256, 0, s>>>(part, nb, C, a->d_gamma, a->d_beta);
    return cudaGetLastError() == cudaSuccess ? VLPROJ_OK : VLPROJ_ERR_CUDA;
}

}  // extern "C"
