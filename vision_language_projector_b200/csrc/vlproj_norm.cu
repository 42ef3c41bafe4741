// Layer norm (declared in vlproj.h as vlproj_layernorm).
#include "norm_host.cuh"

using namespace vlp_ops;

extern "C" {

int vlproj_layernorm(const vlproj_layernorm_args* a, void* stream) {
    if (!a || !shape_ok(a->rows, a->C, a->x_type, a->y_type)) return VLPROJ_ERR_INVALID_ARG;
    if (!matrix_ok(a->x, a->rows, a->C, a->x_ld, a->x_type) || !matrix_ok(a->y, a->rows, a->C, a->y_ld, a->y_type) ||
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
            constexpr int vec = decltype(shape)::vec, words = x.value == VLPROJ_F32 ? 2 : 1;
            // a warp's rows of up to 10 KB; in blocks of 8 warps where 4 would leave an SM with
            // too few rows on their way
            if constexpr (lanes != 0 && vec * words > 20) return false; else {
            constexpr int most = lanes ? (vec * words > 10 ? 256 : 128) : decltype(shape)::threads;
            // Rows in the ring, the one at hand among them: fewer the longer they are, as more of them
            // cost resident blocks. Of a warp's rows four up to 2560 bytes (six: 300000 x 96 bf16 28.7 us
            // instead of 26.8, 160000 x 256 fp32 61.4 and 60.2, others alike), three up to 5120 (100000
            // x 1600 bf16 104 us; two 119, four 146), else two. Of a block's rows two (four: 20000 x 9216
            // bf16 203 us instead of 184, 12000 x 4096 fp32 to bf16 51 and 48, 25000 x 7168 143 and 142,
            // 24693 x 7618 260 and 262).
            constexpr int stages = lanes ? (vec * words <= 5 ? 4 : vec * words <= 10 ? 3 : 2) : 2;
            constexpr bool shifts = vec <= 10;          // longer shifted rows are held by a block
            if (cut == kShifted && !shifts) return false;
            // and so are long rows too few to give every SM one: of the kernel alone, 64 x 5120 bf16
            // takes 4.1 us by blocks and 6.3 us by warps, 512 x 5120 8.1 and 6.5 us
            if (lanes && vec >= 10 && a->rows <= sm_count()) return false;
            auto k = cut == kAligned ? vlp_ln_rows_kernel<x.value, y.value, false, lanes, vec, most, stages>
                                     : vlp_ln_rows_kernel<x.value, y.value, shifts, lanes, vec, most, stages>;
            if (lanes) threads = most;
            const int smem = (lanes ? 64 * nvec : 0) + stages * vec * words * 16 * threads;
            if (smem > kMaxDynamicSmem) return false;
            static ResidentBlocks resident[2];
            const int per_sm = resident[cut].get(k, threads, smem);
            if (per_sm < 1) {
                rc = VLPROJ_ERR_CUDA;
                return true;
            }
            const int64_t groups = lanes ? most / (lanes ? lanes : 1) : 1;
            const int64_t blocks = row_blocks(cut, a->rows, groups, int64_t(per_sm) * sm_count());
            k<<<static_cast<unsigned>(blocks), threads, smem, s>>>(a->x, a->x_ld, a->y, a->y_ld, a->rows, C, a->gamma,
                                                                   a->beta, a->mean, a->rstd, eps);
            return true;
            }
        };
        if (cut != kAny && with_shape<20, LN_FWD_MAX_VEC>(nvec, launch)) return;
        vlp_ln_rows_any_kernel<x.value, y.value><<<static_cast<unsigned>((a->rows + 7) / 8), 256, 0, s>>>(
            a->x, a->x_ld, a->y, a->y_ld, a->rows, C, a->gamma, a->beta, a->mean, a->rstd, eps);
    });
    if (rc != VLPROJ_OK) return rc;
    return cudaGetLastError() == cudaSuccess ? VLPROJ_OK : VLPROJ_ERR_CUDA;
}

}  // extern "C"
