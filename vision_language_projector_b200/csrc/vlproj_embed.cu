// Token-embedding lookup and the gradient of its table (declared in vlproj.h as
// vlproj_embed, vlproj_embed_backward).
#include "kernels_embed.cuh"

#include <algorithm>

using namespace vlp_ops;

namespace {

constexpr int64_t kMaxCount = int64_t(1) << 31;

struct SortPlan {
    int passes, bits, blocks, run, pitch;
};

// Digits of at most SORT_MAX_BITS bits, as equal as possible. One tile a block, more once
// there are SORT_MAX_BLOCKS.
SortPlan sort_plan(int64_t n, int64_t vocab) {
    SortPlan p;
    int bits = 1;
    while ((vocab >> bits) != 0) ++bits;                  // keys 0 .. vocab
    p.passes = (bits + SORT_MAX_BITS - 1) / SORT_MAX_BITS;
    p.bits = (bits + p.passes - 1) / p.passes;
    const int64_t tiles = (n + SORT_TILE - 1) / SORT_TILE;
    const int64_t per = (tiles + SORT_MAX_BLOCKS - 1) / SORT_MAX_BLOCKS;
    p.run = static_cast<int>(per * SORT_TILE);
    p.blocks = static_cast<int>((tiles + per - 1) / per);
    p.pitch = (p.blocks + 3) / 4 * 4;
    return p;
}

// How the rows are cut into chunks: SUM_MAX_ROWS rows, fewer (16 at least) while there are
// too few blocks to fill the GPU (65536 x 2560 bf16, most rows dropped: 222 us with 128 rows,
// 210 us with 64). The same for every alignment, so that the workspace follows from n and N
// alone.
struct SumPlan {
    int rows;
    int64_t chunks;
};
SumPlan sum_plan(int64_t n, int64_t N) {
    const int64_t wide_tiles = (N + 1023) / 1024;
    SumPlan p;
    p.rows = SUM_MAX_ROWS;
    while (p.rows > 16 && n / p.rows * wide_tiles < 2048) p.rows /= 2;
    p.chunks = (n + p.rows - 1) / p.rows;
    return p;
}

bool ids_ok(const int64_t* ids, int64_t n) { return (n == 0 || ids != nullptr) && reinterpret_cast<uintptr_t>(ids) % 8 == 0; }

int64_t round256(int64_t b) { return (b + 255) / 256 * 256; }

}  // namespace

extern "C" {

int vlproj_embed(const vlproj_embed_args* a, void* stream) {
    if (!a || a->n_ids < 0 || a->n_ids >= kMaxCount || a->vocab < 0 || a->vocab >= kMaxCount || a->N < 1 ||
        a->N > VLPROJ_MAX_WIDTH || !known_pair(a->table_type, a->out_type))
        return VLPROJ_ERR_INVALID_ARG;
    if (!ids_ok(a->input_ids, a->n_ids)) return VLPROJ_ERR_INVALID_ARG;
    if (!matrix_ok(a->table, a->vocab, a->N, a->table_ld, a->table_type) ||
        !matrix_ok(a->out, a->n_ids, a->N, a->out_ld, a->out_type))
        return VLPROJ_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(a->status) % 4) return VLPROJ_ERR_INVALID_ARG;
    const Span out[2] = {span_of(a->out, a->n_ids, a->N, a->out_ld, type_size(a->out_type)),
                         span_of(a->status, a->status ? 1 : 0, 1, 1, 4)};
    const Span in[2] = {span_of(a->table, a->vocab, a->N, a->table_ld, type_size(a->table_type)),
                        span_of(a->input_ids, 1, a->n_ids, a->n_ids, 8)};
    if (any_overlap(out, 2, in, 2)) return VLPROJ_ERR_INVALID_ARG;
    if (a->n_ids == 0) return VLPROJ_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool wide = rows_wide(a->table, a->table_ld, a->table_type) && rows_wide(a->out, a->out_ld, a->out_type);
    const int copy = a->table_type == a->out_type && a->scale == 1.0f;
    const int seg = wide ? embed_segment<true>() : embed_segment<false>();
    const dim3 blocks(static_cast<unsigned>((a->n_ids + 7) / 8), static_cast<unsigned>((a->N + seg - 1) / seg));
    dispatch_pair(a->table_type, a->out_type, [&](auto in, auto out) {
        auto k = wide ? vlp_embed_rows_kernel<in.value, out.value, true> : vlp_embed_rows_kernel<in.value, out.value, false>;
        k<<<blocks, 256, 0, s>>>(a->input_ids, a->n_ids, a->image_token_id, a->table, a->vocab, a->table_ld, a->out,
                                 a->out_ld, static_cast<int>(a->N), a->scale, copy, a->status);
    });
    return cudaGetLastError() == cudaSuccess ? VLPROJ_OK : VLPROJ_ERR_CUDA;
}

int64_t vlproj_embed_backward_workspace(int64_t n, int64_t N) {
    if (n < 0 || n >= kMaxCount || N < 1 || N > VLPROJ_MAX_WIDTH) return VLPROJ_ERR_INVALID_ARG;
    if (n <= SMALL_MAX_IDS) return 256;                    // not used
    return 2 * round256(8 * n) + round256(4 * int64_t(SORT_MAX_BLOCKS) * SORT_MAX_BINS) +
           round256(8 * sum_plan(n, N).chunks * N);
}

int vlproj_embed_backward(const vlproj_embed_backward_args* a, void* stream) {
    if (!a || a->n_ids < 0 || a->n_ids >= kMaxCount || a->vocab < 0 || a->vocab >= kMaxCount || a->N < 1 ||
        a->N > VLPROJ_MAX_WIDTH || !known_type(a->d_out_type))
        return VLPROJ_ERR_INVALID_ARG;
    if (!ids_ok(a->input_ids, a->n_ids)) return VLPROJ_ERR_INVALID_ARG;
    if (!matrix_ok(a->d_out, a->n_ids, a->N, a->d_out_ld, a->d_out_type) ||
        !matrix_ok(a->d_table, a->vocab, a->N, a->d_table_ld, VLPROJ_F32))
        return VLPROJ_ERR_INVALID_ARG;
    const int64_t need = vlproj_embed_backward_workspace(a->n_ids, a->N);
    if (!workspace_ok(a->workspace, a->workspace_bytes, need)) return VLPROJ_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(a->status) % 4) return VLPROJ_ERR_INVALID_ARG;
    const Span out[3] = {span_of(a->d_table, a->vocab, a->N, a->d_table_ld, 4), span_of(a->workspace, 1, need, need, 1),
                         span_of(a->status, a->status ? 1 : 0, 1, 1, 4)};
    const Span in[2] = {span_of(a->d_out, a->n_ids, a->N, a->d_out_ld, type_size(a->d_out_type)),
                        span_of(a->input_ids, 1, a->n_ids, a->n_ids, 8)};
    if (any_overlap(out, 3, in, 2)) return VLPROJ_ERR_INVALID_ARG;
    const int64_t n = a->n_ids;
    const bool out_wide = rows_wide(a->d_table, a->d_table_ld, VLPROJ_F32);
    // Elements of an access: 8 or 2 where all rows are aligned for it (83960 x 578 fp16: the
    // sums take 35 us two at a time and 72 us one at a time).
    const int esize = static_cast<int>(type_size(a->d_out_type));
    int width = 1;
    if (rows_wide(a->d_out, a->d_out_ld, a->d_out_type) && out_wide && a->N % 8 == 0) width = 8;
    else if (a->N % 2 == 0 && a->d_out_ld % 2 == 0 && a->d_table_ld % 2 == 0 &&
             reinterpret_cast<uintptr_t>(a->d_out) % (2 * esize) == 0 && reinterpret_cast<uintptr_t>(a->d_table) % 8 == 0)
        width = 2;
    // Few ids are compared with one another instead of sorted, in one launch. Python calls one
    // after another, into 1000 rows of 512: 1024 ids take 10 us so and 17 us by sorting, 2048 ids 16
    // and 20 us, 3000 ids 22 and 19, 4096 ids 28 and 21. Wide rows of a small table lose sooner,
    // as one block adds all rows of a frequent token: 1024 x 4096 22 and 25 us, 2048 x 1024 28 and
    // 23, 2048 x 4096 33 and 27. Into 32000 rows: 2048 x 64 21 and 27, 2048 x 512 27 and 34, 2048 x
    // 4096 114 and 119 us.
    const bool few = n <= SMALL_MAX_IDS;
    const SumPlan plan = sum_plan(n, a->N);
    const int cols = width == 1 ? 4 : 8;                                 // of a thread
    const int64_t threads = (a->N + cols - 1) / cols;
    const int groups = few ? 1 : threads <= 32 ? 4 : threads <= 64 ? 2 : 1;
    const int tiles = static_cast<int>((a->N + cols * (SUM_THREADS / groups) - 1) / (cols * (SUM_THREADS / groups)));
    // The join: a frequent token of a small vocabulary leaves hundreds of partial sums, one
    // behind the other; narrow rows leave threads to share them (83960 x 578, 328 tokens: 34 us
    // by one group, 24 us by four). Wide rows have too many blocks that find nothing.
    const int jgroups = a->N <= 256 ? 8 : a->N <= 1024 ? 4 : a->N <= 2048 ? 2 : 1;
    const int jcols = 4 * JOIN_THREADS / jgroups;
    const int jtiles = static_cast<int>((a->N + jcols - 1) / jcols);
    const int64_t zeros = a->accumulate ? 0 : (a->vocab + ZERO_TOKENS - 1) / ZERO_TOKENS;
    const int64_t sums = (few ? n : (plan.chunks + groups - 1) / groups) * tiles;
    if (sums + zeros >= kMaxCount || plan.chunks * jtiles >= kMaxCount) return VLPROJ_ERR_INVALID_ARG;      // grid size
    // an empty table has no row to write, but its ids, all outside it, are still reported
    if (sums + zeros == 0 || (a->vocab == 0 && a->status == nullptr)) return VLPROJ_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const ScatterOut o{a->d_table, a->d_table_ld, a->vocab, static_cast<int>(a->N), a->scale, a->accumulate != 0};
    const unsigned blocks = static_cast<unsigned>(sums + zeros);
    auto with_type = [&](auto&& f) {
        auto with_width = [&](auto type) {
            if (width == 8) f(type, type_tag<8>());
            else if (width == 2) f(type, type_tag<2>());
            else f(type, type_tag<1>());
        };
        if (a->d_out_type == VLPROJ_BF16) with_width(type_tag<VLPROJ_BF16>());
        else if (a->d_out_type == VLPROJ_F16) with_width(type_tag<VLPROJ_F16>());
        else with_width(type_tag<VLPROJ_F32>());
    };
    if (few) {
        with_type([&](auto type, auto wd) {
            vlp_scatter_few_kernel<type.value, wd.value><<<blocks, SUM_THREADS, 0, s>>>(
                a->input_ids, static_cast<int>(n), a->image_token_id, tiles, static_cast<unsigned>(sums), a->d_out,
                a->d_out_ld, o, a->status);
        });
        return cudaGetLastError() == cudaSuccess ? VLPROJ_OK : VLPROJ_ERR_CUDA;
    }
    uint8_t* w = static_cast<uint8_t*>(a->workspace);
    uint64_t* pairs[2] = {reinterpret_cast<uint64_t*>(w), reinterpret_cast<uint64_t*>(w + round256(8 * n))};
    w += 2 * round256(8 * n);
    uint32_t* counts = reinterpret_cast<uint32_t*>(w);
    float* part = reinterpret_cast<float*>(w + round256(4 * int64_t(SORT_MAX_BLOCKS) * SORT_MAX_BINS));
    SortSource src{a->input_ids, nullptr, n, a->image_token_id, a->vocab, a->status};
    const SortPlan p = sort_plan(n, a->vocab);
    const int bins = 1 << p.bits;
    for (int i = 0; i < p.passes; ++i) {
        if (i == 0)
            vlp_sort_count_kernel<<<p.blocks, SORT_THREADS, 0, s>>>(src, p.run, 0, bins, p.pitch, counts);
        else
            launch_after(vlp_sort_count_kernel, p.blocks, SORT_THREADS, 0, s, src, p.run, i * p.bits, bins, p.pitch, counts);
        launch_after(vlp_sort_scatter_kernel, p.blocks, SORT_THREADS, 0, s, src, p.run, i * p.bits, bins, p.blocks, p.pitch,
                     counts, pairs[i & 1]);
        src.ids = nullptr;
        src.pairs = pairs[i & 1];
    }
    with_type([&](auto type, auto wd) {
        auto k = groups == 4 ? vlp_scatter_sum_kernel<type.value, wd.value, 4>
                 : groups == 2 ? vlp_scatter_sum_kernel<type.value, wd.value, 2>
                               : vlp_scatter_sum_kernel<type.value, wd.value, 1>;
        launch_after(k, blocks, SUM_THREADS, 0, s, src.pairs, n, plan.rows, tiles, static_cast<unsigned>(sums), a->d_out,
                     a->d_out_ld, o, part);
    });
    if (plan.chunks > 1) {
        auto k = jgroups == 8 ? vlp_scatter_join_kernel<8> : jgroups == 4 ? vlp_scatter_join_kernel<4>
                 : jgroups == 2 ? vlp_scatter_join_kernel<2> : vlp_scatter_join_kernel<1>;
        launch_after(k, static_cast<unsigned>((plan.chunks - 1) * jtiles), JOIN_THREADS, 0, s, src.pairs, n, plan.rows,
                     jtiles, part, o);
    }
    return cudaGetLastError() == cudaSuccess ? VLPROJ_OK : VLPROJ_ERR_CUDA;
}

}  // extern "C"
