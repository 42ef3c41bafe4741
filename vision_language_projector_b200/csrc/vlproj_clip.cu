// Global gradient norm and clipping over many tensors (declared in vlproj.h as
// vlproj_clip_grads).
#include "kernels_clip.cuh"

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

using namespace vlp_ops;

namespace {

constexpr int kTable = 448;                             // tensors per launch (a kernel's arguments hold 32 KB)
constexpr int kFewTensors = 32;                         // a smaller table, launched sooner
constexpr int64_t kMaxTensors = 1 << 20;

int tables(int32_t n) { return std::max(1, (n + kTable - 1) / kTable); }

// Whether any of the outputs (the norm and the used bytes of the workspace among them)
// overlaps another tensor's gradient or output.
bool clash(const vlproj_clip_grads_args* a, int64_t workspace_used) {
    const Span norm = span_of(a->norm, a->norm ? 1 : 0, 1, 1, 4);
    const Span scratch = span_of(a->workspace, 1, workspace_used, workspace_used, 1);
    if (overlap(norm, scratch)) return true;
    if (!a->out) {                                     // gradients that are only read may share memory
        for (int32_t i = 0; i < a->n; ++i) {
            const Span g = span_of(a->grads[i], 1, a->numel[i], a->numel[i], type_size(a->type[i]));
            if (overlap(norm, g) || overlap(scratch, g)) return true;
        }
        return false;
    }
    struct Range {
        Span s;
        bool written;
    };
    std::vector<Range> r;
    r.reserve(2 * static_cast<size_t>(a->n) + 2);
    if (a->norm) r.push_back({norm, true});
    if (workspace_used > 0) r.push_back({scratch, true});
    for (int32_t i = 0; i < a->n; ++i) {
        if (a->numel[i] == 0) continue;
        const int64_t sz = type_size(a->type[i]);
        const Span g = span_of(a->grads[i], 1, a->numel[i], a->numel[i], sz);
        const Span o = span_of(a->out[i], 1, a->numel[i], a->numel[i], sz);
        if (g.lo != o.lo && overlap(g, o)) return true;
        r.push_back({o, true});
        if (g.lo != o.lo) r.push_back({g, false});
    }
    std::sort(r.begin(), r.end(), [](const Range& x, const Range& y) { return x.s.lo < y.s.lo; });
    // sweep by start: an overlap with a written range shows against the furthest end so far
    uintptr_t end_any = 0, end_written = 0;
    for (const Range& x : r) {
        if (x.s.lo < end_written || (x.written && x.s.lo < end_any)) return true;
        end_any = std::max(end_any, x.s.hi);
        if (x.written) end_written = std::max(end_written, x.s.hi);
    }
    return false;
}

// Few enough gradients for one launch by one cluster.
bool few(const vlproj_clip_grads_args* a) {
    if (a->n > VLPROJ_CLIP_FEW_TENSORS) return false;
    int64_t total = 0;
    for (int32_t i = 0; i < a->n; ++i) total += a->numel[i];
    return total <= VLPROJ_CLIP_FEW_ELEMENTS;
}

template <int kMax>
int run(const vlproj_clip_grads_args* a, cudaStream_t s) {
    const int sms = sm_count();
    if (sms == 0) return VLPROJ_ERR_CUDA;
    double* part = static_cast<double*>(a->workspace);
    const int nt = std::max(1, (a->n + kMax - 1) / kMax);
    std::vector<ClipTable<kMax>> t(nt);
    std::vector<int> grid(nt);
    for (int q = 0; q < nt; ++q) {
        ClipTable<kMax>& T = t[q];
        T.n = 0;
        int64_t chunks = 0;
        for (int32_t i = q * kMax; i < std::min<int64_t>(a->n, int64_t(q + 1) * kMax); ++i) {
            if (a->numel[i] == 0) continue;
            T.grad[T.n] = a->grads[i];
            T.out[T.n] = a->out ? a->out[i] : nullptr;
            T.numel[T.n] = a->numel[i];
            T.type[T.n] = static_cast<uint8_t>(a->type[i]);
            T.first[T.n++] = static_cast<int32_t>(chunks);
            chunks += (a->numel[i] * type_size(a->type[i]) + CLIP_CHUNK - 1) / CLIP_CHUNK;
            if (chunks >= (int64_t(1) << 30)) return VLPROJ_ERR_INVALID_ARG;
        }
        T.first[T.n] = static_cast<int32_t>(chunks);
        grid[q] = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(chunks, std::min(CLIP_BLOCKS_PER_SM * sms, CLIP_MAX_BLOCKS))));
    }
    if constexpr (kMax == kFewTensors) if (few(a)) {
        vlp_clip_few_kernel<kMax><<<CLIP_CLUSTER, CLIP_THREADS, 0, s>>>(t[0], a->max_norm, a->norm, a->out != nullptr);
        return cudaGetLastError() == cudaSuccess ? VLPROJ_OK : VLPROJ_ERR_CUDA;
    }
    int nparts = 0;
    for (int q = 0; q < nt; ++q) {
        vlp_clip_norm_kernel<<<grid[q], CLIP_THREADS, 0, s>>>(t[q], part + nparts);
        nparts += grid[q];
    }
    // the first scaling launch starts behind the last norm launch, which itself started
    // when all earlier ones had ended
    for (int q = 0; q < (a->out ? nt : 1); ++q)
        launch_after(vlp_clip_scale_kernel<kMax>, a->out ? grid[q] : 1, CLIP_THREADS, 0, s, t[q], part, nparts, a->max_norm,
                     q == 0 ? a->norm : nullptr, a->out != nullptr);
    return cudaGetLastError() == cudaSuccess ? VLPROJ_OK : VLPROJ_ERR_CUDA;
}

}  // namespace

extern "C" {

int64_t vlproj_clip_grads_workspace(int32_t n) {
    if (n < 0 || n > kMaxTensors) return VLPROJ_ERR_INVALID_ARG;
    return int64_t(8) * CLIP_MAX_BLOCKS * tables(n);
}

int vlproj_clip_grads(const vlproj_clip_grads_args* a, void* stream) {
    if (!a || a->n < 0 || a->n > kMaxTensors || (a->n > 0 && (!a->grads || !a->numel || !a->type)))
        return VLPROJ_ERR_INVALID_ARG;
    if ((!a->out && !a->norm) || reinterpret_cast<uintptr_t>(a->norm) % 4) return VLPROJ_ERR_INVALID_ARG;
    if (a->out && !(a->max_norm >= 0. && std::isfinite(a->max_norm))) return VLPROJ_ERR_INVALID_ARG;
    for (int32_t i = 0; i < a->n; ++i) {
        if (a->numel[i] < 0 || a->numel[i] >= (int64_t(1) << 40) || !known_type(a->type[i])) return VLPROJ_ERR_INVALID_ARG;
        if (a->numel[i] == 0) continue;
        const uintptr_t mask = static_cast<uintptr_t>(type_size(a->type[i]) - 1);
        if (!a->grads[i] || (reinterpret_cast<uintptr_t>(a->grads[i]) & mask)) return VLPROJ_ERR_INVALID_ARG;
        if (a->out && (!a->out[i] || (reinterpret_cast<uintptr_t>(a->out[i]) & mask))) return VLPROJ_ERR_INVALID_ARG;
    }
    const int64_t need = few(a) ? 0 : vlproj_clip_grads_workspace(a->n);
    if (need > 0 && !workspace_ok(a->workspace, a->workspace_bytes, need)) return VLPROJ_ERR_INVALID_ARG;
    try {
        if (clash(a, need)) return VLPROJ_ERR_INVALID_ARG;
        return a->n <= kFewTensors ? run<kFewTensors>(a, static_cast<cudaStream_t>(stream))
                                   : run<kTable>(a, static_cast<cudaStream_t>(stream));
    } catch (const std::bad_alloc&) {
        return VLPROJ_ERR_CUDA;
    }
}

}  // extern "C"
