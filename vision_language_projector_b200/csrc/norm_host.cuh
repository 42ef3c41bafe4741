// Host-side pieces of the layer norm entry points: argument checks, how rows are cut and
// held, resident blocks.
#pragma once
#include "kernels_norm.cuh"

#include <algorithm>
#include <mutex>

namespace vlp_ops {

constexpr int64_t kMaxRows = int64_t(1) << 31;

inline bool vec_ok(const float* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }
inline bool shape_ok(int64_t rows, int64_t C, int x_type, int y_type) {
    return rows >= 0 && rows < kMaxRows && C >= 1 && C <= VLPROJ_MAX_WIDTH && known_pair(x_type, y_type);
}

// Most row blocks of the weight gradients' partial sums, a multiple of 8: one for 8 rows, or
// one a row while there are fewer rows than SMs.
inline int part_blocks(int64_t rows, int64_t C) {
    const int64_t want = std::max((rows + 7) / 8, std::min<int64_t>(rows, 148));
    return static_cast<int>(std::min<int64_t>(ln_max_parts(C), std::max<int64_t>(8, (want + 7) / 8 * 8)));
}

// How the matrices' rows can be cut into aligned vectors of 8 elements: all rows aligned and
// C % 8 == 0; or all matrices' rows equally far from an aligned vector; or neither.
enum { kAligned, kShifted, kAny };
struct Rows {
    const void* p;
    int64_t ld;
    int type;
    int64_t start() const { return static_cast<int64_t>(reinterpret_cast<uintptr_t>(p) / type_size(type) % 8); }
};
inline int cut_of(const Rows* m, int n, int64_t C, bool weights_aligned) {
    bool aligned = C % 8 == 0 && weights_aligned, equal = true;
    for (int i = 0; i < n; ++i) {
        aligned = aligned && rows_wide(m[i].p, m[i].ld, m[i].type);
        equal = equal && m[i].start() == m[0].start() && (m[i].ld - m[0].ld) % 8 == 0;
    }
    return aligned ? kAligned : equal ? kShifted : kAny;
}

// Blocks for `rows` rows, `groups` of them a block at a time, at most `most` blocks: for
// shifted rows a multiple of 8.
inline int64_t row_blocks(int cut, int64_t rows, int64_t groups, int64_t most) {
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
// with up to kMaxWarpVec vectors each, or a whole block with up to kMaxBlockVec; f may
// refuse a way (the next one is tried). False when no way fits.
template <int kMaxWarpVec, int kMaxBlockVec, class F>
bool with_shape(int nvec, F&& f) {
    if (nvec <= 8) return f(Shape<4, 2>(), 0);
    if (nvec <= 16) return f(Shape<8, 2>(), 0);
    if (nvec <= 32) return f(Shape<16, 2>(), 0);
    if (nvec <= 64) return f(Shape<16, 4>(), 0);
    if (nvec <= 96) return f(Shape<32, 3>(), 0);
    if (nvec <= 128) return f(Shape<32, 4>(), 0);
    if (nvec <= 160) return f(Shape<32, 5>(), 0);
    if constexpr (kMaxWarpVec > 5) {
        if (nvec <= 256 && f(Shape<32, 8>(), 0)) return true;
        if (nvec <= 320 && f(Shape<32, 10>(), 0)) return true;
        if (nvec <= 512 && f(Shape<32, 16>(), 0)) return true;
        if (nvec <= 640 && f(Shape<32, 20>(), 0)) return true;
    }
    const auto threads = [&](int vec) { return (nvec + 32 * vec - 1) / (32 * vec) * 32; };
    if (nvec <= 1024) return f(Shape<0, 2, 512>(), threads(2));              // 128 registers a thread
    if constexpr (kMaxBlockVec == 2) {
        return nvec <= 2 * LN_MAX_THREADS && f(Shape<0, 2>(), threads(2));
    } else {
        if (nvec <= 4 * 512) return f(Shape<0, 4>(), threads(4));
        return nvec <= kMaxBlockVec * LN_MAX_THREADS && f(Shape<0, kMaxBlockVec>(), threads(kMaxBlockVec));
    }
}

}  // namespace vlp_ops
