// What the C ABI of the language-model operators shares: argument checks, how
// many CTAs of a kernel are resident at once.
#pragma once

#include <algorithm>
#include <map>
#include <mutex>
#include <new>
#include <tuple>

#include "../../include/sgemm_gb300_lm.h"
#include "context.h"
#include "lm_kernels.h"

namespace sg::host {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxBytes = int64_t(1) << 40;
constexpr int kMaxSmem = 227 * 1024;    // dynamic shared memory per CTA

inline int64_t ceil_div(int64_t x, int64_t a) { return (x + a - 1) / a; }
inline int64_t round_up(int64_t x, int64_t a) { return ceil_div(x, a) * a; }
inline size_t align256(int64_t x) { return size_t(round_up(x, 256)); }
inline bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

inline bool type_ok(int t) { return t == SGEMM_TYPE_F32 || t == SGEMM_TYPE_F16 || t == SGEMM_TYPE_BF16; }
inline int type_size(int t) { return t == SGEMM_TYPE_F32 ? 4 : 2; }
inline int out_type(int t) {
    return t == SGEMM_TYPE_F32 ? sg::kOutF32 : t == SGEMM_TYPE_F16 ? sg::kOutF16 : sg::kOutBF16;
}

inline sgemmStatus_t check_matrix(const void *p, int64_t rows, int64_t cols, int64_t ld, int type, bool used) {
    if (ld < std::max<int64_t>(1, cols)) return SGEMM_STATUS_INVALID_VALUE;
    if (!used) return SGEMM_STATUS_SUCCESS;
    if (p == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    if (!aligned(p, type_size(type))) return SGEMM_STATUS_MISALIGNED;
    if (rows > kMaxDim || cols > kMaxDim || ld > kMaxBytes / 4 || rows > kMaxBytes / 4 / ld)
        return SGEMM_STATUS_NOT_SUPPORTED;
    return SGEMM_STATUS_SUCCESS;
}

inline sgemmStatus_t check_device(const sgemmContext *h) {
    int cur = -1;
    if (cudaGetDevice(&cur) != cudaSuccess) return SGEMM_STATUS_LAUNCH_FAILED;
    return cur == h->device ? SGEMM_STATUS_SUCCESS : SGEMM_STATUS_INVALID_VALUE;
}

// CTAs (or SM pairs) of a kernel that are resident at once on the device,
// asked for once per kernel, device and size (to the next KB) after its
// shared-memory opt-in.  The 4-bit products' size follows x, so that a server's
// batches make many.
inline int resident_slots(const sgemmContext *h, const LmKernel &k, int exact_smem) {
    using Key = std::tuple<const void *, int, int, int>;
    static std::map<Key, int> known;
    static std::mutex mutex;
    const int smem = std::min(int(round_up(exact_smem, 1024)), kMaxSmem);
    const Key key(k.fn, h->device, smem, k.threads);
    std::lock_guard<std::mutex> lock(mutex);
    const auto at = known.find(key);
    if (at != known.end()) return at->second;
    // The opt-in is for the most any launch may ask for, so that one launch
    // never lowers it under another.
    if (cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) != cudaSuccess) return -1;
    int n = 0;
    if (k.pair) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(2 * h->sm_count);
        cfg.blockDim = dim3(k.threads);
        cfg.dynamicSmemBytes = size_t(smem);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, k.fn, &cfg) != cudaSuccess) return -1;
    } else {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k.fn, k.threads, smem) != cudaSuccess) return -1;
        n *= h->sm_count;
    }
    if (n < 1) return -1;
    try {
        known.emplace(key, n);
    } catch (const std::bad_alloc &) {       // (asked for again next time)
    }
    return n;
}

inline sgemmStatus_t check_vector(const void *p, int align) {
    if (p == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    return aligned(p, align) ? SGEMM_STATUS_SUCCESS : SGEMM_STATUS_MISALIGNED;
}

// Rows of the output that take vector stores: 16 bytes per lane (columns of
// D as rows), 32 bytes (rows of D).
inline int vec_ok(const void *p, int64_t ld, int64_t stride, int elem, int bytes) {
    return aligned(p, bytes) && ld * elem % bytes == 0 && stride * elem % bytes == 0;
}

}  // namespace sg::host
