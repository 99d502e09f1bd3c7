// C ABI of the language-model operators (declared in
// include/sgemm_gb300_lm.h): argument checks, the choice of tile, operand
// copies into the workspace where TMA cannot read in place, tensor maps and
// launches.
#include <algorithm>
#include <cstring>
#include <mutex>

#include "../../include/sgemm_gb300_lm.h"
#include "context.h"
#include "lm_kernels.h"

namespace {

using sg::LmArgs;
using sg::LmKernel;

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxBytes = int64_t(1) << 40;

inline int64_t ceil_div(int64_t x, int64_t a) { return (x + a - 1) / a; }
inline int64_t round_up(int64_t x, int64_t a) { return ceil_div(x, a) * a; }
inline size_t align256(int64_t x) { return size_t(round_up(x, 256)); }
inline bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool type_ok(int t) { return t == SGEMM_TYPE_F32 || t == SGEMM_TYPE_F16 || t == SGEMM_TYPE_BF16; }
int type_size(int t) { return t == SGEMM_TYPE_F32 ? 4 : 2; }
int out_type(int t) {
    return t == SGEMM_TYPE_F32 ? sg::kOutF32 : t == SGEMM_TYPE_F16 ? sg::kOutF16 : sg::kOutBF16;
}

// A matrix (or a batch of them) as the caller holds it, and where the
// tensor maps find it: in place, or 16-bit copies / three bf16 planes in the
// workspace.
struct Operand {
    const void *ptr = nullptr;
    int64_t rows = 0, cols = 0, ld = 0, batch = 1, stride = 0;
    int type = 0;
    bool copy = false;
    int64_t ld_t = 0, stride_t = 0, plane_t = 0;   // elements of 16 bits
    size_t ws = 0;
    const void *ptr_t = nullptr;

    void plan() {
        copy = type == SGEMM_TYPE_F32 || !aligned(ptr, 16) || ld % 8 != 0 || (batch > 1 && stride % 8 != 0);
        if (copy) {
            ld_t = round_up(std::max<int64_t>(cols, 1), 8);
            stride_t = rows * ld_t;
            plane_t = stride_t * batch;
            ws = align256(plane_t * 2 * (type == SGEMM_TYPE_F32 ? 3 : 1));
        } else {
            ld_t = ld;
            stride_t = batch > 1 ? stride : rows * ld;
            plane_t = stride_t * batch;
        }
    }
    int planes() const { return type == SGEMM_TYPE_F32 ? 3 : 1; }
    // Copies into `at` (ws bytes) if need be.
    bool prepare(void *at, cudaStream_t s) {
        if (!copy) {
            ptr_t = ptr;
            return true;
        }
        ptr_t = at;
        const int64_t st = batch > 1 ? stride : 0;
        return (type == SGEMM_TYPE_F32
                    ? sg::lm_launch_split3(static_cast<const float *>(ptr), ld, st, at, ld_t, plane_t, rows, cols,
                                           batch, s)
                    : sg::lm_launch_pack16(ptr, ld, st, at, ld_t, rows, cols, batch, s)) == cudaSuccess;
    }
    // {cols, rows, batch * planes}, boxes of 64 x box_rows.
    bool map(CUtensorMap *m, int box_rows) const { return map_rows(m, box_rows, 0, rows); }
    bool map_rows(CUtensorMap *m, int box_rows, int64_t row0, int64_t n_rows) const {
        auto enc = sg::tensor_map_encoder();
        if (enc == nullptr) return false;
        const int64_t z = batch * planes();
        cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(n_rows), cuuint64_t(z)};
        cuuint64_t strides[2] = {cuuint64_t(ld_t) * 2, cuuint64_t(stride_t) * 2};
        cuuint32_t box[3] = {64, cuuint32_t(box_rows), 1};
        cuuint32_t one[3] = {1, 1, 1};
        const char *base = static_cast<const char *>(ptr_t) + row0 * ld_t * 2;
        return enc(m, type == SGEMM_TYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                   const_cast<char *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    }
};

sgemmStatus_t check_matrix(const void *p, int64_t rows, int64_t cols, int64_t ld, int type, bool used) {
    if (ld < std::max<int64_t>(1, cols)) return SGEMM_STATUS_INVALID_VALUE;
    if (!used) return SGEMM_STATUS_SUCCESS;
    if (p == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    if (!aligned(p, type_size(type))) return SGEMM_STATUS_MISALIGNED;
    if (rows > kMaxDim || cols > kMaxDim || ld > kMaxBytes / 4 || rows > kMaxBytes / 4 / ld)
        return SGEMM_STATUS_NOT_SUPPORTED;
    return SGEMM_STATUS_SUCCESS;
}

sgemmStatus_t check_device(const sgemmContext *h) {
    int cur = -1;
    if (cudaGetDevice(&cur) != cudaSuccess) return SGEMM_STATUS_LAUNCH_FAILED;
    return cur == h->device ? SGEMM_STATUS_SUCCESS : SGEMM_STATUS_INVALID_VALUE;
}

// CTAs (or SM pairs) of a kernel that are resident at once on the device,
// asked for once per kernel and device after its shared-memory opt-in.
int resident_slots(const sgemmContext *h, const LmKernel &k, int smem) {
    struct Known { const void *fn; int device, slots; };
    static Known known[64];
    static int count = 0;
    static std::mutex mutex;
    std::lock_guard<std::mutex> lock(mutex);
    for (int i = 0; i < count; ++i)
        if (known[i].fn == k.fn && known[i].device == h->device) return known[i].slots;
    if (cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return -1;
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
    if (count < 64) known[count++] = Known{k.fn, h->device, n};
    return n;
}

// Shared memory of a launch: kernels with groups get room for the largest
// table (the opt-in is made once per kernel).
int smem_of(const LmKernel &k, bool groups) { return k.smem + (groups ? 8 * (sg::kLmMaxGroups + 2) : 0); }

sgemmStatus_t launch_lm(sgemmContext *h, const LmKernel &k, bool groups, const CUtensorMap &a, const CUtensorMap &b,
                        LmArgs &args, int64_t tiles, cudaStream_t stream) {
    const int smem = smem_of(k, groups);
    const int slots = resident_slots(h, k, smem);
    if (slots < 1) return SGEMM_STATUS_LAUNCH_FAILED;
    args.err = h->d_err;
    args.timeout_ns = h->timeout_ns;
    args.withhold = h->withhold;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(std::min<int64_t>(std::max<int64_t>(tiles, 1), slots) * (k.pair ? 2 : 1)));
    cfg.blockDim = dim3(k.threads);
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = k.pair ? 2 : 1;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = k.pair ? 2 : 1;
    void *kargs[] = {const_cast<CUtensorMap *>(&a), const_cast<CUtensorMap *>(&b), &args};
    return cudaLaunchKernelExC(&cfg, k.fn, kargs) == cudaSuccess ? SGEMM_STATUS_SUCCESS
                                                                 : SGEMM_STATUS_LAUNCH_FAILED;
}

// Rows of the output that take vector stores: 16 bytes per lane (columns of
// D as rows), 32 bytes (rows of D).
int vec_ok(const void *p, int64_t ld, int64_t stride, int elem, int bytes) {
    return aligned(p, bytes) && ld * elem % bytes == 0 && stride * elem % bytes == 0;
}

// ------------------------------------------------------------ grouped

struct Grouped {
    int type = 0, op = 0;
    int64_t T = 0, N = 0, K = 0, G = 0;
    Operand a, b;
};

sgemmStatus_t plan_grouped(int type, int op, int64_t T, int64_t N, int64_t K, int64_t G, const void *A, int64_t lda,
                           const void *B, int64_t ldb, int64_t strideB, Grouped &q) {
    if (!type_ok(type) || (op != SGEMM_OP_N && op != SGEMM_OP_T)) return SGEMM_STATUS_INVALID_VALUE;
    if (T < 0 || N < 0 || K < 0 || G < 0 || strideB < 0) return SGEMM_STATUS_INVALID_VALUE;
    if (T > kMaxDim - 512 || N > kMaxDim - 512 || K > kMaxDim - 512 || G > SGEMM_MAX_GROUPS)
        return SGEMM_STATUS_NOT_SUPPORTED;
    const bool used = T > 0 && N > 0 && K > 0 && G > 0;
    const int64_t br = op ? N : K, bc = op ? K : N;
    sgemmStatus_t st = check_matrix(A, T, K, lda, type, used);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    st = check_matrix(B, br, bc, ldb, type, used);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    if (used && G > 1) {
        if (strideB < (br - 1) * ldb + bc) return SGEMM_STATUS_INVALID_VALUE;
        if (strideB > kMaxBytes / 4 / G) return SGEMM_STATUS_NOT_SUPPORTED;
    }
    q.type = type;
    q.op = op;
    q.T = T; q.N = N; q.K = K; q.G = G;
    q.a.ptr = A; q.a.rows = T; q.a.cols = K; q.a.ld = lda; q.a.type = type;
    q.b.ptr = B; q.b.rows = br; q.b.cols = bc; q.b.ld = ldb; q.b.type = type;
    q.b.batch = G; q.b.stride = strideB;
    if (used) {
        q.a.plan();
        q.b.plan();
    }
    return SGEMM_STATUS_SUCCESS;
}

struct WeightGrad {
    int type = 0;
    int64_t T = 0, M = 0, N = 0, G = 0;
    Operand a, b;
};

sgemmStatus_t plan_weight_grad(int type, int64_t T, int64_t M, int64_t N, int64_t G, const void *A, int64_t lda,
                               const void *B, int64_t ldb, WeightGrad &q) {
    if (!type_ok(type)) return SGEMM_STATUS_INVALID_VALUE;
    if (T < 0 || M < 0 || N < 0 || G < 0) return SGEMM_STATUS_INVALID_VALUE;
    if (T > kMaxDim - 512 || M > kMaxDim - 512 || N > kMaxDim - 512 || G > SGEMM_MAX_GROUPS)
        return SGEMM_STATUS_NOT_SUPPORTED;
    const bool used = T > 0 && M > 0 && N > 0 && G > 0;
    sgemmStatus_t st = check_matrix(A, T, M, lda, type, used);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    st = check_matrix(B, T, N, ldb, type, used);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    q.type = type;
    q.T = T; q.M = M; q.N = N; q.G = G;
    q.a.ptr = A; q.a.rows = T; q.a.cols = M; q.a.ld = lda; q.a.type = type;
    q.b.ptr = B; q.b.rows = T; q.b.cols = N; q.b.ld = ldb; q.b.type = type;
    if (used) {
        q.a.plan();
        q.b.plan();
    }
    return SGEMM_STATUS_SUCCESS;
}

}  // namespace

extern "C" {

sgemmStatus_t sgemmGroupedWorkspaceSize(sgemmHandle_t h, sgemmDataType_t type, sgemmOperation_t opB, int64_t T,
                                        int64_t N, int64_t K, int64_t G, const void *A, int64_t lda, const void *B,
                                        int64_t ldb, int64_t strideB, size_t *bytes) {
    if (bytes == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    *bytes = 0;
    Grouped q;
    sgemmStatus_t st = plan_grouped(type, opB, T, N, K, G, A, lda, B, ldb, strideB, q);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    if (h == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    *bytes = q.a.ws + q.b.ws;
    return SGEMM_STATUS_SUCCESS;
}

sgemmStatus_t sgemmGrouped(sgemmHandle_t h, sgemmDataType_t type, sgemmOperation_t opB, int64_t T, int64_t N,
                           int64_t K, int64_t G, const void *A, int64_t lda, const void *B, int64_t ldb,
                           int64_t strideB, const int32_t *groupEnds, void *C, int64_t ldc, cudaStream_t stream) {
    Grouped q;
    sgemmStatus_t st = plan_grouped(type, opB, T, N, K, G, A, lda, B, ldb, strideB, q);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    st = check_matrix(C, T, N, ldc, type, T > 0 && N > 0);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    if (G > 0 && T > 0 && N > 0) {
        if (groupEnds == nullptr) return SGEMM_STATUS_INVALID_VALUE;
        if (!aligned(groupEnds, 4)) return SGEMM_STATUS_MISALIGNED;
    }
    if (T == 0 || N == 0) return SGEMM_STATUS_SUCCESS;
    if (h == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    st = check_device(h);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    const int elem = type_size(type);
    if (K == 0 || G == 0)
        return sg::lm_launch_zero(C, ldc, 0, elem, T, N, 1, stream) == cudaSuccess ? SGEMM_STATUS_SUCCESS
                                                                                   : SGEMM_STATUS_LAUNCH_FAILED;
    if (q.a.ws + q.b.ws > 0 && (h->ws == nullptr || h->ws_bytes < q.a.ws + q.b.ws))
        return SGEMM_STATUS_WORKSPACE_REQUIRED;

    const int64_t mean = T / G;
    const int size = mean <= 24 ? 0 : mean <= 128 ? 1 : 2;
    const LmKernel k = sg::lm_grouped_kernel(size, opB == SGEMM_OP_N, type == SGEMM_TYPE_F32);
    LmArgs p{};
    p.M = int(N);
    p.T = int(T);
    p.kb = int(ceil_div(K, 64));
    p.G = int(G);
    p.ends = groupEnds;
    p.tiles_m = int(ceil_div(N, k.tile_m));
    p.tile_n = k.bn;
    p.group_m = 8;
    p.splits = 1;
    p.pairs = type == SGEMM_TYPE_F32 ? 6 : 1;
    p.bf16 = type == SGEMM_TYPE_F16 ? 0 : 1;
    p.C = C;
    p.ldc = ldc;
    p.out = out_type(type);
    p.vec = vec_ok(C, ldc, 0, elem, 16);
    const int64_t tiles = int64_t(p.tiles_m) * (ceil_div(T, k.bn) + G + 1);
    if (tiles > kMaxDim) return SGEMM_STATUS_NOT_SUPPORTED;
    char *ws = static_cast<char *>(h->ws);
    if (!q.a.prepare(ws, stream) || !q.b.prepare(ws + q.a.ws, stream)) return SGEMM_STATUS_LAUNCH_FAILED;
    CUtensorMap tm_w, tm_x;
    if (!q.b.map(&tm_w, k.a_mn ? 64 : k.box_a) || !q.a.map(&tm_x, k.box_b)) return SGEMM_STATUS_LAUNCH_FAILED;
    return launch_lm(h, k, true, tm_w, tm_x, p, tiles, stream);
}

sgemmStatus_t sgemmGroupedWeightGradWorkspaceSize(sgemmHandle_t h, sgemmDataType_t type, int64_t T, int64_t M,
                                                  int64_t N, int64_t G, const void *A, int64_t lda, const void *B,
                                                  int64_t ldb, size_t *bytes) {
    if (bytes == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    *bytes = 0;
    WeightGrad q;
    sgemmStatus_t st = plan_weight_grad(type, T, M, N, G, A, lda, B, ldb, q);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    if (h == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    *bytes = q.a.ws + q.b.ws;
    return SGEMM_STATUS_SUCCESS;
}

sgemmStatus_t sgemmGroupedWeightGrad(sgemmHandle_t h, sgemmDataType_t type, int64_t T, int64_t M, int64_t N,
                                     int64_t G, const void *A, int64_t lda, const void *B, int64_t ldb,
                                     const int32_t *groupEnds, void *C, int64_t ldc, int64_t strideC,
                                     cudaStream_t stream) {
    WeightGrad q;
    sgemmStatus_t st = plan_weight_grad(type, T, M, N, G, A, lda, B, ldb, q);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    const bool any = M > 0 && N > 0 && G > 0;
    st = check_matrix(C, M, N, ldc, type, any);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    if (strideC < 0) return SGEMM_STATUS_INVALID_VALUE;
    if (!any) return SGEMM_STATUS_SUCCESS;
    if (G > 1) {
        if (strideC < (M - 1) * ldc + N) return SGEMM_STATUS_INVALID_VALUE;
        if (strideC > kMaxBytes / 4 / G) return SGEMM_STATUS_NOT_SUPPORTED;
    }
    if (T > 0) {
        if (groupEnds == nullptr) return SGEMM_STATUS_INVALID_VALUE;
        if (!aligned(groupEnds, 4)) return SGEMM_STATUS_MISALIGNED;
    }
    if (h == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    st = check_device(h);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    const int elem = type_size(type);
    const int64_t sc = G > 1 ? strideC : 0;
    if (T == 0)
        return sg::lm_launch_zero(C, ldc, sc, elem, M, N, G, stream) == cudaSuccess ? SGEMM_STATUS_SUCCESS
                                                                                    : SGEMM_STATUS_LAUNCH_FAILED;
    if (q.a.ws + q.b.ws > 0 && (h->ws == nullptr || h->ws_bytes < q.a.ws + q.b.ws))
        return SGEMM_STATUS_WORKSPACE_REQUIRED;

    const int size = M > 128 && N > 128 ? 2 : 1;
    const LmKernel k = sg::lm_weight_grad_kernel(size, type == SGEMM_TYPE_F32);
    LmArgs p{};
    p.M = int(M);
    p.N = int(N);
    p.T = int(T);
    p.G = int(G);
    p.ends = groupEnds;
    p.tiles_m = int(ceil_div(M, k.tile_m));
    p.tile_n = k.bn;
    p.tiles_n = int(ceil_div(N, k.bn));
    const int64_t tiles = int64_t(p.tiles_m) * p.tiles_n * G;
    if (tiles > kMaxDim) return SGEMM_STATUS_NOT_SUPPORTED;
    p.num_tiles = int(tiles);
    p.group_m = 8;
    p.splits = 1;
    p.pairs = type == SGEMM_TYPE_F32 ? 6 : 1;
    p.bf16 = type == SGEMM_TYPE_F16 ? 0 : 1;
    p.C = C;
    p.ldc = ldc;
    p.stride_c = sc;
    p.out = out_type(type);
    p.vec = vec_ok(C, ldc, sc, elem, 32);
    char *ws = static_cast<char *>(h->ws);
    if (!q.a.prepare(ws, stream) || !q.b.prepare(ws + q.a.ws, stream)) return SGEMM_STATUS_LAUNCH_FAILED;
    CUtensorMap tm_a, tm_b;
    if (!q.a.map(&tm_a, 64) || !q.b.map(&tm_b, 64)) return SGEMM_STATUS_LAUNCH_FAILED;
    return launch_lm(h, k, true, tm_a, tm_b, p, tiles, stream);
}

}  // extern "C"
