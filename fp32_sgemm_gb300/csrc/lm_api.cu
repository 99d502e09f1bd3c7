// C ABI of the language-model operators (declared in
// include/sgemm_gb300_lm.h): argument checks, the choice of tile, operand
// copies into the workspace where TMA cannot read in place, tensor maps and
// launches.
#include <algorithm>
#include <cstring>
#include <map>
#include <mutex>
#include <new>
#include <tuple>

#include "../../include/sgemm_gb300_lm.h"
#include "context.h"
#include "lm_kernels.h"
#include "lm_w4.h"

namespace {

using sg::LmArgs;
using sg::LmKernel;

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxBytes = int64_t(1) << 40;
constexpr int kMaxSmem = 227 * 1024;    // dynamic shared memory per CTA

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

    // always: copied even where TMA could read in place.
    void plan(bool always = false) {
        copy = always || type == SGEMM_TYPE_F32 || !aligned(ptr, 16) || ld % 8 != 0 || (batch > 1 && stride % 8 != 0);
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
    // The copy into `at` (ws bytes), if there is one.
    sg::LmCopy place(void *at, sg::LmCopyFilter keep = {}) {
        sg::LmCopy j;
        ptr_t = copy ? at : ptr;
        if (copy) {
            j.src = ptr;
            j.ld = ld;
            j.stride = batch > 1 ? stride : 0;
            j.dst = at;
            j.ld_dst = ld_t;
            j.plane = plane_t;
            j.rows = rows;
            j.cols = cols;
            j.batch = batch;
            j.keep = keep;
        }
        return j;
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

// The copies of two operands (and the scale of a gradient) in one launch, if
// there is anything to do.
bool copy_operands(int type, const sg::LmCopy &a, const sg::LmCopy &b, cudaStream_t s,
                   const sg::LmGradScale &scale = {}) {
    if (a.src == nullptr && b.src == nullptr && scale.scale2 == nullptr) return true;
    return sg::lm_launch_copy(type == SGEMM_TYPE_F32, a, b, scale, s) == cudaSuccess;
}

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
// asked for once per kernel, device and size (to the next KB) after its
// shared-memory opt-in.  The 4-bit products' size follows x, so that a server's
// batches make many.
int resident_slots(const sgemmContext *h, const LmKernel &k, int exact_smem) {
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

// Shared memory of a launch: kernels with groups get room for the largest
// table (the opt-in is made once per kernel).
int smem_of(const LmKernel &k, bool groups) { return k.smem + (groups ? 8 * (sg::kLmMaxGroups + 2) : 0); }

sgemmStatus_t launch_lm(sgemmContext *h, const LmKernel &k, bool groups, const CUtensorMap *a, const CUtensorMap *b,
                        LmArgs &args, int64_t tiles, cudaStream_t stream, sg::LmRows *rows = nullptr) {
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
    void *kargs[] = {const_cast<CUtensorMap *>(a), const_cast<CUtensorMap *>(b), &args}, *rargs[] = {&args, rows};
    return cudaLaunchKernelExC(&cfg, k.fn, rows != nullptr ? rargs : kargs) == cudaSuccess ? SGEMM_STATUS_SUCCESS
                                                                 : SGEMM_STATUS_LAUNCH_FAILED;
}

// Rows of the output that take vector stores: 16 bytes per lane (columns of
// D as rows), 32 bytes (rows of D).
int vec_ok(const void *p, int64_t ld, int64_t stride, int elem, int bytes) {
    return aligned(p, bytes) && ld * elem % bytes == 0 && stride * elem % bytes == 0;
}

// ------------------------------------------------------------ grouped

// Tiles of a grouped product: size as in lm_kernels.h, rows of a group in one
// tile.  The groups' sizes are on the device; half a tile of each group is
// taken to be left over.  Measured, us, with tiles of 128 columns by 32 / 64 /
// 128 rows and 256 columns by 64 / 256 rows:
//   the smallest tiles with which every SM has at most one: 8 groups of 200
//     rows, 512 x 512: 9.0 / 6.9 / 7.6 / 7.6 / 9.6; 4 of 128, 1024 x 1024:
//     8.3 / 9.0 / 9.6 / 9.0 / 10.3;
//   otherwise those of a pair, whose W is read in the fewest and longest
//     pieces: 64 groups of 64, 1408 x 2048: 110 / 73 / 63 / 69 / 61; 8 of 32,
//     4096 x 14336: 159 / 132 / 121 / 128 / 116;
//   with fewer than two for each pair, of as many rows as a group has in the
//     mean, so that the largest groups are cut: 16 of 64, 2048 x 1408 stored
//     1408 x 2048: 31 / 25 / 27 / 24 / 26;
//   and no more rows than there are (8 rows, 8 groups, 4096 x 14336, 256
//     columns by 32 / 256 rows: 96 / 137).
// FP32, whose six products weigh more than reading W, 32 / 128 / 256 rows:
// thin tiles also for few rows in a group (16 of 16, 2048 x 1408: 147 / 150 /
// 174), those of one SM up to 256 rows (16 of 192, 2048 x 1408: 291 / 202
// / 222; of 512: 659 / 307 / 304) and where the pairs' leave SMs idle (2 groups
// of 632, 1024 x 1408: 57 / 34 / 45).
struct Tiling {
    int size, tile_n;
};

Tiling grouped_tiling(int type, int64_t T, int64_t N, int64_t G, int sms) {
    const int64_t mean = T / G, touched = std::min(G, T);
    auto tiles = [&](int64_t height, int64_t rows) { return ceil_div(N, height) * (2 * T / rows + touched) / 2; };
    if (tiles(128, 32) <= sms) return {0, 32};
    if (type == SGEMM_TYPE_F32) {
        if (mean <= 24) return {0, 32};
        return mean <= 256 || tiles(256, 256) < sms / 2 ? Tiling{1, 128} : Tiling{2, 256};
    }
    if (tiles(128, 64) <= sms) return {1, 64};
    if (tiles(128, 128) <= sms) return {1, 128};
    int rows = 256;
    if (ceil_div(N, 256) * G < sms) rows = mean <= 64 ? 64 : mean <= 128 ? 128 : 256;
    return {2, int(std::min<int64_t>(rows, round_up(T, 32)))};
}

// Parts the contraction is cut into where the tiles of a few rows leave most
// SMs without one, each longer than the ring of stages (FP32 takes three a
// block); a launch of its own joins them.  2 rows in 2 of 8 groups, 4096 x 2048:
// 20.3 -> 11.1 us; 128 rows in 2 groups, 4096 x 1024: 19.9 -> 12.4, FP32 75.5 ->
// 39.8; 64 rows in one, 2048 x 2048: 12.4 -> 11.0, FP32 41.0 -> 24.0.
int64_t grouped_parts(int type, int64_t K) { return ceil_div(K, 64) / (type == SGEMM_TYPE_F32 ? 4 : 12); }
int grouped_splits(int type, const Tiling &t, int64_t T, int64_t N, int64_t K, int64_t G, int sms) {
    if (t.size == 2) return 1;
    const int64_t most = ceil_div(N, 128) * (T / t.tile_n + std::min(G, T));
    return int(std::max<int64_t>(1, std::min(sms / std::max<int64_t>(1, most), grouped_parts(type, K))));
}

// Few FP32 rows a group: W as it is, on the FP32 pipes (lm_rows32.cu has both
// sides), unless the contraction is too short for a CTA's warps.  The mean
// decides, the sizes being on the device; skewed ones lose nothing by it (64
// groups of 2048 x 1408, 8 rows in the mean: even 294 us, spread by e^1.5 287, of 9
// rows on the tensor cores 472 and 414), only all rows in one group do (158
// against 130; 256 groups of 1024 x 1024: 251 and 161).
bool few_rows32(int type, int64_t T, int64_t K, int64_t G) {
    return type == SGEMM_TYPE_F32 && T / G <= 8 && K >= 256;
}

struct Grouped {
    int type = 0, op = 0;
    int64_t T = 0, N = 0, K = 0, G = 0;
    Operand a, b;
    bool rows32 = false;         // read as they are, on the FP32 pipes
    // The rest of the plan, on a device of `sms` SMs.
    Tiling tiling{};
    int splits = 1;
    int64_t ld_part = 0;
    size_t ws_part = 0;
    void tile(int sms) {
        if (T == 0 || N == 0 || K == 0 || G == 0 || rows32) return;
        tiling = grouped_tiling(type, T, N, G, sms);
        splits = grouped_splits(type, tiling, T, N, K, G, sms);
        ld_part = round_up(N, 8);
        ws_part = splits > 1 ? align256(splits * T * ld_part * 4) : 0;
    }
    size_t bytes() const { return a.ws + b.ws + ws_part; }
    LmKernel kernel() const {
        return sg::lm_grouped_kernel(tiling.size, op == SGEMM_OP_N, type == SGEMM_TYPE_F32,
                                     K > splits * sg::kLmPlainTerms);
    }
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
    q.rows32 = used && few_rows32(type, T, K, G);
    if (used && !q.rows32) {
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

// Pairs' tiles unless most pairs would have none (8 groups of 512 rows, BF16, 128
// x 128 / 256 x 256: 512 x 512 7.7 / 9.6 us, 768 x 768 10.3 / 10.3, 1024 x 1024
// 15.8 / 14.1).  Sums in runs where a group may be long: one may have all rows.
LmKernel weight_grad_kernel(const WeightGrad &q, int sms) {
    const bool fills = 3 * ceil_div(q.M, 256) * ceil_div(q.N, 256) * q.G >= sms;
    return sg::lm_weight_grad_kernel(q.M > 128 && q.N > 128 && fills ? 2 : 1, q.type == SGEMM_TYPE_F32,
                                     q.T > sg::kLmPlainTerms);
}

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

// ---------------------------------------------------- vocabulary loss

// Bytes of one piece of the logits' gradient: the piece is as many
// vocabulary columns as fit, so that the gradient products are long (pieces
// of 128 / 256 / 512 MB, both gradients: 8192 rows, 131072 x 4096 17.1 / 14.9 /
// 14.9 ms; 16384 rows, 50304 x 1024 5.1 / 3.5 / 3.4; 1024 MB gained nothing).
constexpr int64_t kPieceBytes = int64_t(512) << 20;
constexpr int64_t kMinPieceCols = 2048;

struct Loss {
    int type = 0;
    int64_t T = 0, V = 0, D = 0;
    Operand x, w;
    Operand x_kept;              // gradient: x, rows that take no part as zeros
    bool big = false;
    int bn = 0;                  // columns of a tile at most
    // Forward.
    int tile_n = 0, tiles_n = 0, slabs = 0;
    size_t ws_part = 0, ws_picked = 0;
    // Gradient.
    int64_t piece = 0, pieces = 0, ld_d = 0, ld_acc = 0;
    int d_planes = 1;
    int splits = 1;
    size_t ws_d = 0, ws_planes = 0, ws_acc = 0;
    size_t forward_bytes() const { return x.ws + w.ws + ws_part + ws_picked; }
    size_t grad_bytes() const { return x_kept.ws + w.ws + ws_d + ws_planes + ws_acc + 256; }
};

// Columns per tile of a rows x cols product on `slots` CTAs or pairs: the
// width with the least rounds x (width + what a tile costs beside it).
int balanced_tile_n(int64_t tiles_m, int64_t cols, int64_t slots, int gran, int least, int most) {
    int best = most;
    double best_cost = 0.0;
    for (int n = most; n >= least; n -= gran) {
        const double cost = double(ceil_div(tiles_m * ceil_div(cols, n), slots)) * (n + 8.0);
        if (n == most || cost < best_cost) { best_cost = cost; best = n; }
    }
    return best;
}

sgemmStatus_t plan_loss(int type, int64_t T, int64_t V, int64_t D, const void *X, int64_t ldx, const void *W,
                        int64_t ldw, const sgemmContext *h, Loss &q) {
    if (!type_ok(type) || T < 0 || V < 1 || D < 1) return SGEMM_STATUS_INVALID_VALUE;
    if (T > kMaxDim - 512 || V > kMaxDim - 512 || D > kMaxDim - 512) return SGEMM_STATUS_NOT_SUPPORTED;
    sgemmStatus_t st = check_matrix(X, T, D, ldx, type, T > 0);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    st = check_matrix(W, V, D, ldw, type, T > 0);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    // Tiles of the largest product, with the narrowest tiles.
    if (ceil_div(T, 128) > kMaxDim / ceil_div(V, 128) || ceil_div(V, 128) > kMaxDim / ceil_div(D, 128) ||
        ceil_div(T, 128) > kMaxDim / ceil_div(D, 128))
        return SGEMM_STATUS_NOT_SUPPORTED;
    q.type = type;
    q.T = T; q.V = V; q.D = D;
    q.x.ptr = X; q.x.rows = T; q.x.cols = D; q.x.ld = ldx; q.x.type = type;
    q.w.ptr = W; q.w.rows = V; q.w.cols = D; q.w.ld = ldw; q.w.type = type;
    if (T == 0 || h == nullptr) return SGEMM_STATUS_SUCCESS;
    q.x_kept = q.x;
    q.x.plan();
    q.x_kept.plan(true);
    q.w.plan();
    const bool f32 = type == SGEMM_TYPE_F32;
    // One tile of rows: those of one SM, whose W is read in stages of their own
    // (forward, 32000 x 1024: 128 rows 21.2 us, in pairs' tiles 25.4; 160 rows
    // 31.5 and 25.4).
    q.big = T > 128;
    const int64_t slots = q.big ? h->sm_count / 2 : h->sm_count;
    const int64_t tiles_m = ceil_div(T, q.big ? 256 : 128);
    q.bn = !q.big && f32 ? 128 : 256;
    q.tile_n = balanced_tile_n(tiles_m, V, slots, q.big ? 32 : 16, q.bn / 2, q.bn);
    q.tiles_n = int(ceil_div(V, q.tile_n));
    q.slabs = q.tiles_n * 2;             // an epilogue warp takes half a tile
    q.ws_part = align256(int64_t(q.slabs) * T * 8);
    q.ws_picked = align256(T * 4);
    // Gradient: pieces of the vocabulary, each a multiple of 256 columns.
    // 16 bits hold d with up to half a unit in the last place lost, and a few
    // rows do not average that out (of one row, the target's entry is most of
    // both gradients): up to 128 rows, whose products are bound by reading W
    // and writing its gradient, d is held in two planes, itself and the rest.
    q.d_planes = !f32 && !q.big ? 2 : 1;
    const int64_t elem = f32 ? 10 : 2 * q.d_planes;      // FP32: the piece itself and its three planes
    q.piece = V;
    if (T * V * elem > kPieceBytes) {
        q.piece = std::max<int64_t>(kMinPieceCols, kPieceBytes / (elem * T) / 256 * 256);
        q.piece = std::min(q.piece, V);
    }
    q.pieces = ceil_div(V, q.piece);
    q.piece = std::min(V, round_up(ceil_div(V, q.pieces), 256));
    q.pieces = ceil_div(V, q.piece);
    q.ld_d = round_up(q.piece, 16);
    q.ws_d = align256(T * q.ld_d * (f32 ? 4 : 2 * q.d_planes));
    q.ws_planes = f32 ? align256(T * q.ld_d * 6) : 0;
    // The rows' gradient: one piece, K split when its tiles are few (both
    // gradients of 1024 rows, 32000 x 1024: 172 us, unsplit 265; of 16 rows 97
    // and 396); more pieces, summed in FP32 from one to the next.
    q.ld_acc = round_up(D, 8);
    const int64_t dx_tiles = tiles_m * ceil_div(D, q.bn);
    if (q.pieces == 1) {
        q.splits = int(std::max<int64_t>(1, std::min(slots / dx_tiles, ceil_div(V, 64) / 8)));
        q.ws_acc = q.splits > 1 ? align256(q.splits * T * q.ld_acc * 4) : 0;
    } else {
        q.ws_acc = align256(T * q.ld_acc * 4);
    }
    return SGEMM_STATUS_SUCCESS;
}

sgemmStatus_t check_vector(const void *p, int align) {
    if (p == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    return aligned(p, align) ? SGEMM_STATUS_SUCCESS : SGEMM_STATUS_MISALIGNED;
}

LmArgs loss_args(const Loss &q, const LmKernel &k, int64_t M, int64_t N, int64_t K, int tile_n) {
    LmArgs p{};
    p.M = int(M);
    p.N = int(N);
    p.T = int(M);
    p.kb = p.kb_plane = int(ceil_div(K, 64));
    p.tile_n = tile_n;
    p.tiles_m = int(ceil_div(M, k.tile_m));
    p.tiles_n = int(ceil_div(N, tile_n));
    p.num_tiles = p.tiles_m * p.tiles_n;
    p.splits = 1;
    p.group_m = 8;
    p.bf16 = q.type == SGEMM_TYPE_F16 ? 0 : 1;
    return p;
}

// ------------------------------------------------------ 4-bit weights

struct W4 {
    int type = 0, planes = 1, group = 0;
    int64_t M = 0, N = 0, K = 0;
    int most = 0;                // rows of x per launch
    int slices = 1, k_slice = 0;
    size_t ws = 0;
};

int64_t w4_pitch(int64_t k) {
    // 64 modulo 128 bytes: eight lanes of neighbouring tokens meet no bank twice.
    return round_up(k * 2, 128) + 64;
}

int w4_blocks(int64_t cols) { return cols <= 8 ? 1 : cols <= 16 ? 2 : 4; }

sgemmStatus_t plan_w4(int type, int64_t M, int64_t N, int64_t K, int group, W4 &q) {
    if (!type_ok(type) || M < 0 || N < 0 || K < 0) return SGEMM_STATUS_INVALID_VALUE;
    if (group != 32 && group != 64 && group != 128) return SGEMM_STATUS_INVALID_VALUE;
    if (K % group != 0) return SGEMM_STATUS_INVALID_VALUE;
    // (Row numbers run past N by the rows of one round of CTAs.)
    if (M > kMaxDim - 512 || N > kMaxDim - (1 << 20) || K > kMaxDim - 512) return SGEMM_STATUS_NOT_SUPPORTED;
    q.type = type;
    q.planes = type == SGEMM_TYPE_F32 ? 3 : 1;
    q.group = group;
    q.M = M; q.N = N; q.K = K;
    q.most = int(std::min<int64_t>(M, type == SGEMM_TYPE_F32 ? 10 : 32));
    if (M == 0 || N == 0 || K == 0) return SGEMM_STATUS_SUCCESS;
    // K is cut when x does not fit beside the ring.
    const int64_t cols = int64_t(q.most) * q.planes;
    const int64_t room = kMaxSmem - int64_t(sg::w4_fixed_smem(w4_blocks(cols), true));
    int64_t slices = 1;
    while (cols * w4_pitch(round_up(ceil_div(K, slices), 256)) > room && ceil_div(K, slices) > 256) ++slices;
    q.k_slice = int(round_up(ceil_div(K, slices), 256));
    q.slices = int(ceil_div(K, q.k_slice));
    q.ws = q.slices > 1 ? align256(int64_t(q.slices) * q.most * round_up(N, 8) * 4) : 0;
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
    // (A short contraction is cut on no device.)
    if (grouped_parts(type, K) > 1) q.tile(h->sm_count);
    *bytes = q.bytes();
    return SGEMM_STATUS_SUCCESS;
}

sgemmStatus_t sgemmGroupedQueryPlan(sgemmHandle_t h, sgemmDataType_t type, sgemmOperation_t opB, int64_t T, int64_t N,
                                    int64_t K, int64_t G, const void *A, int64_t lda, const void *B, int64_t ldb,
                                    int64_t strideB, sgemmGroupedPlan_t *plan) {
    if (plan == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    *plan = sgemmGroupedPlan_t{};
    Grouped q;
    sgemmStatus_t st = plan_grouped(type, opB, T, N, K, G, A, lda, B, ldb, strideB, q);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    if (h == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    if (T == 0 || N == 0 || K == 0 || G == 0) return SGEMM_STATUS_SUCCESS;
    plan->splits = 1;
    if (q.rows32) {
        const LmKernel k = sg::lm_rows32_kernel_info(opB == SGEMM_OP_T, false);
        plan->kernel = 1;
        plan->tile_m = k.bn;
        plan->tile_n = k.tile_m;
        return SGEMM_STATUS_SUCCESS;
    }
    q.tile(h->sm_count);
    const LmKernel k = q.kernel();
    plan->kernel = k.pair ? 3 : 2;
    plan->tile_m = q.tiling.tile_n;     // (the rows are on the MMA's N side)
    plan->tile_n = k.tile_m;
    plan->splits = q.splits;
    plan->copies_a = q.a.copy;
    plan->copies_b = q.b.copy;
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
    if (q.rows32) {
        const bool few = ceil_div(N, 32) * std::min(G, T) < h->sm_count;
        const LmKernel k = sg::lm_rows32_kernel_info(opB == SGEMM_OP_T, few);
        LmArgs p{};
        p.M = int(N);
        p.T = int(T);
        p.G = int(G);
        p.ends = groupEnds;
        p.tile_n = k.bn;
        p.tiles_m = int(ceil_div(N, k.tile_m));
        p.C = C;
        p.ldc = ldc;
        sg::LmRows rows{};
        rows.X = static_cast<const float *>(A);
        rows.W = static_cast<const float *>(B);
        rows.ldx = lda;
        rows.ldw = ldb;
        rows.stride = G > 1 ? strideB : 0;
        rows.K = int(K);
        rows.x_vec = vec_ok(A, lda, 0, 4, 16);
        rows.w_vec = vec_ok(B, ldb, rows.stride, 4, 16);
        const int64_t tiles = int64_t(p.tiles_m) * (ceil_div(T, k.bn) + G + 1);
        if (tiles > kMaxDim) return SGEMM_STATUS_NOT_SUPPORTED;
        return launch_lm(h, k, true, nullptr, nullptr, p, tiles, stream, &rows);
    }
    q.tile(h->sm_count);
    if (q.bytes() > 0 && (h->ws == nullptr || h->ws_bytes < q.bytes())) return SGEMM_STATUS_WORKSPACE_REQUIRED;

    const LmKernel k = q.kernel();
    LmArgs p{};
    p.M = int(N);
    p.T = int(T);
    p.kb = int(ceil_div(K, 64));
    p.G = int(G);
    p.ends = groupEnds;
    p.tiles_m = int(ceil_div(N, k.tile_m));
    p.tile_n = q.tiling.tile_n;
    p.group_m = 8;
    p.splits = q.splits;
    p.bf16 = type == SGEMM_TYPE_F16 ? 0 : 1;
    char *ws = static_cast<char *>(h->ws);
    float *part = reinterpret_cast<float *>(ws + q.a.ws + q.b.ws);
    if (q.splits > 1) {
        p.C = part;
        p.ldc = q.ld_part;
        p.stride_c = T * q.ld_part;
        p.out = sg::kOutF32;
    } else {
        p.C = C;
        p.ldc = ldc;
        p.out = out_type(type);
        p.vec = vec_ok(C, ldc, 0, elem, 16);
    }
    const int64_t tiles = int64_t(p.tiles_m) * (ceil_div(T, p.tile_n) + G + 1) * q.splits;
    if (tiles > kMaxDim) return SGEMM_STATUS_NOT_SUPPORTED;
    sg::LmCopyFilter touched;           // matrices of groups that have rows
    touched.ends = groupEnds;
    if (!copy_operands(type, q.a.place(ws), q.b.place(ws + q.a.ws, touched), stream)) return SGEMM_STATUS_LAUNCH_FAILED;
    CUtensorMap tm_w, tm_x;
    if (!q.b.map(&tm_w, k.a_mn ? 64 : k.box_a) || !q.a.map(&tm_x, p.tile_n / (k.pair ? 2 : 1))) return SGEMM_STATUS_LAUNCH_FAILED;
    st = launch_lm(h, k, true, &tm_w, &tm_x, p, tiles, stream);
    if (st != SGEMM_STATUS_SUCCESS || q.splits == 1) return st;
    return sg::lm_launch_join_splits(part, q.ld_part, T * q.ld_part, q.splits, nullptr, int(T), int(N), C, ldc,
                                     out_type(type), stream) == cudaSuccess
               ? SGEMM_STATUS_SUCCESS : SGEMM_STATUS_LAUNCH_FAILED;
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

sgemmStatus_t sgemmGroupedWeightGradQueryPlan(sgemmHandle_t h, sgemmDataType_t type, int64_t T, int64_t M, int64_t N,
                                              int64_t G, const void *A, int64_t lda, const void *B, int64_t ldb,
                                              sgemmGroupedPlan_t *plan) {
    if (plan == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    *plan = sgemmGroupedPlan_t{};
    WeightGrad q;
    sgemmStatus_t st = plan_weight_grad(type, T, M, N, G, A, lda, B, ldb, q);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    if (h == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    if (T == 0 || M == 0 || N == 0 || G == 0) return SGEMM_STATUS_SUCCESS;
    const LmKernel k = weight_grad_kernel(q, h->sm_count);
    plan->kernel = k.pair ? 3 : 2;
    plan->tile_m = k.tile_m;
    plan->tile_n = k.bn;
    plan->splits = 1;
    plan->copies_a = q.a.copy;
    plan->copies_b = q.b.copy;
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

    const LmKernel k = weight_grad_kernel(q, h->sm_count);
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
    p.bf16 = type == SGEMM_TYPE_F16 ? 0 : 1;
    p.C = C;
    p.ldc = ldc;
    p.stride_c = sc;
    p.out = out_type(type);
    p.vec = vec_ok(C, ldc, sc, elem, 32);
    char *ws = static_cast<char *>(h->ws);
    if (!copy_operands(type, q.a.place(ws), q.b.place(ws + q.a.ws), stream)) return SGEMM_STATUS_LAUNCH_FAILED;
    CUtensorMap tm_a, tm_b;
    if (!q.a.map(&tm_a, 64) || !q.b.map(&tm_b, 64)) return SGEMM_STATUS_LAUNCH_FAILED;
    return launch_lm(h, k, true, &tm_a, &tm_b, p, tiles, stream);
}

sgemmStatus_t sgemmCrossEntropyWorkspaceSize(sgemmHandle_t h, sgemmDataType_t type, int64_t T, int64_t V, int64_t D,
                                             const void *X, int64_t ldx, const void *W, int64_t ldw,
                                             size_t *bytes) {
    if (bytes == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    *bytes = 0;
    Loss q;
    sgemmStatus_t st = plan_loss(type, T, V, D, X, ldx, W, ldw, h, q);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    if (h == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    *bytes = T > 0 ? q.forward_bytes() : 0;
    return SGEMM_STATUS_SUCCESS;
}

sgemmStatus_t sgemmCrossEntropy(sgemmHandle_t h, sgemmDataType_t type, int64_t T, int64_t V, int64_t D,
                                const void *X, int64_t ldx, const void *W, int64_t ldw, const int64_t *target,
                                float *loss, float *lse, cudaStream_t stream) {
    Loss q;
    sgemmStatus_t st = plan_loss(type, T, V, D, X, ldx, W, ldw, nullptr, q);      // checks
    if (st != SGEMM_STATUS_SUCCESS) return st;
    if (T == 0) return SGEMM_STATUS_SUCCESS;
    if ((st = check_vector(target, 8)) != SGEMM_STATUS_SUCCESS || (st = check_vector(loss, 4)) != SGEMM_STATUS_SUCCESS ||
        (st = check_vector(lse, 4)) != SGEMM_STATUS_SUCCESS)
        return st;
    if (h == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    st = check_device(h);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    plan_loss(type, T, V, D, X, ldx, W, ldw, h, q);
    if (h->ws == nullptr || h->ws_bytes < q.forward_bytes()) return SGEMM_STATUS_WORKSPACE_REQUIRED;

    const bool f32 = type == SGEMM_TYPE_F32;
    const LmKernel k = sg::lm_lse_kernel(q.big, f32);
    LmArgs p = loss_args(q, k, T, V, D, q.tile_n);
    char *ws = static_cast<char *>(h->ws);
    p.target = target;
    p.vocab = V;
    p.part = reinterpret_cast<float2 *>(ws);
    p.picked = reinterpret_cast<float *>(ws + q.ws_part);
    ws += q.ws_part + q.ws_picked;
    if (!copy_operands(type, q.x.place(ws), q.w.place(ws + q.x.ws), stream)) return SGEMM_STATUS_LAUNCH_FAILED;
    CUtensorMap tm_x, tm_w;
    if (!q.x.map(&tm_x, k.box_a) || !q.w.map(&tm_w, q.tile_n / (k.pair ? 2 : 1))) return SGEMM_STATUS_LAUNCH_FAILED;
    st = launch_lm(h, k, false, &tm_x, &tm_w, p, p.num_tiles, stream);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    return sg::lm_launch_lse_join(p.part, q.slabs, int(T), p.picked, target, V, loss, lse, stream) == cudaSuccess
               ? SGEMM_STATUS_SUCCESS : SGEMM_STATUS_LAUNCH_FAILED;
}

sgemmStatus_t sgemmCrossEntropyGradWorkspaceSize(sgemmHandle_t h, sgemmDataType_t type, int64_t T, int64_t V,
                                                 int64_t D, const void *X, int64_t ldx, const void *W, int64_t ldw,
                                                 size_t *bytes) {
    if (bytes == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    *bytes = 0;
    Loss q;
    sgemmStatus_t st = plan_loss(type, T, V, D, X, ldx, W, ldw, h, q);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    if (h == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    *bytes = T > 0 ? q.grad_bytes() : 0;
    return SGEMM_STATUS_SUCCESS;
}

sgemmStatus_t sgemmCrossEntropyGrad(sgemmHandle_t h, sgemmDataType_t type, int64_t T, int64_t V, int64_t D,
                                    const void *X, int64_t ldx, const void *W, int64_t ldw, const int64_t *target,
                                    const float *lse, const float *dloss, void *dX, int64_t lddx, void *dW,
                                    int64_t lddw, cudaStream_t stream) {
    Loss q;
    sgemmStatus_t st = plan_loss(type, T, V, D, X, ldx, W, ldw, nullptr, q);      // checks
    if (st != SGEMM_STATUS_SUCCESS) return st;
    st = check_matrix(dX, T, D, lddx, type, T > 0);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    st = check_matrix(dW, V, D, lddw, type, true);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    const int elem = type_size(type);
    if (T > 0 && ((st = check_vector(target, 8)) != SGEMM_STATUS_SUCCESS ||
                  (st = check_vector(lse, 4)) != SGEMM_STATUS_SUCCESS ||
                  (st = check_vector(dloss, 4)) != SGEMM_STATUS_SUCCESS))
        return st;
    if (h == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    st = check_device(h);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    plan_loss(type, T, V, D, X, ldx, W, ldw, h, q);
    if (T == 0)
        return sg::lm_launch_zero(dW, lddw, 0, elem, V, D, 1, stream) == cudaSuccess ? SGEMM_STATUS_SUCCESS
                                                                                     : SGEMM_STATUS_LAUNCH_FAILED;
    if (h->ws == nullptr || h->ws_bytes < q.grad_bytes()) return SGEMM_STATUS_WORKSPACE_REQUIRED;

    const bool f32 = type == SGEMM_TYPE_F32, f16 = type == SGEMM_TYPE_F16;
    char *ws = static_cast<char *>(h->ws);
    float *scale2 = reinterpret_cast<float *>(ws);
    void *d = ws + 256;
    void *planes = ws + 256 + q.ws_d;
    float *acc = reinterpret_cast<float *>(ws + 256 + q.ws_d + q.ws_planes);
    ws += 256 + q.ws_d + q.ws_planes + q.ws_acc;
    // Rows that take no part may hold anything, infinities and NaN too: the
    // zeros of d do not keep those out of d^T . X, so X is always a copy
    // (both gradients of 12 rows, 5000 x 768: 38.1 -> 40.5 us; of 128 rows and
    // more, within the noise).
    Operand &x = q.x_kept;
    // d is held over the largest |dloss|, taken in again by the gradient
    // products: then the entries of the targets lie at 1 - p, where all of
    // them are not rounded the same way, as they are when dloss is one over
    // the number of tokens (bf16, 853 tokens: gradients off by 0.28%, all in
    // one direction).  F16 besides times 2^13: its smallest normal number,
    // 2^-14, is above most softmax values over a long vocabulary.
    const bool scaled = f16 || (!f32 && q.d_planes == 1);
    sg::LmCopyFilter part;
    part.target = target;
    part.vocab = V;
    part.grad = dloss;
    sg::LmGradScale scale;
    if (scaled) {
        scale.grad = dloss;
        scale.target = target;
        scale.vocab = V;
        scale.rows = int(T);
        scale.top = f16 ? 8192.f : 1.f;
        scale.scale2 = scale2;
    }
    if (!copy_operands(type, x.place(ws, part), q.w.place(ws + x.ws), stream, scale)) return SGEMM_STATUS_LAUNCH_FAILED;

    const LmKernel kd = sg::lm_dlogits_kernel(q.big, f32);
    // (All pieces are as long as the first, or shorter; d in two planes makes two
    // terms of each.)
    const LmKernel kx = sg::lm_rows_kernel(q.big, false, f32, q.piece * q.d_planes > q.splits * sg::kLmPlainTerms);
    CUtensorMap tm_x, tm_w, tm_d, tm_x_mn, tm_w_mn, tm_d_mn;
    if (!x.map(&tm_x, kd.box_a) || !x.map(&tm_x_mn, 64)) return SGEMM_STATUS_LAUNCH_FAILED;
    for (int64_t i = 0; i < q.pieces; ++i) {
        const int64_t v0 = i * q.piece, width = std::min(q.piece, q.V - v0);
        const bool first = i == 0, last = i == q.pieces - 1;
        // d = (softmax - one at the target) * dloss for this piece.
        const int64_t slots = q.big ? h->sm_count / 2 : h->sm_count;
        // A piece of one round of half-wide tiles at most: narrower ones, down
        // to 32 columns, bring every SM to it.  (Both gradients of one row,
        // 9600 x 1600: 64.7 -> 57.9 us; of 100 rows, 2000 x 512: 39.8 -> 32.8.
        // More rounds of them lose, 128 rows, 50257 x 768: 120 -> 133, and so
        // does the forward pass, which also joins a part for each tile: one
        // row, 9600 x 1600: 20.3 -> 24.9.)
        const int64_t tiles_m = ceil_div(T, kd.tile_m);
        const bool one_round = !q.big && tiles_m * ceil_div(width, kd.bn / 2) <= slots;
        const int tn = balanced_tile_n(tiles_m, width, slots, kd.gran, one_round ? 32 : kd.bn / 2, kd.bn);
        LmArgs p = loss_args(q, kd, T, width, D, tn);
        p.C = d;
        p.ldc = q.ld_d;
        p.out = out_type(type);
        p.vec = 1;
        p.target = target;
        p.vocab = V;
        p.v0 = v0;
        p.lse = lse;
        p.grad = dloss;
        p.gscale = scaled ? scale2 : nullptr;
        if (q.d_planes == 2) p.lo = static_cast<char *>(d) + T * q.ld_d * 2;
        if (!q.w.map_rows(&tm_w, tn / (kd.pair ? 2 : 1), v0, width)) return SGEMM_STATUS_LAUNCH_FAILED;
        st = launch_lm(h, kd, false, &tm_x, &tm_w, p, p.num_tiles, stream);
        if (st != SGEMM_STATUS_SUCCESS) return st;

        Operand dd;
        dd.ptr = d;
        dd.rows = T;
        dd.cols = width;
        dd.ld = q.ld_d;
        dd.type = type;
        dd.batch = q.d_planes;
        dd.stride = T * q.ld_d;
        dd.plan();
        if (!copy_operands(type, dd.place(planes), {}, stream)) return SGEMM_STATUS_LAUNCH_FAILED;
        if (!dd.map(&tm_d, kx.box_a) || !dd.map(&tm_d_mn, 64) || !q.w.map_rows(&tm_w_mn, 64, v0, width))
            return SGEMM_STATUS_LAUNCH_FAILED;

        // Rows' gradient: d . W over this piece of the vocabulary.
        p = loss_args(q, kx, T, D, width, kx.bn);
        p.kb *= q.d_planes;
        p.splits = q.splits;
        p.num_tiles *= q.splits;
        if (q.splits > 1 || !last) {
            p.C = acc;
            p.ldc = q.ld_acc;
            p.stride_c = q.splits > 1 ? T * q.ld_acc : 0;
            p.out = sg::kOutF32;
            p.vec = 1;
        } else {
            p.C = dX;
            p.ldc = lddx;
            p.out = out_type(type);
            p.vec = vec_ok(dX, lddx, 0, elem, 32);
            p.alpha = scaled ? scale2 + 1 : nullptr;
        }
        p.acc_in = first ? nullptr : acc;
        p.ld_acc = q.ld_acc;
        st = launch_lm(h, kx, false, &tm_d, &tm_w_mn, p, p.num_tiles, stream);
        if (st != SGEMM_STATUS_SUCCESS) return st;
        if (q.splits > 1 &&
            sg::lm_launch_join_splits(acc, q.ld_acc, T * q.ld_acc, q.splits, scaled ? scale2 + 1 : nullptr, int(T),
                                      int(D), dX, lddx, out_type(type), stream) != cudaSuccess)
            return SGEMM_STATUS_LAUNCH_FAILED;

        // Vocabulary rows' gradient: d^T . X, complete for this piece.  In
        // pairs' tiles even where they are half empty (4096 rows, both
        // gradients of 100 x 1024: 72 us, in tiles of one SM 78).
        const LmKernel kw = sg::lm_rows_kernel(true, true, f32, T * q.d_planes > sg::kLmPlainTerms);
        p = loss_args(q, kw, width, D, T, kw.bn);
        p.kb *= q.d_planes;
        p.C = static_cast<char *>(dW) + v0 * lddw * elem;
        p.ldc = lddw;
        p.out = out_type(type);
        p.vec = vec_ok(p.C, lddw, 0, elem, 32);
        p.alpha = scaled ? scale2 + 1 : nullptr;
        st = launch_lm(h, kw, false, &tm_d_mn, &tm_x_mn, p, p.num_tiles, stream);
        if (st != SGEMM_STATUS_SUCCESS) return st;
    }
    return SGEMM_STATUS_SUCCESS;
}

sgemmStatus_t sgemmW4WorkspaceSize(sgemmHandle_t h, sgemmDataType_t type, int64_t M, int64_t N, int64_t K, int group,
                                   size_t *bytes) {
    if (bytes == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    *bytes = 0;
    W4 q;
    sgemmStatus_t st = plan_w4(type, M, N, K, group, q);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    if (h == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    *bytes = q.ws;
    return SGEMM_STATUS_SUCCESS;
}

sgemmStatus_t sgemmW4(sgemmHandle_t h, sgemmDataType_t type, int64_t M, int64_t N, int64_t K, int group,
                      const void *X, int64_t ldx, const uint8_t *Q, int64_t ldq, const void *scales, int64_t lds,
                      const uint8_t *zeros, int64_t ldz, void *Y, int64_t ldy, cudaStream_t stream) {
    W4 q;
    sgemmStatus_t st = plan_w4(type, M, N, K, group, q);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    const bool any = M > 0 && N > 0, used = any && K > 0;
    const int64_t groups = K / group;
    if ((st = check_matrix(X, M, K, ldx, type, used)) != SGEMM_STATUS_SUCCESS ||
        (st = check_matrix(scales, N, groups, lds, type, used)) != SGEMM_STATUS_SUCCESS ||
        (st = check_matrix(Y, M, N, ldy, type, any)) != SGEMM_STATUS_SUCCESS)
        return st;
    if (ldq < std::max<int64_t>(1, K / 2) || (zeros != nullptr && ldz < std::max<int64_t>(1, groups)))
        return SGEMM_STATUS_INVALID_VALUE;
    if (used) {
        if (Q == nullptr) return SGEMM_STATUS_INVALID_VALUE;
        if (!aligned(Q, 16) || (N > 1 && ldq % 16 != 0)) return SGEMM_STATUS_MISALIGNED;
        if (ldq > kMaxBytes / N || (zeros != nullptr && ldz > kMaxBytes / N)) return SGEMM_STATUS_NOT_SUPPORTED;
    }
    if (!any) return SGEMM_STATUS_SUCCESS;
    if (h == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    st = check_device(h);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    const int elem = type_size(type);
    if (K == 0)
        return sg::lm_launch_zero(Y, ldy, 0, elem, M, N, 1, stream) == cudaSuccess ? SGEMM_STATUS_SUCCESS
                                                                                   : SGEMM_STATUS_LAUNCH_FAILED;
    if (q.ws > 0 && (h->ws == nullptr || h->ws_bytes < q.ws)) return SGEMM_STATUS_WORKSPACE_REQUIRED;

    // Q as bytes: boxes of 16 rows by 128 bytes (256 columns).
    CUtensorMap tm_q;
    {
        auto enc = sg::tensor_map_encoder();
        if (enc == nullptr) return SGEMM_STATUS_LAUNCH_FAILED;
        cuuint64_t dims[2] = {cuuint64_t(K / 2), cuuint64_t(N)};
        cuuint64_t strides[1] = {cuuint64_t(N > 1 ? ldq : round_up(K / 2, 16))};
        cuuint32_t box[2] = {128, 16}, one[2] = {1, 1};
        if (enc(&tm_q, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(Q), dims, strides, box, one,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return SGEMM_STATUS_LAUNCH_FAILED;
    }
    for (int64_t t0 = 0; t0 < M; t0 += q.most) {
        const int tokens = int(std::min<int64_t>(q.most, M - t0));
        const int cols = tokens * q.planes, nb = w4_blocks(cols);
        sg::W4Args p{};
        p.N = int(N);
        p.K = int(K);
        p.tokens = tokens;
        p.k_slice = q.k_slice;
        p.X = static_cast<const char *>(X) + t0 * ldx * elem;
        p.ldx = ldx;
        p.x_vec = vec_ok(p.X, ldx, 0, elem, 16);
        p.x_pitch = int(w4_pitch(q.k_slice));
        p.Q = Q;
        p.ldq = ldq;
        p.scales = scales;
        p.lds = lds;
        p.zeros = zeros;
        p.ldz = ldz;
        p.s_vec = vec_ok(scales, lds, 0, elem, 16);
        p.z_vec = zeros == nullptr || vec_ok(zeros, ldz, 0, 1, 8);
        p.Y = static_cast<char *>(Y) + t0 * ldy * elem;
        p.ldy = ldy;
        p.part = q.slices > 1 ? static_cast<float *>(h->ws) : nullptr;
        p.ld_part = round_up(N, 8);
        LmKernel k;
        // Two CTAs on an SM where they fit, else one with more warps.
        const int64_t xs = int64_t(cols) * p.x_pitch;
        const bool alone = nb == 4 || int64_t(sg::w4_fixed_smem(nb, false)) + xs > 113 * 1024;
        const int smem = int(int64_t(sg::w4_fixed_smem(nb, alone)) + xs);
        const bool z = zeros != nullptr;
        k.fn = type == SGEMM_TYPE_F32 ? sg::w4_kernel_f32(group, nb, z, alone)
               : type == SGEMM_TYPE_F16 ? sg::w4_kernel_f16(group, nb, z, alone)
                                        : sg::w4_kernel_bf16(group, nb, z, alone);
        k.threads = sg::w4_warps(nb, alone) * 32;
        const int slots = resident_slots(h, k, smem);
        if (slots < 1) return SGEMM_STATUS_LAUNCH_FAILED;
        const int64_t blocks = ceil_div(N, 16);
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(unsigned(std::max<int64_t>(1, std::min<int64_t>(blocks, slots / q.slices))),
                           unsigned(q.slices));
        cfg.blockDim = dim3(unsigned(k.threads));
        cfg.dynamicSmemBytes = size_t(smem);
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        p.err = h->d_err;
        p.timeout_ns = h->timeout_ns;
        p.withhold = h->withhold;
        void *kargs[] = {&tm_q, &p};
        if (cudaLaunchKernelExC(&cfg, k.fn, kargs) != cudaSuccess) return SGEMM_STATUS_LAUNCH_FAILED;
        if (q.slices > 1 &&
            sg::lm_launch_join_splits(p.part, p.ld_part, int64_t(tokens) * p.ld_part, q.slices, nullptr, tokens, int(N),
                                      p.Y, ldy, out_type(type), stream) != cudaSuccess)
            return SGEMM_STATUS_LAUNCH_FAILED;
    }
    return SGEMM_STATUS_SUCCESS;
}

}  // extern "C"
