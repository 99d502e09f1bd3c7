// C ABI of the products in 8-bit integers (declared in
// include/sgemm_gb300_lm.h): argument checks, the choice of kernel, the rows'
// integers in the workspace, launches.
#include "lm_host.h"
#include "lm_int8.h"

namespace {

using namespace sg::host;

sgemmStatus_t status(cudaError_t e) { return e == cudaSuccess ? SGEMM_STATUS_SUCCESS : SGEMM_STATUS_LAUNCH_FAILED; }

struct Int8 {
    int from = 0, to = 0;
    int64_t T = 0, N = 0, K = 0, G = 0;
    bool rows = false;               // lm_int8_rows.cu
    bool x_copy = false;             // x is written to the workspace
    int64_t ldx = 0;                 // pitch of the integers, elements
    bool w_copy = false;
    int64_t ldw = 0, stride_w = 0;
    // rows
    int tokens = 0, warps = 0, ks = 0, slices = 1;
    int64_t k_slice = 0, x_pitch = 0, smem = 0;
    // tensor cores
    bool wide = false;
    int tile_n = 0, splits = 1;
    int64_t ld_part = 0;
    size_t ws_x = 0, ws_scales = 0, ws_w = 0, ws_group = 0, ws_part = 0;
    int parts() const { return rows ? slices : splits; }
    size_t bytes() const { return ws_x + ws_scales + ws_w + ws_group + ws_part; }
};

sgemmStatus_t check_x(int from, const void *X, int64_t T, int64_t K, int64_t ldx, bool used) {
    if (from != SGEMM_TYPE_S8) return check_matrix(X, T, K, ldx, from, used);
    if (ldx < std::max<int64_t>(1, K)) return SGEMM_STATUS_INVALID_VALUE;
    if (!used) return SGEMM_STATUS_SUCCESS;
    if (X == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    return T > kMaxDim || ldx > kMaxBytes / T ? SGEMM_STATUS_NOT_SUPPORTED : SGEMM_STATUS_SUCCESS;
}

// Few rows a group in the mean: straight from memory, W read once for up to 8 of
// them; otherwise the tensor cores (8 rows, 28672 x 8192: 46 and 51 us, 12 rows 84 of
// 16 at a time and 51; 16 groups of 8 rows, 2048 x 1408: 16.8 and 17.9, of 12, 20.0
// and 18.1).  The sizes of the groups are on the device, so T / G decides, and it was
// chosen for even ones.  Where a few groups have all rows, W is read and converted
// again for every 8 of them, and the other kernel would be faster: 512 rows, 64 groups
// of 1024 x 2048, even 31.3 and 31.7 us, in 16 groups 28 and 13.6, in one 27 and 13.5;
// 1024 rows, 128 groups, even 53 and 56, in four 46 and 20.5.
constexpr int64_t kInt8FewRows = 8;
// Bytes of x that every CTA quantises itself instead of a launch of its own (one
// row, 4096 x 4096: 5.5 us, 7.3).
constexpr int64_t kInt8OwnBytes = 16384;

sgemmStatus_t plan_int8(const sgemmContext *h, int from, int to, int64_t T, int64_t N, int64_t K, int64_t G,
                        const void *X, int64_t ldx, const int8_t *W, int64_t ldw, int64_t strideW, Int8 &q) {
    if ((!type_ok(from) && from != SGEMM_TYPE_S8) || !type_ok(to)) return SGEMM_STATUS_INVALID_VALUE;
    if (T < 0 || N < 0 || K < 0 || G < 0 || strideW < 0) return SGEMM_STATUS_INVALID_VALUE;
    if (T > kMaxDim - 512 || N > kMaxDim - 512 || K > sg::kInt8MaxK || G > SGEMM_MAX_GROUPS)
        return SGEMM_STATUS_NOT_SUPPORTED;
    const bool used = T > 0 && N > 0 && K > 0 && G > 0;
    sgemmStatus_t st = check_x(from, X, T, K, ldx, used);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    if (ldw < std::max<int64_t>(1, K)) return SGEMM_STATUS_INVALID_VALUE;
    if (used) {
        if (W == nullptr) return SGEMM_STATUS_INVALID_VALUE;
        if (ldw > kMaxBytes / N) return SGEMM_STATUS_NOT_SUPPORTED;
        if (G > 1) {
            if (strideW < (N - 1) * ldw + K) return SGEMM_STATUS_INVALID_VALUE;
            if (strideW > kMaxBytes / G) return SGEMM_STATUS_NOT_SUPPORTED;
        }
    }
    q.from = from;
    q.to = to;
    q.T = T; q.N = N; q.K = K; q.G = G;
    if (!used || h == nullptr) return SGEMM_STATUS_SUCCESS;
    const bool w_tma = aligned(W, 16) && ldw % 16 == 0 && (G == 1 || strideW % 16 == 0);
    const int64_t mean = T / G;
    q.rows = mean <= kInt8FewRows;
    q.ws_scales = from == SGEMM_TYPE_S8 ? 0 : align256(T * 4);
    if (q.rows) {
        const bool own = from != SGEMM_TYPE_S8 && G == 1 && T * K * type_size(from) <= kInt8OwnBytes;
        q.x_copy = !own && (from != SGEMM_TYPE_S8 || !aligned(X, 16) || ldx % 16 != 0);
        q.ldx = q.x_copy ? round_up(K, 16) : ldx;
        q.ws_x = q.x_copy ? align256(T * q.ldx) : 0;
        // (By group the mean decides, the sizes being on the device: tiles of four
        // tokens where it is about one.)
        if (G == 1) q.tokens = T == 1 ? 1 : T == 2 ? 2 : T <= 4 ? 4 : 8;
        else q.tokens = mean <= 1 ? 4 : 8;
        const int rows = int(std::min<int64_t>(T, q.tokens));
        // x of a tile's tokens beside half of an SM's shared memory, all of it,
        // or the contraction in parts.
        for (q.slices = 1;; ++q.slices) {
            q.k_slice = round_up(ceil_div(K, q.slices), 256);
            q.warps = 8;
            q.smem = sg::int8_rows_smem(q.tokens, rows, 8, q.k_slice, G);
            if (q.smem <= 113 * 1024) break;
            q.warps = 16;
            q.smem = sg::int8_rows_smem(q.tokens, rows, 16, q.k_slice, G);
            if (q.smem <= kMaxSmem) break;
        }
        q.x_pitch = sg::int8_rows_pitch(q.tokens, q.k_slice);
        q.slices = int(ceil_div(K, q.k_slice));
        // Warps that share 16 rows of W, no more than there are steps: with the least
        // rounds of tiles times what a tile costs: its rows, and for its beginning and
        // end about what 24 KB of W take (128 rows over 64 groups of 2048 x 1024: 35 us
        // with tiles of 128 rows, 41 of 32; one row, 28672 x 8192: 41 of 32, 45 of 128).
        const int64_t slots = std::max<int64_t>(1, int64_t(h->sm_count) * (q.warps == 8 ? 2 : 1) / q.slices);
        const int64_t chunks = ceil_div(T, q.tokens) + std::min(G, T) - 1, steps = q.k_slice / 256;
        int64_t best = 0;
        const int least = q.warps == 8 ? 1 : 4;
        for (int ks = q.warps; ks >= least; ks = ks == 4 ? 1 : ks / 2) {
            if (ks > steps && ks > least) continue;
            const int64_t high = 16 * (q.warps / ks), rounds = ceil_div(ceil_div(N, high) * chunks, slots);
            const int64_t cost = rounds * (high + 4 + 24576 / q.k_slice);
            if (best == 0 || cost < best) {
                best = cost;
                q.ks = ks;
            }
        }
    } else {
        q.x_copy = true;
        q.ldx = round_up(K, 8);
        q.ws_x = align256(T * q.ldx * 2);
        q.w_copy = !w_tma;
        if (q.w_copy) {
            q.ldw = round_up(K, 16);
            q.stride_w = q.ldw * N;
            q.ws_w = align256(q.stride_w * G);
        }
        // Kernel and rows of a tile.  One matrix: what has the least rounds of tiles times
        // what a tile costs, which is hardly less for fewer rows, as its W is converted
        // all the same (8192 rows, 4096 x 14336: 48 rounds of 128, 583 us, 32 of 192,
        // 552; 2048 rows: 12 of 128, 152, 9 of 192, 193; 2048 rows, 4096 x 4096: 4 of 128,
        // 68, 3 of 160, 62).  Groups: as many as one has in the mean, wide from 512 on
        // (16 of 2048 rows, 4096 x 2048: 429 us, 441; 64 of 128, 1024 x 2048: 57, 53).
        const int64_t pairs = h->sm_count / 2, high = ceil_div(N, 256);
        const int64_t blocks = ceil_div(K, 256);
        // (Parts of the contraction, of two blocks at least, where the tiles leave
        // pairs idle; joining them takes what ten blocks do.)
        auto parts_of = [&](int64_t tiles) {
            return std::max<int64_t>(1, std::min(pairs / std::max<int64_t>(1, tiles), blocks / 2));
        };
        if (G == 1) {
            int64_t best = 0;
            for (int n = 192; n >= 32; n -= 32) {
                if (n >= T + 32) continue;
                const int64_t tiles = high * ceil_div(T, n), parts = parts_of(tiles);
                const int64_t cost = ceil_div(tiles, pairs) * ceil_div(blocks, parts) * (n > 160 ? 196 : n > 128 ? 184 : 138) +
                                     (parts > 1 ? 1380 : 0);
                if (best != 0 && cost >= best) continue;
                best = cost;
                q.tile_n = n;
            }
            q.splits = int(parts_of(high * ceil_div(T, q.tile_n)));
        } else {
            const int most = sg::int8_mma_kernel(mean >= 512).bn;
            q.tile_n = int(std::min<int64_t>(most, round_up(std::max<int64_t>(mean, 1), 32)));
            q.splits = int(parts_of(high * (T / q.tile_n + std::min(G, T))));
        }
        q.wide = q.tile_n > 128;
    }
    if (q.parts() > 1) {
        q.ld_part = round_up(N, 8);
        q.ws_group = align256(T * 4);
        q.ws_part = align256(q.parts() * T * q.ld_part * 4);
    }
    return SGEMM_STATUS_SUCCESS;
}

}  // namespace

extern "C" {

sgemmStatus_t sgemmInt8Quantize(sgemmHandle_t h, sgemmDataType_t type, int64_t T, int64_t K, const void *X, int64_t ldx,
                                int8_t *Q, int64_t ldq, float *scales, cudaStream_t stream) {
    if (!type_ok(type) || T < 0 || K < 0) return SGEMM_STATUS_INVALID_VALUE;
    if (T > kMaxDim || K > kMaxDim) return SGEMM_STATUS_NOT_SUPPORTED;
    sgemmStatus_t st = check_matrix(X, T, K, ldx, type, T > 0 && K > 0);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    if (ldq < std::max<int64_t>(1, K)) return SGEMM_STATUS_INVALID_VALUE;
    if (T == 0) return SGEMM_STATUS_SUCCESS;
    if (K > 0 && Q == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    if (ldq > kMaxBytes / T) return SGEMM_STATUS_NOT_SUPPORTED;
    if ((st = check_vector(scales, 4)) != SGEMM_STATUS_SUCCESS) return st;
    if (h == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    if ((st = check_device(h)) != SGEMM_STATUS_SUCCESS) return st;
    return status(sg::int8_quantize_launch(type, X, ldx, T, K, Q, ldq, K, false, scales, false, stream));
}

sgemmStatus_t sgemmInt8WorkspaceSize(sgemmHandle_t h, sgemmDataType_t typeX, sgemmDataType_t typeC, int64_t T, int64_t N,
                                     int64_t K, int64_t G, const void *X, int64_t ldx, const int8_t *B, int64_t ldb,
                                     int64_t strideB, size_t *bytes) {
    if (bytes == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    *bytes = 0;
    Int8 q;
    sgemmStatus_t st = plan_int8(h, typeX, typeC, T, N, K, G, X, ldx, B, ldb, strideB, q);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    if (h == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    *bytes = q.bytes();
    return SGEMM_STATUS_SUCCESS;
}

sgemmStatus_t sgemmInt8(sgemmHandle_t h, sgemmDataType_t typeX, sgemmDataType_t typeC, int64_t T, int64_t N, int64_t K,
                        int64_t G, const void *X, int64_t ldx, const float *xScales, const int8_t *B, int64_t ldb,
                        int64_t strideB, const float *scales, const int32_t *groupEnds, void *C, int64_t ldc,
                        cudaStream_t stream) {
    Int8 q;
    sgemmStatus_t st = plan_int8(nullptr, typeX, typeC, T, N, K, G, X, ldx, B, ldb, strideB, q);      // checks
    if (st != SGEMM_STATUS_SUCCESS) return st;
    st = check_matrix(C, T, N, ldc, typeC, T > 0 && N > 0);
    if (st != SGEMM_STATUS_SUCCESS) return st;
    const bool used = T > 0 && N > 0 && K > 0 && G > 0;
    if (groupEnds == nullptr ? G != 1 && T > 0 && N > 0 && G > 0 : !aligned(groupEnds, 4))
        return groupEnds == nullptr ? SGEMM_STATUS_INVALID_VALUE : SGEMM_STATUS_MISALIGNED;
    if ((typeX == SGEMM_TYPE_S8) != (xScales != nullptr) && used) return SGEMM_STATUS_INVALID_VALUE;
    if (used && ((xScales != nullptr && (st = check_vector(xScales, 4)) != SGEMM_STATUS_SUCCESS) ||
                 (st = check_vector(scales, 4)) != SGEMM_STATUS_SUCCESS))
        return st;
    if (T == 0 || N == 0) return SGEMM_STATUS_SUCCESS;
    if (h == nullptr) return SGEMM_STATUS_INVALID_VALUE;
    if ((st = check_device(h)) != SGEMM_STATUS_SUCCESS) return st;
    const int elem = type_size(typeC);
    if (K == 0 || G == 0) return status(sg::lm_launch_zero(C, ldc, 0, elem, T, N, 1, stream));
    plan_int8(h, typeX, typeC, T, N, K, G, X, ldx, B, ldb, strideB, q);
    if (q.bytes() > 0 && (h->ws == nullptr || h->ws_bytes < q.bytes())) return SGEMM_STATUS_WORKSPACE_REQUIRED;

    char *ws = static_cast<char *>(h->ws);
    void *x_ws = ws;
    float *x_scales_ws = reinterpret_cast<float *>(ws + q.ws_x);
    int8_t *w_ws = reinterpret_cast<int8_t *>(ws + q.ws_x + q.ws_scales);
    int32_t *group_ws = reinterpret_cast<int32_t *>(ws + q.ws_x + q.ws_scales + q.ws_w);
    int32_t *part = reinterpret_cast<int32_t *>(ws + q.ws_x + q.ws_scales + q.ws_w + q.ws_group);

    sg::Int8Args a{};
    a.lm.M = int(N);
    a.lm.T = int(T);
    a.lm.G = int(G);
    a.lm.ends = groupEnds;
    a.lm.err = h->d_err;
    a.lm.timeout_ns = h->timeout_ns;
    a.lm.withhold = h->withhold;
    a.lm.group_m = 8;
    a.x_scales = xScales != nullptr ? xScales : x_scales_ws;
    a.scales = scales;
    a.K = int(K);
    const int parts = q.parts();
    a.lm.splits = parts;
    if (parts > 1) {
        a.lm.C = part;
        a.lm.ldc = q.ld_part;
        a.lm.stride_c = T * q.ld_part;
        a.lm.out = sg::kOutF32;
        a.row_group = group_ws;
    } else {
        a.lm.C = C;
        a.lm.ldc = ldc;
        a.lm.out = out_type(typeC);
        a.lm.vec = vec_ok(C, ldc, 0, elem, 16);
    }
    sg::LmKernel k;
    int64_t tiles;
    if (q.rows) {
        k = sg::int8_rows_kernel(q.tokens, q.warps, q.ks);
        a.lm.tile_n = k.bn;
        a.lm.tiles_m = int(ceil_div(N, k.tile_m));
        tiles = int64_t(a.lm.tiles_m) * (ceil_div(T, a.lm.tile_n) + G + 1);
    } else {
        k = sg::int8_mma_kernel(q.wide);
        a.lm.tile_n = q.tile_n;
        a.lm.tiles_m = int(ceil_div(N, k.tile_m));
        a.lm.kb = int(ceil_div(K, k.gran));
        tiles = int64_t(a.lm.tiles_m) * (ceil_div(T, a.lm.tile_n) + G + 1) * q.splits;
    }
    if (tiles > kMaxDim) return SGEMM_STATUS_NOT_SUPPORTED;
    if (q.w_copy && (st = status(sg::int8_copy_launch(B, ldb, G > 1 ? strideB : 0, N, K, G, w_ws, q.ldw, groupEnds,
                                                      stream))) != SGEMM_STATUS_SUCCESS)
        return st;
    if (q.x_copy && (st = status(sg::int8_quantize_launch(typeX, X, ldx, T, K, x_ws, q.ldx, q.ldx, !q.rows, x_scales_ws, true,
                                                          stream))) != SGEMM_STATUS_SUCCESS)
        return st;

    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = k.pair ? 2 : 1;
    cfg.blockDim = dim3(unsigned(k.threads));
    cfg.stream = stream;
    if (q.rows) {
        a.x = q.x_copy ? x_ws : X;
        a.from = q.x_copy ? int(SGEMM_TYPE_S8) : typeX;
        a.x_vec = a.from == SGEMM_TYPE_S8 ? 1 : vec_ok(X, ldx, 0, type_size(typeX), 16);
        a.ldx = q.ldx;
        a.w = B;
        a.ldw = ldb;
        a.stride_w = G > 1 ? strideB : 0;
        a.w_vec = aligned(B, 16) && ldb % 16 == 0 && a.stride_w % 16 == 0;
        a.k_slice = int(q.k_slice);
        a.x_pitch = int(q.x_pitch);
        a.early = q.x_copy && a.w_vec;
        const int slots = resident_slots(h, k, int(q.smem));
        if (slots < 1) return SGEMM_STATUS_LAUNCH_FAILED;
        cfg.gridDim = dim3(unsigned(std::max<int64_t>(1, std::min<int64_t>(tiles, slots / q.slices))), unsigned(q.slices));
        cfg.dynamicSmemBytes = size_t(q.smem);
        void *args[] = {&a};
        st = status(cudaLaunchKernelExC(&cfg, k.fn, args));
    } else {
        auto enc = sg::tensor_map_encoder();
        if (enc == nullptr) return SGEMM_STATUS_LAUNCH_FAILED;
        CUtensorMap tm_w, tm_x;
        const int64_t wl = q.w_copy ? q.ldw : ldb, wst = q.w_copy ? q.stride_w : G > 1 ? strideB : N * ldb;
        cuuint64_t wd[3] = {cuuint64_t(K), cuuint64_t(N), cuuint64_t(G)};
        cuuint64_t wstr[2] = {cuuint64_t(wl), cuuint64_t(wst)};
        cuuint32_t wbox[3] = {128, 128, 1}, one[3] = {1, 1, 1};
        cuuint64_t xd[3] = {cuuint64_t(K), cuuint64_t(T), 1};
        cuuint64_t xstr[2] = {cuuint64_t(q.ldx) * 2, cuuint64_t(q.ldx) * 2 * cuuint64_t(T)};
        cuuint32_t xbox[3] = {64, cuuint32_t(q.tile_n / 2), 1};
        if (enc(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, q.w_copy ? static_cast<void *>(w_ws) : const_cast<int8_t *>(B), wd,
                wstr, wbox, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
            enc(&tm_x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, x_ws, xd, xstr, xbox, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return SGEMM_STATUS_LAUNCH_FAILED;
        const int smem = k.smem + 8 * (sg::kLmMaxGroups + 2);
        const int slots = resident_slots(h, k, smem);
        if (slots < 1) return SGEMM_STATUS_LAUNCH_FAILED;
        cfg.gridDim = dim3(unsigned(std::min<int64_t>(tiles, slots) * 2));
        cfg.dynamicSmemBytes = size_t(smem);
        void *args[] = {&tm_w, &tm_x, &a};
        st = status(cudaLaunchKernelExC(&cfg, k.fn, args));
    }
    if (st != SGEMM_STATUS_SUCCESS || parts == 1) return st;
    return status(sg::int8_join_launch(part, q.ld_part, T * q.ld_part, parts, group_ws, a.x_scales, scales, T, N, C, ldc,
                                       out_type(typeC), stream));
}

}  // extern "C"
