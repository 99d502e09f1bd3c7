// The library handle, shared by the translation units that implement the C
// ABI, and the driver's tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstddef>
#include <cstdint>

#include "../../include/sgemm_gb300.h"

namespace sg {
constexpr uint64_t kDefaultTimeoutNs = 2000000000ull;
// cuTensorMapEncodeTiled, looked up once; NULL without a driver.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();
}  // namespace sg

struct sgemmContext {
    int device = -1;
    int sm_count = 0;
    // Device control block (allocated with the handle): word 0 the error
    // word, words 1-2 the stream-K launch sequence {tag, CTAs finished},
    // from word kCtlFlagsOffset the stream-K flags (kCtlFlagWords words: one
    // per CTA and warp of a launch).
    uint32_t *d_err = nullptr;
    uint32_t *d_flags = nullptr;
    uint32_t *d_sk_seq = nullptr;
    int flag_words = 0;
    void *ws = nullptr;
    size_t ws_bytes = 0;
    uint64_t timeout_ns = sg::kDefaultTimeoutNs;
    int algo = 0;
    int schedule = 0;   // 0 automatic, 1 whole tiles only, 2 stream-K whenever it applies
    int math = 0;       // 0 FP32 FFMA, 1 error-compensated 3xTF32 on the tensor cores
    int withhold = 0;   // test hook: signal the kernels leave out (sg::Withhold)
    cudaEvent_t ev_start = nullptr, ev_stop = nullptr;   // around the main kernel, if set
    // sgemmHostEx pipeline: copy-in and copy-out streams and their events,
    // created with the handle.
    static constexpr int kHostChunks = 8;     // pieces of one sgemmHostEx call (at most 7)
    cudaStream_t s_in = nullptr, s_out = nullptr;
    cudaEvent_t ev_begin = nullptr, ev_end = nullptr;
    cudaEvent_t ev_in[kHostChunks] = {}, ev_done[kHostChunks] = {};
};
