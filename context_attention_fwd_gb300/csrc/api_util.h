// api_util.h -- host helpers shared by the translation units that define
// entry points of the C ABI: logging, NVTX ranges, tensor validation.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <nvtx3/nvToolsExt.h>

#include "../../include/ctx_attn.h"

namespace ctxattn {

// CTX_ATTN_LOG=1: one line per attention call on stderr (schedule, tiles,
// kernel variant).
inline bool log_enabled() {
    static const bool on = [] {
        const char* e = getenv("CTX_ATTN_LOG");
        return e && *e && *e != '0';
    }();
    return on;
}

// An NVTX range around an entry point (visible in a profiler's timeline;
// nearly free when no tool is attached).
struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
};

inline int num_sms() {
    int dev = 0, n = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n > 0 ? n : 148;
}

// Whether a launch in the stream goes into a graph (or that cannot be told).
inline bool stream_captured(cudaStream_t s) {
    cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &st) != cudaSuccess) {
        cudaGetLastError();
        return true;
    }
    return st != cudaStreamCaptureStatusNone;
}

struct Dense {
    void* data;
    int64_t sb, ss, sh;
};

// Validates a logical [B,S,H,D] tensor and resolves its strides.
inline int resolve_strides(const ctx_tensor_t* t, int64_t B, int64_t S, int64_t H, int64_t D, ctx_layout_t layout,
                           Dense* out) {
    if (!t || !t->data) return CTX_ERR_INVALID_ARG;
    if (t->B != B || t->S != S || t->H != H || t->D != D) return CTX_ERR_INVALID_ARG;
    int64_t sb = t->stride_b, ss = t->stride_s, sh = t->stride_h;
    if (sb == 0 && ss == 0 && sh == 0) {
        if (layout == CTX_LAYOUT_BSHD) {
            sh = D; ss = H * D; sb = S * H * D;
        } else if (layout == CTX_LAYOUT_SBHD) {
            sh = D; sb = H * D; ss = B * H * D;
        } else {
            return CTX_ERR_INVALID_ARG;
        }
    }
    if (sb < 0 || ss < 0 || sh < 0) return CTX_ERR_INVALID_ARG;
    if ((B > 1 && sb == 0) || (S > 1 && ss == 0) || (H > 1 && sh == 0)) return CTX_ERR_INVALID_ARG;
    if (sh < D && H > 1) return CTX_ERR_INVALID_ARG;  // heads would overlap
    out->data = t->data;
    out->sb = sb;
    out->ss = ss;
    out->sh = sh;
    return CTX_OK;
}

// The same for the attention calls' tensors, with the alignment that TMA and
// 16-byte vector access need: 16-byte aligned base and strides.
inline int resolve(const ctx_tensor_t* t, int64_t B, int64_t S, int64_t H, int64_t D, ctx_layout_t layout,
                   Dense* out) {
    const int rc = resolve_strides(t, B, S, H, D, layout, out);
    if (rc) return rc;
    if ((reinterpret_cast<uintptr_t>(out->data) & 15) || (out->sb & 7) || (out->ss & 7) || (out->sh & 7))
        return CTX_ERR_UNSUPPORTED;
    return CTX_OK;
}

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

inline int launch_status(cudaError_t launch = cudaSuccess) {
    return launch == cudaSuccess && cudaGetLastError() == cudaSuccess ? CTX_OK : CTX_ERR_CUDA;
}

}  // namespace ctxattn
