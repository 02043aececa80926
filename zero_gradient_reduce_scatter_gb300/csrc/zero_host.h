// Host helpers of the calls that take no context (training losses, gradient clipping): the
// device a call runs on, and which pointers it may hand to its kernels.
#pragma once

#include <cstdint>
#include <utility>

#include <cuda_runtime.h>

#include "zero_gb300.h"
#include "zero_internal.h"

namespace zg {

constexpr int64_t type_size(int32_t type) { return type == ZERO_T_FP32 ? 4 : 2; }
// A temperature whose scale and inverse are ordinary fp32 numbers (false for NaN).
constexpr bool temperature_ok(double t) { return t >= 0x1p-64 && t <= 0x1p64; }
constexpr bool type_ok(int32_t type) { return type >= ZERO_T_BF16 && type <= ZERO_T_FP32; }
inline bool aligned(const void* p, int64_t to) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(to - 1)) == 0; }

// The device of a call: that of its first buffer, made current while the object lives and the
// caller's current device restored after. `rc` is the status so far; the checks below keep the
// first failure. Nothing is remembered between calls.
class CallDevice {
public:
    int rc = ZERO_OK;

    CallDevice(const void* first, void* stream) {
        // Queries about pointers count as unsafe while a stream is being captured in the global
        // mode; they touch no stream, so this thread asks in the relaxed mode.
        if (cudaThreadExchangeStreamCaptureMode(&mode_) != cudaSuccess) cudaGetLastError();
        cudaPointerAttributes at;
        if (!first || cudaPointerGetAttributes(&at, first) != cudaSuccess) {
            cudaGetLastError();  // clear the (non-sticky) error of an unknown pointer
            rc = ZERO_ERR_INVALID_ARG;
            return;
        }
        if (cudaGetDevice(&prev_) != cudaSuccess) prev_ = -1;
        if (at.type == cudaMemoryTypeDevice) dev_ = at.device;
        else if (at.type == cudaMemoryTypeManaged) dev_ = prev_;
        if (dev_ < 0) {
            rc = ZERO_ERR_INVALID_ARG;
            return;
        }
        if (prev_ != dev_) {
            const cudaError_t e = cudaSetDevice(dev_);
            if (e != cudaSuccess) rc = record_cuda_error(e);
            else restore_ = prev_ >= 0;
        }
        int sdev = -1;
        cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
        if (rc == ZERO_OK && stream && cudaStreamIsCapturing((cudaStream_t)stream, &capture) == cudaSuccess &&
            capture == cudaStreamCaptureStatusNone &&
            (cudaStreamGetDevice((cudaStream_t)stream, &sdev) != cudaSuccess || sdev != dev_))
            rc = ZERO_ERR_INVALID_ARG;
        cudaGetLastError();
    }
    ~CallDevice() {
        if (restore_) cudaSetDevice(prev_);
        if (cudaThreadExchangeStreamCaptureMode(&mode_) != cudaSuccess) cudaGetLastError();
    }
    CallDevice(const CallDevice&) = delete;
    CallDevice& operator=(const CallDevice&) = delete;

    // `p` must be memory of the call's device, aligned to `to` bytes.
    void need(const void* p, int64_t to) {
        if (rc != ZERO_OK) return;
        if (!p) {
            rc = ZERO_ERR_INVALID_ARG;
            return;
        }
        cudaPointerAttributes at;
        if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
            cudaGetLastError();
            rc = ZERO_ERR_INVALID_ARG;
        } else if (!(at.type == cudaMemoryTypeManaged || (at.type == cudaMemoryTypeDevice && at.device == dev_))) {
            rc = ZERO_ERR_INVALID_ARG;
        } else if (!aligned(p, to)) {
            rc = ZERO_ERR_MISALIGNED;
        }
    }
    void optional(const void* p, int64_t to) {
        if (p) need(p, to);
    }
    int sm_count() const {
        int n = 0;
        return cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev_) == cudaSuccess && n > 0 ? n : 1;
    }

private:
    int prev_ = -1, dev_ = -1;
    bool restore_ = false;
    cudaStreamCaptureMode mode_ = cudaStreamCaptureModeRelaxed;  // then the caller's own
};

// A launch that may begin while the kernel before it on the stream is still running, in clusters
// of `cluster` CTAs: the kernel waits for its predecessor (griddepcontrol.wait) before it touches
// memory that the predecessor may write or still read.
template <class... P, class... A>
int launch_linked(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, int cluster, cudaStream_t s, A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    launches_without_context(s).fetch_add(1, std::memory_order_relaxed);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
    return e == cudaSuccess ? ZERO_OK : record_cuda_error(e);
}

inline int launched() {
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? ZERO_OK : record_cuda_error(e);
}

}  // namespace zg
