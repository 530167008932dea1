// Host helpers shared by the ABI's translation units: streams, device
// selection, status codes, and NVTX ranges around the entry points (build
// with -DPULSAR_NVTX: header-only NVTX3, no link dependency, no cost when no
// tool is attached; compiled out by default).
#pragma once

#include <cuda_runtime.h>

#include "../../include/pulsar.h"

#ifdef PULSAR_NVTX
#include <nvtx3/nvToolsExt.h>
namespace {
struct NvtxScope {
    explicit NvtxScope(const char* name) { nvtxRangePushA(name); }
    ~NvtxScope() { nvtxRangePop(); }
};
}  // namespace
#define PULSAR_TRACE(name) NvtxScope pulsar_trace_scope_(name)
#else
#define PULSAR_TRACE(name) ((void)0)
#endif

namespace {

inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

inline int cuda_err(cudaError_t e) { return e == cudaSuccess ? PULSAR_OK : PULSAR_ERR_CUDA; }

struct DeviceGuard {
    int prev = -1;
    explicit DeviceGuard(int dev) {
        if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
        if (prev != dev) cudaSetDevice(dev);
    }
    ~DeviceGuard() {
        int cur = -1;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
    }
};

}  // namespace
