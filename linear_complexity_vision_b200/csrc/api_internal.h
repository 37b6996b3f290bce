// Host-side helpers of the C ABI shared by its translation units: the
// thread's last error and kernel, argument checks, and per-device lookups.
// Defined in vrwkv_api.cu unless noted.
#pragma once

#include <atomic>
#include <cstddef>

#include <cuda.h>
#include <cuda_runtime.h>

#include "vrwkv.h"

namespace vrwkv {
namespace api {

// Record the reason of a non-OK status (printf-style) and return it.
vrwkv_status fail(vrwkv_status s, const char* fmt, ...);
vrwkv_status ok();
vrwkv_status cuda_status(cudaError_t e, const char* what);
void set_last_kernel(const char* name);

bool aligned(const void* p, size_t a);
bool overlaps(const void* a, size_t na, const void* b, size_t nb);
int elem_bytes(vrwkv_dtype dt);

// Current device: its SM count, its error word (nullptr if unknown) and the
// limit of bounded waits in nanoseconds.
int sm_count();
unsigned int* device_error_word();
constexpr unsigned long long kDefaultWaitNs = 2000000000ull;
unsigned long long wait_limit_ns();

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn();  // nullptr if the driver does not offer it

// Raise the dynamic shared-memory limit of a kernel once per size needed.
template <typename K>
cudaError_t ensure_smem(K kernel, std::atomic<int>& granted, int bytes) {
    if (bytes <= 48 * 1024 || bytes <= granted.load(std::memory_order_relaxed)) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) {
        int cur = granted.load();
        while (bytes > cur && !granted.compare_exchange_weak(cur, bytes)) {
        }
    }
    return e;
}

// The same for each device: the limit belongs to a device's copy of the kernel.
struct SmemGrants {
    std::atomic<int> of[64] = {};
};
template <typename K>
cudaError_t ensure_smem(K kernel, SmemGrants& granted, int bytes) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64) return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    return ensure_smem(kernel, granted.of[dev], bytes);
}

// One kernel launch.  `follows`: it may begin while the stream's last kernel,
// one of the same call, ends (passes.cuh).
template <typename... P, typename... A>
vrwkv_status launch(void (*kernel)(P...), const char* name, dim3 grid, int threads, int smem, bool follows, cudaStream_t s,
                    const A&... args) {
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = follows ? 1 : 0;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, args...), name);
}
}  // namespace api

// The LayerNorm forward launch (layer_norm_api.cu); its arguments are checked.
struct LayerNormParams;
namespace api {
vrwkv_status launch_layer_norm(const LayerNormParams& p, vrwkv_dtype dtype, cudaStream_t s);
}  // namespace api
}  // namespace vrwkv
