// host_util.cuh -- host helpers shared by the translation units of the library:
// launch counter, NVTX ranges, device scope, fault injection, driver entry points
// and the checks of device pointers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <atomic>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "liteattn.h"

namespace lite {

inline std::atomic<int64_t> g_launches{0};   // kernel launches issued by the library

// NVTX range for the duration of a scope: the host side of each call shows up
// on profiler timelines (header-only NVTX3; a no-op without a tool attached).
struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange &) = delete;
    NvtxRange &operator=(const NvtxRange &) = delete;
};

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
using PtrAttrsFn = CUresult (*)(unsigned int, CUpointer_attribute *, void **, CUdeviceptr);
using CtxGetFn = CUresult (*)(CUcontext *);

struct DriverFns {
    EncodeTiledFn encode = nullptr;
    PtrAttrsFn ptr_attrs = nullptr;
    CtxGetFn ctx_get = nullptr;
    bool ok = false;
};

inline const DriverFns &driver() {
    static DriverFns fns;
    static std::once_flag once;
    std::call_once(once, [] {
        cudaDriverEntryPointQueryResult q1, q2, q3;
        void *p1 = nullptr, *p2 = nullptr, *p3 = nullptr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p1, cudaEnableDefault, &q1) == cudaSuccess &&
            q1 == cudaDriverEntryPointSuccess)
            fns.encode = reinterpret_cast<EncodeTiledFn>(p1);
        if (cudaGetDriverEntryPoint("cuPointerGetAttributes", &p2, cudaEnableDefault, &q2) == cudaSuccess &&
            q2 == cudaDriverEntryPointSuccess)
            fns.ptr_attrs = reinterpret_cast<PtrAttrsFn>(p2);
        if (cudaGetDriverEntryPoint("cuCtxGetCurrent", &p3, cudaEnableDefault, &q3) == cudaSuccess &&
            q3 == cudaDriverEntryPointSuccess)
            fns.ctx_get = reinterpret_cast<CtxGetFn>(p3);
        fns.ok = fns.encode && fns.ptr_attrs && fns.ctx_get;
    });
    return fns;
}

// Makes a plan's device current for the duration of a call and gives the caller
// back its own current device on exit, so a plan works whichever device the
// calling thread has selected (kernels, copies, events and synchronisation all
// go to the device that owns the plan's memory).  A thread that has not used CUDA
// yet has no context, which the driver calls here need: it gets the device's.
struct DeviceScope {
    int prev = -1;
    bool ok = false;
    explicit DeviceScope(int device) {
        if (cudaGetDevice(&prev) != cudaSuccess) {
            cudaGetLastError();
            prev = -1;
            return;
        }
        CUcontext ctx = nullptr;
        const bool bound = prev == device && driver().ok && driver().ctx_get(&ctx) == CUDA_SUCCESS && ctx;
        ok = bound || cudaSetDevice(device) == cudaSuccess;
    }
    ~DeviceScope() {
        int cur = -1;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
    }
    DeviceScope(const DeviceScope &) = delete;
    DeviceScope &operator=(const DeviceScope &) = delete;
};

constexpr int kMaxDevices = 64;

// Fault injection for tests: LITE_ATTN_FAULT=alloc|launch|status makes the
// matching host path report its error without touching the GPU;
// LITE_ATTN_FAULT=device_wait makes the attention kernel's first CTA wait on a
// barrier that nothing arrives on, so its bounded wait runs out and the step
// reports LITE_ERR_DEVICE_TIMEOUT through the status word.
inline bool fault(const char *what) {
    const char *e = std::getenv("LITE_ATTN_FAULT");
    return e && std::strcmp(e, what) == 0;
}

inline int cuda_err(cudaError_t e) { return e == cudaSuccess ? LITE_OK : LITE_ERR_CUDA; }

// Checks that [ptr, ptr + bytes) is device memory of `device` inside one allocation,
// and that ptr is aligned to `align` bytes (a power of two).
// One driver call (a serving step asks a dozen times); a second where the allocation may be a
// reserved range of addresses of which only a part is mapped (virtual memory management, pools):
// there the last byte must be mapped too.
inline bool device_range_ok(const void *ptr, size_t bytes, int device, uintptr_t align = 16) {
    if (!ptr || (reinterpret_cast<uintptr_t>(ptr) & (align - 1u)) || !driver().ok) return false;
    unsigned int type = 0, managed = 0;
    int ordinal = -1;
    CUdeviceptr start = 0, mapped_at = 0;
    size_t size = 0, mapped = 0;
    CUpointer_attribute which[7] = {CU_POINTER_ATTRIBUTE_MEMORY_TYPE, CU_POINTER_ATTRIBUTE_IS_MANAGED, CU_POINTER_ATTRIBUTE_DEVICE_ORDINAL,
                                    CU_POINTER_ATTRIBUTE_RANGE_START_ADDR, CU_POINTER_ATTRIBUTE_RANGE_SIZE,
                                    CU_POINTER_ATTRIBUTE_MAPPING_BASE_ADDR, CU_POINTER_ATTRIBUTE_MAPPING_SIZE};
    void *out[7] = {&type, &managed, &ordinal, &start, &size, &mapped_at, &mapped};
    if (driver().ptr_attrs(7, which, out, reinterpret_cast<CUdeviceptr>(ptr)) != CUDA_SUCCESS) return false;
    if (!managed && (type != CU_MEMORYTYPE_DEVICE || ordinal != device)) return false;
    const uintptr_t b = static_cast<uintptr_t>(start), m = static_cast<uintptr_t>(mapped_at), x = reinterpret_cast<uintptr_t>(ptr);
    if (x < b || bytes > size || x - b > size - bytes) return false;
    if (managed || bytes == 0 || (x >= m && x - m <= mapped && bytes <= mapped - (x - m))) return true;
    return driver().ptr_attrs(3, which, out, static_cast<CUdeviceptr>(x + bytes - 1)) == CUDA_SUCCESS &&
           type == CU_MEMORYTYPE_DEVICE && ordinal == device;
}

}  // namespace lite
