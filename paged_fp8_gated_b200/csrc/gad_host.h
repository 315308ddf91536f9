// gad_host.h - host-side helpers shared by the library's translation units (not
// part of the public interface): device queries, one-time set-up per (device,
// context), launch attributes and the tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>
#include <initializer_list>

#include "gad_attn.h"
#include "gad_error.h"

#define fail gad_fail

namespace gad_host {

constexpr int kMaxDevices = 64;
constexpr size_t kAlign = 256;

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline int current_device_sms(int* sms, int* major) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fail(GAD_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
    e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return fail(GAD_ERR_CUDA, "cudaDeviceGetAttribute: %s", cudaGetErrorString(e));
    e = cudaDeviceGetAttribute(major, cudaDevAttrComputeCapabilityMajor, dev);
    if (e != cudaSuccess) return fail(GAD_ERR_CUDA, "cudaDeviceGetAttribute: %s", cudaGetErrorString(e));
    return GAD_OK;
}

// Whether the byte ranges [a, a + na) and [b, b + nb) share a byte (a NULL one, of an
// argument that is left out, shares none).
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x != 0 && y != 0 && x < y + nb && y < x + na;
}

// A stretch of memory that a call reads or writes.
struct Span {
    const void* p;
    size_t n;
};
// Whether a stretch that is written shares a byte with another one of the call.
inline bool written_overlap(std::initializer_list<Span> written, std::initializer_list<Span> read) {
    for (const Span* w = written.begin(); w != written.end(); ++w) {
        for (const Span* o = w + 1; o != written.end(); ++o)
            if (overlap(w->p, w->n, o->p, o->n)) return true;
        for (const Span& r : read)
            if (overlap(w->p, w->n, r.p, r.n)) return true;
    }
    return false;
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A driver entry point by name (nullptr if the driver does not export it).
inline void* driver_fn(const char* name) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint(name, &f, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
        return nullptr;
    return f;
}

// Unique id of the calling thread's current CUDA context, 0 if there is none
// yet or the driver cannot say.  Per-device set-up done once (function
// attributes, device-symbol addresses) is remembered together with this id,
// so a new context on the device (after cudaDeviceReset, say) repeats it.
inline unsigned long long current_ctx_id() {
    static std::atomic<PFN_cuCtxGetCurrent_v4000> get_cur{nullptr};
    static std::atomic<PFN_cuCtxGetId_v12000> get_id{nullptr};
    PFN_cuCtxGetCurrent_v4000 gc = get_cur.load(std::memory_order_acquire);
    PFN_cuCtxGetId_v12000 gi = get_id.load(std::memory_order_acquire);
    if (gc == nullptr || gi == nullptr) {
        gc = reinterpret_cast<PFN_cuCtxGetCurrent_v4000>(driver_fn("cuCtxGetCurrent"));
        gi = reinterpret_cast<PFN_cuCtxGetId_v12000>(driver_fn("cuCtxGetId"));
        if (gc == nullptr || gi == nullptr) return 0;
        get_cur.store(gc, std::memory_order_release);
        get_id.store(gi, std::memory_order_release);
    }
    CUcontext ctx = nullptr;
    unsigned long long id = 0;
    if (gc(&ctx) != CUDA_SUCCESS || ctx == nullptr || gi(ctx, &id) != CUDA_SUCCESS) return 0;
    return id;
}

// One-time set-up per (device, context): `done[dev]` holds the id of the
// context in which it last ran.
struct OncePerContext {
    std::atomic<unsigned long long> done[kMaxDevices];
    bool is_done(int dev, unsigned long long ctx) const {
        return ctx != 0 && done[dev].load(std::memory_order_acquire) == ctx;
    }
    void mark(int dev) { done[dev].store(current_ctx_id(), std::memory_order_release); }
};

// The current device index, checked against the per-device tables.
inline int current_device(int* dev) {
    cudaError_t e = cudaGetDevice(dev);
    if (e != cudaSuccess) return fail(GAD_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
    if (*dev < 0 || *dev >= kMaxDevices) return fail(GAD_ERR_DEVICE, "device index %d", *dev);
    return GAD_OK;
}

// Raises a kernel's dynamic shared-memory limit once per (device, context).
inline int raise_smem(const void* kern, OncePerContext& once, int bytes) {
    int dev = 0;
    const int ds = current_device(&dev);
    if (ds != GAD_OK) return ds;
    if (!once.is_done(dev, current_ctx_id())) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return fail(GAD_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        once.mark(dev);
    }
    return GAD_OK;
}

inline cudaLaunchAttribute pdl_attr() {
    cudaLaunchAttribute a;
    std::memset(&a, 0, sizeof(a));
    a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a.val.programmaticStreamSerializationAllowed = 1;
    return a;
}

// cuTensorMapEncodeTiled, looked up once through the runtime.
inline int tensor_map_encoder(PFN_cuTensorMapEncodeTiled_v12000* out) {
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> encode{nullptr};
    PFN_cuTensorMapEncodeTiled_v12000 fn = encode.load(std::memory_order_acquire);
    if (fn == nullptr) {
        fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(driver_fn("cuTensorMapEncodeTiled"));
        if (fn == nullptr) return fail(GAD_ERR_CUDA, "cuTensorMapEncodeTiled entry point not found");
        encode.store(fn, std::memory_order_release);
    }
    *out = fn;
    return GAD_OK;
}

}  // namespace gad_host
