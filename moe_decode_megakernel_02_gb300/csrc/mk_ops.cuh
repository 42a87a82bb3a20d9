// mk_ops.cuh -- what the operators on paged caches and logits share: host
// checks and small device helpers.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "../../include/mk.h"

// the library's thread-local message, its wait limit (MK_WAIT_NS) and injected failures (MK_FAULT), of mk_host.cu
extern "C" __attribute__((visibility("hidden"))) int mk_set_error_(int code, const char* msg);
extern "C" __attribute__((visibility("hidden"))) long long mk_wait_ns_(void);
extern "C" __attribute__((visibility("hidden"))) int mk_fault_(const char* what);

namespace mkop {

inline int fail(int code, const char* fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return mk_set_error_(code, buf);
}
inline int cuda_status(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return MK_OK;
    return fail(e == cudaErrorMemoryAllocation ? MK_ERR_OOM : MK_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}
// the current device and how many SMs it has, asked for once each
inline int device_sms(int& dev, int& sms, const char* what) {
    static std::atomic<int> known[64];
    cudaError_t e = cudaGetDevice(&dev);
    sms = e == cudaSuccess && dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (e == cudaSuccess && !sms) {
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess && dev < 64) known[dev].store(sms, std::memory_order_relaxed);
    }
    return cuda_status(e, what);
}
// Dynamic shared memory a kernel is allowed, set once on each device. `done`: a bit a device, one word a kernel.
template <typename K>
inline int allow_smem(K* kern, int bytes, int dev, std::atomic<uint64_t>& done, const char* what) {
    if (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1)) return MK_OK;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_release);
    return cuda_status(e, what);
}
inline int dtype_bytes(int dt) { return dt == MK_DT_F32 ? 4 : (dt == MK_DT_BF16 || dt == MK_DT_F16) ? 2 : 0; }
inline int code_bytes(int format) { return format == MK_KV_BF16 ? 2 : 1; }
inline int log2_exact(int n) { return n > 0 && (n & (n - 1)) == 0 ? __builtin_ctz((unsigned)n) : -1; }

// whether any of some pointers to 32-bit values is off its alignment
template <typename... P>
inline bool off_by4(const P*... p) {
    return ((((uintptr_t)p % 4) | ...)) != 0;
}

// what every operator on pages asks of its cache and table
int check_pages(const mk_pages* p, const mk_page_table* t);
int check_latent(const mk_latent_pages* p, const mk_page_table* t);
int check_rows(const mk_rows* r, const char* what, const char* name);
// whether rows can be read 16 bytes at a time
bool rows_vec(const mk_rows* r);

__device__ __forceinline__ float bf2f(uint32_t h) { return __uint_as_float(h << 16); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

}  // namespace mkop
