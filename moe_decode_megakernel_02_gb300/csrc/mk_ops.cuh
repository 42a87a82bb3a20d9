// mk_ops.cuh -- what the operators on paged caches and logits share: host
// checks and small device helpers.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

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
