// mk_logprobs.cu -- log probabilities of given tokens, entropy and the most
// probable tokens (mk_logprobs).
#include "mk_values.cuh"

namespace {

using namespace mkop;

constexpr int MAX_TOP = 64;

struct LogprobP {
    const uint8_t* logits;
    long long row_s;
    const float* temperature;
    const int* tokens;
    float *logprobs, *entropy, *top_logprobs;
    int* top_ids;
    int V, given, top;
};

constexpr int GT = 512;

template <int DT>
__device__ __forceinline__ float at1(const uint8_t* base, long long i) {
    if constexpr (DT == MK_DT_F32) return reinterpret_cast<const float*>(base)[i];
    else if constexpr (DT == MK_DT_BF16) return bf2f(reinterpret_cast<const uint16_t*>(base)[i]);
    else return __half2float(reinterpret_cast<const __half*>(base)[i]);
}

// A block a row: its maximum, its sums, then the largest tokens one by one.
template <int DT>
__global__ void __launch_bounds__(GT) logprob_rows(const __grid_constant__ LogprobP p) {
    __shared__ float sa[GT / 32], sb[GT / 32];
    __shared__ int si[GT / 32];
    const int r = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint8_t* const x = p.logits + r * p.row_s * (DT == MK_DT_F32 ? 4 : 2);
    float m = -INFINITY;
    bool bad = false;
    for (int i = threadIdx.x; i < p.V; i += GT) {
        const float y = at1<DT>(x, i);
        bad |= !(y < INFINITY);
        m = fmaxf(m, y);
    }
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (lane == 0) sa[warp] = m;
    bad = __syncthreads_or(bad);
    for (int w = 0; w < GT / 32; ++w) m = fmaxf(m, sa[w]);
    const float T = p.temperature ? p.temperature[r] : 1.f;
    bad |= m == -INFINITY || !(T > 0.f);
    const float nan = __uint_as_float(0x7fffffffu);
    auto scaled = [=](float y) { return y == -INFINITY ? y : (y - m) / T; };
    float s1 = 0.f, s2 = 0.f;
    if (!bad)
        for (int i = threadIdx.x; i < p.V; i += GT) {
            const float z = scaled(at1<DT>(x, i)), e = expf(z);
            s1 += e;
            if (e > 0.f) s2 += e * z;
        }
    for (int d = 16; d; d >>= 1) s1 += __shfl_xor_sync(0xffffffffu, s1, d), s2 += __shfl_xor_sync(0xffffffffu, s2, d);
    __syncthreads();
    if (lane == 0) sa[warp] = s1, sb[warp] = s2;
    __syncthreads();
    s1 = s2 = 0.f;
    for (int w = 0; w < GT / 32; ++w) s1 += sa[w], s2 += sb[w];
    const float ls = logf(s1);
    for (int g = threadIdx.x; g < p.given; g += GT) {
        const int id = p.tokens[(long long)r * p.given + g];
        p.logprobs[(long long)r * p.given + g] = bad || (unsigned)id >= (unsigned)p.V ? nan : scaled(at1<DT>(x, id)) - ls;
    }
    if (threadIdx.x == 0 && p.entropy) p.entropy[r] = bad ? nan : ls - s2 / s1;
    float after = INFINITY;  // the last one taken
    int after_i = -1;
    for (int k = 0; k < p.top; ++k) {
        float best = -INFINITY;
        int best_i = INT_MAX;
        if (!bad)
            for (int i = threadIdx.x; i < p.V; i += GT) {
                const float y = at1<DT>(x, i);
                if ((y < after || (y == after && i > after_i)) && (y > best || best_i == INT_MAX)) best = y, best_i = i;
            }
        for (int d = 16; d; d >>= 1) {
            const float y = __shfl_xor_sync(0xffffffffu, best, d);
            const int i = __shfl_xor_sync(0xffffffffu, best_i, d);
            if (i != INT_MAX && (best_i == INT_MAX || y > best || (y == best && i < best_i))) best = y, best_i = i;
        }
        __syncthreads();
        if (lane == 0) sa[warp] = best, si[warp] = best_i;
        __syncthreads();
        for (int w = 0; w < GT / 32; ++w)
            if (si[w] != INT_MAX && (best_i == INT_MAX || sa[w] > best || (sa[w] == best && si[w] < best_i))) best = sa[w], best_i = si[w];
        after = best, after_i = best_i;
        if (threadIdx.x == 0) {
            p.top_ids[(long long)r * p.top + k] = bad ? -1 : best_i;
            p.top_logprobs[(long long)r * p.top + k] = bad ? nan : scaled(best) - ls;
        }
    }
}

}  // namespace

extern "C" int mk_logprobs(const mk_logprob* a, void* stream) {
    if (!a) return fail(MK_ERR_INVALID_ARG, "logprobs: NULL arguments");
    const int e = dtype_bytes(a->dtype);
    if (!e) return fail(MK_ERR_INVALID_ARG, "logprobs: unknown dtype %d", a->dtype);
    if (a->rows < 0 || a->vocab < 1 || a->given < 0 || a->top < 0 || a->row_stride < 0)
        return fail(MK_ERR_INVALID_ARG, "logprobs: rows, given, top or row_stride negative, or vocab below 1");
    if (a->top > a->vocab) return fail(MK_ERR_INVALID_ARG, "logprobs: top %d of a vocabulary of %d", a->top, a->vocab);
    if (a->top > MAX_TOP) return fail(MK_ERR_UNSUPPORTED, "logprobs: top above %d", MAX_TOP);
    if (!a->logits || (a->given && (!a->tokens || !a->logprobs)) || (a->top && (!a->top_ids || !a->top_logprobs)))
        return fail(MK_ERR_INVALID_ARG, "logprobs: logits, tokens, logprobs, top_ids or top_logprobs is NULL");
    if ((uintptr_t)a->logits % e) return fail(MK_ERR_INVALID_ARG, "logprobs: logits not aligned to their type");
    if (off_by4(a->temperature, a->tokens, a->logprobs, a->entropy, a->top_ids, a->top_logprobs))
        return fail(MK_ERR_INVALID_ARG, "logprobs: an argument is not aligned to 4 bytes");
    if (a->rows == 0) return MK_OK;
    LogprobP p = {};
    p.logits = (const uint8_t*)a->logits, p.row_s = a->row_stride, p.temperature = a->temperature, p.tokens = a->tokens;
    p.logprobs = a->logprobs, p.entropy = a->entropy, p.top_ids = a->top_ids, p.top_logprobs = a->top_logprobs;
    p.V = a->vocab, p.given = a->given, p.top = a->top;
    cudaStream_t s = (cudaStream_t)stream;
    if (a->dtype == MK_DT_F32) logprob_rows<MK_DT_F32><<<a->rows, GT, 0, s>>>(p);
    else if (a->dtype == MK_DT_BF16) logprob_rows<MK_DT_BF16><<<a->rows, GT, 0, s>>>(p);
    else logprob_rows<MK_DT_F16><<<a->rows, GT, 0, s>>>(p);
    return cuda_status(cudaGetLastError(), "mk_logprobs");
}
