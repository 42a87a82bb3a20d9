// mk_logprobs.cu -- log probabilities of given tokens, entropy and the most
// probable tokens (mk_logprobs).
//
// One pass over a row's logits x, a cluster of 1 to 8 CTAs a row. With z =
// (x - m) / T, m the largest logit so far, a thread keeps
//   s = sum e^z,  t = sum e^z z    (when m rises by d T: s' = e^-d s, t' = e^-d (t - d s)),
// and at the end log p_i = z_i - log s, entropy = log s - t / s.
//
// The most probable tokens come out of the same pass. Tokens are ordered by one
// 64-bit key (logit, then the lower id). A round is 16 values a thread; before a
// CTA has a threshold, the largest keys of 128 groups of four threads give one
// (the k-th largest of them is no more than the k-th largest of all), after that
// a round whose values all lie below it costs one vote. What lies above goes to
// a list, whose first k are found by counting, for each, how many are larger.
// Ids rise from round to round, so that an equal logit of a later round never
// counts.
//
// Bound by HBM for batches (some 7 instructions a value), by latency for single
// rows: a trip to memory, three votes, the cluster's meeting.
#include <type_traits>

#include "mk_tensor.cuh"
#include "mk_values.cuh"

namespace {

using namespace mkop;
typedef unsigned long long u64;

constexpr int MAX_TOP = 64;
constexpr int GT = 512, BATCH = 16;       // threads, values of a thread's round
constexpr int GROUPS = GT / 4;
// the list: what may be left of it, and what a round may add (k groups of four threads)
constexpr int KEEP = 256, CAP = KEEP + MAX_TOP * 4 * BATCH;
constexpr int MAX_CLUSTER = 8;

struct LogprobP {
    const uint8_t* logits;
    long long row_s;
    const float* temperature;
    const int* tokens;
    float *logprobs, *entropy, *top_logprobs;
    int* top_ids;
    int V, given, top, split;  // split: CTAs of a row
};

struct LogprobShared {
    u64 list[CAP];
    u64 best[MAX_TOP];  // sorted
    u64 group[GROUPS];
    u64 merge[MAX_CLUSTER * MAX_TOP];
    float4 part[GT / 32];  // (m, s, t, -) of the warps
    float4 cta[MAX_CLUSTER];
    int n;
    u64 limit;
};

template <int DT>
__device__ __forceinline__ float at1(const uint8_t* base, long long i) {
    if constexpr (DT == MK_DT_F32) return reinterpret_cast<const float*>(base)[i];
    else if constexpr (DT == MK_DT_BF16) return bf2f(reinterpret_cast<const uint16_t*>(base)[i]);
    else return __half2float(reinterpret_cast<const __half*>(base)[i]);
}
// larger keys first: larger logits, then lower ids (no key is 0)
__device__ __forceinline__ u64 key_of(float x, int id) {
    const uint32_t u = __float_as_uint(x + 0.f);  // (-0 is 0)
    return (u64)(u & 0x80000000u ? ~u : u | 0x80000000u) << 32 | (uint32_t)~id;
}
__device__ __forceinline__ float logit_of(u64 key) {
    const uint32_t u = (uint32_t)(key >> 32);
    return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// (m, s, t) of two parts; c: exponents of 2 a unit of logits
__device__ __forceinline__ void join(float& m, float& s, float& t, float m2, float s2, float t2, float c) {
    const float mn = max_nan(m, m2);
    // a part without an unmasked logit has sums of 0
    const float d = m == -INFINITY ? 0.f : (m - mn) * c, e = m2 == -INFINITY ? 0.f : (m2 - mn) * c;
    const float f = ex2(d), g = ex2(e);
    // (a sum whose weights vanish: its t, 0 times a large d, vanishes too)
    t = f * t + (f > 0.f ? f * d * s : 0.f) + g * t2 + (g > 0.f ? g * e * s2 : 0.f);
    s = f * s + g * s2;
    m = mn;
}

// The first k keys of `n` in sh.list, sorted, to sh.best; returns how many there are.
__device__ int first_keys(LogprobShared& sh, int n, int k) {
    const int tid = threadIdx.x;
    // long lists (adverse orders) are cut by a threshold of theirs first
    while (n > GT) {
        u64 mine[(CAP + GT - 1) / GT], top = 0;
#pragma unroll
        for (int i = 0; i < (CAP + GT - 1) / GT; ++i) {
            mine[i] = i * GT + tid < n ? sh.list[i * GT + tid] : 0;
            top = max(top, mine[i]);
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        if ((tid & 3) == 0) sh.group[tid >> 2] = top;
        __syncthreads();
        if (tid < GROUPS) {
            const u64 x = sh.group[tid];
            int rank = 0;
            for (int i = 0; i < GROUPS; ++i) rank += sh.group[i] > x;
            if (rank == k - 1) sh.limit = x;
        }
        if (tid == 0) sh.n = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < (CAP + GT - 1) / GT; ++i)
            if (mine[i] >= sh.limit) sh.list[atomicAdd(&sh.n, 1)] = mine[i];
        __syncthreads();
        const int left = sh.n;
        __syncthreads();
        if (left == n) break;  // (then nothing is cut any more)
        n = left;
    }
    for (int i = tid; i < n; i += GT) {
        const u64 x = sh.list[i];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) rank += sh.list[j] > x;
        if (rank < k) sh.best[rank] = x;
    }
    __syncthreads();
    return min(n, k);
}

// to the same place in another CTA of the cluster
__device__ __forceinline__ void put_remote(u64* p, int cta, u64 v) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(sm32(p)), "r"(cta));
    asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ void put_remote(float4* p, int cta, float4 v) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(sm32(p)), "r"(cta));
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

template <int DT, bool TOP>
__global__ void __launch_bounds__(GT, 2) logprob_kernel(const __grid_constant__ LogprobP p) {
    constexpr int VEC = DT == MK_DT_F32 ? 4 : 8, U = BATCH / VEC;  // values of 16 bytes, words of a round
    __shared__ LogprobShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, split = p.split;
    const int r = blockIdx.x / split, part = blockIdx.x - r * split;
    const uint8_t* const x = p.logits + (long long)r * p.row_s * (DT == MK_DT_F32 ? 4 : 2);
    // the CTA's values: whole 16-byte words, the row's unaligned ends with the first and the last part
    const int head = min(p.V, (int)((16 - ((uintptr_t)x & 15)) & 15) / (DT == MK_DT_F32 ? 4 : 2));
    const int words = (p.V - head) / VEC, tail = p.V - head - words * VEC;
    const int w0 = (int)((long long)words * part / split), w1 = (int)((long long)words * (part + 1) / split);
    const float T = p.temperature ? p.temperature[r] : 1.f;
    const bool cold = !(T > 0.f);
    const float c = cold ? 0.f : fminf(LOG2E / T, 1e38f);
    const int k = p.top;
    if (TOP && tid == 0) sh.n = 0;

    float m = -INFINITY, s = 0.f, t = 0.f, tt[2] = {0.f, 0.f};  // (t's parts since m last rose)
    bool have = false;  // k keys have been found
    u64 limit = 0;  // a key that the k-th largest one is not below; 0: none yet
    float limit_x = -INFINITY;
    int n = 0;      // of the list
    if (TOP) __syncthreads();

    // N values a thread, ids from `id` in words of VEC that lie GT words apart; `in`: this thread has them
    auto round = [&](auto COUNT, const float (&v)[BATCH], int id, bool in) {
        constexpr int N = decltype(COUNT)::value;
        auto id_of = [&](int i) { return id + i / VEC * GT * VEC + i % VEC; };
        float top = -INFINITY;
        if (in) {
            top = v[0];
#pragma unroll
            for (int i = 1; i < N; ++i) top = max_nan(top, v[i]);
            const float mn = max_nan(m, top);
            if (!(mn == m)) {
                if (m != -INFINITY) {
                    const float d = (m - mn) * c, f = ex2(d);
                    t = f > 0.f ? f * (t + (tt[0] + tt[1]) + d * s) : 0.f;
                    tt[0] = tt[1] = 0.f;
                    s *= f;
                }
                m = mn;
            }
            const float less = m == -INFINITY ? 0.f : -m;
            float sum[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                float a = v[i], b = i + 1 < N ? v[i + 1] : -INFINITY;
                add2(a, b, less, less);
                fma2(a, b, a, b, c, c, 0.f, 0.f);
                // (below 2^-150 a weight is 0; a masked logit times an infinite temperature's 0 is no number, and so too)
                a = fmaxf(a, -150.f), b = fmaxf(b, -150.f);
                const float e = ex2(a), g = ex2(b);
                add2(sum[0], sum[1], e, g);
                fma2(tt[0], tt[1], e, g, a, b, tt[0], tt[1]);
            }
            s += sum[0] + sum[1];
        }
        if constexpr (TOP) {
            const int some = __syncthreads_count(in && (!limit || top > limit_x));
            if (!some) return;
            if (some > k) {
                // a threshold from the groups' largest keys
                u64 best = 0;
                if (in) {
#pragma unroll
                    for (int i = 0; i < N; ++i) best = max(best, key_of(v[i], id_of(i)));
                }
                best = max(best, __shfl_xor_sync(0xffffffffu, best, 1));
                best = max(best, __shfl_xor_sync(0xffffffffu, best, 2));
                if ((lane & 3) == 0) sh.group[tid >> 2] = best;
                if (tid == 0) sh.limit = 0;
                __syncthreads();
                if (tid < GROUPS) {
                    const u64 y = sh.group[tid];
                    int rank = 0;
#pragma unroll 8
                    for (int i = 0; i < GROUPS; ++i) rank += sh.group[i] > y;
                    if (rank == k - 1 && y) sh.limit = y;
                }
                __syncthreads();
                limit = max(limit, sh.limit);  // (keys from it on)
            }
            if (in && (!limit || top >= logit_of(limit))) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const u64 y = key_of(v[i], id_of(i));
                    if (y >= limit) sh.list[atomicAdd(&sh.n, 1)] = y;
                }
            }
            __syncthreads();
            n = sh.n;
            __syncthreads();
            if (n > KEEP || (!have && n >= k)) {
                n = first_keys(sh, n, k);
                if (tid < n) sh.list[tid] = sh.best[tid];
                if (tid == 0) sh.n = n;
                __syncthreads();
                have = true;
            }
            if (have) {
                limit = max(limit, sh.best[k - 1]);
                limit_x = logit_of(limit);
            }
        }
    };
    auto single = [&](int id, bool in) {
        float v[BATCH];
        v[0] = in ? at1<DT>(x, id) : 0.f;
        round(std::integral_constant<int, 1>(), v, id, in);
    };
    if (part == 0 && head) single(tid, tid < head);
    {
        const int id0 = head + w0 * VEC, all = w1 - w0;
        const uint4* const q = reinterpret_cast<const uint4*>(x + (long long)id0 * (DT == MK_DT_F32 ? 4 : 2));
        uint4 next[U];
        auto load = [&](int w) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (w + u * GT < all) next[u] = __ldcs(q + w + u * GT);
        };
#pragma unroll
        for (int u = 0; u < U; ++u) next[u] = make_uint4(0, 0, 0, 0);
        load(tid);
        for (int w = 0; w < all; w += U * GT) {
            float v[BATCH];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t y[4] = {next[u].x, next[u].y, next[u].z, next[u].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (DT == MK_DT_F32) {
                        v[4 * u + i] = __uint_as_float(y[i]);
                    } else if constexpr (DT == MK_DT_BF16) {
                        v[8 * u + 2 * i] = __uint_as_float(y[i] << 16);
                        v[8 * u + 2 * i + 1] = __uint_as_float(y[i] & 0xffff0000u);
                    } else {
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&y[i]));
                        v[8 * u + 2 * i] = f.x, v[8 * u + 2 * i + 1] = f.y;
                    }
                }
            }
            load(w + U * GT + tid);
            if (w + U * GT <= all) {
                round(std::integral_constant<int, BATCH>(), v, id0 + (w + tid) * VEC, true);
            } else {  // the last round, word by word
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (w + u * GT >= all) break;
                    float y[BATCH];
#pragma unroll
                    for (int i = 0; i < VEC; ++i) y[i] = v[u * VEC + i];
                    round(std::integral_constant<int, VEC>(), y, id0 + (w + u * GT + tid) * VEC, w + u * GT + tid < all);
                }
            }
        }
    }
    if (part == split - 1 && tail) single(p.V - tail + tid, tid < tail);

    // ---- the CTA's part, to the row's first CTA
    t += tt[0] + tt[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o),
                    t2 = __shfl_xor_sync(0xffffffffu, t, o);
        join(m, s, t, m2, s2, t2, c);
    }
    if (lane == 0) sh.part[warp] = make_float4(m, s, t, 0.f);
    int found = 0;
    if (TOP) found = first_keys(sh, n, k);  // (and a barrier)
    else __syncthreads();
    m = -INFINITY, s = t = 0.f;
    for (int w = 0; w < GT / 32; ++w) join(m, s, t, sh.part[w].x, sh.part[w].y, sh.part[w].z, c);
    if (split > 1) {
        asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");  // all have begun
        if (tid == 0) put_remote(&sh.cta[part], 0, make_float4(m, s, t, 0.f));
        if (TOP && tid < k) put_remote(&sh.merge[part * k + tid], 0, tid < found ? sh.best[tid] : 0);
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (part) return;
        m = -INFINITY, s = t = 0.f;
        for (int i = 0; i < split; ++i) join(m, s, t, sh.cta[i].x, sh.cta[i].y, sh.cta[i].z, c);
        if (TOP) {
            for (int i = tid; i < split * k; i += GT) {
                const u64 y = sh.merge[i];
                int rank = 0;
#pragma unroll 4
                for (int j = 0; j < split * k; ++j) rank += sh.merge[j] > y;
                if (rank < k && y) sh.best[rank] = y;
            }
            __syncthreads();
        }
    }
    const float nan = __uint_as_float(0x7fffffffu), ls = logf(s);
    const bool bad = cold || !(m < INFINITY) || m == -INFINITY;
    auto logp = [&](float y) { return bad ? nan : y == -INFINITY ? y : (y - m) / T - ls; };
    if (tid == 0 && p.entropy) p.entropy[r] = bad ? nan : ls - t / s * LN2;
    for (int g = tid; g < p.given; g += GT) {
        const int id = p.tokens[(long long)r * p.given + g];
        p.logprobs[(long long)r * p.given + g] = (unsigned)id < (unsigned)p.V ? logp(at1<DT>(x, id)) : nan;
    }
    if (TOP && tid < k) {
        const u64 y = sh.best[tid];
        p.top_ids[(long long)r * k + tid] = bad ? -1 : (int)~(uint32_t)y;
        p.top_logprobs[(long long)r * k + tid] = logp(logit_of(y));
    }
}

template <int DT>
int run(const LogprobP& p, int rows, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * p.split));
    cfg.blockDim = dim3(GT);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = p.split;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = p.split > 1;
    return cuda_status(p.top ? cudaLaunchKernelEx(&cfg, logprob_kernel<DT, true>, p) : cudaLaunchKernelEx(&cfg, logprob_kernel<DT, false>, p),
                       "mk_logprobs");
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
    if ((int64_t)a->rows * MAX_CLUSTER > INT32_MAX) return fail(MK_ERR_UNSUPPORTED, "logprobs: too many rows in one call");
    int dev = 0, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess) return cuda_status(err, "mk_logprobs");
    LogprobP p = {};
    p.logits = (const uint8_t*)a->logits, p.row_s = a->row_stride, p.temperature = a->temperature, p.tokens = a->tokens;
    p.logprobs = a->logprobs, p.entropy = a->entropy, p.top_ids = a->top_ids, p.top_logprobs = a->top_logprobs;
    p.V = a->vocab, p.given = a->given, p.top = a->top;
    // CTAs of a row: two or more an SM, as long as each has a part of a round
    p.split = 1;
    while (p.split < MAX_CLUSTER && (int64_t)a->rows * p.split < 2 * sms && a->vocab / p.split > GT * BATCH / 4) p.split *= 2;
    cudaStream_t s = (cudaStream_t)stream;
    if (a->dtype == MK_DT_F32) return run<MK_DT_F32>(p, a->rows, s);
    return a->dtype == MK_DT_BF16 ? run<MK_DT_BF16>(p, a->rows, s) : run<MK_DT_F16>(p, a->rows, s);
}
