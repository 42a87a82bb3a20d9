// mk_logprobs.cu -- log probabilities of given tokens, entropy and the most
// probable tokens (mk_logprobs).
//
// One pass over a row's logits x, a cluster of 1 to 8 CTAs a row. With z =
// (x - m) / T, m the largest logit so far, a thread keeps
//   s = sum e^z,  t = sum e^z z    (when m rises by d T: s' = e^-d s, t' = e^-d (t - d s)),
// and at the end log p_i = z_i - log s, entropy = log s - t / s.
//
// The most probable tokens come out of the same pass. Tokens are ordered by one
// 64-bit key (logit, then the lower id). A round is 64 bytes a thread; before a
// CTA has a threshold, the largest keys of groups of threads give one
// (the k-th largest of them is no more than the k-th largest of all), after that
// a round whose values all lie below it costs one vote. What lies above goes to
// a list, whose first k are found by counting, for each, how many are larger.
// Ids rise from round to round, so that an equal logit of a later round never
// counts.
//
// 256 rows of 151936 bf16 logits take 19 us without alternatives (60 % of a copy's
// rate): a row a CTA leaves 104 of 152 SMs two rows and 48 one, and 11 instructions a
// value are 10.6 us of all SMs' issue slots, as long as the copy. With 20 alternatives
// 41: 18 instructions a value are 17.4 us; the rest is each round's barrier, at which
// all warps meet also where nothing qualifies, and the list's cuts. Single rows are
// bound by latency, a trip to memory, the threshold's and the ranks' votes, the
// cluster's meeting: 32000 fp32 logits 7.5 us.
#include <climits>
#include <type_traits>

#include "mk_tensor.cuh"
#include "mk_values.cuh"

namespace {

using namespace mkop;
typedef unsigned long long u64;

constexpr int MAX_TOP = 64;
constexpr int GT = 512, U = 4;            // threads, 16-byte words of a thread's round
constexpr int GROUPS = GT / 2;            // of two threads; up to k = 32 half as many, of four
// the list: what may be left of it, and what a round may add (the values of k groups, or of as many threads)
constexpr int SLACK = 8, CAP = MAX_TOP + SLACK + MAX_TOP * 2 * U * 8;
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

template <bool TOP>
struct LogprobShared {
    u64 list[TOP ? CAP : 1];
    u64 best[TOP ? MAX_TOP : 1];  // sorted
    u64 group[TOP ? GROUPS : 1];
    u64 merge[TOP ? MAX_CLUSTER * MAX_TOP : 1];
    float4 part[GT / 32];  // Part of the warps
    float4 cta[MAX_CLUSTER], mine;
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

// the larger of two pairs of 16-bit values, each; no number stays none
template <int DT>
__device__ __forceinline__ uint32_t larger_pair(uint32_t a, uint32_t b) {
    uint32_t y;
    if constexpr (DT == MK_DT_BF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}

// the values of a 16-byte word, and their largest
template <int DT, int N>
__device__ __forceinline__ void unpack(const uint4& z, float (&v)[N]) {
    const uint32_t y[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == MK_DT_F32) {
            v[i] = __uint_as_float(y[i]);
        } else if constexpr (DT == MK_DT_BF16) {
            v[2 * i] = __uint_as_float(y[i] << 16);
            v[2 * i + 1] = __uint_as_float(y[i] & 0xffff0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&y[i]));
            v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
    }
}
template <int DT>
__device__ __forceinline__ float largest(const uint4& z) {
    if constexpr (DT == MK_DT_F32) {
        return max_nan(max_nan(__uint_as_float(z.x), __uint_as_float(z.y)), max_nan(__uint_as_float(z.z), __uint_as_float(z.w)));
    } else {
        const uint32_t y = larger_pair<DT>(larger_pair<DT>(z.x, z.y), larger_pair<DT>(z.z, z.w));
        float v[8];
        unpack<DT>(make_uint4(y, y, y, y), v);
        return max_nan(v[0], v[1]);
    }
}

// Half of x - y: the difference may be beyond the range of 32 bits, where a temperature brings it back.
__device__ __forceinline__ float half_of(float x, float y) { return __fmaf_rn(x, 0.5f, -0.5f * y); }

// Sums of a part of the row, against its largest logit (in exponents of 2, c two units of logits).
struct Part {
    float m, s, t;
};
__device__ __forceinline__ Part join(const Part& x, const Part& y, float c) {
    const bool swap = y.m > x.m;
    const Part a = swap ? y : x, b = swap ? x : y;
    // a part without an unmasked logit has sums of 0; one that vanishes against the other adds nothing
    const float d = b.m == -INFINITY ? 0.f : half_of(b.m, a.m) * c, f = ex2(d);
    return {max_nan(a.m, b.m), a.s + f * b.s, a.t + (f > 0.f ? f * (b.t + d * b.s) : 0.f)};
}

// Ranks of up to 32 M keys (how many are larger): a warp holds all of them, M a lane, and ranks its share by votes.
// found(key, rank) runs in one lane for each key.
template <int M, typename F>
__device__ __forceinline__ void ranks(const u64* keys, int n, F found) {
    constexpr int EACH = 32 * M / (GT / 32);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp * EACH >= n) return;
    u64 mine[M];
#pragma unroll
    for (int i = 0; i < M; ++i) mine[i] = i * 32 + lane < n ? keys[i * 32 + lane] : 0;
#pragma unroll
    for (int g = 0; g < EACH; ++g) {
        const int at = warp * EACH + g;
        const u64 x = at < n ? keys[at] : 0;
        int rank = 0;
#pragma unroll
        for (int i = 0; i < M; ++i) rank += __popc(__ballot_sync(0xffffffffu, mine[i] > x));
        if (lane == 0 && x) found(x, rank);
    }
}

// The first k keys of `n` in sh.list, sorted, to sh.best; returns how many there are.
template <typename S>
__device__ int first_keys(S& sh, int n, int k) {
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
        if ((tid & 1) == 0) sh.group[tid >> 1] = top;
        __syncthreads();
        ranks<8>(sh.group, GROUPS, [&](u64 x, int rank) {
            if (rank == k - 1) sh.limit = x;
        });
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
    if (n <= 32) {
        ranks<1>(sh.list, n, [&](u64 x, int rank) {
            if (rank < k) sh.best[rank] = x;
        });
    } else if (n <= 128) {
        ranks<4>(sh.list, n, [&](u64 x, int rank) {
            if (rank < k) sh.best[rank] = x;
        });
    } else {
        for (int i = tid; i < n; i += GT) {
            const u64 x = sh.list[i];
            int rank = 0;
#pragma unroll 4
            for (int j = 0; j < n; ++j) rank += sh.list[j] > x;
            if (rank < k) sh.best[rank] = x;
        }
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
    constexpr int VEC = DT == MK_DT_F32 ? 4 : 8;  // values of 16 bytes
    __shared__ LogprobShared<TOP> sh;
    extern __shared__ __align__(16) uint8_t ring[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, split = p.split;
    const int r = blockIdx.x / split, part = blockIdx.x - r * split;
    const uint8_t* const x = p.logits + (long long)r * p.row_s * (DT == MK_DT_F32 ? 4 : 2);
    // the CTA's values: whole 16-byte words, the row's unaligned ends with the first and the last part
    const int head = min(p.V, (int)((16 - ((uintptr_t)x & 15)) & 15) / (DT == MK_DT_F32 ? 4 : 2));
    const int words = (p.V - head) / VEC, tail = p.V - head - words * VEC;
    const int w0 = (int)((long long)words * part / split), w1 = (int)((long long)words * (part + 1) / split);
    const float T = p.temperature ? p.temperature[r] : 1.f;
    const bool cold = !(T > 0x1p-120f);
    const float c = cold ? 0.f : 2.f * (LOG2E / T);  // (times half a difference)
    const int k = p.top;
    if (TOP && tid == 0) sh.n = 0;

    // the sums of e = 2^(c (x - m) / 2) and of e c (x - m) / 2, of two lines of values whose arithmetic is paired (two values an
    // instruction; without pairs 256 rows of 151936 bf16 logits take 3 % longer)
    float m = -INFINITY, half_m = m, s[2] = {0.f, 0.f}, t[2] = {0.f, 0.f};
    auto rise = [&](float top) {
        if (m != -INFINITY) {
            const float d = half_of(m, top) * c, f = ex2(d);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                t[i] = f > 0.f ? f * (t[i] + d * s[i]) : 0.f;
                s[i] *= f;
            }
        }
        m = max_nan(m, top);  // (no number stays one)
        half_m = 0.5f * m;
    };
    bool have = false, sorted = false;  // k keys have been found; and nothing since
    u64 limit = 0;  // a key that the k-th largest one is not below; 0: none yet
    float limit_x = -INFINITY;
    int n = 0;      // of the list
    if (TOP) __syncthreads();

    auto add = [&](float x, float y) {
        float z0, z1, e0, e1;
        fma2(z0, z1, x, y, 0.5f, 0.5f, -half_m, -half_m);
        fma2(z0, z1, z0, z1, c, c, 0.f, 0.f);
        // (below 2^-150 a weight is 0; a masked logit times an infinite temperature's 0 is no number, and so too)
        z0 = fmaxf(z0, -150.f), z1 = fmaxf(z1, -150.f);
        e0 = ex2(z0), e1 = ex2(z1);
        add2(s[0], s[1], e0, e1);
        fma2(t[0], t[1], e0, e1, z0, z1, t[0], t[1]);
    };
    // A round's most probable tokens: `top` is this thread's largest logit of the round (`in`: it has any), each(least, f)
    // calls f(logit, id) for all of them, or at least those from `least` on.
    auto pick = [&](float top, bool in, auto each) {
        const int some = __syncthreads_count(in && (!limit || top > limit_x));
        if (!some) return;
        // (the values of 2 MAX_TOP threads find room in the list)
        if (some > (limit ? max(2 * k, 64) : k)) {
            // A threshold from the groups' largest keys, which must differ, or none has rank k - 1 and all values would go to
            // the list: a largest logit that is no number equals none of them, and takes the thread's number for its id.
            int first = INT_MAX;
            each(top, [&](float x, int id) {
                if (x == top) first = min(first, id);
            });
            u64 best = in ? key_of(top, first == INT_MAX ? tid : first) : 0;
            best = max(best, __shfl_xor_sync(0xffffffffu, best, 1));
            if (k <= 32) best = max(best, __shfl_xor_sync(0xffffffffu, best, 2));
            const int by = k <= 32 ? 2 : 1;
            if ((lane & ((1 << by) - 1)) == 0) sh.group[tid >> by] = best;
            if (tid == 0) sh.limit = 0;
            __syncthreads();
            auto found = [&](u64 x, int rank) {
                if (rank == k - 1) sh.limit = x;
            };
            if (k <= 32) ranks<4>(sh.group, GROUPS / 2, found);
            else ranks<8>(sh.group, GROUPS, found);
            __syncthreads();
            limit = max(limit, sh.limit);  // (keys from it on)
        }
        const float least = limit ? logit_of(limit) : -INFINITY;
        if (in && top >= least)
            each(least, [&](float x, int id) {
                if (x >= least) {
                    const u64 y = key_of(x, id);
                    if (y >= limit) sh.list[atomicAdd(&sh.n, 1)] = y;
                }
            });
        __syncthreads();
        n = sh.n;  // (what is written to it or the list from here on is behind another barrier)
        sorted = false;
        // (a threshold that follows closely spares the next rounds more than it costs)
        if (n > k + SLACK || (!have && n >= k)) {
            n = first_keys(sh, n, k);
            if (tid < n) sh.list[tid] = sh.best[tid];
            if (tid == 0) sh.n = n;  // (read behind the next round's barrier)
            have = sorted = true;
        }
        if (have) {
            limit = max(limit, sh.best[k - 1]);
            limit_x = logit_of(limit);
        }
    };
    auto single = [&](int id, bool in) {
        const float x0 = in ? at1<DT>(x, id) : -INFINITY;
        if (in) {
            if (!(x0 <= m)) rise(x0);
            add(x0, -INFINITY);
        }
        if constexpr (TOP)
            pick(x0, in, [&](float, auto f) {
                if (in) f(x0, id);
            });
    };
    if (part == 0 && head) single(tid, tid < head);
    {
        const int id0 = head + w0 * VEC, all = w1 - w0;
        // a thread's own words come through its own places in shared memory, a round ahead
        constexpr int STAGE_B = U * GT * 16;
        const uint32_t mine = sm32(ring) + tid * 16;
        const uint8_t* src = x + (long long)id0 * (DT == MK_DT_F32 ? 4 : 2) + tid * 16;
        int ahead = all - tid;  // words from the next one to ask for on (every GT-th is this thread's)
        auto load = [&](uint32_t to) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (ahead > u * GT) cp16(to + u * GT * 16, src + u * GT * 16, true);
            src += STAGE_B;
            ahead -= U * GT;
            cp_commit();
        };
        load(mine);
        uint32_t stage = 0;
        for (int left = all - tid, id = id0 + tid * VEC; left > -tid; left -= U * GT, id += U * GT * VEC) {
            load(mine + (stage ^ STAGE_B));
            cp_wait<1>();
            const uint8_t* const words = ring + stage + tid * 16;
            float top = -INFINITY;
            auto word = [&](int u) {
                const uint4 z = *reinterpret_cast<const uint4*>(words + u * GT * 16);
                const float mx = largest<DT>(z);
                if (!(mx <= m)) rise(mx);
                top = max_nan(top, mx);
                float y[VEC];
                unpack<DT>(z, y);
#pragma unroll
                for (int e = 0; e < VEC; e += 2) add(y[e], y[e + 1]);
            };
            if (left > (U - 1) * GT) {
#pragma unroll
                for (int u = 0; u < U; ++u) word(u);
            } else {
#pragma unroll 1
                for (int u = 0; u < U && left > u * GT; ++u) word(u);
            }
            if constexpr (TOP)
                pick(top, left > 0, [&](float least, auto f) {
#pragma unroll 1
                    for (int u = 0; u < U && left > u * GT; ++u) {
                        const uint4 z = *reinterpret_cast<const uint4*>(words + u * GT * 16);
                        if (!(largest<DT>(z) >= least)) continue;
                        float y[VEC];
                        unpack<DT>(z, y);
#pragma unroll
                        for (int e = 0; e < VEC; ++e) f(y[e], id + u * GT * VEC + e);
                    }
                });
            stage ^= STAGE_B;
        }
    }
    if (part == split - 1 && tail) single(p.V - tail + tid, tid < tail);

    // ---- the CTA's part, to the row's first CTA
    auto meet = [&](Part a, int lanes) {  // over the first lanes of a warp
        for (int o = 1; o < lanes; o <<= 1)
            a = join(a, Part{__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o),
                             __shfl_xor_sync(0xffffffffu, a.t, o)}, c);
        return a;
    };
    Part all = meet(Part{m, s[0] + s[1], t[0] + t[1]}, 32);
    if (lane == 0) sh.part[warp] = make_float4(all.m, all.s, all.t, 0.f);
    int found = k;
    if constexpr (TOP) {
        if (!sorted) found = first_keys(sh, n, k);
    }
    __syncthreads();
    if (warp == 0) {
        const float4 y = sh.part[lane & (GT / 32 - 1)];
        all = meet(Part{y.x, y.y, y.z}, GT / 32);
        if (lane == 0) {
            if (split > 1) sh.mine = make_float4(all.m, all.s, all.t, 0.f);
            else sh.cta[0] = make_float4(all.m, all.s, all.t, 0.f);
        }
    }
    if (split > 1) {
        asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");  // all have begun
        if (tid == 0) put_remote(&sh.cta[part], 0, sh.mine);
        if constexpr (TOP) {
            if (tid < k) put_remote(&sh.merge[part * k + tid], 0, tid < found ? sh.best[tid] : 0);
        }
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (part) return;
        if constexpr (TOP) {
            for (int i = tid; i < split * k; i += GT) {
                const u64 y = sh.merge[i];
                int rank = 0;
#pragma unroll 4
                for (int j = 0; j < split * k; ++j) rank += sh.merge[j] > y;
                if (rank < k && y) sh.best[rank] = y;
            }
        }
    }
    __syncthreads();
    all = {-INFINITY, 0.f, 0.f};
    for (int i = 0; i < split; ++i) all = join(all, Part{sh.cta[i].x, sh.cta[i].y, sh.cta[i].z}, c);
    m = all.m;
    const float nan = __uint_as_float(0x7fffffffu), ls = logf(all.s);
    const bool bad = cold || !(m < INFINITY) || m == -INFINITY;
    auto logp = [&](float y) { return bad ? nan : y == -INFINITY ? y : half_of(y, m) / T * 2.f - ls; };
    if (tid == 0 && p.entropy) p.entropy[r] = bad ? nan : ls - all.t / all.s * LN2;
    for (int g = tid; g < p.given; g += GT) {
        const int id = p.tokens[(long long)r * p.given + g];
        p.logprobs[(long long)r * p.given + g] = (unsigned)id < (unsigned)p.V ? logp(at1<DT>(x, id)) : nan;
    }
    if constexpr (TOP) {
        if (tid < k) {
            const u64 y = sh.best[tid];
            p.top_ids[(long long)r * k + tid] = bad ? -1 : (int)~(uint32_t)y;
            p.top_logprobs[(long long)r * k + tid] = logp(logit_of(y));
        }
    }
}

template <int DT>
int run(const LogprobP& p, int rows, int dev, cudaStream_t s) {
    constexpr int SMEM = 2 * GT * U * 16;
    static std::atomic<uint64_t> done[2];
    if (const int rc = p.top ? allow_smem(logprob_kernel<DT, true>, SMEM, dev, done[1], "mk_logprobs")
                             : allow_smem(logprob_kernel<DT, false>, SMEM, dev, done[0], "mk_logprobs"))
        return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * p.split));
    cfg.blockDim = dim3(GT);
    cfg.dynamicSmemBytes = SMEM;
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
    if (a->vocab > 1 << 30) return fail(MK_ERR_UNSUPPORTED, "logprobs: vocab above 2^30");
    if (a->top > MAX_TOP) return fail(MK_ERR_UNSUPPORTED, "logprobs: top above %d", MAX_TOP);
    if (!a->logits || (a->given && (!a->tokens || !a->logprobs)) || (a->top && (!a->top_ids || !a->top_logprobs)))
        return fail(MK_ERR_INVALID_ARG, "logprobs: logits, tokens, logprobs, top_ids or top_logprobs is NULL");
    if ((uintptr_t)a->logits % e) return fail(MK_ERR_INVALID_ARG, "logprobs: logits not aligned to their type");
    if (off_by4(a->temperature, a->tokens, a->logprobs, a->entropy, a->top_ids, a->top_logprobs))
        return fail(MK_ERR_INVALID_ARG, "logprobs: an argument is not aligned to 4 bytes");
    if (a->rows == 0) return MK_OK;
    if ((int64_t)a->rows * MAX_CLUSTER > INT32_MAX) return fail(MK_ERR_UNSUPPORTED, "logprobs: too many rows in one call");
    int dev, sms;
    if (const int rc = device_sms(dev, sms, "mk_logprobs")) return rc;
    LogprobP p = {};
    p.logits = (const uint8_t*)a->logits, p.row_s = a->row_stride, p.temperature = a->temperature, p.tokens = a->tokens;
    p.logprobs = a->logprobs, p.entropy = a->entropy, p.top_ids = a->top_ids, p.top_logprobs = a->top_logprobs;
    p.V = a->vocab, p.given = a->given, p.top = a->top;
    // CTAs of a row: one or more an SM, as long as each has a part of a round (a CTA's first threshold and its end cost as
    // much as two rounds: 256 rows of 151936 bf16 logits take 41 us in one part each, 51 in two)
    p.split = 1;
    while (p.split < MAX_CLUSTER && (int64_t)a->rows * p.split < sms && a->vocab / p.split > GT * 4) p.split *= 2;
    cudaStream_t s = (cudaStream_t)stream;
    if (a->dtype == MK_DT_F32) return run<MK_DT_F32>(p, a->rows, dev, s);
    return a->dtype == MK_DT_BF16 ? run<MK_DT_BF16>(p, a->rows, dev, s) : run<MK_DT_F16>(p, a->rows, dev, s);
}
