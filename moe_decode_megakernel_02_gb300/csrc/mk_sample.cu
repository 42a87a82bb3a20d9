// mk_sample.cu -- one token a row from logits: temperature, top-k, top-p and
// min-p, with given random numbers (mk_sample).
//
// A row's weights are w_i = exp((x_i - max x) / T) in 32 bits; every sum of
// weights (the mass that top-p compares, the running sum that u picks from) is
// an integer sum of w_i 2^s, rounded to nearest, with s as large as V weights
// allow in 62 bits. Integer sums are the same in any order, so histograms may
// be built with atomics and the same inputs always give the same token; and a
// token's place among 100,000 others is decided at about 2^-44, far below one
// step of u.
//
// Tokens are ranked by (x descending, index ascending). The k-th rank, and the
// rank where the mass reaches p, are found without sorting: the distance of a
// token's ordered bit pattern from the row's largest, a 32-bit number that
// grows as x falls, is searched 12, 12 and 8 bits at a time with histograms of
// counts (top-k) or masses (top-p); what is left at one exact value are ties,
// taken by index.
//
// A row is one thread-block cluster of C CTAs: each keeps its slice of the row
// in shared memory, so the logits are read from HBM once however many passes
// follow; histograms and sums meet through distributed shared memory.
#include <cooperative_groups.h>

#include "mk_ops.cuh"

namespace {

using namespace mkop;
namespace cg = cooperative_groups;

constexpr int ST = 512;      // threads of a CTA
constexpr int BINS = 4096;   // histogram bins (12 bits a level)
constexpr int MAXC = 8;      // CTAs of a cluster
constexpr int MAX_SLICE = 45056;  // floats of a slice: 176 KB beside the histogram

typedef unsigned long long u64;

struct SampleP {
    const void* logits;
    long long row_stride;
    const float *u, *temperature;
    const int* top_k;
    const float *top_p, *min_p;
    int* tokens;
    float* probs;
    int* kept;
    int V, slice, seg, shift;
};

struct Shared {
    u64 hist[BINS];         // masses, or counts
    u64 warp_sum[ST / 32];
    u64 best;               // this CTA's largest key and its lowest index
    u64 part[MAXC];         // a total of each CTA of the cluster, written by that CTA
    u64 cross_before;       // the level's result, written by the CTA that has it
    unsigned cross_bin;
    unsigned bad;
    unsigned ties[MAXC], kept[MAXC];
};

// order-preserving unsigned image of a float (no NaN; -0 equals +0)
__device__ __forceinline__ unsigned key_of(float x) {
    const unsigned b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// and back
__device__ __forceinline__ float value_of(unsigned key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

struct Weight {
    float m, T, r, up;
    bool plain;  // T far from the ends of the range: the quotient by remainder (Markstein 1990) is the divided one
    __device__ __forceinline__ float operator()(float x) const {
        const float d = x - m;
        if (!plain) return expf(__fdiv_rn(d, T));
        const float q = d * r;
        // far below the smallest 32-bit number: also keeps overflowed quotients out of the remainder
        if (q < -150.f) return 0.f;
        return expf(__fmaf_rn(__fmaf_rn(-q, T, d), r, q));
    }
    // as an integer; a masked token (-infinity) weighs nothing
    __device__ __forceinline__ u64 fixed(float x) const {
        return x == -INFINITY ? 0ull : __float2ull_rn((*this)(x) * up);
    }
};

__device__ __forceinline__ u64 warp_incl(u64 v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 a = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += a;
    }
    return v;
}
// sum over the threads before this one; `total` of all. All threads call it.
__device__ u64 block_excl(u64 v, u64* warp_sum, u64& total) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const u64 inc = warp_incl(v);
    __syncthreads();
    if (lane == 31) warp_sum[w] = inc;
    __syncthreads();
    u64 before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < ST / 32; ++i) {
        if (i < w) before += warp_sum[i];
        total += warp_sum[i];
    }
    return before + inc - v;
}

// One level of the search over the cluster's histograms: the bin at which the
// running sum, `before` in front of bin 0, reaches `target`; `before` becomes
// the sum in front of that bin. With p >= 0 the target is found here, as the
// least whole number that is not below p times this level's total (at least 1:
// the first rank always stays).
__device__ unsigned find_bin(cg::cluster_group& cl, Shared& sh, int C, int rank, u64& before, u64& target, double p) {
    cl.sync();  // every CTA's histogram is complete
    const int per = BINS / C, each = (per + ST - 1) / ST;  // bins of this CTA, of a thread
    u64 mine = 0, bins[BINS / ST];
    const int b0 = rank * per + threadIdx.x * each;
#pragma unroll
    for (int i = 0; i < BINS / ST; ++i) bins[i] = 0;
    if ((int)threadIdx.x * each < per) {
#pragma unroll
        for (int i = 0; i < BINS / ST; ++i) {
            if (i < each)
                for (int c = 0; c < C; ++c) bins[i] += cl.map_shared_rank(sh.hist, c)[b0 + i];
            mine += bins[i];
        }
    }
    u64 slice;
    u64 at = block_excl(mine, sh.warp_sum, slice);
    if ((int)threadIdx.x < C) cl.map_shared_rank(sh.part, threadIdx.x)[rank] = slice;
    cl.sync();  // histograms have been read, the slices' totals are here
    u64 total = 0;
    for (int c = 0; c < C; ++c) {
        if (c == rank) at += total;
        total += sh.part[c];
    }
    if (p >= 0) target = max(1ull, (u64)ceil(p * (double)total));
    u64 run = before + at;
#pragma unroll
    for (int i = 0; i < BINS / ST; ++i) {
        if (run < target && run + bins[i] >= target) {
            for (int c = 0; c < C; ++c) {
                *cl.map_shared_rank(&sh.cross_bin, c) = (unsigned)(b0 + i);
                *cl.map_shared_rank(&sh.cross_before, c) = run;
            }
        }
        run += bins[i];
    }
    cl.sync();  // the result is here
    before = sh.cross_before;
    return sh.cross_bin;
}

__device__ __forceinline__ void clear_hist(Shared& sh) {
    for (int i = threadIdx.x; i < BINS; i += ST) sh.hist[i] = 0;
    __syncthreads();
}

// Bound: one read of the logits from HBM, then a fixed number of passes over
// shared memory (up to 3 each for top-k and top-p, one for the draw) with 3
// cluster barriers each. Small calls are those barriers' latency.
template <int DT>
__global__ void __launch_bounds__(ST) sample_kernel(const SampleP p) {
    extern __shared__ __align__(16) uint8_t smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    float* xs = reinterpret_cast<float*>(smem + sizeof(Shared));
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const long long row = blockIdx.x / C;
    const int i0 = min(p.V, rank * p.slice), n = min(p.V, i0 + p.slice) - i0;
    const int tid = threadIdx.x;

    // ---- the slice into shared memory; the largest logit, lowest index first
    if (tid == 0) {
        sh.best = 0;
        sh.bad = 0;
    }
    __syncthreads();
    u64 best = 0;
    bool bad = false;
    auto take = [&](int i, float x) {
        xs[i] = x;
        bad |= !(x < INFINITY);  // NaN or +infinity
        const u64 b = (u64)key_of(x) << 32 | (0xffffffffu - (unsigned)(i0 + i));
        best = b > best ? b : best;
    };
    if constexpr (DT == MK_DT_F32) {
        const float* src = (const float*)p.logits + row * p.row_stride + i0;
        if ((uintptr_t)src % 16 == 0) {
#pragma unroll 4
            for (int i = tid * 4; i + 3 < n; i += ST * 4) {
                const float4 a = __ldcs(reinterpret_cast<const float4*>(src + i));
                take(i, a.x), take(i + 1, a.y), take(i + 2, a.z), take(i + 3, a.w);
            }
            for (int i = (n & ~3) + tid; i < n; i += ST) take(i, src[i]);
        } else {
#pragma unroll 4
            for (int i = tid; i < n; i += ST) take(i, __ldcs(src + i));
        }
    } else {
        const uint16_t* src = (const uint16_t*)p.logits + row * p.row_stride + i0;
        auto cvt = [](uint32_t h) {
            if constexpr (DT == MK_DT_BF16) return __uint_as_float(h << 16);
            else return __half2float(__ushort_as_half((unsigned short)h));
        };
        if ((uintptr_t)src % 16 == 0) {
#pragma unroll 2
            for (int i = tid * 8; i + 7 < n; i += ST * 8) {
                const uint4 a = __ldcs(reinterpret_cast<const uint4*>(src + i));
                take(i, cvt(a.x & 0xffffu)), take(i + 1, cvt(a.x >> 16));
                take(i + 2, cvt(a.y & 0xffffu)), take(i + 3, cvt(a.y >> 16));
                take(i + 4, cvt(a.z & 0xffffu)), take(i + 5, cvt(a.z >> 16));
                take(i + 6, cvt(a.w & 0xffffu)), take(i + 7, cvt(a.w >> 16));
            }
            for (int i = (n & ~7) + tid; i < n; i += ST) take(i, cvt(src[i]));
        } else {
#pragma unroll 4
            for (int i = tid; i < n; i += ST) take(i, cvt(src[i]));
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const u64 b = __shfl_xor_sync(0xffffffffu, best, o);
        best = b > best ? b : best;
    }
    if ((tid & 31) == 0 && best) atomicMax(&sh.best, best);
    if (bad) sh.bad = 1;
    cl.sync();
    best = 0;
    unsigned any_bad = 0;
    for (int c = 0; c < C; ++c) {
        const u64 b = *cl.map_shared_rank(&sh.best, c);
        best = b > best ? b : best;
        any_bad |= *cl.map_shared_rank(&sh.bad, c);
    }
    const unsigned top = (unsigned)(best >> 32);
    const int argmax = (int)(0xffffffffu - (unsigned)best);
    const float T = p.temperature ? p.temperature[row] : 1.0f;
    if (any_bad || top == key_of(-INFINITY) || !(T > 0.f)) {
        // no distribution (a NaN, a +infinity, or nothing but masked tokens), or greedy
        if (rank == 0 && tid == 0) {
            const bool none = any_bad || top == key_of(-INFINITY);
            p.tokens[row] = none ? -1 : argmax;
            if (p.probs) p.probs[row] = none ? 0.f : 1.f;
            if (p.kept) p.kept[row] = none ? 0 : 1;
        }
        cl.sync();  // no CTA leaves while another reads its shared memory
        return;
    }
    Weight W;
    W.m = value_of(top);
    W.T = T;
    W.r = __frcp_rn(T);
    W.plain = T > 0x1p-60f && T < 0x1p60f;
    W.up = __uint_as_float((unsigned)(127 + p.shift) << 23);  // 2^shift

    const int k_in = p.top_k ? p.top_k[row] : 0;
    const float p_in = p.top_p ? p.top_p[row] : 1.0f;
    const float least = p.min_p ? p.min_p[row] : 0.0f;
    const bool by_k = k_in > 0 && k_in < p.V, by_p = p_in < 1.0f;
    // kept: distance < cut, and the first `quota` of the tokens at distance == cut
    const unsigned masked = top - key_of(-INFINITY);
    unsigned cut = masked;  // masked tokens are never kept
    u64 quota = 0;

    if (by_k) {
        u64 target = (u64)k_in, before = 0;
        unsigned prefix = 0;
#pragma unroll 1
        for (int l = 0; l < 3; ++l) {
            const int lo = l == 0 ? 20 : l == 1 ? 8 : 0, up = l == 0 ? 32 : l == 1 ? 20 : 8;
            clear_hist(sh);
            for (int i = tid; i < n; i += ST) {
                const unsigned d = top - key_of(xs[i]);
                if (l == 0 || (d >> up) == prefix)
                    atomicAdd(reinterpret_cast<unsigned*>(&sh.hist[(d >> lo) & ((1u << (up - lo)) - 1)]), 1u);
            }
            prefix = prefix << (up - lo) | find_bin(cl, sh, C, rank, before, target, -1.0);
        }
        if (prefix < masked) {  // fewer than k unmasked tokens: all of them stay
            cut = prefix;
            quota = (u64)k_in - before;
        }
    }
    if (by_p) {
        u64 target = 0, before = 0;
        unsigned prefix = 0;
        // the ties at top-k's border weigh `quota` times one of them
        const u64 border = quota ? W.fixed(value_of(top - cut)) * quota : 0;
#pragma unroll 1
        for (int l = 0; l < 3; ++l) {
            const int lo = l == 0 ? 20 : l == 1 ? 8 : 0, up = l == 0 ? 32 : l == 1 ? 20 : 8;
            clear_hist(sh);
            for (int i = tid; i < n; i += ST) {
                const float x = xs[i];
                const unsigned d = top - key_of(x);
                if (d < cut && (l == 0 || (d >> up) == prefix)) {
                    const u64 w = W.fixed(x);
                    if (w) atomicAdd(&sh.hist[(d >> lo) & ((1u << (up - lo)) - 1)], w);
                }
            }
            if (rank == 0 && tid == 0 && border && (l == 0 || (cut >> up) == prefix))
                atomicAdd(&sh.hist[(cut >> lo) & ((1u << (up - lo)) - 1)], border);
            prefix = prefix << (up - lo) | find_bin(cl, sh, C, rank, before, target, l == 0 ? fmax((double)p_in, 0.0) : -1.0);
        }
        // ties at the border: as many as have less than the target before
        // them (their weight is not 0: the bin was found by its mass)
        const u64 w = W.fixed(value_of(top - prefix));
        const u64 fit = (target - before + w - 1) / w;
        quota = prefix == cut && quota < fit ? quota : fit;
        cut = prefix;
    }

    // ---- the draw: threads hold consecutive segments, sums run in index order
    const int s0 = min(n, tid * p.seg), s1 = min(n, s0 + p.seg);
    u64 tie_at = 0;
    if (quota) {
        unsigned c = 0;
        for (int i = s0; i < s1; ++i) c += top - key_of(xs[i]) == cut;
        u64 all;
        tie_at = block_excl(c, sh.warp_sum, all);
        if (tid < C) cl.map_shared_rank(sh.ties, tid)[rank] = (unsigned)all;
        cl.sync();
        for (int r = 0; r < rank; ++r) tie_at += sh.ties[r];
    }
    auto keeps = [&](int i, float x, u64& tie, float& w) {
        const unsigned d = top - key_of(x);
        bool in = d < cut;
        if (d == cut) in = tie++ < quota;
        if (!in) return false;
        w = W(x);
        return w >= least || i0 + i == argmax;
    };
    u64 sum = 0;
    unsigned count = 0;
    {
        u64 tie = tie_at;
        for (int i = s0; i < s1; ++i) {
            float w;
            if (keeps(i, xs[i], tie, w)) {
                sum += __float2ull_rn(w * W.up);
                ++count;
            }
        }
    }
    u64 slice_sum, slice_kept;
    u64 at = block_excl(sum, sh.warp_sum, slice_sum);
    block_excl(count, sh.warp_sum, slice_kept);
    if (tid < C) {
        cl.map_shared_rank(sh.part, tid)[rank] = slice_sum;
        cl.map_shared_rank(sh.kept, tid)[rank] = (unsigned)slice_kept;
    }
    cl.sync();
    u64 total = 0;
    unsigned kept = 0;
    for (int c = 0; c < C; ++c) {
        if (c == rank) at += total;
        total += sh.part[c];
        kept += sh.kept[c];
    }
    const float u = fminf(fmaxf(p.u[row], 0.f), 0x1.fffffep-1f);
    // u total lies at or above the running sum of every token before the drawn one
    const u64 target = (u64)((double)u * (double)total);
    if (at <= target && at + sum > target) {
        u64 tie = tie_at, run = at;
        for (int i = s0; i < s1; ++i) {
            float w;
            if (!keeps(i, xs[i], tie, w)) continue;
            run += __float2ull_rn(w * W.up);
            if (run > target) {
                p.tokens[row] = i0 + i;
                if (p.probs) p.probs[row] = (float)((double)w * (double)W.up / (double)total);
                break;
            }
        }
    }
    if (rank == 0 && tid == 0 && p.kept) p.kept[row] = (int)kept;
}

}  // namespace

extern "C" int mk_sample(const mk_sampling* a, void* stream) {
    if (!a) return fail(MK_ERR_INVALID_ARG, "sample: NULL arguments");
    if (a->rows < 0 || a->vocab < 1) return fail(MK_ERR_INVALID_ARG, "sample: rows or vocab");
    const int e = dtype_bytes(a->dtype);
    if (!e) return fail(MK_ERR_INVALID_ARG, "sample: unknown dtype %d", a->dtype);
    if (a->rows == 0) return MK_OK;
    if (!a->logits || !a->u || !a->tokens) return fail(MK_ERR_INVALID_ARG, "sample: logits, u or tokens is NULL");
    if ((uintptr_t)a->logits % e) return fail(MK_ERR_INVALID_ARG, "sample: logits not aligned to their type");
    if (a->vocab > MAXC * MAX_SLICE) return fail(MK_ERR_UNSUPPORTED, "sample: vocab above %d", MAXC * MAX_SLICE);
    if (a->rows > INT32_MAX / MAXC) return fail(MK_ERR_UNSUPPORTED, "sample: too many rows");
    SampleP p;
    p.logits = a->logits, p.row_stride = a->row_stride, p.u = a->u, p.temperature = a->temperature;
    p.top_k = a->top_k, p.top_p = a->top_p, p.min_p = a->min_p;
    p.tokens = a->tokens, p.probs = a->probs, p.kept = a->kept;
    p.V = a->vocab;
    // a slice of 2048 tokens keeps a CTA's threads busy with 4 each
    int C = MAXC;
    while (C > 1 && a->vocab <= 2048 * (C / 2)) C /= 2;
    p.slice = ((a->vocab + C - 1) / C + 7) / 8 * 8;  // whole 16-byte pieces of 16-bit logits
    p.seg = ((p.slice + ST - 1) / ST) | 1;           // an odd stride: segments start in different banks
    p.shift = 61;
    while (p.shift > 0 && ((int64_t)a->vocab << 1) > ((int64_t)1 << (62 - p.shift))) --p.shift;
    auto kern = a->dtype == MK_DT_F32    ? sample_kernel<MK_DT_F32>
                : a->dtype == MK_DT_BF16 ? sample_kernel<MK_DT_BF16>
                                         : sample_kernel<MK_DT_F16>;
    const size_t smem = sizeof(Shared) + (size_t)p.slice * 4;
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return cuda_status(err, "mk_sample");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a->rows * C);
    cfg.blockDim = dim3(ST);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = C;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, kern, p);
    if (err != cudaSuccess) cudaGetLastError();
    return cuda_status(err, "mk_sample");
}
