// mk_sample.cu -- one token a row from logits: temperature, top-k, top-p and
// min-p, with given random numbers (mk_sample).
//
// A row's weights are w_i = exp((x_i - max x) / T) in 32 bits; every sum of
// weights (the mass that top-p compares, the running sum that u picks from) is
// an integer sum of w_i 2^42, each rounded to nearest. Integer sums are the
// same in any order, so they may be split over threads and use atomics, and
// the same inputs always give the same token; a token's place among 100,000
// others is decided to about 2^-42 of the largest weight, far below one step
// of u.
//
// Tokens are ranked by (x descending, index ascending); a rank is a 64-bit
// number, the distance of the token's ordered bit pattern from the row's
// largest above its index. Nothing is sorted but short lists:
//   top-k  the k-th largest of the threads' own maxima bounds the k-th logit
//          from below (to one of 512 equal bins); the few tokens above go to
//          a list in one CTA, which ranks them and does all the rest.
//   top-p  one pass sums all weights; a token lighter than (1 - p) sum / V
//          cannot be kept, the others fill a histogram of masses, 512 bins
//          between that bound and the largest logit. Tokens above the bin
//          where the mass reaches p are kept, the bin's own go to a list,
//          which gives the last rank kept.
//   Where a list would not fit (long runs of nearly equal logits, a large k),
//   the border is searched by histograms over 9, 9, 9 and 5 bits of the
//   distance, and what is left at one exact value are ties, taken by index.
// The kept weights are summed a warp a stretch of tokens, and the warp whose
// stretch u falls into walks it.
//
// A row is one thread-block cluster of C CTAs: each keeps its slice of the row
// in shared memory as it came, so the logits are read from HBM once however
// many passes follow; sums, histograms and lists meet through distributed
// shared memory. A meeting (write to the others, cluster barrier) costs about
// 2500 cycles, as much as a pass: a row takes 2 (no filter), 3 (top-k) or 4
// (top-p) of them, and every CTA works out what it can by itself.
//
// Measured: one fp32 row of 32000 with all filters 10 us, the latency of its
// passes and meetings; 32 fp32 rows of 64000 with top-p 31 us; 256 bf16 rows
// of 151936, each with its own settings, 100 us (0.78 TB/s, 12 % of a copy's
// rate), with top-p on three rows of four 203 and on all 255, top-k alone 77,
// min-p alone 70, no filter 79. Bound by top-p's two passes over the half
// of a normal row's tokens that its bound (1 - p) sum / V leaves (34,000 and
// 27,000 of a row's 75,000 cycles: four shared-memory atomics and an exponential
// a token), and by the meetings, in which a CTA's warps wait (a scheduler issues
// in 44 % of its cycles).
#include <cooperative_groups.h>

#include <atomic>
#include <cfloat>
#include <type_traits>

#include "mk_ops.cuh"

namespace {

using namespace mkop;
namespace cg = cooperative_groups;

constexpr int ST = 512;        // threads of a CTA
constexpr int SW = ST / 32;
constexpr int BINS = ST;       // histogram bins, one a thread
constexpr int LIST = 2 * ST;     // ranks a list holds: ordering more costs more than further histograms
constexpr int MAXC = 8;        // CTAs of a cluster
constexpr int MAX_SLICE_B = 180224;  // bytes of a slice of logits: 176 KB

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
    int V, slice;
    int rows, order;  // order: the costly rows go first
};

// Written by one CTA for another only where it says so; each such place is
// written once, or alternates, so that a late reader is never overtaken.
struct Shared {
    union {
        struct {
            unsigned limb[3][BINS], number[BINS];  // a histogram being filled: masses in 14-bit limbs, counts
        };
        u64 own[LIST];                     // ranks of this CTA's tokens
    };
    u64 mass[2][BINS];                     // complete histograms, read by the cluster; the next one's place is free
                                           // until it is complete, and serves as the warps' queues
    unsigned count[2][BINS];
    u64 list[LIST];                        // ranks, from all CTAs
    u64 part[2][MAXC];                     // totals of each CTA, from it
    u64 sums[MAXC * SW];                   // kept mass of every warp's stretch, from its CTA
    unsigned kept[MAXC];                   // kept tokens of each CTA, from it
    unsigned top[MAXC], low_max[MAXC], bad[MAXC];  // what each CTA saw, from it
    u64 warp_sum[SW];
    u64 cross_before, last;
    unsigned cross_bin, cross_count, cross_ahead;
    unsigned argmax, list_n, own_n, own_base;
    int row;
    unsigned my_top, my_low, my_low_max, my_bad, my_kept;
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
    float m, T, r, low;
    bool plain;  // T far from the ends of the range: the quotient by remainder (Markstein 1990) is the divided one
    // x = -infinity weighs 0 (where T is plain)
    __device__ __forceinline__ float operator()(float x) const {
        // (a difference beyond the range must not meet an infinite T)
        if (!plain) return expf(__fdiv_rn(fmaxf(x - m, -FLT_MAX), T));
        // below -200 T the weight is 0 anyway; the bound keeps infinities out of the remainder
        const float d = fmaxf(x - m, low), q = d * r;
        return expf(__fmaf_rn(__fmaf_rn(-q, T, d), r, q));
    }
};

// Sums of w 2^42 (0 <= w <= 1) over up to 400 weights in two 32-bit integers:
// adding 24 leaves w in steps of 2^-19 in the low bits of the sum, adding
// 1.5 2^-19 what is left of it in steps of 2^-42.
struct Sum {
    unsigned hi = 0, lo = 0;
    __device__ __forceinline__ void add(float w) {
        const float a = w + 24.0f;
        const float b = (w - (a - 24.0f)) + 0x1.8p-19f;
        hi += __float_as_uint(a);
        lo += __float_as_uint(b);
    }
    __device__ __forceinline__ u64 value(unsigned n) const {  // of n weights
        const unsigned h = hi - n * 0x41c00000u;    // the bits of 24
        const int l = (int)(lo - n * 0x36400000u);  // and of 1.5 2^-19
        return ((u64)h << 23) + (u64)(long long)l;
    }
};
__device__ __forceinline__ u64 fixed(float w) {
    Sum s;
    s.add(w);
    return s.value(1);
}

// f t (0 <= f < 1) in whole numbers, rounded down, or up. Integers: 64-bit
// floating point runs at 1/64 of the 32-bit rate here.
__device__ __forceinline__ u64 part_of(float f, u64 t, bool up) {
    const unsigned b = __float_as_uint(f), ex = b >> 23;
    const unsigned man = ex ? (b & 0x7fffffu) | 0x800000u : b;
    const int s = 150 - (int)(ex ? ex : 1u);  // f = man / 2^s, s >= 24
    const u64 hi = __umul64hi(t, man), lo = t * man;
    if (s >= 128) return up && (hi | lo);
    const u64 q = s < 64 ? hi << (64 - s) | lo >> s : s == 64 ? hi : hi >> (s - 64);
    const bool rest = s < 64 ? (lo << (64 - s)) != 0 : lo != 0 || (s > 64 && (hi << (128 - s)) != 0);
    return q + (up && rest);
}

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
    for (int i = 0; i < SW; ++i) {
        if (i < w) before += warp_sum[i];
        total += warp_sum[i];
    }
    return before + inc - v;
}

// A token's weight (below 2^43) into a bin: limbs of 14 bits, whose 32-bit
// sums hold 2^18 tokens, so that no atomic's result is waited for.
__device__ __forceinline__ void tally(Shared& sh, int bin, u64 w) {
    const unsigned a = (unsigned)w & 0x3fffu, b = (unsigned)(w >> 14) & 0x3fffu, c = (unsigned)(w >> 28);
    if (a) atomicAdd(&sh.limb[0][bin], a);
    if (b) atomicAdd(&sh.limb[1][bin], b);
    if (c) atomicAdd(&sh.limb[2][bin], c);
    atomicAdd(&sh.number[bin], 1u);
}

struct Found {
    int bin;         // -1: the total does not reach the target
    u64 before;      // in front of the bin
    unsigned count;  // tokens in it
    unsigned ahead;  // those of them in the CTAs before this one
    u64 total;
};
// The bin of the cluster's histogram at which the running sum (of masses, or
// of counts), `before` in front of bin 0, reaches the target; every CTA finds
// it by itself from all CTAs' bins. `turn` alternates. The histogram is empty again.
__device__ Found find_bin(cg::cluster_group& cl, Shared& sh, int C, int rank, int turn, bool by_count, u64 before, u64 target) {
    const int t = threadIdx.x;
    __syncthreads();
    sh.mass[turn][t] = ((u64)sh.limb[2][t] << 28) + ((u64)sh.limb[1][t] << 14) + sh.limb[0][t];
    sh.count[turn][t] = sh.number[t];
    sh.limb[0][t] = sh.limb[1][t] = sh.limb[2][t] = sh.number[t] = 0;
    if (t == 0) sh.cross_bin = 0xffffffffu;
    cl.sync();
    u64 m = 0;
    unsigned n = 0, ahead = 0;
#pragma unroll
    for (int c = 0; c < MAXC; ++c)  // all at once: each is a round trip through the cluster
        if (c < C) {
            if (!by_count) m += cl.map_shared_rank(sh.mass[turn], c)[t];
            if (c == rank) ahead = n;
            n += cl.map_shared_rank(sh.count[turn], c)[t];
        }
    const u64 v = by_count ? n : m;
    Found f;
    const u64 run = before + block_excl(v, sh.warp_sum, f.total);
    if (run < target && run + v >= target) sh.cross_bin = t, sh.cross_before = run, sh.cross_count = n, sh.cross_ahead = ahead;
    __syncthreads();
    f.bin = (int)sh.cross_bin;
    f.before = sh.cross_before;
    f.count = sh.cross_count;
    f.ahead = sh.cross_ahead;
    __syncthreads();
    return f;
}

// v[0 .. n) ascending; `n2` a power of two not below n, within v, padded with ~0 here
__device__ void sort_list(u64* v, int n, int n2) {
    for (int i = n + threadIdx.x; i < n2; i += ST) v[i] = ~0ull;
    __syncthreads();
    for (int k = 2; k <= n2; k <<= 1)
        for (int j = k >> 1; j; j >>= 1) {
            for (int i = threadIdx.x; i < n2 / 2; i += ST) {
                const int a = 2 * i - (i & (j - 1)), b = a + j;
                const u64 x = v[a], y = v[b];
                if ((x > y) == ((a & k) == 0)) v[a] = y, v[b] = x;
            }
            __syncthreads();
        }
}
// the same for up to ST numbers, one a thread in a register: partners within a
// warp meet by shuffles, the others through v
__device__ void sort_one_each(u64* v, int n) {
    const int t = threadIdx.x;
    int n2 = 32;
    while (n2 < n) n2 *= 2;
    u64 x = t < n ? v[t] : ~0ull;
    __syncthreads();
    for (int k = 2; k <= n2; k <<= 1)
        for (int j = k >> 1; j; j >>= 1) {
            u64 y;
            if (j < 32) {
                y = __shfl_xor_sync(0xffffffffu, x, j);
            } else {
                if (t < n2) v[t] = x;
                __syncthreads();
                y = t < n2 ? v[t ^ j] : 0;
                __syncthreads();
            }
            // the lower place of an ascending pair takes the smaller one
            const bool smaller = ((t & j) == 0) == ((t & k) == 0);
            x = (x < y) == smaller ? x : y;
        }
    if (t < n) v[t] = x;
    __syncthreads();
}
__device__ void order_list(u64* v, int n) {
    if (n <= ST)
        sort_one_each(v, n);
    else
        sort_list(v, n, 2 * ST);
}

// Row number i of the order in which rows are taken: those that need top-p's
// pass over the whole row first, each kind by index, so that none of them (2.5
// times the others' time) begins when the rest is done. Every CTA works it out
// by itself, from all rows' settings.
__device__ int row_in_order(const SampleP& p, Shared& sh, int i) {
    auto costly = [&](int r) {
        const float T = p.temperature ? p.temperature[r] : 1.0f;
        const int k = p.top_k ? p.top_k[r] : 0;
        return T > 0.0f && p.top_p[r] < 1.0f && (k <= 0 || k > LIST);
    };
    int n = 0;
    for (int r0 = 0; r0 < p.rows; r0 += ST) n += __syncthreads_count(r0 + (int)threadIdx.x < p.rows && costly(r0 + (int)threadIdx.x));
    const bool want = i < n;
    int left = want ? i : i - n;  // rows of the kind before the one looked for
    if (threadIdx.x == 0) sh.row = i;
    for (int r0 = 0; r0 < p.rows; r0 += ST) {
        const int r = r0 + (int)threadIdx.x;
        const bool one = r < p.rows && costly(r) == want;
        u64 all;
        const u64 before = block_excl(one, sh.warp_sum, all);
        if (one && before == (u64)left) sh.row = r;
        if ((u64)left < all) break;
        left -= (int)all;
    }
    __syncthreads();
    return sh.row;
}

// Bound: one read of the logits from HBM, then passes over shared memory of 4
// to 25 operations a token (the largest: summing all weights). Small calls are
// the latency of the cluster's meetings.
template <int DT>
__global__ void __launch_bounds__(ST, 2) sample_kernel(const SampleP p) {
    typedef typename std::conditional<DT == MK_DT_F32, float, uint16_t>::type Raw;
    constexpr int E = 16 / sizeof(Raw);  // logits of a 16-byte vector
    extern __shared__ __align__(16) uint8_t smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    uint4* const xs = reinterpret_cast<uint4*>(smem + (sizeof(Shared) + 15) / 16 * 16);
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const long long row = p.order ? row_in_order(p, sh, blockIdx.x / C) : blockIdx.x / C;
    const int i0 = min(p.V, rank * p.slice), n = min(p.V, i0 + p.slice) - i0;
    const int nv = (n + E - 1) / E;  // vectors of the slice
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    auto value = [](uint32_t raw) {  // a 16-bit logit
        if constexpr (DT == MK_DT_BF16) return __uint_as_float(raw << 16);
        else return __half2float(__ushort_as_half((unsigned short)raw));
    };
    auto unpack = [&](float (&x)[E], const uint4& a) {
        if constexpr (DT == MK_DT_F32) {
            x[0] = __uint_as_float(a.x), x[1] = __uint_as_float(a.y);
            x[2] = __uint_as_float(a.z), x[3] = __uint_as_float(a.w);
        } else {
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = value(w[i] & 0xffffu);
                x[2 * i + 1] = value(w[i] >> 16);
            }
        }
    };

    auto larger = [](uint32_t a, uint32_t b) {  // of one 32-bit logit, or of two 16-bit ones; NaN wins
        uint32_t y;
        if constexpr (DT == MK_DT_F32) asm("max.NaN.f32 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
        else if constexpr (DT == MK_DT_BF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
        else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
        return y;
    };
    const uint32_t masked_raw = DT == MK_DT_F32 ? 0xff800000u : DT == MK_DT_BF16 ? 0xff80ff80u : 0xfc00fc00u;

    // ---- the slice into shared memory; the largest logit, a NaN if there is one
    if (tid == 0) {
        sh.my_top = 0, sh.my_low = sh.my_low_max = 0xffffffffu, sh.my_bad = 0, sh.my_kept = 0;
        sh.argmax = 0xffffffffu, sh.list_n = 0, sh.own_n = 0;
    }
    sh.limb[0][tid] = sh.limb[1][tid] = sh.limb[2][tid] = sh.number[tid] = 0;
    __syncthreads();
    float big;
    {
        const Raw* src = (const Raw*)p.logits + row * p.row_stride + i0;
        Raw* raw = reinterpret_cast<Raw*>(xs);
        const int whole = (uintptr_t)src % 16 == 0 ? n / E : 0;
        uint32_t best = masked_raw;
#pragma unroll 4
        for (int i = tid; i < whole; i += ST) {
            const uint4 a = __ldcs(reinterpret_cast<const uint4*>(src) + i);
            xs[i] = a;
            best = larger(best, larger(larger(a.x, a.y), larger(a.z, a.w)));
        }
        for (int i = whole * E + tid; i < nv * E; i += ST) {
            Raw a;
            if constexpr (DT == MK_DT_F32) a = i < n ? src[i] : -INFINITY;  // the last vector's rest is masked
            else a = i < n ? src[i] : (Raw)masked_raw;
            raw[i] = a;
            if constexpr (DT == MK_DT_F32) best = larger(best, __float_as_uint(a));
            else best = larger(best, (masked_raw & 0xffff0000u) | a);
        }
        if constexpr (DT == MK_DT_F32) {
            big = __uint_as_float(best);
        } else {
            const float lo = value(best & 0xffffu), hi = value(best >> 16);
            big = lo != lo || hi != hi ? __uint_as_float(0x7fffffffu) : fmaxf(lo, hi);
        }
    }
    {
        // the least of the threads' largest bounds top-k's search; threads without a token do not count
        const unsigned k = key_of(big), masked_key = key_of(-INFINITY);
        const unsigned a = __reduce_max_sync(0xffffffffu, k);
        const unsigned c = __reduce_min_sync(0xffffffffu, k > masked_key ? k : 0xffffffffu);
        if (lane == 0) {
            atomicMax(&sh.my_top, a);
            atomicMin(&sh.my_low_max, c);
        }
        if (!(big < INFINITY)) sh.my_bad = 1;  // NaN or +infinity
    }
    cl.sync();  // every CTA runs, and has its numbers
    if (tid < C) {
        sh.top[tid] = *cl.map_shared_rank(&sh.my_top, tid);
        sh.low_max[tid] = *cl.map_shared_rank(&sh.my_low_max, tid);
        sh.bad[tid] = *cl.map_shared_rank(&sh.my_bad, tid);
    }
    __syncthreads();
    unsigned top = 0, low_max_key = 0xffffffffu, any_bad = 0;
    for (int c = 0; c < C; ++c) {
        top = max(top, sh.top[c]);
        low_max_key = min(low_max_key, sh.low_max[c]);
        any_bad |= sh.bad[c];
    }
    const float m = value_of(top);
    const float T = p.temperature ? p.temperature[row] : 1.0f;
    const float least = p.min_p ? p.min_p[row] : 0.0f;
    const bool none = any_bad || m == -INFINITY;  // a NaN, a +infinity, or nothing but masked tokens
    if (none || !(T > 0.f) || !(least <= 1.f)) {
        // nothing to draw from, or only the first rank: the lowest index of the largest logit
        if (!none && sh.my_top == top) {
            for (int v = tid; v < nv; v += ST) {
                float x[E];
                unpack(x, xs[v]);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (x[e] == m) atomicMin(cl.map_shared_rank(&sh.argmax, 0), (unsigned)(i0 + v * E + e));
            }
        }
        cl.sync();
        if (rank == 0 && tid == 0) {
            p.tokens[row] = none ? -1 : (int)sh.argmax;
            if (p.probs) p.probs[row] = none ? 0.f : 1.f;
            if (p.kept) p.kept[row] = none ? 0 : 1;
        }
        return;
    }
    const Weight W = {m, T, __frcp_rn(T), -200.f * T, T > 0x1p-60f && T < 0x1p60f};
    const int k_in = p.top_k ? p.top_k[row] : 0;
    const float p_in = p.top_p ? p.top_p[row] : 1.0f;
    const bool by_k = k_in > 0 && k_in < p.V, by_p = p_in < 1.0f;
    const float u = fminf(fmaxf(p.u[row], 0.f), 0x1.fffffep-1f);
    const unsigned masked = top - key_of(-INFINITY);
    auto mass_target = [&](u64 total) {  // the mass that ends top-p; at least 1: the first rank always stays
        return max(1ull, part_of(fmaxf(p_in, 0.f), total, true));
    };

    // a warp's stretch of the slice, in vectors
    const int v0 = (int)((long long)nv * warp / SW), v1 = (int)((long long)nv * (warp + 1) / SW);
    auto each = [&](auto f) {  // f(logit, its index) over the stretch, lanes side by side
        for (int v = v0 + lane; v < v1; v += 32) {
            float x[E];
            unpack(x, xs[v]);
#pragma unroll
            for (int e = 0; e < E; ++e) f(x[e], i0 + v * E + e);
        }
    };
    int turn = 0;  // of what alternates
    // f(logit) for the tokens that `take(logit, index)` says, 32 of them at a time: they wait in a queue of the
    // warp's, so that costly work runs on full warps
    auto dense = [&](auto take, auto f) {
        static_assert(sizeof(sh.mass[0]) >= SW * 64 * sizeof(float), "queues");
        float* q = reinterpret_cast<float*>(sh.mass[turn]) + warp * 64;
        int waiting = 0;
        for (int v = v0; v < v1; v += 32) {
            float x[E];
            unpack(x, v + lane < v1 ? xs[v + lane] : make_uint4(masked_raw, masked_raw, masked_raw, masked_raw));
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const bool in = take(x[e], i0 + (v + lane) * E + e);
                const unsigned who = __ballot_sync(0xffffffffu, in);
                if (who) {
                    if (in) q[waiting + __popc(who & ((1u << lane) - 1))] = x[e];
                    waiting += __popc(who);
                    __syncwarp();
                    if (waiting >= 32) {
                        f(q[lane]);
                        waiting -= 32;
                        const float rest = q[32 + lane];
                        __syncwarp();
                        if (lane < waiting) q[lane] = rest;
                        __syncwarp();
                    }
                }
            }
        }
        if (lane < waiting) f(q[lane]);
        __syncwarp();
    };
    // equal bins from the largest logit down to `edge`; lower ones fall into the last
    struct Linear {
        float m, scale;
        __device__ float place(float x) const { return (m - x) * scale; }
        __device__ int operator()(float x) const { return (int)fminf(place(x), (float)(BINS - 1)); }
        // whether x lies above bin b, and in it, without a conversion
        __device__ bool above(float x, int b) const { return place(x) < (float)b; }
        __device__ bool in(float x, int b) const { return !(place(x) < (float)b) && (place(x) < (float)(b + 1) || b == BINS - 1); }
    };
    auto bins_down_to = [&](float edge) {
        const float s = (float)BINS / (m - edge);
        return Linear{m, s < 1e30f ? s : 0.f};  // no room between the two: one bin
    };
    // The ranks of tokens of the lane's vector v + lane, elements `in`, to this CTA's own list. A list goes on to
    // the cluster as a whole, as every trip there takes about a thousand cycles.
    auto put = [&](int v, const float (&x)[E], unsigned in) {
        if (!in) return;
        unsigned at = atomicAdd(&sh.own_n, (unsigned)__popc(in));
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (in >> e & 1u) {
                if (at < LIST) sh.own[at] = (u64)(top - key_of(x[e])) << 32 | (unsigned)(i0 + (v + lane) * E + e);
                ++at;
            }
    };
    // this CTA's list to the lists of CTAs [0, to), from place `base` on
    auto deliver = [&](int to, unsigned base) {
        const unsigned n_own = min(sh.own_n, (unsigned)LIST);
        for (unsigned i = tid; i < n_own; i += ST)
            if (base + i < LIST)
                for (int c = 0; c < to; ++c) cl.map_shared_rank(sh.list, c)[base + i] = sh.own[i];
    };
    // all tokens from `edge` on that `pick` takes
    auto collect = [&](float edge, auto pick) {
        for (int v = v0; v < v1; v += 32) {
            float x[E];
            unsigned in = 0;
            uint4 a = make_uint4(masked_raw, masked_raw, masked_raw, masked_raw);
            if (v + lane < v1) a = xs[v + lane];
            const uint32_t best = larger(larger(a.x, a.y), larger(a.z, a.w));
            bool some;
            if constexpr (DT == MK_DT_F32) some = __uint_as_float(best) >= edge;
            else some = fmaxf(value(best & 0xffffu), value(best >> 16)) >= edge;
            if (!__any_sync(0xffffffffu, some)) continue;
            unpack(x, a);
#pragma unroll
            for (int e = 0; e < E; ++e) in |= (unsigned)(x[e] >= edge && pick(x[e])) << e;
            put(v, x, in);
        }
    };
    // sums and minima over all threads of the cluster
    auto cluster_sum = [&](u64 v) {
        u64 mine, all = 0;
        block_excl(v, sh.warp_sum, mine);
        if (tid < C) cl.map_shared_rank(sh.part[turn], tid)[rank] = mine;
        cl.sync();
        for (int c = 0; c < C; ++c) all += sh.part[turn][c];
        turn ^= 1;
        return all;
    };
    auto cluster_min = [&](unsigned v) {
        v = __reduce_min_sync(0xffffffffu, v);
        __syncthreads();
        if (lane == 0) sh.warp_sum[warp] = v;
        __syncthreads();
        for (int w = 0; w < SW; ++w) v = min(v, (unsigned)sh.warp_sum[w]);
        if (tid < C) cl.map_shared_rank(sh.part[turn], tid)[rank] = v;
        cl.sync();
        for (int c = 0; c < C; ++c) v = min(v, (unsigned)sh.part[turn][c]);
        turn ^= 1;
        return v;
    };
    // The rank at which a running sum over ranks (of counts, or of masses of tokens up to `up_to`) reaches the
    // target, by histograms over the bits of the distance, then by index among equal logits. All CTAs call it; the
    // sum reaches the target.
    auto search = [&](bool by_count, u64 target, u64 up_to) {
        const float xk = value_of(top - (unsigned)(up_to >> 32));
        const unsigned ik = (unsigned)up_to;
        u64 before = 0;
        unsigned prefix = 0;
#pragma unroll 1
        for (int l = 0; l < 4; ++l) {
            const int lo = l == 3 ? 0 : 23 - 9 * l, up = l == 0 ? 32 : 32 - 9 * l;
            each([&](float x, int i) {
                const unsigned d = top - key_of(x);
                if ((l == 0 || (d >> up) == prefix) && (x > xk || (x == xk && (unsigned)i <= ik)))
                    tally(sh, (d >> lo) & ((1u << (up - lo)) - 1), by_count ? 0 : fixed(W(x)));
            });
            const Found f = find_bin(cl, sh, C, rank, turn, by_count, before, target);
            turn ^= 1;
            prefix = prefix << (up - lo) | (unsigned)f.bin;
            before = f.before;
        }
        // equal logits: their first `want`, in index order
        const float x0 = value_of(top - prefix);
        const u64 w = by_count ? 1 : fixed(W(x0));
        unsigned c = 0;
        each([&](float x, int) { c += x == x0; });
        c = __reduce_add_sync(0xffffffffu, c);
        u64 mine, all = 0, at = block_excl(lane == 0 ? c : 0, sh.warp_sum, mine);
        if (tid < C) cl.map_shared_rank(sh.part[turn], tid)[rank] = mine;
        cl.sync();
        at = __shfl_sync(0xffffffffu, at, 0);
        for (int r = 0; r < C; ++r) {
            if (r == rank) at += all;
            all += sh.part[turn][r];
        }
        const u64 want = min((target - before + w - 1) / w, all);
        if (at < want && at + c >= want) {  // one warp of the cluster
            u64 seen = at;
            for (int v = v0; v < v1 && seen < want; v += 32) {
                float x[E];
                const bool in = v + lane < v1;
                if (in) unpack(x, xs[v + lane]);
                unsigned some = 0;
#pragma unroll
                for (int e = 0; e < E; ++e) some += in && x[e] == x0;
                u64 place = seen + warp_incl(some) - some;
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (in && x[e] == x0 && ++place == want)
                        for (int r = 0; r < C; ++r)
                            *cl.map_shared_rank(&sh.last, r) = (u64)prefix << 32 | (unsigned)(i0 + (v + lane) * E + e);
                seen += __reduce_add_sync(0xffffffffu, some);
            }
        }
        cl.sync();
        turn ^= 1;
        return min(sh.last, up_to);
    };

    // kept: ranks up to `last` (and weights of at least min_p)
    u64 last = ((u64)masked << 32) - 1;  // masked tokens are never kept
    if (by_k) {
        // at least k tokens lie at or above the k-th largest of the threads' maxima; a k beyond what those
        // tell is sought among all tokens
        const bool by_threads = k_in <= min(p.V, C * ST) / 4;
        float edge = value_of(low_max_key);
        if (!by_threads) {
            float small = INFINITY;
            each([&](float x, int) { small = fminf(small, x > -INFINITY ? x : INFINITY); });
            edge = value_of(cluster_min(small < INFINITY ? key_of(small) : 0xffffffffu));
        }
        const Linear bin = bins_down_to(edge);
        if (by_threads) {
            if (big > -INFINITY) atomicAdd(&sh.number[bin(big)], 1u);
        } else {
            each([&](float x, int) {
                if (x > -INFINITY) atomicAdd(&sh.number[bin(x)], 1u);
            });
        }
        const Found f = find_bin(cl, sh, C, rank, turn, true, 0, (u64)k_in);
        turn ^= 1;
        // With fewer than k of them, top-k may still bind: search(). A bin of all tokens is known to fit or not.
        bool listed = f.bin >= 0 && (by_threads || f.before + f.count <= LIST);
        bool binds = f.bin >= 0 || by_threads;
        if (listed) {
            collect(edge, [&](float x) { return f.bin == BINS - 1 || bin.above(x, f.bin + 1); });
            __syncthreads();
            if (tid == 0) sh.own_base = atomicAdd(cl.map_shared_rank(&sh.list_n, 0), sh.own_n);
            __syncthreads();
            deliver(1, sh.own_base);
            cl.sync();
            listed = *cl.map_shared_rank(&sh.list_n, 0) <= LIST;
            if (listed && rank != 0) {
                // CTA 0 has every candidate and goes on alone; it ends after all others have read its count
                asm volatile("barrier.cluster.arrive;" ::: "memory");
                return;
            }
        } else if (by_threads) {
            // how many tokens are there at all
            unsigned c = 0;
            each([&](float x, int) { c += x > -INFINITY; });
            binds = cluster_sum(c) >= (u64)k_in;
        }
        if (listed) {
            {
                int n_l = (int)sh.list_n;
                order_list(sh.list, n_l);
                n_l = min(n_l, k_in);
                // running mass in rank order; top-p and min-p both keep a beginning
                const int each_l = (n_l + ST - 1) / ST, a0 = min(n_l, tid * each_l), a1 = min(n_l, a0 + each_l);
                u64 mass = 0, total;
                for (int i = a0; i < a1; ++i) mass += fixed(W(value_of(top - (unsigned)(sh.list[i] >> 32))));
                u64 run = block_excl(mass, sh.warp_sum, total);
                const u64 target = by_p ? mass_target(total) : ~0ull;
                unsigned keeps = 0;
                for (int i = a0; i < a1; ++i) {
                    const float w = W(value_of(top - (unsigned)(sh.list[i] >> 32)));
                    if (run < target && w >= least) ++keeps;
                    run += fixed(w);
                }
                u64 n_k;
                block_excl(keeps, sh.warp_sum, n_k);
                // in index order now: (index, distance)
                for (int i = tid; i < (int)n_k; i += ST) sh.list[i] = sh.list[i] << 32 | sh.list[i] >> 32;
                __syncthreads();
                order_list(sh.list, (int)n_k);
                const int each_k = ((int)n_k + ST - 1) / ST, b0 = min((int)n_k, tid * each_k),
                          b1 = min((int)n_k, b0 + each_k);
                mass = 0;
                for (int i = b0; i < b1; ++i) mass += fixed(W(value_of(top - (unsigned)sh.list[i])));
                run = block_excl(mass, sh.warp_sum, total);
                const u64 pick = part_of(u, total, false);
                for (int i = b0; i < b1; ++i) {
                    const float w = W(value_of(top - (unsigned)sh.list[i]));
                    const u64 f2 = fixed(w);
                    if (run <= pick && run + f2 > pick) {
                        p.tokens[row] = (int)(sh.list[i] >> 32);
                        if (p.probs) p.probs[row] = (float)((double)w * 0x1p42 / (double)total);
                    }
                    run += f2;
                }
                if (tid == 0 && p.kept) p.kept[row] = (int)n_k;
            }
            asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
            return;
        }
        // the list's place is the histogram's
        sh.limb[0][tid] = sh.limb[1][tid] = sh.limb[2][tid] = sh.number[tid] = 0;
        __syncthreads();
        if (tid == 0) sh.own_n = 0;
        if (binds) last = search(true, (u64)k_in, last);
    }

    const float least_x = least > 0.f ? m + T * (logf(least) - 0.01f) : -INFINITY;  // below: lighter than min_p
    // kept tokens end at `last`; a row that keeps all unmasked tokens needs no comparison, as masked ones weigh 0
    bool all_ranks = last == ((u64)masked << 32) - 1 && W.plain;
    const bool plain_ranks = all_ranks;
    float xc = value_of(top - (unsigned)(last >> 32));
    unsigned ic = (unsigned)last;
    auto up_to_last = [&](float x, int i) { return x > xc || (x == xc && (unsigned)i <= ic); };
    Linear bin = {m, 0.f};
    int border = -1;       // the bin whose tokens are in the list
    unsigned listed = 0;   // how many
    unsigned ahead = 0;    // how many of them in the CTAs before this one
    u64 before = 0, target = 0;
    float low_x = -INFINITY;
    if (by_p) {
        // all of top-k's mass, and the least logit
        Sum s;
        unsigned number = 0;
        float small = INFINITY;
        if (all_ranks) {
            each([&](float x, int) {
                s.add(W(x));
                ++number;
                small = fminf(small, x > -INFINITY ? x : INFINITY);
            });
        } else {
            each([&](float x, int i) {
                if (up_to_last(x, i)) {
                    s.add(W(x));
                    ++number;
                    small = fminf(small, x);
                }
            });
        }
        const unsigned low_key = __reduce_min_sync(0xffffffffu, small < INFINITY ? key_of(small) : 0xffffffffu);
        if (lane == 0) atomicMin(&sh.my_low, low_key);
        const u64 total = cluster_sum(s.value(number));  // its barriers are for my_low too
        target = mass_target(total);
        // Tokens lighter than (1 - p) total / V weigh less than (1 - p) total together: at least p total lies
        // before them. Half of that bound, and a hundredth, leave room for roundings.
        const float light = (1.f - fmaxf(p_in, 0.f)) * (__ull2float_rn(total) * 0x1p-43f) / (float)p.V;
        unsigned low = 0xffffffffu;
#pragma unroll
        for (int c = 0; c < MAXC; ++c)
            if (c < C) low = min(low, *cl.map_shared_rank(&sh.my_low, c));
        low_x = fmaxf(value_of(low), light > 1e-30f ? m + T * (logf(light) - 0.01f) : -INFINITY);
        bin = bins_down_to(low_x);
        dense([&](float x, int i) { return x >= low_x && up_to_last(x, i); },
              [&](float x) { tally(sh, bin(x), fixed(W(x))); });
        const Found f = find_bin(cl, sh, C, rank, turn, false, 0, target);
        turn ^= 1;
        if (f.count <= LIST) {
            border = f.bin;
            listed = f.count;
            ahead = f.ahead;
            before = f.before;
        } else {
            last = search(false, target, last);
            xc = value_of(top - (unsigned)(last >> 32));
            ic = (unsigned)last;
        }
        all_ranks = false;
    }

    // ---- the draw: a warp sums its stretch's kept weights, all CTAs get all sums (and the list)
    auto weigh = [&](float x, float& w) {
        if (x < least_x) return false;
        w = W(x);
        return w >= least;
    };
    Sum s;
    unsigned added = 0, count = 0;  // weights in s, tokens kept
    if (all_ranks && !(least > 0.f)) {
        each([&](float x, int) {
            s.add(W(x));
            ++added;
            count += x > -INFINITY;
        });
    } else if (border >= 0 && plain_ranks && !(least > 0.f)) {
        dense([&](float x, int) { return bin.above(x, border); },
              [&](float x) {
                  s.add(W(x));
                  ++added;
              });
        count = added;
    } else {
        dense([&](float x, int i) { return (border < 0 || bin.above(x, border)) && x >= least_x && up_to_last(x, i); },
              [&](float x) {
                  const float w = W(x);
                  if (w >= least) {
                      s.add(w);
                      ++added;
                  }
              });
        count = added;
    }
    if (border >= 0) {
        for (int v = v0; v < v1; v += 32) {
            float x[E];
            unsigned in = 0;
            if (v + lane < v1) {
                unpack(x, xs[v + lane]);
                if (plain_ranks) {
#pragma unroll
                    for (int e = 0; e < E; ++e) in |= (unsigned)(x[e] >= low_x && bin.in(x[e], border)) << e;
                } else {
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        in |= (unsigned)(x[e] >= low_x && bin.in(x[e], border) && up_to_last(x[e], i0 + (v + lane) * E + e)) << e;
                }
            }
            put(v, x, in);
        }
    }
    u64 sum = s.value(added);
    count = __reduce_add_sync(0xffffffffu, count);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane < C) cl.map_shared_rank(sh.sums, lane)[rank * SW + warp] = sum;
    if (lane == 0) atomicAdd(&sh.my_kept, count);
    __syncthreads();
    if (border >= 0) deliver(C, ahead);
    if (tid < C) cl.map_shared_rank(sh.kept, tid)[rank] = sh.my_kept;
    cl.sync();
    unsigned kept = 0;
    for (int c = 0; c < C; ++c) kept += sh.kept[c];
    if (border >= 0) {
        // the border's tokens in rank order; those kept join their stretches
        const int n_l = (int)listed;
        order_list(sh.list, n_l);
        const int each_l = (n_l + ST - 1) / ST, a0 = min(n_l, tid * each_l), a1 = min(n_l, a0 + each_l);
        u64 mass = 0, all;
        for (int i = a0; i < a1; ++i) mass += fixed(W(value_of(top - (unsigned)(sh.list[i] >> 32))));
        u64 run = before + block_excl(mass, sh.warp_sum, all);
        unsigned keeps = 0;
        for (int i = a0; i < a1; ++i) {
            const float x = value_of(top - (unsigned)(sh.list[i] >> 32));
            const float w = W(x);
            const u64 f = fixed(w);
            if (run < target) {
                if (run + f >= target || i == n_l - 1) sh.last = sh.list[i];  // the last rank kept
                if (w >= least) {
                    const int j = (int)(unsigned)sh.list[i], c = j / p.slice, v = (j - c * p.slice) / E;
                    const int nvc = (min(p.V, (c + 1) * p.slice) - c * p.slice + E - 1) / E;
                    // the warp whose stretch holds vector v of CTA c: floor(nvc w / SW) <= v
                    int w8 = (int)(((long long)v * SW + SW - 1) / nvc);
                    while ((int)((long long)nvc * w8 / SW) > v) --w8;
                    while ((int)((long long)nvc * (w8 + 1) / SW) <= v) ++w8;
                    atomicAdd(&sh.sums[c * SW + w8], f);
                    ++keeps;
                }
            }
            run += f;
        }
        u64 n_k;
        block_excl(keeps, sh.warp_sum, n_k);
        kept += (unsigned)n_k;
        last = sh.last;
        xc = value_of(top - (unsigned)(last >> 32));
        ic = (unsigned)last;
    }
    // running sums over all stretches of the row, in index order
    u64 total;
    u64 at = block_excl(tid < C * SW ? sh.sums[tid] : 0, sh.warp_sum, total);
    // u total lies at or above the running sum of every token before the drawn one
    const u64 pick = part_of(u, total, false);
    if (tid < C * SW && at <= pick && at + sh.sums[tid] > pick) sh.cross_bin = tid, sh.cross_before = at;
    __syncthreads();
    if ((int)sh.cross_bin / SW == rank) {
        // The stretch is this CTA's: its warps sum a part of it each, and the one that u falls into walks that.
        const int w = (int)sh.cross_bin % SW;
        const int s0 = (int)((long long)nv * w / SW), s1 = (int)((long long)nv * (w + 1) / SW);
        const int a0 = s0 + (s1 - s0) * warp / SW, a1 = s0 + (s1 - s0) * (warp + 1) / SW;
        auto weight_of = [&](const float (&x)[E], int v, Sum& mine, unsigned& some) {  // of the kept ones of vector v
            float y;
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (up_to_last(x[e], i0 + v * E + e) && weigh(x[e], y)) mine.add(y), ++some;
        };
        Sum part;
        unsigned parts = 0;
        for (int v = a0 + lane; v < a1; v += 32) {
            float x[E];
            unpack(x, xs[v]);
            weight_of(x, v, part, parts);
        }
        u64 mine = part.value(parts), all;
#pragma unroll
        for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
        u64 seen = block_excl(lane == 0 ? mine : 0, sh.warp_sum, all);
        seen = sh.cross_before + __shfl_sync(0xffffffffu, seen, 0);
        if (seen <= pick && seen + mine > pick) {  // one warp
            for (int v = a0; v < a1 && seen <= pick; v += 32) {
                const int i = i0 + (v + lane) * E;
                float y;
                Sum some;
                unsigned number = 0;
                if (v + lane < a1) {
                    float x[E];
                    unpack(x, xs[v + lane]);
                    weight_of(x, v + lane, some, number);
                }
                const u64 f = some.value(number), incl = warp_incl(f);
                u64 run = seen + incl - f;
                seen += __shfl_sync(0xffffffffu, incl, 31);
                if (run <= pick && run + f > pick) {  // one lane
#pragma unroll 1
                    for (int e = 0; e < E; ++e) {
                        float x;
                        if constexpr (DT == MK_DT_F32) x = reinterpret_cast<const float*>(xs)[(v + lane) * E + e];
                        else x = value(reinterpret_cast<const uint16_t*>(xs)[(v + lane) * E + e]);
                        if (!up_to_last(x, i + e) || !weigh(x, y)) continue;
                        const u64 g = fixed(y);
                        if (run <= pick && run + g > pick) {
                            p.tokens[row] = i + e;
                            if (p.probs) p.probs[row] = (float)((double)y * 0x1p42 / (double)total);
                        }
                        run += g;
                    }
                }
            }
        }
    }
    if (rank == 0 && tid == 0 && p.kept) p.kept[row] = (int)kept;
}

constexpr int MAX_DEV = 32;
constexpr size_t RESERVED = 1024;  // shared memory that the system takes of every CTA
struct Device {
    int sms, smem;  // SMs, and the shared memory of each
};
// asked for once on each device
cudaError_t device_facts(int dev, Device& out) {
    static std::atomic<int> sms[MAX_DEV], smem[MAX_DEV];
    if (dev < MAX_DEV && (out.smem = smem[dev].load(std::memory_order_acquire))) {
        out.sms = sms[dev].load(std::memory_order_relaxed);
        return cudaSuccess;
    }
    cudaError_t e = cudaDeviceGetAttribute(&out.sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&out.smem, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev);
    if (e == cudaSuccess && dev < MAX_DEV) {
        sms[dev].store(out.sms, std::memory_order_relaxed);
        smem[dev].store(out.smem, std::memory_order_release);
    }
    return e;
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
    if (off_by4(a->u, a->temperature, a->top_k, a->top_p, a->min_p, a->tokens, a->probs, a->kept))
        return fail(MK_ERR_INVALID_ARG, "sample: a 32-bit array is not aligned to 4 bytes");
    constexpr int most = MAXC * (MAX_SLICE_B / 4);
    if (a->vocab > most) return fail(MK_ERR_UNSUPPORTED, "sample: vocab above %d", most);
    if (a->rows > INT32_MAX / MAXC) return fail(MK_ERR_UNSUPPORTED, "sample: too many rows");
    SampleP p;
    p.logits = a->logits, p.row_stride = a->row_stride, p.u = a->u, p.temperature = a->temperature;
    p.top_k = a->top_k, p.top_p = a->top_p, p.min_p = a->min_p;
    p.tokens = a->tokens, p.probs = a->probs, p.kept = a->kept;
    p.V = a->vocab;
    // a slice of 2048 tokens keeps a CTA's threads busy with 4 each; where the
    // rows fill the device anyway, larger slices that still leave two CTAs an SM.
    // 256 bf16 rows of 151936, a quarter of them with top-p over the whole
    // vocabulary, take 115 us so, 170 with 8 CTAs a row and 121 with slices that
    // leave one CTA an SM; 512 fp32 rows of 64000 159, 271 and 162; 200 fp32 rows
    // of 8000 31, 47 and 27
    int C = MAXC;
    while (C > 1 && a->vocab <= 2048 * (C / 2)) C /= 2;
    int dev = 0;
    Device of;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess) err = device_facts(dev, of);
    if (err != cudaSuccess) return cuda_status(err, "mk_sample");
    auto slice_of = [&](int c) { return ((a->vocab + c - 1) / c + 7) / 8 * 8; };  // whole 16-byte vectors
    auto smem_of = [&](int c) { return (sizeof(Shared) + 15) / 16 * 16 + (size_t)slice_of(c) * e; };
    auto ctas_of = [&](int c) { return 2 * (smem_of(c) + RESERVED) <= (size_t)of.smem ? 2 : 1; };  // of an SM
    while (C > 1 && (int64_t)a->rows * (C / 2) >= 2 * of.sms && ctas_of(C / 2) == 2) C /= 2;
    p.slice = slice_of(C);
    // More rows than run at once: in the order of their cost. 256 bf16 rows of
    // 151936, an eighth of them costly, take 99 us so and 125 in the order they
    // come, 30 fp32 rows of 300000, one CTA an SM, 97 and 111; where all cost the
    // same 86 and 82 (195 and 192), and 200 fp32 rows of 8000, whose slices of
    // 16 KB are quickly done, 27 and 25. With more waves of rows the last one
    // counts for less.
    p.rows = a->rows;
    p.order = a->top_p && (int64_t)a->rows * C > of.sms * ctas_of(C) && a->rows <= 4 * ST && p.slice * e >= 32768;
    auto kern = a->dtype == MK_DT_F32    ? sample_kernel<MK_DT_F32>
                : a->dtype == MK_DT_BF16 ? sample_kernel<MK_DT_BF16>
                                         : sample_kernel<MK_DT_F16>;
    const size_t smem = smem_of(C);
    // the kernel's shared-memory limit, raised once on each device
    static std::atomic<bool> raised[MAX_DEV][3];
    if (dev >= MAX_DEV || !raised[dev][a->dtype].load()) {
        err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   (int)((sizeof(Shared) + 15) / 16 * 16 + MAX_SLICE_B));
        if (err == cudaSuccess && dev < MAX_DEV) raised[dev][a->dtype] = true;
    }
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
