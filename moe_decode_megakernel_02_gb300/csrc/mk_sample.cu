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
//          from below (to a bin of 1/8 octave); the few tokens above go to a
//          list in one CTA, which ranks them and does all the rest.
//   top-p  one pass sums all weights; a token lighter than (1 - p) sum / V
//          cannot be kept, the others fill a histogram of masses (1/8 octave);
//          the bin where the mass reaches p goes to the list, which gives the
//          last rank kept.
//   Where a list would not fit (long runs of nearly equal logits, a large k),
//   the border is searched by histograms over 12, 12 and 8 bits of the
//   distance, and what is left at one exact value are ties, taken by index.
// Then the kept weights are summed a warp a stretch of tokens, and the warp
// whose stretch u falls into walks it.
//
// A row is one thread-block cluster of C CTAs: each keeps its slice of the row
// in shared memory as it came, so the logits are read from HBM once however
// many passes follow; sums, histograms and lists meet through distributed
// shared memory.
#include <cooperative_groups.h>

#include <type_traits>

#include "mk_ops.cuh"

namespace {

using namespace mkop;
namespace cg = cooperative_groups;

constexpr int ST = 512;        // threads of a CTA
constexpr int SW = ST / 32;
constexpr int BINS = 4096;     // histogram bins (12 bits a level)
constexpr int LIST = BINS;     // ranks a list holds
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
};

struct Shared {
    union {
        u64 hist[BINS];     // masses, or counts
        u64 list[LIST];     // ranks
    };
    u64 warp_sum[SW];
    u64 part[MAXC];         // a total of each CTA of the cluster, written by that CTA
    u64 cross_before;       // a level's result, written by the CTA that has it
    u64 last;               // the last rank kept
    unsigned cross_bin;
    unsigned top, argmax, bad;
    unsigned kept[MAXC];
    unsigned list_n;
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
    float m, T, r;
    bool plain;  // T far from the ends of the range: the quotient by remainder (Markstein 1990) is the divided one
    __device__ __forceinline__ float operator()(float x) const {
        const float d = x - m;
        if (!plain) return expf(__fdiv_rn(d, T));
        const float q = d * r;
        // far below the smallest 32-bit number: also keeps overflowed quotients out of the remainder
        if (q < -150.f) return 0.f;
        return expf(__fmaf_rn(__fmaf_rn(-q, T, d), r, q));
    }
};

// Sums of w 2^42 (0 <= w <= 1) over up to 400 weights in two 32-bit integers:
// adding 24 leaves w in steps of 2^-19 in the low bits of the sum, adding
// 1.5 2^-19 what is left of it in steps of 2^-42.
struct Sum {
    unsigned hi = 0, lo = 0, n = 0;
    __device__ __forceinline__ void add(float w) {
        const float a = w + 24.0f;
        const float b = (w - (a - 24.0f)) + 0x1.8p-19f;
        hi += __float_as_uint(a);
        lo += __float_as_uint(b);
        ++n;
    }
    __device__ __forceinline__ u64 value() const {
        const unsigned h = hi - n * 0x41c00000u;       // the bits of 24
        const int l = (int)(lo - n * 0x36400000u);     // and of 1.5 2^-19
        return ((u64)h << 23) + (u64)(long long)l;
    }
};
__device__ __forceinline__ u64 fixed(float w) {
    Sum s;
    s.add(w);
    return s.value();
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

// The cluster's sum of one number a thread, and the sum over the threads before
// this one. The next call overwrites the parts: a cluster barrier lies between
// any two.
__device__ u64 cluster_sum(cg::cluster_group& cl, Shared& sh, int C, int rank, u64 v, u64& before) {
    u64 mine;
    before = block_excl(v, sh.warp_sum, mine);
    if ((int)threadIdx.x < C) cl.map_shared_rank(sh.part, threadIdx.x)[rank] = mine;
    cl.sync();
    u64 total = 0;
    for (int c = 0; c < C; ++c) {
        if (c == rank) before += total;
        total += sh.part[c];
    }
    return total;
}

// One level of the search over the cluster's histograms: the bin at which the
// running sum, `before` in front of bin 0, reaches `target`; `before` becomes
// the sum in front of that bin.
__device__ unsigned find_bin(cg::cluster_group& cl, Shared& sh, int C, int rank, u64& before, u64 target) {
    cl.sync();  // every CTA's histogram is complete
    const int per = BINS / C, each = per / ST;  // bins of this CTA, of a thread
    u64 mine = 0, bins[BINS / ST];
    const int b0 = rank * per + threadIdx.x * each;
#pragma unroll
    for (int i = 0; i < BINS / ST; ++i) {
        bins[i] = 0;
        if (i < each)
            for (int c = 0; c < C; ++c) bins[i] += cl.map_shared_rank(sh.hist, c)[b0 + i];
        mine += bins[i];
    }
    u64 at;
    cluster_sum(cl, sh, C, rank, mine, at);  // its barrier: histograms have been read
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

// v[0 .. n) ascending; `n2` a power of two not below n, padded with ~0 here
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
// the same for up to ST numbers, all different: each thread finds its own one's place
__device__ void rank_list(u64* v, int n) {
    const int i = threadIdx.x;
    const u64 x = i < n ? v[i] : ~0ull;
    int at = 0;
    for (int j = 0; j < n; ++j) at += v[j] < x;
    __syncthreads();
    if (i < n) v[at] = x;
    __syncthreads();
}
__device__ void order_list(u64* v, int n) {
    if (n <= ST) {
        rank_list(v, n);
    } else {
        int n2 = 2 * ST;
        while (n2 < n) n2 *= 2;
        sort_list(v, n, n2);
    }
}

// Bound: one read of the logits from HBM, then passes over shared memory of 4
// to 25 operations a token (the largest: summing all weights). Small calls are
// the latency of 5 to 12 cluster barriers.
template <int DT>
__global__ void __launch_bounds__(ST, 2) sample_kernel(const SampleP p) {
    typedef typename std::conditional<DT == MK_DT_F32, float, uint16_t>::type Raw;
    constexpr int E = 16 / sizeof(Raw);  // logits of a 16-byte vector
    extern __shared__ __align__(16) uint8_t smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    uint4* const xs = reinterpret_cast<uint4*>(smem + (sizeof(Shared) + 15) / 16 * 16);
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const long long row = blockIdx.x / C;
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

    // ---- the slice into shared memory; this thread's largest logit
    if (tid == 0) sh.top = 0, sh.bad = 0, sh.argmax = 0xffffffffu, sh.list_n = 0;
    __syncthreads();
    float big = -INFINITY;
    bool bad = false;
    {
        const Raw* src = (const Raw*)p.logits + row * p.row_stride + i0;
        const Raw fill = DT == MK_DT_F32 ? (Raw)0 : DT == MK_DT_BF16 ? (Raw)0xff80 : (Raw)0xfc00;  // -infinity
        Raw* raw = reinterpret_cast<Raw*>(xs);
        const int whole = (uintptr_t)src % 16 == 0 ? n / E : 0;
#pragma unroll 4
        for (int i = tid; i < whole; i += ST) {
            const uint4 a = __ldcs(reinterpret_cast<const uint4*>(src) + i);
            xs[i] = a;
            float x[E];
            unpack(x, a);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                big = fmaxf(big, x[e]);
                bad |= !(x[e] < INFINITY);  // NaN or +infinity
            }
        }
        for (int i = whole * E + tid; i < nv * E; i += ST) {
            if (i < n) {
                const Raw a = src[i];
                raw[i] = a;
                float x;
                if constexpr (DT == MK_DT_F32) x = a;
                else x = value(a);
                big = fmaxf(big, x);
                bad |= !(x < INFINITY);
            } else if constexpr (DT == MK_DT_F32) {
                raw[i] = -INFINITY;  // the last vector's rest is masked
            } else {
                raw[i] = fill;
            }
        }
    }
    {
        unsigned k = key_of(big);
#pragma unroll
        for (int o = 16; o; o >>= 1) k = max(k, __shfl_xor_sync(0xffffffffu, k, o));
        if (lane == 0) atomicMax(&sh.top, k);
        if (bad) sh.bad = 1;
    }
    cl.sync();
    unsigned top = 0, any_bad = 0;
    for (int c = 0; c < C; ++c) {
        top = max(top, *cl.map_shared_rank(&sh.top, c));
        any_bad |= *cl.map_shared_rank(&sh.bad, c);
    }
    const float m = value_of(top);
    const float T = p.temperature ? p.temperature[row] : 1.0f;
    const bool none = any_bad || m == -INFINITY;  // a NaN, a +infinity, or nothing but masked tokens

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

    // the lowest index of the largest logit: rank 0, which always stays
    if (!none && sh.top == top) {
        for (int v = tid; v < nv; v += ST) {
            float x[E];
            unpack(x, xs[v]);
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (x[e] == m) atomicMin(&sh.argmax, (unsigned)(i0 + v * E + e));
        }
    }
    cl.sync();
    unsigned argmax = 0xffffffffu;
    for (int c = 0; c < C; ++c) argmax = min(argmax, *cl.map_shared_rank(&sh.argmax, c));
    if (none || !(T > 0.f)) {
        if (rank == 0 && tid == 0) {
            p.tokens[row] = none ? -1 : (int)argmax;
            if (p.probs) p.probs[row] = none ? 0.f : 1.f;
            if (p.kept) p.kept[row] = none ? 0 : 1;
        }
        cl.sync();  // no CTA leaves while another reads its shared memory
        return;
    }
    const Weight W = {m, T, __frcp_rn(T), T > 0x1p-60f && T < 0x1p60f};
    const int k_in = p.top_k ? p.top_k[row] : 0;
    const float p_in = p.top_p ? p.top_p[row] : 1.0f;
    const float least = p.min_p ? p.min_p[row] : 0.0f;
    const bool by_k = k_in > 0 && k_in < p.V, by_p = p_in < 1.0f;
    const float u = fminf(fmaxf(p.u[row], 0.f), 0x1.fffffep-1f);
    const unsigned masked = top - key_of(-INFINITY);
    auto mass_target = [&](u64 total) {  // the mass that ends top-p; at least 1: the first rank always stays
        return max(1ull, (u64)ceil(fmax((double)p_in, 0.0) * (double)total));
    };
    // the least logit at a distance of at most d
    auto at_distance = [&](unsigned d) { return value_of(top - min(d, masked)); };
    // Ranks of the unmasked tokens with low <= x < high, to the first CTA's list; returns how many there are
    // (those that do not fit counted).
    auto collect = [&](float low, float high) {
        u64* list = cl.map_shared_rank(sh.list, 0);
        unsigned* count = cl.map_shared_rank(&sh.list_n, 0);
        each([&](float x, int i) {
            if (x >= low && x < high && x > -INFINITY) {
                const unsigned at = atomicAdd(count, 1u);
                if (at < LIST) list[at] = (u64)(top - key_of(x)) << 32 | (unsigned)i;
            }
        });
        cl.sync();
        const unsigned got = *count;
        cl.sync();  // read everywhere: the first CTA may go on, and leave
        return got;
    };
    // The token at place `quota` (from 1) among those exactly at distance d, by index: its rank.
    auto nth_tie = [&](unsigned d, u64 quota) {
        const float x0 = value_of(top - d);
        unsigned c = 0;
        each([&](float x, int) { c += x == x0; });
        c = __reduce_add_sync(0xffffffffu, c);
        u64 at;
        const u64 all = cluster_sum(cl, sh, C, rank, lane == 0 ? c : 0, at);
        // lanes past 0 come after their warp's count
        at = __shfl_sync(0xffffffffu, at, 0);
        const u64 want = min(quota, all);
        if (at < want && at + c >= want) {  // one warp of the cluster
            u64 seen = at;
            for (int v = v0; v < v1 && seen < want; v += 32) {
                float x[E];
                const bool in = v + lane < v1;
                if (in) unpack(x, xs[v + lane]);
                unsigned mine = 0;
#pragma unroll
                for (int e = 0; e < E; ++e) mine += in && x[e] == x0;
                u64 before = seen + warp_incl(mine) - mine;
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (in && x[e] == x0 && ++before == want)
                        for (int r = 0; r < C; ++r)
                            *cl.map_shared_rank(&sh.last, r) = (u64)d << 32 | (unsigned)(i0 + (v + lane) * E + e);
                seen += __reduce_add_sync(0xffffffffu, mine);
            }
        }
        cl.sync();
        return sh.last;
    };

    // kept: ranks up to `last` (and weights of at least min_p)
    u64 last = ((u64)masked << 32) - 1;  // masked tokens are never kept
    bool listed = false;                 // rank 0's list holds all tokens top-k keeps, and maybe more
    if (by_k) {
        const int holders = min(p.V, C * ST);
        unsigned bin = masked >> 20;
        u64 before = 0;
        clear_hist(sh);
        if (k_in <= holders / 4) {
            // at least k tokens lie at or above the k-th largest of the threads' maxima
            if (big > -INFINITY) atomicAdd(reinterpret_cast<unsigned*>(&sh.hist[(top - key_of(big)) >> 20]), 1u);
        } else {
            each([&](float x, int) {
                if (x > -INFINITY) atomicAdd(reinterpret_cast<unsigned*>(&sh.hist[(top - key_of(x)) >> 20]), 1u);
            });
        }
        if (tid == 0) sh.cross_bin = masked >> 20;  // fewer than k: every unmasked token
        bin = find_bin(cl, sh, C, rank, before, (u64)k_in);
        const unsigned got = collect(at_distance(bin << 20 | 0xfffffu), INFINITY);
        listed = got <= LIST;
        if (!listed) {
            // the k-th rank by three levels of counts
            u64 ahead = 0;
            unsigned prefix = 0;
            bool found = true;
#pragma unroll 1
            for (int l = 0; l < 3 && found; ++l) {
                const int lo = l == 0 ? 20 : l == 1 ? 8 : 0, up = l == 0 ? 32 : l == 1 ? 20 : 8;
                clear_hist(sh);
                each([&](float x, int) {
                    const unsigned d = top - key_of(x);
                    if (x > -INFINITY && (l == 0 || (d >> up) == prefix))
                        atomicAdd(reinterpret_cast<unsigned*>(&sh.hist[(d >> lo) & ((1u << (up - lo)) - 1)]), 1u);
                });
                if (tid == 0) sh.cross_bin = 0xffffffffu;
                const unsigned b = find_bin(cl, sh, C, rank, ahead, (u64)k_in);
                found = b != 0xffffffffu;
                prefix = prefix << (up - lo) | b;
            }
            if (found) last = nth_tie(prefix, (u64)k_in - ahead);
        }
    }

    if (listed) {
        // ---- rank 0 has every candidate: the other CTAs are done
        if (rank == 0) {
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
                if (i == 0 || (run < target && w >= least)) ++keeps;
                run += fixed(w);
            }
            u64 n_k;
            block_excl(keeps, sh.warp_sum, n_k);
            // in index order now: (index, distance)
            for (int i = tid; i < (int)n_k; i += ST) sh.list[i] = sh.list[i] << 32 | sh.list[i] >> 32;
            __syncthreads();
            order_list(sh.list, (int)n_k);
            const int each_k = ((int)n_k + ST - 1) / ST, b0 = min((int)n_k, tid * each_k), b1 = min((int)n_k, b0 + each_k);
            mass = 0;
            for (int i = b0; i < b1; ++i) mass += fixed(W(value_of(top - (unsigned)sh.list[i])));
            run = block_excl(mass, sh.warp_sum, total);
            const u64 pick = (u64)((double)u * (double)total);
            for (int i = b0; i < b1; ++i) {
                const float w = W(value_of(top - (unsigned)sh.list[i]));
                const u64 f = fixed(w);
                if (run <= pick && run + f > pick) {
                    p.tokens[row] = (int)(sh.list[i] >> 32);
                    if (p.probs) p.probs[row] = (float)((double)w * 0x1p42 / (double)total);
                }
                run += f;
            }
            if (tid == 0 && p.kept) p.kept[row] = (int)n_k;
        }
        return;
    }

    const float least_x = least > 0.f ? m + T * (logf(fminf(least, 1.f)) - 0.01f) : -INFINITY;  // below: lighter than min_p
    if (by_p) {
        // all of top-k's mass
        const float xk = value_of(top - (unsigned)(last >> 32));
        const unsigned ik = (unsigned)last;
        Sum s;
        each([&](float x, int i) {
            if (x > xk || (x == xk && (unsigned)i <= ik)) s.add(W(x));
        });
        u64 at, before = 0;
        const u64 total = cluster_sum(cl, sh, C, rank, s.value(), at);
        const u64 target = mass_target(total);
        // Tokens lighter than (1 - p) total / V weigh less than (1 - p) total together: at least p total lies
        // before them. Half of that bound, and a hundredth, leave room for roundings.
        const double light = (1.0 - fmax((double)p_in, 0.0)) * (double)total * 0x1p-43 / (double)p.V;
        const float low_x = light > 1e-30 ? m + T * (logf((float)light) - 0.01f) : -INFINITY;
        clear_hist(sh);
        each([&](float x, int i) {
            if (x >= low_x && (x > xk || (x == xk && (unsigned)i <= ik))) {
                const u64 w = fixed(W(x));
                if (w) atomicAdd(&sh.hist[(top - key_of(x)) >> 20], w);
            }
        });
        unsigned prefix = find_bin(cl, sh, C, rank, before, target);
        const float high = prefix ? at_distance((prefix << 20) - 1) : INFINITY, low = at_distance(prefix << 20 | 0xfffffu);
        if (tid == 0) sh.list_n = 0;
        cl.sync();
        const unsigned got = collect(low, high);  // hist is free: find_bin's barriers are behind
        if (got <= LIST) {
            if (rank == 0) {
                int n_l = (int)got;
                order_list(sh.list, n_l);
                const int each_l = (n_l + ST - 1) / ST, a0 = min(n_l, tid * each_l), a1 = min(n_l, a0 + each_l);
                u64 mass = 0, all;
                for (int i = a0; i < a1; ++i)
                    if (sh.list[i] <= last) mass += fixed(W(value_of(top - (unsigned)(sh.list[i] >> 32))));
                u64 run = before + block_excl(mass, sh.warp_sum, all);
                for (int i = a0; i < a1; ++i) {
                    if (sh.list[i] > last) break;
                    const u64 f = fixed(W(value_of(top - (unsigned)(sh.list[i] >> 32))));
                    // the last one with less than the target before it
                    if (run < target && run + f >= target)
                        for (int r = 0; r < C; ++r) *cl.map_shared_rank(&sh.last, r) = sh.list[i];
                    run += f;
                }
            }
            cl.sync();
            last = sh.last;
        } else {
            unsigned p2 = prefix;
#pragma unroll 1
            for (int l = 1; l < 3; ++l) {
                const int lo = l == 1 ? 8 : 0, up = l == 1 ? 20 : 8;
                clear_hist(sh);
                each([&](float x, int i) {
                    const unsigned d = top - key_of(x);
                    if ((d >> up) == p2 && (x > xk || (x == xk && (unsigned)i <= ik))) {
                        const u64 w = fixed(W(x));
                        if (w) atomicAdd(&sh.hist[(d >> lo) & ((1u << (up - lo)) - 1)], w);
                    }
                });
                p2 = p2 << (up - lo) | find_bin(cl, sh, C, rank, before, target);
            }
            // ties at the border: as many as have less than the target before
            // them (their weight is not 0: the bin was found by its mass)
            const u64 w = fixed(W(value_of(top - p2)));
            last = min(last, nth_tie(p2, (target - before + w - 1) / w));
        }
    }

    // ---- the draw: a warp sums its stretch, the one that u falls into walks it
    const float xc = value_of(top - (unsigned)(last >> 32));
    const unsigned ic = (unsigned)last;
    auto weigh = [&](float x, int i, float& w) {
        if (!(x > xc || (x == xc && (unsigned)i <= ic)) || (x < least_x && i != (int)argmax)) return false;
        w = W(x);
        return w >= least || i == (int)argmax;
    };
    Sum s;
    each([&](float x, int i) {
        float w;
        if (weigh(x, i, w)) s.add(w);
    });
    u64 sum = s.value();
    unsigned count = __reduce_add_sync(0xffffffffu, s.n);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    u64 at, slice_kept;
    block_excl(lane == 0 ? count : 0, sh.warp_sum, slice_kept);
    if (tid < C) cl.map_shared_rank(sh.kept, tid)[rank] = (unsigned)slice_kept;
    cl.sync();  // the parts of an earlier sum have been read
    const u64 total = cluster_sum(cl, sh, C, rank, lane == 0 ? sum : 0, at);
    at = __shfl_sync(0xffffffffu, at, 0);
    // u total lies at or above the running sum of every token before the drawn one
    const u64 pick = (u64)((double)u * (double)total);
    if (at <= pick && at + sum > pick) {  // one warp of the cluster
        const int per = (v1 - v0 + 31) / 32, a0 = min(v1, v0 + lane * per), a1 = min(v1, a0 + per);
        Sum mine;
        for (int v = a0; v < a1; ++v) {
            float x[E], w;
            unpack(x, xs[v]);
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (weigh(x[e], i0 + v * E + e, w)) mine.add(w);
        }
        u64 run = mine.value();
        run = at + warp_incl(run) - run;
        if (run <= pick && run + mine.value() > pick) {
            for (int v = a0; v < a1; ++v) {
                float x[E], w;
                unpack(x, xs[v]);
                for (int e = 0; e < E; ++e) {
                    if (!weigh(x[e], i0 + v * E + e, w)) continue;
                    const u64 f = fixed(w);
                    if (run <= pick && run + f > pick) {
                        p.tokens[row] = i0 + v * E + e;
                        if (p.probs) p.probs[row] = (float)((double)w * 0x1p42 / (double)total);
                    }
                    run += f;
                }
            }
        }
    }
    if (rank == 0 && tid == 0 && p.kept) {
        unsigned kept = 0;
        for (int c = 0; c < C; ++c) kept += sh.kept[c];
        p.kept[row] = (int)kept;
    }
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
    constexpr int most = MAXC * (MAX_SLICE_B / 4);
    if (a->vocab > most) return fail(MK_ERR_UNSUPPORTED, "sample: vocab above %d", most);
    if (a->rows > INT32_MAX / MAXC) return fail(MK_ERR_UNSUPPORTED, "sample: too many rows");
    SampleP p;
    p.logits = a->logits, p.row_stride = a->row_stride, p.u = a->u, p.temperature = a->temperature;
    p.top_k = a->top_k, p.top_p = a->top_p, p.min_p = a->min_p;
    p.tokens = a->tokens, p.probs = a->probs, p.kept = a->kept;
    p.V = a->vocab;
    // a slice of 2048 tokens keeps a CTA's threads busy with 4 each; where the
    // rows fill the device anyway, larger slices that still leave two CTAs an SM
    int C = MAXC;
    while (C > 1 && a->vocab <= 2048 * (C / 2)) C /= 2;
    while (C > 1 && a->rows * (C / 2) >= 304 && ((int64_t)a->vocab * e + C / 2 - 1) / (C / 2) <= 78 * 1024) C /= 2;
    p.slice = ((a->vocab + C - 1) / C + 7) / 8 * 8;  // whole 16-byte vectors
    auto kern = a->dtype == MK_DT_F32    ? sample_kernel<MK_DT_F32>
                : a->dtype == MK_DT_BF16 ? sample_kernel<MK_DT_BF16>
                                         : sample_kernel<MK_DT_F16>;
    const size_t smem = (sizeof(Shared) + 15) / 16 * 16 + (size_t)p.slice * e;
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
