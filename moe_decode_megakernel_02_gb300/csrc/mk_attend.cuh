// mk_attend.cuh -- attention of a few new tokens a sequence over paged K and
// V (mk_pages_attend).
//
// For one query row (a token and a query head) and the positions j it sees,
//   x_j = cap(scale q.k_j) - slope (p - j),  m = max x_j,
//   out = sum_j e^(x_j - m) v_j / sum_j e^(x_j - m),
// in one pass: a running maximum, the sum and the output rescaled when the
// maximum rises. Both products run transposed on the tensor cores
// (m16n8k16): 16 positions by 8 rows of scores, then 16 values by 8 rows of
// output, so that a decode step's 1 to 8 query heads of a kv head fill the
// 8-wide side, K and V fragments are each used once per 8 rows, and a thread
// keeps the same two rows from the scores to the output.
//
// One loop over 64-position tiles (cp.async ring in shared memory); a CTA's
// warps split a tile's positions WP ways and the item's rows WR ways:
//   4 x 1, 4 x 2  up to 8, 16 or 32 rows an item, the usual decode and verify
//                 steps. Bound by the cache's bytes.
//   2 x 4, 1 x 8  64 or 128 rows: chunks of prompts, and a shared prefix, where
//                 the rows of all sequences stand against one copy of K and V;
//                 only where mk_prefix.cuh has no kernel, or for tiles that not
//                 every row sees whole. Bound by the tensor cores and what feeds
//                 them.
// Warps of the same rows hold maxima, sums and outputs of their own positions,
// which meet at the item's end.
//
// Work is cut by tiles, not by sequences: the tiles of all items (sequence,
// kv head, row block) are numbered in one line and every CTA takes an equal
// stretch of it, whatever the lengths are; lengths are read on the device, so
// a captured graph keeps working as they grow. An item that lies within one
// CTA is finished by it; pieces of an item leave (output, maximum, sum) in the
// workspace and a second launch joins them. Small calls, whose time is the
// latency of launches, give every item a cluster of 1 to 8 CTAs instead, which
// join through distributed shared memory: one launch, no workspace.
//
// Measured, 128-wide heads, 40 query heads on 8: 64 sequences of up to 32768
// positions, E4M3, 490 us (5.8 TB/s, 86 % of what a copy reaches); 32 such in
// bf16 396 us (6.9 TB/s); 64 sequences of up to 1024, bf16, 43 us (58 %: the
// start, the join and the ends of pieces are 10 us of it). 16 query heads on 4:
// one sequence of 4096 14.5 us, all latency; 8 sequences of 8192 with 7 new
// tokens each (28 rows), E4M3 and capped scores, 40 us (12 %): issue and
// latency of the conversions, exponentials and shuffles of 4 times the rows.
//
// Rounding. Scores and sums are 32-bit. bf16 pages: queries are exact in bf16
// (16-bit floats: hi + lo parts), probabilities go in as hi + lo bf16 parts
// (split_bf16), so a product keeps 16 bits. 8-bit pages: codes are exact in fp16; a query
// row is scaled by a power of two into fp16 (exact but for values 2^-24 below
// the row's largest); the K scale multiplies the score, the V scale the
// probability, which goes in as one fp16 (11 bits; hi + lo parts for fp16
// outputs, whose own rounding is as fine), scaled by 2^15 over the largest V
// scale that the row has seen so far: products below 2^-29 of the largest
// possible one fall under fp16's normal range and keep steps of 2^-39 of it.
// (A unit for each row costs 1 % of a long context's time and 5 % of 28 rows'.)
#pragma once
#include <cooperative_groups.h>

#include "mk_tensor.cuh"

namespace mkop {

struct AttendP {
    const uint8_t *k, *v;
    const float *ks, *vs;
    long long page_b, head_b, row_b;  // bytes
    long long sc_page, sc_head;       // floats
    const int* table;
    long long table_s;
    int pps, ps_shift, n_pages;
    const int *lens, *starts;
    const float* slopes;
    const uint16_t* q;
    long long qb, qt, qh;
    uint16_t* out;
    long long ob, ot, oh;
    float* lse;
    int* status;
    int B, T, H, G, f16;
    float scale, cap;
    int shared;      // positions in shared pages: the shared launch covers [0, shared), the other one the rest
    int cluster;     // > 0: one item a cluster of so many CTAs, no pieces in the workspace
    int is_shared;   // this is the shared launch (one virtual sequence, rows of the whole batch)
    int wide;        // the tiles that all of a sequence's rows see whole have a launch of their own (mk_prefix.cuh)
    int RB;          // row blocks of an item
    int rows_item;   // rows of one (sequence, kv head): T * G, or B * T * G
    int keep_items;  // finished items go to the workspace too (a shared part joins them)
    int min_units;   // a CTA's least stretch of tiles
    int slot_rows;   // rows of a slot: slot_rows * D outputs, then (maximum, sum) pairs
    int slot_floats;
    float* slots;    // two of each CTA (its first and its last piece), then one of each item
    int* base;       // [B + 1]: first unit of each sequence, written for the joining launch
    unsigned wait_ns;  // limit of the waits in mk_prefix.cuh, below 4 s
    int skip_signal;   // for tests: one of their signals is left out
};

struct JoinP {
    AttendP own, shared;
    int own_grid, shared_grid;  // CTAs; shared_grid 0: no shared part
    int own_rows, shared_rows;  // rows of a row block
    int shared_units;           // tiles of a shared item
    unsigned rows;              // output rows
    int pieces;                 // of a row, about
};

constexpr int MAX_CLUSTER = 8;
constexpr int JT = 128;  // threads of a joining CTA

// units (tiles) of each CTA when `total` are shared out over `grid`
// (the host keeps totals below 2^30)
__host__ __device__ __forceinline__ int units_each(int total, int grid, int min_units) {
    const int e = (total + grid - 1) / grid;
    return e < min_units ? min_units : e;
}

// Whether all of sequence b's tokens see all of the shared positions: it takes
// part in the shared launch. Others (padding, documents that start inside,
// lengths that end inside) are read on their own, so that the shared launch
// has no row that sees a part.
__device__ __forceinline__ bool shares(const AttendP& p, int b) {
    return p.shared > 0 && (long long)p.lens[b] - p.T + 1 >= p.shared && (!p.starts || p.starts[b] <= 0);
}
// Wide calls: the tiles [g0, g1) of 64 positions of sequence b that all of its tokens see whole
__device__ __forceinline__ void whole_tiles(const AttendP& p, int b, int& g0, int& g1) {
    const unsigned lo = p.starts ? max(p.starts[b], 0) : 0;
    const long long hi = min((long long)p.lens[b] - p.T + 1, (long long)p.pps << p.ps_shift);
    g0 = (int)((lo + 63u) / 64u);
    g1 = max(g0, hi < 0 ? 0 : (int)(hi / 64));
}
// The shared launch: the first sequence that takes part (its table row leads to
// the pages; a padded one's may hold anything), INT_MAX when none does. A whole
// CTA asks, of `threads` threads; `at` is shared memory.
__device__ __forceinline__ int first_sharing(const AttendP& p, int threads, int* at) {
    if (threadIdx.x == 0) *at = INT_MAX;
    __syncthreads();
    for (int b = threadIdx.x; b < p.B; b += threads)
        if (shares(p, b)) {
            atomicMin(at, b);
            break;
        }
    __syncthreads();
    return *at;
}
// the positions of sequence b that a launch covers, [lo, hi)
__device__ __forceinline__ void cover(const AttendP& p, int b, int& lo, int& hi) {
    if (p.is_shared) {
        lo = 0;
        hi = p.shared;
        return;
    }
    lo = shares(p, b) ? p.shared : max(p.starts ? p.starts[b] : 0, 0);
    hi = min(p.lens[b], p.pps << p.ps_shift);
}
template <int TILE>
__device__ __forceinline__ int cover_units(const AttendP& p, int b) {
    int lo, hi;
    cover(p, b, lo, hi);
    if (hi <= lo) return 0;
    int n = (hi + TILE - 1) / TILE - lo / TILE;
    if (p.wide) {
        int g0, g1;
        whole_tiles(p, b, g0, g1);
        n -= g1 - g0;
    }
    return n;
}

__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool ok) {
    const int n = ok ? 4 : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// an 8 x 8 matrix of 16-bit values over the warp, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Capped scores as exponents of 2, cap log2(e) tanh z, from y = 2 z log2(e).
// Below |z| = 1/2 y cap/2 times a polynomial in y^2 (Chebyshev interpolation of
// tanh(sqrt t) / sqrt t on [0, 1/4]: 2^-26 off), so that the error is of the
// score's size however large the cap is; from there on tanh z = 1 - 2 / (e^2z + 1),
// whose 2.8 2^-23 of 1 is relative there too. Most scores lie below: a warp
// whose scores all do skips the exponentials.
constexpr float CAP_NEAR = 1.44f;  // |y| of |z| a little below 1/2
__device__ __forceinline__ float cap_near(float y, float half_cap) {
    const float w = y * y;
    float p = 3.5657851e-6f;
    p = __fmaf_rn(p, w, -9.1816237e-5f);
    p = __fmaf_rn(p, w, 1.9223876e-3f);
    p = __fmaf_rn(p, w, -4.0037432e-2f);
    p = __fmaf_rn(p, w, 1.f);
    return y * half_cap * p;
}
__device__ __forceinline__ float cap_any(float y, float cap) {
    const float c2 = cap * LOG2E;
    return fabsf(y) < CAP_NEAR ? cap_near(y, 0.5f * cap) : c2 - 2.f * c2 * rcp(ex2(y) + 1.f);
}

// Two probabilities as bf16 parts: hi cut off, lo the rest, rounded (16 bits
// together). Neither is negative, and lo is not 0, so that an infinity in V,
// times both parts of a probability above 0, stays that infinity (0 x inf is
// NaN, and so is inf - inf).
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t& hi, uint32_t& lo) {
    hi = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
    lo = pack_bf16(x - __uint_as_float(__float_as_uint(x) & 0xffff0000u), y - __uint_as_float(__float_as_uint(y) & 0xffff0000u));
    asm("max.u16x2 %0, %0, %1;" : "+r"(lo) : "r"(0x00010001u));  // 2^-133, the least one; NaN stays
}

// Four E4M3 codes as two registers of two fp16 values, exact.
__device__ __forceinline__ void e4m3_quad(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
// signed bytes plus 128, set into the mantissa of 1024, give 1152 + code
__device__ __forceinline__ uint32_t int8_half2(uint32_t w) {
    const uint32_t c = 0x64806480u;  // 1152, 1152
    const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&w), *reinterpret_cast<const __half2*>(&c));
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <int FMT>
__device__ __forceinline__ void code_quad(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (FMT == MK_KV_E4M3) {
        e4m3_quad(w, lo, hi);
    } else {
        w ^= 0x80808080u;
        lo = int8_half2(__byte_perm(w, 0x64646464u, 0x4140));
        hi = int8_half2(__byte_perm(w, 0x64646464u, 0x4342));
    }
}

// ROWB bytes of a row in shared memory: 16-byte pieces stored at piece ^ f(row),
// so that eight consecutive rows' pieces lie in different banks
template <int ROWB>
__device__ __forceinline__ uint32_t piece(uint32_t base, int row, int c) {
    const int x = ROWB >= 128 ? (row & 7) : ((row >> 1) & 3);
    return base + row * ROWB + ((c ^ x) << 4);
}

// RN: groups of 8 query rows a warp holds.
template <int D, int FMT, bool SPLITQ, int WP, int WR, int RN>
struct Shape {
    static constexpr bool F8 = FMT != MK_KV_BF16;
    static constexpr int EB = F8 ? 1 : 2;                   // bytes of a cached value
    static constexpr int ROWB = D * EB;                     // bytes of a cached row
    static constexpr int SL = 16;                           // positions a warp takes at once
    static constexpr int TILE = 64;                         // positions of a tile
    static constexpr int NT = 32 * WP * WR;                 // threads
    static constexpr int ROWS = WR * 8 * RN;                // query rows of an item
    static constexpr int TILE_B = TILE * ROWB;              // bytes of K (or V) of a tile
    static constexpr int STAGE_B = 2 * TILE_B + (F8 ? 2 * TILE * 4 : 0);
    static constexpr int Q_B = ROWS * D * 2 * (SPLITQ ? 2 : 1);
    static constexpr int MISC_B = 4096;
    static constexpr int OREGS = RN * D / 4;                // registers of the output
    static constexpr bool QREG = RN * D / 8 * (SPLITQ ? 2 : 1) <= 16 || (NT == 128 && RN * D / 8 * (SPLITQ ? 2 : 1) <= 32);
    // CTAs an SM: what the registers allow, and at least two stages of the ring
    static constexpr int WANT = (OREGS <= 64 ? 4 : 2) * 128 / NT;
    static constexpr int fit(int ctas) { return (227 * 1024 / ctas - 1024 - Q_B - MISC_B) / STAGE_B; }
    static constexpr int CTAS = WANT > 3 && fit(WANT) >= 3 ? WANT : WANT >= 3 && fit(3) >= 2 ? 3 : WANT >= 2 && fit(2) >= 2 ? 2 : 1;
    static constexpr int STAGES = fit(CTAS) > 4 ? 4 : fit(CTAS);
    static constexpr int RING_B = STAGES * STAGE_B;
    static constexpr int SMEM = RING_B + Q_B + MISC_B;
    // the warps' outputs meet in the ring's memory
    static_assert(WP == 1 || (WP * ROWS * D * 4 <= RING_B && (WP + 1) * ROWS * 8 <= Q_B), "too small for the merge");
    static_assert(STAGES >= 2 && SMEM <= 227 * 1024, "ring");
};

// per-row facts, and where the rows of the tiles being fetched lie
template <int ROWS, int TILE>
struct Misc {
    long long off[2][TILE];  // bytes after the head's first row; -1: no such row, zeros
    int scan[8];
    int found_base, found_row;
    float slope2[ROWS];  // slope * log2 e
    float qscale[ROWS];  // 8-bit pages: the power of two taken out of the query
    int lo[ROWS], hi[ROWS], at[ROWS];
    int found_b;
};

// four values of a finished row (of the kv head's rows) from column d on, divided and written
__device__ __forceinline__ void emit(const AttendP& p, int row, int h, int d, const float4& y, float mm, float ll) {
    const int bt = row / p.G, g = row - bt * p.G;
    const int b = bt / p.T, t = bt - b * p.T, hq = h * p.G + g;
    const bool none = ll == 0.f;
    const float inv = none ? 0.f : 1.f / ll;
    const float z[4] = {none ? 0.f : y.x * inv, none ? 0.f : y.y * inv, none ? 0.f : y.z * inv, none ? 0.f : y.w * inv};
    uint16_t* dst = p.out + b * p.ob + t * p.ot + hq * p.oh + d;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        dst[i] = p.f16 ? __half_as_ushort(__float2half_rn(z[i])) : __bfloat16_as_ushort(__float2bfloat16_rn(z[i]));
    if (d == 0 && p.lse)
        p.lse[((long long)b * p.T + t) * (p.H * p.G) + hq] = none ? -INFINITY : (mm + log2f(ll)) * LN2;
}

// Joins an item over its cluster: every CTA has its part of all rows in om and
// (maximum, sum) in ml; each joins its share of the values.
template <int D, int ROWS, int AT>
__device__ __forceinline__ void cluster_join(const AttendP& p, float* om, float* ml, const int* lo, const int* hi, int row0,
                                          int h, int nrows, int rank) {
    namespace cg = cooperative_groups;
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    for (int i = rank * AT + (int)threadIdx.x; i < nrows * (D / 4); i += p.cluster * AT) {
        const int r = i / (D / 4), d = (i % (D / 4)) * 4;
        float4 z[MAX_CLUSTER];
        float2 a[MAX_CLUSTER];
#pragma unroll
        for (int c = 0; c < MAX_CLUSTER; ++c)  // all at once: each is a round trip through the cluster
            if (c < p.cluster) {
                z[c] = *reinterpret_cast<const float4*>(cl.map_shared_rank(om, c) + r * D + d);
                a[c] = *reinterpret_cast<const float2*>(cl.map_shared_rank(ml, c) + 2 * r);
            }
        float mm = -INFINITY, ll = 0.f;
#pragma unroll
        for (int c = 0; c < MAX_CLUSTER; ++c)
            if (c < p.cluster) mm = fmaxf(mm, a[c].x);
        const float ref = mm == -INFINITY ? 0.f : mm;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < MAX_CLUSTER; ++c)
            if (c < p.cluster) {
                const float f = ex2(a[c].x - ref);
                ll += a[c].y * f;
                y.x += z[c].x * f, y.y += z[c].y * f, y.z += z[c].z * f, y.w += z[c].w * f;
            }
        emit(p, row0 + r, h, d, y, mm, lo[r] < hi[r] ? ll : 0.f);
    }
    cl.sync();  // no CTA leaves while another reads its shared memory
}

// CL: an item a cluster (small calls)
template <int D, int FMT, bool SPLITQ, int WP, int WR, int RN, bool CL>
__global__ void __launch_bounds__(32 * WP * WR, Shape<D, FMT, SPLITQ, WP, WR, RN>::CTAS)
    attend_kernel(const __grid_constant__ AttendP p) {
    using S = Shape<D, FMT, SPLITQ, WP, WR, RN>;
    constexpr int AT = S::NT;
    const int cluster = CL ? p.cluster : 1;
    constexpr bool F8 = S::F8;
    constexpr int ROWB = S::ROWB, TILE = S::TILE, SL = S::SL, ROWS = S::ROWS, DT = D / 16;
    using M = Misc<ROWS, TILE>;
    static_assert(sizeof(M) <= S::MISC_B, "misc area");
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t ring = sm32(smem), qs = ring + S::RING_B;
    uint8_t* const qmem = smem + S::RING_B;
    M& ms = *reinterpret_cast<M*>(smem + S::RING_B + S::Q_B);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // ---- this CTA's stretch of units
    const int items = p.H * p.RB;  // items of one (virtual) sequence
    const int nb = p.is_shared ? 1 : p.B;
    int total = 0, my_first = 0;
    if (CL) {
        if (p.status && blockIdx.x == 0)
            for (int b = tid; b < p.B; b += AT)
                if (p.lens[b] > (p.pps << p.ps_shift)) *p.status = MK_ERR_INVALID_ARG;
    } else {
        // each thread counts a stretch of sequences; sums before it by shuffles
        const int each = (nb + AT - 1) / AT, b0 = min(nb, tid * each), b1 = min(nb, b0 + each);
        int mine = 0;
        for (int b = b0; b < b1; ++b) {
            mine += cover_units<TILE>(p, b) * items;
            if (p.status && !p.is_shared && blockIdx.x == 0 && p.lens[b] > (p.pps << p.ps_shift))
                *p.status = MK_ERR_INVALID_ARG;
        }
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int a = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += a;
        }
        if (lane == 31) ms.scan[warp] = inc;
        __syncthreads();
        int before = inc - mine;
        total = 0;
#pragma unroll
        for (int w = 0; w < AT / 32; ++w) {
            if (w < warp) before += ms.scan[w];
            total += ms.scan[w];
        }
        if (blockIdx.x == 0 && !p.is_shared) {
            int at = before;
            for (int b = b0; b < b1; ++b) {
                p.base[b] = at;
                at += cover_units<TILE>(p, b) * items;
            }
            if (tid == 0) p.base[p.B] = total;
        }
        const int per = units_each(total, gridDim.x, p.min_units);
        my_first = per * blockIdx.x;
        if (my_first >= total) {
            asm volatile("griddepcontrol.wait;" ::: "memory");
            return;
        }
        if (my_first >= before && my_first < before + mine) {
            int at = before;
            ms.found_b = b0;
            ms.found_base = before;
            for (int b = b0; b < b1; ++b) {
                const int n = cover_units<TILE>(p, b) * items;
                if (my_first < at + n) {
                    ms.found_b = b;
                    ms.found_base = at;
                    break;
                }
                at += n;
            }
        }
        __syncthreads();
    }
    // the sequence whose table row a shared launch reads; no page is looked up when no sequence takes part
    const int row_seq = !CL && p.is_shared ? first_sharing(p, AT, &ms.found_row) : 0;
    // a cluster's item, and this CTA's place in it
    const int c_item = CL ? blockIdx.x / cluster : 0, c_rank = CL ? blockIdx.x - c_item * cluster : 0;
    int b = CL ? c_item / items : ms.found_b;
    int base_b = CL ? 0 : ms.found_base;
    const int my_end = CL ? 1 : min(total, my_first + units_each(total, gridDim.x, p.min_units));
    const int g8 = lane >> 2, q4 = lane & 3;  // a fragment's row (or column) and pair

    for (int u = my_first; u < my_end;) {
        // ---- the item: sequence b, kv head h, row block rb; its tiles [t0, t0 + take)
        int n_b = cover_units<TILE>(p, b), item, off, take;
        if (CL) {
            item = c_item - b * items;
            off = n_b * c_rank / cluster;
            take = n_b * (c_rank + 1) / cluster - off;
        } else {
            while (b < nb && u >= base_b + n_b * items) {
                base_b += n_b * items;
                n_b = ++b < nb ? cover_units<TILE>(p, b) : 0;
            }
            if (n_b == 0) break;  // only if the lengths changed under the launch
            item = (u - base_b) / n_b, off = u - base_b - item * n_b;
            take = min(n_b - off, my_end - u);
        }
        const int h = item / p.RB, rb = item - h * p.RB;
        int clo, chi;
        cover(p, b, clo, chi);
        int gap0 = INT_MAX, gap = 0;  // wide calls: tiles from gap0 on lie `gap` further
        if (!CL && p.wide) {
            whole_tiles(p, b, gap0, gap);
            gap -= gap0;
            gap0 -= clo / TILE + off;
        }
        const int t_first = clo / TILE + off;
        auto t_at = [&](int tile) { return t_first + tile + (!CL && tile >= gap0 ? gap : 0); };
        const int row0 = (p.is_shared ? 0 : b * p.rows_item) + rb * ROWS;
        const int nrows = min(ROWS, p.rows_item - rb * ROWS);
        const int u_first = u;
        u += CL ? 1 : take;

        // ---- fetching: where a tile's rows lie is looked up one tile ahead of the copies, a thread a row
        const uint8_t* const kh = p.k + h * p.head_b;
        const uint8_t* const vh = p.v + h * p.head_b;
        const int* const trow = p.table + (p.is_shared ? (row_seq == INT_MAX ? 0 : row_seq) : b) * p.table_s;
        const int mask = (1 << p.ps_shift) - 1;
        auto page_of = [&](int tile) {  // of position tid of the tile; -1: not this item's, or no such page
            const int pos = t_at(tile) * TILE + tid;
            if (tid >= TILE || tile >= take || pos < clo || pos >= chi || row_seq == INT_MAX) return -1;
            const int pg = trow[pos >> p.ps_shift];
            if ((unsigned)pg < (unsigned)p.n_pages) return pg;
            if (p.status) *p.status = MK_ERR_INVALID_ARG;
            return -1;
        };
        long long sc_at = -1;  // 8-bit pages: where this thread's row of the tile fetched next has its scales
        auto place = [&](int tile, int page) {
            if (tid < TILE) {
                const int r = (t_at(tile) * TILE + tid) & mask;
                ms.off[tile & 1][tid] = page < 0 ? -1 : page * p.page_b + r * p.row_b;
                if constexpr (F8) sc_at = page < 0 ? -1 : page * p.sc_page + h * p.sc_head + r;
            }
        };
        auto fetch = [&](int tile) {
            if (tile < take) {
                const uint32_t st = ring + (tile % S::STAGES) * S::STAGE_B;
                constexpr int CH = ROWB / 16;  // pieces of a row
                static_assert(AT % CH == 0, "a thread copies one column of pieces");
                const long long* off = ms.off[tile & 1];
                const int c = tid % CH;
#pragma unroll
                for (int r = tid / CH; r < TILE; r += AT / CH) {
                    const long long o = off[r];
                    const bool ok = o >= 0;
                    const long long a = ok ? o + c * 16 : 0;
                    const uint32_t to = piece<ROWB>(st, r, c);
                    cp16(to, kh + a, ok);
                    cp16(to + S::TILE_B, vh + a, ok);
                }
                if constexpr (F8) {
                    if (tid < TILE) {
                        const bool ok = sc_at >= 0;
                        const long long a = ok ? sc_at : 0;
                        cp4(st + 2 * S::TILE_B + tid * 4, p.ks + a, ok);
                        cp4(st + 2 * S::TILE_B + (TILE + tid) * 4, p.vs + a, ok);
                    }
                }
            }
            cp_commit();
        };

        const int first_page = page_of(0);
        __syncthreads();  // the previous item is done with every shared area
        for (int r = tid; r < ROWS; r += AT) {
            int lo = 0, hi = 0, at = 0;
            float sl = 0.f;
            if (r < nrows) {
                const int bt = (row0 + r) / p.G, g = (row0 + r) - bt * p.G;
                const int rbq = bt / p.T, t = bt - rbq * p.T;
                const int len = p.lens[rbq];
                at = len - p.T + t;
                lo = clo;
                hi = p.is_shared ? (shares(p, rbq) ? chi : 0) : min(at + 1, chi);
                if (p.slopes) sl = p.slopes[h * p.G + g] * LOG2E;
            }
            ms.lo[r] = lo;
            ms.hi[r] = hi;
            ms.at[r] = at;
            ms.slope2[r] = sl;
        }
        place(0, first_page);
        for (int t = 0; t < S::STAGES - 1; ++t) {
            const int next = page_of(t + 1);
            __syncthreads();
            fetch(t);
            place(t + 1, next);
        }
        // ---- queries into shared memory, a warp a row
        for (int r = warp; r < ROWS; r += AT / 32) {
            constexpr int E = D / 32;  // consecutive values of a lane
            float x[E];
#pragma unroll
            for (int i = 0; i < E; ++i) x[i] = 0.f;
            if (r < nrows) {
                const int bt = (row0 + r) / p.G, g = (row0 + r) - bt * p.G;
                const int rbq = bt / p.T, t = bt - rbq * p.T;
                const uint16_t* src = p.q + rbq * p.qb + t * p.qt + (h * p.G + g) * p.qh + lane * E;
#pragma unroll
                for (int i = 0; i < E; ++i)
                    x[i] = p.f16 ? __half2float(__ushort_as_half(src[i])) : bf2f(src[i]);
            }
            if constexpr (F8) {
                float a = 0.f;
#pragma unroll
                for (int i = 0; i < E; ++i) a = fmaxf(a, fabsf(x[i]));
#pragma unroll
                for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
                // 2^e <= a < 2^(e+1); a row of zeros, infinities or NaN is left as it is
                const unsigned ex = __float_as_uint(a) >> 23;
                const unsigned e = ex == 0 || ex == 255 ? 127u : min(ex, 253u);
                if (lane == 0) ms.qscale[r] = __uint_as_float(e << 23);
                const float inv = __uint_as_float((254u - e) << 23);
#pragma unroll
                for (int i = 0; i < E; ++i) x[i] *= inv;
            }
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                const int d = lane * E + i;
                // 8-bit pages: a lane's four consecutive codes feed slots
                // {2l, 2l+1, 2l+8, 2l+9} of a 16-wide product step
                const int c = F8 ? (d & ~15) + ((d >> 1) & 1) * 8 + ((d >> 2) & 3) * 2 : d;
                uint8_t* dst = qmem + r * (D * 2) + ((((c >> 3) ^ (r & 7))) << 4) + (c & 7) * 2;
                if constexpr (F8) {
                    *reinterpret_cast<uint32_t*>(dst) = pack_f16(x[i], x[i + 1]);
                } else {
                    const uint32_t hi = pack_bf16(x[i], x[i + 1]);
                    *reinterpret_cast<uint32_t*>(dst) = hi;
                    if constexpr (SPLITQ)
                        *reinterpret_cast<uint32_t*>(dst + ROWS * D * 2) =
                            pack_bf16(x[i] - bf2f(hi & 0xffffu), x[i + 1] - bf2f(hi >> 16));
                }
            }
        }
        __syncthreads();

        // ---- the warp's rows; a thread has rows 2 q4 and 2 q4 + 1 of each group of 8
        const int wrow = warp % WR * 8 * RN;
        int rlo[RN][2], rhi[RN][2];
        float f2[RN][2];  // score to exponent of 2 (without a cap: scale log2 e; with one: into tanh's exponential)
#pragma unroll
        for (int n = 0; n < RN; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = wrow + n * 8 + q4 * 2 + e;
                rlo[n][e] = ms.lo[r];
                rhi[n][e] = ms.hi[r];
                f2[n][e] = p.scale * LOG2E * (p.cap > 0.f ? 2.f / p.cap : 1.f) * (F8 ? ms.qscale[r] : 1.f);
            }
        // the range every row sees, and the range some row sees (rows that see something)
        int lo_max = 0, lo_min = INT_MAX, hi_min = INT_MAX, hi_max = 0;
#pragma unroll
        for (int n = 0; n < RN; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (wrow + n * 8 + q4 * 2 + e < nrows && rlo[n][e] < rhi[n][e]) {
                    lo_max = max(lo_max, rlo[n][e]), lo_min = min(lo_min, rlo[n][e]);
                    hi_min = min(hi_min, rhi[n][e]), hi_max = max(hi_max, rhi[n][e]);
                }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            lo_max = max(lo_max, __shfl_xor_sync(0xffffffffu, lo_max, o));
            lo_min = min(lo_min, __shfl_xor_sync(0xffffffffu, lo_min, o));
            hi_min = min(hi_min, __shfl_xor_sync(0xffffffffu, hi_min, o));
            hi_max = max(hi_max, __shfl_xor_sync(0xffffffffu, hi_max, o));
        }
        // queries as B fragments: columns are rows, steps along D
        auto q_frag = [&](uint32_t(&q)[4], int n, int step, int part) {  // of steps `step` and `step + 1`
            const int r = wrow + n * 8 + (lane & 7), c = step * 2 + (lane >> 3);
            ldsm4(q, qs + part * (ROWS * D * 2) + r * (D * 2) + ((c ^ (r & 7)) << 4));
        };
        uint32_t qf[S::QREG ? RN : 1][S::QREG ? DT / 2 : 1][4], ql[S::QREG && SPLITQ ? RN : 1][S::QREG && SPLITQ ? DT / 2 : 1][4];
        if constexpr (S::QREG) {
#pragma unroll
            for (int n = 0; n < RN; ++n)
#pragma unroll
                for (int i = 0; i < DT / 2; ++i) {
                    q_frag(qf[n][i], n, 2 * i, 0);
                    if constexpr (SPLITQ) q_frag(ql[n][i], n, 2 * i, 1);
                }
        }

        float o[RN][DT][4], m[RN][2], l[RN][2];
        // 8-bit pages: a row's output is in units of a power of two, not below any V scale that the row has seen, over
        // 2^15; this is 1 over that. Each row has its own: a scale that only other rows see costs it no bits.
        float vinv[RN][2], vtop = 0x1p115f;  // vtop: the largest of the thread's rows'
#pragma unroll
        for (int n = 0; n < RN; ++n) {
#pragma unroll
            for (int i = 0; i < DT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
            vinv[n][0] = vinv[n][1] = 0x1p115f;  // the least unit
        }

        for (int tile = 0; tile < take; ++tile) {
            cp_wait<S::STAGES - 2>();
            __syncthreads();
            fetch(tile + S::STAGES - 1);
            const int next_page = page_of(tile + S::STAGES);

            const int tile_at = t_at(tile) * TILE;
            const uint32_t st = ring + (tile % S::STAGES) * S::STAGE_B, vt = st + S::TILE_B;
            const float* const scales =
                reinterpret_cast<const float*>(smem + (tile % S::STAGES) * S::STAGE_B + 2 * S::TILE_B);
#pragma unroll 1
            for (int s0 = warp / WR * (TILE / WP), s1 = s0 + TILE / WP; s0 < s1; s0 += SL) {
                const int j0 = tile_at + s0;
                if (j0 + SL <= lo_min || j0 >= hi_max) continue;  // no row sees any of it
                const bool all_see = j0 >= lo_max && j0 + SL <= hi_min;

                // ---- scores, transposed: 16 positions by 8 rows a product.
                // x[n][0..1]: position g8, rows 2 q4 and 2 q4 + 1; x[n][2..3]: position g8 + 8
                float x[RN][4];
#pragma unroll
                for (int n = 0; n < RN; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[n][e] = 0.f;
#pragma unroll
                for (int i = 0; i < DT / 2; ++i) {
                    uint32_t a[2][4];
                    if constexpr (!F8) {
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            ldsm4(a[c], piece<ROWB>(st, s0 + (lane & 15), (2 * i + c) * 2 + (lane >> 4)));
                    } else {
                        uint32_t w[4];
                        ldsm4(w, piece<ROWB>(st, s0 + (lane & 15), 2 * i + (lane >> 4)));
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            code_quad<FMT>(w[2 * c], a[c][0], a[c][2]);
                            code_quad<FMT>(w[2 * c + 1], a[c][1], a[c][3]);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < RN; ++n) {
                        if constexpr (S::QREG) {
                            mma<F8>(x[n], a[0], qf[n][i][0], qf[n][i][1]);
                            mma<F8>(x[n], a[1], qf[n][i][2], qf[n][i][3]);
                            if constexpr (SPLITQ) {
                                mma<F8>(x[n], a[0], ql[n][i][0], ql[n][i][1]);
                                mma<F8>(x[n], a[1], ql[n][i][2], ql[n][i][3]);
                            }
                        } else {
                            uint32_t q[4];
                            q_frag(q, n, 2 * i, 0);
                            mma<F8>(x[n], a[0], q[0], q[1]);
                            mma<F8>(x[n], a[1], q[2], q[3]);
                            if constexpr (SPLITQ) {
                                q_frag(q, n, 2 * i, 1);
                                mma<F8>(x[n], a[0], q[0], q[1]);
                                mma<F8>(x[n], a[1], q[2], q[3]);
                            }
                        }
                    }
                }

                // ---- 8-bit pages: scales of this thread's two positions, and each row's unit
                float vsc[2] = {1.f, 1.f}, grow[RN][2];
#pragma unroll
                for (int n = 0; n < RN; ++n) grow[n][0] = grow[n][1] = 1.f;
                if constexpr (F8) {
                    const float k0 = scales[s0 + g8], k1 = scales[s0 + g8 + 8];
                    vsc[0] = scales[TILE + s0 + g8], vsc[1] = scales[TILE + s0 + g8 + 8];
#pragma unroll
                    for (int n = 0; n < RN; ++n) {
                        x[n][0] *= k0, x[n][1] *= k0;
                        x[n][2] *= k1, x[n][3] *= k1;
                    }
                    // scales (of either sign) above a row's unit
                    const float v0 = fabsf(vsc[0]), v1 = fabsf(vsc[1]);
                    if (__any_sync(0xffffffffu, fmaxf(v0, v1) * vtop > 32768.f)) {
                        const int j = j0 + g8;
                        vtop = 0.f;
#pragma unroll
                        for (int n = 0; n < RN; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                // the largest that the row sees
                                float big = fmaxf(!all_see && (j < rlo[n][e] || j >= rhi[n][e]) ? 0.f : v0,
                                                  !all_see && (j + 8 < rlo[n][e] || j + 8 >= rhi[n][e]) ? 0.f : v1);
#pragma unroll
                                for (int s = 4; s < 32; s <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, s));
                                // a unit above `big`, and far enough from 0 for 2^15 over it
                                const unsigned ex = min((__float_as_uint(big) >> 23) + 1, 250u);
                                const float inv = __uint_as_float((2u * 127u + 15u - max(ex, 27u)) << 23);
                                if (inv < vinv[n][e]) {
                                    grow[n][e] = inv / vinv[n][e];
                                    vinv[n][e] = inv;
                                }
                                vtop = fmaxf(vtop, vinv[n][e]);
                            }
                    }
                }

                // ---- capped scores, as exponents of 2
                if (p.cap > 0.f) {
                    float far = 0.f;
#pragma unroll
                    for (int n = 0; n < RN; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            x[n][e] *= f2[n][e & 1];
                            far = fmaxf(far, fabsf(x[n][e]));
                        }
                    if (__all_sync(0xffffffffu, far < CAP_NEAR)) {
#pragma unroll
                        for (int n = 0; n < RN; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) x[n][e] = cap_near(x[n][e], 0.5f * p.cap);
                    } else {
#pragma unroll
                        for (int n = 0; n < RN; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) x[n][e] = cap_any(x[n][e], p.cap);
                    }
                }

                // ---- softmax: x becomes the probabilities
                uint32_t seen = 0xffffffffu;  // bit n*4+e: the row sees the position
                bool turn = false;
                float f[RN][2];
#pragma unroll
                for (int n = 0; n < RN; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float y0 = x[n][e], y1 = x[n][2 + e];
                        if (!(p.cap > 0.f)) y0 *= f2[n][e], y1 *= f2[n][e];
                        if (p.slopes) {
                            const int r = wrow + n * 8 + q4 * 2 + e;
                            const float sl = ms.slope2[r], far = (float)(ms.at[r] - j0 - g8);  // a whole number: exact
                            y0 -= sl * far;
                            y1 -= sl * (far - 8.f);
                        }
                        if (!all_see) {
                            const int j = j0 + g8;
                            if (j < rlo[n][e] || j >= rhi[n][e]) y0 = -INFINITY, seen &= ~(1u << (n * 4 + e));
                            if (j + 8 < rlo[n][e] || j + 8 >= rhi[n][e]) y1 = -INFINITY, seen &= ~(4u << (n * 4 + e));
                        }
                        float top = fmaxf(y0, y1);
#pragma unroll
                        for (int s = 4; s < 32; s <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
                        const float mn = fmaxf(m[n][e], top);
                        const float ref = mn == -INFINITY ? 0.f : mn;
                        const float keep = ex2(m[n][e] - ref);
                        m[n][e] = mn;
                        const float p0 = ex2(y0 - ref), p1 = ex2(y1 - ref);
                        l[n][e] = l[n][e] * keep + (p0 + p1);
                        x[n][e] = p0, x[n][2 + e] = p1;
                        if constexpr (F8) {
                            x[n][e] *= vsc[0] * vinv[n][e], x[n][2 + e] *= vsc[1] * vinv[n][e];
                            if (!all_see) {  // the scale of a row that is not seen may be anything
                                if (!(seen >> (n * 4 + e) & 1u)) x[n][e] = 0.f;
                                if (!(seen >> (n * 4 + e) & 4u)) x[n][2 + e] = 0.f;
                            }
                        }
                        f[n][e] = keep * grow[n][e];
                        turn |= f[n][e] != 1.f;
                    }
                if (__any_sync(0xffffffffu, turn)) {
#pragma unroll
                    for (int n = 0; n < RN; ++n)
#pragma unroll
                        for (int i = 0; i < DT; ++i) {
                            o[n][i][0] *= f[n][0], o[n][i][1] *= f[n][1];
                            o[n][i][2] *= f[n][0], o[n][i][3] *= f[n][1];
                        }
                }

                // ---- values some row does not see must not reach it, and 0 x NaN would: look for
                // non-finite ones where rows see different parts
                bool odd = false;
                if (!all_see && FMT != MK_KV_INT8) {
                    for (int i = lane; i < SL * (ROWB / 16); i += 32) {
                        uint32_t w[4];
                        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                     : "r"(vt + (s0 * ROWB) + i * 16));
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if constexpr (FMT == MK_KV_BF16) {
                                odd |= (w[e] & 0x7f80u) == 0x7f80u || (w[e] & 0x7f800000u) == 0x7f800000u;
                            } else {
                                // a code is NaN when its low seven bits are all set
                                odd |= (((w[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
                            }
                        }
                    }
                    odd = __any_sync(0xffffffffu, odd);
                }
                if (odd) {
                    // such values go to the rows that see them one by one; below they count as zeros
#pragma unroll 1
                    for (int j = 0; j < SL; ++j) {
#pragma unroll
                        for (int n = 0; n < RN; ++n) {
                            float pv[2];
                            unsigned vis = seen >> (n * 4 + (j >= 8 ? 2 : 0));
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                pv[e] = __shfl_sync(0xffffffffu, j >= 8 ? x[n][2 + e] : x[n][e], ((j & 7) << 2) | q4);
                            vis = __shfl_sync(0xffffffffu, vis, ((j & 7) << 2) | q4);
#pragma unroll
                            for (int i = 0; i < DT; ++i)
#pragma unroll
                                for (int c = 0; c < 2; ++c) {
                                    const int d = F8 ? i * 16 + 2 * g8 + c : i * 16 + g8 + 8 * c;
                                    const uint32_t a = piece<ROWB>(vt, s0 + j, d * S::EB / 16) + (d * S::EB & 15);
                                    if constexpr (F8) {
                                        uint32_t v;
                                        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
                                        if ((v & 0x7fu) == 0x7fu) {
                                            if (vis & 1u) o[n][i][2 * c] = __uint_as_float(0x7fffffffu);
                                            if (vis & 2u) o[n][i][2 * c + 1] = __uint_as_float(0x7fffffffu);
                                        }
                                    } else {
                                        uint16_t v;
                                        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
                                        if ((v & 0x7f80u) == 0x7f80u) {
                                            if (vis & 1u) o[n][i][2 * c] += fmaxf(pv[0], 0x1p-126f) * bf2f(v);
                                            if (vis & 2u) o[n][i][2 * c + 1] += fmaxf(pv[1], 0x1p-126f) * bf2f(v);
                                        }
                                    }
                                }
                        }
                    }
                }

                // ---- outputs, transposed: 16 values by 8 rows a product. Probabilities become B fragments
                // (16 positions by 8 rows) by transposing 8 x 8 pieces; lo: what the 16-bit hi part left
                const bool with_lo = !F8 || p.f16;
                uint32_t ph[RN][2], pl[RN][2];
#pragma unroll
                for (int n = 0; n < RN; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float y0 = x[n][2 * c], y1 = x[n][2 * c + 1];
                        uint32_t hi, lo = 0;
                        if constexpr (F8) {
                            hi = pack_f16(y0, y1);
                            if (with_lo) {
                                const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                                lo = pack_f16(y0 - z.x, y1 - z.y);
                            }
                        } else {
                            split_bf16(y0, y1, hi, lo);
                            if (!all_see) {  // nothing of what is not seen
                                if (!(seen >> (n * 4 + 2 * c) & 1u)) lo &= 0xffff0000u;
                                if (!(seen >> (n * 4 + 2 * c) & 2u)) lo &= 0xffffu;
                            }
                        }
                        ph[n][c] = transpose8(hi);
                        if (with_lo) pl[n][c] = transpose8(lo);
                    }
#pragma unroll
                for (int dt = 0; dt < DT; dt += F8 ? 2 : 1) {
                    uint32_t a[F8 ? 2 : 1][4];
                    if constexpr (!F8) {
                        ldsm4t(a[0], piece<ROWB>(vt, s0 + (lane & 7) + (lane >> 4) * 8, dt * 2 + ((lane >> 3) & 1)));
                        if (odd) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if ((a[0][i] & 0x7f80u) == 0x7f80u) a[0][i] &= 0xffff0000u;
                                if ((a[0][i] & 0x7f800000u) == 0x7f800000u) a[0][i] &= 0xffffu;
                            }
                        }
                    } else {
                        // transposing byte pairs: a register holds values 2 g8, 2 g8 + 1 of two positions;
                        // the even ones are rows 0-7 of the product, the odd ones rows 8-15
                        uint32_t w[4];
                        ldsm4t(w, piece<ROWB>(vt, s0 + (lane & 15), dt + (lane >> 4)));
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            if (FMT == MK_KV_E4M3 && odd) {  // NaN codes to zero
                                const uint32_t z = ((w[c] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                                w[c] &= ~((z >> 7) * 0xffu);
                            }
                            code_quad<FMT>(__byte_perm(w[c], 0, 0x3120), a[c >> 1][(c & 1) * 2], a[c >> 1][(c & 1) * 2 + 1]);
                        }
                    }
#pragma unroll
                    for (int c = 0; c < (F8 ? 2 : 1); ++c)
#pragma unroll
                        for (int n = 0; n < RN; ++n) {
                            mma<F8>(o[n][dt + c], a[c], ph[n][0], ph[n][1]);
                            if (with_lo) mma<F8>(o[n][dt + c], a[c], pl[n][0], pl[n][1]);
                        }
                }
            }
            place(tile + S::STAGES, next_page);
        }

        // ---- the item's (or piece's) result: outputs pass through shared memory, a warp's rows by rows
#pragma unroll
        for (int n = 0; n < RN; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int s = 4; s < 32; s <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], s);
                if constexpr (F8) {
                    const float f = __uint_as_float((254u << 23) - __float_as_uint(vinv[n][e]));  // the unit
#pragma unroll
                    for (int i = 0; i < DT; ++i) o[n][i][e] *= f, o[n][i][2 + e] *= f;
                }
            }
        const bool whole = take == n_b || CL;
        float* slot = nullptr;
        if (whole && p.keep_items)
            slot = p.slots + (2ll * gridDim.x + (long long)b * items + item) * p.slot_floats;
        else if (!whole)
            slot = p.slots + (2ll * blockIdx.x + (u_first == my_first ? 0 : 1)) * p.slot_floats;
        // (m, l) of slot row r at slot + slot_rows * D + 2 r
        auto put = [&](int r, int d, float4 y, float mm, float ll, bool first) {
            // four values of row r from column d on. A row that sees nothing was
            // not masked where all others see everything: it is dropped here.
            if (ms.lo[r] >= ms.hi[r]) mm = -INFINITY, ll = 0.f;
            if (slot) {
                *reinterpret_cast<float4*>(slot + (long long)r * D + d) = y;
                if (first) *reinterpret_cast<float2*>(slot + (long long)p.slot_rows * D + 2 * r) = make_float2(mm, ll);
                return;
            }
            emit(p, row0 + r, h, d, y, mm, ll);
        };
        cp_wait<0>();
        __syncthreads();  // the ring is free
        {
            // WP = 1: a warp's rows one group of 8 after another through the warp's own 8 rows of memory;
            // else the parts of all rows side by side
            float* om = reinterpret_cast<float*>(smem);
            float* oml = reinterpret_cast<float*>(qmem);  // the queries are done with
            auto store = [&](int n, int at_row) {
#pragma unroll
                for (int i = 0; i < DT; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int d = F8 ? i * 16 + 2 * g8 + c : i * 16 + g8 + 8 * c;
                        om[(at_row + q4 * 2) * D + d] = o[n][i][2 * c];
                        om[(at_row + q4 * 2 + 1) * D + d] = o[n][i][2 * c + 1];
                    }
                if (g8 == 0) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        oml[(at_row + q4 * 2 + e) * 2] = m[n][e];
                        oml[(at_row + q4 * 2 + e) * 2 + 1] = l[n][e];
                    }
                }
            };
            if constexpr (WP > 1) {
#pragma unroll
                for (int n = 0; n < RN; ++n) store(n, warp / WR * ROWS + wrow + n * 8);
                __syncthreads();
                for (int i = tid; i < nrows * (D / 4); i += AT) {
                    const int r = i / (D / 4), d = (i % (D / 4)) * 4;
                    float mm = -INFINITY, ll = 0.f;
#pragma unroll
                    for (int w = 0; w < WP; ++w) mm = fmaxf(mm, oml[(w * ROWS + r) * 2]);
                    const float ref = mm == -INFINITY ? 0.f : mm;
                    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < WP; ++w) {
                        const float f = ex2(oml[(w * ROWS + r) * 2] - ref);
                        ll += oml[(w * ROWS + r) * 2 + 1] * f;
                        const float4 z = *reinterpret_cast<const float4*>(om + (w * ROWS + r) * D + d);
                        y.x += z.x * f, y.y += z.y * f, y.z += z.z * f, y.w += z.w * f;
                    }
                    if (CL && cluster > 1) {  // to where only this thread has read
                        *reinterpret_cast<float4*>(om + r * D + d) = y;
                        if (d == 0) *reinterpret_cast<float2*>(oml + WP * ROWS * 2 + 2 * r) = make_float2(mm, ll);
                    } else {
                        put(r, d, y, mm, ll, d == 0);
                    }
                }
                if (CL && cluster > 1)
                    cluster_join<D, ROWS, AT>(p, om, oml + WP * ROWS * 2, ms.lo, ms.hi, row0, h, nrows, c_rank);
            } else {
#pragma unroll
                for (int n = 0; n < RN; ++n) {
                    store(n, warp * 8);
                    __syncwarp();
                    for (int i = lane; i < 8 * (D / 4); i += 32) {
                        const int r = i / (D / 4), d = (i % (D / 4)) * 4, row = wrow + n * 8 + r;
                        if (row < nrows)
                            put(row, d, *reinterpret_cast<const float4*>(om + (warp * 8 + r) * D + d),
                                oml[(warp * 8 + r) * 2], oml[(warp * 8 + r) * 2 + 1], d == 0);
                    }
                    __syncwarp();
                }
            }
        }
    }
    // This launch may have begun before the shared one ended; the joining
    // launch waits for this one alone, so this one ends after the shared one.
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Joins the pieces of one output row: a warp a row (W = 1), or four that take
// every fourth piece each (W = 4: many pieces, whose trips to L2 would follow
// one another). Rows whose only piece went straight to the output are left alone;
// rows without any piece get their zeros here. Reads the pieces from L2: 3 us
// (16 rows) to 6 us (896 rows) of latency, most of it the launch, the lookup of
// the row's pieces and one trip to L2 each.
template <int D, int W>
__global__ void __launch_bounds__(JT) join_kernel(const __grid_constant__ JoinP jp) {
    constexpr int E = D / 32, AHEAD = W == 1 ? (D == 256 ? 4 : 8) : 4;
    __shared__ float om[W][D];
    __shared__ float2 oml[W];
    const AttendP& p = jp.own;
    const int warp = W == 1 ? 0 : threadIdx.x >> 5, lane = threadIdx.x & 31, Hq = p.H * p.G;
    const unsigned orow = W == 1 ? blockIdx.x * (JT / 32) + (threadIdx.x >> 5) : blockIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (orow >= jp.rows) return;
    const int bt = orow / Hq, hq = orow - bt * Hq;
    const int b = bt / p.T, t = bt - b * p.T, h = hq / p.G, g = hq - h * p.G;

    // pieces of a launch: CTAs c0 .. c1, the row's place in a slot
    struct Part {
        const float* slots;
        long long whole_slot;
        int c0, c1, per, first, row, rows, floats, n;
    };
    auto part = [&](const AttendP& a, int grid, int rows_blk, int base, int total, int n_b, int vb, int r) {
        Part x;
        const int rb = r / rows_blk, item = h * a.RB + rb;
        x.n = n_b;
        x.per = units_each(total, grid, a.min_units);
        x.first = base + item * n_b;
        x.c0 = x.first / x.per;
        x.c1 = n_b ? (x.first + n_b - 1) / x.per : x.c0 - 1;
        x.whole_slot = 2ll * grid + (long long)vb * a.H * a.RB + item;
        x.row = r - rb * rows_blk;
        x.rows = a.slot_rows;
        x.floats = a.slot_floats;
        x.slots = a.slots;
        return x;
    };
    const int items = p.H * p.RB;
    const int base = p.base[b];
    const Part own = part(p, jp.own_grid, jp.own_rows, base, p.base[p.B], (p.base[b + 1] - base) / items, b,
                          t * p.G + g);
    const bool with_shared = jp.shared_grid > 0;
    if (own.n && own.c0 == own.c1 && !p.keep_items) return;

    float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = 0.f;
    auto add = [&](const Part& x) {
#pragma unroll AHEAD
        for (int c = x.c0 + warp; c <= x.c1; c += W) {
            const long long slot = x.c0 == x.c1 ? x.whole_slot : 2 * c + (x.first <= c * x.per ? 0 : 1);
            const float* s = x.slots + slot * x.floats;
            const float2 ml = *reinterpret_cast<const float2*>(s + (long long)x.rows * D + 2 * x.row);
            float y[E];
            const float* src = s + (long long)x.row * D + lane * E;
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                const float2 z = *reinterpret_cast<const float2*>(src + i);
                y[i] = z.x, y[i + 1] = z.y;
            }
            const float mn = fmaxf(m, ml.x), ref = mn == -INFINITY ? 0.f : mn;
            const float f = ex2(m - ref), e = ex2(ml.x - ref);
            m = mn;
            l = l * f + ml.y * e;
            // a piece in which the row saw nothing adds nothing
#pragma unroll
            for (int i = 0; i < E; ++i) o[i] = o[i] * f + (ml.x == -INFINITY ? 0.f : y[i] * e);
        }
    };
    if (own.n) add(own);
    if (with_shared) {
        const AttendP& a = jp.shared;
        if (!a.wide)
            add(part(a, jp.shared_grid, jp.shared_rows, 0, jp.shared_units * a.H * a.RB, jp.shared_units, 0,
                     bt * p.G + g));
        else if (const int n = (a.base[b + 1] - a.base[b]) / (a.H * a.RB))
            add(part(a, jp.shared_grid, jp.shared_rows, a.base[b], a.base[a.B], n, b, t * p.G + g));
    }
    uint16_t* dst = p.out + b * p.ob + t * p.ot + hq * p.oh;
    if constexpr (W == 1) {
        const bool none = l == 0.f;
        uint16_t z[E];
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float y = none ? 0.f : o[i] / l;
            z[i] = p.f16 ? __half_as_ushort(__float2half_rn(y)) : __bfloat16_as_ushort(__float2bfloat16_rn(y));
        }
        if (((uintptr_t)dst & 3) == 0) {
#pragma unroll
            for (int i = 0; i < E; i += 2)
                *reinterpret_cast<uint32_t*>(dst + lane * E + i) = z[i] | (uint32_t)z[i + 1] << 16;
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) dst[lane * E + i] = z[i];
        }
        if (lane == 0 && p.lse) p.lse[(long long)orow] = none ? -INFINITY : (m + log2f(l)) * LN2;
        return;
    }
#pragma unroll
    for (int i = 0; i < E; ++i) om[warp][lane * E + i] = o[i];
    if (lane == 0) oml[warp] = make_float2(m, l);
    __syncthreads();
    float mm = -INFINITY, ll = 0.f, w[W];
#pragma unroll
    for (int i = 0; i < W; ++i) mm = fmaxf(mm, oml[i].x);
    const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        w[i] = ex2(oml[i].x - ref);
        ll += oml[i].y * w[i];
    }
    const bool none = ll == 0.f;
    for (int d = threadIdx.x; d < D; d += JT) {
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) y += om[i][d] * w[i];
        const float z = none ? 0.f : y / ll;
        dst[d] = p.f16 ? __half_as_ushort(__float2half_rn(z)) : __bfloat16_as_ushort(__float2bfloat16_rn(z));
    }
    if (threadIdx.x == 0 && p.lse)
        p.lse[((long long)b * p.T + t) * Hq + hq] = none ? -INFINITY : (mm + log2f(ll)) * LN2;
}

// Which kernel a call takes: format, whether queries need a lo part, rows.
struct Kind {
    int format;
    bool splitq;
    int rows;  // of an item: 8, 16, 32, 64 or, below 256 wide heads, 128
};
struct KindInfo {
    int tile, rows, ctas;  // positions of a tile, rows of an item, CTAs an SM
};

// A kernel by its template arguments, with what the host has to know of it.
template <int D, int FMT, bool SPLITQ, int WP, int WR, int RN, bool CL>
int attend_run(const AttendP* p, KindInfo* info, int grid, bool after, cudaStream_t s) {
    using S = Shape<D, FMT, SPLITQ, WP, WR, RN>;
    auto kern = attend_kernel<D, FMT, SPLITQ, WP, WR, RN, CL>;
    if (info) {
        info->tile = S::TILE;
        info->rows = S::ROWS;
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&info->ctas, kern, S::NT, S::SMEM);
        return cuda_status(e, "mk_pages_attend");
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(S::NT);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    if (p->cluster > 1) {
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = p->cluster;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    } else {
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.attrs = at;
    cfg.numAttrs = after || p->cluster > 1 ? 1 : 0;
    return cuda_status(cudaLaunchKernelEx(&cfg, kern, *p), "mk_pages_attend");
}

template <int D, int FMT, bool SPLITQ>
int attend_pick(const Kind& k, const AttendP* p, KindInfo* info, int grid, bool after, cudaStream_t s) {
    // the kernel's attributes are the same with and without clusters, but are set for each
    auto go = [&](auto run, auto run_cl) {
        if (info) {
            if (const int rc = run_cl(nullptr, info, 0, false, nullptr)) return rc;
            return run(nullptr, info, 0, false, nullptr);
        }
        return p->cluster ? run_cl(p, nullptr, grid, after, s) : run(p, nullptr, grid, after, s);
    };
    if (k.rows == 8) return go(attend_run<D, FMT, SPLITQ, 4, 1, 1, false>, attend_run<D, FMT, SPLITQ, 4, 1, 1, true>);
    if (k.rows == 16) return go(attend_run<D, FMT, SPLITQ, 4, 1, 2, false>, attend_run<D, FMT, SPLITQ, 4, 1, 2, true>);
    if (k.rows == 32) return go(attend_run<D, FMT, SPLITQ, 4, 2, 2, false>, attend_run<D, FMT, SPLITQ, 4, 2, 2, true>);
    if constexpr (D < 256) {  // 128 rows of 256 leave no room for the ring
        if (k.rows == 128) return attend_run<D, FMT, SPLITQ, 1, 8, 2, false>(p, info, grid, after, s);
    }
    return attend_run<D, FMT, SPLITQ, 2, 4, 2, false>(p, info, grid, after, s);
}

// With `info`: what the host has to know of the kernel (and its one-time
// attributes on the current device); else the launch, which may begin before
// the previous one of the stream ends when `after` is set.
template <int D>
int attend_d(const Kind& k, const AttendP* p, KindInfo* info, int grid, bool after, cudaStream_t s) {
    if (k.format == MK_KV_E4M3) return attend_pick<D, MK_KV_E4M3, false>(k, p, info, grid, after, s);
    if (k.format == MK_KV_INT8) return attend_pick<D, MK_KV_INT8, false>(k, p, info, grid, after, s);
    if (k.splitq) return attend_pick<D, MK_KV_BF16, true>(k, p, info, grid, after, s);
    return attend_pick<D, MK_KV_BF16, false>(k, p, info, grid, after, s);
}
template <int D>
int join_d(const JoinP& j, cudaStream_t s) {
    // A warp a row where the pieces are few, or the rows so many that the instructions of four warps count more than
    // trips to L2 in turn. Four and one, whole calls: 64 sequences of 1024 positions (40 query heads on 8, 2 pieces)
    // 44.5 and 42.4 us, 256 tokens at 16384 (4096 rows, some 20 pieces) 90.9 and 85.1; 8 x 7 tokens at 8192 (896 rows,
    // 15 pieces) 37.3 and 42.0, 16 x 4 at 4096 (1024 rows, 8 pieces) 31.3 and 33.2.
    const bool one = j.pieces <= 4 || (j.rows >= 2048 && j.pieces <= 32);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(one ? (j.rows + JT / 32 - 1) / (JT / 32) : j.rows);
    cfg.blockDim = dim3(JT);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cuda_status(one ? cudaLaunchKernelEx(&cfg, join_kernel<D, 1>, j) : cudaLaunchKernelEx(&cfg, join_kernel<D, 4>, j),
                       "mk_pages_attend");
}

// one translation unit a head_dim
typedef int (*AttendFn)(const Kind&, const AttendP*, KindInfo*, int, bool, cudaStream_t);
int attend_64(const Kind&, const AttendP*, KindInfo*, int, bool, cudaStream_t);
int attend_128(const Kind&, const AttendP*, KindInfo*, int, bool, cudaStream_t);
int attend_256(const Kind&, const AttendP*, KindInfo*, int, bool, cudaStream_t);
// the launch on the tensor memory (mk_prefix.cuh; head_dim 64 and 128): 128
// rows an item, one CTA an SM. p NULL: one-time attributes.
int prefix_bf16(int head_dim, int format, const AttendP* p, int grid, cudaStream_t s);
int prefix_f16(int head_dim, int format, const AttendP* p, int grid, cudaStream_t s);
int join_64(const JoinP&, cudaStream_t);
int join_128(const JoinP&, cudaStream_t);
int join_256(const JoinP&, cudaStream_t);

}  // namespace mkop
