// mk_latent.cu -- attention over a paged latent cache, in the latent space
// (mk_latent_attend).
//
// For one query row (a token and a head) and the positions j it sees,
//   x_j = scale (q . c_j + q_rope . r_j),  m = max x_j,
//   out = sum_j e^(x_j - m) c_j / sum_j e^(x_j - m):
// one vector a position is key and value of all heads, so the rows of all heads
// (and of a few tokens) stand against one copy of it, up to 64 rows a CTA. A
// tile of 32 positions lies in shared memory once, in the 128-byte-swizzled order
// of tensor maps, and feeds both products on the fifth-generation tensor cores:
//   S  = Q C^T      64 rows x the tile's positions, over rank + 64 values;
//   O' = C^T P^T    rank values x rows: the output transposed, C as the
//                   operand whose rows are the sum's (as it lies there), so
//                   that up to 64 rows of 512 outputs take 256 columns of
//                   tensor memory and few rows cost few of them.
//
// Roles: four warps softmax (S comes as 16-row fragments, a quad of threads a
// row; P goes back through shared memory, rounded to the cache's type: what it
// loses, half a step of each weight, is of the output's own rounding. fp16 has no
// steps of its own for small weights: they are taken 2^7 larger, so that half a
// step is at least 2^-32 of the row's largest), one warp
// copies, one cleans (below), two issue S and O'. O' is rescaled only when some
// row's maximum has risen by more than 2^8 since its reference.
//
// Tiles at the ends of what is seen: scores are masked, and since 0 x NaN is
// NaN, a warp zeroes the rows of such a tile that no row of the block sees. A
// position that only some rows see (a later token of the block) and that is not
// finite is zeroed too, and rows that do see it get NaN.
//
// Work is cut by tiles of all (sequence, row block) items in one line, an equal
// stretch a CTA; pieces of an item leave (output, maximum, sum) in the workspace
// and a second launch joins them. All waits have a limit, after which the CTA
// frees its tensor memory and leaves (MK_ERR_TIMEOUT in `status`, NaN in its
// rows).
//
// Measured, 16 heads on 512 + 64 values, bf16: 64 sequences of up to 32768
// positions 237 us (6.5 TB/s, 95 % of what a copy reaches: HBM). One sequence of
// 8192 15 us, all latency (4 tiles a CTA: 2 us to the first tile's copy, 1 its way,
// 1.7 to its weights, 0.9 a tile, 1 the piece's end; the launches, and 3 us of
// join). Rows past 16 are bound by what feeds the products from shared memory: 64
// rows take 1030 cycles a tile for S (36 steps of 28) and 410 for O', 1600 in
// all: 8 sequences of 8192 with 7 tokens 38 us (9 of them pieces and join), 64 of
// them 160. Tiles of 64 positions feed S better (36 cycles a step of twice the
// positions) but two of them fill shared memory, and copies then wait: 192 us.
//
// Pages of fewer than 8 positions, or overlapping ones (a stride of 0), have no
// tensor map: a block a row takes them, a position a warp at a time.
#include <climits>
#include <type_traits>

#include "mk_tensor.cuh"
#include "mk_values.cuh"

namespace {

using namespace mkop;

struct LatentP {
    const uint8_t *latent, *rope;
    long long page_s, row_s, rope_page_s, rope_row_s;  // elements
    const int* table;
    long long table_s;
    const int *lens, *starts;
    const uint8_t *q, *qr;
    long long qb, qt, qh, rb, rt, rh;
    uint8_t* out;
    long long ob, ot, oh;
    float* lse;
    int* status;
    int pps, ps_shift, n_pages, B, T, H;
    float scale;
    // the tensor cores' kernel
    int nr;          // rows of a block, padded to 16
    int rows_blk;    // rows of a block
    int RB;          // row blocks of a sequence
    int min_units;   // a CTA's least stretch of tiles
    float* slots;    // two of each CTA: its first and its last piece
    int* base;       // [items + 1]: first tile of each item, for the joining launch
    unsigned wait_ns;
    unsigned signals;  // for tests: the tiles of a CTA after which a role's signals are left out
    int q_vec;        // queries can be copied 16 bytes at a time
};

constexpr int LT = 128;

// A block a query row, a position a warp at a time.
template <int DT, int RANK, int ROPE>
__global__ void __launch_bounds__(LT) latent_rows(const __grid_constant__ LatentP p) {
    constexpr int V = RANK / 256;
    __shared__ float om[LT / 32][RANK], ml[LT / 32][2];
    const int row = blockIdx.x, bt = row / p.H, h = row - bt * p.H, b = bt / p.T, t = bt - b * p.T;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cap = p.pps << p.ps_shift, len = p.lens[b];
    if (len > cap && p.status && threadIdx.x == 0) *p.status = MK_ERR_INVALID_ARG;
    const long long last = min((long long)len - p.T + t, (long long)cap - 1);
    const int first = max(p.starts ? p.starts[b] : 0, 0);
    float q[V][8], qr[8], o[V][8] = {};
    const long long qa = b * p.qb + t * p.qt + h * p.qh, ra = b * p.rb + t * p.rt + h * p.rh;
    Values8<DT, false> x;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        x.load(p.q, qa + 8 * (v * 32 + lane));
        x.floats(q[v]);
    }
    if (lane < ROPE / 8) {
        x.load(p.qr, ra + 8 * lane);
        x.floats(qr);
    }
    float m = -INFINITY, l = 0.f;
    for (long long j = first + warp; j <= last; j += LT / 32) {
        const int page = p.table[b * p.table_s + (j >> p.ps_shift)], r = (int)(j & ((1 << p.ps_shift) - 1));
        const bool in = (unsigned)page < (unsigned)p.n_pages;
        if (!in && p.status) *p.status = MK_ERR_INVALID_ARG;
        float c[V][8] = {}, s = 0.f;
        if (in) {
            Values8<DT, true> y;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                y.load(p.latent, page * p.page_s + r * p.row_s + 8 * (v * 32 + lane));
                y.floats(c[v]);
#pragma unroll
                for (int e = 0; e < 8; ++e) s += q[v][e] * c[v][e];
            }
            if (lane < ROPE / 8) {
                float k[8];
                y.load(p.rope, page * p.rope_page_s + r * p.rope_row_s + 8 * lane);
                y.floats(k);
#pragma unroll
                for (int e = 0; e < 8; ++e) s += qr[e] * k[e];
            }
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s = __fmul_rn(s, p.scale);  // (as below: rounded before a maximum is taken off)
        const float mn = fmaxf(m, s), f = __expf(m - mn), w = __expf(s - mn);
        m = mn;
        l = l * f + w;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e) o[v][e] = o[v][e] * f + w * c[v][e];
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) om[warp][8 * (v * 32 + lane) + e] = o[v][e];
    if (lane == 0) ml[warp][0] = m, ml[warp][1] = l;
    __syncthreads();
    float mm = -INFINITY, ll = 0.f;
    for (int w = 0; w < LT / 32; ++w) mm = fmaxf(mm, ml[w][0]);
    const float ref = mm == -INFINITY ? 0.f : mm;
    for (int w = 0; w < LT / 32; ++w) ll += ml[w][1] * __expf(ml[w][0] - ref);
    for (int d = threadIdx.x; d < RANK; d += LT) {
        float y = 0.f;
        for (int w = 0; w < LT / 32; ++w) y += om[w][d] * __expf(ml[w][0] - ref);
        y = ll == 0.f ? 0.f : y / ll;
        if constexpr (DT == MK_DT_F16) reinterpret_cast<__half*>(p.out)[b * p.ob + t * p.ot + h * p.oh + d] = __float2half_rn(y);
        else reinterpret_cast<__nv_bfloat16*>(p.out)[b * p.ob + t * p.ot + h * p.oh + d] = __float2bfloat16_rn(y);
    }
    if (threadIdx.x == 0 && p.lse) p.lse[row] = ll == 0.f ? -INFINITY : mm + logf(ll);
}


// ---------------------------------------------------------------- tensor cores

constexpr int NT = 256, SMEM_MOST = 227 * 1024;
constexpr float RISE = 8.f;  // powers of 2 that a maximum rises above its reference before the output is rescaled
constexpr int TILE = 32;  // positions

// A row block of a sequence and the tiles its rows see.
struct Item {
    int b, rb, row0, rows;  // rows of the block: row0 .. row0 + rows - 1, token-major
    int lo, hi, common;     // positions: [lo, hi) are seen by some row, [lo, common) by all
    int t0, n;              // first tile, tiles
    __device__ __forceinline__ void set(const LatentP& p, int item) {
        b = item / p.RB;
        rb = item - b * p.RB;
        row0 = rb * p.rows_blk;
        rows = min(p.rows_blk, p.T * p.H - row0);
        const long long cap = (long long)p.pps << p.ps_shift, behind = (long long)p.lens[b] - p.T + 1;
        lo = max(p.starts ? p.starts[b] : 0, 0);
        hi = (int)max(0ll, min(behind + (row0 + rows - 1) / p.H, cap));
        common = (int)max(0ll, min(behind + row0 / p.H, cap));
        t0 = lo / TILE;
        n = hi > lo ? (hi + TILE - 1) / TILE - t0 : 0;
    }
};

struct Line {  // a role's place in the line of tiles
    Item it;
    int item, tile;
    __device__ __forceinline__ void start(const LatentP& p, int i, int t) {
        item = i;
        tile = t;
        it.set(p, i);
    }
    // k tiles on; behind the last item is one without an end
    __device__ __forceinline__ void on(const LatentP& p, int k) {
        tile += k;
        while (tile >= it.n) {
            tile -= it.n;
            if (++item >= p.B * p.RB) it.n = INT_MAX, it.hi = 0;
            else it.set(p, item);
        }
    }
    __device__ __forceinline__ int at() const { return (it.t0 + tile) * TILE; }
};

// a ring's stage, its turn, and the tile's number
struct Spot {
    int stage = 0;
    unsigned turn = 0, c = 0;
    template <int STAGES>
    __device__ __forceinline__ void next() {
        ++c;
        if (++stage == STAGES) stage = 0, ++turn;
    }
    __device__ __forceinline__ int buf() const { return (int)(c & 1u); }
    __device__ __forceinline__ unsigned full() const { return turn & 1u; }
    __device__ __forceinline__ unsigned free() const { return (turn - 1) & 1u; }
    __device__ __forceinline__ unsigned pair() const { return c >> 1 & 1u; }
    __device__ __forceinline__ unsigned pair_free() const { return ((c >> 1) - 1) & 1u; }
};

struct LatentMisc {
    unsigned long long kv_full[8], v_ok[8], pv_done[8], s_full[2], s_free[2], p_ready[2], q_ready, drained;
    unsigned tmem, abort;
    int scan[NT / 32], found_item, found_base;
    int bad[16];           // of a piece: the first position of it that is not finite and that only some rows see
    float m[64], f[64];    // of a row: its maximum, its factor
    float sum[64];
    long long to[64];
};

template <int MT, int NR>
struct LatentShape {
    static constexpr int RANK = 128 * MT, KP = 2 * MT + 1;  // 128-byte panels of a position
    static constexpr int Q_B = KP * NR * 128, STAGE_B = KP * TILE * 128, P_B = NR * 128;  // P: two tiles' side by side
    static constexpr int MISC_B = 1984;
    // shared memory: queries, the ring, probabilities, the rest; and room to align to 1024
    static constexpr int FIT = (SMEM_MOST - 1024 - MISC_B - Q_B - P_B) / STAGE_B, STAGES = FIT < 8 ? FIT : 8;
    static constexpr int RING_OFF = Q_B, P_OFF = RING_OFF + STAGES * STAGE_B, MISC_OFF = P_OFF + P_B;
    static constexpr int SMEM = 1024 + MISC_OFF + MISC_B;
    static constexpr int T_S = 0, T_O = 2 * TILE, T_ALL = T_O + MT * NR <= 128 ? 128 : T_O + MT * NR <= 256 ? 256 : 512;
    static_assert(sizeof(LatentMisc) <= MISC_B && STAGES >= 2 && T_O + MT * NR <= T_ALL, "");
};

struct LatentMaps {
    CUtensorMap latent, rope;
};

template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    return F16 ? pack_f16(lo, hi) : pack_bf16(lo, hi);
}
template <bool F16>
__device__ __forceinline__ void put16(uint8_t* out, long long at, float x) {
    if constexpr (F16) reinterpret_cast<__half*>(out)[at] = __float2half_rn(x);
    else reinterpret_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(x);
}
// one 32-bit word with either 16-bit half not finite
template <bool F16>
__device__ __forceinline__ bool not_finite(uint32_t w) {
    constexpr uint32_t E = F16 ? 0x7c00u : 0x7f80u;
    return (w & E) == E || (w & (E << 16)) == E << 16;
}

template <int MT, int NR, bool F16>
__global__ void __launch_bounds__(NT, 1)
    latent_kernel(const __grid_constant__ LatentP p, const __grid_constant__ LatentMaps maps) {
    using S = LatentShape<MT, NR>;
    constexpr int STAGES = S::STAGES;
    extern __shared__ uint8_t raw_smem[];
    uint8_t* const smem = raw_smem + ((1024u - (sm32(raw_smem) & 1023u)) & 1023u);
    const uint32_t qs = sm32(smem), ring = qs + S::RING_OFF, ps = qs + S::P_OFF;
    uint8_t* const psm = smem + S::P_OFF;
    LatentMisc& ms = *reinterpret_cast<LatentMisc*>(smem + S::MISC_OFF);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Limit limit = {&ms.abort, p.wait_ns};
    // weights are 2^(x - m), m being UP below a maximum: in fp16 up to 2^15, of 65504
    constexpr float UP = F16 ? 7.f : 0.f;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // the line: each thread counts a stretch of items; sums before it by shuffles
    const int items = p.B * p.RB, each = (items + NT - 1) / NT, i0 = min(items, tid * each), i1 = min(items, i0 + each);
    int mine = 0, own = 0;
    for (int i = i0; i < i1; ++i) {
        Item it;
        it.set(p, i);
        own = it.n;
        mine += own;
    }
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += a;
    }
    if (lane == 31) ms.scan[warp] = inc;
    if (tid == 0) {
        for (int i = 0; i < STAGES; ++i) {
            bar_init(&ms.kv_full[i], 1);
            bar_init(&ms.v_ok[i], 1);
            bar_init(&ms.pv_done[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&ms.s_full[i], 1);
            bar_init(&ms.s_free[i], 128);
            bar_init(&ms.p_ready[i], 128);
        }
        bar_init(&ms.q_ready, 128);
        bar_init(&ms.drained, 2);
        ms.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 5) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sm32(&ms.tmem)),
                     "n"(S::T_ALL)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    __syncthreads();
    int before = inc - mine, total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += ms.scan[w];
        total += ms.scan[w];
    }
    const int per = max((total + (int)gridDim.x - 1) / (int)gridDim.x, p.min_units);
    const int first = per * blockIdx.x, end = min(total, first + per);
    if (blockIdx.x == 0 || (first >= before && first < before + mine)) {
        int at = before;
        for (int i = i0; i < i1; ++i) {
            if (each > 1) {
                Item it;
                it.set(p, i);
                own = it.n;
            }
            if (blockIdx.x == 0) {
                p.base[i] = at;  // for the joining launch
                if (p.status && (long long)p.lens[i / p.RB] > (long long)p.pps << p.ps_shift) *p.status = MK_ERR_INVALID_ARG;
            }
            if (first >= at && first < at + own) ms.found_item = i, ms.found_base = at;
            at += own;
        }
    }
    if (blockIdx.x == 0 && tid == 0) p.base[items] = total;
    tm_before();
    __syncthreads();
    tm_after();
    const uint32_t tm = ms.tmem;
    int sent = 0;  // tiles that the copying warp has asked for
    if (first < end) {
        Line w;
        w.start(p, ms.found_item, first - ms.found_base);
        if (warp < 4) {
            // ================ softmax, and the pieces' ends ================
            const int r0 = 16 * warp + (lane >> 2);  // this thread's rows: r0 and r0 + 8
            const bool act = 16 * warp < NR;
            const uint32_t my = tm + ((uint32_t)(warp * 32) << 16);
            const float scale2 = p.scale * LOG2E;
            Spot at_c, back;
            bool ok = true;
            unsigned piece = 0;
            for (int u = first; u < end; ++piece) {
                const int take = min(w.it.n - w.tile, end - u);
                const Item& it = w.it;
                // queries, a row a warp: every product that read the last ones has ended (all its scores came)
                for (int r = warp; r < NR; r += 4) {
                    const int g = it.row0 + r, t = g / p.H, h = g - t * p.H;
                    const uint8_t* const a = p.q + 2 * (it.b * p.qb + t * p.qt + h * p.qh);
                    const uint8_t* const e = p.qr + 2 * (it.b * p.rb + t * p.rt + h * p.rh);
                    const bool in = r < it.rows;
                    if (p.q_vec) {
#pragma unroll
                        for (int c = lane; c < 8 * S::KP; c += 32)
                            cp16(qs + panel_at(0, NR, r, c), in ? (c < 16 * MT ? a + 16 * c : e + 16 * (c - 16 * MT)) : p.q, in);
                    } else {
                        for (int c = lane; c < 8 * S::KP; c += 32) {
                            uint32_t x[4] = {0, 0, 0, 0};
                            if (in) {
                                const uint16_t* const s2 =
                                    reinterpret_cast<const uint16_t*>(c < 16 * MT ? a + 16 * c : e + 16 * (c - 16 * MT));
#pragma unroll
                                for (int i = 0; i < 4; ++i) x[i] = s2[2 * i] | (uint32_t)s2[2 * i + 1] << 16;
                            }
                            *reinterpret_cast<uint4*>(smem + panel_at(0, NR, r, c)) = make_uint4(x[0], x[1], x[2], x[3]);
                        }
                    }
                }
                // where the rows' outputs go
                if (tid < it.rows) {
                    const int g = it.row0 + tid, t = g / p.H, h = g - t * p.H;
                    ms.to[tid] = it.b * p.ob + t * p.ot + h * p.oh;
                }
                cp_commit();
                cp_wait<0>();
                fence_async();
                bar_arrive(&ms.q_ready);
                int last[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = r0 + 8 * i;
                    const long long x = (long long)p.lens[it.b] - p.T + (it.row0 + r) / p.H;
                    last[i] = r < it.rows ? (int)max(-1ll, min(x, (long long)it.hi - 1)) : -1;
                }
                float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
                for (int i = 0; i < take; ++i) {
                    const int j0 = (it.t0 + w.tile + i) * TILE;
                    float x[2][TILE / 4];  // of row r0 and r0 + 8: columns 8 k + 2 (lane % 4) + {0, 1}
                    ok = ok && warp_wait(&ms.s_full[at_c.buf()], at_c.pair(), limit);
                    tm_after();
                    if (act) {
#pragma unroll
                        for (int h = 0; h < TILE / 32; ++h) {
                            uint32_t s[16];
                            tm_frag32(s, my + S::T_S + at_c.buf() * TILE + 32 * h);
                            tm_wait_ld();
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                // (rounded before a maximum is taken off: of large scores a fused step would leave their rounding)
                                x[0][8 * h + 2 * k] = __fmul_rn(__uint_as_float(s[4 * k]), scale2);
                                x[0][8 * h + 2 * k + 1] = __fmul_rn(__uint_as_float(s[4 * k + 1]), scale2);
                                x[1][8 * h + 2 * k] = __fmul_rn(__uint_as_float(s[4 * k + 2]), scale2);
                                x[1][8 * h + 2 * k + 1] = __fmul_rn(__uint_as_float(s[4 * k + 3]), scale2);
                            }
                        }
                    }
                    tm_before();
                    bar_arrive(&ms.s_free[at_c.buf()]);
                    float mx[2] = {-INFINITY, -INFINITY};
                    bool rise = false;
                    if (act) {
                        if (j0 < it.lo || j0 + TILE > it.common) {
#pragma unroll
                            for (int k = 0; k < TILE / 4; ++k) {
                                const int j = j0 + 8 * (k >> 1) + 2 * (lane & 3) + (k & 1);
                                if (j < it.lo || j > last[0]) x[0][k] = -INFINITY;
                                if (j < it.lo || j > last[1]) x[1][k] = -INFINITY;
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float a = x[e][0], b = x[e][1];
#pragma unroll
                            for (int k = 2; k < TILE / 4; k += 2) a = fmaxf(a, x[e][k]), b = fmaxf(b, x[e][k + 1]);
                            a = fmaxf(a, b);
                            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
                            mx[e] = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
                        }
                        rise = mx[0] - m[0] > UP + RISE || mx[1] - m[1] > UP + RISE;
                    }
                    if (i == 0) {
                        m[0] = mx[0] - UP, m[1] = mx[1] - UP;
                    } else if (bar_any(1, 128, rise)) {
                        // rows whose maximum rose: their outputs so far shrink
                        if (act) {
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float mn = mx[e] - m[e] > UP + RISE ? mx[e] - UP : m[e];
                                const float f = m[e] == -INFINITY ? 1.f : ex2(m[e] - mn);  // (nothing so far: zeros)
                                m[e] = mn;
                                l[e] *= f;
                                if ((lane & 3) == 0) ms.f[r0 + 8 * e] = f;
                            }
                        }
                        // every product so far is in the output
                        ok = ok && warp_wait(&ms.pv_done[back.stage], back.full(), limit);
                        bar_named(1, 128);
                        tm_after();
#pragma unroll 1
                        for (int mb = 0; mb < MT; ++mb)
#pragma unroll 1
                            for (int c = 0; c < NR; c += 16) {
                                uint32_t o[16];
                                tm_ld16(o, my + S::T_O + mb * NR + c);
                                tm_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * ms.f[c + e]);
                                tm_st16(my + S::T_O + mb * NR + c, o);
                            }
                        tm_wait_st();
                        tm_before();
                        bar_named(1, 128);
                    }
                    // the buffer is free when the product of the tile that it held last has read it
                    if (at_c.c >= 2) {  // (its stage is the one before `back`)
                        Spot two = back;
                        if (two.stage == 0) two.stage = STAGES - 1, --two.turn;
                        else --two.stage;
                        ok = ok && warp_wait(&ms.pv_done[two.stage], two.full(), limit);
                    }
                    if (act) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float ref = m[e] == -INFINITY ? 0.f : m[e];
                            const int r = r0 + 8 * e;
                            uint8_t* const row = psm + r * 128 + 4 * (lane & 3);
                            float s0 = 0.f, s1 = 0.f;
#pragma unroll
                            for (int k = 0; k < TILE / 8; ++k) {
                                const float a = ex2(x[e][2 * k] - ref), b = ex2(x[e][2 * k + 1] - ref);
                                s0 += a, s1 += b;
                                const int c = at_c.buf() * 4 + k;
                                *reinterpret_cast<uint32_t*>(row + ((c ^ (r & 7)) << 4)) = pack16<F16>(a, b);
                            }
                            l[e] += s0 + s1;
                        }
                    }
                    fence_async();
                    tm_before();
                    bar_arrive(&ms.p_ready[at_c.buf()]);
                    back = at_c;
                    at_c.next<STAGES>();
                }
                // ---- the piece: maxima and sums by row, then the output out of tensor memory
                if (act) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
                        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
                    }
                }
                ok = ok && warp_wait(&ms.pv_done[back.stage], back.full(), limit);
                if (act && (lane & 3) == 0) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // what sees a latent that is no number is none
                        const float l2 = last[e] >= ms.bad[piece & 15] ? __uint_as_float(0x7fffffffu) : l[e];
                        ms.m[r0 + 8 * e] = m[e];
                        ms.sum[r0 + 8 * e] = l2;
                        ms.f[r0 + 8 * e] = l2 == 0.f ? 0.f : 1.f / l2;
                    }
                }
                tm_before();
                // nor what a CTA that gave up leaves: a row's weights are one warp's, its outputs all four's
                const bool none = bar_any(1, 128, !ok);
                tm_after();
                const bool whole = take == it.n;
                float* const slot = p.slots + (2ll * blockIdx.x + (u == first ? 0 : 1)) * ((long long)NR * (S::RANK + 2));
#pragma unroll 1
                for (int c = 0; c < it.rows; c += 16) {
#pragma unroll 2
                    for (int mb = 0; mb < MT; ++mb) {
                        uint32_t o[16];
                        tm_ld16(o, my + S::T_O + mb * NR + c);
                        tm_wait_ld();
                        const int d = mb * 128 + warp * 32 + lane;
                        if (whole) {
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (c + e < it.rows)
                                    put16<F16>(p.out, ms.to[c + e] + d, none ? __uint_as_float(0x7fffffffu) : __uint_as_float(o[e]) * ms.f[c + e]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (c + e < it.rows) slot[(c + e) * S::RANK + d] = __uint_as_float(o[e]);
                        }
                    }
                }
                if (tid < it.rows) {
                    const float l2 = none ? __uint_as_float(0x7fffffffu) : ms.sum[tid];
                    if (!whole)
                        *reinterpret_cast<float2*>(slot + (long long)NR * S::RANK + 2 * tid) = make_float2(ms.m[tid], l2);
                    else if (p.lse)
                        p.lse[(long long)it.b * p.T * p.H + it.row0 + tid] = l2 == 0.f ? -INFINITY : (ms.m[tid] + log2f(l2)) * LN2;
                }
                tm_before();
                bar_named(1, 128);  // the outputs have been read
                u += take;
                w.on(p, take);
            }
        } else if (warp == 4) {
            // ================ copies ================
            // A tile is `parts` boxes of up to TILE rows of one page. The lanes hold the pages of the next 32 boxes, and
            // of the 32 after them.
            const int rows = min(TILE, 1 << p.ps_shift), parts = TILE / rows, mask = (1 << p.ps_shift) - 1;
            const int tiles = end - first, pshift = __ffs(parts) - 1;
            Line ahead = w;
            int ahead_c = lane >> pshift;
            ahead.on(p, ahead_c);
            auto page_next = [&] {  // of this lane's box of the next 32; one that nothing sees reads as zeros
                int page = p.n_pages;
                if (ahead_c < tiles) {
                    const int pos = ahead.at() + (lane & (parts - 1)) * rows;
                    if (pos < ahead.it.hi && pos + rows > ahead.it.lo) {
                        page = p.table[ahead.it.b * p.table_s + (pos >> p.ps_shift)];
                        if ((unsigned)page >= (unsigned)p.n_pages) {
                            page = p.n_pages;
                            if (p.status) *p.status = MK_ERR_INVALID_ARG;
                        }
                    }
                    ahead_c += 32 >> pshift;
                    ahead.on(p, 32 >> pshift);
                }
                return page;
            };
            int now = page_next(), next = 0;
            int box = 0;
            Spot pl;
            for (int c = 0; c < tiles; ++c, pl.next<STAGES>()) {
                const int j0 = w.at();
                w.on(p, 1);
                const uint32_t st = ring + pl.stage * S::STAGE_B;
                unsigned long long* const bar = &ms.kv_full[pl.stage];
                if (c >= STAGES && !warp_wait(&ms.pv_done[pl.stage], pl.free(), limit)) break;
                if (lane == 0) bar_expect(bar, S::STAGE_B);
                sent = c + 1;
                for (int i = 0; i < parts; ++i, ++box) {
                    const int page = __shfl_sync(0xffffffffu, now, box & 31);
                    if (lane == 0) {
                        const int row = (j0 + i * rows) & mask;
#pragma unroll
                        for (int x = 0; x < 2 * MT; ++x)
                            tma_3d(st + x * TILE * 128 + i * rows * 128, &maps.latent, x * 64, row, page, bar);
                        tma_3d(st + 2 * MT * TILE * 128 + i * rows * 128, &maps.rope, 0, row, page, bar);
                    }
                    if ((box & 31) == 0) next = page_next();
                    if ((box & 31) == 31) now = next;
                }
            }
        } else if (warp == 7) {
            // ================ rows that must not reach the output ================
            Spot pl;
            unsigned piece = 0;
            bool ok = true;
            for (int u = first; u < end && ok; ++piece) {
                const int take = min(w.it.n - w.tile, end - u);
                const Item& it = w.it;
                int bad = INT_MAX;
                for (int i = 0; i < take; ++i, pl.next<STAGES>()) {
                    const int j0 = (it.t0 + w.tile + i) * TILE;
                    if (!(ok = warp_wait(&ms.kv_full[pl.stage], pl.full(), limit))) break;
                    if (j0 < it.lo || j0 + TILE > it.common) {
                        uint8_t* const st = smem + S::RING_OFF + pl.stage * S::STAGE_B;
                        for (int r = 0; r < TILE; ++r) {
                            const int j = j0 + r;
                            const bool hidden = j < it.lo || j >= it.hi;
                            if (!hidden && j < it.common) continue;
                            for (int c = lane; c < 16 * MT; c += 32) {  // (the order within a panel's row does not matter)
                                uint4* const at = reinterpret_cast<uint4*>(st + (c >> 3) * TILE * 128 + r * 128 + (c & 7) * 16);
                                if (hidden) {
                                    *at = make_uint4(0, 0, 0, 0);
                                } else {
                                    const uint4 v = *at;
                                    if (not_finite<F16>(v.x) || not_finite<F16>(v.y) || not_finite<F16>(v.z) || not_finite<F16>(v.w)) {
                                        *at = make_uint4(0, 0, 0, 0);
                                        bad = min(bad, j);
                                    }
                                }
                            }
                        }
                        fence_async();
                    }
                    if (i == take - 1) {
                        bad = __reduce_min_sync(0xffffffffu, bad);
                        if (lane == 0) ms.bad[piece & 15] = bad;
                    }
                    __syncwarp();
                    if (lane == 0) bar_arrive(&ms.v_ok[pl.stage]);
                }
                u += take;
                w.on(p, take);
            }
        } else {
            // ================ products: two warps, one lane of each issues ================
            const uint32_t tmu = __shfl_sync(0xffffffffu, tm, 0);
            Spot at_c;
            unsigned piece = 0;
            bool ok = true;
            if (warp == 5) {
                constexpr uint32_t QK = mma_desc(64, TILE, false, false, F16);
                const uint64_t q = smem_desc(qs, 16, 1024), k0 = smem_desc(ring, 16, 1024);
                for (int u = first; u < end && ok; ++piece) {
                    const int take = min(w.it.n - w.tile, end - u);
                    u += take;
                    w.on(p, take);
                    ok = warp_wait(&ms.q_ready, piece & 1u, limit);
                    for (int i = 0; i < take && ok; ++i) {
                        // the tile is here; the softmax has read what the S buffer held two tiles ago
                        ok = warp_wait(&ms.kv_full[at_c.stage], at_c.full(), limit) &&
                             (at_c.c < 2 || warp_wait(&ms.s_free[at_c.buf()], at_c.pair_free(), limit));
                        if (!ok) break;
                        tm_after();
                        if (elect_one()) {
                            const uint64_t k = desc_on(k0, at_c.stage * S::STAGE_B);
                            const uint32_t d = tmu + S::T_S + at_c.buf() * TILE;
#pragma unroll
                            for (int j = 0; j < 4 * S::KP; ++j)
                                mma_ss(d, desc_on(q, (j >> 2) * NR * 128 + (j & 3) * 32),
                                       desc_on(k, (j >> 2) * TILE * 128 + (j & 3) * 32), QK, j > 0);
                            mma_commit(&ms.s_full[at_c.buf()]);
                        }
                        __syncwarp();
                        at_c.next<STAGES>();
                    }
                }
            } else {
                constexpr uint32_t PV = mma_desc(128, NR, false, true, F16);
                const uint64_t v0 = smem_desc(ring, TILE * 128, 1024), p0 = smem_desc(ps, 16, 1024);
                for (int u = first; u < end && ok; ++piece) {
                    const int take = min(w.it.n - w.tile, end - u);
                    u += take;
                    w.on(p, take);
                    for (int i = 0; i < take; ++i) {
                        ok = warp_wait(&ms.p_ready[at_c.buf()], at_c.pair(), limit) &&
                             warp_wait(&ms.v_ok[at_c.stage], at_c.full(), limit);
                        if (!ok) break;
                        tm_after();
                        if (elect_one()) {
                            const uint64_t v = desc_on(v0, at_c.stage * S::STAGE_B);
                            const uint64_t pb = desc_on(p0, at_c.buf() * 64);
                            // the first tile of a piece overwrites
#pragma unroll
                            for (int mb = 0; mb < MT; ++mb)
#pragma unroll
                                for (int j = 0; j < TILE / 16; ++j)
                                    mma_ss(tmu + S::T_O + mb * NR, desc_on(v, mb * 2 * TILE * 128 + j * 2048),
                                           desc_on(pb, j * 32), PV, i > 0 || j > 0);
                            if (at_c.c < p.signals) mma_commit(&ms.pv_done[at_c.stage]);
                        }
                        __syncwarp();
                        at_c.next<STAGES>();
                    }
                }
            }
            // the last products end before the tensor memory goes, also when a role gave up
            if (elect_one()) mma_commit(&ms.drained);
            const long long t0 = now_ns();
            while (!bar_try(&ms.drained, 0) && now_ns() - t0 < DRAIN_NS) {
            }
        }
    }
    __syncwarp();
    tm_before();
    __syncthreads();
    tm_after();
    if (ms.abort) {
        // copies may still be on their way into this CTA's memory: at most the ring's last tiles
        if (warp == 4) {
            const long long t0 = now_ns();
            for (int c = max(0, sent - STAGES); c < sent; ++c)
                while (!bar_try(&ms.kv_full[c % STAGES], (unsigned)(c / STAGES) & 1u) && now_ns() - t0 < DRAIN_NS) {
                }
        }
        if (tid == 0 && p.status) *p.status = MK_ERR_TIMEOUT;
        __syncthreads();
    }
    if (warp == 5)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "n"(S::T_ALL) : "memory");
}

// Joins the pieces of an output row. MANY rows: a block a row, a warp 128 values of it, piece after piece; else a block takes
// 128 values of a row and its four warps every fourth piece each, whose trips to memory would follow one another. Rows
// without a piece get their zeros, rows whose only piece went straight to the output are left alone.
constexpr int JT = 128;
template <int RANK, bool F16, bool MANY>
__global__ void __launch_bounds__(JT) latent_join(const __grid_constant__ LatentP p, int main_grid) {
    constexpr int CH = RANK / 128, W = MANY ? 1 : JT / 32;  // parts of a row; warps that share its pieces
    __shared__ float4 om[W][32];
    __shared__ float2 oml[W];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = MANY ? blockIdx.x : blockIdx.x / CH, d0 = (MANY ? warp : (int)blockIdx.x - row * CH) * 128, first = MANY ? 0 : warp;
    const int rows = p.T * p.H, b = row / rows, g = row - b * rows, rb = g / p.rows_blk, r = g - rb * p.rows_blk;
    const int item = b * p.RB + rb, t = g / p.H, h = g - t * p.H;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int total = p.base[p.B * p.RB], t0 = p.base[item], n = p.base[item + 1] - t0;
    const int per = max((total + main_grid - 1) / main_grid, p.min_units);
    const int c0 = t0 / per, c1 = n ? (t0 + n - 1) / per : c0 - 1;
    if (n && c0 == c1) return;
    const long long slot_f = (long long)p.nr * (RANK + 2);
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int c = c0 + first; c <= c1; c += W) {
        // a CTA's first piece is the one that its stretch begins with
        const float* const s = p.slots + (2ll * c + (t0 <= c * per ? 0 : 1)) * slot_f;
        const float2 ml = *reinterpret_cast<const float2*>(s + p.nr * RANK + 2 * r);
        const float4 y = *reinterpret_cast<const float4*>(s + r * RANK + d0 + 4 * lane);
        const float mn = fmaxf(m, ml.x), ref = mn == -INFINITY ? 0.f : mn, f = ex2(m - ref), w = ex2(ml.x - ref);
        m = mn;
        l = l * f + ml.y * w;
        o.x = o.x * f + y.x * w, o.y = o.y * f + y.y * w, o.z = o.z * f + y.z * w, o.w = o.w * f + y.w * w;
    }
    const long long to = b * p.ob + t * p.ot + h * p.oh + d0;
    if constexpr (MANY) {
        const float x[4] = {o.x, o.y, o.z, o.w};
        uint16_t z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) put16<F16>(reinterpret_cast<uint8_t*>(z), i, l == 0.f ? 0.f : x[i] / l);
        uint16_t* const at = reinterpret_cast<uint16_t*>(p.out) + to + 4 * lane;
        if (((uintptr_t)at & 7) == 0) {
            *reinterpret_cast<uint2*>(at) = make_uint2(z[0] | (uint32_t)z[1] << 16, z[2] | (uint32_t)z[3] << 16);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) at[i] = z[i];
        }
        if (threadIdx.x == 0 && p.lse) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
        return;
    }
    om[first][lane] = o;
    if (lane == 0) oml[first] = make_float2(m, l);
    __syncthreads();
    float mm = -INFINITY, ll = 0.f, y = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) mm = fmaxf(mm, oml[i].x);
    const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const float w = ex2(oml[i].x - ref);
        ll += oml[i].y * w;
        y += reinterpret_cast<const float*>(om[i])[threadIdx.x] * w;
    }
    put16<F16>(p.out, to + threadIdx.x, ll == 0.f ? 0.f : y / ll);
    if (threadIdx.x == 0 && d0 == 0 && p.lse) p.lse[row] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * LN2;
}

// ---- host

// latents or rope parts as a tensor [page][row][value]; a box is up to TILE rows of a page by 64 values, in the 128-byte
// swizzled order the products read
int map_of(const void* base, int width, const mk_latent_pages& g, int64_t page_s, int64_t row_s, CUtensorMap* out) {
    const EncodeFn encode = encode_fn();
    if (!encode) return fail(MK_ERR_CUDA, "latent attend: the driver has no cuTensorMapEncodeTiled");
    const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)g.page_size, (cuuint64_t)g.n_pages};
    const cuuint64_t strides[2] = {(cuuint64_t)row_s * 2, (cuuint64_t)page_s * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)(g.page_size < TILE ? g.page_size : TILE), 1}, one[3] = {1, 1, 1};
    const CUresult r = encode(out, g.dtype == MK_DT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                              const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(MK_ERR_CUDA, "latent attend: cuTensorMapEncodeTiled failed (%d)", (int)r);
    return MK_OK;
}

struct Plan {
    bool rows;  // a block a row
    int nr, rows_blk, RB, grid, dev, sms;
    int64_t slots_off, bytes;
};

// Tiles a CTA takes at least: fewer make more pieces for the join, more a longer line. One sequence of 8192, 16
// heads: 2 18.4 us, 3 16.2, 4 15.1, 8 15.8; of 1024: 2 10.3, 3 10.5, 4 11.1, 8 13.8.
constexpr int MIN_UNITS = 4;

template <int MT, int NR, bool F16>
int run(const LatentP* p, const mk_latent_pages* g, int dev, int sms, int grid, cudaStream_t s) {
    using S = LatentShape<MT, NR>;
    auto kern = latent_kernel<MT, NR, F16>;
    static std::atomic<uint64_t> done;
    if (const int rc = allow_smem(kern, S::SMEM, dev, done, "mk_latent_attend")) return rc;
    LatentMaps maps;
    if (const int rc = map_of(g->latent, g->rank, *g, g->page_stride, g->row_stride, &maps.latent)) return rc;
    if (const int rc = map_of(g->rope, 64, *g, g->rope_page_stride, g->rope_row_stride, &maps.rope)) return rc;
    kern<<<grid, NT, S::SMEM, s>>>(*p, maps);
    if (const int rc = cuda_status(cudaGetLastError(), "mk_latent_attend")) return rc;
    cudaLaunchConfig_t cfg = {};
    // Many rows of a few pieces each. Whole calls with and without: 64 sequences of 7 tokens at up to 8192 (7168 rows, 2 pieces)
    // 161 and 182 us, 16 of 128 heads (2048 rows, 5 pieces) 53 and 57; 8 of 7 tokens (896 rows, 10 pieces) 43 and 38.
    const int rows = p->B * p->T * p->H;
    const bool many = rows >= 4 * sms && grid <= 6 * (int64_t)p->B * p->RB;
    cfg.gridDim = dim3((unsigned)(many ? rows : rows * MT));
    cfg.blockDim = dim3(many ? 32 * MT : JT);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cuda_status(many ? cudaLaunchKernelEx(&cfg, latent_join<128 * MT, F16, true>, *p, grid)
                            : cudaLaunchKernelEx(&cfg, latent_join<128 * MT, F16, false>, *p, grid), "mk_latent_attend");
}

int check(const mk_latent_attention* a) {
    if (!a) return fail(MK_ERR_INVALID_ARG, "latent attend: NULL arguments");
    if (const int rc = check_latent(a->pages, a->table)) return rc;
    const mk_latent_pages& g = *a->pages;
    if (a->n_tokens < 1 || a->n_heads < 1) return fail(MK_ERR_INVALID_ARG, "latent attend: n_tokens or n_heads below 1");
    if (!a->lens || off_by4(a->lens, a->starts, a->lse, a->status))
        return fail(MK_ERR_INVALID_ARG, "latent attend: lens is NULL, or lens, starts, lse or status not aligned to 4 bytes");
    if (const int rc = check_rows(a->q, "latent attend", "q")) return rc;
    if (const int rc = check_rows(a->q_rope, "latent attend", "q_rope")) return rc;
    if (const int rc = check_rows(a->out, "latent attend", "out")) return rc;
    if (a->q->dtype != g.dtype || a->q_rope->dtype != g.dtype || a->out->dtype != g.dtype)
        return fail(MK_ERR_INVALID_ARG, "latent attend: q, q_rope and out must have the cache's type");
    if (!(a->scale >= -1e30f && a->scale <= 1e30f)) return fail(MK_ERR_INVALID_ARG, "latent attend: scale is not a number in range");
    if ((g.rank != 256 && g.rank != 512) || g.rope_dim != 64)
        return fail(MK_ERR_UNSUPPORTED, "latent attend: rank must be 256 or 512, rope_dim 64");
    if ((int64_t)a->table->batch * a->n_tokens * a->n_heads > INT32_MAX / 16)
        return fail(MK_ERR_UNSUPPORTED, "latent attend: too many queries in one call");
    return MK_OK;
}

int make_plan(const mk_latent_attention* a, Plan& pl) {
    if (const int rc = check(a)) return rc;
    const mk_latent_pages& g = *a->pages;
    const mk_page_table& t = *a->table;
    pl = {};
    pl.rows = g.page_size < 8 || !g.page_stride || !g.row_stride || !g.rope_page_stride || !g.rope_row_stride;
    if (pl.rows) return MK_OK;
    if (const int rc = device_sms(pl.dev, pl.sms, "mk_latent_attend")) return rc;
    const int rows = a->n_tokens * a->n_heads;
    pl.RB = (rows + 63) / 64;
    pl.rows_blk = (rows + pl.RB - 1) / pl.RB;
    pl.RB = (rows + pl.rows_blk - 1) / pl.rows_blk;
    pl.nr = pl.rows_blk <= 16 ? 16 : pl.rows_blk <= 32 ? 32 : 64;
    const int64_t items = (int64_t)t.batch * pl.RB, cap = (int64_t)t.pages_per_seq * g.page_size;
    const int64_t most = items * ((cap + TILE - 1) / TILE + 1);
    if (most > (1 << 30)) return fail(MK_ERR_UNSUPPORTED, "latent attend: too many positions in one call");
    const int64_t want = (most + MIN_UNITS - 1) / MIN_UNITS;
    pl.grid = (int)(want < pl.sms ? want : pl.sms);
    pl.slots_off = ((items + 1) * 4 + 255) / 256 * 256;
    pl.bytes = pl.slots_off + 2ll * pl.grid * pl.nr * (g.rank + 2) * 4;
    pl.bytes = (pl.bytes + 255) / 256 * 256;
    return MK_OK;
}

}  // namespace

extern "C" int mk_latent_attend_workspace(const mk_latent_attention* a, int64_t* bytes) {
    Plan pl;
    if (const int rc = make_plan(a, pl)) return rc;
    if (!bytes) return fail(MK_ERR_INVALID_ARG, "latent attend: NULL bytes");
    *bytes = pl.bytes;
    return MK_OK;
}

extern "C" int mk_latent_attend(const mk_latent_attention* a, void* workspace, int64_t workspace_bytes, void* stream) {
    Plan pl;
    if (const int rc = make_plan(a, pl)) return rc;
    if (pl.bytes && (!workspace || (uintptr_t)workspace % 256 || workspace_bytes < pl.bytes))
        return fail(MK_ERR_INVALID_ARG, "latent attend: the workspace must be %lld bytes, aligned to 256", (long long)pl.bytes);
    const mk_latent_pages& g = *a->pages;
    const mk_page_table& t = *a->table;
    LatentP p = {};
    p.latent = (const uint8_t*)g.latent, p.rope = (const uint8_t*)g.rope;
    p.page_s = g.page_stride, p.row_s = g.row_stride, p.rope_page_s = g.rope_page_stride, p.rope_row_s = g.rope_row_stride;
    p.table = t.table, p.table_s = t.stride, p.lens = a->lens, p.starts = a->starts;
    p.q = (const uint8_t*)a->q->data, p.qb = a->q->seq_stride, p.qt = a->q->token_stride, p.qh = a->q->head_stride;
    p.qr = (const uint8_t*)a->q_rope->data, p.rb = a->q_rope->seq_stride, p.rt = a->q_rope->token_stride, p.rh = a->q_rope->head_stride;
    p.out = (uint8_t*)a->out->data, p.ob = a->out->seq_stride, p.ot = a->out->token_stride, p.oh = a->out->head_stride;
    p.lse = a->lse, p.status = a->status;
    p.pps = t.pages_per_seq, p.ps_shift = log2_exact(g.page_size), p.n_pages = g.n_pages, p.B = t.batch;
    p.T = a->n_tokens, p.H = a->n_heads, p.scale = a->scale;
    cudaStream_t s = (cudaStream_t)stream;
    const bool f16 = g.dtype == MK_DT_F16, wide = g.rank == 512;
    if (pl.rows) {
        const int grid = p.B * p.T * p.H;
        if (f16) wide ? latent_rows<MK_DT_F16, 512, 64><<<grid, LT, 0, s>>>(p) : latent_rows<MK_DT_F16, 256, 64><<<grid, LT, 0, s>>>(p);
        else wide ? latent_rows<MK_DT_BF16, 512, 64><<<grid, LT, 0, s>>>(p) : latent_rows<MK_DT_BF16, 256, 64><<<grid, LT, 0, s>>>(p);
        return cuda_status(cudaGetLastError(), "mk_latent_attend");
    }
    p.nr = pl.nr, p.rows_blk = pl.rows_blk, p.RB = pl.RB, p.min_units = MIN_UNITS;
    p.base = (int*)workspace, p.slots = (float*)((uint8_t*)workspace + pl.slots_off);
    const long long ns = mk_wait_ns_();
    p.wait_ns = (unsigned)(ns < 4000000000ll ? ns : 4000000000ll);
    p.signals = signalled_tiles();
    p.q_vec = rows_vec(a->q) && rows_vec(a->q_rope);
    auto go = [&](auto MT, auto NR) {
        constexpr int mt = decltype(MT)::value, nr = decltype(NR)::value;
        return f16 ? run<mt, nr, true>(&p, &g, pl.dev, pl.sms, pl.grid, s) : run<mt, nr, false>(&p, &g, pl.dev, pl.sms, pl.grid, s);
    };
    using std::integral_constant;
    auto rank = [&](auto MT) {
        if (pl.nr == 16) return go(MT, integral_constant<int, 16>());
        return pl.nr == 32 ? go(MT, integral_constant<int, 32>()) : go(MT, integral_constant<int, 64>());
    };
    return wide ? rank(integral_constant<int, 4>()) : rank(integral_constant<int, 2>());
}
