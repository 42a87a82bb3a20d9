// mk_prefix.cuh -- attention over positions that all rows of an item see, on
// the fifth-generation tensor cores: a prefix that the sequences of a batch
// share (rows of the whole batch), or, in calls with many rows a sequence, the
// tiles that all of its tokens see whole. Everything that is masked for some
// row stays with mk_attend.cuh, so that no row here sees a part of a tile.
//
// The rows of a kv head (tokens and query heads of the group) stand against
// one copy of K and V, 128 rows a CTA, 64 positions a tile:
//   S = Q K^T   128 x 64, both operands in shared memory, S in tensor memory;
//   P = 2^(x - m) per row, one thread a row (tensor memory gives a thread its
//       row, so that no value crosses threads);
//   O += P V    P as the tensor-memory operand, V from shared memory as it
//       lies there (rows are the product's K: the transposed form), O in
//       tensor memory for the item's whole stretch of tiles.
// P goes in as bf16 hi + lo parts (16 bits of each probability) in two chains
// of products. O is rescaled only when a row's maximum has risen by more than
// 2^8 since its reference: until then probabilities up to 2^8 and their sum are
// as exact as ones below 1.
//
// Two groups of four warps: softmax, a row a thread, of the even and of the odd
// tiles; each group keeps its own maxima, sums and output, which meet at the
// piece's end. Then loads (bf16 pages: one warp, by tensor maps; 8-bit pages:
// four warps, which turn staged codes into bf16 -- E4M3 and INT8 codes are
// exact in it; the K scale multiplies the score, the V scale the probability)
// and two warps, an elected thread of each issuing Q K^T and P V; S of the next
// tile comes before P V of this one, so that the tensor cores work while the
// softmax does. fp16 queries are two bf16 parts, one more chain of Q K^T. All
// waits are on mbarriers with a limit; a wait that runs out raises a flag that
// every role sees, and the CTA leaves after freeing its tensor memory
// (MK_ERR_TIMEOUT in `status`, NaN in its rows).
//
// Bound by latency: a tile of 128-wide heads takes about 2000 cycles (54 tiles a
// CTA in 106,000, bf16). Q K^T of 128 x 64 takes 48 cycles a 16-wide step (its
// operands' shared-memory reads), the two chains of P V 64 each, 875 cycles of
// products (the tensor pipe is busy 39 % of the time); the tile's 2980 warp
// instructions are 745 issue slots of each scheduler, 8192 exponentials at 16 a
// cycle 512. What is left is the chain from a tile's scores to its
// probabilities, of which two warps a scheduler are on the way. 8-bit pages: the
// four warps that convert, 3400 (E4M3) to 4100 (INT8) cycles a tile. Work is cut
// as in mk_attend.cuh; every piece goes to the workspace for the joining launch.
//
// Measured, 64 sequences on 16384 shared positions, 40 query heads on 8 of 128,
// bf16: 50 us for this launch by a profiler that runs launches one by one (0.65
// PFLOP/s with both parts of P counted, 34 % of a large product's rate), 91 us
// for the call with up to 1024 positions of each sequence's own; INT8 118 us,
// fp16 queries 99 us. 256 tokens at 16384 positions of one sequence, 16 query
// heads on 4: 84 us.
#pragma once
#include "mk_attend.cuh"

namespace mkop {

// SPLITQ: fp16 queries, as two bf16 parts (their 11 bits and range fit them)
template <int D, int FMT, bool SPLITQ>
struct PrefixShape {
    static constexpr bool F8 = FMT != MK_KV_BF16;
    static constexpr int ROWS = 128, TILE = 64;
    static constexpr int PANELS = D / 64;          // 128-byte wide panels of a row
    static constexpr int Q_PART = PANELS * ROWS * 128, Q_B = Q_PART * (SPLITQ ? 2 : 1);
    static constexpr int KV_B = PANELS * TILE * 128;  // K (or V) of a tile
    static constexpr int STAGE_B = 2 * KV_B;
    static constexpr int SCALE_B = 2 * TILE * 4;   // of a stage: K scales, V scales (8-bit pages)
    static constexpr int STAGES = D == 128 ? (F8 ? 3 : SPLITQ ? 4 : 5) : (F8 ? 6 : 8);
    static constexpr int RAW_B = 2 * TILE * D + SCALE_B, RAWS = 3;  // staged codes and scales of a tile
    static constexpr int SC_OFF = Q_B + STAGES * STAGE_B;
    static constexpr int RAW_OFF = SC_OFF + STAGES * SCALE_B;
    static constexpr int MISC_OFF = RAW_OFF + (F8 ? RAWS * RAW_B : 0);
    static constexpr int MISC_B = 4096;
    static constexpr int SMEM = MISC_OFF + MISC_B + 1024;  // and room to align to 1024
    static constexpr int LOADERS = F8 ? 4 : 1, NT = 32 * (8 + LOADERS + 2);  // warps: softmax, loads, products
    // tensor memory columns of the two groups: S, P (hi, lo), O
    static constexpr int T_S = 0, T_P = 2 * TILE, T_O = T_P + 2 * TILE, T_ALL = 512;
    static_assert(T_O + 2 * D <= T_ALL && SMEM <= 227 * 1024, "");
};

struct PrefixMisc {
    unsigned long long kv_full[8], pv_done[8], s_full[2], s_free[2], p_ready[2], q_ready, drained;
    unsigned tmem, abort;
    int scan[16], found_b, found_base;
    long long off[2][64];  // where a tile's rows lie (bytes), -1: zeros
    float2 stat[2][128];   // (maximum, sum) of each group's rows
};

// A role's place in the line of items and their tiles. Shared launch: one
// sequence, whose items all have n tiles. Wide calls: the tiles that a
// sequence's rows see whole, sequence after sequence.
struct Walk {
    int b, item, tile, n, t0;  // sequence, item of it, tile of the item, tiles of the item, the first one's number
    __device__ __forceinline__ void count(const AttendP& p) {
        if (p.wide) {
            int g1;
            whole_tiles(p, b, t0, g1);
            n = g1 - t0;
        } else {
            t0 = 0;
            n = (p.shared + 63) / 64;
        }
    }
    // to tile u of the line; tiles of sequence b begin at `base`
    __device__ __forceinline__ void start(const AttendP& p, int u, int seq, int base) {
        b = seq;
        count(p);
        n = max(n, 1);
        item = min((u - base) / n, p.H * p.RB - 1);
        tile = u - base - item * n;
    }
    // k tiles on; behind the last item is one without an end
    __device__ __forceinline__ void on(const AttendP& p, int k) {
        tile += k;
        while (tile >= n) {
            tile -= n;
            if (++item < p.H * p.RB) continue;
            item = 0;
            do {
                if (p.wide && b + 1 < p.B) {
                    ++b;
                    count(p);
                } else {
                    n = INT_MAX;
                }
            } while (n == 0);
        }
    }
    __device__ __forceinline__ int at() const { return (t0 + tile) * 64; }
};

// Four codes as two bf16 pairs, exact. E4M3: through fp16 and fp32. INT8: the
// low seven bits as the mantissa of 128 (whose bf16 step is 1), less 128, or
// less 256 where the sign bit is set.
template <int FMT>
__device__ __forceinline__ void codes_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (FMT == MK_KV_E4M3) {
        uint32_t a, b;
        e4m3_quad(w, a, b);
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
        lo = pack_bf16(x.x, x.y);
        hi = pack_bf16(y.x, y.y);
    } else {
        auto pair = [](uint32_t v) {
            const uint32_t x = v & 0xff7fff7fu, c = v & 0xff80ff80u;
            const __nv_bfloat162 r =
                __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&c));
            return *reinterpret_cast<const uint32_t*>(&r);
        };
        lo = pair(__byte_perm(w, 0x43434343u, 0x4140));
        hi = pair(__byte_perm(w, 0x43434343u, 0x4342));
    }
}

// K and V as tensors [page][kv head][row][value] (bf16 pages)
struct PrefixMaps {
    CUtensorMap k, v;
};
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int x, int row, int head, int page,
                                         unsigned long long* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(row), "r"(head), "r"(page), "r"(sm32(bar))
        : "memory");
}
template <int D, int FMT, bool SPLITQ>
__global__ void __launch_bounds__(PrefixShape<D, FMT, SPLITQ>::NT, 1)
    prefix_kernel(const __grid_constant__ AttendP p, const __grid_constant__ PrefixMaps maps) {
    using S = PrefixShape<D, FMT, SPLITQ>;
    constexpr bool F8 = S::F8;
    constexpr int TILE = S::TILE, ROWS = S::ROWS;
    extern __shared__ uint8_t raw_smem[];
    uint8_t* const smem = raw_smem + ((1024u - (sm32(raw_smem) & 1023u)) & 1023u);
    const uint32_t qs = sm32(smem), ring = qs + S::Q_B;
    float* const scales = reinterpret_cast<float*>(smem + S::SC_OFF);
    PrefixMisc& ms = *reinterpret_cast<PrefixMisc*>(smem + S::MISC_OFF);
    static_assert(sizeof(PrefixMisc) <= S::MISC_B, "");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Limit wait_limit = {&ms.abort, p.wait_ns};

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // (the host sees to it that the tiles of all items fit 32 bits)
    const int items = p.H * p.RB;  // of a sequence
    int limit = p.wide ? p.pps << p.ps_shift : p.shared;  // positions
    int total, mine = 0, before = 0;
    const int each = (p.B + S::NT - 1) / S::NT, b0 = min(p.B, tid * each), b1 = min(p.B, b0 + each);
    auto tiles_of = [&](int b) {
        int g0, g1;
        whole_tiles(p, b, g0, g1);
        return (g1 - g0) * items;
    };
    if (p.wide) {
        // each thread counts a stretch of sequences; sums before it by shuffles
        for (int b = b0; b < b1; ++b) mine += tiles_of(b);
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int a = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += a;
        }
        if (lane == 31) ms.scan[warp] = inc;
        __syncthreads();
        before = inc - mine;
        total = 0;
#pragma unroll
        for (int w = 0; w < S::NT / 32; ++w) {
            if (w < warp) before += ms.scan[w];
            total += ms.scan[w];
        }
        if (blockIdx.x == 0) {  // for the joining launch
            int at = before;
            for (int b = b0; b < b1; ++b) {
                p.base[b] = at;
                at += tiles_of(b);
            }
            if (tid == 0) p.base[p.B] = total;
        }
    } else {
        total = items * ((p.shared + TILE - 1) / TILE);
    }
    const int per = (int)units_each(total, gridDim.x, p.min_units);
    const int first = per * blockIdx.x, end = min(total, first + per);
    if (first >= end) return;
    if (p.wide) {
        if (first >= before && first < before + mine) {
            ms.found_b = b0;
            ms.found_base = before;
            for (int b = b0, at = before; b < b1; ++b) {
                const int n = tiles_of(b);
                if (first < at + n) {
                    ms.found_b = b;
                    ms.found_base = at;
                    break;
                }
                at += n;
            }
        }
    } else {
        const int b = first_sharing(p, S::NT, &ms.scan[0]);
        if (b == INT_MAX) limit = 0;  // no sequence takes part, and no page is looked up
        if (tid == 0) ms.found_b = b == INT_MAX ? 0 : b, ms.found_base = 0;
    }
    // warps of a group that have rows at all
    const int act = p.RB > 1 ? 4 : (p.rows_item + 31) / 32;

    if (tid == 0) {
        for (int i = 0; i < S::STAGES; ++i) {
            bar_init(&ms.kv_full[i], F8 ? 128 : 1);
            bar_init(&ms.pv_done[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&ms.s_full[i], 1);
            bar_init(&ms.s_free[i], 32 * act);
            bar_init(&ms.p_ready[i], 32 * act);
        }
        bar_init(&ms.q_ready, 64 * act);
        bar_init(&ms.drained, 2);
        ms.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    constexpr int MMA_WARP = 8 + S::LOADERS;
    if (warp == MMA_WARP) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sm32(&ms.tmem)),
                     "n"(S::T_ALL)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tm_before();
    __syncthreads();
    tm_after();
    const uint32_t tm = ms.tmem;
    Walk w;
    w.start(p, first, ms.found_b, ms.found_base);
    int sent = 0;  // tiles that the tensor maps' warp has asked for

    // Tiles are counted over all pieces: tile c uses stage c % STAGES, S and P buffer c & 1.
    if (warp < 8 && (warp & 3) >= act) {
        // rows that no item has: nothing of them is read
    } else if (warp < 8) {
        // ================ softmax, a row a thread ================
        const int wg = warp >> 2, lrow = tid & 127;
        const uint32_t my = tm + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t my_s = my + S::T_S + wg * TILE, my_p = my + S::T_P + wg * TILE, my_o = my + S::T_O + wg * D;
        Place<S::STAGES> at_c, back;  // the group's tile, and its last one
        int parity = 0;               // of the tile that comes next, over both groups
        if (wg) at_c.next();
        bool ok = true;
        for (int u = first; u < end;) {
            const int take = min(w.n - w.tile, end - u);
            const int h = w.item / p.RB, rb = w.item - h * p.RB;
            const int row = rb * ROWS + lrow;
            const bool real = row < p.rows_item;
            const int bt = real ? row / p.G : 0, g = real ? row - bt * p.G : 0;
            const int b = p.wide ? w.b : bt / p.T, t = p.wide ? bt : bt - b * p.T;
            // half of the row's query, fetched while the length is; every product that read the last one has
            // ended (all scores came)
            bool live;
            {
                const uint16_t* src = p.q + b * p.qb + t * p.qt + (long long)(h * p.G + g) * p.qh + wg * (D / 2);
                uint4 x[D / 16];
                if (((uintptr_t)src & 15) == 0) {
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) x[j] = reinterpret_cast<const uint4*>(src)[j];
                } else {
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[e] = src[8 * j + 2 * e] | (uint32_t)src[8 * j + 2 * e + 1] << 16;
                        x[j] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                live = real && (p.wide || shares(p, b));
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    uint4 hi = live ? x[j] : make_uint4(0, 0, 0, 0);
                    const uint32_t to = panel_at(0, ROWS, lrow, wg * (D / 16) + j);
                    if constexpr (SPLITQ) {
                        uint4 lo;
                        auto split = [](uint32_t& v, uint32_t& rest) {
                            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
                            v = pack_bf16(f.x, f.y);
                            rest = pack_bf16(f.x - bf2f(v & 0xffffu), f.y - __uint_as_float(v & 0xffff0000u));
                        };
                        split(hi.x, lo.x), split(hi.y, lo.y), split(hi.z, lo.z), split(hi.w, lo.w);
                        *reinterpret_cast<uint4*>(smem + S::Q_PART + to) = lo;
                    }
                    *reinterpret_cast<uint4*>(smem + to) = hi;
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                bar_arrive(&ms.q_ready);
            }
            // score to exponent of 2, or to the cap's argument
            const float scale2 = p.scale * LOG2E, in2 = p.cap > 0.f ? scale2 * (2.f / p.cap) : scale2;
            const float slope2 = p.slopes ? p.slopes[h * p.G + g] * LOG2E : 0.f;
            const int at = live ? p.lens[b] - p.T + t : 0;
            float m = -INFINITY, l = 0.f;
            bool fresh = true;  // no tile of this piece yet
            for (int i = (parity ^ wg) & 1; i < take && ok; i += 2) {
                const int stage = at_c.stage;
                const int j0 = w.at() + i * TILE;
                if (!(ok = warp_wait(&ms.s_full[wg], at_c.pair(), wait_limit))) break;
                tm_after();
                uint32_t s0[32], s1[32];
                tm_ld32(s0, my_s);
                tm_ld32(s1, my_s + 32);
                tm_wait_ld();
                tm_before();
                bar_arrive(&ms.s_free[wg]);
                const float* ksc = scales + stage * 2 * TILE;
                // the scales come with the tile
                if (F8 && !(ok = warp_wait(&ms.kv_full[stage], at_c.full(), wait_limit))) break;
                if constexpr (F8) {
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 a = *reinterpret_cast<const float4*>(ksc + j);
                        const float4 e = *reinterpret_cast<const float4*>(ksc + 32 + j);
                        s0[j] = __float_as_uint(__uint_as_float(s0[j]) * a.x), s0[j + 1] = __float_as_uint(__uint_as_float(s0[j + 1]) * a.y);
                        s0[j + 2] = __float_as_uint(__uint_as_float(s0[j + 2]) * a.z), s0[j + 3] = __float_as_uint(__uint_as_float(s0[j + 3]) * a.w);
                        s1[j] = __float_as_uint(__uint_as_float(s1[j]) * e.x), s1[j + 1] = __float_as_uint(__uint_as_float(s1[j + 1]) * e.y);
                        s1[j + 2] = __float_as_uint(__uint_as_float(s1[j + 2]) * e.z), s1[j + 3] = __float_as_uint(__uint_as_float(s1[j + 3]) * e.w);
                    }
                }
                if (p.cap > 0.f || p.slopes) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        s0[j] = __float_as_uint(__uint_as_float(s0[j]) * in2);
                        s1[j] = __float_as_uint(__uint_as_float(s1[j]) * in2);
                    }
                    if (p.cap > 0.f) {
                        float far = 0.f;
#pragma unroll
                        for (int j = 0; j < 32; ++j) far = fmaxf(far, fmaxf(fabsf(__uint_as_float(s0[j])), fabsf(__uint_as_float(s1[j]))));
                        if (__all_sync(0xffffffffu, far < CAP_NEAR)) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) {
                                s0[j] = __float_as_uint(cap_near(__uint_as_float(s0[j]), 0.5f * p.cap));
                                s1[j] = __float_as_uint(cap_near(__uint_as_float(s1[j]), 0.5f * p.cap));
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < 32; ++j) {
                                s0[j] = __float_as_uint(cap_any(__uint_as_float(s0[j]), p.cap));
                                s1[j] = __float_as_uint(cap_any(__uint_as_float(s1[j]), p.cap));
                            }
                        }
                    }
                    if (p.slopes) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            s0[j] = __float_as_uint(__uint_as_float(s0[j]) - slope2 * (float)(at - j0 - j));
                            s1[j] = __float_as_uint(__uint_as_float(s1[j]) - slope2 * (float)(at - j0 - 32 - j));
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        s0[j] = __float_as_uint(__uint_as_float(s0[j]) * scale2);
                        s1[j] = __float_as_uint(__uint_as_float(s1[j]) * scale2);
                    }
                }
                if (j0 > limit - TILE) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if (j0 + j >= limit) s0[j] = 0xff800000u;
                        if (j0 + 32 + j >= limit) s1[j] = 0xff800000u;
                    }
                }
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int j = 0; j < 32; ++j) top[j & 3] = fmaxf(top[j & 3], fmaxf(__uint_as_float(s0[j]), __uint_as_float(s1[j])));
                const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                // the reference: the first tile's maximum, or a new one past 2^8 of the old
                const bool rise = mx > m + 8.f;
                if (fresh) {
                    m = mx;
                } else if (__any_sync(0xffffffffu, rise)) {
                    const float mn = rise ? mx : m;
                    const float f = ex2((m == -INFINITY ? (mn == -INFINITY ? 0.f : -INFINITY) : m) - (mn == -INFINITY ? 0.f : mn));
                    m = mn;
                    l *= f;
                    // every product so far is in O
                    if (!(ok = warp_wait(&ms.pv_done[back.stage], back.full(), wait_limit))) break;
                    tm_after();
#pragma unroll 1
                    for (int d = 0; d < D; d += 32) {
                        uint32_t o[32];
                        tm_ld32(o, my_o + d);
                        tm_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tm_st32(my_o + d, o);
                    }
                    tm_wait_st();
                }
                const float ref = m == -INFINITY ? 0.f : m;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
                uint32_t hi[32], lo[32];
                auto pair = [&](uint32_t a, uint32_t b2, float va, float vb, uint32_t& ph, uint32_t& pl, float& s) {
                    float x = ex2(__uint_as_float(a) - ref), y = ex2(__uint_as_float(b2) - ref);
                    s += x + y;
                    if constexpr (F8) {
                        x *= va, y *= vb;
                        ph = pack_bf16(x, y);
                        pl = pack_bf16(x - bf2f(ph & 0xffffu), y - __uint_as_float(ph & 0xffff0000u));
                    } else {
                        split_bf16(x, y, ph, pl);
                    }
                };
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    float4 va = make_float4(1.f, 1.f, 1.f, 1.f), vb = va;
                    if constexpr (F8) {
                        va = *reinterpret_cast<const float4*>(ksc + TILE + 2 * j);
                        vb = *reinterpret_cast<const float4*>(ksc + TILE + 32 + 2 * j);
                    }
                    pair(s0[2 * j], s0[2 * j + 1], va.x, va.y, hi[j], lo[j], sum[0]);
                    pair(s0[2 * j + 2], s0[2 * j + 3], va.z, va.w, hi[j + 1], lo[j + 1], sum[1]);
                    pair(s1[2 * j], s1[2 * j + 1], vb.x, vb.y, hi[16 + j], lo[16 + j], sum[2]);
                    pair(s1[2 * j + 2], s1[2 * j + 3], vb.z, vb.w, hi[17 + j], lo[17 + j], sum[3]);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                // the P buffer is free when the group's last product has read it
                if (at_c.c >= 2 && !(ok = warp_wait(&ms.pv_done[back.stage], back.full(), wait_limit))) break;
                tm_after();
                tm_st32(my_p, hi);
                tm_st32(my_p + 32, lo);
                tm_wait_st();
                tm_before();
                bar_arrive(&ms.p_ready[wg]);
                fresh = false;
                back = at_c;
                at_c.next();
                at_c.next();
            }
            parity ^= take & 1;
            // ---- the piece: both groups' outputs join out of tensor memory, half of the columns by each
            // (a group that gave up keeps the barriers)
            if (ok && !fresh) ok = warp_wait(&ms.pv_done[back.stage], back.full(), wait_limit);
            // what a group that gave up leaves is no number, in every row's output
            ms.stat[wg][lrow] = make_float2(m, ok ? l : __uint_as_float(0x7fffffffu));
            tm_before();
            asm volatile("bar.sync 2, %0;" ::"r"(64 * act) : "memory");
            tm_after();
            const float2 s0 = ms.stat[0][lrow], s1 = ms.stat[1][lrow];
            const float mm = fmaxf(s0.x, s1.x), mr = mm == -INFINITY ? 0.f : mm;
            const float f0 = ex2(s0.x - mr), f1 = ex2(s1.x - mr), ll = s0.y * f0 + s1.y * f1;  // (0 x NaN stays NaN)
            // a group without a tile (or without a finite score) has nothing in its output
            const bool has0 = s0.x != -INFINITY, has1 = s1.x != -INFINITY;
            const bool whole = take == w.n;
            float* slot = p.slots + (whole ? 2ll * gridDim.x + (p.wide ? (long long)w.b * items : 0) + w.item : 2ll * blockIdx.x + (u == first ? 0 : 1)) * p.slot_floats;
#pragma unroll 1
            for (int d = wg * (D / 2); d < (wg + 1) * (D / 2); d += 32) {
                uint32_t x[32], y[32];
                tm_ld32(x, my + S::T_O + d);
                tm_ld32(y, my + S::T_O + D + d);
                tm_wait_ld();
                if (real) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        float z[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            z[i] = (has0 ? __uint_as_float(x[e + i]) * f0 : 0.f) + (has1 ? __uint_as_float(y[e + i]) * f1 : 0.f);
                        *reinterpret_cast<float4*>(slot + (long long)lrow * D + d + e) = make_float4(z[0], z[1], z[2], z[3]);
                    }
                }
            }
            tm_before();
            if (real && wg == 0)
                *reinterpret_cast<float2*>(slot + (long long)p.slot_rows * D + 2 * lrow) =
                    live ? make_float2(mm, ll) : make_float2(-INFINITY, 0.f);
            asm volatile("bar.sync 2, %0;" ::"r"(64 * act) : "memory");  // the outputs have been read
            u += take;
            w.on(p, take);
        }
    } else if (!F8 && warp < MMA_WARP) {
        // ================ loads by tensor maps: one warp ================
        {
            // A tile is `parts` boxes of up to 64 rows of one page. The lanes hold the pages of the next 32 boxes,
            // and of the 32 after them.
            const int rows = min(TILE, 1 << p.ps_shift), parts = TILE / rows, mask = (1 << p.ps_shift) - 1;
            const int tiles = end - first, pshift = __ffs(parts) - 1;
            Walk ahead = w;
            int ahead_c = lane >> pshift;
            ahead.on(p, ahead_c);
            auto page_next = [&] {  // of this lane's box of the next 32; one that does not exist reads as zeros
                int page = p.n_pages;
                if (ahead_c < tiles) {
                    const int pos = ahead.at() + (lane & (parts - 1)) * rows;
                    if ((unsigned)pos < (unsigned)limit) {
                        page = p.table[ahead.b * p.table_s + (pos >> p.ps_shift)];
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
            int now = page_next(), next = page_next();
            int box = 0;
            Place<S::STAGES> pl;
            for (int c = 0; c < tiles; ++c, pl.next()) {
                const int stage = pl.stage, h = w.item / p.RB, j0 = w.at();
                w.on(p, 1);
                const uint32_t st = ring + stage * S::STAGE_B;
                if (c >= S::STAGES && !warp_wait(&ms.pv_done[stage], pl.free(), wait_limit)) break;
                if (lane == 0) bar_expect(&ms.kv_full[stage], S::STAGE_B);
                sent = c + 1;
                for (int i = 0; i < parts; ++i, ++box) {
                    const int page = __shfl_sync(0xffffffffu, now, box & 31);
                    if (lane == 0) {
                        const int row = (j0 + i * rows) & mask;
#pragma unroll
                        for (int x = 0; x < S::PANELS; ++x) {
                            const uint32_t to = st + x * TILE * 128 + i * rows * 128;
                            tma_rows(to, &maps.k, x * 64, row, h, page, &ms.kv_full[stage]);
                            tma_rows(to + S::KV_B, &maps.v, x * 64, row, h, page, &ms.kv_full[stage]);
                        }
                    }
                    if ((box & 31) == 31) {
                        now = next;
                        next = page_next();
                    }
                }
            }
        }
    } else if (F8 && warp < MMA_WARP) {
        // ================ loads of codes ================
        const int t = tid - 256;
        const int mask = (1 << p.ps_shift) - 1;
        constexpr int CH = D / 16;             // 16-byte pieces of a cached row
        constexpr int EACH = TILE * CH / 128;      // pieces of K (and of V) a thread copies
        const int cc = t % CH;
        const int tiles = end - first;
        const uint32_t raw0 = qs + S::RAW_OFF;
        // Row t of a tile: its page, looked up two tiles ahead of the copies, which are two ahead of their use. A
        // thread turns what it copied itself, so only the rows' places pass between threads.
        struct At {
            int page, r, h;  // of row t: its page (-1: none) and row there; the tile's kv head
        };
        auto look = [&](int c) {  // tiles in their order
            At x = {-1, 0, 0};
            if (c >= tiles) return x;
            const int pos = w.at() + t;
            x.r = pos & mask;
            x.h = w.item / p.RB;
            if (t < TILE && (unsigned)pos < (unsigned)limit) {
                x.page = p.table[w.b * p.table_s + (pos >> p.ps_shift)];
                if ((unsigned)x.page >= (unsigned)p.n_pages) {
                    x.page = -1;
                    if (p.status) *p.status = MK_ERR_INVALID_ARG;
                }
            }
            w.on(p, 1);
            return x;
        };
        auto note = [&](int c, const At& x) {
            if (t < TILE && c < tiles) ms.off[c & 1][t] = x.page < 0 ? -1 : x.page * p.page_b + x.r * p.row_b;
        };
        auto copy = [&](int c, const At& x) {
            if (c < tiles) {
                const int h = x.h;
                const uint8_t* const kh = p.k + h * p.head_b;
                const uint8_t* const vh = p.v + h * p.head_b;
                const uint32_t to = raw0 + c % S::RAWS * S::RAW_B;
#pragma unroll
                for (int i = 0; i < EACH; ++i) {
                    const int r = t / CH + i * (128 / CH);
                    const long long o = ms.off[c & 1][r];
                    const bool in = o >= 0;
                    const long long a = in ? o + cc * 16 : 0;
                    cp16(to + (i * 128 + t) * 16, kh + a, in);
                    cp16(to + TILE * D + (i * 128 + t) * 16, vh + a, in);
                }
                if (t < TILE) {
                    const long long o = x.page < 0 ? 0 : x.page * p.sc_page + h * p.sc_head + x.r;
                    cp4(to + 2 * TILE * D + t * 4, p.ks + o, x.page >= 0);
                    cp4(to + 2 * TILE * D + (TILE + t) * 4, p.vs + o, x.page >= 0);
                }
            }
            cp_commit();
        };
        auto here = [] { asm volatile("bar.sync 1, 128;" ::: "memory"); };
        const At at0 = look(0), at1 = look(1);
        At at2 = look(2);
        note(0, at0);
        note(1, at1);
        here();
        copy(0, at0);
        copy(1, at1);
        here();
        Place<S::STAGES> pl;
        bool ok = true;
        for (int c = 0; c < tiles; ++c, pl.next()) {
            const int stage = pl.stage;
            const uint32_t st = ring + stage * S::STAGE_B;
            const At at3 = look(c + 3);
            note(c + 2, at2);  // over the places of tile c, which were read two barriers ago
            here();
            copy(c + 2, at2);
            at2 = at3;
            // a thread that gave up keeps the loop's barriers
            if (ok && c >= S::STAGES) ok = bar_wait(&ms.pv_done[stage], pl.free(), wait_limit);
            cp_wait<2>();
            if (ok) {
                const uint8_t* const raw = smem + S::RAW_OFF + c % S::RAWS * S::RAW_B;
                auto put = [&](uint32_t base, int r, const uint4& w) {
                    uint4 a, b;
                    codes_bf16<FMT>(w.x, a.x, a.y);
                    codes_bf16<FMT>(w.y, a.z, a.w);
                    codes_bf16<FMT>(w.z, b.x, b.y);
                    codes_bf16<FMT>(w.w, b.z, b.w);
                    *reinterpret_cast<uint4*>(smem + (panel_at(base, TILE, r, 2 * cc) - qs)) = a;
                    *reinterpret_cast<uint4*>(smem + (panel_at(base, TILE, r, 2 * cc + 1) - qs)) = b;
                };
#pragma unroll
                for (int i = 0; i < EACH; ++i) {
                    const int r = t / CH + i * (128 / CH);
                    put(st, r, *reinterpret_cast<const uint4*>(raw + (i * 128 + t) * 16));
                    put(st + S::KV_B, r, *reinterpret_cast<const uint4*>(raw + TILE * D + (i * 128 + t) * 16));
                }
                if (t < TILE) {
                    const float* sc = reinterpret_cast<const float*>(raw + 2 * TILE * D);
                    scales[stage * 2 * TILE + t] = sc[t];
                    scales[stage * 2 * TILE + TILE + t] = sc[TILE + t];
                }
                // this thread's part of the tile lies in shared memory
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                bar_arrive(&ms.kv_full[stage]);
            }
        }
        cp_wait<0>();
    } else {
        // ================ products: two warps in step, one lane of each issues ================
        const uint32_t tmu = __shfl_sync(0xffffffffu, tm, 0);
        Place<S::STAGES> at_c;
        unsigned piece_no = 0;
        bool ok = true;
        if (warp == MMA_WARP) {
            constexpr uint32_t QK = mma_desc(ROWS, TILE, false);
            const uint64_t q = smem_desc(qs, 16, 1024), k0 = smem_desc(ring, 16, 1024);
            for (int u = first; u < end && ok; ++piece_no) {
                const int take = min(w.n - w.tile, end - u);
                u += take;
                w.on(p, take);
                ok = warp_wait(&ms.q_ready, piece_no & 1u, wait_limit);
                for (int i = 0; i < take && ok; ++i) {
                    // K is here; the softmax has read what the S buffer held two tiles ago
                    ok = warp_wait(&ms.kv_full[at_c.stage], at_c.full(), wait_limit) &&
                         (at_c.c < 2 || warp_wait(&ms.s_free[at_c.buf()], at_c.pair_free(), wait_limit));
                    if (!ok) break;
                    tm_after();
                    if (elect_one()) {
                        const uint64_t k = desc_on(k0, at_c.stage * S::STAGE_B);
                        const uint32_t d = tmu + S::T_S + at_c.buf() * TILE;
#pragma unroll
                        for (int part = 0; part < (SPLITQ ? 2 : 1); ++part)
#pragma unroll
                            for (int j = 0; j < D / 16; ++j)
                                mma_ss(d, desc_on(q, part * S::Q_PART + (j >> 2) * ROWS * 128 + (j & 3) * 32),
                                       desc_on(k, (j >> 2) * TILE * 128 + (j & 3) * 32), QK, part > 0 || j > 0);
                        mma_commit(&ms.s_full[at_c.buf()]);
                    }
                    __syncwarp();
                    at_c.next();
                }
            }
        } else {
            constexpr uint32_t PV = mma_desc(ROWS, D, true);
            const uint64_t v0 = smem_desc(ring + S::KV_B, TILE * 128, 1024);
            for (int u = first; u < end && ok;) {
                const int take = min(w.n - w.tile, end - u);
                u += take;
                w.on(p, take);
                for (int i = 0; i < take; ++i) {
                    // the probabilities are here, and so V (their scores came from the same stage)
                    if (!(ok = warp_wait(&ms.p_ready[at_c.buf()], at_c.pair(), wait_limit))) break;
                    tm_after();
                    if (elect_one()) {
                        const uint64_t v = desc_on(v0, at_c.stage * S::STAGE_B);
                        const uint32_t pa = tmu + S::T_P + at_c.buf() * TILE, d = tmu + S::T_O + at_c.buf() * D;
                        // the first tile of each group's piece overwrites
#pragma unroll
                        for (int part = 0; part < 2; ++part)
#pragma unroll
                            for (int j = 0; j < TILE / 16; ++j)
                                mma_ts(d, pa + part * 32 + j * 8, desc_on(v, j * 2048), PV, i > 1 || part > 0 || j > 0);
                        if (!p.skip_signal) mma_commit(&ms.pv_done[at_c.stage]);
                    }
                    __syncwarp();
                    at_c.next();
                }
            }
        }
        // the last products end before the tensor memory goes, also when a role gave up
        if (elect_one()) mma_commit(&ms.drained);
        const long long t0 = now_ns();
        while (!bar_try(&ms.drained, 0) && now_ns() - t0 < DRAIN_NS) {
        }
    }
    __syncwarp();
    tm_before();
    __syncthreads();
    tm_after();
    if (ms.abort) {
        // Whichever role gave up, copies by the tensor maps may still be on their way into this CTA's memory: at most
        // the ring's last tiles. (The loads of codes and the products have waited for theirs.)
        if (!F8 && warp == 8) {
            const long long t0 = now_ns();
            for (int c = max(0, sent - S::STAGES); c < sent; ++c)
                while (!bar_try(&ms.kv_full[c % S::STAGES], (unsigned)(c / S::STAGES) & 1u) && now_ns() - t0 < DRAIN_NS) {
                }
        }
        if (tid == 0 && p.status) *p.status = MK_ERR_TIMEOUT;
    }
    if (warp == MMA_WARP)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "n"(S::T_ALL) : "memory");
}

// ---- launches (p NULL: one-time attributes)

// K or V as a 4-D tensor; a box is up to 64 rows of a page by 64 values, in
// the 128-byte swizzled order the products read
inline int map_of(const AttendP& p, const void* base, int head_dim, CUtensorMap* out) {
    const EncodeFn encode = encode_fn();
    if (!encode) return fail(MK_ERR_CUDA, "attend: the driver has no cuTensorMapEncodeTiled");
    const cuuint32_t rows = 1u << p.ps_shift;
    const cuuint64_t dims[4] = {(cuuint64_t)head_dim, rows, (cuuint64_t)p.H, (cuuint64_t)p.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)p.row_b, (cuuint64_t)p.head_b, (cuuint64_t)p.page_b};
    const cuuint32_t box[4] = {64, rows < 64 ? rows : 64, 1, 1}, one[4] = {1, 1, 1, 1};
    const CUresult r = encode(out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, one,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(MK_ERR_CUDA, "attend: cuTensorMapEncodeTiled failed (%d)", (int)r);
    return MK_OK;
}

template <int D, int FMT, bool SPLITQ>
int prefix_go(const AttendP* p, int grid, cudaStream_t s) {
    using S = PrefixShape<D, FMT, SPLITQ>;
    auto kern = prefix_kernel<D, FMT, SPLITQ>;
    if (!p) return cuda_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM), "mk_pages_attend");
    PrefixMaps maps = {};
    if constexpr (FMT == MK_KV_BF16) {
        if (const int rc = map_of(*p, p->k, D, &maps.k)) return rc;
        if (const int rc = map_of(*p, p->v, D, &maps.v)) return rc;
    }
    kern<<<grid, S::NT, S::SMEM, s>>>(*p, maps);
    return cuda_status(cudaGetLastError(), "mk_pages_attend");
}
template <int D, bool SPLITQ>
int prefix_pick(int format, const AttendP* p, int grid, cudaStream_t s) {
    if (format == MK_KV_E4M3) return prefix_go<D, MK_KV_E4M3, SPLITQ>(p, grid, s);
    if (format == MK_KV_INT8) return prefix_go<D, MK_KV_INT8, SPLITQ>(p, grid, s);
    return prefix_go<D, MK_KV_BF16, SPLITQ>(p, grid, s);
}

}  // namespace mkop
