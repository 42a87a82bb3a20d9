// mk_prompt.cu -- causal attention of prompts over expanded keys and values
// (mk_prompt_attend).
//
// For one query row (a token and a head) and the keys j it sees,
//   x_j = scale (q . k_j + q_rope . r_j),  m = max x_j,
//   out = sum_j e^(x_j - m) v_j / sum_j e^(x_j - m),
// in one pass over tiles of 128 keys on the fifth-generation tensor cores. A CTA
// takes 256 queries of a sequence and head as two blocks of 128 rows against the
// same tiles:
//   S = Q K^T   128 x 128 over 192 values, both operands in shared memory by
//               tensor maps, S in tensor memory;
//   P = 2^(x - m), a row a thread, over the columns that S took, rounded to the
//               values' type (what a weight loses, half a step, is of the
//               output's own rounding; fp16 has no steps of its own for small
//               weights, which are taken 2^7 larger: half a step is at least
//               2^-32 of the row's largest);
//   O += P V    P as the tensor-memory operand, V from shared memory as it lies
//               there (its rows are the product's K), O in tensor memory.
// While the tensor cores work for one block, the other's four softmax warps
// turn its scores into probabilities. Each block has a warp that issues its
// products, in their order: O of a tile (either half as soon as its P is there),
// then the next S, which overwrites the P that the O before it has read. O is
// rescaled only when a row's maximum has risen by more than 2^8 since its
// reference.
//
// Shared memory is full: queries 96 KB, a ring of five 16 KB panels of keys (64
// values of 128 keys), one of three 16 KB halves of values (64 keys).
//
// At the end of what is seen scores are masked, and since 0 x NaN is NaN, a
// warp cleans the tiles there: values that no row of the CTA sees become zeros;
// so do values that are not finite and that only some rows see, and rows that
// do see them get NaN.
//
// A few blocks with long contexts share each block's tiles out to a cluster of 2 to
// 8 CTAs, whose outputs, maxima and sums meet through distributed shared memory.
//
// Longest CTAs first: blocks of a sequence in falling order, all heads of one
// after another, so that short ones fill the end. All waits have a limit.
//
// Measured, 16 heads, bf16: 8192 tokens 251 us (1.37 PFLOP/s of what is seen, 71 %
// of a large product's rate), 4 x 4096 283, 8 x 2048 183, 1 x 1024 23. A tile of
// both blocks takes 3500 cycles, 2590 of them products; the rest is the turns'
// hand-over and waits (a wait that is already over costs some 100). A CTA has all
// of an SM's memory and nothing runs beside its 8 us before the first scores and
// after the last ones: these bound short prompts, and are some 50 of the 183 us of
// 8 x 2048 (6.7 CTAs an SM).
#include <climits>
#include <type_traits>

#include "mk_tensor.cuh"

namespace {

using namespace mkop;

constexpr int NOPE = 128, ROPE = 64, VD = 128;
constexpr int ROWS = 128, TILE = 128, PAIR = 2 * ROWS;
constexpr int PANELS = (NOPE + ROPE) / 64;      // 64 values wide
constexpr int PANEL_B = TILE * 128;             // of keys, and of queries
constexpr int Q_B = PANELS * PANEL_B;           // a block's queries
constexpr int KS = 5, VS = 3;                   // ring slots: panels of keys, halves of values
constexpr int VHALF_B = 64 * VD * 2;
constexpr int K_OFF = 2 * Q_B, V_OFF = K_OFF + KS * PANEL_B, MISC_OFF = V_OFF + VS * VHALF_B;
constexpr int NT = 384;                         // warps: softmax 2 x 4, copies, products 2, cleaning
// registers of a softmax thread's row and of the others: of the launch's 384 x 168
constexpr int REGS_SOFTMAX = 208, REGS_REST = 80;
static_assert(256 * REGS_SOFTMAX + 128 * REGS_REST <= NT * 168, "");
constexpr int T_S = 0, T_O = 2 * TILE, T_ALL = 512;  // tensor memory: S (and P) of both blocks, O of both
static_assert(T_O + 2 * VD <= T_ALL && PANEL_B == VHALF_B, "");

struct PromptMisc {
    unsigned long long q_full[2], k_full[2], k_free[KS], v_full[VS], v_ok[VS], v_free[VS], s_full[2], p_ready[2][2], o_done[2],
        turn[2], drained;
    unsigned tmem, abort;
    int scan[NT / 32], seq, pair, bad;
};
constexpr int MISC_B = 1024, SMEM = 1024 + MISC_OFF + MISC_B;
// A row among the CTAs of a block: its output, maximum and sum, floats.
constexpr int OUT_ROW = VD + 4;
static_assert(PAIR * OUT_ROW * 4 <= MISC_OFF && sizeof(PromptMisc) <= MISC_B && SMEM <= 227 * 1024, "");

struct PromptP {
    const int *q_starts, *k_starts;
    uint8_t* out;
    float* lse;
    int* status;
    long long ot, oh;           // elements
    int B, n_q, n_k, H;
    int q_heads, k_heads, v_heads;  // 0: all heads are one (a stride of 0)
    float scale;
    int split;                  // CTAs of a block, a cluster: each takes a part of its tiles
    unsigned wait_ns;
    unsigned signals;           // for tests: the tiles of a CTA after which a role's signals are left out
};
struct PromptMaps {
    CUtensorMap q, k, r, v;
};

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, unsigned long long* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(sm32(bar))
        : "memory");
}
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    return F16 ? pack_f16(lo, hi) : pack_bf16(lo, hi);
}
// all CTAs of the cluster, their shared memory with them
__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// a ring slot and its turn
template <int N>
struct Slot {
    int i = 0;
    unsigned turn = 0;
    __device__ __forceinline__ void next() {
        if (++i == N) i = 0, ++turn;
    }
};

// blocks of 256 queries of a sequence; 0 where its bounds are none
__device__ __forceinline__ int pairs_of(const PromptP& p, int b) {
    const int q0 = p.q_starts[b], q1 = p.q_starts[b + 1], k0 = p.k_starts[b], k1 = p.k_starts[b + 1];
    if (q0 < 0 || q1 < q0 || q1 > p.n_q || k0 < 0 || k1 < k0 || k1 > p.n_k) return -1;
    return (q1 - q0 + PAIR - 1) / PAIR;
}

template <bool F16>
__global__ void __launch_bounds__(NT, 1)
    prompt_kernel(const __grid_constant__ PromptP p, const __grid_constant__ PromptMaps maps) {
    extern __shared__ uint8_t raw_smem[];
    uint8_t* const smem = raw_smem + ((1024u - (sm32(raw_smem) & 1023u)) & 1023u);
    const uint32_t qs = sm32(smem);
    PromptMisc& ms = *reinterpret_cast<PromptMisc*>(smem + MISC_OFF);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Limit limit = {&ms.abort, p.wait_ns};

    // the CTA's block: each thread counts a stretch of sequences; sums before it by shuffles
    const int block = blockIdx.x / p.split, part = blockIdx.x - block * p.split;
    const int h = block % p.H, u = block / p.H;
    const int each = (p.B + NT - 1) / NT, b0 = min(p.B, tid * each), b1 = min(p.B, b0 + each);
    int mine = 0;
    for (int b = b0; b < b1; ++b) {
        const int n = pairs_of(p, b);
        mine += max(n, 0);
        if (n < 0 && blockIdx.x == 0 && p.status) *p.status = MK_ERR_INVALID_ARG;
    }
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += a;
    }
    if (lane == 31) ms.scan[warp] = inc;
    if (tid == 0) ms.seq = -1;
    __syncthreads();
    int before = inc - mine;
    for (int w = 0; w < warp; ++w) before += ms.scan[w];
    if (u >= before && u < before + mine) {
        for (int b = b0, at = before; b < b1; ++b) {
            const int n = max(pairs_of(p, b), 0);
            if (u < at + n) {
                ms.seq = b;
                ms.pair = n - 1 - (u - at);  // the longest first
                break;
            }
            at += n;
        }
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            bar_init(&ms.q_full[i], 1);
            bar_init(&ms.k_full[i], 1);
            bar_init(&ms.s_full[i], 1);
            bar_init(&ms.turn[i], 1);
            bar_init(&ms.p_ready[i][0], 128);
            bar_init(&ms.p_ready[i][1], 128);
            bar_init(&ms.o_done[i], 1);
        }
        for (int i = 0; i < KS; ++i) bar_init(&ms.k_free[i], 2);
        for (int i = 0; i < VS; ++i) bar_init(&ms.v_full[i], 1), bar_init(&ms.v_ok[i], 1), bar_init(&ms.v_free[i], 2);
        bar_init(&ms.drained, 2);
        ms.abort = 0;
        ms.bad = INT_MAX;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    if (ms.seq < 0) return;  // (the grid has room for a block more a sequence than there may be)
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sm32(&ms.tmem)), "n"(T_ALL)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tm_before();
    __syncthreads();
    tm_after();
    const uint32_t tm = ms.tmem;
    const int b = ms.seq, q0 = p.q_starts[b], n = p.q_starts[b + 1] - q0, k0 = p.k_starts[b], m = p.k_starts[b + 1] - k0;
    const int i0 = ms.pair * PAIR, behind = m - n;  // query i sees keys 0 .. behind + i
    // tiles that block g's rows see
    auto tiles_of = [&](int g) {
        const int first = i0 + g * ROWS, last = min(first + ROWS, n) - 1;
        return first < n && behind + last >= 0 ? (behind + last) / TILE + 1 : 0;
    };
    // of them this CTA's: from tile `from` on, counted from there
    const int all0 = tiles_of(0), all1 = tiles_of(1), most = max(all0, all1);
    const int from = (int)((long long)most * part / p.split), to_tile = (int)((long long)most * (part + 1) / p.split);
    const int nt0 = max(0, min(all0, to_tile) - from), nt1 = max(0, min(all1, to_tile) - from), nt = max(nt0, nt1);
    float row_m = -INFINITY, row_l = 0.f;  // of a softmax thread's row
    int sent_k = 0, sent_v = 0;  // panels and halves that the copying warp has asked for

    if (warp < 8) {
        // ================ softmax, a row a thread ================
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
        const int g = warp >> 2, row = i0 + g * ROWS + (tid & 127), mine_nt = g ? nt1 : nt0;
        const uint32_t my = tm + ((uint32_t)((warp & 3) * 32) << 16), my_s = my + T_S + g * TILE, my_o = my + T_O + g * VD;
        const int last = behind + row, least = behind + i0 + g * ROWS;  // the row's last key, and the block's first row's
        const bool neg = p.scale < 0.f;  // (then the smallest product counts: signs turned)
        const float scale2 = fabsf(p.scale) * LOG2E;
        // the row's reference: UP below a maximum (weights in fp16 are up to 2^15, of 65504)
        constexpr float UP = F16 ? 7.f : 0.f, RISE = 8.f;
        float mx = -INFINITY, l = 0.f;
        bool ok = true, large = false;  // large: some row's reference in the warp is, so that its own rounding counts
        auto is_large = [&] { return __any_sync(0xffffffffu, mx != -INFINITY && fabsf(mx) >= 0x1p20f); };
        // a reference moves: the output so far shrinks
        auto raise = [&](bool rise, float to, int j) {
            const float mn = rise ? to : mx, f = mx == -INFINITY ? 1.f : ex2(mx - mn);
            mx = mn;
            l *= f;
            if (j == 0) return true;
            // the last product is in the output
            if (!warp_wait(&ms.o_done[g], (j - 1) & 1, limit)) return false;
            tm_after();
#pragma unroll 1
            for (int d = 0; d < VD; d += 16) {
                uint32_t o[16];
                tm_ld16(o, my_o + d);
                tm_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tm_st16(my_o + d, o);
            }
            tm_wait_st();
            return true;
        };
        // A tile where references are large: products are rounded as those were before they are taken off (a fused step would
        // leave their rounding, which at 2^31 is past any exponent). Rare, so in small parts out of the tensor memory,
        // where a part's weights only replace scores that have been read. (Its being here costs prompts without any up to 1 %.)
        auto large_tile = [&](int j) {
            const int j0 = (from + j) * TILE;
            auto part = [&](int c, float (&x)[16]) {
                uint32_t y[16];
                tm_ld16(y, my_s + c);
                tm_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    x[e] = j0 + c + e > last ? -INFINITY : __fmul_rn(__uint_as_float(neg ? y[e] ^ 0x80000000u : y[e]), scale2);
            };
            float x[16], tile_m = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < TILE; c += 16) {
                part(c, x);
#pragma unroll
                for (int e = 0; e < 16; ++e) tile_m = fmaxf(tile_m, x[e]);
            }
            const bool rise = tile_m - mx > UP + RISE;
            if (__any_sync(0xffffffffu, rise)) {
                if (!(ok = raise(rise, tile_m - UP, j))) return;
            }
            large = is_large();
            const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll 1
            for (int c = 0; c < TILE; c += 16) {
                part(c, x);
                uint32_t y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float a = ex2(x[2 * e] - ref), d = ex2(x[2 * e + 1] - ref);
                    l += a + d;
                    y[e] = pack16<F16>(a, d);
                }
                tm_st8(my_s + (c >> 1), y);
                if ((c & 48) == 48) {
                    tm_wait_st();
                    tm_before();
                    bar_arrive(&ms.p_ready[g][c >> 6]);
                }
            }
        };
        // one tile; EDGE: some row of the block does not see all of it. A reference that turns out large leaves the tile to
        // large_tile (which finds nothing risen any more).
        auto tile = [&](auto EDGE, int j) {
            constexpr bool edge = decltype(EDGE)::value;
            const int j0 = (from + j) * TILE;
            uint32_t s[TILE];
#pragma unroll
            for (int c = 0; c < TILE; c += 32) tm_ld32(*reinterpret_cast<uint32_t(*)[32]>(s + c), my_s + c);
            tm_wait_ld();
            if (neg) {
#pragma unroll
                for (int e = 0; e < TILE; ++e) s[e] ^= 0x80000000u;
            }
            if constexpr (edge) {
#pragma unroll
                for (int e = 0; e < TILE; ++e)
                    if (j0 + e > last) s[e] = 0xff800000u;
            }
            float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < TILE; e += 8)
#pragma unroll
                for (int i = 0; i < 4; ++i) t[i] = fmaxf(t[i], fmaxf(__uint_as_float(s[e + 2 * i]), __uint_as_float(s[e + 2 * i + 1])));
            // (a scale of 0 times a masked -infinity is no number)
            const float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])), tile_m = top == -INFINITY ? top : __fmul_rn(top, scale2);
            const bool rise = tile_m - mx > UP + RISE;
            if (__any_sync(0xffffffffu, rise)) {
                if (!(ok = raise(rise, tile_m - UP, j))) return;
                if ((large = is_large())) return;
            }
            const float ref = mx == -INFINITY ? 0.f : mx;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < TILE; c += 32) {
                uint32_t x[16];
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    float a, d;
                    fma2(a, d, __uint_as_float(s[c + e]), __uint_as_float(s[c + e + 1]), scale2, scale2, -ref, -ref);
                    a = ex2(a), d = ex2(d);
                    if constexpr (edge) {  // (a scale of 0 again)
                        if (j0 + c + e > last) a = 0.f;
                        if (j0 + c + e + 1 > last) d = 0.f;
                    }
                    add2(sum[e & 2], sum[(e & 2) + 1], a, d);
                    x[e >> 1] = pack16<F16>(a, d);
                }
                tm_st16(my_s + (c >> 1), x);
                if (c & 32) {  // half of the keys: its product need not wait for the other half
                    tm_wait_st();
                    tm_before();
                    bar_arrive(&ms.p_ready[g][c >> 6]);
                }
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        };
        for (int j = 0; j < mine_nt; ++j) {
            if (!(ok = warp_wait(&ms.s_full[g], j & 1, limit))) break;
            tm_after();
            if (!large) {
                if ((from + j) * TILE + TILE - 1 > least) tile(std::true_type(), j);
                else tile(std::false_type(), j);
            }
            if (ok && large) large_tile(j);
            if (!ok) break;
        }
        // ---- the block's end
        if (ok && mine_nt) ok = warp_wait(&ms.o_done[g], (mine_nt - 1) & 1, limit);
        tm_after();
        // what a CTA that gave up leaves is no number, nor what sees a value that is none
        if (!ok || last >= ms.bad) l = __uint_as_float(0x7fffffffu);
        row_m = mx, row_l = l;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const bool real = row < n;
        uint4* const to = reinterpret_cast<uint4*>(p.out + 2 * ((long long)(q0 + row) * p.ot + (long long)h * p.oh));
#pragma unroll 1
        for (int d = 0; d < VD && p.split == 1; d += 32) {
            uint32_t o[32];
            tm_ld32(o, my_o + d);
            tm_wait_ld();
            if (real) {
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    uint32_t y[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        y[i] = l == 0.f ? 0u  // (nothing seen: what lies in the tensor memory may be anything)
                                        : pack16<F16>(__uint_as_float(o[e + 2 * i]) * inv, __uint_as_float(o[e + 2 * i + 1]) * inv);
                    to[(d + e) / 8] = make_uint4(y[0], y[1], y[2], y[3]);
                }
            }
        }
        if (real && p.lse && p.split == 1) p.lse[(long long)(q0 + row) * p.H + h] = l == 0.f ? -INFINITY : (mx + log2f(l)) * LN2;
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_REST));
    }
    if (warp < 8) {
    } else if (warp == 8) {
        // ================ copies ================
        Slot<KS> ks;
        Slot<VS> vs;
        bool ok = true;
        for (int j = 0; j < nt && ok; ++j) {
            const int key = k0 + (from + j) * TILE;
            for (int c = 0; c < PANELS; ++c, ks.next()) {
                ok = ok && (!ks.turn || warp_wait(&ms.k_free[ks.i], (ks.turn - 1) & 1, limit));
                if (!ok && c == 0) break;  // (a tile that has begun is finished all the same: its barrier counts all of it)
                ++sent_k;
                if (lane == 0) {
                    unsigned long long* const bar = &ms.k_full[j & 1];  // a tile's panels meet there
                    if (c == 0) bar_expect(bar, Q_B);
                    const uint32_t to = qs + K_OFF + ks.i * PANEL_B;
                    if (c < NOPE / 64) tma_3d(to, &maps.k, 64 * c, p.k_heads ? h : 0, key, bar);
                    else tma_2d(to, &maps.r, 0, key, bar);
                }
                if (j == 0 && c == 0) {  // queries: with the first keys
                    for (int g = 0; g < 2; ++g) {
                        if (lane || !(g ? nt1 : nt0)) continue;
                        bar_expect(&ms.q_full[g], Q_B);
                        for (int x = 0; x < PANELS; ++x)
                            tma_3d(qs + g * Q_B + x * PANEL_B, &maps.q, 64 * x, p.q_heads ? h : 0, q0 + i0 + g * ROWS, &ms.q_full[g]);
                    }
                }
            }
            for (int c = 0; c < 2 && ok; ++c, vs.next()) {
                if (!(ok = !vs.turn || warp_wait(&ms.v_free[vs.i], (vs.turn - 1) & 1, limit))) break;
                ++sent_v;
                if (lane == 0) {
                    unsigned long long* const bar = &ms.v_full[vs.i];
                    bar_expect(bar, VHALF_B);
                    for (int x = 0; x < 2; ++x)
                        tma_3d(qs + V_OFF + vs.i * VHALF_B + x * 8192, &maps.v, 64 * x, p.v_heads ? h : 0, key + 64 * c, bar);
                }
            }
        }
    } else if (warp == 11) {
        // ================ values that must not reach the output ================
        Slot<VS> vs;
        bool ok = true;
        const int all = behind + i0, some = behind + min(i0 + PAIR, n) - 1;  // keys up to which all rows, and any row, see
        for (int j = 0; j < 2 * nt && ok; ++j, vs.next()) {
            if (!(ok = warp_wait(&ms.v_full[vs.i], vs.turn & 1, limit))) break;
            const int j0 = from * TILE + 64 * j;
            if (j0 + 63 > all) {
                // 16-byte piece c: value panel c / 512, key c / 8 % 64 of the half
                uint4* const at = reinterpret_cast<uint4*>(smem + V_OFF + vs.i * VHALF_B) + lane;
                int bad = INT_MAX;
                // keys that some rows see, eight pieces a thread at a time: an exponent of ones carries into the sign
                constexpr uint32_t E = F16 ? 0x7c007c00u : 0x7f807f80u, ONE = F16 ? 0x04000400u : 0x00800080u;
                if (j0 <= some) {
#pragma unroll 1
                    for (int i = 0; i < VHALF_B / 512; i += 8) {
                        uint4 v[8];
                        uint32_t ones = 0;
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = at[(i + e) * 32];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            ones |= ((v[e].x & E) + ONE) | ((v[e].y & E) + ONE) | ((v[e].z & E) + ONE) | ((v[e].w & E) + ONE);
                        if (!(ones & 0x80008000u)) continue;
                        for (int e = 0; e < 8; ++e) {
                            const int key = j0 + (((i + e) * 32 + lane) >> 3 & 63);
                            const uint4 x = at[(i + e) * 32];
                            if (key <= all || key > some ||
                                !((((x.x & E) + ONE) | ((x.y & E) + ONE) | ((x.z & E) + ONE) | ((x.w & E) + ONE)) & 0x80008000u))
                                continue;
                            at[(i + e) * 32] = make_uint4(0, 0, 0, 0);
                            bad = min(bad, key);
                        }
                    }
                }
                if (j0 + 63 > some) {
                    for (int i = 0; i < VHALF_B / 512; ++i)
                        if (j0 + ((i * 32 + lane) >> 3 & 63) > some) at[i * 32] = make_uint4(0, 0, 0, 0);
                }
                if (bad != INT_MAX) atomicMin(&ms.bad, bad);
                fence_async();
            }
            __syncwarp();
            if (lane == 0) bar_arrive(&ms.v_ok[vs.i]);
        }
    } else {
        // ================ products: a warp for each block, an elected lane issues ================
        // (a constant block: operands then stay in uniform registers)
        auto products = [&](auto G) {
        constexpr int g = decltype(G)::value;
        const int mine_nt = g ? nt1 : nt0;
        const uint32_t tmu = __shfl_sync(0xffffffffu, tm, 0);
        constexpr uint32_t QK = mma_desc(ROWS, TILE, false, false, F16), PV = mma_desc(ROWS, VD, true, false, F16);
        const uint64_t qd = smem_desc(qs + g * Q_B, 16, 1024), kd = smem_desc(qs + K_OFF, 16, 1024), vd = smem_desc(qs + V_OFF, 8192, 1024);
        const uint32_t ts = tmu + T_S + g * TILE, to = tmu + T_O + g * VD;
        bool ok = true;
        Slot<KS> ks;
        Slot<VS> vs;
        // (the whole warp runs this and one lane issues: the shuffle above and the votes of a wait need all 32)
        auto here = [&](unsigned long long* bar, unsigned parity) { return bar_wait(bar, parity & 1u, limit); };
        // S of a tile; one that the block does not see is let go as it comes
        auto scores = [&](int j) {
            if (j == 0 && mine_nt) ok = ok && warp_wait(&ms.q_full[g], 0, limit);
            if (j == 0 && g) ok = ok && warp_wait(&ms.turn[1], 0, limit);
            if (!(ok = ok && warp_wait(&ms.k_full[j & 1], (unsigned)j >> 1 & 1u, limit))) return;
            tm_after();
            if (elect_one()) {
                Slot<KS> at = ks;
                if (j < mine_nt) {
#pragma unroll
                    for (int c = 0; c < PANELS; ++c, at.next()) {
                        if (c == PANELS - 1) bar_arrive(&ms.turn[g ^ 1]);  // (the other's next products follow these)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_ss(ts, desc_on(qd, c * PANEL_B + k * 32), desc_on(kd, at.i * PANEL_B + k * 32), QK, c > 0 || k > 0);
                        mma_commit(&ms.k_free[at.i]);
                    }
                    if ((unsigned)j < p.signals) mma_commit(&ms.s_full[g]);
                } else {
                    bar_arrive(&ms.turn[g ^ 1]);
                    for (int c = 0; c < PANELS; ++c, at.next()) bar_arrive(&ms.k_free[at.i]);
                }
            }
            __syncwarp();
            for (int c = 0; c < PANELS; ++c) ks.next();
        };
        // O of half a tile
        auto half = [&](int j, int c) {
            tm_after();
            if (elect_one()) {
                if (j < mine_nt) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_ts(to, ts + (4 * c + k) * 8, desc_on(vd, vs.i * VHALF_B + k * 2048), PV, j > 0 || c > 0 || k > 0);
                    mma_commit(&ms.v_free[vs.i]);
                    if (c == 1) mma_commit(&ms.o_done[g]);
                } else {
                    bar_arrive(&ms.v_free[vs.i]);
                }
            }
            __syncwarp();
            vs.next();
        };
        if (nt) scores(0);
        for (int j = 0; j < nt && ok; ++j) {
            // V and the first half's weights are here; block 0's turn is after block 1's S of this tile, block 1's after
            // block 0's S of the next one
            const unsigned turn1 = vs.i == VS - 1 ? vs.turn + 1 : vs.turn;
            const int i1 = vs.i == VS - 1 ? 0 : vs.i + 1;
            ok = __all_sync(0xffffffffu, here(&ms.v_ok[vs.i], vs.turn) && here(&ms.v_ok[i1], turn1) && (j >= mine_nt || here(&ms.p_ready[g][0], j)) &&
                                             (j + g >= nt || here(&ms.turn[g], j + g)));
            if (!ok) break;
            half(j, 0);
            if (j < mine_nt) ok = __all_sync(0xffffffffu, here(&ms.p_ready[g][1], j));
            if (!ok) break;
            half(j, 1);
            if (j + 1 < nt) scores(j + 1);
        }
        };
        if (warp == 9) products(std::integral_constant<int, 0>());
        else products(std::integral_constant<int, 1>());
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
        // copies may still be on their way into this CTA's memory (the queries, at most the rings' last ones): they land before
        // anything else is written there, the marks of rows without a number among it
        if (warp == 8 && sent_k) {
            const long long t0 = now_ns();
            auto gone = [&](unsigned long long* bar, unsigned parity) {
                while (!bar_try(bar, parity) && now_ns() - t0 < DRAIN_NS) {
                }
            };
            if (nt0) gone(&ms.q_full[0], 0);
            if (nt1) gone(&ms.q_full[1], 0);
            for (int c = max(0, sent_k / PANELS - 2); c < sent_k / PANELS; ++c) gone(&ms.k_full[c & 1], (unsigned)c >> 1 & 1u);
            for (int c = max(0, sent_v - VS); c < sent_v; ++c) gone(&ms.v_full[c % VS], (unsigned)(c / VS) & 1u);
        }
        if (tid == 0 && p.status) *p.status = MK_ERR_TIMEOUT;
        __syncthreads();
    }
    if (p.split > 1) {
        // ================ the block's parts meet: outputs over the queries and rings, which nothing uses any more ================
        float* const outs = reinterpret_cast<float*>(smem);
        if (warp < 8) {
            const uint32_t my_o = tm + ((uint32_t)((warp & 3) * 32) << 16) + T_O + (warp >> 2) * VD;
            const bool some = (warp >> 2) ? nt1 : nt0;
            float* const row = outs + tid * OUT_ROW;
#pragma unroll 1
            for (int d = 0; d < VD; d += 16) {
                uint32_t o[16];
                tm_ld16(o, my_o + d);
                tm_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; e += 4)  // (without a tile: what lies in the tensor memory may be anything)
                    *reinterpret_cast<float4*>(row + d + e) =
                        some ? make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]), __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]))
                             : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            *reinterpret_cast<float2*>(row + VD) = make_float2(row_m, ms.abort ? __uint_as_float(0x7fffffffu) : row_l);
        }
        cluster_meet();
        // a warp a row, four values a lane
        const int r1 = PAIR * (part + 1) / p.split;
        for (int r = PAIR * part / p.split + warp; r < r1; r += NT / 32) {
            const int row = i0 + r;
            if (row >= n) break;
            float mx = -INFINITY, l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int c = 0; c < p.split; ++c) {
                float2 st;
                float4 y;
                uint32_t a;
                asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(sm32(outs + r * OUT_ROW)), "r"(c));
                asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(st.x), "=f"(st.y) : "r"(a + VD * 4) : "memory");
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(y.x), "=f"(y.y), "=f"(y.z), "=f"(y.w) : "r"(a + 16 * lane) : "memory");
                const float mn = fmaxf(mx, st.x), ref = mn == -INFINITY ? 0.f : mn, f = ex2(mx - ref), w = ex2(st.x - ref);
                mx = mn;
                l = l * f + st.y * w;
                o.x = o.x * f + y.x * w, o.y = o.y * f + y.y * w, o.z = o.z * f + y.z * w, o.w = o.w * f + y.w * w;
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;
            *reinterpret_cast<uint2*>(p.out + 2 * ((long long)(q0 + row) * p.ot + (long long)h * p.oh + 4 * lane)) =
                make_uint2(pack16<F16>(o.x * inv, o.y * inv), pack16<F16>(o.z * inv, o.w * inv));
            if (lane == 0 && p.lse) p.lse[(long long)(q0 + row) * p.H + h] = l == 0.f ? -INFINITY : (mx + log2f(l)) * LN2;
        }
        cluster_meet();  // the others have read what lies here
    }
    if (warp == 9)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "n"(T_ALL) : "memory");
}

// [rows][heads][width] as a tensor, boxes of `box` rows by 64 values of one head (heads 0: one for all, a stride of 0)
int map_of(const void* base, int dtype, int width, int heads, int rows, int64_t head_s, int64_t row_s, int box, CUtensorMap* out) {
    const EncodeFn encode = encode_fn();
    if (!encode) return fail(MK_ERR_CUDA, "prompt: the driver has no cuTensorMapEncodeTiled");
    // one row or head: its stride is never used, but has to be one
    const cuuint64_t rs = rows > 1 ? (cuuint64_t)row_s * 2 : 16, hs = heads > 1 ? (cuuint64_t)head_s * 2 : 16;
    const bool flat = heads < 0;
    const cuuint64_t dims[3] = {(cuuint64_t)width, flat ? (cuuint64_t)rows : (cuuint64_t)(heads ? heads : 1), (cuuint64_t)rows};
    const cuuint64_t strides[2] = {flat ? rs : hs, rs};
    const cuuint32_t boxes[3] = {64, flat ? (cuuint32_t)box : 1, (cuuint32_t)box}, one[3] = {1, 1, 1};
    const CUresult r = encode(out, dtype == MK_DT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                              flat ? 2 : 3, const_cast<void*>(base), dims, strides, boxes, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(MK_ERR_CUDA, "prompt: cuTensorMapEncodeTiled failed (%d)", (int)r);
    return MK_OK;
}

template <bool F16>
int run(PromptP& p, const PromptMaps& maps, int some, int64_t blocks, cudaStream_t s) {
    auto kern = prompt_kernel<F16>;
    static std::atomic<uint64_t> done;
    int dev, sms;
    if (const int rc = device_sms(dev, sms, "mk_prompt_attend")) return rc;
    if (const int rc = allow_smem(kern, SMEM, dev, done, "mk_prompt_attend")) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    // how many clusters of 2, 4, 8 CTAs the device holds at once, asked for once
    static std::atomic<int> room[64][3];
    auto fits = [&](int i) {
        int n = dev < 64 ? room[dev][i].load(std::memory_order_relaxed) : 0;
        if (!n) {
            at[0].val.clusterDim.x = 2 << i;
            cfg.gridDim = dim3((unsigned)(2 << i));
            if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) n = 1, cudaGetLastError();
            if (dev < 64) room[dev][i].store(n, std::memory_order_relaxed);
        }
        return n;
    };
    // Few blocks share their tiles out to clusters, as long as these run all at once and a CTA has four tiles or more (of an
    // average over the sequences that may have queries: the lengths are on the device, so one long context among many short
    // ones is not shared, nor where a ragged batch's bound on blocks is past the room). 16 heads, 256 tokens at 8192
    // positions: 136 us by one CTA a block, 48 by four; by eight, which do not all find room at once, 63. One token behind
    // 16000 keys beside 15 sequences without any: 204 us by one, 59 by eight.
    p.split = 1;
    for (int i = 0; i < 3 && p.n_k / some >= (4 * TILE << (i + 1)) && blocks <= fits(i); ++i) p.split = 2 << i;
    cfg.gridDim = dim3((unsigned)(blocks * p.split));
    at[0].val.clusterDim.x = p.split;
    cfg.numAttrs = p.split > 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, kern, p, maps), "mk_prompt_attend");
}

}  // namespace

extern "C" int mk_prompt_attend(const mk_prompt_attention* a, void* stream) {
    if (!a) return fail(MK_ERR_INVALID_ARG, "prompt: NULL arguments");
    if (!a->q_starts || !a->k_starts || off_by4(a->q_starts, a->k_starts, a->lse, a->status))
        return fail(MK_ERR_INVALID_ARG, "prompt: q_starts or k_starts is NULL, or they, lse or status not aligned to 4 bytes");
    if (a->dtype != MK_DT_BF16 && a->dtype != MK_DT_F16) return fail(MK_ERR_INVALID_ARG, "prompt: q, k and v must be bf16 or fp16");
    if (a->batch < 1 || a->n_tokens < 0 || a->n_keys < 0 || a->n_heads < 1) return fail(MK_ERR_INVALID_ARG, "prompt: non-positive dimension");
    if (!(a->scale >= -1e30f && a->scale <= 1e30f)) return fail(MK_ERR_INVALID_ARG, "prompt: scale is not a number in range");
    if (a->nope_dim != NOPE || a->rope_dim != ROPE || a->v_dim != VD)
        return fail(MK_ERR_UNSUPPORTED, "prompt: heads must have nope_dim 128, rope_dim 64, v_dim 128");
    if (a->n_tokens == 0) return MK_OK;
    if (!a->q || !a->out || (a->n_keys && (!a->k || !a->k_rope || !a->v))) return fail(MK_ERR_INVALID_ARG, "prompt: q, k, k_rope, v or out is NULL");
    if (((uintptr_t)a->q | (uintptr_t)a->k | (uintptr_t)a->k_rope | (uintptr_t)a->v | (uintptr_t)a->out) % 16 ||
        (a->q_token | a->q_head | a->k_token | a->k_head | a->rope_token | a->v_token | a->v_head | a->out_token | a->out_head) % 8)
        return fail(MK_ERR_INVALID_ARG, "prompt: q, k, k_rope, v, out and their strides must be multiples of 16 bytes");
    if (a->q_token < 0 || a->q_head < 0 || a->k_token < 0 || a->k_head < 0 || a->rope_token < 0 || a->v_token < 0 ||
        a->v_head < 0 || a->out_token < 0 || a->out_head < 0)
        return fail(MK_ERR_INVALID_ARG, "prompt: negative stride");
    if (a->n_keys > 1 << 30) return fail(MK_ERR_UNSUPPORTED, "prompt: more than 2^30 keys in one call");
    if (a->batch > (1 << 20) || (int64_t)a->n_tokens * a->n_heads > INT32_MAX / 16)
        return fail(MK_ERR_UNSUPPORTED, "prompt: too many sequences or queries in one call");
    if ((a->n_tokens > 1 && (!a->q_token || !a->out_token)) || (a->n_keys > 1 && (!a->k_token || !a->rope_token || !a->v_token)) ||
        (a->n_heads > 1 && !a->out_head))
        return fail(MK_ERR_UNSUPPORTED, "prompt: tokens must not share their rows (a stride of 0), nor heads those of out");
    // sequences with queries at most (the others are padding), and blocks of them
    const int some = a->batch < a->n_tokens ? a->batch : a->n_tokens;
    const int64_t blocks = (a->n_tokens + (int64_t)(PAIR - 1) * some) / PAIR * a->n_heads;
    if (blocks > INT32_MAX / 8) return fail(MK_ERR_UNSUPPORTED, "prompt: too many sequences or queries in one call");
    PromptP p = {};
    p.q_starts = a->q_starts, p.k_starts = a->k_starts;
    p.out = (uint8_t*)a->out, p.lse = a->lse, p.status = a->status, p.ot = a->out_token, p.oh = a->out_head;
    p.B = a->batch, p.n_q = a->n_tokens, p.n_k = a->n_keys, p.H = a->n_heads, p.scale = a->scale;
    p.q_heads = a->q_head != 0, p.k_heads = a->k_head != 0, p.v_heads = a->v_head != 0;
    const long long ns = mk_wait_ns_();
    p.wait_ns = (unsigned)(ns < 4000000000ll ? ns : 4000000000ll);
    p.signals = signalled_tiles();
    const int H = a->n_heads, dt = a->dtype, M = a->n_keys;
    PromptMaps maps = {};
    if (const int rc = map_of(a->q, dt, NOPE + ROPE, p.q_heads ? H : 0, a->n_tokens, a->q_head, a->q_token, ROWS, &maps.q)) return rc;
    if (M) {  // (without keys nothing is copied)
        if (const int rc = map_of(a->k, dt, NOPE, p.k_heads ? H : 0, M, a->k_head, a->k_token, TILE, &maps.k)) return rc;
        if (const int rc = map_of(a->k_rope, dt, ROPE, -1, M, 0, a->rope_token, TILE, &maps.r)) return rc;
        if (const int rc = map_of(a->v, dt, VD, p.v_heads ? H : 0, M, a->v_head, a->v_token, 64, &maps.v)) return rc;
    }
    cudaStream_t s = (cudaStream_t)stream;
    return dt == MK_DT_F16 ? run<true>(p, maps, some, blocks, s) : run<false>(p, maps, some, blocks, s);
}
