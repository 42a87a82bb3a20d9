// mk_rotary.cu -- rotation by positions (mk_rotate), and rows into a latent
// cache, normalised and rotated on the way (mk_latent_write).
//
// Angles. A frequency becomes 2^-64ths of a turn a position, an integer, out of
// a product kept as the sum of two 64-bit numbers; times the position, modulo
// 2^64, it is the angle, however far the position is (a 32-bit product of
// radians would be 0.06 off at position 10^6). Its upper 32 bits, rounded to 24,
// go to the half-turn sine and cosine: 2^-25 half turns.
//
// Measured: 16004 tokens of 40 heads of 128, bf16, 56 us (5.9 TB/s, 86 % of a copy's
// rate); 8 tokens 3 us, a launch. The last 64 values of 4096 tokens' 16 heads of 192
// with the rest copied 18 (40 %): 320 blocks on 304 places (124 registers a thread),
// and a warp's turning and copying units run one after the other. Rows into a latent
// cache, 16 ragged prompts of up to 4096 tokens from fp32 28 us (5.2 TB/s, 77 %); 65536
// rows from bf16 32 (4.7 TB/s: as many instructions a row for fewer bytes, the rope
// part's of two bytes a lane); 8 tokens 2.7 us.
#include "mk_values.cuh"

namespace mkop {

int check_latent(const mk_latent_pages* p, const mk_page_table* t) {
    if (!p || !t || !p->latent || !p->rope || !t->table) return fail(MK_ERR_INVALID_ARG, "latent: NULL pages, table, latent or rope");
    if (p->dtype != MK_DT_BF16 && p->dtype != MK_DT_F16) return fail(MK_ERR_INVALID_ARG, "latent: the cache must be bf16 or fp16");
    if (p->n_pages < 1 || p->rank < 1 || p->rope_dim < 1 || t->batch < 1 || t->pages_per_seq < 1 || t->stride < 0)
        return fail(MK_ERR_INVALID_ARG, "latent: non-positive dimension");
    if (t->batch > (1 << 20)) return fail(MK_ERR_UNSUPPORTED, "latent: too many sequences");
    if (p->rank % 8 || p->rank > 1024 || p->rope_dim % 8 || p->rope_dim > 256)
        return fail(MK_ERR_UNSUPPORTED, "latent: rank must be a multiple of 8 up to 1024, rope_dim of 8 up to 256");
    if (log2_exact(p->page_size) < 0) return fail(MK_ERR_UNSUPPORTED, "latent: page_size must be a power of two");
    if ((int64_t)t->pages_per_seq * p->page_size > (1 << 30))
        return fail(MK_ERR_UNSUPPORTED, "latent: a sequence has at most 2^30 positions");
    if (off_by4(t->table)) return fail(MK_ERR_INVALID_ARG, "latent: table not aligned to 4 bytes");
    if ((uintptr_t)p->latent % 16 || (uintptr_t)p->rope % 16 || p->page_stride % 8 || p->row_stride % 8 ||
        p->rope_page_stride % 8 || p->rope_row_stride % 8)
        return fail(MK_ERR_INVALID_ARG, "latent: latent, rope and their strides must be multiples of 16 bytes");
    if (p->page_stride < 0 || p->row_stride < 0 || p->rope_page_stride < 0 || p->rope_row_stride < 0)
        return fail(MK_ERR_INVALID_ARG, "latent: negative stride");
    return MK_OK;
}

}  // namespace mkop

namespace {

using namespace mkop;

constexpr int MAX_HALF = 128;  // pairs of a rotation

// 2^-64ths of a turn a position, off by less than 2 (and 2^-40 |radians|): the quotient by 2 pi is high + low, the product's
// rounded value and what it left, each reduced to half a turn without loss (the sums of their 2^-64ths come round at 2^64)
__device__ __forceinline__ unsigned long long turns_of(double radians) {
    constexpr double INV = 0.15915494309189535, INV_LOW = -9.839338337591243e-18;  // 1 / (2 pi)
    const double high = __dmul_rn(radians, INV), low = fma(radians, INV_LOW, fma(radians, INV, -high));
    return (unsigned long long)__double2ll_rn((high - rint(high)) * 0x1p64) + (unsigned long long)__double2ll_rn((low - rint(low)) * 0x1p64);
}
// (cos, sin) at a position; sign -1: of the angle turned back
__device__ __forceinline__ float2 turn(unsigned long long turns, long long position, float magnitude, float sign) {
    const unsigned long long at = turns * (unsigned long long)position;
    float s, c;
    sincospif((float)(int)(at >> 32) * 0x1p-31f, &s, &c);
    return make_float2(c * magnitude, s * magnitude * sign);
}

template <int DT>
__device__ __forceinline__ float load1(const uint8_t* base, long long at) {
    if constexpr (DT == MK_DT_F32) return reinterpret_cast<const float*>(base)[at];
    else if constexpr (DT == MK_DT_BF16) return bf2f(reinterpret_cast<const uint16_t*>(base)[at]);
    else return __half2float(reinterpret_cast<const __half*>(base)[at]);
}
template <int DT>
__device__ __forceinline__ void store1(uint8_t* base, long long at, float x) {
    if constexpr (DT == MK_DT_F32) reinterpret_cast<float*>(base)[at] = x;
    else if constexpr (DT == MK_DT_BF16) reinterpret_cast<__nv_bfloat16*>(base)[at] = __float2bfloat16_rn(x);
    else reinterpret_cast<__half*>(base)[at] = __float2half_rn(x);
}

// ---------------------------------------------------------------- mk_rotate

struct RotateP {
    const double* freq;
    const int* positions;
    long long position_s;
    const uint8_t* x;
    uint8_t* out;
    long long xb, xt, xh, ob, ot, oh;  // elements
    float magnitude, sign;
    int T, H, half, first, n, pairs;  // pairs: neighbours turn together
    int turned, units;                // of a head: units that turn, all of them
    int heads, chunks;                // heads that one thread takes in turn, such parts of a token
    long long items;                  // units of all parts of all tokens
};

constexpr int RT = 256;

// A thread takes a unit (8 pairs: two 16-byte words in, two out; without VEC one pair) of a token through some of its heads:
// its sines and cosines are computed once and stay in registers. Values of a head that do not turn are copied, 8 or one a
// unit. A block's frequencies become turns once, in shared memory (64-bit arithmetic is slow here). Bound by HBM for
// prompts, by a launch and two trips to memory for single tokens.
template <int DT, bool VEC>
__global__ void __launch_bounds__(RT) rotate_kernel(const __grid_constant__ RotateP p) {
    constexpr int E = VEC ? 8 : 1, HEADS = DT == MK_DT_F32 ? 2 : 4;  // pairs of a unit, heads in flight
    __shared__ unsigned long long turns[MAX_HALF];
    for (int i = threadIdx.x; i < p.half; i += RT) turns[i] = turns_of(p.freq[i]);
    __syncthreads();
    for (long long item = (long long)blockIdx.x * RT + threadIdx.x; item < p.items; item += (long long)gridDim.x * RT) {
        const long long part = item / p.units;
        const int c = (int)(item - part * p.units), tok = (int)(part / p.chunks), ch = (int)(part - (long long)tok * p.chunks);
        const int b = tok / p.T, t = tok - b * p.T, h0 = ch * p.heads, h1 = min(p.H, h0 + p.heads);
        const uint8_t* const x = p.x;
        const long long xr = b * p.xb + t * p.xt, orow = b * p.ob + t * p.ot;
        if (c < p.turned) {
            const long long at = p.position_s ? p.positions[b * p.position_s + t] : (long long)p.positions[b] + t;
            float2 w[E];
#pragma unroll
            for (int i = 0; i < E; ++i) w[i] = turn(turns[E * c + i], at, p.magnitude, p.sign);
            // values from ia and ib on: of a half layout the two halves' parts, else neighbours
            const int ia = p.first + (p.pairs ? 2 * E * c : E * c), ib = p.pairs ? ia + E : ia + p.half;
            if constexpr (VEC) {
                for (int h = h0; h < h1; h += HEADS) {
                    Values8<DT, true> va[HEADS], vb[HEADS];
#pragma unroll
                    for (int k = 0; k < HEADS; ++k)
                        if (h + k < h1) {
                            va[k].load(x, xr + (h + k) * p.xh + ia);
                            vb[k].load(x, xr + (h + k) * p.xh + ib);
                        }
#pragma unroll
                    for (int k = 0; k < HEADS; ++k) {
                        if (h + k >= h1) break;
                        float a[8], e[8];
                        va[k].floats(a);
                        vb[k].floats(e);
                        if (p.pairs) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float a0 = a[2 * i], a1 = a[2 * i + 1], e0 = e[2 * i], e1 = e[2 * i + 1];
                                a[2 * i] = a0 * w[i].x - a1 * w[i].y, a[2 * i + 1] = a0 * w[i].y + a1 * w[i].x;
                                e[2 * i] = e0 * w[4 + i].x - e1 * w[4 + i].y, e[2 * i + 1] = e0 * w[4 + i].y + e1 * w[4 + i].x;
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float a0 = a[i], e0 = e[i];
                                a[i] = a0 * w[i].x - e0 * w[i].y, e[i] = a0 * w[i].y + e0 * w[i].x;
                            }
                        }
                        store8<DT, true>(p.out, orow + (h + k) * p.oh + ia, a);
                        store8<DT, true>(p.out, orow + (h + k) * p.oh + ib, e);
                    }
                }
            } else {
                for (int h = h0; h < h1; ++h) {
                    const float a = load1<DT>(x, xr + h * p.xh + ia), e = load1<DT>(x, xr + h * p.xh + ib);
                    store1<DT>(p.out, orow + h * p.oh + ia, a * w[0].x - e * w[0].y);
                    store1<DT>(p.out, orow + h * p.oh + ib, a * w[0].y + e * w[0].x);
                }
            }
        } else {
            int i = (c - p.turned) * E;
            if (i >= p.first) i += p.n;
            if constexpr (VEC) {
                for (int h = h0; h < h1; h += 2 * HEADS) {
                    Values8<DT, true> v[2 * HEADS];
#pragma unroll
                    for (int k = 0; k < 2 * HEADS; ++k)
                        if (h + k < h1) v[k].load(x, xr + (h + k) * p.xh + i);
#pragma unroll
                    for (int k = 0; k < 2 * HEADS; ++k) {
                        if (h + k >= h1) break;
                        float y[8];
                        v[k].floats(y);
                        store8<DT, true>(p.out, orow + (h + k) * p.oh + i, y);
                    }
                }
            } else {
                for (int h = h0; h < h1; ++h) store1<DT>(p.out, orow + h * p.oh + i, load1<DT>(x, xr + h * p.xh + i));
            }
        }
    }
}

int check_rotary(const mk_rotary* r, const char* what) {
    if (!r || !r->inv_freq) return fail(MK_ERR_INVALID_ARG, "%s: NULL rotary or inv_freq", what);
    if (r->n < 2 || r->n > 2 * MAX_HALF || r->n % 2) return fail(MK_ERR_INVALID_ARG, "%s: rotary n must be even, 2 to 256", what);
    if (r->layout != MK_ROTARY_HALF && r->layout != MK_ROTARY_PAIRS) return fail(MK_ERR_INVALID_ARG, "%s: unknown rotary layout %d", what, r->layout);
    if ((uintptr_t)r->inv_freq % 8) return fail(MK_ERR_INVALID_ARG, "%s: inv_freq not aligned to 8 bytes", what);
    if (!(r->magnitude >= -1e30f && r->magnitude <= 1e30f)) return fail(MK_ERR_INVALID_ARG, "%s: rotary magnitude is not a number in range", what);
    return MK_OK;
}

template <int DT>
void rotate_go(const RotateP& p, bool vec, int grid, cudaStream_t s) {
    if (vec) rotate_kernel<DT, true><<<grid, RT, 0, s>>>(p);
    else rotate_kernel<DT, false><<<grid, RT, 0, s>>>(p);
}

// ---------------------------------------------------------------- mk_latent_write

struct LatentWriteP {
    uint8_t *latent, *rope;
    long long page_s, row_s, rope_page_s, rope_row_s;  // elements
    const int* table;
    long long table_s;
    const int *positions, *counts;
    const uint8_t* rows;
    long long rb, rt;
    const uint8_t* gain;
    const double* freq;
    float eps, magnitude, sign;
    int pps, ps_shift, n_pages, rank, rope_dim, B, n, gain_dt, f16, pairs;
    int* status;
};

constexpr int WT = 128;

__device__ __forceinline__ float gain_at(const LatentWriteP& p, int i) {
    if (p.gain_dt == MK_DT_F32) return load1<MK_DT_F32>(p.gain, i);
    return p.gain_dt == MK_DT_BF16 ? load1<MK_DT_BF16>(p.gain, i) : load1<MK_DT_F16>(p.gain, i);
}

// A warp a row, two rows in flight: V pieces of 8 latent values a lane, their squares summed by shuffles; a pair of the rope
// part a lane. Gains and frequencies are loaded once for all of a block's rows. Bound by HBM for prompts.
template <int DT, bool VEC, int V, int RP>
__global__ void __launch_bounds__(WT, V <= 2 && RP == 1 ? 8 : 4) latent_write_kernel(const __grid_constant__ LatentWriteP p) {
    constexpr int R = V <= 2 ? 2 : 1;  // rows in flight; RP: pairs of a lane at most
    const int lane = threadIdx.x & 31, warps = gridDim.x * (WT / 32), half = p.rope_dim / 2;
    const long long total = (long long)p.B * p.n;
    // gains lie in shared memory by lanes: value e of piece v of lane l at (v 8 + e) 32 + l
    __shared__ float gain[V * 256];
    __shared__ unsigned long long all_turns[RP * 32];
    unsigned long long turns[RP];
    if (p.gain)
        for (int i = threadIdx.x; i < p.rank; i += WT) gain[(i >> 8) * 256 + (i & 7) * 32 + (i >> 3 & 31)] = gain_at(p, i);
    if (p.freq && threadIdx.x < half) all_turns[threadIdx.x] = turns_of(p.freq[threadIdx.x]);  // (64-bit arithmetic: once a block)
    __syncthreads();
    if (p.freq) {
#pragma unroll
        for (int j = 0; j < RP; ++j)
            if (j * 32 + lane < half) turns[j] = all_turns[j * 32 + lane];
    }
    auto pair_of = [&](int j, int& ia, int& ib) {
        const int i = j * 32 + lane;
        ia = p.pairs ? 2 * i : i, ib = p.pairs ? ia + 1 : i + half;
        return i < half;
    };
    for (long long row0 = (long long)blockIdx.x * (WT / 32) + (threadIdx.x >> 5); row0 < total; row0 += (long long)warps * R) {
        Values8<DT, VEC> x[R][V];
        float ra[R], rb[R];  // the first pair of the rope part
        long long src[R], pos[R];
        int page[R];         // -1: no row, -2: out of range
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const long long row = row0 + (long long)k * warps;
            page[k] = -1;
            if (row >= total) continue;
            const int b = (int)((unsigned)row / (unsigned)p.n), t = (int)((unsigned)row - (unsigned)b * (unsigned)p.n);
            if (p.counts && t >= p.counts[b]) continue;
            src[k] = b * p.rb + t * p.rt;
            pos[k] = (long long)p.positions[b] + t;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int i = 8 * (v * 32 + lane);
                if (i < p.rank) x[k][v].load(p.rows, src[k] + i);
                else x[k][v].zero();
            }
            int ia, ib;
            if (pair_of(0, ia, ib)) {
                ra[k] = load1<DT>(p.rows, src[k] + p.rank + ia);
                rb[k] = load1<DT>(p.rows, src[k] + p.rank + ib);
            }
            const long long col = pos[k] >> p.ps_shift;
            page[k] = pos[k] >= 0 && col < p.pps ? p.table[b * p.table_s + col] : -2;
            if ((unsigned)page[k] >= (unsigned)p.n_pages) page[k] = -2;
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (page[k] < 0) {
                if (page[k] == -2 && p.status) *p.status = MK_ERR_INVALID_ARG;
                continue;
            }
            const int r = (int)(pos[k] & ((1 << p.ps_shift) - 1));
            float f = 1.f;
            if (p.gain) {
                float sum = 0.f;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float y[8];
                    x[k][v].floats(y);
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum += y[e] * y[e];
                }
                sum *= 0x1p-8f;  // (a lane's 32 squares below 2^120 are in range, a row's 1024 would not be)
#pragma unroll
                for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                f = rsqrtf(sum / ((float)p.rank * 0x1p-8f) + p.eps);
            }
            const long long to = page[k] * p.page_s + r * p.row_s;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int i = 8 * (v * 32 + lane);
                if (i >= p.rank) continue;
                float y[8];
                x[k][v].floats(y);
                if (p.gain) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = y[e] * f * gain[(v * 8 + e) * 32 + lane];
                }
                if (p.f16) store8<MK_DT_F16, true>(p.latent, to + i, y);
                else store8<MK_DT_BF16, true>(p.latent, to + i, y);
            }
            const long long rto = page[k] * p.rope_page_s + r * p.rope_row_s;
#pragma unroll
            for (int j = 0; j < RP; ++j) {
                int ia, ib;
                if (!pair_of(j, ia, ib)) break;
                float a = j ? load1<DT>(p.rows, src[k] + p.rank + ia) : ra[k], e = j ? load1<DT>(p.rows, src[k] + p.rank + ib) : rb[k];
                if (p.freq) {
                    const float2 w = turn(turns[j], pos[k], p.magnitude, p.sign);
                    const float y = a * w.x - e * w.y;
                    e = a * w.y + e * w.x;
                    a = y;
                }
                if (p.f16) {
                    store1<MK_DT_F16>(p.rope, rto + ia, a);
                    store1<MK_DT_F16>(p.rope, rto + ib, e);
                } else {
                    store1<MK_DT_BF16>(p.rope, rto + ia, a);
                    store1<MK_DT_BF16>(p.rope, rto + ib, e);
                }
            }
        }
    }
}

template <int DT, bool VEC>
void write_go(const LatentWriteP& p, int grid, cudaStream_t s) {
    const bool one = p.rope_dim <= 64;
    if (p.rank <= 512) {
        if (one) latent_write_kernel<DT, VEC, 2, 1><<<grid, WT, 0, s>>>(p);
        else latent_write_kernel<DT, VEC, 2, 4><<<grid, WT, 0, s>>>(p);
    } else {
        if (one) latent_write_kernel<DT, VEC, 4, 1><<<grid, WT, 0, s>>>(p);
        else latent_write_kernel<DT, VEC, 4, 4><<<grid, WT, 0, s>>>(p);
    }
}

}  // namespace

extern "C" int mk_rotate(const mk_rotation* a, void* stream) {
    if (!a) return fail(MK_ERR_INVALID_ARG, "rotate: NULL arguments");
    if (const int rc = check_rotary(a->rotary, "rotate")) return rc;
    const mk_rotary& r = *a->rotary;
    if (!a->positions || off_by4(a->positions)) return fail(MK_ERR_INVALID_ARG, "rotate: positions is NULL or not aligned to 4 bytes");
    if (const int rc = check_rows(a->x, "rotate", "x")) return rc;
    if (const int rc = check_rows(a->out, "rotate", "out")) return rc;
    const mk_rows &x = *a->x, &o = *a->out;
    if (x.dtype != o.dtype) return fail(MK_ERR_INVALID_ARG, "rotate: x and out must have one type");
    if (a->batch < 0 || a->n_tokens < 0 || a->n_heads < 0 || a->head_dim < 1 || a->position_stride < 0)
        return fail(MK_ERR_INVALID_ARG, "rotate: negative dimension");
    if (a->first < 0 || a->first > a->head_dim - r.n)
        return fail(MK_ERR_INVALID_ARG, "rotate: values %d to %d of heads of %d", a->first, a->first + r.n - 1, a->head_dim);
    if (!a->batch || !a->n_tokens || !a->n_heads) return MK_OK;
    if ((int64_t)a->batch * a->n_tokens > INT32_MAX / 64 || a->n_heads > 4096 || a->head_dim > 65536)
        return fail(MK_ERR_UNSUPPORTED, "rotate: too many tokens, or heads beyond 4096 or 65536 values");
    RotateP p = {};
    p.freq = r.inv_freq, p.positions = a->positions, p.position_s = a->position_stride;
    p.x = (const uint8_t*)x.data, p.xb = x.seq_stride, p.xt = x.token_stride, p.xh = x.head_stride;
    p.out = (uint8_t*)o.data, p.ob = o.seq_stride, p.ot = o.token_stride, p.oh = o.head_stride;
    p.magnitude = r.magnitude, p.sign = r.inverse ? -1.f : 1.f;
    p.T = a->n_tokens, p.H = a->n_heads, p.half = r.n / 2, p.first = a->first, p.n = r.n;
    p.pairs = r.layout == MK_ROTARY_PAIRS;
    const bool in_place = x.data == o.data && x.seq_stride == o.seq_stride && x.token_stride == o.token_stride &&
                          x.head_stride == o.head_stride;
    const bool vec = rows_vec(&x) && rows_vec(&o) && r.n % 16 == 0 && a->first % 8 == 0 && a->head_dim % 8 == 0;
    const int e = vec ? 8 : 1;
    p.turned = p.half / e;
    p.units = p.turned + (in_place ? 0 : (a->head_dim - r.n) / e);
    int dev, sms;
    if (const int rc = device_sms(dev, sms, "mk_rotate")) return rc;
    // as many heads a thread (whose angles they share) as leave the device 1024 threads an SM
    const int64_t tokens = (int64_t)a->batch * a->n_tokens, all = tokens * p.units;
    p.chunks = (int)(1024ll * sms / all);
    if (p.chunks < 1) p.chunks = 1;
    p.heads = (p.H + p.chunks - 1) / p.chunks;
    p.chunks = (p.H + p.heads - 1) / p.heads;
    p.items = all * p.chunks;
    const int64_t want = (p.items + RT - 1) / RT;
    const int grid = (int)(want < 8 * sms ? want : 8 * sms);
    cudaStream_t s = (cudaStream_t)stream;
    if (x.dtype == MK_DT_F32) rotate_go<MK_DT_F32>(p, vec, grid, s);
    else if (x.dtype == MK_DT_BF16) rotate_go<MK_DT_BF16>(p, vec, grid, s);
    else rotate_go<MK_DT_F16>(p, vec, grid, s);
    return cuda_status(cudaGetLastError(), "mk_rotate");
}

extern "C" int mk_latent_write(const mk_latent_pages* g, const mk_page_table* t, const int32_t* positions,
                               const int32_t* counts, int32_t n, const mk_rows* rows, const void* gain,
                               int32_t gain_dtype, float eps, const mk_rotary* rotary, int32_t* status, void* stream) {
    if (const int rc = check_latent(g, t)) return rc;
    if (!positions) return fail(MK_ERR_INVALID_ARG, "latent: positions is NULL");
    if (off_by4(positions, counts, status))
        return fail(MK_ERR_INVALID_ARG, "latent: positions, counts or status not aligned to 4 bytes");
    if (n < 0) return fail(MK_ERR_INVALID_ARG, "latent: negative token count");
    if (const int rc = check_rows(rows, "latent", "rows")) return rc;
    if (gain) {
        const int e = dtype_bytes(gain_dtype);
        if (!e || (uintptr_t)gain % e) return fail(MK_ERR_INVALID_ARG, "latent: gain's type is unknown, or it is not aligned to it");
        if (!(eps >= 0.f && eps <= 1e30f)) return fail(MK_ERR_INVALID_ARG, "latent: eps is negative or no number in range");
    }
    if (rotary) {
        if (const int rc = check_rotary(rotary, "latent")) return rc;
        if (rotary->n != g->rope_dim) return fail(MK_ERR_INVALID_ARG, "latent: rotary n %d, rope_dim %d", rotary->n, g->rope_dim);
    }
    if (n == 0) return MK_OK;
    if ((int64_t)t->batch * n > INT32_MAX) return fail(MK_ERR_UNSUPPORTED, "latent: too many rows in one call");
    LatentWriteP p = {};
    p.latent = (uint8_t*)g->latent, p.rope = (uint8_t*)g->rope;
    p.page_s = g->page_stride, p.row_s = g->row_stride, p.rope_page_s = g->rope_page_stride, p.rope_row_s = g->rope_row_stride;
    p.table = t->table, p.table_s = t->stride, p.pps = t->pages_per_seq;
    p.positions = positions, p.counts = counts;
    p.rows = (const uint8_t*)rows->data, p.rb = rows->seq_stride, p.rt = rows->token_stride;
    p.gain = (const uint8_t*)gain, p.gain_dt = gain_dtype, p.eps = eps;
    p.freq = rotary ? rotary->inv_freq : nullptr;
    p.magnitude = rotary ? rotary->magnitude : 1.f, p.sign = rotary && rotary->inverse ? -1.f : 1.f;
    p.pairs = rotary && rotary->layout == MK_ROTARY_PAIRS;
    p.ps_shift = log2_exact(g->page_size), p.n_pages = g->n_pages, p.rank = g->rank, p.rope_dim = g->rope_dim;
    p.B = t->batch, p.n = n, p.f16 = g->dtype == MK_DT_F16, p.status = status;
    int dev, sms;
    if (const int rc = device_sms(dev, sms, "mk_latent_write")) return rc;
    const int unit = rows->dtype == MK_DT_F32 ? 4 : 8;
    const bool vec = (uintptr_t)rows->data % 16 == 0 && rows->seq_stride % unit == 0 && rows->token_stride % unit == 0;
    const int64_t want = ((int64_t)t->batch * n + WT / 32 - 1) / (WT / 32);
    const int grid = (int)(want < 8 * sms ? want : 8 * sms);
    cudaStream_t s = (cudaStream_t)stream;
    auto go = [&](auto f, auto slow) { vec ? f(p, grid, s) : slow(p, grid, s); };
    if (rows->dtype == MK_DT_F32) go(write_go<MK_DT_F32, true>, write_go<MK_DT_F32, false>);
    else if (rows->dtype == MK_DT_BF16) go(write_go<MK_DT_BF16, true>, write_go<MK_DT_BF16, false>);
    else go(write_go<MK_DT_F16, true>, write_go<MK_DT_F16, false>);
    return cuda_status(cudaGetLastError(), "mk_latent_write");
}
