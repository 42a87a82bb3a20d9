// mk_rotary.cu -- rotation by positions (mk_rotate), and rows into a latent
// cache, normalised and rotated on the way (mk_latent_write).
//
// Angles. A frequency becomes 2^-64ths of a turn a position, an integer; times
// the position, modulo 2^64, it is the angle exactly, however far the position
// is (a 32-bit product of radians would be 0.06 off at position 10^6). Its upper
// 32 bits, rounded to 24, go to the half-turn sine and cosine: 2^-25 half turns.
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

// 2^-64ths of a turn a position
__device__ __forceinline__ unsigned long long turns_of(double radians) {
    const double t = radians * 0.15915494309189533577;  // 1 / (2 pi)
    return __double2ull_rn((t - floor(t)) * 18446744073709551616.0);
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
    int B, T, half, first, n, pairs;  // pairs: neighbours turn together
    int turned, units, upt;           // of a head: units that turn, all of them; of a token
    unsigned magic_h, magic_t;        // u / units and u / upt by the high word of a product
    int toks, tokens;                 // of a block's turn, of the call
};

constexpr int RT = 256;

// A block's turn is some tokens: their cosines and sines once, in shared
// memory, then units of 8 pairs (VEC; two 16-byte words in, two out) or of one
// pair. Values of a head that do not turn are copied in units of 8 or one.
// Bound by HBM for prompts (the angles are an n-th of a head's work for each of
// the heads), by a launch and three trips to memory for single tokens.
template <int DT, bool VEC>
__global__ void __launch_bounds__(RT) rotate_kernel(const __grid_constant__ RotateP p) {
    extern __shared__ float2 cs[];  // [toks][half]
    __shared__ unsigned long long turns[MAX_HALF];
    for (int i = threadIdx.x; i < p.half; i += RT) turns[i] = turns_of(p.freq[i]);
    __syncthreads();
    constexpr int E = VEC ? 8 : 1;
    for (int n0 = blockIdx.x * p.toks; n0 < p.tokens; n0 += gridDim.x * p.toks) {
        const int toks = min(p.toks, p.tokens - n0);
        for (int i = threadIdx.x; i < toks * p.half; i += RT) {
            const int tok = i / p.half, j = i - tok * p.half;
            const int b = (n0 + tok) / p.T, t = n0 + tok - b * p.T;
            const long long at = p.position_s ? p.positions[b * p.position_s + t] : (long long)p.positions[b] + t;
            cs[i] = turn(turns[j], at, p.magnitude, p.sign);
        }
        __syncthreads();
        for (int u = threadIdx.x; u < toks * p.upt; u += RT) {
            const int tok = toks > 1 ? (p.upt > 1 ? (int)__umulhi((unsigned)u, p.magic_t) : u) : 0;
            const int r = u - tok * p.upt, h = p.units > 1 ? (int)__umulhi((unsigned)r, p.magic_h) : r;
            const int c = r - h * p.units;
            const int b = (n0 + tok) / p.T, t = n0 + tok - b * p.T;
            const long long xr = b * p.xb + t * p.xt + h * p.xh, orow = b * p.ob + t * p.ot + h * p.oh;
            if (c < p.turned) {
                // values a .. and b .. : of a half layout the two halves' parts, else neighbours
                const int ia = p.first + (p.pairs ? 2 * E * c : E * c), ib = p.pairs ? ia + E : ia + p.half;
                const float2* const w = cs + tok * p.half + E * c;
                if constexpr (VEC) {
                    Values8<DT, true> va, vb;
                    va.load(p.x, xr + ia);
                    vb.load(p.x, xr + ib);
                    float x[8], y[8];
                    va.floats(x);
                    vb.floats(y);
                    if (p.pairs) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 f = w[i], g = w[4 + i];
                            const float x0 = x[2 * i], x1 = x[2 * i + 1], y0 = y[2 * i], y1 = y[2 * i + 1];
                            x[2 * i] = x0 * f.x - x1 * f.y, x[2 * i + 1] = x0 * f.y + x1 * f.x;
                            y[2 * i] = y0 * g.x - y1 * g.y, y[2 * i + 1] = y0 * g.y + y1 * g.x;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 f = w[i];
                            const float a = x[i], e = y[i];
                            x[i] = a * f.x - e * f.y, y[i] = a * f.y + e * f.x;
                        }
                    }
                    store8<DT, true>(p.out, orow + ia, x);
                    store8<DT, true>(p.out, orow + ib, y);
                } else {
                    const float a = load1<DT>(p.x, xr + ia), e = load1<DT>(p.x, xr + ib);
                    store1<DT>(p.out, orow + ia, a * w->x - e * w->y);
                    store1<DT>(p.out, orow + ib, a * w->y + e * w->x);
                }
            } else {
                int i = (c - p.turned) * E;
                if (i >= p.first) i += p.n;
                if constexpr (VEC) {
                    Values8<DT, true> v;
                    v.load(p.x, xr + i);
                    float x[8];
                    v.floats(x);
                    store8<DT, true>(p.out, orow + i, x);
                } else {
                    store1<DT>(p.out, orow + i, load1<DT>(p.x, xr + i));
                }
            }
        }
        __syncthreads();
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

int sm_count(int& sms, const char* what) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return cuda_status(e, what);
}

template <int DT>
void rotate_go(const RotateP& p, bool vec, int grid, cudaStream_t s) {
    const size_t smem = sizeof(float2) * p.toks * p.half;
    if (vec) rotate_kernel<DT, true><<<grid, RT, smem, s>>>(p);
    else rotate_kernel<DT, false><<<grid, RT, smem, s>>>(p);
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

// A warp a row: V pieces of 8 latent values a lane, their squares summed by
// shuffles; a pair of the rope part a lane. A warp's gains and frequencies are
// loaded once for all its rows. Bound by HBM for prompts.
template <int DT, bool VEC, int V>
__global__ void __launch_bounds__(WT) latent_write_kernel(const __grid_constant__ LatentWriteP p) {
    const int lane = threadIdx.x & 31, warps = gridDim.x * (WT / 32);
    const long long total = (long long)p.B * p.n;
    float gain[V][8];
    unsigned long long turns[4];
    if (p.gain) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = 8 * (v * 32 + lane);
            if (i < p.rank) {
#pragma unroll
                for (int e = 0; e < 8; ++e) gain[v][e] = gain_at(p, i + e);
            }
        }
    }
    if (p.freq) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j * 32 + lane < p.rope_dim / 2) turns[j] = turns_of(p.freq[j * 32 + lane]);
    }
    for (long long row = (long long)blockIdx.x * (WT / 32) + (threadIdx.x >> 5); row < total; row += warps) {
        const int b = (int)(row / p.n), t = (int)(row - (long long)b * p.n);
        if (p.counts && t >= p.counts[b]) continue;
        const long long src = b * p.rb + t * p.rt;
        Values8<DT, VEC> x[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = 8 * (v * 32 + lane);
            if (i < p.rank) x[v].load(p.rows, src + i);
            else x[v].zero();
        }
        const long long pos = (long long)p.positions[b] + t, col = pos >> p.ps_shift;
        const int page = pos >= 0 && col < p.pps ? p.table[b * p.table_s + col] : -1;
        if ((unsigned)page >= (unsigned)p.n_pages) {
            if (p.status) *p.status = MK_ERR_INVALID_ARG;
            continue;
        }
        const int r = (int)(pos & ((1 << p.ps_shift) - 1));
        float f = 1.f;
        if (p.gain) {
            float sum = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float y[8];
                x[v].floats(y);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum += y[e] * y[e];
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            f = rsqrtf(sum / (float)p.rank + p.eps);
        }
        const long long to = page * p.page_s + r * p.row_s;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = 8 * (v * 32 + lane);
            if (i >= p.rank) continue;
            float y[8];
            x[v].floats(y);
            if (p.gain) {
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = y[e] * f * gain[v][e];
            }
            if (p.f16) store8<MK_DT_F16, true>(p.latent, to + i, y);
            else store8<MK_DT_BF16, true>(p.latent, to + i, y);
        }
        const long long rto = page * p.rope_page_s + r * p.rope_row_s;
        const int half = p.rope_dim / 2;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = j * 32 + lane;
            if (i >= half) break;
            const int ia = p.pairs ? 2 * i : i, ib = p.pairs ? ia + 1 : i + half;
            float a = load1<DT>(p.rows, src + p.rank + ia), e = load1<DT>(p.rows, src + p.rank + ib);
            if (p.freq) {
                const float2 w = turn(turns[j], pos, p.magnitude, p.sign);
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

template <int DT, bool VEC>
void write_go(const LatentWriteP& p, int grid, cudaStream_t s) {
    if (p.rank <= 256) latent_write_kernel<DT, VEC, 1><<<grid, WT, 0, s>>>(p);
    else if (p.rank <= 512) latent_write_kernel<DT, VEC, 2><<<grid, WT, 0, s>>>(p);
    else latent_write_kernel<DT, VEC, 4><<<grid, WT, 0, s>>>(p);
}

}  // namespace

extern "C" int mk_rotate(const mk_rotation* a, void* stream) {
    if (!a) return fail(MK_ERR_INVALID_ARG, "rotate: NULL arguments");
    if (const int rc = check_rotary(a->rotary, "rotate")) return rc;
    const mk_rotary& r = *a->rotary;
    if (!a->positions || off_by4(a->positions)) return fail(MK_ERR_INVALID_ARG, "rotate: positions is NULL or not aligned to 4 bytes");
    if (const int rc = check_rows(a->x, "x")) return rc;
    if (const int rc = check_rows(a->out, "out")) return rc;
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
    p.B = a->batch, p.T = a->n_tokens, p.half = r.n / 2, p.first = a->first, p.n = r.n;
    p.pairs = r.layout == MK_ROTARY_PAIRS;
    const bool in_place = x.data == o.data && x.seq_stride == o.seq_stride && x.token_stride == o.token_stride &&
                          x.head_stride == o.head_stride;
    const bool vec = rows_vec(&x) && rows_vec(&o) && r.n % 16 == 0 && a->first % 8 == 0 && a->head_dim % 8 == 0;
    const int e = vec ? 8 : 1;
    p.turned = p.half / e;
    p.units = p.turned + (in_place ? 0 : (a->head_dim - r.n) / e);
    p.upt = a->n_heads * p.units;
    p.tokens = a->batch * a->n_tokens;
    int sms = 0;
    if (const int rc = sm_count(sms, "mk_rotate")) return rc;
    // a block's turn: four units a thread, as long as every SM has a block, and its angles fit 16 KB
    int toks = 4 * RT / p.upt, most = 2048 / p.half, spread = (p.tokens + sms - 1) / sms;
    toks = toks < most ? toks : most;
    toks = toks < spread ? toks : spread;
    p.toks = toks < 1 ? 1 : toks;
    // exact for units of a token (some below 2^28) only where the product with the divisor stays below 2^32
    if ((int64_t)p.toks * p.upt * (int64_t)p.upt >= (1ll << 32) && p.toks > 1) p.toks = 1;
    if ((int64_t)p.upt * p.units >= (1ll << 32)) return fail(MK_ERR_UNSUPPORTED, "rotate: heads too many or too wide");
    p.magic_h = (unsigned)(0x100000000ull / p.units + 1);
    p.magic_t = (unsigned)(0x100000000ull / p.upt + 1);
    const int turns = (p.tokens + p.toks - 1) / p.toks, grid = turns < 8 * sms ? turns : 8 * sms;
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
    if (const int rc = check_rows(rows, "rows")) return rc;
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
    int sms = 0;
    if (const int rc = sm_count(sms, "mk_latent_write")) return rc;
    const int unit = rows->dtype == MK_DT_F32 ? 4 : 8;
    const bool vec = (uintptr_t)rows->data % 16 == 0 && rows->seq_stride % unit == 0 && rows->token_stride % unit == 0;
    const int64_t want = ((int64_t)t->batch * n + WT / 32 - 1) / (WT / 32);
    const int grid = (int)(want < 16 * sms ? want : 16 * sms);
    cudaStream_t s = (cudaStream_t)stream;
    auto go = [&](auto f, auto slow) { vec ? f(p, grid, s) : slow(p, grid, s); };
    if (rows->dtype == MK_DT_F32) go(write_go<MK_DT_F32, true>, write_go<MK_DT_F32, false>);
    else if (rows->dtype == MK_DT_BF16) go(write_go<MK_DT_BF16, true>, write_go<MK_DT_BF16, false>);
    else go(write_go<MK_DT_F16, true>, write_go<MK_DT_F16, false>);
    return cuda_status(cudaGetLastError(), "mk_latent_write");
}
