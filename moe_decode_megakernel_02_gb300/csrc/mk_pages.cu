// mk_pages.cu -- rows into a paged cache and back (mk_pages_write,
// mk_pages_read): 8-bit codes with one fp32 scale a row, or bf16.
//
// A row's scale is its largest magnitude over the format's largest code; a
// block takes some tokens of a sequence with all their kv heads, looks up where
// they go once, and its threads take 8 or 16 values of a row each.
//
// Measured, 8 kv heads of 128, 16 ragged prompts of up to 4096 tokens: bf16
// rows into INT8 58 us (4.5 TB/s of reads and writes, 68 % of what a copy
// reaches), E4M3 back to bf16 65.9 us (6.2 TB/s, 92 %). The same into bf16 pages
// 62 us (83 %), and back 81 us (99 %). One new token of 8 sequences: 2.8 us, a
// launch.
#include <type_traits>

#include "mk_ops.cuh"

namespace mkop {

int check_pages(const mk_pages* p, const mk_page_table* t) {
    if (!p || !t || !p->k || !p->v || !t->table) return fail(MK_ERR_INVALID_ARG, "pages: NULL pages, table, k or v");
    if (p->format != MK_KV_BF16 && p->format != MK_KV_E4M3 && p->format != MK_KV_INT8)
        return fail(MK_ERR_INVALID_ARG, "pages: unknown format %d", p->format);
    if ((p->format != MK_KV_BF16) != (p->k_scale != nullptr) || (p->format != MK_KV_BF16) != (p->v_scale != nullptr))
        return fail(MK_ERR_INVALID_ARG, "pages: 8-bit formats need k_scale and v_scale, bf16 pages have none");
    if (p->n_pages < 1 || p->n_kv_heads < 1 || p->head_dim < 1 || t->batch < 1 || t->pages_per_seq < 1 || t->stride < 0)
        return fail(MK_ERR_INVALID_ARG, "pages: non-positive dimension");
    if (p->n_kv_heads > 65535 || t->batch > (1 << 20)) return fail(MK_ERR_UNSUPPORTED, "pages: too many heads or sequences");
    if (p->head_dim % 8 || p->head_dim > 256)
        return fail(MK_ERR_UNSUPPORTED, "pages: head_dim must be a multiple of 8, at most 256");
    if (log2_exact(p->page_size) < 0) return fail(MK_ERR_UNSUPPORTED, "pages: page_size must be a power of two");
    if ((int64_t)t->pages_per_seq * p->page_size > (1 << 30))
        return fail(MK_ERR_UNSUPPORTED, "pages: a sequence has at most 2^30 positions");
    if (off_by4(t->table, p->k_scale, p->v_scale))
        return fail(MK_ERR_INVALID_ARG, "pages: table or scales not aligned to 4 bytes");
    const int e = code_bytes(p->format);
    if ((uintptr_t)p->k % (8 * e) || (uintptr_t)p->v % (8 * e) || p->page_stride % 8 || p->head_stride % 8 ||
        p->row_stride % 8)
        return fail(MK_ERR_INVALID_ARG, "pages: k, v and their strides must be multiples of 8 elements");
    if (p->page_stride < 0 || p->head_stride < 0 || p->row_stride < 0 || p->scale_page_stride < 0 ||
        p->scale_head_stride < 0)
        return fail(MK_ERR_INVALID_ARG, "pages: negative stride");
    return MK_OK;
}

}  // namespace mkop

namespace {

using namespace mkop;

struct CopyP {
    uint8_t *k, *v;
    float *ks, *vs;
    long long page_s, head_s, row_s, sc_page, sc_head;  // elements
    const int* table;
    long long table_s;
    const int *positions, *counts;
    uint8_t *xk, *xv;                                  // the rows outside the cache
    long long kb, kt, kh, vb, vt, vh;                  // their strides, elements
    int pps, ps_shift, n_pages, H, n;
    int lanes, lanes_shift;  // threads of a row (8 or 16 values each), and the power of two they are spaced by
    int units, toks;         // of a token: H rows' threads; tokens of a block
    unsigned magic;          // unit / units by the high word of a product
    int chunks;              // blocks of a sequence
    int* status;
};

constexpr int CT = 256;    // threads of a block
constexpr int AHEAD = 4;   // rows of K and of V a reading thread has in flight
constexpr int TOKS = 64;   // most tokens of a block

// the larger of magnitudes (of one 32-bit number, or of two 16-bit ones); NaN wins
template <int DT>
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    if constexpr (DT == MK_DT_F32) return max(a, b);
    uint32_t y;
    if constexpr (DT == MK_DT_BF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}

// Eight values of a row outside the cache, as they lie there. VEC: 16-byte
// aligned.
template <int DT, bool VEC>
struct Values8 {
    static constexpr int W = DT == MK_DT_F32 ? 8 : 4;  // 32-bit words
    uint32_t w[W];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void load(const uint8_t* base, long long at) {
        if constexpr (VEC) {
            const uint4* p = reinterpret_cast<const uint4*>(base + at * (DT == MK_DT_F32 ? 4 : 2));
#pragma unroll
            for (int i = 0; i < W / 4; ++i) {
                const uint4 a = __ldcs(p + i);
                w[4 * i] = a.x, w[4 * i + 1] = a.y, w[4 * i + 2] = a.z, w[4 * i + 3] = a.w;
            }
        } else if constexpr (DT == MK_DT_F32) {
            const uint32_t* p = reinterpret_cast<const uint32_t*>(base) + at;
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = p[i];
        } else {
            const uint16_t* p = reinterpret_cast<const uint16_t*>(base) + at;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = p[2 * i] | (uint32_t)p[2 * i + 1] << 16;
        }
    }
    // 16-bit types are exact in 32 bits
    __device__ __forceinline__ void floats(float (&x)[8]) const {
        if constexpr (DT == MK_DT_F32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (DT == MK_DT_BF16) {
                    x[2 * i] = __uint_as_float(w[i] << 16);
                    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
                } else {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                    x[2 * i] = f.x;
                    x[2 * i + 1] = f.y;
                }
            }
        }
    }
    // the largest magnitude's bits; 16-bit types: of the even and of the odd values, side by side
    __device__ __forceinline__ uint32_t largest() const {
        constexpr uint32_t ABS = DT == MK_DT_F32 ? 0x7fffffffu : 0x7fff7fffu;
        uint32_t m = w[0] & ABS;
#pragma unroll
        for (int i = 1; i < W; ++i) m = larger<DT>(m, w[i] & ABS);
        return m;
    }
};
template <int DT>
__device__ __forceinline__ float magnitude(uint32_t bits) {
    if constexpr (DT == MK_DT_F32) return __uint_as_float(bits);
    else if constexpr (DT == MK_DT_BF16) return __uint_as_float(bits << 16);
    else return __half2float(__ushort_as_half((unsigned short)bits));
}

template <int DT, bool VEC>
__device__ __forceinline__ void store8(uint8_t* base, long long at, const float (&x)[8]) {
    if constexpr (DT == MK_DT_F32) {
        float* p = reinterpret_cast<float*>(base) + at;
        if constexpr (VEC) {
            __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
            __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = x[i];
        }
    } else {
        uint16_t* p = reinterpret_cast<uint16_t*>(base) + at;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = DT == MK_DT_BF16 ? pack_bf16(x[2 * i], x[2 * i + 1]) : pack_f16(x[2 * i], x[2 * i + 1]);
        if constexpr (VEC) {
            __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[2 * i] = (uint16_t)w[i];
                p[2 * i + 1] = (uint16_t)(w[i] >> 16);
            }
        }
    }
}

// The quotients x / s of a row, correctly rounded, from r = 1 / s: q = x r is
// within one unit of the last place, the remainder x - q s is exact in one
// fused multiply-add, and q + r (x - q s) rounds correctly when r is the
// correctly rounded reciprocal (Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990). Three operations a
// value. Scales so small that a remainder could be subnormal take the division.
__device__ __forceinline__ float quotient(float x, float s, float r) {
    const float q = x * r;
    return __fmaf_rn(__fmaf_rn(-q, s, x), r, q);
}
// largest / Q in the same way; r = 1 / Q
__device__ __forceinline__ float scale_of(float largest, float q, float r) {
    return largest < 0x1p-80f ? fmaxf(__fdiv_rn(largest, q), 0x1p-126f) : quotient(largest, q, r);
}

template <int FMT>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float scale) {
    float q[8];
    if (scale < 0x1p-80f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(x[i], scale);
    } else {
        const float r = __frcp_rn(scale);
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = quotient(x[i], scale, r);
    }
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if constexpr (FMT == MK_KV_E4M3) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q[4 * h], q[4 * h + 1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q[4 * h + 2], q[4 * h + 3]), __NV_SATFINITE, __NV_E4M3);
            w[h] = lo | hi << 16;
        } else {
            // adding 1.5 * 2^23 leaves the value rounded to an integer (ties
            // to even) in the low mantissa bits, as two's complement
            uint32_t c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = __float_as_uint(q[4 * h + i] + 12582912.0f);
            w[h] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
        }
    }
    return make_uint2(w[0], w[1]);
}

// A block's tokens: where each one's rows lie in the cache, -1 where they are
// to be left alone (past the count, or no such place).
struct Tokens {
    long long at[TOKS], scale[TOKS];
};
__device__ __forceinline__ void find_tokens(const CopyP& p, Tokens& tk, int b, int t0) {
    for (int i = threadIdx.x; i < p.toks; i += CT) {
        const int t = t0 + i;
        long long at = -1, scale = -1;
        if (t < p.n && (!p.counts || t < p.counts[b])) {
            const long long pos = (long long)p.positions[b] + t, col = pos >> p.ps_shift;
            const int page = pos >= 0 && col < p.pps ? p.table[b * p.table_s + col] : -1;
            if ((unsigned)page < (unsigned)p.n_pages) {
                const int r = (int)(pos & ((1 << p.ps_shift) - 1));
                at = page * p.page_s + r * p.row_s;
                scale = page * p.sc_page + r;
            } else if (p.status) {
                *p.status = MK_ERR_INVALID_ARG;
            }
        }
        tk.at[i] = at;
        tk.scale[i] = scale;
    }
}
// Unit u of a block: 8 values (piece c) of the row of kv head h of token `tok`.
__device__ __forceinline__ void unit_of(const CopyP& p, int u, int& tok, int& h, int& c) {
    tok = p.units == 1 ? u : p.toks > 1 ? (int)__umulhi((unsigned)u, p.magic) : 0;
    const int rest = u - tok * p.units;  // (a token of one unit: the magic number does not fit 32 bits)
    h = rest >> p.lanes_shift;
    c = rest & ((1 << p.lanes_shift) - 1);
}

// One thread: 8 G values of a row, of K and of V, WAHEAD rows at a time; the
// threads of a row lie in one warp and find its largest magnitude by shuffles,
// K's and V's together where they fit one word. The rows are fetched before the
// block knows where they go, so that the two trips to memory overlap. Reads 2
// or 4 bytes a value, writes 1 + 4 / head_dim, with 15.5 instructions a value (3
// of them the quotient); a thread takes 16 values where rows allow: 58 us in
// place of 73 for the prompts above. Neither issue (2.35 instructions a cycle of
// 4) nor HBM (45 %) is full there: 1326 blocks for the some 600 that run at once
// are 2.2 waves that cost 3, and a thread has one row in flight.
template <int FMT, int DT, bool VEC, int G>
__global__ void __launch_bounds__(CT, 3) write_kernel(const __grid_constant__ CopyP p) {
    constexpr int WAHEAD = G == 2 ? 1 : 2;
    __shared__ Tokens tk;
    const int b = blockIdx.x / p.chunks, t0 = (blockIdx.x - b * p.chunks) * p.toks;
    const int limit = p.counts ? min(p.counts[b], p.n) : p.n;
    if (t0 >= limit) return;
    const int all = min(p.toks, limit - t0) * p.units;
    const uint8_t* const xk = p.xk + (b * p.kb + t0 * p.kt) * (DT == MK_DT_F32 ? 4 : 2);
    const uint8_t* const xv = p.xv + (b * p.vb + t0 * p.vt) * (DT == MK_DT_F32 ? 4 : 2);
#pragma unroll 1
    for (int u0 = 0; u0 < all; u0 += CT * WAHEAD) {
        Values8<DT, VEC> k[WAHEAD][G], v[WAHEAD][G];
#pragma unroll
        for (int i = 0; i < WAHEAD; ++i) {
            if (u0 + i * CT >= all) break;
            int tok, h, c;
            unit_of(p, u0 + i * CT + threadIdx.x, tok, h, c);
            const bool in = u0 + i * CT + (int)threadIdx.x < all && c < p.lanes;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                if (in) {
                    k[i][g].load(xk, tok * p.kt + h * p.kh + 8 * (G * c + g));
                    v[i][g].load(xv, tok * p.vt + h * p.vh + 8 * (G * c + g));
                } else {
                    k[i][g].zero();
                    v[i][g].zero();
                }
            }
        }
        if (u0 == 0) {
            find_tokens(p, tk, b, t0);
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < WAHEAD; ++i) {
            if (u0 + i * CT >= all) break;
            int tok, h, c;
            const int u = u0 + i * CT + threadIdx.x;
            unit_of(p, u, tok, h, c);
            const long long row = u < all && c < p.lanes ? tk.at[tok] : -1;
            const long long at = row + h * p.head_s + 8 * G * c;
            if constexpr (FMT == MK_KV_BF16) {
                if (row >= 0) {
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        float x[8];
                        k[i][g].floats(x);
                        store8<MK_DT_BF16, true>(p.k, at + 8 * g, x);
                        v[i][g].floats(x);
                        store8<MK_DT_BF16, true>(p.v, at + 8 * g, x);
                    }
                }
            } else {
                uint32_t mk = k[i][0].largest(), mv = v[i][0].largest();
#pragma unroll
                for (int g = 1; g < G; ++g) {
                    mk = larger<DT>(mk, k[i][g].largest());
                    mv = larger<DT>(mv, v[i][g].largest());
                }
                if constexpr (DT == MK_DT_F32) {
                    for (int o = (1 << p.lanes_shift) >> 1; o; o >>= 1) {
                        mk = larger<DT>(mk, __shfl_xor_sync(0xffffffffu, mk, o));
                        mv = larger<DT>(mv, __shfl_xor_sync(0xffffffffu, mv, o));
                    }
                } else {  // both in one word
                    uint32_t m = larger<DT>(__byte_perm(mk, mv, 0x5410), __byte_perm(mk, mv, 0x7632));
                    for (int o = (1 << p.lanes_shift) >> 1; o; o >>= 1)
                        m = larger<DT>(m, __shfl_xor_sync(0xffffffffu, m, o));
                    mk = m & 0xffffu;
                    mv = m >> 16;
                }
                constexpr float QMAX = FMT == MK_KV_E4M3 ? 448.0f : 127.0f, QINV = 1.0f / QMAX;
                // the upper bound keeps code x scale finite for the largest 32-bit inputs
                constexpr float SMAX = FMT == MK_KV_E4M3 ? 0x1.249248p+119f : 0x1.020406p+121f;
                if (row < 0) continue;
                auto out = [&](const Values8<DT, VEC>(&x)[G], uint32_t bits, uint8_t* codes, float* scales) {
                    const float a = magnitude<DT>(bits);
                    const bool bad = !(a < INFINITY);
                    const float s = fminf(scale_of(a, QMAX, QINV), SMAX);
                    uint2 w[G];
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        float y[8];
                        x[g].floats(y);
                        w[g] = encode8<FMT>(y, s);
                        if (bad) w[g] = make_uint2(0, 0);
                    }
                    if constexpr (G == 2)
                        *reinterpret_cast<uint4*>(codes + at) = make_uint4(w[0].x, w[0].y, w[1].x, w[1].y);
                    else
                        *reinterpret_cast<uint2*>(codes + at) = w[0];
                    if (c == 0) scales[tk.scale[tok] + h * p.sc_head] = bad ? __uint_as_float(0x7fffffffu) : s;
                };
                out(k[i], mk, p.k, p.ks);
                out(v[i], mv, p.v, p.vs);
            }
        }
    }
}

// 8 cached values as they lie there: codes, or bf16
template <int FMT>
struct Raw8 {
    typename std::conditional<FMT == MK_KV_BF16, uint4, uint2>::type w;
    __device__ __forceinline__ void load(const uint8_t* base, long long at) {
        if constexpr (FMT == MK_KV_BF16) w = __ldcs(reinterpret_cast<const uint4*>(base + 2 * at));
        else w = __ldcs(reinterpret_cast<const uint2*>(base + at));
    }
    __device__ __forceinline__ void decode(float (&x)[8], float scale) const {
        if constexpr (FMT == MK_KV_BF16) {
            const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(v[i] << 16);
                x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t byte = ((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 0xffu;
                if constexpr (FMT == MK_KV_E4M3)
                    x[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3))) * scale;
                else
                    x[i] = (float)(int8_t)byte * scale;
            }
        }
    }
};

// The write's way back, the same threads for the same values; bound by HBM
// (93 % of a copy's rate).
template <int FMT, int DT, bool VEC>
__global__ void __launch_bounds__(CT) read_kernel(const __grid_constant__ CopyP p) {
    __shared__ Tokens tk;
    const int b = blockIdx.x / p.chunks, t0 = (blockIdx.x - b * p.chunks) * p.toks;
    const int limit = p.counts ? min(p.counts[b], p.n) : p.n;
    if (t0 >= limit) return;
    const int all = min(p.toks, limit - t0) * p.units;
    find_tokens(p, tk, b, t0);
    __syncthreads();
#pragma unroll 1
    for (int u0 = 0; u0 < all; u0 += CT * AHEAD) {
        Raw8<FMT> k[AHEAD], v[AHEAD];
        float sk[AHEAD], sv[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            int tok, h, c;
            const int u = u0 + i * CT + threadIdx.x;
            unit_of(p, u, tok, h, c);
            const long long row = u < all && c < p.lanes ? tk.at[tok] : -1;
            sk[i] = sv[i] = 1.f;
            if (row >= 0) {
                k[i].load(p.k, row + h * p.head_s + 8 * c);
                v[i].load(p.v, row + h * p.head_s + 8 * c);
                if constexpr (FMT != MK_KV_BF16) {
                    sk[i] = p.ks[tk.scale[tok] + h * p.sc_head];
                    sv[i] = p.vs[tk.scale[tok] + h * p.sc_head];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            int tok, h, c;
            const int u = u0 + i * CT + threadIdx.x;
            unit_of(p, u, tok, h, c);
            if (u < all && c < p.lanes && tk.at[tok] >= 0) {
                float x[8];
                k[i].decode(x, sk[i]);
                store8<DT, VEC>(p.xk, b * p.kb + (t0 + tok) * p.kt + h * p.kh + 8 * c, x);
                v[i].decode(x, sv[i]);
                store8<DT, VEC>(p.xv, b * p.vb + (t0 + tok) * p.vt + h * p.vh + 8 * c, x);
            }
        }
    }
}

template <bool WRITE, int FMT, int DT>
void launch3(const CopyP& p, bool vec, bool wide, unsigned blocks, cudaStream_t s) {
    if constexpr (WRITE) {
        if (vec && wide) write_kernel<FMT, DT, true, 2><<<blocks, CT, 0, s>>>(p);
        else if (vec) write_kernel<FMT, DT, true, 1><<<blocks, CT, 0, s>>>(p);
        else write_kernel<FMT, DT, false, 1><<<blocks, CT, 0, s>>>(p);
    } else {
        if (vec) read_kernel<FMT, DT, true><<<blocks, CT, 0, s>>>(p);
        else read_kernel<FMT, DT, false><<<blocks, CT, 0, s>>>(p);
    }
}

template <bool WRITE, int FMT>
void launch2(const CopyP& p, int dt, bool vec, bool wide, unsigned blocks, cudaStream_t s) {
    if (dt == MK_DT_F32) launch3<WRITE, FMT, MK_DT_F32>(p, vec, wide, blocks, s);
    else if (dt == MK_DT_BF16) launch3<WRITE, FMT, MK_DT_BF16>(p, vec, wide, blocks, s);
    else launch3<WRITE, FMT, MK_DT_F16>(p, vec, wide, blocks, s);
}

int check_rows(const mk_rows* r, const char* name) {
    if (!r || !r->data) return fail(MK_ERR_INVALID_ARG, "pages: %s is NULL", name);
    const int e = dtype_bytes(r->dtype);
    if (!e) return fail(MK_ERR_INVALID_ARG, "pages: unknown dtype %d of %s", r->dtype, name);
    if ((uintptr_t)r->data % e) return fail(MK_ERR_INVALID_ARG, "pages: %s is not aligned to its type", name);
    return MK_OK;
}

bool rows_vec(const mk_rows* r) {
    const int unit = r->dtype == MK_DT_F32 ? 4 : 8;  // elements in 16 bytes
    return (uintptr_t)r->data % 16 == 0 && r->seq_stride % unit == 0 && r->token_stride % unit == 0 &&
           r->head_stride % unit == 0;
}

template <bool WRITE>
int copy(const mk_pages* g, const mk_page_table* t, const int32_t* positions, const int32_t* counts, int32_t n,
         const mk_rows* k, const mk_rows* v, int32_t* status, void* stream) {
    if (const int rc = check_pages(g, t)) return rc;
    if (!positions) return fail(MK_ERR_INVALID_ARG, "pages: positions is NULL");
    if (off_by4(positions, counts, status))
        return fail(MK_ERR_INVALID_ARG, "pages: positions, counts or status not aligned to 4 bytes");
    if (n < 0) return fail(MK_ERR_INVALID_ARG, "pages: negative token count");
    if (const int rc = check_rows(k, "k")) return rc;
    if (const int rc = check_rows(v, "v")) return rc;
    if (k->dtype != v->dtype) return fail(MK_ERR_INVALID_ARG, "pages: k and v rows must have one type");
    if (n == 0) return MK_OK;
    CopyP p;
    p.k = (uint8_t*)g->k, p.v = (uint8_t*)g->v, p.ks = g->k_scale, p.vs = g->v_scale;
    p.page_s = g->page_stride, p.head_s = g->head_stride, p.row_s = g->row_stride;
    p.sc_page = g->scale_page_stride, p.sc_head = g->scale_head_stride;
    p.table = t->table, p.table_s = t->stride, p.pps = t->pages_per_seq;
    p.positions = positions, p.counts = counts;
    p.xk = (uint8_t*)k->data, p.kb = k->seq_stride, p.kt = k->token_stride, p.kh = k->head_stride;
    p.xv = (uint8_t*)v->data, p.vb = v->seq_stride, p.vt = v->token_stride, p.vh = v->head_stride;
    p.ps_shift = log2_exact(g->page_size), p.n_pages = g->n_pages, p.H = g->n_kv_heads, p.n = n;
    p.status = status;
    const bool vec = rows_vec(k) && rows_vec(v);
    // 16 values a thread: 16-byte stores of codes
    const bool wide = WRITE && vec && g->head_dim % 16 == 0 && g->page_stride % 16 == 0 && g->head_stride % 16 == 0 &&
                      g->row_stride % 16 == 0 && (uintptr_t)g->k % 16 == 0 && (uintptr_t)g->v % 16 == 0;
    p.lanes = g->head_dim / (wide ? 16 : 8), p.lanes_shift = 0;
    while ((1 << p.lanes_shift) < p.lanes) ++p.lanes_shift;
    p.units = p.H << p.lanes_shift;
    // a block's tokens keep its threads busy twice over, or are all there are
    int toks = 2 * CT * AHEAD / p.units;
    p.toks = toks < 1 ? 1 : toks > TOKS ? TOKS : toks;
    if (p.toks > n) p.toks = n;
    p.magic = (unsigned)(0x100000000ull / p.units + 1);  // exact for the units of a block: below 2^16
    p.chunks = (n + p.toks - 1) / p.toks;
    const int64_t blocks64 = (int64_t)t->batch * p.chunks;
    if (blocks64 > INT32_MAX) return fail(MK_ERR_UNSUPPORTED, "pages: too many rows in one call");
    const unsigned blocks = (unsigned)blocks64;
    cudaStream_t s = (cudaStream_t)stream;
    if (g->format == MK_KV_BF16)
        launch2<WRITE, MK_KV_BF16>(p, k->dtype, vec, wide, blocks, s);
    else if (g->format == MK_KV_E4M3)
        launch2<WRITE, MK_KV_E4M3>(p, k->dtype, vec, wide, blocks, s);
    else
        launch2<WRITE, MK_KV_INT8>(p, k->dtype, vec, wide, blocks, s);
    return cuda_status(cudaGetLastError(), WRITE ? "mk_pages_write" : "mk_pages_read");
}

}  // namespace

extern "C" int mk_pages_write(const mk_pages* pages, const mk_page_table* table, const int32_t* positions,
                              const int32_t* counts, int32_t n, const mk_rows* k, const mk_rows* v, int32_t* status,
                              void* stream) {
    return copy<true>(pages, table, positions, counts, n, k, v, status, stream);
}

extern "C" int mk_pages_read(const mk_pages* pages, const mk_page_table* table, const int32_t* positions,
                             const int32_t* counts, int32_t n, const mk_rows* k, const mk_rows* v, int32_t* status,
                             void* stream) {
    return copy<false>(pages, table, positions, counts, n, k, v, status, stream);
}
