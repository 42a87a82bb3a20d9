// mk_pages.cu -- rows into a paged cache and back (mk_pages_write,
// mk_pages_read): 8-bit codes with one fp32 scale a row, or bf16.
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
    int pps, ps_shift, n_pages, H, D, n;
    unsigned rows;  // B * n * H
    int* status;
};

constexpr int CT = 256;

// eight values of a row outside the cache, as fp32. VEC: 8 elements' bytes
// aligned. The fp32 values of 16-bit types are exact.
template <int DT, bool VEC>
__device__ __forceinline__ void load8(float (&x)[8], const uint8_t* base, long long at) {
    if constexpr (DT == MK_DT_F32) {
        const float* p = reinterpret_cast<const float*>(base) + at;
        if constexpr (VEC) {
            const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
            x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = p[i];
        }
    } else {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(base) + at;
        uint32_t w[4];
        if constexpr (VEC) {
            const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
            w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = p[2 * i] | (uint32_t)p[2 * i + 1] << 16;
        }
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
__device__ __forceinline__ float quotient(float x, float s, float r, bool tiny) {
    if (tiny) return __fdiv_rn(x, s);
    const float q = x * r;
    return __fmaf_rn(__fmaf_rn(-q, s, x), r, q);
}

template <int FMT>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float scale) {
    const float r = __frcp_rn(scale);
    const bool tiny = scale < 0x1p-80f;
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if constexpr (FMT == MK_KV_E4M3) {
            float q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = quotient(x[4 * h + i], scale, r, tiny);
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q[0], q[1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q[2], q[3]), __NV_SATFINITE, __NV_E4M3);
            w[h] = lo | hi << 16;
        } else {
            // adding 1.5 * 2^23 leaves the value rounded to an integer (ties
            // to even) in the low mantissa bits, as two's complement
            uint32_t c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = __float_as_uint(quotient(x[4 * h + i], scale, r, tiny) + 12582912.0f);
            w[h] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
        }
    }
    return make_uint2(w[0], w[1]);
}

// One thread: 8 values of a row, of K and of V; `lanes` = head_dim / 8 threads
// of a warp hold a row, the row's largest magnitude by shuffles among them.
// Magnitudes are compared as the bits of |x|, so a NaN wins and is seen. Bound
// by HBM (reads 2-4 bytes a value, writes 1 + 4/head_dim): K and V together
// keep two 16-byte loads a thread in flight. Measured times: at the launch.
template <int FMT, int DT, bool VEC>
__global__ void __launch_bounds__(CT) write_kernel(const CopyP p, int lanes, int lanes_shift) {
    const unsigned gid = blockIdx.x * CT + threadIdx.x;
    const unsigned row = gid >> lanes_shift;
    const int c = (int)(gid & ((1u << lanes_shift) - 1));
    bool live = row < p.rows && c < lanes;
    float xk[8], xv[8];
    long long at = 0, sat = 0;
    if (live) {
        const unsigned bt = row / (unsigned)p.H;
        const int h = (int)(row - bt * p.H);
        const int b = (int)(bt / (unsigned)p.n), t = (int)(bt - (unsigned)b * p.n);
        if (p.counts && t >= p.counts[b]) {
            live = false;
        } else {
            const long long pos = (long long)p.positions[b] + t;
            const long long col = pos >> p.ps_shift;
            const int page = pos >= 0 && col < p.pps ? p.table[b * p.table_s + col] : -1;
            if ((unsigned)page >= (unsigned)p.n_pages) {
                if (p.status) *p.status = MK_ERR_INVALID_ARG;
                live = false;
            } else {
                const int r = (int)(pos & ((1 << p.ps_shift) - 1));
                at = page * p.page_s + h * p.head_s + r * p.row_s + 8 * c;
                sat = page * p.sc_page + h * p.sc_head + r;
                load8<DT, VEC>(xk, p.xk, b * p.kb + t * p.kt + h * p.kh + 8 * c);
                load8<DT, VEC>(xv, p.xv, b * p.vb + t * p.vt + h * p.vh + 8 * c);
            }
        }
    }
    if constexpr (FMT == MK_KV_BF16) {
        if (!live) return;
        store8<MK_DT_BF16, true>(p.k, at, xk);
        store8<MK_DT_BF16, true>(p.v, at, xv);
    } else {
        uint32_t mk = 0, mv = 0;
        if (live) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                mk = max(mk, __float_as_uint(xk[i]) & 0x7fffffffu);
                mv = max(mv, __float_as_uint(xv[i]) & 0x7fffffffu);
            }
        }
        for (int o = (1 << lanes_shift) >> 1; o; o >>= 1) {
            mk = max(mk, __shfl_xor_sync(0xffffffffu, mk, o));
            mv = max(mv, __shfl_xor_sync(0xffffffffu, mv, o));
        }
        if (!live) return;
        constexpr float QMAX = FMT == MK_KV_E4M3 ? 448.0f : 127.0f;
        // the upper bound keeps code x scale finite for the largest 32-bit inputs
        constexpr float SMAX = FMT == MK_KV_E4M3 ? 0x1.249248p+119f : 0x1.020406p+121f;
        const float sk = fminf(fmaxf(__fdiv_rn(__uint_as_float(mk), QMAX), 0x1p-126f), SMAX);
        const float sv = fminf(fmaxf(__fdiv_rn(__uint_as_float(mv), QMAX), 0x1p-126f), SMAX);
        const bool bad_k = mk >= 0x7f800000u, bad_v = mv >= 0x7f800000u;
        const uint2 ck = bad_k ? make_uint2(0, 0) : encode8<FMT>(xk, sk);
        const uint2 cv = bad_v ? make_uint2(0, 0) : encode8<FMT>(xv, sv);
        *reinterpret_cast<uint2*>(p.k + at) = ck;
        *reinterpret_cast<uint2*>(p.v + at) = cv;
        if (c == 0) {
            p.ks[sat] = bad_k ? __uint_as_float(0x7fffffffu) : sk;
            p.vs[sat] = bad_v ? __uint_as_float(0x7fffffffu) : sv;
        }
    }
}

template <int FMT>
__device__ __forceinline__ void decode8(float (&x)[8], const uint8_t* base, long long at, float scale) {
    if constexpr (FMT == MK_KV_BF16) {
        load8<MK_DT_BF16, true>(x, base, at);
    } else {
        const uint2 w = __ldcs(reinterpret_cast<const uint2*>(base + at));
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

// The write's way back, the same threads for the same values; bound by HBM.
template <int FMT, int DT, bool VEC>
__global__ void __launch_bounds__(CT) read_kernel(const CopyP p, int lanes, int lanes_shift) {
    const unsigned gid = blockIdx.x * CT + threadIdx.x;
    const unsigned row = gid >> lanes_shift;
    const int c = (int)(gid & ((1u << lanes_shift) - 1));
    if (row >= p.rows || c >= lanes) return;
    const unsigned bt = row / (unsigned)p.H;
    const int h = (int)(row - bt * p.H);
    const int b = (int)(bt / (unsigned)p.n), t = (int)(bt - (unsigned)b * p.n);
    if (p.counts && t >= p.counts[b]) return;
    const long long pos = (long long)p.positions[b] + t;
    const long long col = pos >> p.ps_shift;
    const int page = pos >= 0 && col < p.pps ? p.table[b * p.table_s + col] : -1;
    if ((unsigned)page >= (unsigned)p.n_pages) {
        if (p.status) *p.status = MK_ERR_INVALID_ARG;
        return;
    }
    const int r = (int)(pos & ((1 << p.ps_shift) - 1));
    const long long at = page * p.page_s + h * p.head_s + r * p.row_s + 8 * c;
    const long long sat = page * p.sc_page + h * p.sc_head + r;
    float xk[8], xv[8];
    decode8<FMT>(xk, p.k, at, FMT == MK_KV_BF16 ? 1.f : p.ks[sat]);
    decode8<FMT>(xv, p.v, at, FMT == MK_KV_BF16 ? 1.f : p.vs[sat]);
    store8<DT, VEC>(p.xk, b * p.kb + t * p.kt + h * p.kh + 8 * c, xk);
    store8<DT, VEC>(p.xv, b * p.vb + t * p.vt + h * p.vh + 8 * c, xv);
}

template <bool WRITE, int FMT, int DT>
void launch3(const CopyP& p, bool vec, int lanes, int shift, unsigned blocks, cudaStream_t s) {
    if constexpr (WRITE) {
        if (vec)
            write_kernel<FMT, DT, true><<<blocks, CT, 0, s>>>(p, lanes, shift);
        else
            write_kernel<FMT, DT, false><<<blocks, CT, 0, s>>>(p, lanes, shift);
    } else {
        if (vec)
            read_kernel<FMT, DT, true><<<blocks, CT, 0, s>>>(p, lanes, shift);
        else
            read_kernel<FMT, DT, false><<<blocks, CT, 0, s>>>(p, lanes, shift);
    }
}

template <bool WRITE, int FMT>
void launch2(const CopyP& p, int dt, bool vec, int lanes, int shift, unsigned blocks, cudaStream_t s) {
    if (dt == MK_DT_F32)
        launch3<WRITE, FMT, MK_DT_F32>(p, vec, lanes, shift, blocks, s);
    else if (dt == MK_DT_BF16)
        launch3<WRITE, FMT, MK_DT_BF16>(p, vec, lanes, shift, blocks, s);
    else
        launch3<WRITE, FMT, MK_DT_F16>(p, vec, lanes, shift, blocks, s);
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
    if (n < 0) return fail(MK_ERR_INVALID_ARG, "pages: negative token count");
    if (const int rc = check_rows(k, "k")) return rc;
    if (const int rc = check_rows(v, "v")) return rc;
    if (k->dtype != v->dtype) return fail(MK_ERR_INVALID_ARG, "pages: k and v rows must have one type");
    if (n == 0) return MK_OK;
    const long long rows = (long long)t->batch * n * g->n_kv_heads;
    const int lanes = g->head_dim / 8;
    int shift = 0;
    while ((1 << shift) < lanes) ++shift;
    if (rows << shift > UINT32_MAX - CT) return fail(MK_ERR_UNSUPPORTED, "pages: too many rows in one call");
    CopyP p;
    p.k = (uint8_t*)g->k, p.v = (uint8_t*)g->v, p.ks = g->k_scale, p.vs = g->v_scale;
    p.page_s = g->page_stride, p.head_s = g->head_stride, p.row_s = g->row_stride;
    p.sc_page = g->scale_page_stride, p.sc_head = g->scale_head_stride;
    p.table = t->table, p.table_s = t->stride, p.pps = t->pages_per_seq;
    p.positions = positions, p.counts = counts;
    p.xk = (uint8_t*)k->data, p.kb = k->seq_stride, p.kt = k->token_stride, p.kh = k->head_stride;
    p.xv = (uint8_t*)v->data, p.vb = v->seq_stride, p.vt = v->token_stride, p.vh = v->head_stride;
    p.ps_shift = log2_exact(g->page_size), p.n_pages = g->n_pages, p.H = g->n_kv_heads, p.D = g->head_dim, p.n = n;
    p.rows = (unsigned)rows, p.status = status;
    const bool vec = rows_vec(k) && rows_vec(v);
    const unsigned blocks = (unsigned)(((rows << shift) + CT - 1) / CT);
    cudaStream_t s = (cudaStream_t)stream;
    if (g->format == MK_KV_BF16)
        launch2<WRITE, MK_KV_BF16>(p, k->dtype, vec, lanes, shift, blocks, s);
    else if (g->format == MK_KV_E4M3)
        launch2<WRITE, MK_KV_E4M3>(p, k->dtype, vec, lanes, shift, blocks, s);
    else
        launch2<WRITE, MK_KV_INT8>(p, k->dtype, vec, lanes, shift, blocks, s);
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
