// mk_latent.cu -- attention over a paged latent cache, in the latent space
// (mk_latent_attend).
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
        s *= p.scale;
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

int check(const mk_latent_attention* a) {
    if (!a) return fail(MK_ERR_INVALID_ARG, "latent attend: NULL arguments");
    if (const int rc = check_latent(a->pages, a->table)) return rc;
    const mk_latent_pages& g = *a->pages;
    if (a->n_tokens < 1 || a->n_heads < 1) return fail(MK_ERR_INVALID_ARG, "latent attend: n_tokens or n_heads below 1");
    if (!a->lens || off_by4(a->lens, a->starts, a->lse, a->status))
        return fail(MK_ERR_INVALID_ARG, "latent attend: lens is NULL, or lens, starts, lse or status not aligned to 4 bytes");
    if (const int rc = check_rows(a->q, "q")) return rc;
    if (const int rc = check_rows(a->q_rope, "q_rope")) return rc;
    if (const int rc = check_rows(a->out, "out")) return rc;
    if (a->q->dtype != g.dtype || a->q_rope->dtype != g.dtype || a->out->dtype != g.dtype)
        return fail(MK_ERR_INVALID_ARG, "latent attend: q, q_rope and out must have the cache's type");
    if (!(a->scale >= -1e30f && a->scale <= 1e30f)) return fail(MK_ERR_INVALID_ARG, "latent attend: scale is not a number in range");
    if ((g.rank != 256 && g.rank != 512) || g.rope_dim != 64)
        return fail(MK_ERR_UNSUPPORTED, "latent attend: rank must be 256 or 512, rope_dim 64");
    if ((int64_t)a->table->batch * a->n_tokens * a->n_heads > INT32_MAX / 16)
        return fail(MK_ERR_UNSUPPORTED, "latent attend: too many queries in one call");
    return MK_OK;
}

}  // namespace

extern "C" int mk_latent_attend_workspace(const mk_latent_attention* a, int64_t* bytes) {
    if (const int rc = check(a)) return rc;
    if (!bytes) return fail(MK_ERR_INVALID_ARG, "latent attend: NULL bytes");
    *bytes = 0;
    return MK_OK;
}

extern "C" int mk_latent_attend(const mk_latent_attention* a, void*, int64_t, void* stream) {
    if (const int rc = check(a)) return rc;
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
    const int grid = p.B * p.T * p.H;
    cudaStream_t s = (cudaStream_t)stream;
    if (g.dtype == MK_DT_F16) g.rank == 512 ? latent_rows<MK_DT_F16, 512, 64><<<grid, LT, 0, s>>>(p) : latent_rows<MK_DT_F16, 256, 64><<<grid, LT, 0, s>>>(p);
    else g.rank == 512 ? latent_rows<MK_DT_BF16, 512, 64><<<grid, LT, 0, s>>>(p) : latent_rows<MK_DT_BF16, 256, 64><<<grid, LT, 0, s>>>(p);
    return cuda_status(cudaGetLastError(), "mk_latent_attend");
}
