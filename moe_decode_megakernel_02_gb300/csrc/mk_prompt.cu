// mk_prompt.cu -- causal attention of prompts over expanded keys and values
// (mk_prompt_attend).
#include "mk_values.cuh"

namespace {

using namespace mkop;

constexpr int NOPE = 128, ROPE = 64, VD = 128;

struct PromptP {
    const int *q_starts, *k_starts;
    const uint8_t *q, *k, *kr, *v;
    uint8_t* out;
    float* lse;
    int* status;
    long long qt, qh, kt, kh, rt, vt, vh, ot, oh;  // elements
    int B, n_q, n_k, H;
    float scale;
};

constexpr int PT = 128;

// A block a query row, a key a warp at a time.
template <int DT>
__global__ void __launch_bounds__(PT) prompt_rows(const __grid_constant__ PromptP p) {
    __shared__ float om[PT / 32][VD], ml[PT / 32][2];
    const int row = blockIdx.x / p.H, h = blockIdx.x - row * p.H;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int q0, q1, k0, k1, mine = -1;
    for (int b = 0; b < p.B; ++b) {
        q0 = p.q_starts[b], q1 = p.q_starts[b + 1], k0 = p.k_starts[b], k1 = p.k_starts[b + 1];
        const bool good = 0 <= q0 && q0 <= q1 && q1 <= p.n_q && 0 <= k0 && k0 <= k1 && k1 <= p.n_k;
        if (!good && blockIdx.x == 0 && p.status) *p.status = MK_ERR_INVALID_ARG;
        if (good && q0 <= row && row < q1 && mine < 0) mine = b;
    }
    if (mine < 0) return;
    q0 = p.q_starts[mine], q1 = p.q_starts[mine + 1], k0 = p.k_starts[mine], k1 = p.k_starts[mine + 1];
    const int last = k1 - q1 + row;  // a row of k
    float q[8] = {}, o[4] = {};
    if (lane < (NOPE + ROPE) / 8) {
        Values8<DT, true> x;
        x.load(p.q, row * p.qt + h * p.qh + 8 * lane);
        x.floats(q);
    }
    float m = -INFINITY, l = 0.f;
    for (int j = k0 + warp; j <= last; j += PT / 32) {
        float s = 0.f, k[8] = {};
        Values8<DT, true> x;
        if (lane < NOPE / 8) {
            x.load(p.k, j * p.kt + h * p.kh + 8 * lane);
            x.floats(k);
        } else if (lane < (NOPE + ROPE) / 8) {
            x.load(p.kr, j * p.rt + 8 * lane - NOPE);
            x.floats(k);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) s += q[e] * k[e];
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= p.scale;
        const float mn = fmaxf(m, s), f = __expf(m - mn), w = __expf(s - mn);
        m = mn;
        l = l * f + w;
        const uint2 v2 = *reinterpret_cast<const uint2*>(p.v + 2 * (j * p.vt + h * p.vh + 4 * lane));
        float v[4];
        if constexpr (DT == MK_DT_BF16) {
            v[0] = bf2f(v2.x & 0xffffu), v[1] = bf2f(v2.x >> 16), v[2] = bf2f(v2.y & 0xffffu), v[3] = bf2f(v2.y >> 16);
        } else {
            const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v2.x)), c = __half22float2(*reinterpret_cast<const __half2*>(&v2.y));
            v[0] = a.x, v[1] = a.y, v[2] = c.x, v[3] = c.y;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = o[e] * f + w * v[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) om[warp][4 * lane + e] = o[e];
    if (lane == 0) ml[warp][0] = m, ml[warp][1] = l;
    __syncthreads();
    float mm = -INFINITY, ll = 0.f, y = 0.f;
    for (int w = 0; w < PT / 32; ++w) mm = fmaxf(mm, ml[w][0]);
    const float ref = mm == -INFINITY ? 0.f : mm;
    for (int w = 0; w < PT / 32; ++w) {
        ll += ml[w][1] * __expf(ml[w][0] - ref);
        y += om[w][threadIdx.x] * __expf(ml[w][0] - ref);
    }
    y = ll == 0.f ? 0.f : y / ll;
    const long long at = row * p.ot + h * p.oh + threadIdx.x;
    if constexpr (DT == MK_DT_F16) reinterpret_cast<__half*>(p.out)[at] = __float2half_rn(y);
    else reinterpret_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(y);
    if (threadIdx.x == 0 && p.lse) p.lse[(long long)row * p.H + h] = ll == 0.f ? -INFINITY : mm + logf(ll);
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
    if (a->batch > (1 << 20) || (int64_t)a->n_tokens * a->n_heads > INT32_MAX / 16)
        return fail(MK_ERR_UNSUPPORTED, "prompt: too many sequences or queries in one call");
    PromptP p = {};
    p.q_starts = a->q_starts, p.k_starts = a->k_starts;
    p.q = (const uint8_t*)a->q, p.k = (const uint8_t*)a->k, p.kr = (const uint8_t*)a->k_rope, p.v = (const uint8_t*)a->v;
    p.out = (uint8_t*)a->out, p.lse = a->lse, p.status = a->status;
    p.qt = a->q_token, p.qh = a->q_head, p.kt = a->k_token, p.kh = a->k_head, p.rt = a->rope_token;
    p.vt = a->v_token, p.vh = a->v_head, p.ot = a->out_token, p.oh = a->out_head;
    p.B = a->batch, p.n_q = a->n_tokens, p.n_k = a->n_keys, p.H = a->n_heads, p.scale = a->scale;
    const int grid = p.n_q * p.H;
    if (a->dtype == MK_DT_F16) prompt_rows<MK_DT_F16><<<grid, PT, 0, (cudaStream_t)stream>>>(p);
    else prompt_rows<MK_DT_BF16><<<grid, PT, 0, (cudaStream_t)stream>>>(p);
    return cuda_status(cudaGetLastError(), "mk_prompt_attend");
}
