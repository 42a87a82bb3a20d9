// mk_attend.cu -- host side of mk_pages_attend: checks, the choice of kernels,
// the workspace's layout and the launches.
#include <mutex>

#include "mk_attend.cuh"

namespace {

using namespace mkop;

constexpr int MAX_DEV = 32;
// Small calls: an item is one cluster's while that leaves a CTA at most so many
// tiles. One launch in place of two, and no workspace: 6 us less of the host's
// time, and for 8 sequences of 1024 positions (4 kv heads of 128) 10.6 us in
// place of 13.3 on the device, of 4096 16.6 in place of 17.8. One sequence,
// whose 4 clusters leave most of the device idle: 1024 positions 9.4 and 9.5,
// 4096 (8 tiles) 14.1 and 11.1, which the host's time outweighs, 6144 18.6 and
// 12.4, which it does not. Clusters of 16 take one sequence of 4096 to 11.4,
// but cost the others 1 to 3 us (and are not portable).
constexpr int CLUSTER_TILES = 8;
// Wide calls: from so many rows x tiles an SM on, the tiles that a sequence's
// tokens all see whole go to the tensor memory's kernel, the rest and the join
// being worth some 10 us. Measured without and with it, 16 query heads on 4 kv
// heads of 128, bf16: 8 sequences of 8192 positions, 28 rows 37 and 43 us, 128
// rows 88 and 71; 16 sequences of 16384, 28 rows 118 and 107, 56 rows 190 and
// 117; 256 tokens at 16384 217 and 83. 8-bit pages: 128 rows 96 and 80, 256
// tokens 242 and 125, but 28 rows at 65536 191 and 265: their conversion costs
// the same for fewer rows.
constexpr int64_t WIDE_WORK = 2000;

// KindInfo of each kernel on each device, asked for once
int kind_info(int dev, int d, const Kind& k, KindInfo& out) {
    static KindInfo cache[MAX_DEV][3][5][6];
    static bool have[MAX_DEV][3][5][6];
    static std::mutex lock;
    const int di = d == 64 ? 0 : d == 128 ? 1 : 2;
    const int ri = log2_exact(k.rows) - 3, fi = k.format * 2 + (k.splitq ? 1 : 0);
    const AttendFn fn = d == 64 ? attend_64 : d == 128 ? attend_128 : attend_256;
    if (dev >= MAX_DEV) return fn(k, nullptr, &out, 0, false, nullptr);
    std::lock_guard<std::mutex> g(lock);
    if (!have[dev][di][ri][fi]) {
        if (const int rc = fn(k, nullptr, &cache[dev][di][ri][fi], 0, false, nullptr)) return rc;
        have[dev][di][ri][fi] = true;
    }
    out = cache[dev][di][ri][fi];
    return MK_OK;
}

// one-time attributes of the kernels of mk_prefix.cuh
int prefix_info(int dev, int d, int format, bool f16, KindInfo& out) {
    static bool have[MAX_DEV][2][3][2];
    static std::mutex lock;
    out = KindInfo{64, 128, 1};
    std::lock_guard<std::mutex> g(lock);
    if (dev < MAX_DEV && have[dev][d == 128][format][f16]) return MK_OK;
    const int rc = (f16 ? prefix_f16 : prefix_bf16)(d, format, nullptr, 0, nullptr);
    if (dev < MAX_DEV && !rc) have[dev][d == 128][format][f16] = true;
    return rc;
}

struct Plan {
    Kind own_k, sh_k;
    int cluster;  // > 0: small call, an item a cluster
    bool prefix, wide;
    KindInfo own_i, sh_i;
    int own_grid, sh_grid;  // sh_grid 0: nothing shared
    int own_rb, sh_rb;
    int own_slot_rows, sh_slot_rows, own_floats, sh_floats;
    int64_t base_off, sh_base_off, own_off, sh_off, bytes;
};

int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }
int slot_floats(int rows, int d) { return rows * d + (2 * rows + 3) / 4 * 4; }

int make_plan(const mk_attention* a, Plan& pl) {
    if (!a) return fail(MK_ERR_INVALID_ARG, "attend: NULL arguments");
    if (const int rc = check_pages(a->pages, a->table)) return rc;
    const mk_pages& g = *a->pages;
    const mk_page_table& t = *a->table;
    const int D = g.head_dim, H = g.n_kv_heads, B = t.batch, T = a->n_tokens, Hq = a->n_q_heads;
    if (D != 64 && D != 128 && D != 256) return fail(MK_ERR_UNSUPPORTED, "attend: head_dim must be 64, 128 or 256");
    if (T < 1 || Hq < 1 || Hq % H) return fail(MK_ERR_INVALID_ARG, "attend: n_tokens, or n_q_heads not a multiple of n_kv_heads");
    const int eb = code_bytes(g.format);
    if ((uintptr_t)g.k % 16 || (uintptr_t)g.v % 16 || g.page_stride * eb % 16 || g.head_stride * eb % 16 ||
        g.row_stride * eb % 16)
        return fail(MK_ERR_INVALID_ARG, "attend: k, v and their strides must be multiples of 16 bytes");
    if (!a->lens || !a->q || !a->out || !a->q->data || !a->out->data)
        return fail(MK_ERR_INVALID_ARG, "attend: lens, q or out is NULL");
    if ((a->q->dtype != MK_DT_BF16 && a->q->dtype != MK_DT_F16) || a->out->dtype != a->q->dtype)
        return fail(MK_ERR_INVALID_ARG, "attend: q must be bf16 or fp16, out of the same type");
    if ((uintptr_t)a->q->data % 2 || (uintptr_t)a->out->data % 2)
        return fail(MK_ERR_INVALID_ARG, "attend: q or out not aligned to its type");
    if (off_by4(a->lens, a->starts, a->slopes, a->lse, a->status))
        return fail(MK_ERR_INVALID_ARG, "attend: lens, starts, slopes, lse or status not aligned to 4 bytes");
    if (!(a->scale == a->scale) || !(a->softcap == 0.f || (a->softcap >= 1e-30f && a->softcap <= 1e30f)))
        return fail(MK_ERR_INVALID_ARG, "attend: scale is NaN, or softcap not 0 and outside 1e-30 .. 1e30");
    const int64_t cap = (int64_t)t.pages_per_seq * g.page_size;
    if (a->shared_len < 0 || a->shared_len % g.page_size || a->shared_len > cap)
        return fail(MK_ERR_INVALID_ARG, "attend: shared_len must be whole pages of the table");
    if ((int64_t)B * T * Hq > INT32_MAX / 2) return fail(MK_ERR_UNSUPPORTED, "attend: too many queries in one call");
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_status(e, "mk_pages_attend");

    const int rows = T * (Hq / H);
    const bool splitq = g.format == MK_KV_BF16 && a->q->dtype == MK_DT_F16;
    // the least row block that holds the rows, or the largest there is
    auto block_of = [D](int64_t n) { return n <= 8 ? 8 : n <= 16 ? 16 : n <= 32 ? 32 : n <= 64 || D == 256 ? 64 : 128; };
    pl.own_k = Kind{g.format, splitq, block_of(rows)};
    if (const int rc = kind_info(dev, D, pl.own_k, pl.own_i)) return rc;
    if (pl.own_i.ctas < 1) return fail(MK_ERR_UNSUPPORTED, "attend: the kernel does not fit this device");
    pl.own_rb = (rows + pl.own_i.rows - 1) / pl.own_i.rows;
    pl.own_slot_rows = rows < pl.own_i.rows ? rows : pl.own_i.rows;
    pl.own_floats = slot_floats(pl.own_slot_rows, D);
    const int min_units = 2;
    const int64_t items = (int64_t)B * H * pl.own_rb;
    if (items > INT32_MAX / 16) return fail(MK_ERR_UNSUPPORTED, "attend: too many queries in one call");
    // (all items' clusters are resident at once, or nearly)
    pl.cluster = 0;
    pl.wide = false;
    if (!a->shared_len && pl.own_k.rows <= 32) {
        const int64_t tiles = (cap + pl.own_i.tile - 1) / pl.own_i.tile;
        int c = 1;
        while (c < MAX_CLUSTER && tiles > 4 * c && items * c * 2 <= (int64_t)sms * pl.own_i.ctas) c *= 2;
        if (tiles <= CLUSTER_TILES * c && items * c <= (int64_t)sms * pl.own_i.ctas * 2) {
            pl.cluster = c;
            pl.own_grid = (int)(items * c);
            pl.sh_grid = 0;
            pl.base_off = pl.own_off = pl.sh_off = pl.bytes = 0;
            return MK_OK;
        }
    }
    const int64_t most = items * ((cap + pl.own_i.tile - 1) / pl.own_i.tile + 1);
    if (most > (1 << 30)) return fail(MK_ERR_UNSUPPORTED, "attend: too many positions in one call");
    int64_t grid = (int64_t)sms * pl.own_i.ctas;
    if (grid > (most + min_units - 1) / min_units) grid = (most + min_units - 1) / min_units;
    pl.own_grid = (int)grid;
    // what the kernels of mk_prefix.cuh read (their tensor maps want distinct rows, 8 or more of them a page)
    const bool fits = D <= 128 && g.page_size >= 8 && g.row_stride > 0 && g.head_stride > 0 && g.page_stride > 0;
    if (!a->shared_len && fits && rows > (g.format == MK_KV_BF16 ? 16 : 32)) {
        const int64_t tiles = (int64_t)B * H * ((rows + 127) / 128) * (cap / 64);
        pl.wide = tiles * (rows < 128 ? rows : 128) >= WIDE_WORK * sms;
    }
    pl.base_off = 0;
    pl.sh_base_off = up256((int64_t)(B + 1) * 4);
    pl.own_off = 2 * pl.sh_base_off;
    const int64_t own_slots = 2 * grid + (a->shared_len || pl.wide ? items : 0);
    pl.bytes = up256(pl.own_off + own_slots * pl.own_floats * 4);
    pl.sh_grid = 0;
    pl.sh_off = pl.bytes;
    if (a->shared_len || pl.wide) {
        const int64_t all = pl.wide ? rows : (int64_t)B * rows;
        pl.sh_k = Kind{g.format, splitq, block_of(all)};
        // 8-bit pages: their conversion costs the same for few rows. A prefix of 16384 positions in 8 heads of 128,
        // without and with it: INT8 8 rows 31 and 44 us, 16 rows 40 and 44, 32 rows 53 and 49; bf16 4 rows 34 and
        // 34, 16 rows 44 and 38, 32 rows 55 and 42.
        pl.prefix = pl.wide || (fits && (g.format == MK_KV_BF16 || all > 16));
        if (const int rc = pl.prefix ? prefix_info(dev, D, g.format, a->q->dtype == MK_DT_F16, pl.sh_i) : kind_info(dev, D, pl.sh_k, pl.sh_i))
            return rc;
        if (pl.sh_i.ctas < 1) return fail(MK_ERR_UNSUPPORTED, "attend: the kernel does not fit this device");
        pl.sh_rb = (int)((all + pl.sh_i.rows - 1) / pl.sh_i.rows);
        pl.sh_slot_rows = (int)(all < pl.sh_i.rows ? all : pl.sh_i.rows);
        pl.sh_floats = slot_floats(pl.sh_slot_rows, D);
        const int64_t sh_items = (int64_t)H * pl.sh_rb * (pl.wide ? B : 1);
        const int64_t units = sh_items * (((pl.wide ? cap : a->shared_len) + pl.sh_i.tile - 1) / pl.sh_i.tile);
        if (units > (1 << 30)) return fail(MK_ERR_UNSUPPORTED, "attend: too many positions in one call");
        int64_t sg = (int64_t)sms * pl.sh_i.ctas;
        if (sg > (units + min_units - 1) / min_units) sg = (units + min_units - 1) / min_units;
        pl.sh_grid = (int)sg;
        pl.bytes = up256(pl.sh_off + (2 * sg + sh_items) * pl.sh_floats * 4);
    }
    return MK_OK;
}

}  // namespace

extern "C" int mk_pages_attend_workspace(const mk_attention* args, int64_t* bytes) {
    if (!bytes) return fail(MK_ERR_INVALID_ARG, "attend: bytes is NULL");
    Plan pl;
    if (const int rc = make_plan(args, pl)) return rc;
    *bytes = pl.bytes;
    return MK_OK;
}

extern "C" int mk_pages_attend(const mk_attention* a, void* workspace, int64_t workspace_bytes, void* stream) {
    Plan pl;
    if (const int rc = make_plan(a, pl)) return rc;
    if (pl.bytes && (!workspace || (uintptr_t)workspace % 256 || workspace_bytes < pl.bytes))
        return fail(MK_ERR_INVALID_ARG, "attend: the workspace needs %lld bytes, 256-byte aligned", (long long)pl.bytes);
    const mk_pages& g = *a->pages;
    const int eb = code_bytes(g.format), D = g.head_dim;
    uint8_t* ws = (uint8_t*)workspace;
    AttendP p = {};
    p.k = (const uint8_t*)g.k, p.v = (const uint8_t*)g.v, p.ks = g.k_scale, p.vs = g.v_scale;
    p.page_b = g.page_stride * eb, p.head_b = g.head_stride * eb, p.row_b = g.row_stride * eb;
    p.sc_page = g.scale_page_stride, p.sc_head = g.scale_head_stride;
    p.table = a->table->table, p.table_s = a->table->stride, p.pps = a->table->pages_per_seq;
    p.ps_shift = log2_exact(g.page_size), p.n_pages = g.n_pages;
    p.lens = a->lens, p.starts = a->starts, p.slopes = a->slopes;
    p.q = (const uint16_t*)a->q->data, p.qb = a->q->seq_stride, p.qt = a->q->token_stride, p.qh = a->q->head_stride;
    p.out = (uint16_t*)a->out->data, p.ob = a->out->seq_stride, p.ot = a->out->token_stride, p.oh = a->out->head_stride;
    p.lse = a->lse, p.status = a->status;
    p.B = a->table->batch, p.T = a->n_tokens, p.H = g.n_kv_heads, p.G = a->n_q_heads / g.n_kv_heads;
    p.f16 = a->q->dtype == MK_DT_F16;
    p.scale = a->scale, p.cap = a->softcap, p.shared = a->shared_len;
    p.min_units = 2;
    p.RB = pl.own_rb, p.rows_item = p.T * p.G, p.keep_items = a->shared_len > 0 || pl.wide, p.wide = pl.wide;
    p.slot_rows = pl.own_slot_rows, p.slot_floats = pl.own_floats;
    p.slots = (float*)(ws + pl.own_off), p.base = (int*)(ws + pl.base_off);
    JoinP j = {};
    j.own = p, j.own_grid = pl.own_grid, j.own_rows = pl.own_i.rows;
    const AttendFn fn = D == 64 ? attend_64 : D == 128 ? attend_128 : attend_256;
    cudaStream_t s = (cudaStream_t)stream;
    if (pl.sh_grid) {
        const long long ns = mk_wait_ns_();
        p.wait_ns = (unsigned)(ns < 4000000000ll ? ns : 4000000000ll), p.skip_signal = mk_fault_("skip_attend_signal");
        AttendP q = p;
        q.is_shared = !pl.wide;
        q.RB = pl.sh_rb, q.rows_item = pl.wide ? p.T * p.G : p.B * p.T * p.G;
        q.base = (int*)(ws + pl.sh_base_off);
        q.slot_rows = pl.sh_slot_rows, q.slot_floats = pl.sh_floats, q.slots = (float*)(ws + pl.sh_off);
        j.shared = q, j.shared_grid = pl.sh_grid, j.shared_rows = pl.sh_i.rows;
        j.shared_units = (a->shared_len + pl.sh_i.tile - 1) / pl.sh_i.tile;
        if (const int rc = pl.prefix ? (p.f16 ? prefix_f16 : prefix_bf16)(D, g.format, &q, pl.sh_grid, s)
                                     : fn(pl.sh_k, &q, nullptr, pl.sh_grid, false, s))
            return rc;
    }
    p.cluster = pl.cluster;
    if (const int rc = fn(pl.own_k, &p, nullptr, pl.own_grid, pl.sh_grid > 0, s)) return rc;
    if (pl.cluster) return MK_OK;
    j.rows = (unsigned)((int64_t)p.B * p.T * a->n_q_heads);
    j.pieces = pl.own_grid / (p.B * p.H * pl.own_rb) + 1;
    if (pl.sh_grid) j.pieces += pl.sh_grid / (p.H * pl.sh_rb * (pl.wide ? p.B : 1)) + 1;
    return D == 64 ? join_64(j, s) : D == 128 ? join_128(j, s) : join_256(j, s);
}
