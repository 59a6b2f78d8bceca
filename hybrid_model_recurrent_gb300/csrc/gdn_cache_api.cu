// gdn_cache_api.cu - host side of gdn_cache.h: argument checks, plans and launches on the caller's stream.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "../../include/gdn_cache.h"
#include "gdn_cache.cuh"

#define GDN_EXPORT extern "C" __attribute__((visibility("default")))

namespace gdn {
// gdn_api.cu
uint64_t wait_limit_ns();
int32_t stall_after();
}  // namespace gdn

namespace {

using namespace gdn::cache;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool supported_d(int d) { return d == 32 || d == 64 || d == 128; }
bool known_dtype(gdn_dtype t) { return t == GDN_F32 || t == GDN_BF16; }
int64_t es(gdn_dtype t) { return t == GDN_BF16 ? 2 : 4; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
gdn_status launched(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

gdn_status check_ws(const void* ws, size_t bytes) {
    return ws && bytes >= gdn_workspace_size() && aligned(ws, 16) ? GDN_OK : GDN_ERR_INVALID_ARG;
}

// A stream of rows of `width` elements: its stride, packed where 0.
gdn_status check_stride(int64_t& s, int64_t width, gdn_dtype t) {
    if (s == 0) s = width;
    if (s < width || s % (16 / es(t))) return GDN_ERR_INVALID_ARG;
    return s < (1ll << 36) ? GDN_OK : GDN_ERR_UNSUPPORTED;
}

gdn_status check_cache(const gdn_cache* c, bool refs) {
    if (!c || c->num_layers < 1 || c->num_pages < 1 || c->num_kv_heads < 1 || c->num_rows < 1 || c->row_pages < 1)
        return GDN_ERR_INVALID_ARG;
    if (!c->pages || !c->scales || !c->table || !c->lens || (refs && !c->refs)) return GDN_ERR_INVALID_ARG;
    if (!aligned(c->pages, 16) || !aligned(c->scales, 4) || !aligned(c->table, 4) || !aligned(c->lens, 4) || !aligned(c->refs, 4))
        return GDN_ERR_INVALID_ARG;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) return GDN_ERR_UNSUPPORTED;
    if (!supported_d(c->head_dim) || c->num_kv_heads > 4096) return GDN_ERR_UNSUPPORTED;
    if ((int64_t)c->row_pages * c->page_size >= (1ll << 31) - 512 || c->num_pages >= (1 << 30)) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

int log2i(int x) {
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

int64_t layer_scales(const gdn_cache* c) { return (int64_t)c->num_pages * 2 * c->num_kv_heads; }

Cache cache_of(const gdn_cache* c, int layer) {
    Cache x{};
    x.scales = c->scales + layer * layer_scales(c);
    x.pages = static_cast<unsigned char*>(c->pages) + layer * layer_scales(c) * c->page_size * c->head_dim;
    x.table = c->table, x.lens = c->lens;
    x.N = c->num_pages, x.page = c->page_size, x.page_log2 = log2i(c->page_size);
    x.Hkv = c->num_kv_heads, x.R = c->num_rows, x.W = c->row_pages;
    return x;
}

gdn_status check_batch(const gdn_cache* c, const gdn_batch* b, Batch& t) {
    if (!b || b->num_requests < 1 || b->max_new < 1 || b->num_tokens < 0 || b->max_len < 0) return GDN_ERR_INVALID_ARG;
    if (!b->cu_new || !aligned(b->cu_new, 4) || !aligned(b->rows, 4) || (!b->rows && b->num_requests > c->num_rows))
        return GDN_ERR_INVALID_ARG;
    if (b->num_requests > kMaxBatch || b->num_tokens >= (1ll << 30) || b->max_new >= (1 << 30)) return GDN_ERR_UNSUPPORTED;
    t.cu = b->cu_new, t.rows = b->rows, t.B = b->num_requests, t.T = (int32_t)b->num_tokens;
    t.max_new = (int32_t)std::min<int64_t>(b->max_new, std::max<int64_t>(b->num_tokens, 1));
    const int64_t cap = (int64_t)c->row_pages * c->page_size;
    t.max_len = (int32_t)(b->max_len ? std::min(b->max_len, cap) : cap);
    return GDN_OK;
}

// ---- attention ----------------------------------------------------------------------------------------------------

struct PagedPlan {
    bool tc, join;
    int tiles, ctas;   // row tiles of 16 a CTA (without tensor cores of the 5th generation); CTAs
    int tile_rows;
    int min_rows, max_rows;
    size_t ml_off, o_off, total;
};

// The launches for requests with rows in min_rows .. max_rows.
gdn_status plan_rows(const gdn_cache* c, const Batch& t, gdn_dtype dtype, int G, int64_t min_rows, int64_t max_rows, PagedPlan& pl) {
    const int64_t rows = std::min(t.max_new * (int64_t)G, max_rows);
    pl.min_rows = (int)min_rows, pl.max_rows = (int)max_rows;
    // The tensor cores of the 5th generation take 256 rows a tile, filled or not, warp-level products 16 or 32.  Measured, us, warp-level /
    // tensor cores: 16 requests x 4 heads on 8192 tokens 42 / 57 at 16 rows a head, 63 / 58 at 24, 93 / 60 at 40, 169 / 66 at 128; 4 x 8
    // heads on 30000 59 / 90, 87 / 90, - , 264 / 102; 1 x 2 heads on 100000 40 / 41, 48 / 41, 64 / 43, 84 / 44.
    pl.tc = dtype == GDN_BF16 && c->head_dim >= 64 && rows > 16;
    // Warp-level products: rows beyond 16 take tiles of 32, which halve the reads; the second tile of 16 costs a third of the warps at
    // once (in bf16, where both were possible: 16 x 4 heads at 24 rows 63 us against 65, 4 x 8 heads 87 against 94).
    pl.tiles = rows > 16 ? 2 : 1;
    pl.tile_rows = pl.tc ? kTcRows : 16 * pl.tiles;
    const int unit = pl.tc ? kTcUnit : kUnit;
    const int64_t per_item = std::max<int64_t>(ceil_div(t.max_len, unit), 1) + kLead;
    const int64_t items =
        std::min(t.B * ceil_div(rows, pl.tile_rows), ceil_div((int64_t)t.T * G, pl.tile_rows) + t.B) * c->num_kv_heads;
    if (items > kMostUnits / per_item) return GDN_ERR_UNSUPPORTED;
    const int per_sm = pl.tc ? 1 : pl.tiles == 1 ? 3 : 2;
    pl.ctas = (int)std::max<int64_t>(1, std::min<int64_t>(items * per_item, (int64_t)kSms * per_sm));
    pl.join = t.max_len > unit && pl.ctas > 1;
    pl.ml_off = (size_t)pl.ctas * sizeof(Cut);
    pl.o_off = pl.ml_off + (size_t)2 * pl.ctas * pl.tile_rows * 8;
    pl.total = pl.o_off + (size_t)2 * pl.ctas * pl.tile_rows * c->head_dim * 4;
    return GDN_OK;
}

// One plan, or two: where the average request has at most a quarter of the longest one's new tokens (a prompt among single tokens),
// those with 16 rows at most go ahead by themselves, for tiles of 256 rows cost them two to four times as much; the other two launches
// cost 8 to 20 us, as 4096 units of 128 tokens do.  Measured, us, one plan / two: 255 single tokens on 2000 x 4 heads of 64 and a prompt of
// 2000 278 / 159; 63 on 4096 x 8 heads of 128 and one of 8192 677 / 572; on 4000 x 4 heads of 128 with one of 300 new tokens 134 / 95 for 64
// requests (8192 units), 81 / 73 for 32, 54 / 62 for 16.
gdn_status plan_paged(const gdn_cache* c, const Batch& t, gdn_dtype dtype, int Hq, PagedPlan (&pl)[2], int& plans, size_t& bytes) {
    const int G = Hq / c->num_kv_heads;
    const int64_t rows = t.max_new * (int64_t)G, most = (1ll << 31) - 1024;
    if (rows >= most) return GDN_ERR_UNSUPPORTED;
    plans = 1;
    const gdn_status st = plan_rows(c, t, dtype, G, 0, most, pl[0]);
    if (st != GDN_OK) return st;
    bytes = pl[0].total;
    if (pl[0].tc && G <= 16 && (int64_t)t.B * t.max_new >= 4ll * t.T &&
        t.B * ceil_div(t.max_len, kTcUnit) * c->num_kv_heads >= 4096 && plan_rows(c, t, dtype, G, 0, 16, pl[1]) == GDN_OK) {
        std::swap(pl[0], pl[1]);
        pl[1].min_rows = 17;
        plans = 2, bytes = std::max(bytes, pl[0].total);   // (one after the other)
    }
    return GDN_OK;
}

gdn_status check_heads(const gdn_cache* c, gdn_dtype dtype, int Hq) {
    if (!known_dtype(dtype) || Hq < 1 || Hq % c->num_kv_heads) return GDN_ERR_INVALID_ARG;
    return Hq / c->num_kv_heads <= 128 && Hq <= (1 << 16) ? GDN_OK : GDN_ERR_UNSUPPORTED;
}

// ---- upkeep ---------------------------------------------------------------------------------------------------------

// scratch: the number of copies, then three lists of N pages
size_t upkeep_bytes(const gdn_cache* c) { return 16 + (size_t)3 * c->num_pages * 4; }

gdn_status upkeep_params(const gdn_cache* c, void* scratch, size_t scratch_bytes, void* ws, size_t ws_bytes, UpkeepParams& p) {
    const gdn_status st = check_cache(c, true);
    if (st != GDN_OK) return st;
    if (c->num_rows > kMaxRows) return GDN_ERR_UNSUPPORTED;
    if (check_ws(ws, ws_bytes) != GDN_OK) return GDN_ERR_INVALID_ARG;
    if (!scratch || !aligned(scratch, 16) || scratch_bytes < upkeep_bytes(c)) return GDN_ERR_INVALID_ARG;
    p.table = c->table, p.lens = c->lens, p.refs = c->refs;
    p.N = c->num_pages, p.R = c->num_rows, p.W = c->row_pages, p.page = c->page_size, p.page_log2 = log2i(c->page_size);
    p.n_copies = static_cast<int32_t*>(scratch);
    p.free_list = p.n_copies + 4;
    p.copy_from = p.free_list + c->num_pages;
    p.copy_to = p.copy_from + c->num_pages;
    p.pages = static_cast<unsigned char*>(c->pages), p.scales = c->scales;
    p.page_scales = 2 * c->num_kv_heads;
    p.page_bytes = (int64_t)p.page_scales * c->page_size * c->head_dim;
    p.layer_bytes = p.page_bytes * c->num_pages, p.layer_scales = layer_scales(c);
    p.L = c->num_layers;
    p.status = static_cast<unsigned int*>(ws);
    return GDN_OK;
}

}  // namespace

GDN_EXPORT gdn_status gdn_qk_norm_rope(const gdn_rope_problem* f, const void* q, const void* k, const int32_t* positions,
                                       const double* inv_freq, const void* q_weight, const void* k_weight, void* q_out,
                                       void* k_out, gdn_stream_t stream) {
    if (!f || f->num_tokens < 0 || f->num_q_heads < 1 || f->num_k_heads < 0 || f->rotary_dim < 0 || !known_dtype(f->dtype))
        return GDN_ERR_INVALID_ARG;
    if (f->layout != GDN_ROPE_HALF && f->layout != GDN_ROPE_INTERLEAVED) return GDN_ERR_INVALID_ARG;
    if (!(f->eps >= 0.f) || !std::isfinite(f->eps) || !std::isfinite(f->mscale)) return GDN_ERR_INVALID_ARG;
    if (!supported_d(f->head_dim)) return GDN_ERR_UNSUPPORTED;
    if (f->rotary_dim > f->head_dim || f->rotary_dim % 16) return GDN_ERR_INVALID_ARG;
    if (f->num_q_heads > (1 << 16) || f->num_k_heads > (1 << 16) || f->num_tokens >= (1ll << 31)) return GDN_ERR_UNSUPPORTED;
    RopeParams p{};
    p.q_stride = f->q_stride, p.k_stride = f->k_stride, p.qo_stride = f->q_out_stride, p.ko_stride = f->k_out_stride;
    const int64_t qw = (int64_t)f->num_q_heads * f->head_dim, kw = (int64_t)f->num_k_heads * f->head_dim;
    gdn_status st;
    if ((st = check_stride(p.q_stride, qw, f->dtype)) != GDN_OK || (st = check_stride(p.qo_stride, qw, f->dtype)) != GDN_OK)
        return st;
    if (f->num_k_heads > 0 && ((st = check_stride(p.k_stride, kw, f->dtype)) != GDN_OK ||
                               (st = check_stride(p.ko_stride, kw, f->dtype)) != GDN_OK))
        return st;
    for (const void* x : {q_weight, k_weight})
        if (!aligned(x, 16)) return GDN_ERR_INVALID_ARG;
    if (f->num_tokens == 0) return GDN_OK;
    if (!q || !q_out || !aligned(q, 16) || !aligned(q_out, 16)) return GDN_ERR_INVALID_ARG;
    if (f->num_k_heads > 0 && (!k || !k_out || !aligned(k, 16) || !aligned(k_out, 16))) return GDN_ERR_INVALID_ARG;
    if (f->rotary_dim > 0 && (!positions || !inv_freq || !aligned(positions, 4) || !aligned(inv_freq, 8)))
        return GDN_ERR_INVALID_ARG;
    // in place: the same rows
    if ((q_out == q && p.qo_stride != p.q_stride) || (k && k_out == k && p.ko_stride != p.k_stride)) return GDN_ERR_INVALID_ARG;
    p.q = q, p.k = k, p.q_out = q_out, p.k_out = k_out;
    p.positions = positions, p.inv_freq = inv_freq, p.qw = q_weight, p.kw = k_weight;
    p.T = f->num_tokens, p.Hq = f->num_q_heads, p.Hk = f->num_k_heads, p.rd = f->rotary_dim;
    p.normalize = f->normalize != 0, p.eps = f->eps, p.mscale = f->mscale;
    // A token's heads go to one warp, whose sines then serve them all, unless there are too few tokens to fill the GPU.
    const bool bf16 = f->dtype == GDN_BF16;
    const int passes = rope_passes(p.Hq, p.Hk, f->head_dim, bf16);
    const int64_t wanted = (int64_t)kSms * 16;
    p.parts = (int)std::min<int64_t>(passes, std::max<int64_t>(1, wanted / p.T));
    p.per_part = (int)ceil_div(passes, p.parts);
    p.parts = (int)ceil_div(passes, p.per_part);
    return launched(launch_rope(p, f->head_dim, bf16, f->layout == GDN_ROPE_HALF, (cudaStream_t)stream));
}

GDN_EXPORT gdn_status gdn_cache_append(const gdn_cache* c, int32_t layer, const gdn_batch* b, const void* k, const void* v,
                                       gdn_dtype dtype, int64_t k_stride, int64_t v_stride, void* workspace, size_t ws_bytes,
                                       gdn_stream_t stream) {
    gdn_status st = check_cache(c, false);
    if (st != GDN_OK) return st;
    AppendParams p{};
    if ((st = check_batch(c, b, p.t)) != GDN_OK) return st;
    if (layer < 0 || layer >= c->num_layers || !known_dtype(dtype)) return GDN_ERR_INVALID_ARG;
    if ((st = check_ws(workspace, ws_bytes)) != GDN_OK) return st;
    const int64_t width = (int64_t)c->num_kv_heads * c->head_dim;
    p.k_stride = k_stride, p.v_stride = v_stride;
    if ((st = check_stride(p.k_stride, width, dtype)) != GDN_OK || (st = check_stride(p.v_stride, width, dtype)) != GDN_OK) return st;
    if (p.t.T == 0) return GDN_OK;
    if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return GDN_ERR_INVALID_ARG;
    if (ceil_div(p.t.max_new, c->page_size) * 2 * c->num_kv_heads >= (1ll << 30)) return GDN_ERR_UNSUPPORTED;
    p.c = cache_of(c, layer);
    p.t.max_len = c->row_pages * c->page_size;   // (a bound that is too low would move tokens)
    p.k = k, p.v = v;
    p.status = static_cast<unsigned int*>(workspace);
    return launched(launch_append(p, c->head_dim, dtype == GDN_BF16, (cudaStream_t)stream));
}

GDN_EXPORT size_t gdn_paged_scratch_bytes(const gdn_cache* c, const gdn_batch* b, gdn_dtype dtype, int32_t num_q_heads) {
    Batch t{};
    PagedPlan pl[2];
    int plans;
    size_t bytes;
    if (check_cache(c, false) != GDN_OK || check_batch(c, b, t) != GDN_OK || check_heads(c, dtype, num_q_heads) != GDN_OK ||
        plan_paged(c, t, dtype, num_q_heads, pl, plans, bytes) != GDN_OK)
        return 0;
    return bytes;
}

GDN_EXPORT gdn_status gdn_paged_attention(const gdn_cache* c, int32_t layer, const gdn_batch* b, const void* q, gdn_dtype dtype,
                                          int32_t num_q_heads, int64_t q_stride, float softmax_scale, void* o, float* lse,
                                          void* scratch, size_t scratch_bytes, void* workspace, size_t ws_bytes,
                                          gdn_stream_t stream) {
    gdn_status st = check_cache(c, false);
    if (st != GDN_OK) return st;
    PagedParams p{};
    if ((st = check_batch(c, b, p.t)) != GDN_OK || (st = check_heads(c, dtype, num_q_heads)) != GDN_OK) return st;
    if (layer < 0 || layer >= c->num_layers) return GDN_ERR_INVALID_ARG;
    if ((st = check_ws(workspace, ws_bytes)) != GDN_OK) return st;
    p.scale_log2 = (float)((double)softmax_scale * 1.4426950408889634);
    if (!std::isfinite(p.scale_log2)) return GDN_ERR_INVALID_ARG;
    p.q_stride = q_stride;
    if ((st = check_stride(p.q_stride, (int64_t)num_q_heads * c->head_dim, dtype)) != GDN_OK) return st;
    PagedPlan plan[2];
    int plans;
    size_t bytes;
    if ((st = plan_paged(c, p.t, dtype, num_q_heads, plan, plans, bytes)) != GDN_OK) return st;
    if (!scratch || !aligned(scratch, 32) || scratch_bytes < bytes || !aligned(lse, 4)) return GDN_ERR_INVALID_ARG;
    if (p.t.T == 0) return GDN_OK;
    if (!q || !o || !aligned(q, 16) || !aligned(o, 16)) return GDN_ERR_INVALID_ARG;
    p.c = cache_of(c, layer);
    p.q = q, p.o = o, p.lse = lse;
    unsigned char* sc = static_cast<unsigned char*>(scratch);
    p.cuts = reinterpret_cast<Cut*>(sc);
    p.status = static_cast<unsigned int*>(workspace);
    p.Hq = num_q_heads, p.G = num_q_heads / c->num_kv_heads;
    p.wait_limit_ns = gdn::wait_limit_ns();
    p.stall_after = gdn::stall_after();
    const bool bf16 = dtype == GDN_BF16;
    const cudaStream_t s = (cudaStream_t)stream;
    for (int i = 0; st == GDN_OK && i < plans; ++i) {
        const PagedPlan& pl = plan[i];
        p.part_ml = reinterpret_cast<float2*>(sc + pl.ml_off), p.part_o = reinterpret_cast<float*>(sc + pl.o_off);
        p.ctas = pl.ctas, p.min_rows = pl.min_rows, p.max_rows = pl.max_rows;
        st = launched(pl.tc ? launch_paged_tc(p, c->head_dim, s) : launch_paged(p, c->head_dim, bf16, pl.tiles, s));
        if (st == GDN_OK && pl.join) st = launched(launch_paged_join(p, c->head_dim, bf16, pl.tile_rows, s));
    }
    return st;
}

GDN_EXPORT size_t gdn_cache_scratch_bytes(const gdn_cache* c) { return check_cache(c, true) == GDN_OK ? upkeep_bytes(c) : 0; }

GDN_EXPORT gdn_status gdn_cache_update(const gdn_cache* c, int32_t num_drop, const int32_t* drop, int32_t num_fork,
                                       const int32_t* fork_from, const int32_t* fork_to, const int32_t* grow, int32_t* granted,
                                       void* scratch, size_t scratch_bytes, void* workspace, size_t ws_bytes,
                                       gdn_stream_t stream) {
    UpkeepParams p{};
    const gdn_status st = upkeep_params(c, scratch, scratch_bytes, workspace, ws_bytes, p);
    if (st != GDN_OK) return st;
    if (num_drop < 0 || num_fork < 0 || (num_drop > 0 && !drop) || (num_fork > 0 && (!fork_from || !fork_to)))
        return GDN_ERR_INVALID_ARG;
    for (const void* x : {(const void*)drop, (const void*)fork_from, (const void*)fork_to, (const void*)grow, (const void*)granted})
        if (!aligned(x, 4)) return GDN_ERR_INVALID_ARG;
    if (num_drop > (1 << 24) || num_fork > (1 << 24)) return GDN_ERR_UNSUPPORTED;
    p.n_drop = num_drop, p.drop = drop, p.n_fork = num_fork, p.from = fork_from, p.to = fork_to;
    p.grow = grow, p.granted = granted;
    if (num_drop == 0 && num_fork == 0 && !grow) return GDN_OK;
    return launched(launch_update(p, (cudaStream_t)stream));
}

GDN_EXPORT gdn_status gdn_cache_compact(const gdn_cache* c, int32_t* live, void* scratch, size_t scratch_bytes, void* workspace,
                                        size_t ws_bytes, gdn_stream_t stream) {
    UpkeepParams p{};
    const gdn_status st = upkeep_params(c, scratch, scratch_bytes, workspace, ws_bytes, p);
    if (st != GDN_OK) return st;
    if (!live || !aligned(live, 4)) return GDN_ERR_INVALID_ARG;
    p.live = live;
    return launched(launch_compact(p, (cudaStream_t)stream));
}
