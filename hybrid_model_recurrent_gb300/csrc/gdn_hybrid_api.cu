// gdn_hybrid_api.cu - host side of gdn_hybrid.h: argument checks, job tables, the split of few long scans and of
// the prefix, and launches on the caller's stream.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <memory>
#include <vector>

#include "../../include/gdn_hybrid.h"
#include "gdn_linear.cuh"
#include "gdn_prefix.cuh"

#define GDN_EXPORT extern "C" __attribute__((visibility("default")))

namespace gdn {
// gdn_api.cu
uint64_t wait_limit_ns();
int32_t stall_after();
void* encode_tiled_fn();
}  // namespace gdn

namespace {

constexpr int kSms = gdn::prefix::kSms;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool supported_d(int d) { return d == 32 || d == 64 || d == 128; }
bool known_dtype(gdn_dtype t) { return t == GDN_F32 || t == GDN_BF16; }
int64_t es(gdn_dtype t) { return t == GDN_BF16 ? 2 : 4; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

gdn_status check_ws(const void* ws, size_t bytes) {
    return ws && bytes >= gdn_workspace_size() && aligned(ws, 16) ? GDN_OK : GDN_ERR_INVALID_ARG;
}

// No exception leaves a C entry point: running out of host memory is reported as GDN_ERR_CUDA.
template <class F>
gdn_status guarded(F&& f) {
    try {
        return f();
    } catch (...) {
        return GDN_ERR_CUDA;
    }
}

// ---- linear attention -----------------------------------------------------------------

struct LinStrides {
    int64_t q, k, v;
};

gdn_status check_linear(const gdn_linear_problem* p, LinStrides& s) {
    if (!p || p->num_seqs < 1 || p->num_heads < 1 || p->num_qk_heads < 1 || p->d_k < 1 || p->d_v < 1)
        return GDN_ERR_INVALID_ARG;
    if (p->num_heads % p->num_qk_heads) return GDN_ERR_INVALID_ARG;
    if (!known_dtype(p->qkv_dtype) || !known_dtype(p->out_dtype) || !std::isfinite(p->scale)) return GDN_ERR_INVALID_ARG;
    if (!supported_d(p->d_k) || !supported_d(p->d_v)) return GDN_ERR_UNSUPPORTED;
    if (p->num_heads > (1 << 16)) return GDN_ERR_UNSUPPORTED;
    const int64_t qk = (int64_t)p->num_qk_heads * p->d_k, vv = (int64_t)p->num_heads * p->d_v;
    s = {p->q_stride ? p->q_stride : qk, p->k_stride ? p->k_stride : qk, p->v_stride ? p->v_stride : vv};
    const int64_t e = 16 / es(p->qkv_dtype);
    if (s.q < qk || s.k < qk || s.v < vv || s.q % e || s.k % e || s.v % e) return GDN_ERR_INVALID_ARG;
    if (s.q >= (1ll << 36) || s.k >= (1ll << 36) || s.v >= (1ll << 36)) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

gdn_status check_lengths(const gdn_linear_problem* p) {
    if (!p->cu_seqlens || p->cu_seqlens[0] != 0) return GDN_ERR_INVALID_ARG;
    for (int b = 0; b < p->num_seqs; ++b)
        if (p->cu_seqlens[b + 1] < p->cu_seqlens[b]) return GDN_ERR_INVALID_ARG;
    if (p->cu_seqlens[p->num_seqs] >= (1ll << 31) - 256) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

// How a prefill's scans are cut.  seg_len 0: one job a sequence.
struct LinPlan {
    bool tc;            // the tensor-core kernel
    int rows_per_cta;   // state rows of a CTA
    int64_t seg_len;
    int64_t slots;   // states of all segments but the last of each sequence
};

LinPlan plan_linear(const gdn_linear_problem* p) {
    LinPlan pl{};
    const int B = p->num_seqs;
    const int64_t T = p->cu_seqlens[B];
    int64_t longest = 0;
    for (int b = 0; b < B; ++b) longest = std::max(longest, p->cu_seqlens[b + 1] - p->cu_seqlens[b]);
    // The tensor-core kernel rounds the readout's operands to bf16, which a bf16 output hides and an fp32 one does not.
    pl.tc = p->d_k >= 64 && p->d_v >= 64 && p->qkv_dtype == GDN_BF16 && p->out_dtype == GDN_BF16;
    // FP32 pipes: CTAs of 64 state rows when that still gives two a multiprocessor, else smaller ones
    pl.rows_per_cta = pl.tc ? p->d_v : std::min(64, p->d_v);
    while (!pl.tc && pl.rows_per_cta > 16 && (int64_t)B * p->num_heads * (p->d_v / pl.rows_per_cta) < 2 * kSms) pl.rows_per_cta /= 2;
    const int64_t per_seq = (int64_t)p->num_heads * (p->d_v / pl.rows_per_cta);
    // A scan is sequential, so a call with few long ones leaves multiprocessors idle.  Its scans may then be cut into
    // segments: each segment's own state from zero (keys and values read once more), the chain of the states, and all
    // segments side by side.  Both ways are estimated, in us, from what was measured: a token's time in a CTA with a readout
    // and without, a CTA's start, the chain's time a segment, two more launches, five passes of memory over the segments'
    // states; the FP32 pipes' CTAs are small and run four to a multiprocessor.  At d = 128 in bf16, 8192 tokens, 16 / 32 / 48
    // / 64 heads took 55 / 92 / 121 / 162 us cut and 190 whole, 1024 tokens of 16 heads 34 cut and 30 whole; in fp32, 4096
    // tokens of 32 heads of 64 x 64 205 us cut and 456 whole.
    const double read = pl.tc ? 0.026 : 0.1, update = pl.tc ? 0.014 : 0.06, start = 6, link = 0.8;
    const int64_t slots = kSms * (pl.tc ? 1 : 4), share = ceil_div(T * per_seq, slots);
    double best = (double)std::max(longest, share) * read + start;
    auto segments = [&](int64_t len) {   // of all scans
        int64_t n = 0;
        for (int b = 0; b < B; ++b) n += ceil_div(p->cu_seqlens[b + 1] - p->cu_seqlens[b], len);
        return n;
    };
    for (int waves = 1; waves <= 4 && (double)share * (read + update) < best; ++waves) {
        // the shortest segments that all run in `waves` waves, if about the even share's length will do
        const int64_t even = ceil_div(std::max<int64_t>(256, ceil_div(share, waves)), 128) * 128;
        int64_t len = even, n = segments(len);
        for (int i = 0; i < 10 && n * per_seq > waves * slots; ++i) len += ceil_div(len, 2048) * 128, n = segments(len);
        if (n * per_seq > waves * slots) len = even, n = segments(len);
        if (len >= longest) continue;
        const int64_t tokens = std::min(ceil_div(n * per_seq, slots) * len, share + len);   // of the busiest CTA slot
        const double cost = (double)tokens * (read + update) + 2 * start * waves + link * (double)ceil_div(longest, len) + 6 +
                            (double)(n * p->num_heads) * p->d_v * p->d_k * 20 / 6e6;
        if (cost < 0.95 * best) best = cost, pl.seg_len = len;
    }
    if (pl.seg_len) {
        for (int b = 0; b < B; ++b) {
            const int64_t n = p->cu_seqlens[b + 1] - p->cu_seqlens[b];
            if (n > 0) pl.slots += ceil_div(n, pl.seg_len) - 1;
        }
    }
    return pl;
}

// A sequence with more checkpoints than a job holds takes several launches in a row, in a call of at most this many sequences.
// The limit is one of the call, not of the plan: how the scans are cut does not decide what is accepted.
constexpr int kLongListSeqs = 256;

struct LinHostJob {
    gdn::lin::Job job;
    std::vector<gdn::lin::Ckpt> ckpts;
    int round = 0;   // jobs of a round start from checkpoints of the round before
};

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// bf16 tensor map over `rank` dimensions (the innermost of them contiguous), boxes of 64 columns x 1 head x `tokens`
// (x 1 request), 128-byte swizzle; strides of the outer dimensions in elements
bool bf16_map(CUtensorMap* m, const void* base, int rank, const int64_t (&dim)[4], const int64_t (&stride)[3], int tokens) {
    const auto enc = reinterpret_cast<EncodeFn>(gdn::encode_tiled_fn());
    if (!enc) return false;
    cuuint64_t dims[4], strides[3];
    for (int i = 0; i < 4; ++i) dims[i] = (cuuint64_t)std::max<int64_t>(dim[i], 1);
    for (int i = 0; i < 3; ++i) strides[i] = (cuuint64_t)(stride[i] * 2);
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)tokens, 1}, one[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Batch jobs into parameter blocks, a round after the other, longest first.
template <class F>
gdn_status launch_jobs(gdn::lin::Params& prm, std::vector<LinHostJob>& jobs, F&& launch) {
    std::stable_sort(jobs.begin(), jobs.end(), [](const LinHostJob& a, const LinHostJob& b) {
        return a.round != b.round ? a.round < b.round : a.job.len > b.job.len;
    });
    size_t i = 0;
    while (i < jobs.size()) {
        int nj = 0, nc = 0;
        while (i + nj < jobs.size() && nj < gdn::lin::kMaxJobs && jobs[i + nj].round == jobs[i].round &&
               nc + (int)jobs[i + nj].ckpts.size() <= gdn::lin::kMaxCkpts) {
            gdn::lin::Job j = jobs[i + nj].job;
            j.ck_begin = nc;
            j.ck_count = (int32_t)jobs[i + nj].ckpts.size();
            for (const gdn::lin::Ckpt& c : jobs[i + nj].ckpts) prm.ckpts[nc++] = c;
            prm.jobs[nj++] = j;
        }
        prm.n_jobs = nj;
        if (launch(prm) != cudaSuccess) return GDN_ERR_CUDA;
        i += nj;
    }
    return GDN_OK;
}

gdn_status linear_prefill(const gdn_linear_problem* p, const void* q, const void* k, const void* v, const float* alpha,
                          const float* S0, const int32_t* s0_index, int64_t s0_slots, void* o, float* S_final,
                          const int64_t* ckpt_pos, const int64_t* cu_ckpt, float* ckpt_states, void* scratch,
                          size_t scratch_bytes, void* workspace, size_t ws_bytes, cudaStream_t stream) {
    LinStrides sd{};
    gdn_status st = check_linear(p, sd);
    if (st != GDN_OK) return st;
    if ((st = check_lengths(p)) != GDN_OK) return st;
    if ((st = check_ws(workspace, ws_bytes)) != GDN_OK) return st;
    const int B = p->num_seqs, H = p->num_heads;
    const int64_t T = p->cu_seqlens[B];
    if (!alpha || !aligned(alpha, 4) || !S_final || !aligned(S_final, 16)) return GDN_ERR_INVALID_ARG;
    if (T > 0) {
        if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return GDN_ERR_INVALID_ARG;
        if (o && (!q || !aligned(q, 16))) return GDN_ERR_INVALID_ARG;
    }
    if (o && !aligned(o, 16)) return GDN_ERR_INVALID_ARG;
    if (S0) {
        if (!aligned(S0, 16) || s0_slots < 0 || (!s0_index && s0_slots < B)) return GDN_ERR_INVALID_ARG;
        for (int b = 0; s0_index && b < B; ++b)
            if (s0_index[b] < -1 || s0_index[b] >= s0_slots) return GDN_ERR_INVALID_ARG;
    }
    int64_t n_ck = 0;
    if (cu_ckpt) {
        if (cu_ckpt[0] != 0) return GDN_ERR_INVALID_ARG;
        for (int b = 0; b < B; ++b)
            if (cu_ckpt[b + 1] < cu_ckpt[b]) return GDN_ERR_INVALID_ARG;
        n_ck = cu_ckpt[B];
        if (n_ck > 0 && (!ckpt_pos || !ckpt_states || !aligned(ckpt_states, 16))) return GDN_ERR_INVALID_ARG;
        for (int b = 0; b < B; ++b) {
            const int64_t n = p->cu_seqlens[b + 1] - p->cu_seqlens[b];
            for (int64_t i = cu_ckpt[b]; i < cu_ckpt[b + 1]; ++i)
                if (ckpt_pos[i] < 1 || ckpt_pos[i] > n || (i > cu_ckpt[b] && ckpt_pos[i] <= ckpt_pos[i - 1]))
                    return GDN_ERR_INVALID_ARG;
        }
        if (n_ck >= (1ll << 23)) return GDN_ERR_UNSUPPORTED;
        for (int b = 0; b < B; ++b)
            if (cu_ckpt[b + 1] - cu_ckpt[b] > gdn::lin::kMaxCkpts && B > kLongListSeqs) return GDN_ERR_UNSUPPORTED;
    }
    const LinPlan pl = plan_linear(p);
    const size_t state = (size_t)H * p->d_v * p->d_k;
    if (pl.slots > 0 && (!scratch || !aligned(scratch, 16) || scratch_bytes < (size_t)pl.slots * state * 4))
        return GDN_ERR_INVALID_ARG;
    if ((int64_t)H * (p->d_v / pl.rows_per_cta) * gdn::lin::kMaxJobs >= (1ll << 31)) return GDN_ERR_UNSUPPORTED;

    // the jobs: every sequence, or its segments; `own` the segments' own states
    std::vector<LinHostJob> jobs, own;
    std::vector<gdn::lin::Chain> chains;
    float* seg_states = static_cast<float*>(scratch);
    int64_t slot = 0;
    for (int b = 0; b < B; ++b) {
        const int64_t beg = p->cu_seqlens[b], n = p->cu_seqlens[b + 1] - beg;
        const int64_t L = pl.seg_len ? pl.seg_len : std::max<int64_t>(n, 1);
        const int64_t segs = std::max<int64_t>(ceil_div(n, L), 1);
        const int32_t from = s0_index ? s0_index[b] : b;
        const float* s0 = S0 && from >= 0 ? S0 + (size_t)from * state : nullptr;
        int64_t ck = cu_ckpt ? cu_ckpt[b] : 0;
        const int64_t ck_end = cu_ckpt ? cu_ckpt[b + 1] : 0;
        if (segs > 1) chains.push_back({s0, (int32_t)slot, (int32_t)(segs - 1)});
        for (int64_t j = 0; j < segs; ++j) {
            LinHostJob w{};
            w.job.tok_begin = beg + j * L;
            w.job.len = (int32_t)std::min(L, n - j * L);
            w.job.s0 = j == 0 ? s0 : seg_states + (size_t)(slot + j - 1) * state;
            w.job.s_final = j == segs - 1 ? S_final + (size_t)b * state : nullptr;
            if (j < segs - 1) {
                LinHostJob z{};
                z.job = w.job;
                z.job.s0 = nullptr;
                z.job.s_final = seg_states + (size_t)(slot + j) * state;
                own.push_back(std::move(z));
            }
            const int64_t end = j * L + w.job.len;
            int64_t from_pos = j * L;
            for (; ck < ck_end && ckpt_pos[ck] <= end; ++ck) {
                if (w.ckpts.size() == (size_t)gdn::lin::kMaxCkpts) {
                    // a full list: the job ends at its last checkpoint, and the next round's takes that state up
                    const int64_t cut = ckpt_pos[ck - 1];
                    LinHostJob rest{};
                    rest.job = w.job;
                    rest.job.tok_begin = beg + cut;
                    rest.job.len = (int32_t)(end - cut);
                    rest.job.s0 = ckpt_states + (size_t)(ck - 1) * state;
                    rest.round = w.round + 1;
                    w.job.len = (int32_t)(cut - from_pos);
                    w.job.s_final = nullptr;
                    jobs.push_back(std::move(w));
                    w = std::move(rest);
                    from_pos = cut;
                }
                w.ckpts.push_back({(int32_t)(ckpt_pos[ck] - from_pos), (int32_t)ck});
            }
            // without a readout a segment that ends in no wanted state has nothing to do
            if (o || w.job.s_final || !w.ckpts.empty()) jobs.push_back(std::move(w));
        }
        slot += segs - 1;
    }

    auto prm = std::make_unique<gdn::lin::Params>();
    std::memset(prm.get(), 0, sizeof(gdn::lin::Params));
    prm->q = q, prm->k = k, prm->v = v;
    prm->q_stride = sd.q, prm->k_stride = sd.k, prm->v_stride = sd.v;
    prm->alpha = alpha;
    prm->ckpt_states = ckpt_states;
    prm->status = static_cast<unsigned int*>(workspace);
    prm->wait_limit_ns = gdn::wait_limit_ns();
    prm->stall_after = gdn::stall_after();
    prm->scale = p->scale;
    prm->H = H, prm->rep = H / p->num_qk_heads;
    prm->dv = p->d_v;
    prm->rows_per_cta = pl.rows_per_cta;
    const bool in_bf16 = p->qkv_dtype == GDN_BF16, out_bf16 = p->out_dtype == GDN_BF16;
    if (pl.tc && T > 0) {
        const int Hk = p->num_qk_heads;
        bool maps = bf16_map(&prm->tm_k, k, 3, {p->d_k, Hk, T, 1}, {p->d_k, sd.k, 0}, 128) &&
                    bf16_map(&prm->tm_v, v, 3, {p->d_v, H, T, 1}, {p->d_v, sd.v, 0}, 128);
        if (maps && o)
            maps = bf16_map(&prm->tm_q, q, 3, {p->d_k, Hk, T, 1}, {p->d_k, sd.q, 0}, 128) &&
                   bf16_map(&prm->tm_o, o, 3, {p->d_v, H, T, 1}, {p->d_v, (int64_t)H * p->d_v, 0}, 128);
        if (!maps) return GDN_ERR_CUDA;
    }
    auto launch = [&](const gdn::lin::Params& pr) {
        return pl.tc ? gdn::lin::launch_tc(pr, p->d_k, stream) : gdn::lin::launch_simt(pr, p->d_k, in_bf16, out_bf16, stream);
    };
    if (!own.empty()) {
        prm->o = nullptr;
        if ((st = launch_jobs(*prm, own, launch)) != GDN_OK) return st;
        auto ch = std::make_unique<gdn::lin::ChainParams>();
        ch->states = seg_states;
        ch->alpha = alpha;
        ch->H = H, ch->state = p->d_v * p->d_k;
        ch->seg_len = (int32_t)pl.seg_len;
        for (size_t i = 0; i < chains.size(); i += gdn::lin::kMaxJobs) {
            ch->n_scans = (int32_t)std::min<size_t>(gdn::lin::kMaxJobs, chains.size() - i);
            std::copy_n(chains.begin() + i, ch->n_scans, ch->scans);
            if (gdn::lin::launch_chain(*ch, stream) != cudaSuccess) return GDN_ERR_CUDA;
        }
    }
    prm->o = o;
    return launch_jobs(*prm, jobs, launch);
}

// ---- shared-prefix attention ------------------------------------------------------------

struct PrefixPlan {
    bool tc, joined;
    int row_tiles;         // tensor cores: row tiles of a CTA
    int pre_splits, pre_chunk, tail_splits, pre_tiles, tail_tiles;
    int groups;            // groups of 32 stacked rows of a key/value head
    int64_t rows;          // query rows of all heads
    size_t ml_off, o_off, total;
    int parts() const { return pre_splits + tail_splits; }
};

// what the kernels multiply scores by: exponentials of base 2
float scale_log2(const gdn_prefix_problem& f) { return (float)((double)f.softmax_scale * 1.4426950408889634); }

gdn_status check_prefix(const gdn_prefix_problem* p, gdn_prefix_problem& f) {
    if (!p) return GDN_ERR_INVALID_ARG;
    f = *p;
    if (f.batch < 1 || f.num_queries < 1 || f.num_q_heads < 1 || f.num_kv_heads < 1 || f.head_dim < 1)
        return GDN_ERR_INVALID_ARG;
    if (f.num_q_heads % f.num_kv_heads || !known_dtype(f.dtype) || !std::isfinite(scale_log2(f)))
        return GDN_ERR_INVALID_ARG;
    if (f.prefix_len < 0 || f.tail_cap < 0 || f.max_tail < 0 || f.max_tail > f.tail_cap) return GDN_ERR_INVALID_ARG;
    if (!supported_d(f.head_dim)) return GDN_ERR_UNSUPPORTED;
    if (f.prefix_len >= (1ll << 31) - 512 || f.tail_cap >= (1ll << 31) - 512) return GDN_ERR_UNSUPPORTED;
    if (f.num_q_heads > (1 << 16) || (int64_t)f.batch * f.num_queries * f.num_q_heads >= (1ll << 31) - 512)
        return GDN_ERR_UNSUPPORTED;
    const int64_t D = f.head_dim, e = 16 / es(f.dtype);
    auto fill = [](int64_t& s, int64_t packed) { if (s == 0) s = packed; };
    fill(f.q_stride_h, D), fill(f.q_stride_n, D * f.num_q_heads), fill(f.q_stride_b, D * f.num_q_heads * f.num_queries);
    fill(f.kp_stride_h, D), fill(f.kp_stride_t, D * f.num_kv_heads);
    fill(f.vp_stride_h, D), fill(f.vp_stride_t, D * f.num_kv_heads);
    const int64_t cap = std::max<int64_t>(f.tail_cap, 1);
    fill(f.kt_stride_h, D), fill(f.kt_stride_t, D * f.num_kv_heads), fill(f.kt_stride_b, D * f.num_kv_heads * cap);
    fill(f.vt_stride_h, D), fill(f.vt_stride_t, D * f.num_kv_heads), fill(f.vt_stride_b, D * f.num_kv_heads * cap);
    for (int64_t s : {f.q_stride_b, f.q_stride_n, f.q_stride_h, f.kp_stride_t, f.kp_stride_h, f.vp_stride_t, f.vp_stride_h,
                      f.kt_stride_b, f.kt_stride_t, f.kt_stride_h, f.vt_stride_b, f.vt_stride_t, f.vt_stride_h}) {
        if (s < 0 || s % e) return GDN_ERR_INVALID_ARG;
        if (s >= (1ll << 36)) return GDN_ERR_UNSUPPORTED;
    }
    return GDN_OK;
}

// In how many ranges to cut `tiles` tiles of tokens that `items` row tiles take, with `slots` CTAs at once: the fewest
// tile times, counting whole waves, two tile times for a CTA's start and end, and the join's reading and writing of
// each range's partial sums (at about 10 TB/s from L2, against a tile time of about 1.2 us).
int best_splits(int64_t tiles, int64_t items, int64_t slots, int64_t part_bytes) {
    int64_t best = 1;
    double best_cost = 1e300;
    for (int64_t s = 1; s <= std::min<int64_t>(tiles, 256); ++s) {
        const int64_t per = ceil_div(tiles, s);
        if (ceil_div(tiles, per) != s) continue;   // the same ranges as fewer splits
        const double cost = (double)ceil_div(items * s, slots) * (double)(per + 2) + (double)(s * part_bytes) / 1.2e7;
        if (cost < best_cost) best_cost = cost, best = s;
    }
    return (int)best;
}

PrefixPlan plan_prefix(const gdn_prefix_problem& f) {
    PrefixPlan pl{};
    pl.rows = (int64_t)f.batch * f.num_queries * f.num_q_heads;
    const int64_t group = f.num_q_heads / f.num_kv_heads, own = f.num_queries * group, stacked = own * f.batch;
    pl.groups = (int)ceil_div(stacked, 32);
    pl.tc = f.dtype == GDN_BF16 && f.head_dim >= 64;
    const int64_t part_bytes = pl.rows * (f.head_dim * 4 + 8) * 2;
    int64_t unit;   // tokens of a tile
    int64_t slots;
    if (pl.tc) {
        unit = gdn::prefix::kTcKeys;
        // A request with a whole row tile of its own needs no stacking: when such tiles fill the GPU, each takes prefix
        // and tail in one go and writes its rows itself.
        const int64_t pairs = ceil_div(own, 2 * gdn::prefix::kTcRows);
        if (own > gdn::prefix::kTcRows && f.batch * f.num_kv_heads * pairs >= kSms && f.prefix_len + f.max_tail > 0) {
            pl.joined = true;
            pl.row_tiles = 2;
            pl.tail_tiles = (int)pairs;
            pl.tail_splits = 1;
            return pl;
        }
        // Two row tiles a CTA halve the reads of the prefix when more than one is stacked; one leaves room for two CTAs.
        pl.row_tiles = std::max(f.prefix_len > 0 ? stacked : 0, own) > gdn::prefix::kTcRows ? 2 : 1;
        pl.pre_tiles = (int)ceil_div(stacked, pl.row_tiles * gdn::prefix::kTcRows);
        pl.tail_tiles = (int)ceil_div(own, pl.row_tiles * gdn::prefix::kTcRows);
        slots = kSms * (3 - pl.row_tiles);
    } else {
        unit = gdn::prefix::kSimtKeys;
        pl.pre_tiles = (int)ceil_div(stacked, gdn::prefix::kSimtRows);
        pl.tail_tiles = (int)ceil_div(own, gdn::prefix::kSimtRows);
        slots = kSms * 5;   // CTAs that 43 KB of shared memory let run at once
    }
    if (f.prefix_len > 0) {
        const int64_t tiles = ceil_div(f.prefix_len, unit);
        const int s = best_splits(tiles, (int64_t)f.num_kv_heads * pl.pre_tiles, slots, part_bytes);
        pl.pre_chunk = (int)(ceil_div(tiles, s) * unit);
        pl.pre_splits = (int)ceil_div(f.prefix_len, pl.pre_chunk);
    }
    if (f.max_tail > 0)
        pl.tail_splits = best_splits(ceil_div(f.max_tail, unit), (int64_t)f.batch * f.num_kv_heads * pl.tail_tiles,
                                     slots, part_bytes);
    const int64_t parts = pl.parts();
    if (parts == 0 || (pl.tc && parts == 1)) return pl;
    pl.ml_off = 0;
    const int64_t rows = parts * f.num_kv_heads * pl.groups * 32;   // groups of 32 stacked rows
    pl.o_off = (size_t)rows * 8;
    pl.total = pl.o_off + (size_t)rows * f.head_dim * 4;
    return pl;
}

gdn_status prefix_attention(const gdn_prefix_problem* p, const void* q, const void* k_prefix, const void* v_prefix,
                            const void* k_tail, const void* v_tail, const int32_t* tail_len, void* o, float* lse,
                            void* scratch, size_t scratch_bytes, void* workspace, size_t ws_bytes, cudaStream_t stream) {
    gdn_prefix_problem f;
    gdn_status st = check_prefix(p, f);
    if (st != GDN_OK) return st;
    if ((st = check_ws(workspace, ws_bytes)) != GDN_OK) return st;
    if (!q || !o || !aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4)) return GDN_ERR_INVALID_ARG;
    if (f.prefix_len > 0 && (!k_prefix || !v_prefix || !aligned(k_prefix, 16) || !aligned(v_prefix, 16)))
        return GDN_ERR_INVALID_ARG;
    if (f.max_tail > 0 && (!k_tail || !v_tail || !tail_len || !aligned(k_tail, 16) || !aligned(v_tail, 16) ||
                           !aligned(tail_len, 4)))
        return GDN_ERR_INVALID_ARG;
    const PrefixPlan pl = plan_prefix(f);
    if (pl.total > 0 && (!scratch || !aligned(scratch, 32) || scratch_bytes < pl.total)) return GDN_ERR_INVALID_ARG;
    const int64_t items = f.num_kv_heads * ((int64_t)pl.pre_splits * pl.pre_tiles + (int64_t)pl.tail_splits * pl.tail_tiles * f.batch);
    if (items >= (1ll << 31) || (int64_t)f.num_kv_heads * pl.groups * (f.head_dim / 8) >= (1ll << 31))
        return GDN_ERR_UNSUPPORTED;

    auto prm = std::make_unique<gdn::prefix::Params>();
    std::memset(prm.get(), 0, sizeof(gdn::prefix::Params));
    prm->q = q, prm->kp = k_prefix, prm->vp = v_prefix, prm->kt = k_tail, prm->vt = v_tail;
    prm->q_sb = f.q_stride_b, prm->q_sn = f.q_stride_n, prm->q_sh = f.q_stride_h;
    prm->kp_st = f.kp_stride_t, prm->kp_sh = f.kp_stride_h, prm->vp_st = f.vp_stride_t, prm->vp_sh = f.vp_stride_h;
    prm->kt_sb = f.kt_stride_b, prm->kt_st = f.kt_stride_t, prm->kt_sh = f.kt_stride_h;
    prm->vt_sb = f.vt_stride_b, prm->vt_st = f.vt_stride_t, prm->vt_sh = f.vt_stride_h;
    prm->tail_len = tail_len;
    prm->o = o, prm->lse = lse;
    unsigned char* sc = static_cast<unsigned char*>(scratch);
    prm->part_ml = reinterpret_cast<float2*>(sc + pl.ml_off);
    prm->part_o = reinterpret_cast<float*>(sc + pl.o_off);
    prm->status = static_cast<unsigned int*>(workspace);
    prm->wait_limit_ns = gdn::wait_limit_ns();
    prm->stall_after = gdn::stall_after();
    prm->prefix_len = f.prefix_len, prm->max_tail = f.max_tail;
    prm->scale_log2 = scale_log2(f);
    prm->B = f.batch, prm->n = f.num_queries, prm->Hq = f.num_q_heads, prm->Hkv = f.num_kv_heads;
    prm->G = f.num_q_heads / f.num_kv_heads;
    prm->pre_splits = pl.pre_splits, prm->pre_chunk = pl.pre_chunk, prm->tail_splits = pl.tail_splits;
    prm->pre_tiles = pl.pre_tiles, prm->tail_tiles = pl.tail_tiles, prm->groups = pl.groups;
    prm->by_hkv.set(f.num_kv_heads), prm->by_b.set(f.batch), prm->by_g.set(prm->G);
    prm->by_ng.set((uint32_t)(f.num_queries * prm->G));
    prm->by_pre_tiles.set(std::max(pl.pre_tiles, 1)), prm->by_tail_tiles.set(std::max(pl.tail_tiles, 1));
    prm->by_tail_splits.set(std::max(pl.tail_splits, 1));
    const bool bf16 = f.dtype == GDN_BF16;
    const int64_t pre_items = (int64_t)f.num_kv_heads * pl.pre_splits * pl.pre_tiles;
    const int64_t tail_items = items - pre_items;
    if (pl.tc) {
        bool maps = true;
        const int64_t D = f.head_dim, Hkv = f.num_kv_heads, pre_dim[4] = {D, Hkv, f.prefix_len, 1},
                      tail_dim[4] = {D, Hkv, f.tail_cap, f.batch};
        if (f.prefix_len > 0)
            maps = bf16_map(&prm->tm_kp, k_prefix, 3, pre_dim, {f.kp_stride_h, f.kp_stride_t, 0}, gdn::prefix::kTcKeys) &&
                   bf16_map(&prm->tm_vp, v_prefix, 3, pre_dim, {f.vp_stride_h, f.vp_stride_t, 0}, gdn::prefix::kTcKeys);
        if (maps && f.max_tail > 0)
            maps = bf16_map(&prm->tm_kt, k_tail, 4, tail_dim, {f.kt_stride_h, f.kt_stride_t, f.kt_stride_b},
                            gdn::prefix::kTcKeys) &&
                   bf16_map(&prm->tm_vt, v_tail, 4, tail_dim, {f.vt_stride_h, f.vt_stride_t, f.vt_stride_b},
                            gdn::prefix::kTcKeys);
        if (!maps) return GDN_ERR_CUDA;
        const bool direct = pl.parts() == 1;
        if (gdn::prefix::launch_tc(*prm, f.head_dim, pl.row_tiles, pre_items, tail_items, pl.joined, direct, stream) !=
            cudaSuccess)
            return GDN_ERR_CUDA;
        if (direct) return GDN_OK;
    } else if (gdn::prefix::launch_simt(*prm, f.head_dim, bf16, stream) != cudaSuccess) {
        return GDN_ERR_CUDA;
    }
    return gdn::prefix::launch_join(*prm, f.head_dim, bf16, pl.parts(), stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

GDN_EXPORT size_t gdn_linear_scratch_bytes(const gdn_linear_problem* p) {
    LinStrides sd{};
    if (check_linear(p, sd) != GDN_OK || check_lengths(p) != GDN_OK) return 0;
    return (size_t)plan_linear(p).slots * p->num_heads * p->d_v * p->d_k * 4;
}

GDN_EXPORT gdn_status gdn_linear_prefill(const gdn_linear_problem* p, const void* q, const void* k, const void* v,
                                         const float* alpha, const float* S0, const int32_t* s0_index, int64_t s0_slots,
                                         void* o, float* S_final, const int64_t* ckpt_pos, const int64_t* cu_ckpt,
                                         float* ckpt_states, void* scratch, size_t scratch_bytes, void* workspace,
                                         size_t ws_bytes, gdn_stream_t stream) {
    return guarded([&] {
        return linear_prefill(p, q, k, v, alpha, S0, s0_index, s0_slots, o, S_final, ckpt_pos, cu_ckpt, ckpt_states,
                              scratch, scratch_bytes, workspace, ws_bytes, (cudaStream_t)stream);
    });
}

GDN_EXPORT gdn_status gdn_linear_step(const gdn_linear_problem* p, const void* q, const void* k, const void* v,
                                      const float* alpha, float* states, int64_t num_slots, const int32_t* slots,
                                      void* o, gdn_stream_t stream) {
    LinStrides sd{};
    const gdn_status st = check_linear(p, sd);
    if (st != GDN_OK) return st;
    if (!q || !k || !v || !alpha || !states || !o || num_slots < 0 || (!slots && num_slots < p->num_seqs))
        return GDN_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(alpha, 4) || !aligned(states, 16) ||
        !aligned(o, 16) || !aligned(slots, 4))
        return GDN_ERR_INVALID_ARG;
    if ((int64_t)p->num_seqs * p->num_heads * (p->d_v / 8) >= (1ll << 31)) return GDN_ERR_UNSUPPORTED;
    gdn::lin::StepParams s{};
    s.q = q, s.k = k, s.v = v;
    s.q_stride = sd.q, s.k_stride = sd.k, s.v_stride = sd.v;
    s.alpha = alpha, s.states = states, s.slots = slots, s.o = o;
    s.num_slots = num_slots, s.scale = p->scale;
    s.B = p->num_seqs, s.H = p->num_heads, s.rep = p->num_heads / p->num_qk_heads, s.dv = p->d_v;
    return gdn::lin::launch_step(s, p->d_k, p->qkv_dtype == GDN_BF16, p->out_dtype == GDN_BF16, (cudaStream_t)stream) ==
                   cudaSuccess
               ? GDN_OK
               : GDN_ERR_CUDA;
}

GDN_EXPORT size_t gdn_prefix_scratch_bytes(const gdn_prefix_problem* p) {
    gdn_prefix_problem f;
    return check_prefix(p, f) == GDN_OK ? plan_prefix(f).total : 0;
}

GDN_EXPORT gdn_status gdn_prefix_attention(const gdn_prefix_problem* p, const void* q, const void* k_prefix,
                                           const void* v_prefix, const void* k_tail, const void* v_tail,
                                           const int32_t* tail_len, void* o, float* lse, void* scratch,
                                           size_t scratch_bytes, void* workspace, size_t ws_bytes,
                                           gdn_stream_t stream) {
    return guarded([&] {
        return prefix_attention(p, q, k_prefix, v_prefix, k_tail, v_tail, tail_len, o, lse, scratch, scratch_bytes,
                                workspace, ws_bytes, (cudaStream_t)stream);
    });
}
