// gdn_prefix.cuh - attention for a batch that shares a long prefix: the parameter block and launchers shared by
// the kernels (gdn_prefix_tc.cu: tensor cores, bf16 of width 64 and 128; gdn_prefix.cu: every other size and type, and
// the join) and the host side (gdn_hybrid_api.cu).
//
// The work falls into parts: `pre_splits` ranges of the prefix, taken by the stacked query rows of all requests,
// and `tail_splits` ranges of each request's own tail, taken by its own rows.  A part leaves, for every query row,
// the maximum m of its scores (times log2 e), l = sum 2^(x - m) and the unnormalised sum of values; the join adds the
// parts up.  Query rows of one key/value head are ordered by request, query and head of the group, and a part's sums are
// kept in groups of 32 such rows, column by column: the threads that hold and that join them have a row each, so a warp
// writes and reads whole lines.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn {
namespace prefix {

// Division of 0 <= x < 2^31 by a fixed d >= 1 as a multiplication, by Granlund and Montgomery's method ("Division by invariant
// integers using multiplication", 1994: m = floor(2^32 (2^s - d) / d) + 1, s = ceil(log2 d):
// x / d = (mulhi(x, m) + x) >> s).  A CTA finds its item with half a dozen of them, and starts on a cold instruction
// cache, where the divisions' code took longer than their arithmetic.
struct Div {
    uint32_t d, m, s;
    __host__ void set(uint32_t by) {
        d = by;
        for (s = 0; s < 32 && (1ull << s) < by; ++s) {}
        m = (uint32_t)((((1ull << s) - by) << 32) / by + 1);
    }
    __device__ __forceinline__ int div(int x) const { return (int)((__umulhi((uint32_t)x, m) + (uint32_t)x) >> s); }
    __device__ __forceinline__ int divmod(int x, int* rest) const {
        const int q = div(x);
        *rest = x - q * (int)d;
        return q;
    }
};

struct Params {
    CUtensorMap tm_kp, tm_vp, tm_kt, tm_vt;   // tensor-core kernel only
    const void* q;
    const void* kp;
    const void* vp;
    const void* kt;
    const void* vt;
    int64_t q_sb, q_sn, q_sh;                  // strides in elements
    int64_t kp_st, kp_sh, vp_st, vp_sh;
    int64_t kt_sb, kt_st, kt_sh, vt_sb, vt_st, vt_sh;
    const int32_t* tail_len;
    void* o;           // [B, n, Hq, D]
    float* lse;        // [B, n, Hq] or nullptr
    float* part_o;     // [parts][Hkv][groups][D][32]
    float2* part_ml;   // [parts][Hkv][groups][32]: m, l (l = 0: an empty part, whose part_o is not read)
    unsigned int* status;
    unsigned long long wait_limit_ns;
    int64_t prefix_len, max_tail;
    float scale_log2;               // softmax_scale * log2 e
    int32_t B, n, Hq, Hkv, G;       // G = Hq / Hkv
    int32_t pre_splits, pre_chunk;  // prefix range s: [s * pre_chunk, (s + 1) * pre_chunk) cut at prefix_len
    int32_t tail_splits;            // tail range s of S: a share of the request's own length (tail_range)
    int32_t pre_tiles, tail_tiles;  // row tiles of the stacked rows, and of one request's rows
    Div by_hkv, by_b, by_pre_tiles, by_tail_tiles, by_tail_splits, by_ng, by_g;   // ng = n G
    int32_t groups;                 // groups of 32 stacked rows of a key/value head
    int32_t stall_after;
};

// The group that stacked row `row` of a head belongs to, within part_o and part_ml.
__host__ __device__ inline int64_t part_group(const Params& p, int part, int head, int row) {
    return ((int64_t)part * p.Hkv + head) * p.groups + (row >> 5);
}

// Range s of a tail of `len` tokens cut in tail_splits: equal shares, rounded up to whole tiles of `tile` tokens.
__device__ __forceinline__ void tail_range(const Params& p, int len, int tile, int s, int* lo, int* hi) {
    const int share = (p.by_tail_splits.div(len + (int)p.by_tail_splits.d - 1) + tile - 1) / tile * tile;
    const int64_t a = (int64_t)s * share, b = a + share;
    *lo = (int)min(a, (int64_t)len);
    *hi = (int)min(b, (int64_t)len);
}

constexpr int kSimtRows = 16;    // query rows of a tile of the FP32-pipe kernel
constexpr int kSimtKeys = 32;    // tokens of a staged tile

constexpr int kSms = 152;        // multiprocessors of a GB300, by which the host estimates how many CTAs run at once
constexpr int kTcRows = 128;     // query rows of a row tile, and tokens of a tile, of the tensor-core kernel
constexpr int kTcKeys = 128;

cudaError_t launch_simt(const Params& p, int D, bool bf16, cudaStream_t stream);
// `row_tiles` (1 or 2) row tiles a CTA.  joined: an item takes the whole prefix and then the whole tail of one request's
// rows (pre_items = 0); direct: the items write o and lse themselves (one part in all)
cudaError_t launch_tc(const Params& p, int D, int row_tiles, int64_t pre_items, int64_t tail_items, bool joined,
                      bool direct, cudaStream_t stream);
cudaError_t launch_join(const Params& p, int D, bool bf16, int parts, cudaStream_t stream);

}  // namespace prefix
}  // namespace gdn
