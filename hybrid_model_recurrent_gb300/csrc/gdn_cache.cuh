// gdn_cache.cuh - the operators around a paged 8-bit cache (gdn_cache.h): parameter blocks and launchers shared by the
// kernels (gdn_cache.cu: norm and rotation, append, upkeep; gdn_paged.cu: attention of few rows, fp32, and the join;
// gdn_paged_tc.cu: attention of many rows) and the host side (gdn_cache_api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn {
namespace cache {

constexpr int kSms = 152;

struct RopeParams {
    const void* q;
    const void* k;
    void* q_out;
    void* k_out;
    const int32_t* positions;
    const double* inv_freq;
    const void* qw;
    const void* kw;
    int64_t q_stride, k_stride, qo_stride, ko_stride;   // elements between tokens
    int64_t T;
    int32_t Hq, Hk, rd;
    int32_t parts, per_part;   // shares of a token's passes over its heads, and passes of a share
    int32_t normalize;
    float eps, mscale;
};

struct Cache {
    unsigned char* pages;   // of the layer
    float* scales;          // of the layer
    const int32_t* table;
    const int32_t* lens;
    int32_t N, page, page_log2, Hkv, R, W;
};

struct Batch {
    const int32_t* cu;
    const int32_t* rows;
    int32_t B, max_new, max_len;
    int32_t T;
};

// Request b's row of the table, its tokens and where its new ones start in the packed streams.  row < 0: padding.
// Device values are taken within their bounds, whatever they say.
struct Request {
    int row, len, n, first;
    bool bad;   // more new tokens than the call's bound
};
__device__ __forceinline__ Request request_at(const Cache& c, const Batch& t, int b) {
    Request q;
    q.first = min(max(t.cu[b], 0), t.T);
    q.n = min(max(t.cu[b + 1], q.first), t.T) - q.first;
    q.row = t.rows ? t.rows[b] : b;
    if (q.row < 0 || q.row >= c.R) q.row = -1;
    q.len = q.row < 0 ? 0 : min(max(c.lens[q.row], 0), t.max_len);
    q.bad = q.n > t.max_new;
    if (q.bad) q.n = t.max_new;
    return q;
}

struct AppendParams {
    Cache c;
    Batch t;
    const void* k;
    const void* v;
    int64_t k_stride, v_stride;
    unsigned int* status;
};

struct UpkeepParams {
    int32_t* table;
    int32_t* lens;
    int32_t* refs;
    int32_t N, R, W, page, page_log2;
    int32_t n_drop, n_fork;
    const int32_t* drop;
    const int32_t* from;
    const int32_t* to;
    const int32_t* grow;
    int32_t* granted;
    int32_t* live;
    // scratch: copies asked for, then lists of N each (pages to take; a copy's source and destination)
    int32_t* n_copies;
    int32_t* free_list;
    int32_t* copy_from;
    int32_t* copy_to;
    // what the copies move
    unsigned char* pages;
    float* scales;
    int64_t page_bytes, layer_bytes, layer_scales;
    int32_t L, page_scales;
    unsigned int* status;
};

constexpr int kMaxRows = 16384;
constexpr int kMaxBatch = 4096;

cudaError_t launch_rope(const RopeParams& p, int D, bool bf16, bool half, cudaStream_t s);
int rope_passes(int heads, int D, bool bf16);
cudaError_t launch_append(const AppendParams& p, int D, bool bf16, cudaStream_t s);
cudaError_t launch_update(const UpkeepParams& p, cudaStream_t s);
cudaError_t launch_compact(const UpkeepParams& p, cudaStream_t s);

// ---- attention ----------------------------------------------------------------------------------------------------
//
// The work is cut evenly over the CTAs: an item is a tile of the query rows of one request and key/value head, a unit is
// `kUnit` tokens of an item, and CTA c takes the units [c share, (c + 1) share) of them all, in the order of requests,
// heads, row tiles and tokens.  A CTA has so at most one item that it begins in the middle (its part goes to slot 2 c) and one that
// it begins and leaves unfinished (slot 2 c + 1); a join adds the parts up.
struct PagedParams {
    Cache c;
    Batch t;
    const void* q;
    int64_t q_stride;
    void* o;             // [T, Hq, D]
    float* lse;          // [T, Hq] or nullptr
    float* part_o;       // [2 CTAs][rows of a tile][D]
    float2* part_ml;     // [2 CTAs][rows of a tile]: m, l
    int32_t* starts;     // [B + 1] units before each request, written by the first CTA for the join
    unsigned int* status;
    float scale_log2;
    int32_t Hq, G, ctas;
};
constexpr int kUnit = 64;

// `tiles`: row tiles of 16 that a CTA takes at once (1 or 2)
cudaError_t launch_paged(const PagedParams& p, int D, bool bf16, int tiles, bool join, cudaStream_t s);

}  // namespace cache
}  // namespace gdn
