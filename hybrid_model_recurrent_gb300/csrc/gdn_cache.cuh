// gdn_cache.cuh - the operators around a paged 8-bit cache (gdn_cache.h): parameter blocks and launchers shared by the
// kernels (gdn_cache.cu: norm and rotation, append, upkeep; gdn_paged.cu: attention of few rows, fp32, and the join;
// gdn_paged_tc.cu: attention of many rows) and the host side (gdn_cache_api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn_kernel.cuh"

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
    bool bad;   // more tokens, or more new ones, than the call's bounds
};
__device__ __forceinline__ Request request_at(const Cache& c, const Batch& t, int b) {
    Request q;
    q.first = min(max(t.cu[b], 0), t.T);
    q.n = min(max(t.cu[b + 1], q.first), t.T) - q.first;
    q.row = t.rows ? t.rows[b] : b;
    if (q.row < 0 || q.row >= c.R) q.row = -1;
    const int len = q.row < 0 ? 0 : c.lens[q.row];
    q.len = min(max(len, 0), t.max_len);
    q.bad = q.n > t.max_new || len > t.max_len;
    q.n = min(q.n, t.max_new);
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
int rope_passes(int Hq, int Hk, int D, bool bf16);
cudaError_t launch_append(const AppendParams& p, int D, bool bf16, cudaStream_t s);
cudaError_t launch_update(const UpkeepParams& p, cudaStream_t s);
cudaError_t launch_compact(const UpkeepParams& p, cudaStream_t s);

// ---- attention ----------------------------------------------------------------------------------------------------
//
// The work is cut evenly over the CTAs: an item is a tile of RT query rows of one request and key/value head (rows in the
// order of tokens and of the heads of the group), a unit is a number of tokens that an item's rows see, and CTA c takes the
// units [c share, (c + 1) share) of them all, in the order of requests, heads, row tiles and tokens.  What an item costs besides its
// tokens counts as kLead units before them, which are nobody's work: else the CTAs that have a prompt's first tiles, of few tokens, are
// late (a prompt of 8192 x 32 heads, bf16: 616 us without lead, 494, 479, 489 with 3, 4, 6
// units; in fp32 3700 and, with 2, 4, 6, 10, 3418, 3085, 2805, 2693; but 128 single tokens on 100 to 4800 122, 124, 128 with 4, 6, 10).  So a CTA has at most one
// item that it begins in the middle (its part goes to slot 2 c) and one that it begins and leaves unfinished (slot 2 c + 1).
// Every CTA describes the item that it begins in the middle, if the CTA before began it (a cut), and a join, whose grid follows the
// CTAs and not the batch, adds the cut items' parts up.  Lengths are read on the device only, and differ at will.
struct Cut {
    int32_t rows, row0, h, first;   // 0 rows: no cut here
    int32_t last, unused[3];        // CTAs c - 1 .. last have the item's parts
};
struct PagedParams {
    Cache c;
    Batch t;
    const void* q;
    int64_t q_stride;
    void* o;             // [T, Hq, D]
    float* lse;          // [T, Hq] or nullptr
    float* part_o;       // [2 CTAs][RT][D]: sums of 2^(x - m) v
    float2* part_ml;     // [2 CTAs][RT]: m, l
    Cut* cuts;           // [CTAs]
    unsigned int* status;
    float scale_log2;
    int32_t Hq, G, ctas;
    int32_t min_rows, max_rows;         // requests with other numbers of query rows a key/value head are another launch's
    unsigned long long wait_limit_ns;   // (tensor-core kernel)
    int32_t stall_after;
};

__device__ __forceinline__ Request attended(const PagedParams& p, int b) {
    Request q = request_at(p.c, p.t, b);
    if (q.n * p.G < p.min_rows || q.n * p.G > p.max_rows) q.n = 0;
    return q;
}

// The join's CTAs may be started (they wait for this kernel's end before they read anything of it).
__device__ __forceinline__ void join_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

constexpr int kUnit = 64;       // tokens of a unit: warp-level products
constexpr int kTcUnit = 128;    // 5th-generation tensor cores
constexpr int kTcRows = 256;
constexpr int kLead = 4;
constexpr int kMostUnits = 0x7fffffff - (1 << 20) + 1;   // of all items

// Tokens that a row tile's last row sees (its units are one at least: rows that see nothing are written too).
__device__ __forceinline__ int tile_sees(const Request& q, int G, int RT, int tile) {
    const int last = (min((tile + 1) * RT, q.n * G) - 1) / G;
    return max(0, min(q.len, q.len - q.n + last + 1));
}
// The units of a request's tiles with their lead, one after the other (without a division for each).
template <int RT, int UNIT>
struct TileWalk {
    int base, len, last, qi, rest, G, step_qi, step_rest;   // qi, rest: the tile's last row is `rest` of token qi
    __device__ __forceinline__ TileWalk(const Request& q, int G_) : base(q.len - q.n + 1), len(q.len), last(q.n - 1), G(G_) {
        qi = (RT - 1) / G, rest = (RT - 1) - qi * G;
        step_qi = RT / G, step_rest = RT - step_qi * G;
    }
    __device__ __forceinline__ int next() {
        const int u = kLead + max(1, (max(0, min(len, base + min(qi, last))) + UNIT - 1) / UNIT);
        qi += step_qi, rest += step_rest;
        if (rest >= G) rest -= G, ++qi;
        return u;
    }
};
// units of a request for one head (none without queries)
template <int RT, int UNIT>
__device__ __forceinline__ int head_units(const Request& q, int G) {
    int n = 0;
    const int tiles = (q.n * G + RT - 1) / RT;
    TileWalk<RT, UNIT> w(q, G);
    for (int t = 0; t < tiles; ++t) n += w.next();
    return n;
}

// Units before every group of requests into s_cum, by all THREADS threads of a CTA, a thread a request; a group is the least power of two
// with which kMaxGroups of them hold the batch (one request up to 256).  The host's plan keeps the total
// to kMostUnits for counts as the call describes them (CTAs round their shares up: sums stay in 31 bits); the sums here stop at kNoTotal, and
// a larger total (cu_new that falls) is reported and nothing is done.
constexpr unsigned kNoTotal = 0x7fffffffu;
constexpr int kMaxGroups = 256;
__device__ __forceinline__ int group_log2(int B) {
    int s = 0;
    while (((B - 1) >> s) >= kMaxGroups) ++s;
    return s;
}
__device__ __forceinline__ int groups_of(int B) { return ((B - 1) >> group_log2(B)) + 1; }
template <int THREADS, int RT, int UNIT>
__device__ __forceinline__ void count_units(const PagedParams& p, int* s_cum) {
    const int tid = threadIdx.x, lane = tid & 31, B = p.t.B, shift = group_log2(B), width = 1 << shift, groups = groups_of(B);
    for (int b0 = 0; b0 < B; b0 += THREADS) {
        const int b = b0 + tid;
        unsigned n = 0;
        if (b < B) {
            const Request q = attended(p, b);
            if (q.bad && blockIdx.x == 0) atomicOr(p.status, STATUS_BAD_INDEX);
            n = (unsigned)(head_units<RT, UNIT>(q, p.G) * p.c.Hkv);
        }
        unsigned y = n;
        for (int o = 1; o < width; o <<= 1) {
            const unsigned z = __shfl_up_sync(0xffffffffu, y, o, width);
            if ((tid & (width - 1)) >= o) y = min(y + z, kNoTotal);
        }
        if ((tid & (width - 1)) == width - 1 && (b >> shift) < groups) s_cum[(b >> shift) + 1] = (int)y;
    }
    __syncthreads();
    if (tid < 32) {
        constexpr int PER = kMaxGroups / 32;
        unsigned sum = 0;
        for (int i = 0; i < PER; ++i)
            if (lane * PER + i < groups) sum = min(sum + s_cum[lane * PER + i + 1], kNoTotal);
        unsigned y = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y = min(y + z, kNoTotal);
        }
        const bool none = __shfl_sync(0xffffffffu, y, 31) > (unsigned)kMostUnits;
        if (none && lane == 0 && blockIdx.x == 0) atomicOr(p.status, STATUS_BAD_INDEX);
        y -= sum;
        for (int i = 0; i < PER; ++i)
            if (lane * PER + i < groups) y += s_cum[lane * PER + i + 1], s_cum[lane * PER + i + 1] = none ? 0 : (int)y;
        if (lane == 0) s_cum[0] = 0;
    }
    __syncthreads();
}

// What a CTA does of one item: rows row0 .. of `rows` of the request, tokens lo .. hi; it has the units u0 .. u1 of the item's `units`.
struct Segment {
    Request rq;
    int h, row0, rows, lo, hi, u0, u1, units;
    __device__ __forceinline__ bool whole() const { return u0 == 0 && u1 == units; }
    __device__ __forceinline__ int64_t slot() const { return 2 * (int64_t)blockIdx.x + (u0 == 0); }
};
// The item at unit x, looked for; returns its units before x.  Called by whole warps.
template <int RT, int UNIT>
__device__ __forceinline__ int find_item(const PagedParams& p, const int* s_cum, int x, Segment& s) {
    const int shift = group_log2(p.t.B);
    int g = 0, top = groups_of(p.t.B);   // cum[g] <= x < cum[top]
    while (top - g > 1) {
        const int mid = (g + top) >> 1;
        if (s_cum[mid] <= x) g = mid;
        else top = mid;
    }
    int mine = x - s_cum[g], head;   // the unit within its request, and the request's units a head
    if (shift == 0) {
        s.rq = request_at(p.c, p.t, g);
        head = (s_cum[g + 1] - s_cum[g]) / p.c.Hkv;
    } else {   // the requests of the group, a lane each
        const int lane = threadIdx.x & 31, b = (g << shift) + lane, width = 1 << shift;
        Request q{-1, 0, 0, 0, false};
        if (lane < width && b < p.t.B) q = attended(p, b);
        const int per_head = head_units<RT, UNIT>(q, p.G), n = per_head * p.c.Hkv;
        int after = n;
        for (int o = 1; o < width; o <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, after, o);
            if (lane >= o) after += z;
        }
        const int at = __ffs(__ballot_sync(0xffffffffu, lane < width && mine < after)) - 1;
        s.rq.row = __shfl_sync(0xffffffffu, q.row, at), s.rq.len = __shfl_sync(0xffffffffu, q.len, at);
        s.rq.n = __shfl_sync(0xffffffffu, q.n, at), s.rq.first = __shfl_sync(0xffffffffu, q.first, at);
        mine -= __shfl_sync(0xffffffffu, after - n, at);
        head = __shfl_sync(0xffffffffu, per_head, at);
    }
    s.h = mine / head;
    mine -= s.h * head;
    int tile = 0;
    TileWalk<RT, UNIT> w(s.rq, p.G);
    for (const int last = (s.rq.n * p.G - 1) / RT;; ++tile) {   // (it ends, whatever becomes of the lengths meanwhile)
        const int units = w.next();
        if (mine < units || tile >= last) break;
        mine -= units;
    }
    s.row0 = tile * RT;
    return mine;
}
// The next item of which the CTA has tokens, from unit x on, where the one of `s` ended: the request's next tile or head (found step by
// step from its first, the tiles of prompts cost more than their products), another request's, or, after segment_none(), the CTA's
// first.  x moves behind what the CTA has of it; false: it has no more.
template <int RT, int UNIT>
__device__ __forceinline__ bool next_segment(const PagedParams& p, const int* s_cum, int& x, int end, Segment& s) {
    while (x < end) {
        s.row0 += RT;
        int v0 = 0;   // units of the item, with its lead, that are other CTAs'
        if (s.row0 >= s.rq.n * p.G) {
            s.row0 = 0;
            if (++s.h >= p.c.Hkv) v0 = find_item<RT, UNIT>(p, s_cum, x, s);
        }
        const int seen = tile_sees(s.rq, p.G, RT, s.row0 / RT);
        s.units = max(1, (seen + UNIT - 1) / UNIT);
        const int v1 = min(kLead + s.units, v0 + (end - x));
        x += v1 - v0;
        s.u0 = max(0, v0 - kLead), s.u1 = v1 - kLead;
        if (s.u1 <= s.u0) continue;
        s.rows = min(s.rq.n * p.G - s.row0, RT);
        s.lo = s.u0 * UNIT;
        s.hi = min(s.u1 * UNIT, seen);
        return true;
    }
    return false;
}
__device__ __forceinline__ Segment segment_none() {
    Segment s{};
    s.h = 1 << 30;
    return s;
}
// The CTA's cut, written by one thread; `s`: its first segment.
__device__ __forceinline__ void describe_cut(const PagedParams& p, const Segment& s, int begin, int share) {
    const int at = begin - s.u0;   // the item's first tokens
    Cut c{};
    if (s.u0 > 0 && at >= begin - share)
        c.rows = s.rows, c.row0 = s.row0, c.h = s.h, c.first = s.rq.first, c.last = (at + s.units - 1) / share;
    p.cuts[blockIdx.x] = c;
}

// `tiles`: row tiles of 16 that a CTA takes at once (1 or 2)
cudaError_t launch_paged(const PagedParams& p, int D, bool bf16, int tiles, cudaStream_t s);
cudaError_t launch_paged_tc(const PagedParams& p, int D, cudaStream_t s);
cudaError_t launch_paged_join(const PagedParams& p, int D, bool bf16, int tile_rows, cudaStream_t s);

}  // namespace cache
}  // namespace gdn
