// gdn_paged_tc.cu - attention over a paged 8-bit cache for many query rows a key/value head (turns and prompts, bf16,
// head_dim 64 or 128), on the 5th-generation tensor cores.
//
// A CTA takes two tiles of 128 query rows of one request and key/value head against tiles of 128 tokens:
//     S = Q K^T  (TMEM, fp32)  ->  P = 2^(x - m) (f16, over S's own columns)  ->  O += P V  (TMEM, fp32)
// with each row's running maximum m and sum l in the thread that owns the row, and O rescaled only when m has risen by more
// than 2^8.  Scores, statistics and sums are fp32; the weights are rounded to f16 for the product (half a step, 2^-11 of each).
//
// All operands are f16, which holds e4m3 exactly and takes one conversion for two values.  What f16 lacks in range is carried
// beside it, by factors that cost nothing a value: a row of Q is brought to [2^14, 2^15) by a power of two, the scale of
// the keys' block joins that of the row in the exponent, the scale of the values' block goes into it too, relative to the
// largest of the item so far (and is taken out again where l is summed); raising that one rescales O as a risen maximum does.
// (With bf16 operands the converting warps below, three then, made two conversions and a product for each value, and a tile took 10 k cycles; a product
// of f16 pairs for blocks that differ within a tile took as long as conversion and copies together.)
//
// Bulk copies bring the pages' bytes (a block is contiguous) into a ring of their own, five warps convert them and write
// the swizzled tiles that the products read.  Tokens behind what the rows see are written as zeros, whatever the page holds
// there.
//
// The units (128 tokens of an item) are dealt out evenly over the CTAs, one a multiprocessor (gdn_cache.cuh).
// Roles: warps 0 .. 7 softmax (one warpgroup a row tile), warps 8 and 15 issue the products of one row tile each, warp 9 copies, warps
// 10 .. 14 convert (three the first 64 tokens of a tile, two the others).  An item of at most 128 rows takes one row tile, in turn.
//
// A step is half a tile, 64 tokens, and S has room for two: the scores of step i + 2 are issued behind the product of step i, so
// a row tile's softmax finds its next scores ready and runs without a pause.  It takes a step's 64 scores of a row at once and
// compares with the maximum so far; O is rescaled, rarely, once the product before is done.  (16 x 256 new tokens x 32 heads on
// 17 k tokens: scores of whole tiles, one after the softmax of the other, 662 us; two halves issued by one warp for both row
// tiles 826, its barriers and elections in turn.  Rows of 128 scores held by 384 threads, three warps converting, 887: a lone warp's
// instructions came at 7 to 9 cycles each, waiting for the instruction cache.)
// What bounds it: that case takes 588 us, 1090 TFLOP/s of the products asked for, 0.57 of a library product's rate, 3.4 k cycles a tile
// of 128 tokens of which the products take 2.1 k, and 7 us an item besides; a step of the softmax takes 1.5 k whatever is left out of
// its arithmetic (at 601 us: without exponentials 578, without the maximum 569): its waits, the scores' way from TMEM and the weights'
// back.  With one row tile the conversion takes as long: neither more converting warps nor both row tiles on every other tile gain.
//
// Every wait is bounded: a role that gives up sets the CTA's abort flag and the sticky status, every role leaves its
// loop, copies and products in flight are waited for, and TMEM is freed.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "gdn_cache.cuh"
#include "gdn_tc_util.cuh"

namespace gdn {
namespace cache {
namespace {

using tc::idesc;
using tc::proxy_fence;
using tc::tc_fence_after;
using tc::tc_fence_before;
using tc::tmem_ld32;
using tc::tmem_ld32x2;
using tc::tmem_st16;
using tc::tmem_st_wait;
using tc::umma_commit;
using tc::umma_ss;
using tc::umma_ts;
using tcu::cols_step;
using tcu::elect_one;
using tcu::pack2;
using tcu::rows_step;
using tcu::store32;
using tcu::tile_desc;
using tcu::warp_wait_bar;

constexpr int kRows = 128;    // rows of a tile
constexpr int kKeys = kTcUnit;
constexpr float kRise = 8.f;  // O is rescaled when a maximum has risen by more than this (log2)
constexpr float kLift = 7.f;  // log2 of a weight at the maximum: with the rise 2^15 in f16
constexpr int kConv0 = 3, kConv1 = 2;   // converting warps for the first half of a tile, and for the second
// A weight's exponent is score * scale + (kLift - m), and two roundings can carry it past the 15 that a maximum which has not risen
// leaves it: that of the score as the rise was judged by it, and that of the bracket.  Up to 2^22 each is a quarter at most, and 2^15.5 is
// in f16's range (with 2^28 here exponents reached 24, and the weights infinity).  Rows further from zero round the product by itself
// first, as the maximum was, and take that off it, exactly where their difference counts.
constexpr float kFar = 4194304.f;
// Factors of scores are not below the smallest normal number: a hidden token's -infinity stays that.
constexpr float kTiny = 1.17549435e-38f;
constexpr int kThreads = 512;

template <int D>
struct Cfg {
    static constexpr int kTile = kKeys * D * 2;               // bytes of a K, V or Q tile
    static constexpr int ST = D == 128 ? 4 : 8;               // K and V tiles in turn
    static constexpr int RS = D == 128 ? 4 : 8;               // halves of them as bytes of the pages
    static constexpr int kHalf = kKeys / 2 * D;               // bytes of such a half
    static constexpr int kRing = 2 * kTile;                   // after the Q tiles
    static constexpr int kRaw = kRing + ST * kTile;
    static constexpr int kBar = kRaw + RS * kHalf;
    static constexpr int kInfos = ST == 4 ? 4 : 8;            // tiles described: when one is, V of ST / 2 + 1 tiles before is done
    static constexpr int kArea = ST == 4 ? 2048 : 2816;       // barriers, units before each group of requests, the descriptions
    static constexpr int kSmem = kBar + kArea + 1024;
    static constexpr uint32_t kO = 256;                       // TMEM: S of each row tile, then O of each
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t half2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// instruction descriptor of kind::f16: D fp32, A and B f16, M = 128
__host__ __device__ constexpr uint32_t idesc_f16(int N, bool b_mn) { return idesc(N, false, b_mn) & ~((1u << 7) | (1u << 10)); }

// 16 columns, waited for
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// What a risen maximum changes: O, in `pieces` of 16 columns from to on.  A function by itself, so that the loop of the softmax
// stays small.
__device__ __noinline__ void rescale(uint32_t to, int pieces, float fo) {
#pragma unroll 1
    for (int k = 0; k < pieces; ++k) {
        uint32_t o[16];
        tmem_ld16(to + 16 * k, o);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * fo);
        tmem_st16(to + 16 * k, o);
    }
}

// 16 e4m3 as f16
__device__ __forceinline__ void widen16(const uint4& u, uint32_t (&y)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(y[2 * i]), "=r"(y[2 * i + 1])
            : "r"(w[i]));
}

// What the rows need to know of a tile: for each 16 of its tokens (a page has as many at least) the scale of the keys, the log2
// of a weight at the maximum, and that weight's inverse; the largest scale of the item's values so far (a power of two).
struct TileInfo {
    float4 part[kKeys / 16];
    float v, unused[3];
};

// The weights of a tile's chunk c for rows far from zero, over its scores; returns their sum.
__device__ __noinline__ float far_weights(uint32_t ts, int c, int seen, float row_scale, float base, float4 f) {
    const float scale = fmaxf(row_scale * f.x, kTiny);
    float sum = 0.f;
    uint32_t x[16], w[8];
    tmem_ld16(ts + 16 * c, x);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float y = __fsub_rn(__fmul_rn(__uint_as_float(x[i]), scale), base);
        const float e = 16 * c + i < seen ? ex2(y + f.y) : 0.f;
        x[i] = __float_as_uint(e);
        sum += e * f.z;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = half2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
    tmem_st8(ts + 8 * c, w);
    return sum;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) paged_tc_kernel(const __grid_constant__ PagedParams p) {
    using F = Cfg<D>;
    static_assert(F::kSmem <= 232448, "shared memory");
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_addr(smem);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + F::kBar);   // [ST][2] half a K or V tile written
    uint64_t* empty = full + 2 * F::ST;                              // [ST][2] every product that reads it is done
    uint64_t* s_full = empty + 2 * F::ST;                            // [2][2] S of a row tile done, in the one or the other half
    uint64_t* p_ready = s_full + 4;                                  // [2][2] P written over it, O rescaled
    uint64_t* pv_done = p_ready + 4;                                 // [2] and multiplied by V
    uint64_t* q_ready = pv_done + 2;                                 // [2] an item's Q tile written
    uint64_t* end_bar = q_ready + 2;                                 // [2] every product of an issuing warp done
    uint64_t* raw_full = end_bar + 2;                                // [RS] half a tile's bytes landed
    uint64_t* raw_empty = raw_full + F::RS;                          // [RS] and read by the converting warps
    uint32_t* tslot = reinterpret_cast<uint32_t*>(raw_empty + F::RS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
    int* issued = reinterpret_cast<int*>(tslot + 2);                 // halves whose copies were issued
    int* s_cum = issued + 1;                                         // units before each group of requests
    TileInfo* info = reinterpret_cast<TileInfo*>(smem + F::kBar + F::kArea - sizeof(TileInfo) * F::kInfos);
    static_assert((4 * F::ST + 2 * F::RS + 14) * 8 + 12 + (kMaxGroups + 1) * 4 + sizeof(TileInfo) * F::kInfos <= F::kArea, "barrier area");

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint64_t limit = p.wait_limit_ns;

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tslot)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (tid == 0) {
        // (a half tile is released by the products of both row tiles)
        for (int i = 0; i < 2 * F::ST; ++i) mbar_init(&full[i], i & 1 ? kConv1 : kConv0), mbar_init(&empty[i], 2);
        for (int i = 0; i < 4; ++i) mbar_init(&s_full[i], 1), mbar_init(&p_ready[i], 128);
        for (int i = 0; i < 2; ++i) mbar_init(&pv_done[i], 1), mbar_init(&q_ready[i], 128), mbar_init(&end_bar[i], 1);
        for (int i = 0; i < F::RS; ++i) mbar_init(&raw_full[i], 1), mbar_init(&raw_empty[i], i & 1 ? kConv1 : kConv0);
        *abort_flag = 0;
        *issued = 0;
        fence_barrier_init();
    }
    join_may_start();
    count_units<kThreads, kTcRows, kTcUnit>(p, s_cum);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tslot;
    auto warp_wait = [&](uint64_t* bar, int parity) { return warp_wait_bar(bar, (uint32_t)parity & 1u, abort_flag, limit); };

    const int total = s_cum[groups_of(p.t.B)], share = (total + (int)gridDim.x - 1) / (int)gridDim.x;
    const int begin = (int)min((int64_t)blockIdx.x * share, (int64_t)total), end = (int)min((int64_t)begin + share, (int64_t)total);

    if (tid == 0) p.cuts[blockIdx.x] = Cut{};

    // Every role walks the CTA's items; an item of at most 128 rows takes one row tile, the two in turn, so that one tile's sums
    // leave and its next Q arrives while the other computes.
    Segment x = segment_none();
    auto takes = [&](int& turn) {
        const int one = turn;
        if (x.rows <= kRows) turn ^= 1;
        return x.rows > kRows ? 3 : 1 << one;   // bit a: row tile a
    };
    auto tiles_of = [&] { return max(0, (x.hi - x.lo + kKeys - 1) / kKeys); };

    if (warp >= 8) {
        if (warp == 8 || warp == 15) {
            // ---- products of row tile a (the whole warp walks along, one elected lane issues); K of tile i is ring entry 2 i, V
            // 2 i + 1.  Step i: the values' product of its weights, and the scores of step i + 2 over their place ----
            const int a = warp == 15;
            auto slot_at = [&](int e) { return sbase + F::kRing + (uint32_t)(e % F::ST) * F::kTile; };
            auto landed = [&](int e, int half) { return warp_wait(&full[2 * (e % F::ST) + half], e / F::ST); };
            bool ok = true;
            int it = 0, turn = 0, steps = 0, nth = 0;   // tiles of all items; steps and items of this row tile
            const uint64_t q = tile_desc(sbase + a * F::kTile, false);
            for (int at = begin; ok && next_segment<kTcRows, kTcUnit>(p, s_cum, at, end, x);) {
                const int n = 2 * tiles_of(), on = takes(turn);
                if (n == 0) continue;
                if (!(on >> a & 1)) {   // the other row tile's alone: pass by, entry after entry, so that no barrier gets ahead
                    for (int i = 0; ok && i < 2 * n; ++i) {
                        const int e = 2 * it + (i >> 1 & 1) + 2 * (i >> 2), half = i & 1;   // K's halves, then V's
                        ok = landed(e, half);
                        if (ok && lane == 0) mbar_arrive(&empty[2 * (e % F::ST) + half]);
                    }
                    it += n / 2;
                    continue;
                }
                ok = warp_wait(&q_ready[a], nth++);
#pragma unroll 1
                for (int i = -2; ok && i < n; ++i) {
                    const int half = i & 1, ev = (2 * (it + (i >> 1)) + 1) & 0x7fffffff, ek = 2 * (it + (i >> 1)) + 2;
                    const bool pv = i >= 0, qk = i + 2 < n;
                    const int g = steps + i, region = g & 1;
                    ok = (!pv || landed(ev, half)) && (!qk || landed(ek, half)) && (!pv || warp_wait(&p_ready[2 * a + region], g >> 1));
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t v = tile_desc(slot_at(ev) + half * 8192, true), k = tile_desc(slot_at(ek) + half * 8192, false);
                    const uint32_t at_s = tbase + a * 128 + region * 64;
                    if (elect_one()) {
                        if (pv) {
#pragma unroll
                            for (int s = 0; s < 4; ++s)
                                umma_ts(tbase + F::kO + a * D, at_s + 8 * s, rows_step(v, s), idesc_f16(D, true), i > 0 || s > 0);
                            umma_commit(&pv_done[a]);
                            umma_commit(&empty[2 * (ev % F::ST) + half]);
                        }
                        if (qk) {
#pragma unroll
                            for (int s = 0; s < D / 16; ++s)
                                umma_ss(at_s, cols_step(q, s), cols_step(k, s), idesc_f16(64, false), s > 0);
                            umma_commit(&s_full[2 * a + region]);
                            umma_commit(&empty[2 * (ek % F::ST) + half]);
                        }
                    }
                }
                it += n / 2;
                steps += n;
            }
            if (elect_one()) umma_commit(&end_bar[a]);   // also after giving up: the end waits for the products in flight
        } else {
            // ---- keys and values: copied by a warp, a lane a page, and converted by five, in halves of 64 tokens ----
            const int64_t block = (int64_t)p.c.page * D;
            auto checked = [&](int id) {   // a table's entry, where it is used
                if ((unsigned)id >= (unsigned)p.c.N) {
                    atomicOr(p.status, STATUS_BAD_INDEX);
                    id = 0;
                }
                return id;
            };
            // (loaded by name where they stand, a tile before their use: the compiler moved plain loads down to it)
            auto load = [](const void* a) {
                uint32_t y;
                asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(y) : "l"(a));
                return y;
            };
            bool ok = true;
            int seq = 0;   // ring entries of the items so far
            if (warp == 9) {
                const int piece_log2 = min(p.c.page_log2, 6), lanes = kKeys >> piece_log2;   // a page or half of one a lane
                const uint32_t piece = (uint32_t)D << piece_log2;
                const int own_half = lane >= lanes / 2;
                const uint32_t own_to = sbase + F::kRaw + (uint32_t)(lane & (lanes / 2 - 1)) * piece;
                const int64_t kv_bytes = p.c.Hkv * block;
                const int stop = p.stall_after >= 0 ? 4 * p.stall_after : 0x7fffffff;   // testing hook
                int asked = 0;
                for (int at = begin; ok && next_segment<kTcRows, kTcUnit>(p, s_cum, at, end, x);) {
                    const int n = tiles_of();
                    if (n == 0) continue;
                    const int32_t* table = p.c.table + (int64_t)x.rq.row * p.c.W;   // (a row without tokens has no tiles)
                    // this lane's piece of tile j, and where it lies: found a tile ahead, so that a copy is a few instructions
                    auto token = [&](int j) { return x.lo + j * kKeys + (lane << piece_log2); };
                    auto copies = [&](int j) { return lane < lanes && j < n && token(j) < x.hi; };
                    auto copied = [&](int j) { return copies(j) ? (int)load(table + (token(j) >> p.c.page_log2)) : 0; };
                    int id = copied(0);
#pragma unroll 1
                    for (int j = 0; ok && j < n; ++j) {
                        const unsigned char* src = p.c.pages + ((int64_t)checked(id) * 2 * p.c.Hkv + x.h) * block +
                                                   (int64_t)(token(j) & (p.c.page - 1)) * D;
                        const bool some = copies(j);
                        const uint32_t who = __ballot_sync(0xffffffffu, some);
                        id = copied(j + 1);
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {   // the halves of the keys, then of the values
                            const int r = 2 * seq + 4 * j + c, at_r = r % F::RS, half = c & 1;
                            ok = r < stop && (r < F::RS || warp_wait(&raw_empty[at_r], r / F::RS - 1));
                            if (!ok) break;
                            if (lane == 0)
                                mbar_arrive_expect_tx(&raw_full[at_r], __popc(who >> (half * lanes / 2) & ((1u << lanes / 2) - 1)) * piece);
                            __syncwarp();
                            if (some && own_half == half)
                                asm volatile(
                                    "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                                        own_to + (uint32_t)at_r * F::kHalf),
                                    "l"(src + (c & 2 ? kv_bytes : 0)), "r"(piece), "r"(smem_addr(&raw_full[at_r]))
                                    : "memory");
                            asked = r + 1;
                        }
                    }
                    seq += 2 * n;
                }
                if (lane == 0) *issued = asked;
            } else {
                // A warp converts the tokens 8 g .. 8 g + 7 of its half for every second or third g, 64 bytes of a token by four lanes.  At
                // width 128 odd tokens take their 64 bytes the other way round: a quarter of a warp then meets every bank once,
                // reading and writing.
                const int half = warp >= 13, g0 = half ? warp - 13 : warp - 10, stride = half ? kConv1 : kConv0, sub = lane >> 2, quad = lane & 3;
                constexpr int kParts = D / 64;
                const int turned = kParts == 2 ? sub & 1 : 0;
                const int chunk0 = ((2 * quad) ^ sub) << 4, chunk1 = ((2 * quad + 1) ^ sub) << 4;   // (token & 7 = sub)
                const unsigned char* raw0 = smem + F::kRaw + (8 * g0 + sub) * D + quad * 16;
                unsigned char* to0 = smem + F::kRing + (64 * half + 8 * g0 + sub) * 128;
                const bool describes = warp == 12;   // (with two groups of 8 tokens, others have three)
                for (int at = begin; ok && next_segment<kTcRows, kTcUnit>(p, s_cum, at, end, x);) {
                    const int n = tiles_of();
                    if (n == 0) continue;
                    const int32_t* table = p.c.table + (int64_t)x.rq.row * p.c.W;
                    // the scales of the tokens 16 l .. 16 l + 15 of tile j
                    auto holds = [&](int j) { return lane < 8 && j < n && x.lo + j * kKeys + 16 * lane < x.hi; };
                    auto held = [&](int j) { return holds(j) ? (int)load(table + ((x.lo + j * kKeys + 16 * lane) >> p.c.page_log2)) : 0; };
                    auto scale_of = [&](int j, int id, int kv) {
                        return holds(j) ? __uint_as_float(load(p.c.scales + ((int64_t)checked(id) * 2 + kv) * p.c.Hkv + x.h)) : 0.f;
                    };
                    int id1 = 0;
                    float ks = 0.f, vs = 0.f;
                    int item_e = 0;   // exponent bits of the largest scale of the item's values so far
                    if (describes) {
                        const int id0 = held(0);
                        id1 = held(1);
                        ks = scale_of(0, id0, 0), vs = scale_of(0, id0, 1);
                    }
#pragma unroll 1
                    for (int c = 0; c < 2 * n; ++c) {
                        const int j = c >> 1, e = seq + c, r = 2 * e + half;
                        if (describes && (c & 1) == 0) {
                            const int id2 = held(j + 2);
                            const float ks1 = scale_of(j + 1, id1, 0), vs1 = scale_of(j + 1, id1, 1);
                            const uint32_t bits = __float_as_uint(vs);
                            item_e = max(item_e, (int)(__reduce_max_sync(0xffffffffu, bits) >> 23));
                            // log2 of the scale over the item's largest (far below it, where f16 holds nothing of the weight, the
                            // sum's share of it still counts); a power of two has no rest
                            const float below = (float)max((int)(bits >> 23) - item_e, -80);
                            float rest;
                            asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(rest) : "f"(__uint_as_float((bits & 0x7fffffu) | 0x3f800000u)));
                            TileInfo& ti = info[(e / 2) % F::kInfos];
                            if (lane < 8) ti.part[lane] = make_float4(ks, kLift + below + rest, ex2(-kLift - below) * ex2(-rest), 0.f);
                            if (lane == 0) ti.v = __uint_as_float((uint32_t)item_e << 23);
                            __syncwarp();
                            id1 = id2, ks = ks1, vs = vs1;
                        }
                        ok = warp_wait(&raw_full[r % F::RS], r / F::RS) && (e < F::ST || warp_wait(&empty[2 * (e % F::ST) + half], e / F::ST - 1));
                        if (!ok) break;
                        const unsigned char* raw = raw0 + (r % F::RS) * F::kHalf;
                        unsigned char* to = to0 + (e % F::ST) * F::kTile;
                        const int left = x.hi - x.lo - j * kKeys - 64 * half - 8 * g0 - sub;   // tokens seen from this lane's first on
                        const bool part = __any_sync(0xffffffffu, left <= 48);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (g0 + stride * i >= 8) break;
                            uint4 u[kParts];
#pragma unroll
                            for (int h = 0; h < kParts; ++h)
                                u[h] = *reinterpret_cast<const uint4*>(raw + i * (8 * stride) * D + (h ^ turned) * 64);
                            if (part && 8 * stride * i >= left) {
#pragma unroll
                                for (int h = 0; h < kParts; ++h) u[h] = make_uint4(0, 0, 0, 0);
                            }
#pragma unroll
                            for (int h = 0; h < kParts; ++h) {
                                uint32_t y[8];
                                widen16(u[h], y);
                                unsigned char* row = to + i * (8 * stride) * 128 + (h ^ turned) * 16384;
                                *reinterpret_cast<uint4*>(row + chunk0) = make_uint4(y[0], y[1], y[2], y[3]);
                                *reinterpret_cast<uint4*>(row + chunk1) = make_uint4(y[4], y[5], y[6], y[7]);
                            }
                        }
                        proxy_fence();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&raw_empty[r % F::RS]), mbar_arrive(&full[2 * (e % F::ST) + half]);
                    }
                    seq += 2 * n;
                }
            }
        }
    } else {
        // ---- softmax of row tile a; this thread's row ----
        const int a = warp >> 2, r = tid & 127;
        const uint32_t trow = tbase + ((uint32_t)(32 * (warp & 3)) << 16);
        bool ok = true, first = true;
        int turn = 0, it = 0, g = 0;   // tiles of all items; steps of this row tile
        for (int at = begin; ok && next_segment<kTcRows, kTcUnit>(p, s_cum, at, end, x);) {
            if (first && tid == 0) describe_cut(p, x, begin, share);
            first = false;
            const int on = takes(turn), n = tiles_of(), it0 = it;
            it += n;
            if (!(on >> a & 1)) continue;
            const int rr = (on == 3 ? a * kRows : 0) + r;   // row of the item
            const bool valid = rr < x.rows;
            const int R = x.row0 + (valid ? rr : 0), qi = R / p.G;
            const int vis = min(x.rq.len, x.rq.len - x.rq.n + qi + 1);   // tokens that this row sees end here
            const int64_t at_o = (int64_t)(x.rq.first + qi) * p.Hq + x.h * p.G + (R - qi * p.G);
            const bool busy = __any_sync(0xffffffffu, valid);   // a warp without rows only keeps the barriers going
            // Q, its tile free since the last item's last scores: a power of two times the row, negated where the scale is
            // negative, so that a maximum of scores is one of products
            float row_scale = 0.f;
            if (n > 0) {
                // a warp loads its own 32 rows, 16 bytes a lane, as many rows at a time as its lanes cover (each lane knows
                // one row's address)
                constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
                // (past the rows: the item's first row once more, whose results are not stored)
                const int64_t own = (int64_t)(x.rq.first + qi) * p.q_stride + (int64_t)(x.h * p.G + (R - qi * p.G)) * D;
                const int c = lane % kLanes, rows = __popc(__ballot_sync(0xffffffffu, valid));
                for (int k0 = 0; k0 < rows; k0 += 8 * kAtOnce) {   // (rolled, for the instruction cache)
                    uint4 y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int64_t off = __shfl_sync(0xffffffffu, own, k0 + i * kAtOnce + lane / kLanes);
                        y[i] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + off + 8 * c);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint32_t top = __vmaxu2(__vmaxu2(y[i].x & 0x7fff7fffu, y[i].y & 0x7fff7fffu),
                                                __vmaxu2(y[i].z & 0x7fff7fffu, y[i].w & 0x7fff7fffu));
#pragma unroll
                        for (int o = kLanes / 2; o > 0; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
                        const int e = max((int)(max(top & 0xffffu, top >> 16) >> 7) - 127, -100);
                        const float f = __uint_as_float((uint32_t)(14 - min(e, 127) + 127) << 23);
                        const int first = k0 + i * kAtOnce;
                        const float fr = __shfl_sync(0xffffffffu, f, ((lane - first) & (kAtOnce - 1)) * kLanes);
                        if (lane >= first && lane < first + kAtOnce) row_scale = fr;
                        const float g = p.scale_log2 < 0.f ? -f : f;
                        const uint32_t w[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
                        uint32_t z[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            z[k] = half2(__uint_as_float(w[k] << 16) * g, __uint_as_float(w[k] & 0xffff0000u) * g);
                        const int row = (r & 96) + first + lane / kLanes;
                        *reinterpret_cast<uint4*>(smem + a * F::kTile + (c >> 3) * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4)) =
                            make_uint4(z[0], z[1], z[2], z[3]);
                    }
                }
                row_scale = valid ? fabsf(p.scale_log2) / row_scale : 0.f;
                proxy_fence();
                mbar_arrive(&q_ready[a]);
            }
            float m = -INFINITY, item_v = 0.f;
            float2 la = make_float2(0.f, 0.f), lb = la;
            for (int j = 0; j < 2 * n; ++j, ++g) {
                ok = warp_wait(&s_full[2 * a + (g & 1)], g >> 1);
                if (!ok) break;
                tc_fence_after();
                if (busy) {
                    const int seen = valid ? vis - x.lo - j * 64 : 64;
                    const bool hide = __any_sync(0xffffffffu, seen < 64);
                    const TileInfo& ti = info[(it0 + j / 2) % F::kInfos];
                    const uint32_t ts = trow + a * 128 + (g & 1) * 64, to = trow + F::kO + a * D;
                    do {
                        float s0[32], s1[32];
                        tmem_ld32x2(ts, ts + 32, s0, s1);
                        if (hide) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                if (i >= seen) s0[i] = -INFINITY;
                                if (32 + i >= seen) s1[i] = -INFINITY;
                            }
                        }
                        const float4* parts = ti.part + 4 * (j & 1);
                        float top = -INFINITY;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float* s = (k < 2 ? s0 : s1) + 16 * (k & 1);
                            float t0 = fmaxf(s[0], s[1]), t1 = fmaxf(s[8], s[9]);
#pragma unroll
                            for (int i = 2; i < 8; i += 2) t0 = fmaxf(fmaxf(t0, s[i]), s[i + 1]), t1 = fmaxf(fmaxf(t1, s[8 + i]), s[9 + i]);
                            top = fmaxf(top, fmaxf(t0, t1) * fmaxf(row_scale * parts[k].x, kTiny));
                        }
                        const bool rise = valid && (top - m > kRise || m == -INFINITY), grow = ti.v > item_v;   // (m + kRise may round up)
                        if (__any_sync(0xffffffffu, rise || grow)) {
                            // by a power of two: exact for l and O; far from zero by what m rises, there as exact
                            const float up = ceilf(top - m);   // (infinite for a first maximum)
                            const bool anew = !(up <= 100.f), far = fabsf(top) > kFar;
                            const float f = !rise ? 1.f : anew ? 0.f : ex2(far ? m - top : -up);
                            if (rise) m = anew || far ? top : m + up;
                            la = make_float2(la.x * f, la.y * f), lb = make_float2(lb.x * f, lb.y * f);
                            float fo = f;
                            if (grow) fo *= item_v / ti.v, item_v = ti.v;
                            if (j > 0) ok = warp_wait(&pv_done[a], g - 1), tc_fence_after(), rescale(to, D / 16, fo);
                        }
                        const float base = m == -INFINITY ? 0.f : m;
                        if (__any_sync(0xffffffffu, fabsf(base) > kFar)) {
#pragma unroll 1
                            for (int k = 0; k < 4; ++k) la.x += far_weights(ts, k, seen, row_scale, base, parts[k]);
                            break;
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float* s = (k < 2 ? s0 : s1) + 16 * (k & 1);
                            const float4 f4 = parts[k];
                            const float fx = fmaxf(row_scale * f4.x, kTiny), fb = f4.y - base;
                            const float2 scale2 = make_float2(fx, fx), base2 = make_float2(fb, fb), drop2 = make_float2(f4.z, f4.z);
                            uint32_t w[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                float2 e = __ffma2_rn(make_float2(s[2 * i], s[2 * i + 1]), scale2, base2);
                                e = make_float2(ex2(e.x), ex2(e.y));
                                if (i & 1) lb = __ffma2_rn(e, drop2, lb);
                                else la = __ffma2_rn(e, drop2, la);
                                w[i] = half2(e.x, e.y);
                            }
                            tmem_st8(ts + 8 * k, w);
                        }
                    } while (false);
                    tmem_st_wait();
                }
                // The item's end waits for its last step's product.  A barrier tells a phase from the next one only, so the one before is
                // waited for here; elsewhere the scores of step g are made behind the product of step g - 2.
                if (j == 2 * n - 1) ok = warp_wait(&pv_done[a], g - 1);
                if (!ok) break;
                tc_fence_before();
                mbar_arrive(&p_ready[2 * a + (g & 1)]);
            }
            if (!ok) break;
            if (n > 0) {
                ok = warp_wait(&pv_done[a], g - 1);
                if (!ok) break;
                tc_fence_after();
            }
            if (!busy) continue;
            const float l = (la.x + la.y) + (lb.x + lb.y);
            const bool some = l != 0.f, whole = x.whole();
            const float unit = item_v * 0.0078125f;   // of O: 2^-kLift
            const float inv = some ? unit / l : 0.f;
            const int64_t part = x.slot() * kTcRows + rr;
            if (valid && !whole) p.part_ml[part] = make_float2(m, l);
            if (valid && whole && p.lse) p.lse[at_o] = some ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
            const bool wide = (reinterpret_cast<uintptr_t>(p.o) & 31) == 0;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                float o[32];
                if (n > 0) {
                    tmem_ld32(trow + F::kO + a * D + 32 * c, o);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0.f;
                }
                if (valid && whole) {
                    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) + at_o * D + 32 * c;
#pragma unroll
                    for (int i = 0; i < 32; i += 16) {
                        uint32_t u[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            u[k] = some ? pack2(o[i + 2 * k] * inv, o[i + 2 * k + 1] * inv) : 0u;
                        store32(dst + i, u, wide);
                    }
                } else if (valid) {
                    float* dst = p.part_o + part * D + 32 * c;
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        uint32_t u[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) u[k] = __float_as_uint(o[i + k] * unit);
                        store32(dst + i, u, true);
                    }
                }
            }
        }
    }

    // ---- leave only with no copy and no product still writing into this CTA's shared memory or TMEM ----
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *abort_flag) {
        const uint64_t drain = limit > kDrainLimitNs ? limit : kDrainLimitNs;
        for (int e = max(0, *issued - F::RS); e < *issued; ++e)
            tc::drain_phase(&raw_full[e % F::RS], (uint32_t)((e / F::RS) & 1), drain);
        tc::drain_phase(&end_bar[0], 0, drain), tc::drain_phase(&end_bar[1], 0, drain);
        atomicOr(p.status, STATUS_TIMEOUT);
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(512));
}

template <int D>
cudaError_t launch(const PagedParams& p, cudaStream_t s) {
    using F = Cfg<D>;
    static std::atomic<int> optin[kMaxOptinDevices];
    const cudaError_t e = smem_optin(reinterpret_cast<const void*>(paged_tc_kernel<D>), F::kSmem, optin);
    if (e != cudaSuccess) return e;
    paged_tc_kernel<D><<<p.ctas, kThreads, F::kSmem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_tc(const PagedParams& p, int D, cudaStream_t s) { return D == 64 ? launch<64>(p, s) : launch<128>(p, s); }

}  // namespace cache
}  // namespace gdn
