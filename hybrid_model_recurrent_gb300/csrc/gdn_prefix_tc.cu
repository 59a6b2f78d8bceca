// gdn_prefix_tc.cu - attention for a batch that shares a long prefix, on the 5th-generation tensor cores (bf16,
// head_dim 64 or 128).
//
// A CTA takes NT tiles of 128 query rows of one key/value head (stacked over requests, queries and the heads of the
// group) against a range of the prefix, a range of one request's tail, or both in turn, in tiles of 128 tokens:
//     S = Q K^T  (TMEM, fp32)  ->  P = 2^(x - m) (bf16, over S's own columns)  ->  O += P V  (TMEM, fp32)
// one pass over keys and values with each row's running maximum m and sum l.  A thread owns a row, so the statistics
// need no exchange.  O is rescaled only when a row's maximum has risen by more than 2^8 since m was set: until then the
// weights are at most 2^8 and only their common scale differs.  Scores, statistics and sums are fp32; the weights are
// rounded to bf16 for the product (half a step, 2^-8 of each weight), as the tensor cores take them.
//
// Roles: warps 0 .. 4 NT - 1 softmax (one warpgroup a row tile), then a warp that issues products and one copying thread.
// K and V tiles arrive by TMA in a ring of ST tiles; with NT = 2 both row tiles use each tile, and one tile's softmax
// runs beside the other's products (an item of at most 128 rows uses one).  With NT = 1 two CTAs share a multiprocessor and
// overlap each other instead.  A CTA takes one item after the other, the copies running ahead into the next one.
//
// What bounds it: where queries are many, a tile's chain of product, softmax and product (16 requests x 256 tokens x 32
// heads on 16384 + 700 tokens, d = 128: 784 us, 1440 TFLOP/s, 0.76 of a library product's rate); where they are few, the
// reading of the prefix and the start and end of each CTA (64 x 32 heads on 32768 + 1024 tokens: 74 us, 3.6 TB/s).
//
// A masked token's score is replaced (not multiplied), and value rows past the range are zeroed in shared memory
// before the product, so nothing that lies past a tail's end reaches a result.
//
// Every wait is bounded: a role that gives up sets the CTA's abort flag and the sticky status, every role leaves its
// loop, copies and products in flight are waited for, and TMEM is freed.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "gdn_prefix.cuh"
#include "gdn_tc_util.cuh"

namespace gdn {
namespace prefix {
namespace {

using tc::idesc;
using tc::proxy_fence;
using tc::sw128;
using tc::tc_fence_after;
using tc::tc_fence_before;
using tc::tmem_ld32;
using tc::tmem_ld32x2;
using tc::tmem_st16;
using tc::tmem_st32;
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
using tcu::wait_bar;
using tcu::warp_wait_bar;

constexpr int kRows = 128;   // rows of a tile
constexpr int kKeys = 128;   // tokens of a tile
constexpr float kRise = 8.f; // O is rescaled when a maximum has risen by more than this (log2)
// A weight's exponent is score * scale - m in one rounding, but m is a product already rounded: for the largest score its
// rounding error is left, half a step of m, 16 at 2^28 and past what an exponential holds from 2^31 on.  Rows further from zero
// than this round the product by itself first.
constexpr float kFar = 268435456.f;

template <int D, int NT>
struct Cfg {
    static constexpr int kTile = kKeys * D * 2;                            // bytes of a K, V or Q tile
    static constexpr int ST = NT == 2 ? (D == 128 ? 5 : 8) : (D == 128 ? 2 : 5);
    static constexpr int kRing = NT * kTile;                               // after the Q tiles
    static constexpr int kBar = kRing + ST * kTile;
    static constexpr int kSmem = kBar + 512 + 1024;
    // softmax warpgroups, then a warp that issues products and one that issues copies; with NT = 2 two idle warps fill up
    // their warpgroup, which then hands registers to the others
    static constexpr int kThreads = NT == 2 ? 384 : 192;
    static constexpr int kTmem = NT == 2 ? 512 : 256;
    static constexpr uint32_t kO = NT * 128;                               // TMEM: S of each row tile, then O of each
    static_assert(kSmem <= 232448 / (NT == 1 ? 2 : 1) - (NT == 1 ? 1024 : 0), "shared memory");
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* tm, int x, int y, int z, int w, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
        : "memory");
}
// What one item computes: rows [row0, row0 + NT 128) of `rows`, against prefix tokens [lo1, hi1) and tail tokens
// [lo2, hi2) of request b0, in n_tiles tiles, the first n1 of them the prefix's.
struct Item {
    bool stacked;   // rows of all requests (prefix only), else one request's
    int na;         // row tiles that hold rows
    int h, b0, part, len, lo1, hi1, lo2, hi2, rows, row0, n1, n_tiles;
};
template <int NT>
__device__ __forceinline__ Item item_at(const Params& p, int item, int pre_items, bool joined) {
    Item x;
    const int nG = (int)p.by_ng.d;
    x.stacked = item < pre_items;
    x.b0 = x.len = x.lo1 = x.hi1 = x.lo2 = x.hi2 = 0;
    int tile;
    if (x.stacked) {
        item = p.by_hkv.divmod(item, &x.h);
        x.part = p.by_pre_tiles.divmod(item, &tile);
        x.rows = p.B * nG;
        x.lo1 = x.part * p.pre_chunk;
        x.hi1 = (int)min((int64_t)x.lo1 + p.pre_chunk, p.prefix_len);
    } else {
        item = p.by_hkv.divmod(item - pre_items, &x.h);
        item = p.by_tail_tiles.divmod(item, &tile);
        x.part = p.by_b.divmod(item, &x.b0);
        x.rows = nG;
        x.len = p.max_tail > 0 ? min(max(p.tail_len[x.b0], 0), (int)p.max_tail) : 0;
        if (joined) {
            x.hi1 = (int)p.prefix_len;
            // what the tile's last row sees
            const int last = p.by_g.div(min((tile + 1) * NT * kRows, x.rows) - 1);
            x.hi2 = min(x.len, max(0, x.len - p.n + last + 1));
        } else {
            tail_range(p, x.len, kKeys, x.part, &x.lo2, &x.hi2);
        }
        x.part += p.pre_splits;
    }
    x.row0 = tile * (NT * kRows);
    x.na = NT == 1 || x.rows - x.row0 <= kRows ? 1 : 2;
    x.n1 = (x.hi1 - x.lo1 + kKeys - 1) / kKeys;
    x.n_tiles = x.n1 + (x.hi2 - x.lo2 + kKeys - 1) / kKeys;
    return x;
}

// The weights of a tile's row, over its own scores in TMEM, for rows far from zero; returns their sum.  A function by itself:
// inlined, it made the kernel 4 % slower where no row is far (turns of 16 x 256 tokens: 806 us against 778), a call 1 % (787).
__device__ __noinline__ float far_weights(uint32_t taddr, int seen, float scale, float base) {
    float sum = 0.f;
#pragma unroll 1
    for (int c = 0; c < kKeys / 32; ++c) {
        float x[32];
        uint32_t w[16];
        tmem_ld32(taddr + 32 * c, x);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float y = __fsub_rn(__fmul_rn(x[i], scale), base);
            x[i] = 32 * c + i < seen ? ex2(y) : 0.f;
            sum += x[i];
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = pack2(x[2 * i], x[2 * i + 1]);
        tmem_st16(taddr + 16 * c, w);
    }
    return sum;
}

template <int D, int NT>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, NT == 1 ? 2 : 1)
    prefix_tc_kernel(const __grid_constant__ Params p, const int pre_items, const bool joined, const bool direct) {
    using F = Cfg<D, NT>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_addr(smem);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + F::kBar);   // [ST] a K or V tile landed
    uint64_t* empty = full + F::ST;                                  // [ST] every product that reads it is done
    uint64_t* s_full = empty + F::ST;                                // [NT] S (and every earlier product) done
    uint64_t* p_ready = s_full + NT;                                 // [NT] P written, O rescaled, V's end zeroed
    uint64_t* q_ready = p_ready + NT;                                // [NT] an item's Q tile written
    uint64_t* o_full = q_ready + NT;                                 // [NT] every product of an item done
    uint32_t* tslot = reinterpret_cast<uint32_t*>(o_full + NT);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
    int* issued = reinterpret_cast<int*>(tslot + 2);                 // tiles whose copy was issued; items asked for
    uint64_t* end = reinterpret_cast<uint64_t*>(tslot + 4);          // every product done
    uint64_t* q_asked = end + 1;                                     // the first item's Q loads are under way
    uint64_t* n_full = q_asked + 1;                                  // [2] an item's description written
    uint64_t* n_empty = n_full + 2;                                  // [2] and read by every role
    uint64_t* answered = n_empty + 2;                                // the answer to a request for another item
    uint4* answer = reinterpret_cast<uint4*>((reinterpret_cast<uintptr_t>(answered + 1) + 15) & ~(uintptr_t)15);
    Item* described = reinterpret_cast<Item*>(answer + 1);           // [2]
    static_assert((2 * F::ST + 4 * NT) * 8 + 32 + 5 * 8 + 32 + 2 * sizeof(Item) <= 512, "barrier area");

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint64_t limit = p.wait_limit_ns;

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tslot)),
                     "r"(F::kTmem));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (warp == NT * 4 + 1 && lane == 0) {   // the descriptors that there are: none without a prefix, none without tails
        for (const CUtensorMap* tm : {&p.tm_kp, &p.tm_vp, &p.tm_kt, &p.tm_vt})
            if (tm == &p.tm_kp || tm == &p.tm_vp ? p.prefix_len > 0 : p.max_tail > 0)
                asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tm)) : "memory");
    }
    if (tid == 0) {
        for (int i = 0; i < F::ST; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
        for (int i = 0; i < NT; ++i) {
            mbar_init(&s_full[i], 1), mbar_init(&p_ready[i], 128);
            mbar_init(&q_ready[i], 128), mbar_init(&o_full[i], 1);
        }
        mbar_init(end, 1);
        mbar_init(q_asked, NT * 128);
        for (int i = 0; i < 2; ++i) mbar_init(&n_full[i], 1), mbar_init(&n_empty[i], 1 + 4 * NT);
        mbar_init(answered, 1);
        *abort_flag = 0;
        issued[0] = issued[1] = 0;
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tslot;
    auto warp_wait = [&](uint64_t* bar, int parity) { return warp_wait_bar(bar, (uint32_t)parity & 1u, abort_flag, limit); };

    // 384 threads start with 168 registers each (64512 in all): 256 x 200 + 128 x 96 = 63488
    constexpr bool kKeep = NT == 2;   // a row's 128 scores stay in registers between the maximum and the weights

    // The grid has a CTA an item, and a running CTA takes over items whose CTAs have not started (cluster launch control):
    // lengths differ, and the items of a fixed share of them summed up to a third more for the unluckiest CTA.  The copying
    // thread asks for the next item while it copies one, and describes each item to the other roles ahead of time.
    auto next_item = [&](int n, Item& x) {   // the CTA's n-th item, for a warp; false: no more, or given up
        if (!warp_wait(&n_full[n & 1], n >> 1)) return false;
        x = described[n & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(&n_empty[n & 1]);
        return x.n_tiles >= 0;
    };

    // An item of at most 128 rows takes one row tile; with two, such items take them in turn (every role counts alike), so
    // that one tile's sums leave and its next Q arrives, 6000 cycles, while the other tile computes.
    auto takes = [&](const Item& x, int& turn) {
        const int one = turn;
        if (NT == 2 && x.na == 1) turn ^= 1;
        return x.na == 2 ? 3 : 1 << one;   // bit a: row tile a
    };

    // Every role walks the CTA's items; tiles are counted through all of them (it: tiles so far, K of tile i is copy 2 i,
    // V copy 2 i + 1), so the copies of the next item begin while the last one is still computed.
    if (warp >= NT * 4) {
        if constexpr (kKeep) asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        if (warp == NT * 4) {
            // ---- products (the whole warp walks along, one elected lane issues) ----
            auto slot_at = [&](int seq) { return sbase + F::kRing + (uint32_t)(seq % F::ST) * F::kTile; };
            auto landed = [&](int seq) { return warp_wait(&full[seq % F::ST], seq / F::ST); };
            auto done = [&](uint64_t* bar) {
                if (elect_one()) umma_commit(bar);
            };
            bool ok = true;
            int it = 0, turn = 0, tiles[NT] = {}, nth[NT] = {};   // tiles of the ring; tiles and items of each row tile
            Item x;
            for (int nn = 0; ok && next_item(nn, x); ++nn) {
                const int n = x.n_tiles, on = takes(x, turn), last = on >> 1;
                if (n == 0) continue;
                auto scores = [&](int a, int i) {
                    const uint64_t q = tile_desc(sbase + a * F::kTile, false), k = tile_desc(slot_at(2 * i), false);
                    if (elect_one()) {
#pragma unroll
                        for (int s = 0; s < D / 16; ++s)
                            umma_ss(tbase + a * 128, cols_step(q, s), cols_step(k, s), idesc(kKeys, false, false), s > 0);
                        umma_commit(&s_full[a]);
                        if (a == last) umma_commit(&empty[2 * i % F::ST]);
                    }
                };
                ok = landed(2 * it);
#pragma unroll
                for (int a = 0; a < NT; ++a) {
                    if (!(on >> a & 1)) continue;
                    ok = ok && warp_wait(&q_ready[a], nth[a]);
                    if (ok) scores(a, it);
                }
                for (int j = 0; ok && j < n; ++j) {
                    const int i = it + j, vs = 2 * i + 1;
                    ok = landed(vs);
#pragma unroll
                    for (int a = 0; a < NT; ++a) {
                        if (!(on >> a & 1)) continue;
                        ok = ok && warp_wait(&p_ready[a], tiles[a] + j);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t v = tile_desc(slot_at(vs), true);
                        if (elect_one()) {
#pragma unroll
                            for (int s = 0; s < kKeys / 16; ++s)
                                umma_ts(tbase + F::kO + a * D, tbase + a * 128 + 8 * s, rows_step(v, s), idesc(D, false, true),
                                        j > 0 || s > 0);
                            if (a == last) umma_commit(&empty[vs % F::ST]);
                        }
                        if (j + 1 < n) {
                            ok = landed(2 * i + 2);
                            if (!ok) break;
                            scores(a, i + 1);
                        } else {
                            done(&o_full[a]);
                        }
                    }
                }
                it += n;
#pragma unroll
                for (int a = 0; a < NT; ++a)
                    if (on >> a & 1) tiles[a] += n, ++nth[a];
            }
            done(end);   // also after giving up: the end waits for the products in flight
        } else if (warp == NT * 4 + 1) {
            // ---- copies ----
            if (lane == 0) {
                bool ok = true;
                int seq = 0;   // (the copies of a whole wave, asked for first, keep the Q loads waiting for 5 us)
                int item = blockIdx.x;
                for (int nn = 0; ok; ++nn) {
                    const int k = nn & 1;
                    if (nn >= 2) ok = wait_bar(&n_empty[k], (uint32_t)(nn / 2 - 1) & 1u, abort_flag, limit);
                    if (!ok) break;
                    Item x;
                    if (item >= 0) x = item_at<NT>(p, item, pre_items, joined);
                    else x.n_tiles = -1;
                    described[k] = x;
                    mbar_arrive(&n_full[k]);
                    if (item < 0) break;
                    // Asked for once the item's first copy is under way: a CTA that has only just started would take over
                    // what the next multiprocessor is about to start.
                    auto ask = [&] {
                        proxy_fence();   // the last answer has been read
                        mbar_arrive_expect_tx(answered, 16);
                        asm volatile(
                            "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::
                                "r"(smem_addr(answer)),
                            "r"(smem_addr(answered))
                            : "memory");
                        issued[1] = nn + 1;
                    };
                    for (int c = 0; c < 2 * x.n_tiles; ++c, ++seq) {
                        const int s = seq % F::ST, j = c >> 1;
                        ok = !(p.stall_after >= 0 && seq / 2 >= p.stall_after) &&   // testing hook
                             (seq > 0 || wait_bar(q_asked, 0, abort_flag, limit)) &&
                             (seq < F::ST || wait_bar(&empty[s], (uint32_t)((seq / F::ST - 1) & 1), abort_flag, limit));
                        if (!ok) break;
                        unsigned char* dst = smem + F::kRing + s * F::kTile;
                        mbar_arrive_expect_tx(&full[s], F::kTile);
                        const bool v = c & 1;
#pragma unroll
                        for (int y = 0; y < D / 64; ++y) {
                            if (j < x.n1)
                                tma_load_3d(dst + y * 16384, v ? &p.tm_vp : &p.tm_kp, y * 64, x.h, x.lo1 + j * kKeys, &full[s]);
                            else
                                tma_load_4d(dst + y * 16384, v ? &p.tm_vt : &p.tm_kt, y * 64, x.h, x.lo2 + (j - x.n1) * kKeys, x.b0,
                                            &full[s]);
                        }
                        *issued = seq + 1;
                        if (c == 0) ask();
                    }
                    if (x.n_tiles == 0) ask();
                    ok = ok && wait_bar(answered, (uint32_t)nn & 1u, abort_flag, limit);
                    if (!ok) break;
                    uint32_t some, first;
                    asm volatile(
                        "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\tld.shared.b128 r, [%2];\n\t"
                        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\tselp.u32 %0, 1, 0, p;\n\t"
                        "mov.u32 %1, 0;\n\t"
                        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
                        : "=r"(some), "=r"(first)
                        : "r"(smem_addr(answer))
                        : "memory");
                    item = some ? (int)first : -1;
                }
            }
        }
    } else {
        // ---- softmax of row tile a; this thread's row ----
        if constexpr (kKeep) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        const int a = warp >> 2, r = tid & 127;
        const uint32_t trow = tbase + ((uint32_t)(32 * (warp & 3)) << 16);
        // (a scale of 0 as the smallest normal number: every weight is 1, and a hidden token's -infinity stays that)
        const float scale = fmaxf(fabsf(p.scale_log2), 1.17549435e-38f);
        const int nG = (int)p.by_ng.d;
        bool ok = true, first = true;
        int it = 0, turn = 0, mine = 0, nth = 0;   // tiles of the ring, of this row tile, its items
        Item x;
        for (int nn = 0; ok && next_item(nn, x); ++nn) {
            const int on = takes(x, turn);
            if (!(on >> a & 1)) {   // no rows for this row tile
                if (first && x.n_tiles > 0) mbar_arrive(q_asked), first = false;
                it += x.n_tiles;
                continue;
            }
            const int R = x.row0 + (on == 3 ? a * kRows : 0) + r;
            const bool valid = R < x.rows;
            int e, g;
            const int bs = p.by_ng.divmod(R, &e), b = x.stacked ? bs : x.b0;   // (one request's rows are below n G, or invalid)
            const int qi = p.by_g.divmod(e, &g), head = x.h * p.G + g;
            const int vis2 = min(x.hi2, max(0, x.len - p.n + qi + 1));   // tail tokens that this row sees end here
            const int64_t at = ((int64_t)b * p.n + qi) * p.Hq + head;
            const bool busy = __any_sync(0xffffffffu, valid);   // a warp without rows only keeps the barriers going
            // Q, its tile free since the last item's last scores; negated where the scale is negative, so that a maximum of
            // scores is one of products
            if (x.n_tiles > 0) {
                // a warp loads its own 32 rows, 16 bytes a lane, as many rows at a time as its lanes cover (each lane knows
                // one row's address)
                constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
                const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
                // past the rows: the item's first row once more, whose results are not stored (its address is good, and
                // no load waits for a condition)
                const int64_t own = valid ? b * p.q_sb + qi * p.q_sn + head * p.q_sh
                                          : (x.stacked ? 0 : b * p.q_sb) + (int64_t)x.h * p.G * p.q_sh;
                const int c = lane % kLanes, rows = __popc(__ballot_sync(0xffffffffu, valid));
                for (int k0 = 0; k0 < rows; k0 += 8 * kAtOnce) {   // (rolled, for the instruction cache)
                    uint4 y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int64_t off = __shfl_sync(0xffffffffu, own, k0 + i * kAtOnce + lane / kLanes);
                        y[i] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + off + 8 * c);
                    }
                    if (first && k0 + 8 * kAtOnce >= rows) mbar_arrive(q_asked);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int row = (r & 96) + k0 + i * kAtOnce + lane / kLanes;
                        *reinterpret_cast<uint4*>(smem + a * F::kTile + (c >> 3) * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4)) =
                            make_uint4(y[i].x ^ flip, y[i].y ^ flip, y[i].z ^ flip, y[i].w ^ flip);
                    }
                }
                if (first && rows == 0) mbar_arrive(q_asked);
                first = false;
                proxy_fence();
                mbar_arrive(&q_ready[a]);
            }
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < x.n_tiles; ++j, ++it, ++mine) {
                const int t0 = j < x.n1 ? x.lo1 + j * kKeys : x.lo2 + (j - x.n1) * kKeys;
                ok = warp_wait(&s_full[a], mine);
                if (!ok) break;
                tc_fence_after();
                if (busy) {
                    // With NT = 2 a row's scores stay in registers; with NT = 1 (two CTAs of 6 warps and 168 registers a
                    // thread) they are read again for the weights.
                    const int seen = valid ? (j < x.n1 ? x.hi1 : vis2) - t0 : kKeys;
                    const bool hide = __any_sync(0xffffffffu, seen < kKeys);
                    float s[kKeep ? 4 : 2][32];
                    auto load = [&](int half, float (&s0)[32], float (&s1)[32]) {
                        tmem_ld32x2(trow + a * 128 + 64 * half, trow + a * 128 + 64 * half + 32, s0, s1);
                        if (hide) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                if (64 * half + i >= seen) s0[i] = -INFINITY;
                                if (64 * half + 32 + i >= seen) s1[i] = -INFINITY;
                            }
                        }
                    };
                    float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        float(&s0)[32] = s[kKeep ? 2 * half : 0], (&s1)[32] = s[kKeep ? 2 * half + 1 : 1];
                        load(half, s0, s1);
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            t[0] = fmaxf(fmaxf(t[0], s0[i]), s0[i + 1]);
                            t[1 + (i & 2)] = fmaxf(fmaxf(t[1 + (i & 2)], s1[i]), s1[i + 1]);
                        }
                    }
                    const float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * scale;
                    const bool rise = valid && (top > m + kRise || m == -INFINITY);
                    if (__any_sync(0xffffffffu, rise)) {
                        const float mn = rise ? fmaxf(m, top) : m;
                        const float f = mn == -INFINITY ? 1.f : ex2(m - mn);
                        m = mn;
                        l *= f;
                        if (j > 0) {   // every earlier product into O is done: s_full came after them
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                float o[32];
                                tmem_ld32(trow + F::kO + a * D + 32 * c, o);
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] *= f;
                                tmem_st32(trow + F::kO + a * D + 32 * c, o);
                            }
                        }
                    }
                    const float base = m == -INFINITY ? 0.f : m;
                    const float2 scale2 = make_float2(scale, scale), base2 = make_float2(-base, -base);
                    float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
                    if (__any_sync(0xffffffffu, fabsf(base) > kFar)) {
                        sum0.x = far_weights(trow + a * 128, seen, scale, base);
                    } else {
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            float(&s0)[32] = s[kKeep ? 2 * half : 0], (&s1)[32] = s[kKeep ? 2 * half + 1 : 1];
                            if (!kKeep) load(half, s0, s1);
                            uint32_t w0[16], w1[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                float2 e = __ffma2_rn(make_float2(s0[2 * i], s0[2 * i + 1]), scale2, base2);
                                float2 g = __ffma2_rn(make_float2(s1[2 * i], s1[2 * i + 1]), scale2, base2);
                                e = make_float2(ex2(e.x), ex2(e.y)), g = make_float2(ex2(g.x), ex2(g.y));
                                sum0 = __fadd2_rn(sum0, e), sum1 = __fadd2_rn(sum1, g);
                                w0[i] = pack2(e.x, e.y), w1[i] = pack2(g.x, g.y);
                            }
                            tmem_st16(trow + a * 128 + 32 * half, w0);
                            tmem_st16(trow + a * 128 + 32 * half + 16, w1);
                        }
                    }
                    l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
                    tmem_st_wait();
                }
                if ((a == 0 || on != 3) && j >= x.n1 && t0 + kKeys > x.hi2) {
                    // the tail's last tile: zero the value rows past the range
                    const int vs = 2 * it + 1;
                    ok = warp_wait(&full[vs % F::ST], vs / F::ST);
                    if (!ok) break;
                    if (r >= x.hi2 - t0) {
                        unsigned char* v = smem + F::kRing + (vs % F::ST) * F::kTile + r * 128;
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                *reinterpret_cast<uint4*>(v + c * 16384 + 16 * i) = make_uint4(0, 0, 0, 0);
                    }
                    proxy_fence();
                }
                tc_fence_before();
                mbar_arrive(&p_ready[a]);
            }
            if (!ok) break;
            if (x.n_tiles > 0) {
                ok = warp_wait(&o_full[a], nth++);
                if (!ok) break;
                tc_fence_after();
            }
            if (!busy) continue;
            const bool some = l != 0.f;
            const float inv = some ? 1.f / l : 0.f;
            const int64_t group = part_group(p, x.part, x.h, x.stacked ? R : x.b0 * nG + R);
            const int in_group = (x.stacked ? R : x.b0 * nG + R) & 31;
            if (valid && !direct) p.part_ml[group * 32 + in_group] = make_float2(m, l);
            if (valid && direct && p.lse) p.lse[at] = some ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
            if (x.n_tiles == 0 && !direct) continue;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                float o[32];
                if (x.n_tiles > 0) {
                    tmem_ld32(trow + F::kO + a * D + 32 * c, o);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0.f;
                }
                if (valid && direct) {
                    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) + at * D + 32 * c;
                    const bool wide = (reinterpret_cast<uintptr_t>(p.o) & 31) == 0;
#pragma unroll
                    for (int i = 0; i < 32; i += 16) {
                        uint32_t u[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            u[k] = some ? pack2(o[i + 2 * k] * inv, o[i + 2 * k + 1] * inv) : 0u;
                        store32(dst + i, u, wide);
                    }
                } else if (valid) {
                    float* dst = p.part_o + (group * D + 32 * c) * 32 + in_group;
#pragma unroll
                    for (int i = 0; i < 32; ++i) dst[32 * i] = o[i];
                }
            }
        }
    }

    // ---- leave only with no copy and no product still writing into this CTA's shared memory or TMEM ----
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
        if (*abort_flag) {
            const uint64_t drain = limit > kDrainLimitNs ? limit : kDrainLimitNs;
            for (int seq = max(0, *issued - F::ST); seq < *issued; ++seq)
                tc::drain_phase(&full[seq % F::ST], (uint32_t)((seq / F::ST) & 1), drain);
            if (issued[1] > 0)
                tc::drain_phase(answered, (uint32_t)(issued[1] - 1) & 1u, drain);
            tc::drain_phase(end, 0, drain);
            atomicOr(p.status, STATUS_TIMEOUT);
        }
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(F::kTmem));
}

template <int D, int NT>
cudaError_t launch(const Params& p, int64_t pre_items, int64_t tail_items, bool joined, bool direct, cudaStream_t s) {
    using F = Cfg<D, NT>;
    if (pre_items + tail_items == 0) return cudaSuccess;
    auto kern = prefix_tc_kernel<D, NT>;
    static std::atomic<int> optin[kMaxOptinDevices];
    const cudaError_t e = smem_optin(reinterpret_cast<const void*>(kern), F::kSmem, optin);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)(pre_items + tail_items), F::kThreads, F::kSmem, s>>>(p, (int)pre_items, joined, direct);
    return cudaGetLastError();
}
template <int D>
cudaError_t launch_d(const Params& p, int row_tiles, int64_t pre_items, int64_t tail_items, bool joined, bool direct,
                     cudaStream_t s) {
    return row_tiles == 2 ? launch<D, 2>(p, pre_items, tail_items, joined, direct, s)
                          : launch<D, 1>(p, pre_items, tail_items, joined, direct, s);
}

}  // namespace

cudaError_t launch_tc(const Params& p, int D, int row_tiles, int64_t pre_items, int64_t tail_items, bool joined,
                      bool direct, cudaStream_t s) {
    return D == 64 ? launch_d<64>(p, row_tiles, pre_items, tail_items, joined, direct, s)
                   : launch_d<128>(p, row_tiles, pre_items, tail_items, joined, direct, s);
}

}  // namespace prefix
}  // namespace gdn
