// gdn_linear_tc.cu - linear attention with a decay for each head, chunked form on the 5th-generation tensor cores
// (d_k, d_v of 64 or 128, bf16 in and out).
//
//     S_t = a S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t
//
// regrouped over a chunk of n <= 128 tokens that starts from the state S (rows t, s = 0 .. n-1 of the chunk):
//
//     o_t = scale (a^{t+1} S q_t + sum_{s <= t} a^{t-s} (q_t . k_s) v_s)
//     S'  = a^n S + sum_s v_s (a^{n-1-s} k_s)^T
//
// Every power of a is at most 1, so no decay in [0, 1] leaves the range of fp32.  A chunk ends after 128 tokens, at a
// checkpoint and at the end of its job.  Products, all M = 128 with fp32 sums in TMEM:
//     G = Q K^T;  O = Q S^T, its rows scaled by a^{t+1} in place, O += P V with P = G masked and decayed;
//     V'^T K with V' = diag(a^{n-1-s}) V, added to a^n S in registers
// V' is not exact in bf16: it is split into hi - mid + lo (mid is formed negated and the product negates it back), 24 bits,
// all multiplied; and the tensor cores' sums, which are not rounded to nearest, run over one chunk only.  So a state is
// within 6e-7 of itself against 64 bits, as fp32 sums are; with two parts, and the sums running through all chunks, it was
// within 2.5e-6.  P and the copy of S that the readout multiplies are rounded to bf16 once
// (half a step, 2^-8 of each term): the readout itself is rounded to bf16, and its error stays of that order.
//
// What bounds it: shared memory's 128 bytes a cycle, of which a product with both operands there takes nearly all.  So
// P and V'^T are operands in TMEM: with K' = diag(.) K split in shared memory instead (written, and read again beside V),
// a chunk moved 590 KB through shared memory, now 430 KB, and the room of K' gives every input tile a second buffer.
//
// What it measured (d = 128): 8 x 16 scans of 8192 tokens with 16 checkpoints each, 1.22 GB in 207 us, 5.9 of the 6.7 TB/s
// that a copy reaches (128 of 152 multiprocessors have a scan); 2.9 us a chunk without a checkpoint, where the products need
// 1.6.  32 scans of 131072, cut into segments and read twice: 1.04 ms.
//
// One CTA takes one (job, head) from its first chunk to its last.  Roles:
//   state  (warps 0-3):  S, a row a thread, in registers: a^n S + the chunk's products; its bf16 copy; checkpoints,
//                        initial, final state; a^{t+1} into O; rows past a cut chunk zeroed
//   tokens (warps 4-7):  the first half of G's columns -> P and of V^T -> V', both in TMEM
//   output (warps 8-11): the second half of P and V'; O to memory, staged for TMA
// (without a readout the last two only form V', into two buffers in turn, so the next chunk's while this one's is multiplied)
//   one thread each that issues the products, the copies of K and V, of Q and of staged output
// They hand over through mbarriers, one phase a chunk, and no barrier completes a phase before everyone who waits for
// the last one has seen it (a parity tells only two phases apart).  The critical path is the products' own order: V' hi and
// mid of the next chunk are formed while P V and G are multiplied, lo waits in registers until G's columns are free, and the
// update starts before Q S^T does.  Each role's chunk is written as short rolled loops, the products' issue among them:
// unrolled, the roles' code streamed through the instruction cache once a chunk (24 products took 3600 cycles to issue
// instead of 1400).
//
// A sequence's tiles may reach past its end into its neighbour's tokens: P and V' are replaced by zeros there and the
// key and value rows are zeroed, so a neighbour's values, infinities and NaN included, never reach a result.
//
// Every wait is bounded: a role that gives up sets the abort flag, every role leaves, copies and products in flight
// are waited for, TMEM is freed and the sticky status is set.
#include <cuda_bf16.h>

#include "gdn_linear.cuh"
#include "gdn_tc_util.cuh"

namespace gdn {
namespace lin {
namespace {

using tc::idesc;
using tc::proxy_fence;
using tc::sw128;
using tc::tc_fence_after;
using tc::tc_fence_before;
using tc::tmem_ld32;
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

constexpr int kTok = 128;                   // tokens of a chunk
constexpr int kTile = kTok * 128 * 2;       // bytes of a tile: two 64-column blocks of [128][128 B] (one used at width 64)
constexpr int kThreads = 16 * 32;
constexpr int OFF_O = 5 * kTile;            // after the input tiles (with a readout): staged output
constexpr int OFF_S = 6 * kTile;            // the bf16 copy of S
constexpr int OFF_POW = 7 * kTile;          // a^0 .. a^128; a^128 .. a^0; a^127 .. a^0
constexpr int OFF_BAR = OFF_POW + 3 * 528;
constexpr int kSmem = OFF_BAR + 256 + 1024;
static_assert(kSmem <= 232448, "227 KB of shared memory per block");
// With a readout, P and V' lo go over G, each role's over the 64 columns of its tokens, which only it reads: P's two blocks
// of 32 tokens (16 columns each) first, then V' lo's.
__host__ __device__ constexpr uint32_t p_block(int cb) { return 128u + 16u * cb + (cb >= 2 ? 32u : 0u); }
constexpr uint32_t T_S = 0, T_G = 128, T_O = 256;
// V' hi, then mid; without a readout the columns of G and O give room to two whole V', and the next one is formed during an update
__host__ __device__ constexpr uint32_t t_hi(bool readout, int buf) { return readout ? 384u : 128u + 192u * buf; }
__host__ __device__ constexpr uint32_t lo_block(bool readout, int buf, int cb) {
    return readout ? p_block(cb) + 32u : t_hi(false, buf) + 128u + 16u * cb;
}

// b - z for two values, b as bf16
__device__ __forceinline__ float2 less(uint32_t b, float2 z) {
    float2 r;
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; sub.rn.f32.bf16 %0, l, %3; sub.rn.f32.bf16 %1, h, %4;}"
        : "=f"(r.x), "=f"(r.y)
        : "r"(b), "f"(z.x), "f"(z.y));
    return r;
}
__device__ __forceinline__ void tma_store_3d(const void* src, const CUtensorMap* tm, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(tm)),
                 "r"(x), "r"(y), "r"(z), "r"(smem_addr(src))
                 : "memory");
}

__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* tm, int x, int y, int z) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(reinterpret_cast<uint64_t>(tm)),
                 "r"(x), "r"(y), "r"(z)
                 : "memory");
}
// four 8 x 8 matrices of 16-bit elements, transposed: register m of lane l holds rows 2 (l % 4), + 1 of column l / 4
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// 16 TMEM lanes x 32 columns: register 2 g + k of lane l goes to TMEM lane 8 k + l / 4, column 4 g + l % 4
__device__ __forceinline__ void tmem_st_16x128b_x8(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]));
}

// the chunks of a job, walked alike by every role
struct Walk {
    int pos, n, ck;
    const int len, ck_end;
    const Ckpt* const ckpts;
    __device__ Walk(const Params& p, const Job& j)
        : pos(0), ck(j.ck_begin), len(j.len), ck_end(j.ck_begin + j.ck_count), ckpts(p.ckpts) {
        size();
    }
    __device__ void size() { n = min(kTok, (ck < ck_end ? ckpts[ck].pos : len) - pos); }
    __device__ bool more() const { return pos < len; }
    // whether the chunk ends at a checkpoint
    __device__ bool dump() const { return ck < ck_end && ckpts[ck].pos == pos + n; }
    __device__ void next() {
        if (dump()) ++ck;
        pos += n;
        size();
    }
};

// 512 threads leave 128 registers a thread, by which the compiler spills although the state role has 208 later: with a readout
// 236 bytes of stores and 256 of loads a thread (128 x 128), 200 and 240 (128 x 64), 100 or less otherwise; without one 172 and
// 140 (128 x 64), else 80 or less.  What that costs has not been measured by itself.
template <int DK, int DV, bool READOUT>
__global__ void __launch_bounds__(kThreads, 1) linear_tc_kernel(const __grid_constant__ Params p) {
    constexpr int NB = READOUT ? 2 : 3;               // buffers of K and of V (Q is spent early in its chunk: one)
    constexpr int NV = READOUT ? 1 : 2;               // V'
    constexpr int NT = READOUT ? 2 * NB + 1 : 2 * NB; // input tiles
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_addr(smem);
    float* pw = reinterpret_cast<float*>(smem + OFF_POW);   // pw[i] = a^i
    float* wp = pw + 132;                                   // wp[i] = a^(128 - i)
    float* vp = wp + 132;                                   // vp[i] = a^(127 - i): both orders of 16-byte pieces
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);   // [NT] an input tile landed
    uint64_t* empty = full + NT;        // [NT] everything that reads it is done
    uint64_t* g_done = empty + NT;      // G
    uint64_t* q_done = g_done + 1;      // Q S^T
    uint64_t* st_done = q_done + 1;     // [NV] the state's update (and Q S^T before it)
    uint64_t* o_done = st_done + NV;    // O
    uint64_t* s_ready = o_done + 1;     // state: the bf16 copy written
    uint64_t* p_ready = s_ready + 1;    // tokens, output: P written; state: O scaled
    uint64_t* v_ready = p_ready + 1;    // [NV] the last products read, V' hi and mid written, key and value rows zeroed
    uint64_t* lo_ready = v_ready + NV;  // V' lo written
    uint64_t* o_free = lo_ready + 1;    // output: O read
    uint64_t* o_staged = o_free + 1;    // output: a chunk's output staged
    uint64_t* o_left = o_staged + 1;    // the staged output has been copied out
    uint64_t* end = o_left + 1;         // every product done
    uint32_t* tslot = reinterpret_cast<uint32_t*>(end + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
    int* issued = reinterpret_cast<int*>(tslot + 2);   // [3] chunks whose K, V, Q copy was issued
    static_assert((2 * NT + 10 + 2 * NV) * 8 + 20 <= 256, "barrier area");

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x % p.H;
    const Job& job = p.jobs[blockIdx.x / p.H];
    const int hk = h / p.rep;
    const uint64_t limit = p.wait_limit_ns;

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tslot)),
                     "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (tid == 0) {
        for (int i = 0; i < 2 * NT + 3 + NV; ++i) mbar_init(&full[i], 1);
        mbar_init(o_left, 1);
        for (uint64_t* b : {s_ready, o_free, o_staged}) mbar_init(b, 128);
        mbar_init(p_ready, 384);
        for (int i = 0; i < NV; ++i) mbar_init(&v_ready[i], 384);
        mbar_init(lo_ready, 256);
        mbar_init(end, 1);
        *abort_flag = 0;
        issued[0] = issued[1] = issued[2] = 0;
        fence_barrier_init();
    }
    if (tid == 13 * 32 && job.len > 0) {   // the copies' descriptors, on their way while the barriers are made (a call without
                                           // tokens has none)
        for (const CUtensorMap* tm : {&p.tm_k, &p.tm_v, &p.tm_q})
            if (READOUT || tm != &p.tm_q)
                asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tm)) : "memory");
    }
    if (tid >= 128 && tid - 128 <= kTok) {
        // a^i by binary powers in fp64, rounded once
        double x = 1.0, sq = (double)p.alpha[h];
        for (int i = tid - 128; i; i >>= 1, sq *= sq)
            if (i & 1) x *= sq;
        const int i = tid - 128;
        pw[i] = wp[kTok - i] = (float)x;
        if (i < kTok) vp[kTok - 1 - i] = (float)x;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tslot;
    const uint32_t trow = tbase + ((uint32_t)(32 * (warp & 3)) << 16);   // this warp's lane quarter
    const int row = tid & 127;                                           // this thread's TMEM lane or tile row
    // chunk j's input tiles (0 K, 1 V, 2 Q): index of the tile and its barriers, offset, phase
    auto bar = [&](int in, int j) { return in == 2 ? 2 * NB : in * NB + j % NB; };
    auto at = [&](int in, int j) { return (uint32_t)(bar(in, j) * kTile); };
    auto phase = [&](int in, int j) { return in == 2 ? j : j / NB; };
    auto warp_wait = [&](uint64_t* bar, int parity) {
        return tcu::warp_wait_bar(bar, (uint32_t)parity & 1u, abort_flag, limit);
    };
    auto update_wait = [&](int j) { return warp_wait(&st_done[j % NV], j / NV); };   // chunk j's update is done
    Walk w(p, job);
    // 64 tokens from 32 sb of V'^T, 16 of this warp's 32 value dimensions (TMEM lanes): transposed on the way from shared memory by
    // ldmatrix, whose fragment (lane l: dimension l / 4, token pair l % 4 of an 8 x 8 matrix) is the 16x128b form's.  hi and
    // mid are stored, lo is handed back.
    auto scale_values = [&](int j, int n, int sb, int a, uint32_t (&v)[16]) {
        const int q4 = warp & 3, s0 = 32 * sb + 2 * (lane & 3);   // this lane's tokens s0 + 8 g and the next
        if (32 * q4 >= DV) return;   // rows past d_v: never read
        // row addresses, matrix lane / 8 of a load: token 8 (lane / 16) + (lane & 7), dimensions 16 a + 8 (lane / 8 % 2) ..
        const uint32_t src = sbase + at(1, j) + (q4 >> 1) * 16384 + (32 * sb + 8 * (lane >> 4) + (lane & 7)) * 128 +
                             ((((q4 & 1) * 4 + 2 * a + (lane >> 3 & 1)) ^ (lane & 7)) << 4);
        // v: [8-token group g, 8 dimensions of the 16]
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t x[4];
            ldsm_x4_trans(src + i * 16 * 128, x);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[4 * i + k] = x[k];
        }
        float2 f[8];   // a^{127-s}, a^{126-s}
#pragma unroll
        for (int g = 0; g < 8; ++g) f[g] = *reinterpret_cast<const float2*>(vp + s0 + 8 * g);
        if (n < kTok) {
#pragma unroll
            for (int g = 0; g < 8; ++g) {
                const int s = s0 + 8 * g;
                f[g].x = pw[max(n - 1 - s, 0)], f[g].y = pw[max(n - 2 - s, 0)];
                // past the chunk: another chunk's or sequence's values, not taken in
                const uint32_t in = (s < n ? 0xffffu : 0u) | (s + 1 < n ? 0xffff0000u : 0u);
                v[2 * g] &= in, v[2 * g + 1] &= in;
            }
        }
        const uint32_t t = trow + (16u * a << 16);
        float2 z[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            z[i] = __fmul2_rn(bf16x2_to_float2(v[i]), f[i >> 1]);
            v[i] = pack2(z[i].x, z[i].y);
        }
        tmem_st_16x128b_x8(t + t_hi(READOUT, j % NV) + 16 * sb, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            z[i] = less(v[i], z[i]);
            v[i] = pack2(z[i].x, z[i].y);
        }
        tmem_st_16x128b_x8(t + t_hi(READOUT, j % NV) + 64 + 16 * sb, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            z[i] = less(v[i], z[i]);
            v[i] = pack2(z[i].x, z[i].y);
        }
    };
    auto put_low = [&](int j, int sb, int a, const uint32_t (&lo)[16]) {
        if (32 * (warp & 3) < DV) tmem_st_16x128b_x8(trow + (16u * a << 16) + lo_block(READOUT, j % NV, sb), lo);
    };
    // Column block cb of P over G's columns, for this warp's token rows [32 rb, 32 rb + 32), lane a row.
    auto decay_scores = [&](int cb, float rowf) {
        const int rb = warp & 3;
        uint32_t pk[16];
        if (cb <= rb) {
            float g[32];
            if (cb < rb) {
                // a^{t-s} = a^{lane} a^{32 (rb - cb) - i}: both exponents are at least 0
                const float4* col = reinterpret_cast<const float4*>(wp + kTok - 32 * (rb - cb));
                const float2 rf = make_float2(rowf, rowf);
                float2 f[16];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 x = col[i];
                    f[2 * i] = __fmul2_rn(make_float2(x.x, x.y), rf), f[2 * i + 1] = __fmul2_rn(make_float2(x.z, x.w), rf);
                }
                tmem_ld32(trow + T_G + 32 * cb, g);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 y = __fmul2_rn(f[i], make_float2(g[2 * i], g[2 * i + 1]));
                    pk[i] = pack2(y.x, y.y);
                }
            } else {
                tmem_ld32(trow + T_G + 32 * cb, g);
#pragma unroll
                for (int i = 0; i < 32; ++i) g[i] = i <= lane ? g[i] * pw[max(lane - i, 0)] : 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) pk[i] = pack2(g[2 * i], g[2 * i + 1]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) pk[i] = 0u;
        }
        tmem_st16(trow + p_block(cb), pk);
    };

    if (warp < 4) {
        // ---- state ----
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");   // 512 threads start with 128: 208 + 120 + 120 + 64 = 4 x 128
        auto zero_rows = [&](int j) {   // a cut chunk's key and value rows past it
            if (w.n == kTok) return true;
            if (!warp_wait(&full[bar(0, j)], phase(0, j)) || !warp_wait(&full[bar(1, j)], phase(1, j))) return false;
            if (row >= w.n) {
#pragma unroll 1
                for (int in = 0; in < 2; ++in) {
                    unsigned char* x = smem + at(in, j) + row * 128;
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        *reinterpret_cast<uint4*>(x + (c >> 3) * 16384 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                }
            }
            proxy_fence();
            return true;
        };
        const float2 inter2 = make_float2(pw[row + 1], pw[row + 1]);
        auto scale_out = [&](int j) {   // O = Q S^T's rows, one a thread, by a^{t+1}
            if (!READOUT) return true;
            if (!warp_wait(q_done, j)) return false;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < DV / 32; ++c) {
                float x[32];
                tmem_ld32(trow + T_O + 32 * c, x);
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    const float2 z = __fmul2_rn(inter2, make_float2(x[i], x[i + 1]));
                    x[i] = z.x, x[i + 1] = z.y;
                }
                tmem_st32(trow + T_O + 32 * c, x);
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(p_ready);
            return true;
        };
        if (DV < 128 && 32 * warp >= DV) {
            // lanes past d_v hold nothing that is read: these warps only keep the barriers going (and zero their rows)
            for (int j = 0; w.more(); w.next(), ++j) {
                if (j > 0 && !update_wait(j - 1)) break;
                mbar_arrive(s_ready);
                if (!zero_rows(j)) break;
                mbar_arrive(&v_ready[j % NV]);
                if (!scale_out(j)) break;
            }
        } else {
            const size_t warp_off = ((size_t)h * DV + 32 * warp) * DK;
            // A thread holds a row, and 32 rows' 16 bytes at a time would take the load/store unit 32 lines an instruction, so
            // 32 x 32 pieces of the state pass through this warp's rows of the S tile, which is free then (two pieces in turn).
            unsigned char* const piece = smem + OFF_S + 32 * warp * 128;
            const int pr = lane >> 3, pc = lane & 7;   // by lines: row 4 k + pr, 16-byte column pc
            auto by_row = [&](int c, int i) {
                return reinterpret_cast<float4*>(piece + (c & 1) * 16384 + lane * 128 + ((i ^ (lane & 7)) << 4));
            };
            auto by_line = [&](int c, int k) {
                const int r = 4 * k + pr;
                return reinterpret_cast<float4*>(piece + (c & 1) * 16384 + r * 128 + ((pc ^ (r & 7)) << 4));
            };
            float2 S[DK / 2];   // this thread's row of the state
#pragma unroll
            for (int i = 0; i < DK / 2; ++i) S[i] = make_float2(0.f, 0.f);
            if (job.s0) {
                const float* src = job.s0 + warp_off + pr * DK + 4 * pc;
#pragma unroll
                for (int c = 0; c < DK / 32; ++c) {
                    float4 x[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[k] = *reinterpret_cast<const float4*>(src + 4 * k * DK + 32 * c);
#pragma unroll
                    for (int k = 0; k < 8; ++k) *by_line(c, k) = x[k];
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 y = *by_row(c, i);
                        S[16 * c + 2 * i] = make_float2(y.x, y.y), S[16 * c + 2 * i + 1] = make_float2(y.z, y.w);
                    }
                }
                __syncwarp();
            }
            float decay = 1.f;   // a^n of the last chunk
            bool ok = true;
            int j = 0, slot = -1;   // slot: where the last chunk's state goes
            for (;; w.next(), ++j) {
                if (j > 0) {
                    ok = update_wait(j - 1);
                    if (!ok) break;
                    tc_fence_after();
                    {
                        // S = a^n S + what the chunk's products added up
                        const float2 d = make_float2(decay, decay);
#pragma unroll
                        for (int c = 0; c < DK / 32; ++c) {
                            float v[32];
                            tmem_ld32(trow + T_S + 32 * c, v);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                S[16 * c + i] = __ffma2_rn(d, S[16 * c + i], make_float2(v[2 * i], v[2 * i + 1]));
                        }
                    }
                }
                if (w.more()) {   // the update may begin; only Q S^T waits for what follows
                    ok = zero_rows(j);
                    if (!ok) break;
                    tc_fence_before();
                    mbar_arrive(&v_ready[j % NV]);
                }
                // the states wanted here: a checkpoint's, the final one (S stays in registers only while it is used in one place)
#pragma unroll 1
                for (int k = 0; k < 2; ++k) {
                    float* dst = k == 0 ? (slot >= 0 ? p.ckpt_states + (size_t)slot * p.H * DV * DK : nullptr)
                                        : (w.more() ? nullptr : job.s_final);
                    if (!dst) continue;
                    dst += warp_off + pr * DK + 4 * pc;
#pragma unroll
                    for (int c = 0; c < DK / 32; ++c) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 x = S[16 * c + 2 * i], y = S[16 * c + 2 * i + 1];
                            *by_row(c, i) = make_float4(x.x, x.y, y.x, y.y);
                        }
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 8; ++i) *reinterpret_cast<float4*>(dst + 4 * i * DK + 32 * c) = *by_line(c, i);
                    }
                    __syncwarp();
                }
                if (!w.more()) break;
                decay = pw[w.n];
                if (READOUT) {
#pragma unroll
                    for (int c = 0; c < DK / 8; ++c)
                        *reinterpret_cast<uint4*>(smem + OFF_S + (c >> 3) * 16384 + sw128(row, (c & 7) * 8)) =
                            make_uint4(pack2(S[4 * c].x, S[4 * c].y), pack2(S[4 * c + 1].x, S[4 * c + 1].y),
                                       pack2(S[4 * c + 2].x, S[4 * c + 2].y), pack2(S[4 * c + 3].x, S[4 * c + 3].y));
                }
                if (READOUT) proxy_fence();
                mbar_arrive(s_ready);
                slot = w.dump() ? p.ckpts[w.ck].slot : -1;
                ok = scale_out(j);
                if (!ok) break;
            }
        }
    } else if (warp < 12) {
        // ---- tokens, output: lane = token row, this warp's rows are [32 rb, 32 rb + 32) ----
        asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
        const bool tokens = warp < 8;
        const bool wide = (reinterpret_cast<uintptr_t>(p.o) & 31) == 0;
        const float rowf = pw[lane];
        const float2 scale2 = make_float2(p.scale, p.scale);
        const int b0 = tokens ? 0 : 2;   // the blocks of 32 tokens of this role
        int pos = 0, n = 0;              // the chunk before j, whose O is still to be taken
        for (int j = 0;; w.next(), ++j) {
            const bool more = w.more();
            // V' hi and mid as soon as the last update is done with theirs, while PV and G are made; lo stays here until G is
            // read
            uint32_t lo[2][16];
            if (more) {
                if (!warp_wait(&full[bar(1, j)], phase(1, j)) || (j >= NV && !update_wait(j - NV))) break;
                tc_fence_after();
#pragma unroll 1
                for (int a = 0; a < 2; ++a) {
                    uint32_t v[16];
                    scale_values(j, w.n, b0, a, v);
                    if (READOUT) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) lo[0][i] = a == 0 ? v[i] : lo[0][i], lo[1][i] = v[i];
                    } else {
                        put_low(j, b0, a, v);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&v_ready[j % NV]);
            }
            if (READOUT && !tokens && j > 0) {
                if (!warp_wait(o_done, j - 1) || (j > 1 && !warp_wait(o_left, j - 2))) break;
                tc_fence_after();
                // A whole chunk is staged and copied out by TMA: a thread holds a row, and stores of 32 rows at a time,
                // 32 bytes each, kept the load/store unit from everyone for 1200 cycles.  A cut one is stored like that.
                __nv_bfloat16* const dst =
                    static_cast<__nv_bfloat16*>(p.o) + ((job.tok_begin + pos + row) * p.H + h) * (int64_t)DV;
#pragma unroll 1
                for (int c = 0; c < DV / 32; ++c) {
                    float x[32];
                    tmem_ld32(trow + T_O + 32 * c, x);
                    uint32_t u[2][8];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 z = __fmul2_rn(scale2, make_float2(x[2 * i], x[2 * i + 1]));
                        u[i >> 3][i & 7] = pack2(z.x, z.y);
                    }
                    if (n == kTok) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            *reinterpret_cast<uint4*>(smem + OFF_O + (c >> 1) * 16384 + sw128(row, ((c & 1) * 4 + i) * 8)) =
                                make_uint4(u[i >> 1][(i & 1) * 4], u[i >> 1][(i & 1) * 4 + 1], u[i >> 1][(i & 1) * 4 + 2],
                                           u[i >> 1][(i & 1) * 4 + 3]);
                    } else if (row < n) {
                        store32(dst + 32 * c, u[0], wide);
                        store32(dst + 32 * c + 16, u[1], wide);
                    }
                }
                tc_fence_before();
                mbar_arrive(o_free);
                proxy_fence();
                mbar_arrive(o_staged);
            }
            if (!more) break;
            pos = w.pos, n = w.n;
            if (!READOUT) continue;
            if (!warp_wait(g_done, j)) break;
            tc_fence_after();
#pragma unroll 1
            for (int b = b0; b < b0 + 2; ++b) decay_scores(b, rowf);
            put_low(j, b0, 0, lo[0]);
            put_low(j, b0, 1, lo[1]);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(lo_ready);
            mbar_arrive(p_ready);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == 12) {
            // ---- products (the whole warp walks along, one elected lane issues) ----
            const uint32_t id_g = idesc(kTok, false, false), id_q = idesc(DV, false, false), id_o = idesc(DV, false, true),
                           id_s = idesc(DK, false, true);
            const uint64_t s_desc = tile_desc(sbase + OFF_S, false);
            auto scores = [&](int j) {   // G of chunk j
                if (!warp_wait(&full[bar(0, j)], phase(0, j)) || !warp_wait(&full[bar(2, j)], phase(2, j))) return false;
                const uint64_t q = tile_desc(sbase + at(2, j), false), k = tile_desc(sbase + at(0, j), false);
                if (elect_one()) {
#pragma unroll 2
                    for (int i = 0; i < DK / 16; ++i) umma_ss(tbase + T_G, cols_step(q, i), cols_step(k, i), id_g, i > 0);
                    umma_commit(g_done);
                }
                return true;
            };
            bool ok = !READOUT || !w.more() || scores(0);
            for (int j = 0; ok && w.more(); ++j) {
                w.next();
                ok = warp_wait(&v_ready[j % NV], j / NV) && warp_wait(&full[bar(0, j)], phase(0, j));
                if (!ok) break;
                tc_fence_after();
                const uint64_t k = tile_desc(sbase + at(0, j), true), v = tile_desc(sbase + at(1, j), true);
                const uint32_t vh = tbase + t_hi(READOUT, j % NV);
                if (elect_one()) {
#pragma unroll 2
                    for (int i = 0; i < 8; ++i) {   // the key rows of 16 tokens
                        umma_ts(tbase + T_S, vh + 8 * i, rows_step(k, i), id_s, i > 0);
                        umma_ts(tbase + T_S, vh + 64 + 8 * i, rows_step(k, i), id_s | 1u << 13, 1);   // A negated
                    }
                }
                if (READOUT) {
                    ok = warp_wait(s_ready, j) && (j == 0 || warp_wait(o_free, j - 1));
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t q = tile_desc(sbase + at(2, j), false);
                    if (elect_one()) {
#pragma unroll 2
                        for (int i = 0; i < DK / 16; ++i)
                            umma_ss(tbase + T_O, cols_step(q, i), cols_step(s_desc, i), id_q, i > 0);
                        umma_commit(q_done);
                        umma_commit(&empty[bar(2, j)]);
                    }
                    ok = warp_wait(lo_ready, j);
                    if (!ok) break;
                    tc_fence_after();
                }
                if (elect_one()) {
#pragma unroll 2
                    for (int i = 0; i < 8; ++i)
                        umma_ts(tbase + T_S, tbase + lo_block(READOUT, j % NV, i >> 1) + 8 * (i & 1), rows_step(k, i), id_s, 1);
                    umma_commit(&st_done[j % NV]);
                    umma_commit(&empty[bar(0, j)]);
                }
                if (READOUT) {
                    ok = warp_wait(p_ready, j) && warp_wait(&full[bar(1, j)], phase(1, j));
                    if (!ok) break;
                    tc_fence_after();
                }
                if (elect_one()) {
                    if (READOUT) {
#pragma unroll 2
                        for (int i = 0; i < 8; ++i) umma_ts(tbase + T_O, tbase + p_block(i >> 1) + 8 * (i & 1), rows_step(v, i), id_o, 1);
                        umma_commit(o_done);
                    }
                    umma_commit(&empty[bar(1, j)]);
                }
                if (READOUT) ok = !w.more() || scores(j + 1);
            }
            if (elect_one()) umma_commit(end);   // also after giving up: the end waits for the products in flight
        } else if (warp == 14) {
            // ---- staged output to memory ----
            if (READOUT && lane == 0) {
                for (int j = 0; w.more(); w.next(), ++j) {
                    if (!wait_bar(o_staged, (uint32_t)j & 1u, abort_flag, limit)) break;
                    if (w.n == kTok) {
                        const int t0 = (int)(job.tok_begin + w.pos);
#pragma unroll
                        for (int x = 0; x < DV / 64; ++x) tma_store_3d(smem + OFF_O + x * 16384, &p.tm_o, 64 * x, h, t0);
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    }
                    mbar_arrive(o_left);
                }
            }
        } else if (lane == 0 && (warp == 13 || READOUT)) {
            // ---- copies: warp 13 K and V, warp 15 Q, whose buffer comes free at another time of the chunk ----
            const int first = warp == 13 ? 0 : 2, last = warp == 13 ? 1 : 2;
            bool ok = true;
            for (int j = 0; ok && w.more(); w.next(), ++j) {
                if (p.stall_after >= 0 && j >= p.stall_after) break;   // testing hook
                const int t0 = (int)(job.tok_begin + w.pos);
                for (int in = first; in <= last; ++in) {
                    if (phase(in, j) > 0 &&
                        !wait_bar(&empty[bar(in, j)], (uint32_t)(phase(in, j) - 1) & 1u, abort_flag, limit)) {
                        ok = false;
                        break;
                    }
                    const CUtensorMap* tm = in == 0 ? &p.tm_k : in == 1 ? &p.tm_v : &p.tm_q;
                    const int head = in == 1 ? h : hk;
                    uint64_t* b = &full[bar(in, j)];
                    const int blocks = (in == 1 ? DV : DK) / 64;
                    mbar_arrive_expect_tx(b, blocks * 16384);
                    for (int x = 0; x < blocks; ++x) tma_load_3d(smem + at(in, j) + x * 16384, tm, 64 * x, head, t0, b);
                    issued[in] = j + 1;
                    // Q has one buffer, and the next chunk's scores wait for it: on its way into the L2 cache before there is room
                    if (in == 2 && w.pos + w.n < w.len)
                        for (int x = 0; x < blocks; ++x) tma_prefetch_3d(tm, 64 * x, head, t0 + w.n);
                }
            }
        }
    }

    // ---- leave only with no copy and no product still writing into this CTA's shared memory or TMEM ----
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *abort_flag) {
        const uint64_t drain = limit > kDrainLimitNs ? limit : kDrainLimitNs;
        for (int in = 0; in < 3; ++in)
            for (int j = max(0, issued[in] - (in == 2 ? 1 : NB)); j < issued[in]; ++j)
                tc::drain_phase(&full[bar(in, j)], (uint32_t)phase(in, j) & 1u, drain);
        tc::drain_phase(end, 0, drain);
        atomicOr(p.status, STATUS_TIMEOUT);
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(512));
}

template <int DK, int DV, bool READOUT>
cudaError_t launch(const Params& p, cudaStream_t s) {
    auto kern = linear_tc_kernel<DK, DV, READOUT>;
    static std::atomic<int> optin[kMaxOptinDevices];
    const cudaError_t e = smem_optin(reinterpret_cast<const void*>(kern), kSmem, optin);
    if (e != cudaSuccess) return e;
    kern<<<p.n_jobs * p.H, kThreads, kSmem, s>>>(p);
    return cudaGetLastError();
}
template <int DK, int DV>
cudaError_t launch_d(const Params& p, cudaStream_t s) {
    return p.o ? launch<DK, DV, true>(p, s) : launch<DK, DV, false>(p, s);
}

}  // namespace

cudaError_t launch_tc(const Params& p, int dk, cudaStream_t s) {
    if (dk == 128) return p.dv == 128 ? launch_d<128, 128>(p, s) : launch_d<128, 64>(p, s);
    return p.dv == 128 ? launch_d<64, 128>(p, s) : launch_d<64, 64>(p, s);
}

}  // namespace lin
}  // namespace gdn
