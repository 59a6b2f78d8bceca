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
//     S += V'^T K with V' = diag(a^{n-1-s}) V
// V' is not exact in bf16: it is split into hi + lo halves and both are multiplied, so a state loses 2^-16 of an added
// term, as the delta rule scan's does.  P and the copy of S that the readout multiplies are rounded to bf16 once (half a
// step, 2^-8 of each term): the readout itself is rounded to bf16, and its error stays of that order.
//
// What bounds it: shared memory's 128 bytes a cycle, of which a product with both operands there takes nearly all.  So
// P and V'^T are operands in TMEM: with K' = diag(.) K split in shared memory instead (written, and read again beside V),
// a chunk moved 590 KB through shared memory, now 430 KB, and the room of K' gives every input tile a second buffer.
//
// One CTA takes one (job, head) from its first chunk to its last.  Roles:
//   state  (warps 0-3):  S out of TMEM into its bf16 copy, S scaled by a^n in place; half of V^T -> V' hi and lo in
//                        TMEM; checkpoints, initial, final state; key and value rows past a cut chunk zeroed
//   tokens (warps 4-7):  the first half of G's columns -> P in TMEM; a^{t+1} into O
//   output (warps 8-11): the second half of P; the other half of the next V'; O to memory, staged for TMA
// (without a readout the last two only form V')
//   one thread each that issues the products, the copies of K and V, of Q and of staged output
// They hand over through mbarriers, one phase a chunk, and no barrier completes a phase before everyone who waits for
// the last one has seen it (a parity tells only two phases apart).  The state's own chain (S and V' converted, Q S^T and
// the update multiplied) is the critical path; G, P and P V of a chunk run beside it.  Each role's chunk is written as
// short rolled loops: unrolled, the roles' code streamed through the instruction cache once a chunk, 1.5 times as slow.
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
using tc::split_pair;
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

constexpr int kTok = 128;                   // tokens of a chunk
constexpr int kTile = kTok * 128 * 2;       // bytes of a tile: two 64-column blocks of [128][128 B] (one used at width 64)
constexpr int kThreads = 16 * 32;
constexpr int OFF_O = 5 * kTile;            // after the input tiles (with a readout): staged output
constexpr int OFF_S = 6 * kTile;            // the bf16 copy of S
constexpr int OFF_POW = 7 * kTile;          // a^0 .. a^128; a^128 .. a^0; a^127 .. a^0
constexpr int OFF_BAR = OFF_POW + 3 * 528;
constexpr int kSmem = OFF_BAR + 256 + 1024;
static_assert(kSmem <= 232448, "227 KB of shared memory per block");
// P, a block of 32 tokens (16 columns) at a time, goes over columns of G that only the writing role reads: blocks 0 and 1
// over G's first 32 columns (tokens), 2 and 3 over the third (output)
__host__ __device__ constexpr uint32_t p_block(int cb) { return 128u + 16u * cb + (cb >= 2 ? 32u : 0u); }
constexpr uint32_t T_S = 0, T_G = 128, T_O = 256, T_VH = 384, T_VL = 448;

__device__ __forceinline__ void tma_store_3d(const void* src, const CUtensorMap* tm, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(tm)),
                 "r"(x), "r"(y), "r"(z), "r"(smem_addr(src))
                 : "memory");
}

// four 8 x 8 matrices of 16-bit elements, transposed: register m of lane l holds rows 2 (l % 4), + 1 of column l / 4
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// 16 TMEM lanes x 16 columns: register 2 g + k of lane l goes to TMEM lane 8 k + l / 4, column 4 g + l % 4
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]));
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

template <int DK, int DV, bool READOUT>
__global__ void __launch_bounds__(kThreads, 1) linear_tc_kernel(const __grid_constant__ Params p) {
    constexpr int NB = READOUT ? 2 : 3;               // buffers of K and of V (Q is spent early in its chunk: one)
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
    uint64_t* st_done = q_done + 1;     // the state's update (and Q S^T before it)
    uint64_t* o_done = st_done + 1;     // O
    uint64_t* s_ready = o_done + 1;     // state: the bf16 copy written, S scaled
    uint64_t* p_ready = s_ready + 1;    // tokens, output: P written, O scaled
    uint64_t* v_ready = p_ready + 1;    // V' written, key and value rows zeroed
    uint64_t* o_free = v_ready + 1;     // output: O read
    uint64_t* o_staged = o_free + 1;    // output: a chunk's output staged
    uint64_t* o_left = o_staged + 1;    // the staged output has been copied out
    uint64_t* end = o_left + 1;         // every product done
    uint32_t* tslot = reinterpret_cast<uint32_t*>(end + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
    int* issued = reinterpret_cast<int*>(tslot + 2);   // [3] chunks whose K, V, Q copy was issued
    static_assert((2 * NT + 11) * 8 + 20 <= 256, "barrier area");

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
        for (int i = 0; i < 2 * NT + 4; ++i) mbar_init(&full[i], 1);
        mbar_init(o_left, 1);
        for (uint64_t* b : {s_ready, o_free, o_staged}) mbar_init(b, 128);
        mbar_init(p_ready, 256);
        mbar_init(v_ready, READOUT ? 256 : 384);
        mbar_init(end, 1);
        *abort_flag = 0;
        issued[0] = issued[1] = issued[2] = 0;
        fence_barrier_init();
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
    Walk w(p, job);
    // Tokens 32 sb .. of V'^T, this warp's 32 value dimensions (TMEM lanes): transposed on the way from shared memory by
    // ldmatrix, whose fragment (lane l: dimension l / 4, token pair l % 4 of an 8 x 8 matrix) is the 16x128b form's.
    auto scale_values = [&](int j, int n, int sb) {
        const int q4 = warp & 3, pr = lane & 3;
        if (32 * q4 >= DV) return;   // rows past d_v: never read
        // row addresses: token 8 g + (lane & 7) of the block, dimensions 8 (lane / 8) .. of this warp's 32
        const uint32_t src = sbase + at(1, j) + (q4 >> 1) * 16384 + (32 * sb + (lane & 7)) * 128 +
                             ((((q4 & 1) * 4 + (lane >> 3)) ^ (lane & 7)) << 4);
        uint32_t hi[2][8], lo[2][8];   // [16 dimensions][8-token group g, 8 dimensions of those]
        // every load first: one at a time, each of the four would wait out its latency and its arithmetic's
        uint32_t v[4][4];
        float2 f[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            ldsm_x4_trans(src + g * 8 * 128, v[g]);
            f[g] = *reinterpret_cast<const float2*>(vp + 32 * sb + 8 * g + 2 * pr);   // a^{127-s}, a^{126-s}
        }
        if (n < kTok) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int s = 32 * sb + 8 * g + 2 * pr;   // this lane's tokens s and s + 1
                f[g].x = pw[max(n - 1 - s, 0)], f[g].y = pw[max(n - 2 - s, 0)];
                // past the chunk: another chunk's or sequence's values, not taken in
                const uint32_t in = (s < n ? 0xffffu : 0u) | (s + 1 < n ? 0xffff0000u : 0u);
#pragma unroll
                for (int m = 0; m < 4; ++m) v[g][m] &= in;
            }
        }
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float2 z = __fmul2_rn(bf16x2_to_float2(v[g][m]), f[g]);
                split_pair(z.x, z.y, hi[m >> 1][2 * g + (m & 1)], lo[m >> 1][2 * g + (m & 1)]);
            }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            tmem_st_16x128b_x4(trow + (16u * m << 16) + T_VH + 16 * sb, hi[m]);
            tmem_st_16x128b_x4(trow + (16u * m << 16) + T_VL + 16 * sb, lo[m]);
        }
    };
    // Two blocks of chunk j's V', by a role that has not waited for the last update yet.
    auto form_values = [&](int j, int n, int sb) {
        if (!warp_wait(&full[bar(1, j)], phase(1, j)) || (j > 0 && !warp_wait(st_done, j - 1))) return false;
        tc_fence_after();
#pragma unroll 1
        for (int i = sb; i < sb + 2; ++i) scale_values(j, n, i);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(v_ready);
        return true;
    };
    // Column block cb of P over G's columns, for this warp's token rows [32 rb, 32 rb + 32), lane a row; diag[i] =
    // a^{lane - i}, the same in every chunk.
    auto decay_scores = [&](int cb, float rowf, const float (&diag)[32]) {
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
                for (int i = 0; i < 32; ++i) g[i] = i <= lane ? g[i] * diag[i] : 0.f;
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
        const bool mine = row < DV;   // whole warps: lanes past d_v hold nothing that is read
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
        auto dump = [&](float* dst) {   // this warp's rows of TMEM to dst
            if (!mine) return;
            dst += warp_off + pr * DK + 4 * pc;
#pragma unroll 1
            for (int c = 0; c < DK / 32; ++c) {
                float v[32];
                tmem_ld32(trow + T_S + 32 * c, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) *by_row(c, i) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 8; ++k) *reinterpret_cast<float4*>(dst + 4 * k * DK + 32 * c) = *by_line(c, k);
            }
            __syncwarp();
        };
        if (w.more() && mine) {
            // the initial state into TMEM, so that the first chunk is like the others
#pragma unroll 1
            for (int c0 = 0; c0 < DK / 32; c0 += 2) {
                if (job.s0) {
                    const float* src = job.s0 + warp_off + pr * DK + 4 * pc + 32 * c0;
                    float4 x[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = *reinterpret_cast<const float4*>(src + 4 * (i & 7) * DK + 32 * (i >> 3));
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 16; ++i) *by_line(i >> 3, i & 7) = x[i];
                    __syncwarp();
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 x = job.s0 ? *by_row(c, i) : make_float4(0.f, 0.f, 0.f, 0.f);
                        v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
                    }
                    tmem_st32(trow + T_S + 32 * (c0 + c), v);
                }
            }
            tmem_st_wait();
            __syncwarp();
        }
        bool ok = true;
        int j = 0, slot = -1;   // slot: where the last chunk's state is dumped
        for (; w.more(); w.next(), ++j) {
            if (j > 0) {
                ok = warp_wait(st_done, j - 1);
                if (!ok) break;
                tc_fence_after();
                if (slot >= 0) dump(p.ckpt_states + (size_t)slot * p.H * DV * DK);
            }
            const float2 decay = make_float2(pw[w.n], pw[w.n]);
#pragma unroll 1
            for (int c = 0; c < (mine ? DK / 64 : 0); ++c) {
                float v[2][32];
                tmem_ld32x2(trow + T_S + 64 * c, trow + T_S + 64 * c + 32, v[0], v[1]);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (READOUT) {
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            *reinterpret_cast<uint4*>(smem + OFF_S + c * 16384 + sw128(row, k * 32 + i)) =
                                make_uint4(pack2(v[k][i], v[k][i + 1]), pack2(v[k][i + 2], v[k][i + 3]),
                                           pack2(v[k][i + 4], v[k][i + 5]), pack2(v[k][i + 6], v[k][i + 7]));
                    }
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float2 x = __fmul2_rn(make_float2(v[k][i], v[k][i + 1]), decay);
                        v[k][i] = x.x, v[k][i + 1] = x.y;
                    }
                    tmem_st32(trow + T_S + 64 * c + 32 * k, v[k]);
                }
            }
            tmem_st_wait();
            if (READOUT) proxy_fence();
            tc_fence_before();
            mbar_arrive(s_ready);
            // then half of V', on the chain as well (without a readout the tokens role has nothing else to do)
            if (READOUT) {
                ok = warp_wait(&full[bar(1, j)], phase(1, j));
                if (!ok) break;
#pragma unroll 1
                for (int sb = 0; sb < 2; ++sb) scale_values(j, w.n, sb);
            }
            if (w.n < kTok) {
                ok = warp_wait(&full[bar(0, j)], phase(0, j)) && warp_wait(&full[bar(1, j)], phase(1, j));
                if (!ok) break;
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
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(v_ready);
            slot = w.dump() ? p.ckpts[w.ck].slot : -1;
        }
        if (ok && j > 0) {
            ok = warp_wait(st_done, j - 1);
            if (ok) {
                tc_fence_after();
                if (slot >= 0) dump(p.ckpt_states + (size_t)slot * p.H * DV * DK);
                if (job.s_final) dump(job.s_final);
            }
        } else if (ok && job.s_final && mine) {
            // no tokens: the final state is the initial one
            for (int i = lane; i < 32 * DK / 4; i += 32)
                reinterpret_cast<float4*>(job.s_final + warp_off)[i] =
                    job.s0 ? reinterpret_cast<const float4*>(job.s0 + warp_off)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    } else if (warp < 8) {
        // ---- tokens: lane = token row, this warp's rows are [32 rb, 32 rb + 32) ----
        if (!READOUT) {
            for (int j = 0; w.more() && form_values(j, w.n, 0); w.next()) ++j;
        }
        if (READOUT) {
            const float rowf = pw[lane], inter = pw[row + 1];
            const float2 inter2 = make_float2(inter, inter);
            float diag[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) diag[i] = pw[max(lane - i, 0)];
            for (int j = 0; w.more(); w.next(), ++j) {
                if (!warp_wait(g_done, j)) break;
                tc_fence_after();
#pragma unroll 1
                for (int cb = 0; cb < 2; ++cb) decay_scores(cb, rowf, diag);
                if (!warp_wait(q_done, j)) break;
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
            }
        }
    } else if (warp < 12) {
        // ---- output: lane = token row ----
        if (!READOUT) {
            for (int j = 0; w.more() && form_values(j, w.n, 2); w.next()) ++j;
        } else if (w.more() && form_values(0, w.n, 2)) {
            const bool wide = (reinterpret_cast<uintptr_t>(p.o) & 31) == 0;
            const float2 scale2 = make_float2(p.scale, p.scale);
            const float rowf = pw[lane];
            float diag[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) diag[i] = pw[max(lane - i, 0)];
            for (int j = 0; w.more(); ++j) {
                const int pos = w.pos, n = w.n;
                if (!warp_wait(g_done, j)) break;
                tc_fence_after();
#pragma unroll 1
                for (int cb = 2; cb < 4; ++cb) decay_scores(cb, rowf, diag);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(p_ready);
                // the other half of the next chunk's V', for which the update is done before this chunk's O
                w.next();
                if (w.more() && !form_values(j + 1, w.n, 2)) break;
                if (!warp_wait(o_done, j)) break;
                tc_fence_after();
                // the whole row into registers first, so that the next chunk's O can begin before the stores are through
                uint32_t u[DV / 16][8];
#pragma unroll
                for (int c = 0; c < DV / 32; ++c) {
                    float x[32];
                    tmem_ld32(trow + T_O + 32 * c, x);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 z = __fmul2_rn(scale2, make_float2(x[2 * i], x[2 * i + 1]));
                        u[2 * c + (i >> 3)][i & 7] = pack2(z.x, z.y);
                    }
                }
                tc_fence_before();
                mbar_arrive(o_free);
                // A whole chunk is staged and copied out by TMA: a thread holds a row, and stores of 32 rows at a time,
                // 32 bytes each, kept the load/store unit from everyone for 1200 cycles.  A cut one is stored like that.
                if (j > 0 && !warp_wait(o_left, j - 1)) break;
                if (n == kTok) {
#pragma unroll
                    for (int c = 0; c < DV / 8; ++c)
                        *reinterpret_cast<uint4*>(smem + OFF_O + (c >> 3) * 16384 + sw128(row, (c & 7) * 8)) =
                            make_uint4(u[c >> 1][(c & 1) * 4], u[c >> 1][(c & 1) * 4 + 1], u[c >> 1][(c & 1) * 4 + 2],
                                       u[c >> 1][(c & 1) * 4 + 3]);
                    proxy_fence();
                } else if (row < n) {
                    __nv_bfloat16* dst =
                        static_cast<__nv_bfloat16*>(p.o) + ((job.tok_begin + pos + row) * p.H + h) * (int64_t)DV;
#pragma unroll
                    for (int c = 0; c < DV / 16; ++c) store32(dst + 16 * c, u[c], wide);
                }
                mbar_arrive(o_staged);
            }
        }
    } else if (warp == 12) {
        // ---- products (the whole warp walks along, one elected lane issues) ----
        const uint32_t id_g = idesc(kTok, false, false), id_q = idesc(DV, false, false), id_o = idesc(DV, false, true),
                       id_s = idesc(DK, false, true);
        const uint64_t s_desc = tile_desc(sbase + OFF_S, false);
        auto scores = [&](int j) {   // G of chunk j
            if (!warp_wait(&full[bar(0, j)], phase(0, j)) || !warp_wait(&full[bar(2, j)], phase(2, j))) return false;
            const uint64_t q = tile_desc(sbase + at(2, j), false), k = tile_desc(sbase + at(0, j), false);
            if (elect_one()) {
#pragma unroll
                for (int i = 0; i < DK / 16; ++i) umma_ss(tbase + T_G, cols_step(q, i), cols_step(k, i), id_g, i > 0);
                umma_commit(g_done);
            }
            return true;
        };
        bool ok = !READOUT || !w.more() || scores(0);
        for (int j = 0; ok && w.more(); ++j) {
            w.next();
            ok = warp_wait(s_ready, j);
            if (!ok) break;
            if (READOUT) {
                ok = j == 0 || warp_wait(o_free, j - 1);
                if (!ok) break;
                tc_fence_after();
                const uint64_t q = tile_desc(sbase + at(2, j), false);
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < DK / 16; ++i)
                        umma_ss(tbase + T_O, cols_step(q, i), cols_step(s_desc, i), id_q, i > 0);
                    umma_commit(q_done);
                    umma_commit(&empty[bar(2, j)]);
                }
            }
            ok = warp_wait(v_ready, j) && warp_wait(&full[bar(0, j)], phase(0, j));
            if (!ok) break;
            tc_fence_after();
            const uint64_t k = tile_desc(sbase + at(0, j), true), v = tile_desc(sbase + at(1, j), true);
            if (elect_one()) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    umma_ts(tbase + T_S, tbase + T_VH + 8 * i, rows_step(k, i), id_s, 1);
                    umma_ts(tbase + T_S, tbase + T_VL + 8 * i, rows_step(k, i), id_s, 1);
                }
                umma_commit(st_done);
                umma_commit(&empty[bar(0, j)]);
            }
            if (READOUT) {
                ok = warp_wait(p_ready, j) && warp_wait(&full[bar(1, j)], phase(1, j));
                if (!ok) break;
                tc_fence_after();
            }
            if (elect_one()) {
                if (READOUT) {
#pragma unroll
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
