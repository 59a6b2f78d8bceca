// gdn_linear_tc.cu - linear attention with a decay for each head, chunked form on the 5th-generation tensor cores
// (d_k = d_v = 128, bf16 in and out).
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
//     G = Q K^T;  O1 = Q S^T;  O2 = P V, P = G masked and decayed;  S += V^T K' with K' = diag(a^{n-1-s}) K
// K' is not exact in bf16: it is split into hi + lo halves and both are multiplied, so a state loses 2^-16 of an added
// term, as the delta rule scan's does.  P and the copy of S that the readout multiplies are rounded to bf16 once (half a
// step, 2^-8 of each term): the readout itself is rounded to bf16, and its error stays of that order.
//
// One CTA takes one (job, head) from its first chunk to its last.  Roles:
//   state  (warps 0-3):  S out of TMEM into its bf16 copy, S scaled by a^n in place; checkpoints, initial, final state
//   tokens (warps 4-7):  G -> P in TMEM; the readout a^{t+1} O1 + O2 to memory
//   keys   (warps 8-11): K -> K' hi (in place) and lo; value rows past a cut chunk zeroed
//   one thread that issues the products, one that issues the copies (TMA, a ring of 5 tiles in the order K, Q, V)
// They hand over through mbarriers, one phase a chunk.  The state's own chain (S and K' converted, O1 and the update
// multiplied) is the critical path; G, P and O2 of a chunk run beside it.
//
// A sequence's tiles may reach past its end into its neighbour's tokens: P and K' are replaced by zeros there and the
// value rows are zeroed, so a neighbour's values, infinities and NaN included, never reach a result.
//
// Every wait is bounded: a role that gives up sets the abort flag, every role leaves, copies and products in flight
// are waited for, TMEM is freed and the sticky status is set.
#include <cuda_bf16.h>

#include "gdn_chunk_tc.cuh"
#include "gdn_linear.cuh"

namespace gdn {
namespace lin {
namespace {

using tc::idesc;
using tc::proxy_fence;
using tc::sdesc;
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

constexpr int D = 128;
constexpr int kTok = 128;                   // tokens of a chunk
constexpr int kTile = kTok * D * 2;         // bytes of a K, Q, V, K' or S tile: two 64-column blocks of [128][128 B]
constexpr int ST = 5;                       // tiles of the ring
constexpr int kThreads = 14 * 32;
constexpr int OFF_KLO = ST * kTile;         // K' lo
constexpr int OFF_S = OFF_KLO + kTile;      // bf16 S
constexpr int OFF_POW = OFF_S + kTile;      // a^0 .. a^128, then a^128 .. a^0
constexpr int OFF_BAR = OFF_POW + 2 * 528;
constexpr int kSmem = OFF_BAR + 256 + 1024;
static_assert(kSmem <= 232448, "227 KB of shared memory per block");
constexpr uint32_t T_S = 0, T_G = 128, T_O1 = 256, T_O2 = 384;

// bounded wait of one thread; gives up when another role has given up
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint64_t limit) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (;;) {
        if (mbar_try_wait_suspend(bar, parity, 2000)) return true;
        if (*abort_flag) return false;
        if (global_ns() - t0 > limit) {
            *abort_flag = 1;
            return false;
        }
    }
}
__device__ __forceinline__ void tma_store_3d(const void* src, const CUtensorMap* tm, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(tm)),
                 "r"(x), "r"(y), "r"(z), "r"(smem_addr(src))
                 : "memory");
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
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

template <bool READOUT>
__global__ void __launch_bounds__(kThreads, 1) linear_tc_kernel(const __grid_constant__ Params p) {
    constexpr int PER = READOUT ? 3 : 2;   // tiles a chunk: K, Q, V or K, V
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_addr(smem);
    float* pw = reinterpret_cast<float*>(smem + OFF_POW);   // pw[i] = a^i
    float* wp = pw + 132;                                   // wp[i] = a^(128 - i)
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);   // [ST] a tile landed
    uint64_t* empty = full + ST;        // [ST] every product that reads it is done
    uint64_t* g_done = empty + ST;      // G
    uint64_t* st_done = g_done + 1;     // the state's update (and O1 before it)
    uint64_t* o_done = st_done + 1;     // O1 and O2
    uint64_t* s_ready = o_done + 1;     // state: the bf16 copy written, S scaled
    uint64_t* p_ready = s_ready + 1;    // tokens: P written
    uint64_t* k_ready = p_ready + 1;    // keys: K' written, value rows zeroed
    uint64_t* o_free = k_ready + 1;     // tokens: O1 and O2 read
    uint64_t* o_staged = o_free + 1;    // tokens: the chunk's output in the spent Q tile
    uint64_t* end = o_staged + 1;       // every product done
    uint32_t* tslot = reinterpret_cast<uint32_t*>(end + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
    int* issued = reinterpret_cast<int*>(tslot + 2);
    static_assert((2 * ST + 9) * 8 + 12 <= 256, "barrier area");

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
        for (int i = 0; i < 2 * ST + 3; ++i) mbar_init(&full[i], 1);
        for (uint64_t* b : {s_ready, p_ready, k_ready, o_free, o_staged}) mbar_init(b, 128);
        mbar_init(end, 1);
        *abort_flag = 0;
        *issued = 0;
        fence_barrier_init();
    }
    if (tid >= 128 && tid - 128 <= kTok) {
        // a^i by binary powers in fp64, rounded once
        double x = 1.0, sq = (double)p.alpha[h];
        for (int i = tid - 128; i; i >>= 1, sq *= sq)
            if (i & 1) x *= sq;
        pw[tid - 128] = wp[kTok - (tid - 128)] = (float)x;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tslot;
    const uint32_t trow = tbase + ((uint32_t)(32 * (warp & 3)) << 16);   // this warp's lane quarter
    const int row = tid & 127;                                           // this thread's TMEM lane or tile row
    auto tile = [&](int seq) { return (uint32_t)(seq % ST) * kTile; };
    auto warp_wait = [&](uint64_t* bar, int parity) {
        return __all_sync(0xffffffffu, wait_bar(bar, (uint32_t)parity & 1u, abort_flag, limit)) != 0;
    };
    auto full_parity = [&](int seq) { return (seq / ST) & 1; };
    Walk w(p, job);

    if (warp < 4) {
        // ---- state ----
        const size_t state_off = ((size_t)h * D + row) * D;
        auto dump = [&](float* dst) {   // this thread's row, from TMEM
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                float v[32];
                tmem_ld32(trow + T_S + 32 * c, v);
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    *reinterpret_cast<float4*>(dst + 32 * c + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
        };
        if (w.more()) {
            // the initial state into TMEM, so that the first chunk is like the others
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                float v[32];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 x = job.s0 ? reinterpret_cast<const float4*>(job.s0 + state_off + 32 * c)[i]
                                            : make_float4(0.f, 0.f, 0.f, 0.f);
                    v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
                }
                tmem_st32(trow + T_S + 32 * c, v);
            }
            tmem_st_wait();
        }
        bool ok = true;
        int j = 0, slot = -1;   // slot: where the last chunk's state is dumped
        for (; w.more(); w.next(), ++j) {
            if (j > 0) {
                ok = warp_wait(st_done, j - 1);
                if (!ok) break;
                tc_fence_after();
                if (slot >= 0) dump(p.ckpt_states + (size_t)slot * p.H * D * D + state_off);
            }
            const float2 decay = make_float2(pw[w.n], pw[w.n]);
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
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
            slot = w.dump() ? p.ckpts[w.ck].slot : -1;
        }
        if (ok && j > 0) {
            ok = warp_wait(st_done, j - 1);
            if (ok) {
                tc_fence_after();
                if (slot >= 0) dump(p.ckpt_states + (size_t)slot * p.H * D * D + state_off);
                if (job.s_final) dump(job.s_final + state_off);
            }
        } else if (ok && job.s_final) {
            // no tokens: the final state is the initial one
            for (int i = 0; i < D; i += 4)
                *reinterpret_cast<float4*>(job.s_final + state_off + i) =
                    job.s0 ? *reinterpret_cast<const float4*>(job.s0 + state_off + i) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    } else if (warp < 8) {
        // ---- tokens: lane = token row, this warp's rows are [32 rb, 32 rb + 32) ----
        if (READOUT) {
            const int rb = warp & 3;
            const float rowf = pw[lane], inter = pw[row + 1] * p.scale;
            const float2 inter2 = make_float2(inter, inter), scale2 = make_float2(p.scale, p.scale);
            int held = -1;   // ring slot of the last chunk's Q tile, until its output has been copied out of it
            auto release = [&] {
                if (held >= 0) {
                    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    mbar_arrive(&empty[held]);
                    held = -1;
                }
                __syncwarp();
            };
            for (int j = 0; w.more(); w.next(), ++j) {
                if (!warp_wait(g_done, j)) break;
                tc_fence_after();
#pragma unroll 1
                for (int cb = 0; cb < 4; ++cb) {
                    uint32_t pk[16];
                    if (cb <= rb) {
                        float g[32];
                        tmem_ld32(trow + T_G + 32 * cb, g);
                        if (cb < rb) {
                            // a^{t-s} = a^{lane} a^{32 (rb - cb) - i}: both exponents are at least 0
                            const float4* col = reinterpret_cast<const float4*>(wp + kTok - 32 * (rb - cb));
                            const float2 rf = make_float2(rowf, rowf);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float4 x = col[i];
                                const float2 y0 = __fmul2_rn(__fmul2_rn(make_float2(x.x, x.y), rf), make_float2(g[4 * i], g[4 * i + 1]));
                                const float2 y1 = __fmul2_rn(__fmul2_rn(make_float2(x.z, x.w), rf), make_float2(g[4 * i + 2], g[4 * i + 3]));
                                pk[2 * i] = pack2(y0.x, y0.y), pk[2 * i + 1] = pack2(y1.x, y1.y);
                            }
                        } else {
                            const float* d = wp + kTok - lane;   // d[i] = a^{lane - i}, not read past the diagonal
#pragma unroll
                            for (int i = 0; i < 32; ++i) g[i] = i <= lane ? g[i] * d[i] : 0.f;
#pragma unroll
                            for (int i = 0; i < 16; ++i) pk[i] = pack2(g[2 * i], g[2 * i + 1]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) pk[i] = 0u;
                    }
                    tmem_st16(trow + T_G + 16 * cb, pk);   // over the columns of G that are read by now
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(p_ready);
                release();
                if (!warp_wait(o_done, j)) break;
                tc_fence_after();
                const int qs = PER * j + 1;
                const bool whole = w.n == kTok;
                __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) + ((job.tok_begin + w.pos + row) * p.H + h) * (int64_t)D;
                // A whole chunk is staged in its spent Q tile and copied out by TMA: a thread holds a row, and 16-byte
                // stores of 32 rows at a time took 3100 of the 8300 cycles of a chunk.  A cut one is stored directly.
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    float x[32], y[32];
                    tmem_ld32x2(trow + T_O1 + 32 * c, trow + T_O2 + 32 * c, x, y);
                    unsigned char* piece = smem + tile(qs) + (c >> 1) * 16384;
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        uint32_t u[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int k = i + 2 * e;
                            const float2 z = __ffma2_rn(inter2, make_float2(x[k], x[k + 1]),
                                                        __fmul2_rn(scale2, make_float2(y[k], y[k + 1])));
                            u[e] = pack2(z.x, z.y);
                        }
                        const uint4 q4 = make_uint4(u[0], u[1], u[2], u[3]);
                        if (whole)
                            *reinterpret_cast<uint4*>(piece + sw128(row, (c & 1) * 32 + i)) = q4;
                        else if (row < w.n)
                            *reinterpret_cast<uint4*>(dst + 32 * c + i) = q4;
                    }
                }
                proxy_fence();
                tc_fence_before();
                mbar_arrive(o_free);
                mbar_arrive(o_staged);
                bool staged = true;
                if (tid == 128) {
                    staged = wait_bar(o_staged, (uint32_t)j & 1u, abort_flag, limit);
                    if (staged && whole) {
                        const int t0 = (int)(job.tok_begin + w.pos);
                        tma_store_3d(smem + tile(qs), &p.tm_o, 0, h, t0);
                        tma_store_3d(smem + tile(qs) + 16384, &p.tm_o, 64, h, t0);
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    }
                    held = qs % ST;
                }
                if (!__all_sync(0xffffffffu, staged)) break;
            }
            release();
        }
    } else if (warp < 12) {
        // ---- keys: row = token s ----
        for (int j = 0; w.more(); w.next(), ++j) {
            const int ks = PER * j, vs = PER * j + PER - 1;
            // G has read K; the last update has read K' lo
            if (READOUT && !warp_wait(g_done, j)) break;
            if (!warp_wait(&full[ks % ST], full_parity(ks))) break;
            if (j > 0 && !warp_wait(st_done, j - 1)) break;
            const bool in = row < w.n;
            const float f = in ? pw[w.n - 1 - row] : 0.f;
            unsigned char* hi = smem + tile(ks);
            unsigned char* lo = smem + OFF_KLO;
            const float2 f2 = make_float2(f, f);
#pragma unroll 1
            for (int c0 = 0; c0 < 4; ++c0) {
                // all loads of a quarter row before its stores: the compiler may not move a load over a store
                uint4 x[4];
                const uint32_t off = (c0 >> 1) * 16384 + row * 128;
#pragma unroll
                for (int c = 0; c < 4; ++c)   // past the chunk: another chunk's or sequence's keys, not taken in
                    x[c] = in ? *reinterpret_cast<const uint4*>(hi + off + (((4 * (c0 & 1) + c) ^ (row & 7)) << 4))
                              : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t a[4] = {x[c].x, x[c].y, x[c].z, x[c].w}, b[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 y = __fmul2_rn(bf16x2_to_float2(a[i]), f2);
                        split_pair(y.x, y.y, a[i], b[i]);
                    }
                    const uint32_t at = off + (((4 * (c0 & 1) + c) ^ (row & 7)) << 4);
                    *reinterpret_cast<uint4*>(hi + at) = make_uint4(a[0], a[1], a[2], a[3]);
                    *reinterpret_cast<uint4*>(lo + at) = make_uint4(b[0], b[1], b[2], b[3]);
                }
            }
            if (w.n < kTok) {
                if (!warp_wait(&full[vs % ST], full_parity(vs))) break;
                if (!in) {
                    unsigned char* v = smem + tile(vs) + row * 128;
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        *reinterpret_cast<uint4*>(v + (c >> 3) * 16384 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                }
            }
            proxy_fence();
            mbar_arrive(k_ready);
        }
    } else if (warp == 12) {
        // ---- products ----
        if (lane == 0) {
            const uint32_t id = idesc(D, false, false), id_b = idesc(D, false, true), id_ab = idesc(D, true, true);
            auto wait = [&](uint64_t* bar, int parity) { return wait_bar(bar, (uint32_t)parity & 1u, abort_flag, limit); };
            for (int j = 0; w.more(); w.next(), ++j) {
                const int ks = PER * j, qs = ks + 1, vs = PER * j + PER - 1;
                const uint32_t k = sbase + tile(ks), q = sbase + tile(qs), v = sbase + tile(vs);
                if (READOUT) {
                    if (!wait(&full[ks % ST], full_parity(ks)) || !wait(&full[qs % ST], full_parity(qs))) break;
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        const uint32_t off = (uint32_t)((kk >> 2) * 16384 + (kk & 3) * 32);
                        umma_ss(tbase + T_G, sdesc(q + off, 16, 1024), sdesc(k + off, 16, 1024), id, kk > 0);
                    }
                    umma_commit(g_done);
                }
                if (!wait(s_ready, j)) break;
                if (READOUT) {
                    if (j > 0 && !wait(o_free, j - 1)) break;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        const uint32_t off = (uint32_t)((kk >> 2) * 16384 + (kk & 3) * 32);
                        umma_ss(tbase + T_O1, sdesc(q + off, 16, 1024), sdesc(sbase + OFF_S + off, 16, 1024), id, kk > 0);
                    }
                }
                if (!wait(&full[vs % ST], full_parity(vs))) break;
                if (READOUT) {
                    if (!wait(p_ready, j)) break;
                    if (w.n < kTok && !wait(k_ready, j)) break;   // a cut chunk's value rows are zeroed by then
                    tc_fence_after();
#pragma unroll
                    for (int kt = 0; kt < 8; ++kt)
                        umma_ts(tbase + T_O2, tbase + T_G + 8 * kt, sdesc(v + kt * 2048, 16384, 1024), id_b, kt > 0);
                    umma_commit(o_done);
                }
                if (!wait(k_ready, j)) break;
                tc_fence_after();
#pragma unroll
                for (int kt = 0; kt < 8; ++kt) {
                    const uint64_t av = sdesc(v + kt * 2048, 16384, 1024);
                    umma_ss(tbase + T_S, av, sdesc(k + kt * 2048, 16384, 1024), id_ab, 1);
                    umma_ss(tbase + T_S, av, sdesc(sbase + OFF_KLO + kt * 2048, 16384, 1024), id_ab, 1);
                }
                umma_commit(st_done);
                umma_commit(&empty[ks % ST]);
                umma_commit(&empty[vs % ST]);
            }
            umma_commit(end);   // also after giving up: the end waits for the products in flight
        }
    } else if (lane == 0) {
        // ---- copies ----
        bool ok = true;
        for (int j = 0; ok && w.more(); w.next(), ++j) {
            if (p.stall_after >= 0 && j >= p.stall_after) break;   // testing hook
            const int t0 = (int)(job.tok_begin + w.pos);
            for (int i = 0; i < PER; ++i) {
                const int seq = PER * j + i, s = seq % ST;
                if (seq >= ST && !wait_bar(&empty[s], (uint32_t)((seq / ST - 1) & 1), abort_flag, limit)) {
                    ok = false;
                    break;
                }
                const CUtensorMap* tm = i == 0 ? &p.tm_k : i == PER - 1 ? &p.tm_v : &p.tm_q;
                const int head = i == PER - 1 ? h : hk;
                mbar_arrive_expect_tx(&full[s], kTile);
                tma_load_3d(smem + s * kTile, tm, 0, head, t0, &full[s]);
                tma_load_3d(smem + s * kTile + 16384, tm, 64, head, t0, &full[s]);
                *issued = seq + 1;
            }
        }
    }

    // ---- leave only with no copy and no product still writing into this CTA's shared memory or TMEM ----
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *abort_flag) {
        const uint64_t drain = limit > kDrainLimitNs ? limit : kDrainLimitNs;
        for (int seq = max(0, *issued - ST); seq < *issued; ++seq)
            tc::drain_phase(&full[seq % ST], (uint32_t)((seq / ST) & 1), drain);
        tc::drain_phase(end, 0, drain);
        atomicOr(p.status, STATUS_TIMEOUT);
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(512));
}

template <bool READOUT>
cudaError_t launch(const Params& p, cudaStream_t s) {
    auto kern = linear_tc_kernel<READOUT>;
    static std::atomic<int> optin[kMaxOptinDevices];
    const cudaError_t e = smem_optin(reinterpret_cast<const void*>(kern), kSmem, optin);
    if (e != cudaSuccess) return e;
    kern<<<p.n_jobs * p.H, kThreads, kSmem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tc(const Params& p, cudaStream_t stream) { return p.o ? launch<true>(p, stream) : launch<false>(p, stream); }

}  // namespace lin
}  // namespace gdn
