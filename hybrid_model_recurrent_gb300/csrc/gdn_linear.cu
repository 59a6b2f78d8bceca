// gdn_linear.cu - linear attention with a decay for each head, on the FP32 pipes: the token-by-token scan for
// every size and type, the chaining of a split scan's segments, and the single-token step.
//
// The scan.  Row i of S evolves only from v_{t,i}, so the rows of a head split over warps and CTAs with no
// exchange.  A warp holds 16 rows: 4 row groups of 8 column lanes, a lane 4 rows x d_k/8 columns in registers.
// A token costs three FP32 operations per state element (decay, update, readout) and one reduction of the
// readout over the 8 column lanes.  The recurrence itself is one multiply and one FMA deep; loads and reductions of
// 4 or 8 tokens go together, round by round.  q, k and v arrive by cp.async in tiles of 16 (fp32) or 32 (bf16) tokens,
// 2 to 6 of them at a time.
//
// What bounds it: a few scans, the latency of a token's steps (2 heads of 32 x 32, 256 tokens, fp32: 21 us, 38 with each
// token's reduction by itself and two tiles; 4 heads of 64 x 64, 512 tokens: 58 us, 87); many, the issue of its FP32
// instructions (8 x 16 x 2048, 128 x 128, fp32: 637 us, 20 of the
// pipes' 37 T instructions a second).
//
// The step.  A warp holds 16 or 8 rows of one head's state, read and written once: 268 MB in 46 us (64 requests x 32 heads
// at d = 128, or 256 x 32 at d = 64), a call among others, are 5.9 of the 6.7 TB/s that a copy reaches.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "gdn_linear.cuh"

namespace gdn {
namespace lin {
namespace {

__device__ __forceinline__ uint32_t saddr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
// 16-byte asynchronous copy; bytes = 0 fills with zeros
__device__ __forceinline__ void cp_async(void* dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(saddr(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// N consecutive values as fp32
template <int N>
__device__ __forceinline__ void load_vec(const float* p, float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4 f = *reinterpret_cast<const float4*>(p + i);
        x[i] = f.x, x[i + 1] = f.y, x[i + 2] = f.z, x[i + 3] = f.w;
    }
}
template <int N>
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, float (&x)[N]) {
    static_assert(N == 4 || N == 8, "8 or 16 bytes");
    uint32_t w[N / 2];
    if constexpr (N == 8) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        w[0] = u.x, w[1] = u.y;
    }
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store_out(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// The columns that a lane holds: NV pieces of VW consecutive ones, piece i at (c + 8 i) VW, so that the 8 column
// lanes of a row group read 128 consecutive bytes of a fp32 (or 16-byte pieces of a bf16) vector at a time.
template <int DK, typename T>
struct Cols {
    static constexpr int CT = DK / 8;
    static constexpr int VW = std::is_same<T, float>::value ? 4 : (CT < 8 ? CT : 8);
    static constexpr int NV = CT / VW;
    __device__ static __forceinline__ int at(int c, int i) { return (c + 8 * i) * VW; }
    __device__ static __forceinline__ void load(const T* row, int c, float (&x)[CT]) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float y[VW];
            load_vec<VW>(row + at(c, i), y);
#pragma unroll
            for (int j = 0; j < VW; ++j) x[i * VW + j] = y[j];
        }
    }
    __device__ static __forceinline__ void load_state(const float* row, int c, float (&x)[CT]) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float y[VW];
            load_vec<VW>(row + at(c, i), y);
#pragma unroll
            for (int j = 0; j < VW; ++j) x[i * VW + j] = y[j];
        }
    }
    __device__ static __forceinline__ void store_state(float* row, int c, const float (&x)[CT]) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VW; j += 4)
                *reinterpret_cast<float4*>(row + at(c, i) + j) =
                    make_float4(x[i * VW + j], x[i * VW + j + 1], x[i * VW + j + 2], x[i * VW + j + 3]);
    }
};

// Sums of four rows' partial values of U tokens over the 8 column lanes: each round keeps half of the values and sends the
// other half.  Lane c ends with row c >> 1, of every token for U = 1 (lanes c and c ^ 1 the same sum) and of token 2 i +
// (c & 1) in x[i] otherwise.  All tokens go through a round together: one after the other, each would wait out its three
// shuffles.
template <int U>
__device__ __forceinline__ void reduce_rows(const float (&p)[U][4], int c, float (&x)[(U + 1) / 2]) {
    const bool u4 = c & 4, u2 = c & 2, u1 = c & 1;
    float a[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        a[u] = (u4 ? p[u][2] : p[u][0]) + __shfl_xor_sync(0xffffffffu, u4 ? p[u][0] : p[u][2], 4);
        b[u] = (u4 ? p[u][3] : p[u][1]) + __shfl_xor_sync(0xffffffffu, u4 ? p[u][1] : p[u][3], 4);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) a[u] = (u2 ? b[u] : a[u]) + __shfl_xor_sync(0xffffffffu, u2 ? a[u] : b[u], 2);
    if constexpr (U == 1) {
        x[0] = a[0] + __shfl_xor_sync(0xffffffffu, a[0], 1);
    } else {
#pragma unroll
        for (int u = 0; u < U; u += 2)
            x[u / 2] = (u1 ? a[u + 1] : a[u]) + __shfl_xor_sync(0xffffffffu, u1 ? a[u] : a[u + 1], 1);
    }
}

template <int DK, bool READOUT, typename T, typename OutT>
__global__ void __launch_bounds__(128) linear_scan_kernel(const __grid_constant__ Params p) {
    using CM = Cols<DK, T>;
    constexpr int CT = CM::CT;
    constexpr int kPiece = 16 / (int)sizeof(T);         // elements of a 16-byte copy
    constexpr int kTile = sizeof(T) == 4 ? 16 : 32;     // tokens of a staged tile
    // As many tiles as 48 KB of static memory hold: a narrow one's tokens take less time than its copy from memory.
    constexpr int NB = 49152 / (kTile * (2 * DK + 64) * (int)sizeof(T));
    static_assert(NB >= 2, "a tile being read and one on its way");
    __shared__ __align__(16) T sk[NB][kTile][DK];
    __shared__ __align__(16) T sq[NB][kTile][DK];
    __shared__ __align__(16) T sv[NB][kTile][64];

    const int RB = p.rows_per_cta;
    const int blocks = p.dv / RB;
    const int rb = blockIdx.x % blocks;
    const int h = (blockIdx.x / blocks) % p.H;
    const Job& job = p.jobs[blockIdx.x / (blocks * p.H)];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c = lane & 7, rg = lane >> 3;
    const int row0 = rb * RB + warp * kWarpRows + rg * 4;   // first of this lane's 4 state rows
    const int hk = h / p.rep;
    const int len = job.len;
    const float a = p.alpha[h];
    const size_t head = (size_t)h * p.dv * DK;

    float S[4][CT];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        if (job.s0) {
            CM::load_state(job.s0 + head + (size_t)(row0 + r) * DK, c, S[r]);
        } else {
#pragma unroll
            for (int j = 0; j < CT; ++j) S[r][j] = 0.f;
        }
    }

    const T* gk = static_cast<const T*>(p.k) + job.tok_begin * p.k_stride + (int64_t)hk * DK;
    const T* gq = READOUT ? static_cast<const T*>(p.q) + job.tok_begin * p.q_stride + (int64_t)hk * DK : nullptr;
    const T* gv = static_cast<const T*>(p.v) + job.tok_begin * p.v_stride + (int64_t)h * p.dv + rb * RB;
    OutT* go = READOUT ? static_cast<OutT*>(p.o) + (job.tok_begin * p.H + h) * (int64_t)p.dv + row0 : nullptr;

    const int tiles = (len + kTile - 1) / kTile;
    auto stage = [&](int tile) {   // one group of copies, empty past the end
        const int t0 = tile * kTile, buf = tile % NB;
        for (int i = tid; tile < tiles && i < kTile * (DK / kPiece); i += blockDim.x) {
            const int t = i / (DK / kPiece), x = (i % (DK / kPiece)) * kPiece;
            const int ts = min(t0 + t, len - 1);   // past the end: a valid address, nothing copied
            const int n = t0 + t < len ? 16 : 0;
            cp_async(&sk[buf][t][x], gk + (int64_t)ts * p.k_stride + x, n);
            if (READOUT) cp_async(&sq[buf][t][x], gq + (int64_t)ts * p.q_stride + x, n);
        }
        for (int i = tid; tile < tiles && i < kTile * (RB / kPiece); i += blockDim.x) {
            const int t = i / (RB / kPiece), x = (i % (RB / kPiece)) * kPiece;
            const int ts = min(t0 + t, len - 1);
            cp_async(&sv[buf][t][x], gv + (int64_t)ts * p.v_stride + x, t0 + t < len ? 16 : 0);
        }
        cp_commit();
    };

    int ck = job.ck_begin;
    const int ck_end = job.ck_begin + job.ck_count;
    int next_ck = ck < ck_end ? p.ckpts[ck].pos : INT32_MAX;
#pragma unroll 1
    for (int i = 0; i < NB - 1; ++i) stage(i);
    for (int tile = 0; tile < tiles; ++tile) {
        stage(tile + NB - 1);
        cp_wait<NB - 1>();
        __syncthreads();
        const int buf = tile % NB, n = min(kTile, len - tile * kTile);
        auto tokens = [&](int t, auto count) {
            constexpr int U = decltype(count)::value;
            [[maybe_unused]] float part[U][4];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float kk[CT], vv[4];
                CM::load(sk[buf][t + u], c, kk);
                load_vec<4>(&sv[buf][t + u][warp * kWarpRows + rg * 4], vv);
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int j = 0; j < CT; ++j) S[r][j] = fmaf(vv[r], kk[j], a * S[r][j]);
                if constexpr (READOUT) {
                    float qq[CT];
                    CM::load(sq[buf][t + u], c, qq);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        float x = 0.f;
#pragma unroll
                        for (int j = 0; j < CT; ++j) x = fmaf(S[r][j], qq[j], x);
                        part[u][r] = x;
                    }
                }
            }
            if constexpr (READOUT) {
                float x[(U + 1) / 2];
                reduce_rows<U>(part, c, x);
                const int own = U > 1 ? c & 1 : 0;   // the token of a pair that this lane has
#pragma unroll
                for (int u = 0; u < U; u += 2)
                    if (U > 1 || (c & 1) == 0)
                        store_out(go + (int64_t)(tile * kTile + t + u + own) * p.H * p.dv + (c >> 1), x[u / 2] * p.scale);
            }
        };
        for (int t = 0; t < n;) {
            // up to the next checkpoint without a branch, several tokens at a time: a token's loads, its reduction and its
            // store have no part in the recurrence and overlap the next token's
            const int stop = min(n, next_ck - tile * kTile);
            constexpr int U = CT >= 16 ? 4 : 8;
            for (; t + U <= stop; t += U) tokens(t, std::integral_constant<int, U>{});
            for (; t < stop; ++t) tokens(t, std::integral_constant<int, 1>{});
            if (tile * kTile + t == next_ck) {
                float* dst = p.ckpt_states + (size_t)p.ckpts[ck].slot * p.H * p.dv * DK + head;
#pragma unroll
                for (int r = 0; r < 4; ++r) CM::store_state(dst + (size_t)(row0 + r) * DK, c, S[r]);
                ++ck;
                next_ck = ck < ck_end ? p.ckpts[ck].pos : INT32_MAX;
            }
        }
        __syncthreads();   // the next tile's copies overwrite this buffer
    }
    if (job.s_final) {
#pragma unroll
        for (int r = 0; r < 4; ++r) CM::store_state(job.s_final + head + (size_t)(row0 + r) * DK, c, S[r]);
    }
}

// Initial states of a split scan's segments: start_{j+1} = alpha^L start_j + own_j, in place (slot j holds own_j and
// receives start_{j+1}).  One thread takes four elements of one head's state through all segments; bound by the
// traffic of the states.  alpha^L is formed by binary powers in fp64 (once a block, which lies within one
// head) and rounded once.
__global__ void __launch_bounds__(128) chain_kernel(const __grid_constant__ ChainParams p) {
    const int per_head = p.state / 4;
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;   // per_head is a multiple of the block
    const int e = (int)(i % per_head) * 4;
    const int h = (int)(i / per_head % p.H);
    const Chain& sc = p.scans[i / per_head / p.H];
    __shared__ float w_sh;
    if (threadIdx.x == 0) {
        double y = 1.0, sq = (double)p.alpha[h];
        for (int k = p.seg_len; k; k >>= 1, sq *= sq)
            if (k & 1) y *= sq;
        w_sh = (float)y;
    }
    __syncthreads();
    const float w = w_sh;
    const size_t all = (size_t)p.H * p.state, off = (size_t)h * p.state + e;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (sc.s0) x = *reinterpret_cast<const float4*>(sc.s0 + off);
    float* st = p.states + (size_t)sc.slot * all + off;
    for (int j = 0; j < sc.n; ++j, st += all) {
        const float4 y = *reinterpret_cast<const float4*>(st);
        x.x = fmaf(w, x.x, y.x), x.y = fmaf(w, x.y, y.y), x.z = fmaf(w, x.z, y.z), x.w = fmaf(w, x.w, y.w);
        *reinterpret_cast<float4*>(st) = x;
    }
}

// One token a request.  A warp takes 4 R rows of one (request, head)'s state, held as in the scan (a lane R rows), with
// every load issued before the first use; bound by the state's traffic (read and written once).
template <int DK, int R, typename T, typename OutT>
__global__ void __launch_bounds__(128) linear_step_kernel(const __grid_constant__ StepParams p) {
    using CM = Cols<DK, T>;
    constexpr int CT = CM::CT;
    const int lane = threadIdx.x & 31;
    const int c = lane & 7, rg = lane >> 3;
    const int per_head = p.dv / (4 * R);
    const int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (w >= (int64_t)p.B * p.H * per_head) return;
    const int row0 = ((int)(w % per_head) * 4 + rg) * R;
    const int h = (int)(w / per_head % p.H);
    const int b = (int)(w / per_head / p.H);
    OutT* o = static_cast<OutT*>(p.o) + ((int64_t)b * p.H + h) * p.dv + row0;
    const int64_t slot = p.slots ? p.slots[b] : b;
    // after the reduction lane c holds row c / (8 / R), with 8 / R lanes alike
    const bool writes = c % (8 / R) == 0;
    if (slot < 0 || slot >= p.num_slots) {
        if (writes) store_out(o + c / (8 / R), 0.f);
        return;
    }
    float* st = p.states + ((slot * p.H + h) * p.dv + row0) * DK;
    float S[R][CT], kk[CT], qq[CT], vv[R];
#pragma unroll
    for (int r = 0; r < R; ++r) CM::load_state(st + r * DK, c, S[r]);
    const int hk = h / p.rep;
    CM::load(static_cast<const T*>(p.k) + b * p.k_stride + (int64_t)hk * DK, c, kk);
    CM::load(static_cast<const T*>(p.q) + b * p.q_stride + (int64_t)hk * DK, c, qq);
    const T* v = static_cast<const T*>(p.v) + b * p.v_stride + (int64_t)h * p.dv + row0;
#pragma unroll
    for (int r = 0; r < R; ++r) vv[r] = (float)v[r];
    const float a = p.alpha[h];
    float part[1][R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float x = 0.f;
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            S[r][j] = fmaf(vv[r], kk[j], a * S[r][j]);
            x = fmaf(S[r][j], qq[j], x);
        }
        part[0][r] = x;
        CM::store_state(st + r * DK, c, S[r]);
    }
    float sum[1];
    if constexpr (R == 4) {
        reduce_rows<1>(part, c, sum);
    } else {
        static_assert(R == 2, "rows of a lane");
        const bool up = c & 4;
        float x = (up ? part[0][1] : part[0][0]) + __shfl_xor_sync(0xffffffffu, up ? part[0][0] : part[0][1], 4);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        sum[0] = x + __shfl_xor_sync(0xffffffffu, x, 1);
    }
    if (writes) store_out(o + c / (8 / R), sum[0] * p.scale);
}

template <int DK>
cudaError_t scan_types(const Params& p, bool in_bf16, bool out_bf16, cudaStream_t s) {
    const int grid = p.n_jobs * p.H * (p.dv / p.rows_per_cta);
    const int threads = 32 * (p.rows_per_cta / kWarpRows);
    auto run = [&](auto kernel) { kernel<<<grid, threads, 0, s>>>(p); };
    using B = __nv_bfloat16;
    if (!p.o) in_bf16 ? run(linear_scan_kernel<DK, false, B, float>) : run(linear_scan_kernel<DK, false, float, float>);
    else if (in_bf16) out_bf16 ? run(linear_scan_kernel<DK, true, B, B>) : run(linear_scan_kernel<DK, true, B, float>);
    else out_bf16 ? run(linear_scan_kernel<DK, true, float, B>) : run(linear_scan_kernel<DK, true, float, float>);
    return cudaGetLastError();
}

template <int DK>
cudaError_t step_types(const StepParams& p, bool in_bf16, bool out_bf16, cudaStream_t s) {
    // rows of a lane: 2 keep twice the warps in flight (GPU time, 64 requests x 32 heads at d = 128: 43 us against 57 with 4;
    // 256 x 32 at d = 64, fp32: 44 against 51); at d_k = 32 a lane has 16 bytes of a row and takes 4
    constexpr int R = DK >= 64 ? 2 : 4;
    const int64_t warps = (int64_t)p.B * p.H * (p.dv / (4 * R));
    const int per = 4;
    const int grid = (int)((warps + per - 1) / per), threads = 32 * per;
    if (in_bf16 && out_bf16) linear_step_kernel<DK, R, __nv_bfloat16, __nv_bfloat16><<<grid, threads, 0, s>>>(p);
    else if (in_bf16) linear_step_kernel<DK, R, __nv_bfloat16, float><<<grid, threads, 0, s>>>(p);
    else if (out_bf16) linear_step_kernel<DK, R, float, __nv_bfloat16><<<grid, threads, 0, s>>>(p);
    else linear_step_kernel<DK, R, float, float><<<grid, threads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_simt(const Params& p, int dk, bool in_bf16, bool out_bf16, cudaStream_t stream) {
    if (dk == 32) return scan_types<32>(p, in_bf16, out_bf16, stream);
    if (dk == 64) return scan_types<64>(p, in_bf16, out_bf16, stream);
    return scan_types<128>(p, in_bf16, out_bf16, stream);
}
cudaError_t launch_step(const StepParams& p, int dk, bool in_bf16, bool out_bf16, cudaStream_t stream) {
    if (dk == 32) return step_types<32>(p, in_bf16, out_bf16, stream);
    if (dk == 64) return step_types<64>(p, in_bf16, out_bf16, stream);
    return step_types<128>(p, in_bf16, out_bf16, stream);
}
cudaError_t launch_chain(const ChainParams& p, cudaStream_t stream) {
    const int64_t n = (int64_t)p.n_scans * p.H * (p.state / 4);
    chain_kernel<<<(unsigned)((n + 127) / 128), 128, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace lin
}  // namespace gdn
