// gdn_prefix.cu - attention for a batch that shares a long prefix, on the FP32 pipes (fp32, and bf16 of width 32), and the
// join of the parts.
//
// A CTA takes 16 query rows against one range of tokens, in tiles of 32: a lane scores one token for its warp's 4
// rows, the warp keeps each row's running maximum and sum, and the value product runs with a lane holding D/32
// columns of the 4 rows.  One pass over the keys and values; scores, statistics and sums in fp32.
//
// What bounds it: few rows, latency (7 requests x 8 heads on 2047 + 77 tokens, d = 64, fp32: 17 us for 9.5 MB, join and
// all); many, the FP32 pipes.  The join reads each part's sums once, from the L2 cache.
#include <cuda_bf16.h>

#include <cmath>

#include "gdn_prefix.cuh"

namespace gdn {
namespace prefix {
namespace {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

template <int D, typename T>
__global__ void __launch_bounds__(128) prefix_part_kernel(const __grid_constant__ Params p) {
    constexpr int RT = kSimtRows, KT = kSimtKeys, CL = D / 32;
    __shared__ __align__(16) float sq[RT][D];
    __shared__ __align__(16) float sk[KT][D + 4];   // + 4: a lane's float4 of its own row without bank conflicts
    __shared__ __align__(16) float sv[KT][D];
    __shared__ float sp[RT][KT];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nG = p.n * p.G;
    const int pre_items = p.pre_splits * p.pre_tiles * p.Hkv;
    int item = blockIdx.x;
    const bool pre = item < pre_items;
    int b0 = 0, h, tile, split, lo, hi, len = 0;
    int64_t rows;
    const T *gk, *gv;
    int64_t ks, vs;
    if (pre) {
        h = item % p.Hkv, item /= p.Hkv;
        tile = item % p.pre_tiles;
        split = item / p.pre_tiles;
        rows = (int64_t)p.B * nG;
        lo = split * p.pre_chunk;
        hi = (int)min((int64_t)lo + p.pre_chunk, p.prefix_len);
        gk = static_cast<const T*>(p.kp) + h * p.kp_sh, ks = p.kp_st;
        gv = static_cast<const T*>(p.vp) + h * p.vp_sh, vs = p.vp_st;
    } else {
        item -= pre_items;
        h = item % p.Hkv, item /= p.Hkv;
        tile = item % p.tail_tiles, item /= p.tail_tiles;
        b0 = item % p.B;
        split = item / p.B;
        rows = nG;
        len = min(max(p.tail_len[b0], 0), (int)p.max_tail);
        tail_range(p, len, KT, split, &lo, &hi);
        gk = static_cast<const T*>(p.kt) + b0 * p.kt_sb + h * p.kt_sh, ks = p.kt_st;
        gv = static_cast<const T*>(p.vt) + b0 * p.vt_sb + h * p.vt_sh, vs = p.vt_st;
        split += p.pre_splits;
    }
    const int64_t row0 = (int64_t)tile * RT;
    for (int i = tid; i < RT * D; i += blockDim.x) {
        const int64_t r = row0 + i / D;
        float x = 0.f;
        if (r < rows) {
            const int b = pre ? (int)(r / nG) : b0, e = (int)(r % nG);
            x = to_f(static_cast<const T*>(p.q)[b * p.q_sb + (e / p.G) * p.q_sn + (h * p.G + e % p.G) * p.q_sh + i % D]);
        }
        sq[i / D][i % D] = x;
    }
    int vis[4];   // tokens that each of the warp's rows sees
    float m[4], l[4], acc[4][CL];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int64_t row = row0 + warp * 4 + r;
        vis[r] = row >= rows ? 0 : pre ? hi : min(len, max(0, len - p.n + (int)(row % nG) / p.G + 1));
        m[r] = -INFINITY, l[r] = 0.f;
#pragma unroll
        for (int j = 0; j < CL; ++j) acc[r][j] = 0.f;
    }
    for (int t0 = lo; t0 < hi; t0 += KT) {
        __syncthreads();
        for (int i = tid; i < KT * D; i += blockDim.x) {
            const int t = i / D, x = i % D;
            const bool in = t0 + t < hi;   // past the range: zeros, whatever the buffer holds there
            sk[t][x] = in ? to_f(gk[(int64_t)(t0 + t) * ks + x]) : 0.f;
            sv[t][x] = in ? to_f(gv[(int64_t)(t0 + t) * vs + x]) : 0.f;
        }
        __syncthreads();
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int x = 0; x < D; x += 4) {
            const float4 k4 = *reinterpret_cast<const float4*>(&sk[lane][x]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float4 q4 = *reinterpret_cast<const float4*>(&sq[warp * 4 + r][x]);
                s[r] = fmaf(q4.x, k4.x, fmaf(q4.y, k4.y, fmaf(q4.z, k4.z, fmaf(q4.w, k4.w, s[r]))));
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float x = t0 + lane < min(hi, vis[r]) ? s[r] * p.scale_log2 : -INFINITY;
            float top = x;
#pragma unroll
            for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float mn = fmaxf(m[r], top);
            const float base = mn == -INFINITY ? 0.f : mn;   // nothing seen yet: every term is 2^-inf = 0
            const float f = exp2f(m[r] - base), e = exp2f(x - base);
            m[r] = mn;
            l[r] = l[r] * f + e;   // this lane's tokens; added up at the end
#pragma unroll
            for (int j = 0; j < CL; ++j) acc[r][j] *= f;
            sp[warp * 4 + r][lane] = e;
        }
        __syncwarp();
#pragma unroll 4
        for (int t = 0; t < KT; ++t) {
            float v[CL];
#pragma unroll
            for (int j = 0; j < CL; ++j) v[j] = sv[t][lane + 32 * j];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float e = sp[warp * 4 + r][t];
#pragma unroll
                for (int j = 0; j < CL; ++j) acc[r][j] = fmaf(e, v[j], acc[r][j]);
            }
        }
        __syncwarp();
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int64_t row = row0 + warp * 4 + r;
#pragma unroll
        for (int d = 16; d; d >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], d);
        if (row >= rows) continue;
        const int stacked = (int)(pre ? row : (int64_t)b0 * nG + row);
        const int64_t group = part_group(p, split, h, stacked);
        if (lane == 0) p.part_ml[group * 32 + (stacked & 31)] = make_float2(m[r], l[r]);
#pragma unroll
        for (int j = 0; j < CL; ++j) p.part_o[(group * D + lane + 32 * j) * 32 + (stacked & 31)] = acc[r][j];
    }
}

// o = sum_p 2^(m_p - m) o_p / sum_p 2^(m_p - m) l_p.  A CTA joins CC columns of a group of 32 rows, lane = row, whole lines
// at a time; its 8 warps share the parts and add up in shared memory, so that few rows of many parts are not read one
// behind the other.  Bound by reading the parts (from L2).
constexpr int kJoinWarps = 8;
template <int D, int CC, typename T>
__global__ void __launch_bounds__(32 * kJoinWarps) prefix_join_kernel(const __grid_constant__ Params p, int parts) {
    constexpr int W = kJoinWarps;
    __shared__ float top[W][32], sum[W][CC + 1][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c0 = blockIdx.x % (D / CC) * CC;
    const int g = blockIdx.x / (D / CC) % p.groups, h = blockIdx.x / (D / CC) / p.groups;
    const int nG = p.n * p.G, row = g * 32 + lane;
    const bool valid = row < p.B * nG;
    const int64_t step = (int64_t)p.Hkv * p.groups, first = (int64_t)h * p.groups + g;
    const float2* ml = p.part_ml + first * 32 + lane;
    float m = -INFINITY;
#pragma unroll 4
    for (int s = warp; s < parts; s += W) {
        const float2 x = valid ? ml[s * step * 32] : make_float2(0.f, 0.f);
        if (x.y != 0.f) m = fmaxf(m, x.x);   // (a NaN sum counts as one)
    }
    top[warp][lane] = m;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < W; ++k) m = fmaxf(m, top[k][lane]);
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f, acc[CC];
#pragma unroll
    for (int j = 0; j < CC; ++j) acc[j] = 0.f;
    // parts at a time: few rows have few warps to hide their loads behind (7 rows a head in 67 parts: 17 us with the FP32-pipe
    // kernel against 19 with 1; 16 columns have as many loads in one part)
    constexpr int U = CC == 8 ? 2 : 1;
#pragma unroll 1
    for (int s0 = warp; s0 < parts; s0 += W * U) {
        // every load first, of valid addresses whatever they hold: an empty part's values were not written and are not used
        float2 x[U];
        float y[U][CC];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t at = min(s0 + u * W, parts - 1) * step + first;
            const float* src = p.part_o + (at * D + c0) * 32 + lane;
            x[u] = p.part_ml[at * 32 + lane];
#pragma unroll
            for (int j = 0; j < CC; ++j) y[u][j] = src[32 * j];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool some = valid && s0 + u * W < parts && x[u].y != 0.f;
            const float w = some ? exp2f(x[u].x - base) : 0.f;
            l += some ? w * x[u].y : 0.f;
#pragma unroll
            for (int j = 0; j < CC; ++j) acc[j] = fmaf(w, some ? y[u][j] : 0.f, acc[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < CC; ++j) sum[warp][j][lane] = acc[j];
    sum[warp][CC][lane] = l;
    __syncthreads();
    if (warp != 0 || !valid) return;
#pragma unroll
    for (int k = 1; k < W; ++k) {
        l += sum[k][CC][lane];
#pragma unroll
        for (int j = 0; j < CC; ++j) acc[j] += sum[k][j][lane];
    }
    int e, k;
    const int b = p.by_ng.divmod(row, &e), i = p.by_g.divmod(e, &k);
    const int64_t at = ((int64_t)b * p.n + i) * p.Hq + h * p.G + k;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    struct alignas(16) Out {
        T x[CC];
    } out;
#pragma unroll
    for (int j = 0; j < CC; ++j) put(&out.x[j], acc[j] * inv);
    const uint4* src = reinterpret_cast<const uint4*>(&out);
    uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.o) + at * D + c0);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(Out) / 16); ++i) dst[i] = src[i];
    if (p.lse && c0 == 0) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

template <int D, typename T>
cudaError_t part(const Params& p, cudaStream_t s) {
    const int64_t items = (int64_t)p.Hkv * ((int64_t)p.pre_splits * p.pre_tiles + (int64_t)p.tail_splits * p.tail_tiles * p.B);
    if (items == 0) return cudaSuccess;
    prefix_part_kernel<D, T><<<(unsigned)items, 128, 0, s>>>(p);
    return cudaGetLastError();
}
template <int D, typename T>
cudaError_t join(const Params& p, int parts, cudaStream_t s) {
    // 16 columns a CTA read each row's weights half as often as 8; few rows take 8, for twice the CTAs (64 rows: 6 us against 8)
    const int64_t wide = (int64_t)p.Hkv * p.groups * (D / 16);
    if (wide >= 2 * kSms)
        prefix_join_kernel<D, 16, T><<<(unsigned)wide, 32 * kJoinWarps, 0, s>>>(p, parts);
    else
        prefix_join_kernel<D, 8, T><<<(unsigned)(2 * wide), 32 * kJoinWarps, 0, s>>>(p, parts);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_simt(const Params& p, int D, bool bf16, cudaStream_t s) {
    if (D == 32) return bf16 ? part<32, __nv_bfloat16>(p, s) : part<32, float>(p, s);
    return D == 64 ? part<64, float>(p, s) : part<128, float>(p, s);   // (wider bf16: launch_tc)
}
cudaError_t launch_join(const Params& p, int D, bool bf16, int parts, cudaStream_t s) {
    if (D == 32) return bf16 ? join<32, __nv_bfloat16>(p, parts, s) : join<32, float>(p, parts, s);
    if (D == 64) return bf16 ? join<64, __nv_bfloat16>(p, parts, s) : join<64, float>(p, parts, s);
    return bf16 ? join<128, __nv_bfloat16>(p, parts, s) : join<128, float>(p, parts, s);
}

}  // namespace prefix
}  // namespace gdn
