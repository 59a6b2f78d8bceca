// gdn_cache.cu - kernels around a paged 8-bit cache: norm of the heads and rotation in one pass, append with a
// power-of-two scale a block, and the upkeep of pages (free, fork, growth with copy on write, compaction).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cfloat>

#include "gdn_cache.cuh"

namespace gdn {
namespace cache {
namespace {

// 16 bytes of T as fp32, and back
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(const uint4& u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void get(const uint4& u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};

// ---- norm and rotation ----------------------------------------------------------------------------------------------
//
// A warp takes a share of one token's heads, L = D / (2 N) lanes a head and 32 / L heads at a time.  A lane holds two
// 16-byte pieces of its head that make whole pairs (the pieces i and i + rotary_dim / 2 apart, or two neighbours), so the
// rotation needs no exchange, and it has the same N pairs in every head: their sines are formed once a token.
//
// An angle is position * frequency.  The frequency is held as a 64-bit fraction of a turn, so the product's low 64 bits
// are the angle without whole turns, to 2^-33 of a turn at any position; the nearest quarter turn is then
// taken off as an integer, and what is left (an eighth of a turn at most) goes to fp32.
//
// Bound by memory: each element is read and written once.
template <typename T, int D, bool HALF>
__global__ void __launch_bounds__(128) rope_kernel(const __grid_constant__ RopeParams p) {
    using V = Vec<T>;
    constexpr int N = V::N, L = D / (2 * N), HP = 32 / L, U = 2;
    const int lane = threadIdx.x & 31, j = lane % L, hsub = lane / L;
    const int heads = p.Hq + p.Hk;
    const bool turned = 2 * N * j < p.rd;
    // the lane's two pieces, in elements
    int ea, eb;
    if (HALF) {
        ea = (turned ? j : 2 * j) * N;
        eb = turned ? ea + p.rd / 2 : ea + N;
    } else {
        ea = 2 * j * N, eb = ea + N;
    }
    uint64_t freq[N];
    float wq[2][N], wk[2][N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        freq[i] = 0;
        wq[0][i] = wq[1][i] = wk[0][i] = wk[1][i] = 1.f;
    }
    if (turned) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const double turns = p.inv_freq[j * N + i] * 0.15915494309189535;
            freq[i] = __double2ull_rn((turns - floor(turns)) * 18446744073709551616.0);
        }
    }
    if (p.normalize) {
        if (p.qw) {
            V::get(*reinterpret_cast<const uint4*>(static_cast<const T*>(p.qw) + ea), wq[0]);
            V::get(*reinterpret_cast<const uint4*>(static_cast<const T*>(p.qw) + eb), wq[1]);
        }
        if (p.kw) {
            V::get(*reinterpret_cast<const uint4*>(static_cast<const T*>(p.kw) + ea), wk[0]);
            V::get(*reinterpret_cast<const uint4*>(static_cast<const T*>(p.kw) + eb), wk[1]);
        }
    }
    const int64_t units = p.T * p.parts, warps = (int64_t)gridDim.x * 4;
    for (int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5); u < units; u += warps) {
        const int64_t t = u / p.parts;
        const int first = (int)(u - t * p.parts) * p.per_part, last = min(first + p.per_part, (heads + HP - 1) / HP);
        float cs[N], sn[N];
        const int64_t pos = turned ? p.positions[t] : 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint64_t a = (uint64_t)pos * freq[i];
            const uint32_t quarter = (uint32_t)((a + (1ull << 61)) >> 62);
            const int64_t rest = (int64_t)(a - ((uint64_t)quarter << 62));
            float s, c;
            sincospif(__ll2float_rn(rest) * 1.0842021724855044e-19f, &s, &c);   // 2^-63: half turns
            const float cc = quarter & 1 ? s : c, ss = quarter & 1 ? c : s;
            cs[i] = ((quarter + 1) & 2 ? -cc : cc) * p.mscale;
            sn[i] = (quarter & 2 ? -ss : ss) * p.mscale;
        }
        for (int g = first; g < last; g += U) {
            uint4 in[U][2];
#pragma unroll
            for (int x = 0; x < U; ++x) {
                const int head = (g + x) * HP + hsub;
                if (g + x < last && head < heads) {
                    const T* src = head < p.Hq ? static_cast<const T*>(p.q) + t * p.q_stride + head * D
                                               : static_cast<const T*>(p.k) + t * p.k_stride + (head - p.Hq) * D;
                    in[x][0] = *reinterpret_cast<const uint4*>(src + ea);
                    in[x][1] = *reinterpret_cast<const uint4*>(src + eb);
                } else {
                    in[x][0] = in[x][1] = make_uint4(0, 0, 0, 0);
                }
            }
#pragma unroll
            for (int x = 0; x < U; ++x) {
                const int head = (g + x) * HP + hsub;
                const bool is_q = head < p.Hq;
                float a[N], b[N];
                V::get(in[x][0], a);
                V::get(in[x][1], b);
                if (p.normalize) {
                    float sum = 0.f;
#pragma unroll
                    for (int i = 0; i < N; ++i) sum = fmaf(a[i], a[i], sum), sum = fmaf(b[i], b[i], sum);
#pragma unroll
                    for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    const float r = rsqrtf(sum * (1.f / D) + p.eps);
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        a[i] *= r * (is_q ? wq[0][i] : wk[0][i]);
                        b[i] *= r * (is_q ? wq[1][i] : wk[1][i]);
                    }
                }
                if (turned) {
                    if (HALF) {
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            const float y = a[i];
                            a[i] = y * cs[i] - b[i] * sn[i];
                            b[i] = b[i] * cs[i] + y * sn[i];
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < N / 2; ++i) {
                            const float y = a[2 * i], z = b[2 * i];
                            a[2 * i] = y * cs[i] - a[2 * i + 1] * sn[i];
                            a[2 * i + 1] = a[2 * i + 1] * cs[i] + y * sn[i];
                            b[2 * i] = z * cs[N / 2 + i] - b[2 * i + 1] * sn[N / 2 + i];
                            b[2 * i + 1] = b[2 * i + 1] * cs[N / 2 + i] + z * sn[N / 2 + i];
                        }
                    }
                }
                if (g + x < last && head < heads) {
                    T* dst = is_q ? static_cast<T*>(p.q_out) + t * p.qo_stride + head * D
                                  : static_cast<T*>(p.k_out) + t * p.ko_stride + (head - p.Hq) * D;
                    *reinterpret_cast<uint4*>(dst + ea) = V::put(a);
                    *reinterpret_cast<uint4*>(dst + eb) = V::put(b);
                }
            }
        }
    }
}

template <typename T, int D>
cudaError_t rope(const RopeParams& p, bool half, cudaStream_t s) {
    const int64_t units = p.T * p.parts, need = (units + 3) / 4;
    // four CTAs of 128 threads a multiprocessor's worth of registers hold; more units than that take turns
    const unsigned grid = (unsigned)std::min<int64_t>(need, (int64_t)kSms * 8);
    if (half) rope_kernel<T, D, true><<<grid, 128, 0, s>>>(p);
    else rope_kernel<T, D, false><<<grid, 128, 0, s>>>(p);
    return cudaGetLastError();
}

// ---- append -----------------------------------------------------------------------------------------------------------
//
// A block (page x head, keys or values) is taken by TPB threads: they read its new tokens once into registers, agree on the
// largest value, and write the bytes.  Tokens that the block holds already are touched only when the scale grows.
// TPB is 32 for calls with at most 8 new tokens a request (decode, drafts: a block has little to do, and eight of them
// share a CTA), 256 else.
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t u) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)u, __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// the exponent of the least power of two with which `top` is at most 448 (1.75 * 2^8) times it: the bits below 1.75 carry
__device__ __forceinline__ int scale_exponent(float top) {
    return min(max((int)((__float_as_uint(top) + 0x1fffffu) >> 23) - 127 - 8, -126), 120);
}

template <typename T, int D, int TPB, int NCH>
__global__ void __launch_bounds__(256) append_kernel(const __grid_constant__ AppendParams p) {
    constexpr int PER = 256 / TPB;            // blocks of a CTA
    constexpr int VEC = 16 / sizeof(T), LD = 8 / VEC;   // a chunk is 8 values: LD loads
    constexpr int CPT = D / 8;                // chunks of a token
    __shared__ float s_top[8];
    const Cache& c = p.c;
    const int tid = threadIdx.x % TPB, sub = threadIdx.x / TPB;
    const int blocks = 2 * c.Hkv, groups = (blocks + PER - 1) / PER;
    const int b = blockIdx.y;
    const int i0 = blockIdx.x / groups, block = (blockIdx.x - i0 * groups) * PER + sub;
    const Request rq = request_at(c, p.t, b);
    if (rq.bad && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.status, STATUS_BAD_INDEX);
    if (rq.row < 0 || rq.n == 0 || rq.bad) return;
    const int start = max(rq.len - rq.n, 0), skip = max(rq.n - rq.len, 0);   // (new tokens before a row's first position)
    const int i = (start >> c.page_log2) + i0, base = i << c.page_log2;
    if (base >= rq.len) return;
    const int pg = c.table[(int64_t)rq.row * c.W + i];
    if (pg < 0 || pg >= c.N) {
        if (threadIdx.x == 0) atomicOr(p.status, STATUS_BAD_INDEX);
        return;
    }
    const int lo = max(start - base, 0), n = min(rq.len - base, c.page) - lo;   // the block's new tokens: lo .. lo + n
    const bool work = block < blocks;
    const int kv = block >= c.Hkv, h = block - kv * c.Hkv;
    const T* src = (kv ? static_cast<const T*>(p.v) + (rq.first + skip + (int64_t)(base + lo - start)) * p.v_stride
                       : static_cast<const T*>(p.k) + (rq.first + skip + (int64_t)(base + lo - start)) * p.k_stride) + h * D;
    const int64_t stride = kv ? p.v_stride : p.k_stride;
    const int64_t at = ((int64_t)pg * 2 + kv) * c.Hkv + h;
    const int chunks = work ? n * CPT : 0;
    float was = 0.f;
    if (work && lo > 0) was = c.scales[at];   // (before anyone writes it)

    uint4 in[NCH][LD];
#pragma unroll
    for (int x = 0; x < NCH; ++x) {
        const int ch = x * TPB + tid;
        if (ch < chunks) {
            const T* a = src + (int64_t)(ch / CPT) * stride + (ch % CPT) * 8;
#pragma unroll
            for (int y = 0; y < LD; ++y) in[x][y] = *reinterpret_cast<const uint4*>(a + y * VEC);
        }
    }
    float top = 0.f;
#pragma unroll
    for (int x = 0; x < NCH; ++x) {
        if (x * TPB + tid < chunks) {
#pragma unroll
            for (int y = 0; y < LD; ++y) {
                float f[VEC];
                Vec<T>::get(in[x][y], f);
#pragma unroll
                for (int z = 0; z < VEC; ++z) top = fmaxf(top, fabsf(f[z]) <= FLT_MAX ? fabsf(f[z]) : 0.f);
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (TPB > 32) {
        if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = top;
        __syncthreads();
#pragma unroll
        for (int x = 0; x < 8; ++x) top = fmaxf(top, s_top[x]);
    } else {
        __syncwarp();   // every lane has `was`
    }
    if (!work) return;
    float scale = __uint_as_float((uint32_t)(scale_exponent(top) + 127) << 23);
    const bool grows = lo > 0 && scale > was;
    if (lo > 0 && !grows) scale = was;
    const float inv = 1.f / scale;
    unsigned char* dst = c.pages + at * c.page * D;
#pragma unroll
    for (int x = 0; x < NCH; ++x) {
        const int ch = x * TPB + tid;
        if (ch < chunks) {
            float f[8];
#pragma unroll
            for (int y = 0; y < LD; ++y) {
                float g[VEC];
                Vec<T>::get(in[x][y], g);
#pragma unroll
                for (int z = 0; z < VEC; ++z) f[y * VEC + z] = fabsf(g[z]) <= FLT_MAX ? g[z] * inv : __uint_as_float(0x7fc00000u);
            }
            *reinterpret_cast<uint2*>(dst + (int64_t)lo * D + ch * 8) =
                make_uint2(to_e4m3x4(f[0], f[1], f[2], f[3]), to_e4m3x4(f[4], f[5], f[6], f[7]));
        }
    }
    if (grows) {
        const float ratio = was * inv;   // a power of two
        for (int ch = tid; ch < lo * CPT; ch += TPB) {
            uint2* a = reinterpret_cast<uint2*>(dst + ch * 8);
            uint2 u = *a;
            const float2 x0 = from_e4m3x2(u.x & 0xffff), x1 = from_e4m3x2(u.x >> 16), x2 = from_e4m3x2(u.y & 0xffff),
                         x3 = from_e4m3x2(u.y >> 16);
            u = make_uint2(to_e4m3x4(x0.x * ratio, x0.y * ratio, x1.x * ratio, x1.y * ratio),
                           to_e4m3x4(x2.x * ratio, x2.y * ratio, x3.x * ratio, x3.y * ratio));
            *a = u;
        }
    }
    if (tid == 0) c.scales[at] = scale;
}

template <typename T, int D, int TPB, int NCH>
cudaError_t append_n(const AppendParams& p, cudaStream_t s) {
    const int touched = (p.t.max_new + p.c.page - 2) / p.c.page + 1;   // pages that a request's new tokens may lie in
    const int groups = (2 * p.c.Hkv + 256 / TPB - 1) / (256 / TPB);
    append_kernel<T, D, TPB, NCH><<<dim3(touched * groups, p.t.B), 256, 0, s>>>(p);
    return cudaGetLastError();
}
template <typename T, int D>
cudaError_t append_d(const AppendParams& p, cudaStream_t s) {
    const int most = std::min(p.t.max_new, p.c.page) * (D / 8);   // chunks of a block
    if (p.t.max_new <= 8) return most <= 32 ? append_n<T, D, 32, 1>(p, s) : append_n<T, D, 32, (D / 8 + 3) / 4>(p, s);
    if (most <= 256) return append_n<T, D, 256, 1>(p, s);
    if (most <= 512) return append_n<T, D, 256, 2>(p, s);
    if constexpr (D >= 64)
        if (most <= 1024) return append_n<T, D, 256, 4>(p, s);
    if constexpr (D >= 128) return append_n<T, D, 256, 8>(p, s);
    return cudaErrorInvalidValue;   // (a page has at most 128 tokens)
}

// ---- upkeep of pages ------------------------------------------------------------------------------------------------
//
// The tables are small and their changes depend on one another, so one CTA makes them; the copies of pages that it asks
// for follow in a launch of their own over the whole GPU.  Pages are found in rising order by scanning the holders'
// counts, 16384 a round (64 KB), as far as there is need: no list of free pages has to be kept in step with them.
constexpr int kCtl = 1024;

// Counts change under atomics and are read past the L1 cache.
__device__ __forceinline__ int now(const int32_t* p) { return __ldcg(p); }

// exclusive prefix sum of x over the CTA's threads; *total: of all.  Every thread calls it.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* s_part, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
    }
    if (lane == 31) s_part[warp] = y;
    __syncthreads();
    if (warp == 0) {
        int64_t z = s_part[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t w = __shfl_up_sync(0xffffffffu, z, o);
            if (lane >= o) z += w;
        }
        s_part[lane] = z;
    }
    __syncthreads();
    const int64_t before = warp ? s_part[warp - 1] : 0;
    *total = s_part[31];
    __syncthreads();
    return before + y - x;
}

// 16 counts from `at` on; -1 behind the last
__device__ __forceinline__ void load16(const int32_t* refs, int N, int at, int (&x)[16]) {
    if (at + 16 <= N && (reinterpret_cast<uintptr_t>(refs) & 15) == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int4 v = __ldcg(reinterpret_cast<const int4*>(refs + at) + i);
            x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = at + i < N ? now(refs + at + i) : -1;
    }
}

__global__ void __launch_bounds__(kCtl) update_kernel(const __grid_constant__ UpkeepParams p) {
    extern __shared__ int32_t s_rows[];   // [R] pages needed, then their first one; [R] the fork that a row is; bit 30: freed
    int32_t* s_need = s_rows;
    int32_t* s_fork = s_rows + p.R;
    __shared__ int64_t s_part[32];
    __shared__ int s_copies;
    constexpr int kNone = 0x7fffffff;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto pages_of = [&](int len) { return min((int)(((int64_t)max(len, 0) + p.page - 1) >> p.page_log2), p.W); };
    auto good = [&](int pg) {
        const bool ok = pg >= 0 && pg < p.N;
        if (!ok) atomicOr(p.status, STATUS_BAD_INDEX);
        return ok;
    };
    if (tid == 0) s_copies = 0;
    for (int r = tid; r < p.R; r += kCtl) s_need[r] = 0, s_fork[r] = kNone;
    __syncthreads();

    // which rows give up their pages, and which pair each fork follows (the first that names it)
    for (int i = tid; i < p.n_drop; i += kCtl) {
        const int r = p.drop[i];
        if (r >= 0 && r < p.R) s_need[r] = 1;
    }
    for (int i = tid; i < p.n_fork; i += kCtl) {
        const int a = p.from[i], r = p.to[i];
        if (a < 0 || a >= p.R || r < 0 || r >= p.R || a == r) continue;
        s_need[r] = 1;
        atomicMin(&s_fork[r], i);
    }
    __syncthreads();
    if (p.n_drop + p.n_fork > 0) {
        for (int r = warp; r < p.R; r += kCtl / 32) {
            if (!s_need[r]) continue;
            const int used = pages_of(p.lens[r]);
            for (int w = lane; w < used; w += 32) {
                const int pg = p.table[(int64_t)r * p.W + w];
                if (good(pg)) atomicSub(&p.refs[pg], 1);
            }
            __syncwarp();
            if (lane == 0) p.lens[r] = 0;
        }
        __syncthreads();
        for (int r = warp; r < p.R; r += kCtl / 32) {
            if (s_fork[r] == kNone) continue;
            const int a = p.from[s_fork[r]];
            if (s_need[a]) continue;   // freed just now: an empty row
            const int len = p.lens[a], used = pages_of(len);
            for (int w = lane; w < p.W; w += 32) {
                const int pg = p.table[(int64_t)a * p.W + w];
                p.table[(int64_t)r * p.W + w] = pg;
                if (w < used && good(pg)) atomicAdd(&p.refs[pg], 1);
            }
            if (lane == 0) p.lens[r] = len;
        }
        __syncthreads();
    }
    if (!p.grow) {
        if (tid == 0) *p.n_copies = 0;
        return;
    }

    // pages that each row needs, and their places among all that are taken.  s_need: the first place; s_fork: bit 31 refused,
    // bit 30 copy the last page, below: the number of pages
    constexpr unsigned kRefused = 1u << 31, kCopy = 1u << 30;
    int64_t carry = 0;
    for (int r0 = 0; r0 < p.R; r0 += kCtl) {
        const int r = r0 + tid;
        int need = 0;
        unsigned flags = 0;
        if (r < p.R) {
            const int len = max(p.lens[r], 0), more = max(p.grow[r], 0);
            if ((int64_t)len + more > (int64_t)p.W * p.page) {
                flags = kRefused;
            } else if (more > 0) {
                const int have = pages_of(len);
                need = pages_of(len + more) - have;
                if (len & (p.page - 1)) {
                    const int last = p.table[(int64_t)r * p.W + have - 1];
                    if (good(last) && now(p.refs + last) > 1) ++need, flags = kCopy;
                }
            }
        }
        int64_t total;
        const int64_t first = carry + block_scan(need, s_part, &total);
        carry += total;
        if (r < p.R) {
            s_need[r] = (int)min(first, (int64_t)kNone);
            s_fork[r] = (int)(flags | (unsigned)need);
        }
    }
    // the free pages with the lowest numbers, as many as are needed
    int64_t found = 0;
    for (int base = 0; base < p.N && found < carry; base += kCtl * 16) {
        int x[16], c = 0;
        load16(p.refs, p.N, base + 16 * tid, x);
#pragma unroll
        for (int i = 0; i < 16; ++i) c += x[i] == 0;
        int64_t total;
        int64_t at = found + block_scan(c, s_part, &total);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (x[i] == 0) {
                if (at < carry) p.free_list[at] = base + 16 * tid + i;
                ++at;
            }
        found += total;
    }
    __syncthreads();
    for (int r = warp; r < p.R; r += kCtl / 32) {
        const unsigned f = (unsigned)s_fork[r];
        const int need = (int)(f & (kCopy - 1)), first = s_need[r];
        const bool copy = f & kCopy;
        const int more = max(p.grow[r], 0);
        if ((f & kRefused) || (need > 0 && (int64_t)first + need > found)) {
            if (lane == 0 && p.granted) p.granted[r] = -1;
            continue;
        }
        const int len = max(p.lens[r], 0), have = pages_of(len);
        int32_t* row = p.table + (int64_t)r * p.W;
        for (int w = lane; w < need; w += 32) {
            const int pg = __ldcg(p.free_list + first + w);
            p.refs[pg] = 1;
            if (copy && w == 0) {
                const int old = row[have - 1];
                const int at = atomicAdd(&s_copies, 1);
                p.copy_from[at] = old, p.copy_to[at] = pg;
                atomicSub(&p.refs[old], 1);
                row[have - 1] = pg;
            } else {
                row[have + w - copy] = pg;
            }
        }
        if (lane == 0) {
            if (more > 0) p.lens[r] = len + more;
            if (p.granted) p.granted[r] = more;
        }
    }
    __syncthreads();
    if (tid == 0) *p.n_copies = s_copies;
}

__global__ void __launch_bounds__(kCtl) compact_kernel(const __grid_constant__ UpkeepParams p) {
    __shared__ int64_t s_part[32];
    const int tid = threadIdx.x;
    int64_t n = 0;
    for (int base = 0; base < p.N; base += kCtl * 16) {
        int x[16];
        load16(p.refs, p.N, base + 16 * tid, x);
#pragma unroll
        for (int i = 0; i < 16; ++i) n += x[i] > 0;
    }
    int64_t live;
    block_scan(n, s_part, &live);
    // holes below `live` and pages in use from it on, the k-th of the ones to the k-th of the others; counted together, the
    // holes in the low half
    int64_t found = 0;
    for (int base = 0; base < p.N; base += kCtl * 16) {
        int x[16];
        load16(p.refs, p.N, base + 16 * tid, x);
        int64_t c = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int pg = base + 16 * tid + i;
            if (pg >= p.N) break;
            if (pg < live) c += x[i] <= 0;
            else c += x[i] > 0 ? 1ll << 32 : 0;
        }
        int64_t total;
        const int64_t at = found + block_scan(c, s_part, &total);
        int hole = (int)(at & 0xffffffff), mover = (int)(at >> 32);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int pg = base + 16 * tid + i;
            if (pg >= p.N) break;
            if (pg < live) {
                if (x[i] <= 0) p.copy_to[hole++] = pg;
            } else if (x[i] > 0) {
                p.copy_from[mover] = pg;
                p.free_list[pg] = mover++;   // where a table's entry finds its new place
            } else {
                p.free_list[pg] = -1;
            }
        }
        found += total;
    }
    __syncthreads();
    const int moves = (int)(found >> 32);
    for (int i = tid; i < moves; i += kCtl) {
        const int a = __ldcg(p.copy_from + i), b = __ldcg(p.copy_to + i);
        p.refs[b] = now(p.refs + a);
        p.refs[a] = 0;
    }
    if (tid == 0) {
        *p.live = (int)live;
        *p.n_copies = moves;
    }
}

// The copies of pages, of every layer, in pieces of 16 KB; with `remap` the tables' entries first.
constexpr int kPiece = 16384;
__global__ void __launch_bounds__(256) copy_pages_kernel(const __grid_constant__ UpkeepParams p, const bool remap) {
    const int n = *p.n_copies;
    const int tid = threadIdx.x;
    if (remap) {
        const int live = *p.live;
        for (int r = blockIdx.x; r < p.R; r += gridDim.x) {
            const int used = min((int)(((int64_t)max(p.lens[r], 0) + p.page - 1) >> p.page_log2), p.W);
            for (int w = tid; w < used; w += 256) {
                const int pg = p.table[(int64_t)r * p.W + w];
                if (pg >= 0 && pg < live) continue;
                const int move = pg >= 0 && pg < p.N ? p.free_list[pg] : -1;
                if (move >= 0) p.table[(int64_t)r * p.W + w] = p.copy_to[move];
                else atomicOr(p.status, STATUS_BAD_INDEX);   // outside the pool, or held by nobody
            }
        }
    }
    const int pieces = (int)((p.page_bytes + kPiece - 1) / kPiece);
    const int64_t units = (int64_t)n * p.L * pieces;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t x = u / pieces;
        const int piece = (int)(u - x * pieces), layer = (int)(x % p.L), i = (int)(x / p.L);
        const int64_t from = p.copy_from[i], to = p.copy_to[i];
        const int64_t off = (int64_t)piece * kPiece;
        const unsigned char* src = p.pages + layer * p.layer_bytes + from * p.page_bytes + off;
        unsigned char* dst = p.pages + layer * p.layer_bytes + to * p.page_bytes + off;
        const int bytes = (int)min((int64_t)kPiece, p.page_bytes - off);
        uint4 y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int at = (j * 256 + tid) * 16;
            if (at < bytes) y[j] = __ldcs(reinterpret_cast<const uint4*>(src + at));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int at = (j * 256 + tid) * 16;
            if (at < bytes) __stcs(reinterpret_cast<uint4*>(dst + at), y[j]);
        }
        if (piece == 0)
            for (int j = tid; j < p.page_scales; j += 256)
                p.scales[layer * p.layer_scales + to * p.page_scales + j] = p.scales[layer * p.layer_scales + from * p.page_scales + j];
    }
}

cudaError_t launch_copies(const UpkeepParams& p, bool remap, int64_t most, cudaStream_t s) {
    const int64_t pieces = (p.page_bytes + kPiece - 1) / kPiece;
    const int64_t grid = std::min<int64_t>((int64_t)kSms * 8, std::max<int64_t>(most * p.L * pieces, remap ? p.R : 1));
    copy_pages_kernel<<<(unsigned)grid, 256, 0, s>>>(p, remap);
    return cudaGetLastError();
}

}  // namespace

int rope_passes(int heads, int D, bool bf16) {
    const int at_once = 32 / (D / (bf16 ? 16 : 8));
    return (heads + at_once - 1) / at_once;
}

cudaError_t launch_rope(const RopeParams& p, int D, bool bf16, bool half, cudaStream_t s) {
    if (p.T == 0) return cudaSuccess;
    switch (D * 2 + bf16) {
        case 64: return rope<float, 32>(p, half, s);
        case 65: return rope<__nv_bfloat16, 32>(p, half, s);
        case 128: return rope<float, 64>(p, half, s);
        case 129: return rope<__nv_bfloat16, 64>(p, half, s);
        case 256: return rope<float, 128>(p, half, s);
        default: return rope<__nv_bfloat16, 128>(p, half, s);
    }
}

cudaError_t launch_append(const AppendParams& p, int D, bool bf16, cudaStream_t s) {
    switch (D * 2 + bf16) {
        case 64: return append_d<float, 32>(p, s);
        case 65: return append_d<__nv_bfloat16, 32>(p, s);
        case 128: return append_d<float, 64>(p, s);
        case 129: return append_d<__nv_bfloat16, 64>(p, s);
        case 256: return append_d<float, 128>(p, s);
        default: return append_d<__nv_bfloat16, 128>(p, s);
    }
}

cudaError_t launch_update(const UpkeepParams& p, cudaStream_t s) {
    static std::atomic<int> optin[kMaxOptinDevices];
    const int smem = p.R * 8;
    if (smem > 40000) {
        const cudaError_t e = smem_optin(reinterpret_cast<const void*>(update_kernel), kMaxRows * 8, optin);
        if (e != cudaSuccess) return e;
    }
    update_kernel<<<1, kCtl, smem, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !p.grow) return e;
    return launch_copies(p, false, std::min(p.R, p.N), s);
}

cudaError_t launch_compact(const UpkeepParams& p, cudaStream_t s) {
    compact_kernel<<<1, kCtl, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_copies(p, true, p.N / 2 + 1, s);
}

}  // namespace cache
}  // namespace gdn
