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
// An angle is position * frequency.  The frequency is held as a 64-bit fraction of a turn, formed from inv_freq in two parts of
// 53 bits (fp64, once a CTA), so the product's low 64 bits are the angle without whole turns, to 2^-33 of a turn at any position
// (one product of fp64 left 2^-25 at the farthest); the nearest quarter turn is then taken off as an integer, and what
// is left (an eighth of a turn at most) goes to fp32.
//
// Bound by memory: each element is read and written once.  The next heads' loads are issued before the ones at hand are
// computed, and the arithmetic is on pairs of fp32 (without both 272 us): 65536 tokens x 40 heads of 128 in bf16 take 224 us, 6.0 TB/s, 88 %
// of a copy's rate; 67 tokens x 32 heads of 64 in fp32 4.5 us, a launch.
template <typename T, int D, bool HALF>
__global__ void __launch_bounds__(128) rope_kernel(const __grid_constant__ RopeParams p) {
    using V = Vec<T>;
    constexpr int N = V::N, L = D / (2 * N), HP = 32 / L, U = 2;
    __shared__ uint64_t s_freq[D / 2];
    const int lane = threadIdx.x & 31, j = lane % L, hsub = lane / L;
    const int q_passes = (p.Hq + HP - 1) / HP, passes = q_passes + (p.Hk + HP - 1) / HP;
    const bool turned = 2 * N * j < p.rd;
    const int ea = (HALF && turned ? j : 2 * j) * N, eb = HALF && turned ? ea + p.rd / 2 : ea + N;   // the lane's two pieces
    for (int i = threadIdx.x; i < p.rd / 2; i += 128) {
        // in 2^-64 of a turn: the product with 1 / 2 pi, and what it leaves, for 1 / 2 pi in two parts; whole turns are taken off exactly
        constexpr double kTurn = 18446744073709551616.0;
        const double f = p.inv_freq[i], x = f * (0.15915494309189535 * kTurn);
        const double rest = fma(f, -9.839338337591243e-18 * kTurn, fma(f, 0.15915494309189535 * kTurn, -x));
        s_freq[i] = (uint64_t)__double2ll_rn(fma(rint(x * (1.0 / kTurn)), -kTurn, x)) + (uint64_t)__double2ll_rn(rest);
    }
    __syncthreads();
    const int64_t units = p.T * p.parts, warps = (int64_t)gridDim.x * 4;
    for (int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5); u < units; u += warps) {
        const int64_t t = u / p.parts;
        const int first = (int)(u - t * p.parts) * p.per_part, last = min(first + p.per_part, passes);
        // the queries' passes, then the keys'
        auto place = [&](int g, bool out) -> T* {   // of this lane's head of pass g; nullptr: none
            const bool k = g >= q_passes;
            const int head = (k ? g - q_passes : g) * HP + hsub;
            if (g >= last || head >= (k ? p.Hk : p.Hq)) return nullptr;
            const void* base = k ? (out ? p.k_out : p.k) : (out ? p.q_out : p.q);
            const int64_t stride = k ? (out ? p.ko_stride : p.k_stride) : (out ? p.qo_stride : p.q_stride);
            return static_cast<T*>(const_cast<void*>(base)) + t * stride + head * D;
        };
        uint4 next[U][2];
        auto fetch = [&](int g) {
#pragma unroll
            for (int x = 0; x < U; ++x) {
                const T* src = place(g + x, false);
                next[x][0] = next[x][1] = make_uint4(0, 0, 0, 0);
                if (src) {
                    next[x][0] = *reinterpret_cast<const uint4*>(src + ea);
                    next[x][1] = *reinterpret_cast<const uint4*>(src + eb);
                }
            }
        };
        fetch(first);
        float2 cs[N / 2], sn[N / 2];
        const int64_t pos = turned ? p.positions[t] : 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint64_t a = (uint64_t)pos * (turned ? s_freq[j * N + i] : 0);
            const uint32_t quarter = (uint32_t)((a + (1ull << 61)) >> 62);
            const int64_t rest = (int64_t)(a - ((uint64_t)quarter << 62));
            float s, c;
            sincospif(__ll2float_rn(rest) * 1.0842021724855044e-19f, &s, &c);   // 2^-63: half turns
            const float cc = quarter & 1 ? s : c, ss = quarter & 1 ? c : s;
            const float cv = ((quarter + 1) & 2 ? -cc : cc) * p.mscale, sv = (quarter & 2 ? -ss : ss) * p.mscale;
            if (i & 1) cs[i / 2].y = cv, sn[i / 2].y = sv;
            else cs[i / 2].x = cv, sn[i / 2].x = sv;
        }
        float2 wa[N / 2], wb[N / 2];
        auto weights = [&](const void* w) {
            float a[N], b[N];
#pragma unroll
            for (int i = 0; i < N; ++i) a[i] = b[i] = 1.f;
            if (w) {
                V::get(*reinterpret_cast<const uint4*>(static_cast<const T*>(w) + ea), a);
                V::get(*reinterpret_cast<const uint4*>(static_cast<const T*>(w) + eb), b);
            }
#pragma unroll
            for (int i = 0; i < N / 2; ++i) wa[i] = make_float2(a[2 * i], a[2 * i + 1]), wb[i] = make_float2(b[2 * i], b[2 * i + 1]);
        };
        if (p.normalize) weights(first < q_passes ? p.qw : p.kw);
        for (int g = first; g < last; g += U) {
            uint4 in[U][2];
#pragma unroll
            for (int x = 0; x < U; ++x) in[x][0] = next[x][0], in[x][1] = next[x][1];
            fetch(g + U);
#pragma unroll
            for (int x = 0; x < U; ++x) {
                if (p.normalize && g + x == q_passes) weights(p.kw);   // (the same for the whole warp)
                float fa[N], fb[N];
                V::get(in[x][0], fa);
                V::get(in[x][1], fb);
                float2 a[N / 2], b[N / 2];
#pragma unroll
                for (int i = 0; i < N / 2; ++i) a[i] = make_float2(fa[2 * i], fa[2 * i + 1]), b[i] = make_float2(fb[2 * i], fb[2 * i + 1]);
                if (p.normalize) {
                    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < N / 2; ++i) s2 = __ffma2_rn(a[i], a[i], s2), s2 = __ffma2_rn(b[i], b[i], s2);
                    float sum = s2.x + s2.y;
#pragma unroll
                    for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    const float r = rsqrtf(sum * (1.f / D) + p.eps);
                    const float2 r2 = make_float2(r, r);
#pragma unroll
                    for (int i = 0; i < N / 2; ++i)
                        a[i] = __fmul2_rn(a[i], __fmul2_rn(r2, wa[i])), b[i] = __fmul2_rn(b[i], __fmul2_rn(r2, wb[i]));
                }
                if (turned) {
                    if (HALF) {
#pragma unroll
                        for (int i = 0; i < N / 2; ++i) {
                            const float2 y = a[i], ns = make_float2(-sn[i].x, -sn[i].y);
                            a[i] = __ffma2_rn(y, cs[i], __fmul2_rn(b[i], ns));
                            b[i] = __ffma2_rn(b[i], cs[i], __fmul2_rn(y, sn[i]));
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < N / 2; ++i) {   // pair 2 i, 2 i + 1 of one piece; N / 2 of them in each
                            const float ca = i & 1 ? cs[i / 2].y : cs[i / 2].x, sa = i & 1 ? sn[i / 2].y : sn[i / 2].x;
                            const float cb = i & 1 ? cs[N / 4 + i / 2].y : cs[N / 4 + i / 2].x;
                            const float sb = i & 1 ? sn[N / 4 + i / 2].y : sn[N / 4 + i / 2].x;
                            a[i] = make_float2(a[i].x * ca - a[i].y * sa, a[i].y * ca + a[i].x * sa);
                            b[i] = make_float2(b[i].x * cb - b[i].y * sb, b[i].y * cb + b[i].x * sb);
                        }
                    }
                }
                if (T* dst = place(g + x, true)) {
#pragma unroll
                    for (int i = 0; i < N / 2; ++i) fa[2 * i] = a[i].x, fa[2 * i + 1] = a[i].y, fb[2 * i] = b[i].x, fb[2 * i + 1] = b[i].y;
                    *reinterpret_cast<uint4*>(dst + ea) = V::put(fa);
                    *reinterpret_cast<uint4*>(dst + eb) = V::put(fb);
                }
            }
        }
    }
}

template <typename T, int D>
cudaError_t rope(const RopeParams& p, bool half, cudaStream_t s) {
    const int64_t units = p.T * p.parts, need = (units + 3) / 4;
    const unsigned grid = (unsigned)std::min<int64_t>(need, (int64_t)kSms * 12);   // more units than warps take turns
    if (half) rope_kernel<T, D, true><<<grid, 128, 0, s>>>(p);
    else rope_kernel<T, D, false><<<grid, 128, 0, s>>>(p);
    return cudaGetLastError();
}

// ---- append -----------------------------------------------------------------------------------------------------------
//
// A block (page x head, keys or values) is taken by TPB threads: they read its new tokens once into registers, agree on the
// largest value, and write the bytes.  Tokens that the block holds already are touched only when the scale grows.
// TPB is 32 for calls with at most 8 new tokens a request (decode, drafts: a block has little to do, and eight of them
// share a CTA), 256 else.  A CTA takes `share` blocks of one page in turn: what it has to find out first, four loads that wait
// for one another, took half of its time where every block had a CTA of its own.  (Loading the next block's tokens ahead cost 10 %:
// fewer CTAs fit.)  32 turns of up to 1999 tokens x 8 heads of 128 take 46 us, 82 % of a copy's rate; one token of 64 requests 3.5 us, four
// loads that wait for one another.
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
__device__ __forceinline__ int scale_exponent(uint32_t top) {   // (as bits)
    return min(max((int)((top + 0x1fffffu) >> 23) - 127 - 8, -126), 120);
}

template <typename T, int D, int TPB, int NCH>
__global__ void __launch_bounds__(256) append_kernel(const __grid_constant__ AppendParams p, const int share) {
    constexpr int PER = 256 / TPB;            // blocks of a CTA
    constexpr int VEC = 16 / sizeof(T), LD = 8 / VEC;   // a chunk is 8 values: LD loads
    constexpr int CPT = D / 8;                // chunks of a token
    __shared__ uint32_t s_top[8];
    const Cache& c = p.c;
    const int tid = threadIdx.x % TPB, sub = threadIdx.x / TPB;
    const int blocks = 2 * c.Hkv, groups = (blocks + share - 1) / share;
    const int b = blockIdx.y;
    const int i0 = blockIdx.x / groups, block0 = (blockIdx.x - i0 * groups) * share;
    const Request rq = request_at(c, p.t, b);
    if (rq.bad && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.status, STATUS_BAD_INDEX);
    if (rq.row < 0 || rq.n == 0 || rq.bad) return;
    const int start = max(rq.len - rq.n, 0), skip = max(rq.n - rq.len, 0);   // (new tokens before a row's first position)
    const int i = (start >> c.page_log2) + i0;
    if (i > (rq.len - 1) >> c.page_log2) return;   // (in pages: behind the longest rows the tokens' numbers leave 32 bits)
    const int base = i << c.page_log2;
    const int pg = c.table[(int64_t)rq.row * c.W + i];
    if (pg < 0 || pg >= c.N) {
        if (threadIdx.x == 0) atomicOr(p.status, STATUS_BAD_INDEX);
        return;
    }
    const int lo = max(start - base, 0), n = min(rq.len - base, c.page) - lo;   // the block's new tokens: lo .. lo + n
    const int end = min(block0 + share, blocks);
    const int64_t first = rq.first + skip + (int64_t)(base + lo - start);   // the block's first new token in the streams
    uint4 in[NCH][LD];
    auto fetch = [&](int block) {
        const bool kv = block >= c.Hkv;
        const int64_t stride = kv ? p.v_stride : p.k_stride;
        const T* src = static_cast<const T*>(kv ? p.v : p.k) + first * stride + (int64_t)(kv ? block - c.Hkv : block) * D;
        const int chunks = block < end ? n * CPT : 0;
#pragma unroll
        for (int x = 0; x < NCH; ++x) {
            const int ch = x * TPB + tid;
            if (ch < chunks) {
                const T* a = src + (int64_t)(ch / CPT) * stride + (ch % CPT) * 8;
#pragma unroll
                for (int y = 0; y < LD; ++y) in[x][y] = *reinterpret_cast<const uint4*>(a + y * VEC);
            }
        }
    };
    for (int at0 = block0; at0 < end; at0 += PER) {
        const int block = at0 + sub;
        const bool work = block < end;
        const int kv = block >= c.Hkv, h = block - kv * c.Hkv;
        const int64_t at = ((int64_t)pg * 2 + kv) * c.Hkv + h;
        const int chunks = work ? n * CPT : 0;
        float was = 0.f;
        if (work && lo > 0) was = c.scales[at];   // (before anyone writes it)
        fetch(block);
        // The largest value (two of bf16 at a time; a maximum passes over NaN, which the conversion holds as it is).  Where that is an
        // infinity, which is rare, the others are looked through again.
        auto agree = [&](uint32_t y) {
            y = __reduce_max_sync(0xffffffffu, y);
            if (TPB > 32) {
                __syncthreads();
                if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = y;
                __syncthreads();
#pragma unroll
                for (int x = 0; x < 8; ++x) y = max(y, s_top[x]);
            } else {
                __syncwarp();   // every lane has `was`
            }
            return y;
        };
        uint32_t bits = 0;
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int x = 0; x < NCH; ++x)
                if (x * TPB + tid < chunks)
#pragma unroll
                    for (int y = 0; y < LD; ++y)
#pragma unroll
                        for (uint32_t w : {in[x][y].x, in[x][y].y, in[x][y].z, in[x][y].w})
                            asm("max.bf16x2 %0, %1, %2;" : "=r"(bits) : "r"(bits), "r"(w & 0x7fff7fffu));
            bits = max(bits & 0xffffu, bits >> 16) << 16;
        } else {
            float top = 0.f;
#pragma unroll
            for (int x = 0; x < NCH; ++x)
                if (x * TPB + tid < chunks)
#pragma unroll
                    for (int y = 0; y < LD; ++y)
#pragma unroll
                        for (uint32_t w : {in[x][y].x, in[x][y].y, in[x][y].z, in[x][y].w}) top = fmaxf(top, fabsf(__uint_as_float(w)));
            bits = __float_as_uint(top);
        }
        bits = agree(bits);
        const bool odd = bits == 0x7f800000u;
        if (odd) {
            bits = 0;
#pragma unroll
            for (int x = 0; x < NCH; ++x) {
                if (x * TPB + tid < chunks) {
#pragma unroll
                    for (int y = 0; y < LD; ++y) {
                        float f[VEC];
                        Vec<T>::get(in[x][y], f);
#pragma unroll
                        for (int z = 0; z < VEC; ++z)
                            if (fabsf(f[z]) <= FLT_MAX) bits = max(bits, __float_as_uint(fabsf(f[z])));
                    }
                }
            }
            bits = agree(bits);
        }
        if (!work) continue;
        float scale = __uint_as_float((uint32_t)(scale_exponent(bits) + 127) << 23);
        const bool grows = lo > 0 && scale > was;
        if (lo > 0 && !grows) scale = was;
        const float inv = 1.f / scale;
        unsigned char* dst = c.pages + at * c.page * D;
        auto convert = [&](bool check) {   // (checked values apart, so that the others take one product and half a conversion each)
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
                        for (int z = 0; z < VEC; ++z)
                            f[y * VEC + z] = !check || fabsf(g[z]) <= FLT_MAX ? g[z] * inv : __uint_as_float(0x7fc00000u);
                    }
                    *reinterpret_cast<uint2*>(dst + (int64_t)lo * D + ch * 8) =
                        make_uint2(to_e4m3x4(f[0], f[1], f[2], f[3]), to_e4m3x4(f[4], f[5], f[6], f[7]));
                }
            }
        };
        if (odd) convert(true);
        else convert(false);
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
}

template <typename T, int D, int TPB, int NCH>
cudaError_t append_n(const AppendParams& p, cudaStream_t s) {
    const int touched = (p.t.max_new + p.c.page - 2) / p.c.page + 1;   // pages that a request's new tokens may lie in
    // about three CTAs for each that runs at once, blocks of one page in a CTA
    constexpr int PER = 256 / TPB;
    const int64_t blocks = 2 * p.c.Hkv, all = (int64_t)touched * p.t.B * blocks;
    const int share = (int)std::min<int64_t>(blocks, std::max<int64_t>(PER, all / (kSms * 4 * 3)));
    append_kernel<T, D, TPB, NCH><<<dim3((unsigned)(touched * ((blocks + share - 1) / share)), p.t.B), 256, 0, s>>>(p, share);
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
// The tables are small and their changes depend on one another, so one cluster makes them, its CTAs (one for small tables) sharing
// the rows; the copies of pages that it asks for follow in a launch of their own over the whole GPU.  Pages are found in rising order by scanning the holders'
// counts, 16384 a round (64 KB), as far as there is need: no list of free pages has to be kept in step with them.  128 forks of 8191 tokens
// (pages of 64) with growth take 19 us here (35 with one CTA), their 128 copied pages in 8 layers 22 more; four forks of 64 pages 10 in all,
// the phases' loads one after another.
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

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Every CTA of the cluster works out the same lists in its shared memory; the rows' pages are taken in turns by all warps.
__global__ void __launch_bounds__(kCtl) update_kernel(const __grid_constant__ UpkeepParams p) {
    extern __shared__ int32_t s_rows[];   // [R] whether a row is freed, then its first new page's place; [R] the fork that it is, then needs
    int32_t* s_need = s_rows;
    int32_t* s_fork = s_rows + p.R;
    __shared__ int64_t s_part[32];
    constexpr int kNone = 0x7fffffff;
    const int tid = threadIdx.x, lane = tid & 31, first_row = blockIdx.x * (kCtl / 32) + (tid >> 5), step = gridDim.x * (kCtl / 32);
    auto pages_of = [&](int len) { return min((int)(((int64_t)max(len, 0) + p.page - 1) >> p.page_log2), p.W); };
    auto good = [&](int pg) {
        const bool ok = pg >= 0 && pg < p.N;
        if (!ok) atomicOr(p.status, STATUS_BAD_INDEX);
        return ok;
    };
    if (blockIdx.x == 0 && tid == 0) *p.n_copies = 0;
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
        for (int r = first_row; r < p.R; r += step) {
            if (!s_need[r]) continue;
            const int used = pages_of(p.lens[r]);
#pragma unroll 4
            for (int w = lane; w < used; w += 32) {
                const int pg = p.table[(int64_t)r * p.W + w];
                if (good(pg)) atomicSub(&p.refs[pg], 1);
            }
            __syncwarp();
            if (lane == 0) p.lens[r] = 0;
        }
        cluster_sync();
        for (int r = first_row; r < p.R; r += step) {
            if (s_fork[r] == kNone) continue;
            const int a = p.from[s_fork[r]];
            if (s_need[a]) continue;   // freed just now: an empty row
            const int len = now(p.lens + a), used = pages_of(len);
#pragma unroll 4
            for (int w = lane; w < p.W; w += 32) {
                const int pg = p.table[(int64_t)a * p.W + w];
                p.table[(int64_t)r * p.W + w] = pg;
                if (w < used && good(pg)) atomicAdd(&p.refs[pg], 1);
            }
            if (lane == 0) p.lens[r] = len;
        }
    }
    cluster_sync();
    if (!p.grow) return;

    // pages that each row needs, and their places among all that are taken.  s_need: the first place; s_fork: bit 31 refused,
    // bit 30 copy the last page, below: the number of pages
    constexpr unsigned kRefused = 1u << 31, kCopy = 1u << 30;
    int64_t carry = 0;
    for (int r0 = 0; r0 < p.R; r0 += kCtl) {
        const int r = r0 + tid;
        int need = 0;
        unsigned flags = 0;
        if (r < p.R) {
            const int len = max(now(p.lens + r), 0), more = max(p.grow[r], 0);
            if ((int64_t)len + more > (int64_t)p.W * p.page) {
                flags = kRefused;
            } else if (more > 0) {
                const int have = pages_of(len);
                need = pages_of(len + more) - have;
                if (len & (p.page - 1)) {
                    const int last = now(p.table + (int64_t)r * p.W + have - 1);
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
    if (blockIdx.x == 0) {
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
        if (tid == 0) p.n_copies[1] = (int)found;
    }
    cluster_sync();   // (what each row needs was read by all before any row changes)
    const int found = now(p.n_copies + 1);
    for (int r = first_row; r < p.R; r += step) {
        const unsigned f = (unsigned)s_fork[r];
        const int need = (int)(f & (kCopy - 1)), first = s_need[r];
        const bool copy = f & kCopy;
        const int more = max(p.grow[r], 0);
        if ((f & kRefused) || (need > 0 && (int64_t)first + need > found)) {
            if (lane == 0 && p.granted) p.granted[r] = -1;
            continue;
        }
        const int len = max(now(p.lens + r), 0), have = pages_of(len);
        int32_t* row = p.table + (int64_t)r * p.W;
        for (int w = lane; w < need; w += 32) {
            const int pg = now(p.free_list + first + w);
            p.refs[pg] = 1;
            if (copy && w == 0) {
                const int old = now(row + have - 1);
                const int at = atomicAdd(p.n_copies, 1);
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

// The copies of pages, of every layer, in pieces of 32 KB (16 KB: 3 % slower); with `remap` the tables' entries first.  Bound by memory: 1.6 GB
// read and written in 247 us, 94 % of a copy's rate.
constexpr int kPiece = 32768;
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
        uint4 y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int at = (j * 256 + tid) * 16;
            if (at < bytes) y[j] = __ldcs(reinterpret_cast<const uint4*>(src + at));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
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

int rope_passes(int Hq, int Hk, int D, bool bf16) {
    const int at_once = 32 / (D / (bf16 ? 16 : 8));
    return (Hq + at_once - 1) / at_once + (Hk + at_once - 1) / at_once;
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
    // eight CTAs where the rows' pages are many: one alone took 35 us to fork 128 rows of 128 pages, most of it waiting for loads
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (int64_t)p.R * p.W > 4096 ? 8 : 1;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(attr.val.clusterDim.x), cfg.blockDim = dim3(kCtl);
    cfg.dynamicSmemBytes = smem, cfg.stream = s;
    cfg.attrs = &attr, cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, update_kernel, p);
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
