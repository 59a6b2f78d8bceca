// gdn_paged.cu - attention over a paged 8-bit cache for few query rows a key/value head (decode, drafts) and for fp32
// queries, and the join of the parts.
//
// Bound by memory, so the keys and values go from global memory straight into the registers that warp-level products take
// them from: nothing is staged.  A product's contraction index and its columns may be numbered at will as long as both
// sides agree, which lets a lane's operand be whole 16-byte pieces: of the keys the pieces c and c + 4 of a token's row
// (lane 4 t + c of token t, 8 tokens a load), of the values the piece t of the tokens 2 c, 2 c + 1 (+ 8).  e4m3 becomes f16
// exactly, two values an instruction; values of two tokens are interleaved by byte permutes first.
//
// Per 16 tokens of a warp:  S = Q K^T (rows x 16),  x = S * scale of the keys' block,  p = 2^(x - m),  O += P V.
// Queries are brought to [2^14, 2^15) by a power of two for each row and held as one f16 (bf16 queries: exact) or the sum of two
// (fp32: 22 bits); the weights likewise, times 2^11 and, in bf16, the block's scale over the largest met (a power of two).
// m is raised only when a score is more than 2^4 above it, so the weights stay below 2^15.  Statistics and sums are fp32.
//
// The units of all items are dealt out evenly (gdn_cache.cuh), so lengths may differ at will; a CTA's four warps take
// 16-token steps in turn and add their sums up in shared memory at the end of an item.
//
// 64 requests x 8 heads of 128 (4 query heads each) on 17 to 34 k tokens take 528 us, 6.18 TB/s, 91 % of a copy's rate; 4 requests x 2 heads
// on 1 k tokens 12, the join 4 of them: a chain of loads (counts, rows, lengths, pages, keys) and two launches.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "gdn_cache.cuh"

namespace gdn {
namespace cache {
namespace {

constexpr int kWarps = 4;
constexpr float kRise = 4.f;       // log2: how far a score may be above m
constexpr float kLift = 2048.f;    // weights are held times this: 2^11 2^4 = 2^15 in f16

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// four e4m3 as two pairs of f16
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ void mma(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
// d += f times the products of both parts of a, for fp32: the tensor cores cut their sums, every time by up to a step of fp32, so the running
// sum is kept outside them (with it inside, the outputs were off by 4.7e-6 where fp32 sums of the plain form were by 1.8e-6)
__device__ __forceinline__ void mma_two(float (&d)[4], const uint4& a, const uint4& rest, uint32_t b0, uint32_t b1, float f) {
    float t[4] = {0.f, 0.f, 0.f, 0.f};
    mma(t, rest, b0, b1);
    mma(t, a, b0, b1);
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = fmaf(t[i], f, d[i]);
}
__device__ __forceinline__ uint32_t half2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// x minus its f16 rounding, in f16
__device__ __forceinline__ uint32_t half2_rest(float a, float b, uint32_t h) {
    const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return half2(a - r.x, b - r.y);
}
template <int BYTES>
__device__ __forceinline__ void load_bytes(uint32_t* to, const unsigned char* p) {   // read once: not kept in L1
    if constexpr (BYTES == 16)
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(to[0]), "=r"(to[1]), "=r"(to[2]), "=r"(to[3]) : "l"(p));
    else if constexpr (BYTES == 8)
        asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(to[0]), "=r"(to[1]) : "l"(p));
    else
        asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(to[0]) : "l"(p));
}
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

template <int D, typename T, int MT>
struct Cfg {
    static constexpr int PARTS = sizeof(T) == 2 ? 1 : 2;
    static constexpr int RT = 16 * MT;        // rows of a tile
    static constexpr int U = 128 / D;         // 16-token pieces of a step: the same bytes in flight at every width
    static constexpr int KW = D / 16;         // words of a key that a lane holds
    static constexpr int VW = D / 32;         // and of a value
    static constexpr int NT = D / 8;          // column tiles of the output
    static constexpr int kQ = 0;              // queries: [PARTS][MT][KW][32] uint4
    static constexpr int kO = kQ + PARTS * MT * KW * 512;            // sums: [warps][MT][NT][4][32] fp32
    static constexpr int kMl = kO + kWarps * MT * NT * 512;          // m, l: [warps][RT] float2
    static constexpr int kQe = kMl + kWarps * RT * 8;                // factors of the rows [RT]
    static constexpr int kCum = kQe + RT * 4;                        // units before each group of requests
    static constexpr int kSmem = kCum + (kMaxGroups + 1) * 4;
};

template <int D, typename T, int MT>
__global__ void __launch_bounds__(kWarps * 32, MT == 1 ? 3 : 2) paged_kernel(const __grid_constant__ PagedParams p) {
    using F = Cfg<D, T, MT>;
    constexpr int PARTS = F::PARTS, U = F::U, KW = F::KW, VW = F::VW, NT = F::NT, RT = F::RT;
    extern __shared__ __align__(16) unsigned char smem[];
    uint4* s_q = reinterpret_cast<uint4*>(smem + F::kQ);
    float* s_o = reinterpret_cast<float*>(smem + F::kO);
    float2* s_ml = reinterpret_cast<float2*>(smem + F::kMl);
    float* s_f = reinterpret_cast<float*>(smem + F::kQe);
    int* s_cum = reinterpret_cast<int*>(smem + F::kCum);
    const Cache& c = p.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q4 = lane & 3;

    join_may_start();
    count_units<kWarps * 32, RT, kUnit>(p, s_cum);
    const int total = s_cum[groups_of(p.t.B)], share = (total + gridDim.x - 1) / gridDim.x;
    int x = (int)min((int64_t)blockIdx.x * share, (int64_t)total);
    const int begin = x, end = (int)min((int64_t)x + share, (int64_t)total);

    Segment sg = segment_none();
    if (tid == 0) p.cuts[blockIdx.x] = Cut{};
    for (bool first = true; next_segment<RT, kUnit>(p, s_cum, x, end, sg); first = false) {
        if (first && tid == 0) describe_cut(p, sg, begin, share);
        const Request& rq = sg.rq;
        const int h = sg.h, row0 = sg.row0, rows = sg.rows, lo = sg.lo, hi = sg.hi;
        const int shift = rq.len - rq.n;              // query i sees the tokens below shift + i + 1
        const int all_see = shift + row0 / p.G + 1;   // tokens that every row sees end here
        const int32_t* table = c.table + (int64_t)max(rq.row, 0) * c.W;

        // ---- loads of a step: pages one step ahead of the data ----
        struct Data {
            uint32_t k[U][2][KW], v[U][4][VW];
            float ks[U], vs[U];
        };
        const unsigned char* pages = c.pages + (int64_t)h * c.page * D;
        const int64_t kv_bytes = (int64_t)c.Hkv * c.page * D;
        auto ids = [&](int t0, int (&id)[U]) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int t = t0 + 16 * u;
                id[u] = t < hi ? __ldg(table + (t >> c.page_log2)) : 0;
            }
        };
        auto fetch = [&](int t0, int (&id)[U], Data& d) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int t = t0 + 16 * u;
                if (t < hi) {
                    if ((unsigned)id[u] >= (unsigned)c.N) {
                        if (lane == 0) atomicOr(p.status, STATUS_BAD_INDEX);
                        id[u] = 0;
                    }
                    const unsigned char* a = pages + (int64_t)id[u] * 2 * kv_bytes + (int64_t)(t & (c.page - 1)) * D;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const unsigned char* row = a + (8 * j + g) * D;
                        if constexpr (D == 128) {
                            load_bytes<16>(&d.k[u][j][0], row + 16 * q4);
                            load_bytes<16>(&d.k[u][j][4], row + 64 + 16 * q4);
                        } else {
                            load_bytes<D / 4>(&d.k[u][j][0], row + D / 4 * q4);
                        }
                    }
                    a += kv_bytes;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        load_bytes<D / 8>(&d.v[u][j][0], a + (8 * (j >> 1) + 2 * q4 + (j & 1)) * D + D / 8 * g);
                    const float* sc = c.scales + (int64_t)id[u] * 2 * c.Hkv + h;
                    d.ks[u] = __ldg(sc), d.vs[u] = __ldg(sc + c.Hkv);
                } else {
                    d.ks[u] = d.vs[u] = 0.f;
                }
            }
        };
        constexpr int STEP = 16 * U;
        int id[U];
        Data d;
        int t0 = lo + warp * STEP;
        ids(t0, id);

        // ---- queries: a power of two for each row, then the products' operands ----
        const T* q = static_cast<const T*>(p.q);
        for (int r = warp; r < RT; r += kWarps) {
            float most = 0.f;
            if (r < rows) {
                const int R = row0 + r;
                const T* a = q + (int64_t)(rq.first + R / p.G) * p.q_stride + (int64_t)(h * p.G + R % p.G) * D;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) most = fmaxf(most, fabsf(to_f(a[lane + 32 * i])));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
            const int e = max((int)(__float_as_uint(most) >> 23) - 127, -100);
            if (lane == 0) s_f[r] = __uint_as_float((uint32_t)(14 - min(e, 127) + 127) << 23);
        }
        fetch(t0, id, d);
        ids(t0 + kWarps * STEP, id);
        __syncthreads();
        for (int i = tid; i < MT * KW * 32; i += kWarps * 32) {
            const int l = i & 31, w = (i >> 5) % KW, mt = i / (32 * KW);
            const int col = (D == 128 ? 64 * (w >> 2) + 16 * (l & 3) + 4 * (w & 3) : D / 4 * (l & 3) + 4 * w);
            float y[2][4];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int r = mt * 16 + half * 8 + (l >> 2), R = row0 + r;
                const float f = s_f[r];
                const T* a = q + (int64_t)(rq.first + R / p.G) * p.q_stride + (int64_t)(h * p.G + R % p.G) * D + col;
#pragma unroll
                for (int k = 0; k < 4; ++k) y[half][k] = r < rows ? to_f(a[k]) * f : 0.f;
            }
            uint4 hi4 = make_uint4(half2(y[0][0], y[0][1]), half2(y[1][0], y[1][1]), half2(y[0][2], y[0][3]), half2(y[1][2], y[1][3]));
            s_q[i] = hi4;
            if constexpr (PARTS == 2)
                s_q[MT * KW * 32 + i] = make_uint4(half2_rest(y[0][0], y[0][1], hi4.x), half2_rest(y[1][0], y[1][1], hi4.y),
                                                   half2_rest(y[0][2], y[0][3], hi4.z), half2_rest(y[1][2], y[1][3], hi4.w));
        }
        float fr[MT][2];
        int sees[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int r = mt * 16 + half * 8 + g;
                fr[mt][half] = p.scale_log2 / s_f[r];
                sees[mt][half] = r < rows ? min(rq.len, shift + (row0 + r) / p.G + 1) : 0;
            }
        __syncthreads();

        // ---- the tokens ----
        float m[MT][2], l[MT][2], o[MT][NT][4], vref = 0.f, vinv = 0.f;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            m[mt][0] = m[mt][1] = -INFINITY, l[mt][0] = l[mt][1] = 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[mt][n][i] = 0.f;
        }
        for (; t0 < hi; t0 += kWarps * STEP) {
            Data e = d;
            fetch(t0 + kWarps * STEP, id, d);
            ids(t0 + 2 * kWarps * STEP, id);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int t = t0 + 16 * u;
                if (t >= hi) break;
                float s[MT][2][4];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[mt][j][i] = 0.f;
#pragma unroll
                for (int w = 0; w < KW; ++w) {
                    uint32_t b0, b1, b2, b3;
                    widen4(e.k[u][0][w], b0, b1);
                    widen4(e.k[u][1][w], b2, b3);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        uint4 a[PARTS];
#pragma unroll
                        for (int part = 0; part < PARTS; ++part) a[part] = s_q[(part * MT + mt) * KW * 32 + w * 32 + lane];
                        if constexpr (PARTS == 1) {
                            mma(s[mt][0], a[0], b0, b1);
                            mma(s[mt][1], a[0], b2, b3);
                        } else {
                            mma_two(s[mt][0], a[0], a[1], b0, b1, 1.f);
                            mma_two(s[mt][1], a[0], a[1], b2, b3, 1.f);
                        }
                    }
                }
                bool rise = false;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const float f = fr[mt][half] * e.ks[u];
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int i = 0; i < 2; ++i) s[mt][j][2 * half + i] = __fmul_rn(s[mt][j][2 * half + i], f);   // (as m is)
                    }
                if (t + 16 > all_see) {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (t + 8 * j + 2 * q4 + (i & 1) >= sees[mt][i >> 1]) s[mt][j][i] = -INFINITY;
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const float t4 = fmaxf(fmaxf(s[mt][0][2 * half], s[mt][0][2 * half + 1]),
                                               fmaxf(s[mt][1][2 * half], s[mt][1][2 * half + 1]));
                        rise |= t4 - m[mt][half] > kRise;   // (m = -infinity: any score; m + kRise may round up)
                    }
                if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            float t4 = fmaxf(fmaxf(s[mt][0][2 * half], s[mt][0][2 * half + 1]),
                                             fmaxf(s[mt][1][2 * half], s[mt][1][2 * half + 1]));
                            t4 = fmaxf(t4, __shfl_xor_sync(0xffffffffu, t4, 1));
                            t4 = fmaxf(t4, __shfl_xor_sync(0xffffffffu, t4, 2));
                            const float mn = fmaxf(m[mt][half], t4);
                            const float f = mn == -INFINITY ? 1.f : ex2(m[mt][half] - mn);
                            m[mt][half] = mn;
                            l[mt][half] *= f;
#pragma unroll
                            for (int n = 0; n < NT; ++n) o[mt][n][2 * half] *= f, o[mt][n][2 * half + 1] *= f;
                        }
                }
                if (e.vs[u] > vref) {   // (the same for the whole warp)
                    const float f = vref / e.vs[u];
                    vref = e.vs[u];
                    if constexpr (PARTS == 2) vinv = 1.f / vref;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int i = 0; i < 4; ++i) o[mt][n][i] *= f;
                }
                // The block's scale over the largest met: in bf16 the weights carry it, in fp32 the products' sums, so that every block's
                // weights keep their 22 bits (with it, those of a block 2^-20 of the largest kept 15).
                float lift = kLift, ratio = 1.f;
                if constexpr (PARTS == 1) lift = vref > 0.f ? e.vs[u] / vref * kLift : 0.f;
                else ratio = e.vs[u] * vinv;
                uint4 a[PARTS][MT];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    uint32_t w[4], w2[4];
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const float base = m[mt][half] == -INFINITY ? 0.f : m[mt][half];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float p0 = ex2(s[mt][j][2 * half] - base), p1 = ex2(s[mt][j][2 * half + 1] - base);
                            l[mt][half] += p0 + p1;
                            w[2 * j + half] = half2(p0 * lift, p1 * lift);
                            if constexpr (PARTS == 2) w2[2 * j + half] = half2_rest(p0 * lift, p1 * lift, w[2 * j + half]);
                        }
                    }
                    a[0][mt] = make_uint4(w[0], w[1], w[2], w[3]);
                    if constexpr (PARTS == 2) a[1][mt] = make_uint4(w2[0], w2[1], w2[2], w2[3]);
                }
                if (t + 16 > hi) {   // what lies behind the row's tokens
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (t + 8 * (j >> 1) + 2 * q4 + (j & 1) >= hi)
#pragma unroll
                            for (int w = 0; w < VW; ++w) e.v[u][j][w] = 0;
                }
#pragma unroll
                for (int w = 0; w < VW; ++w) {
                    const uint32_t l01 = __byte_perm(e.v[u][0][w], e.v[u][1][w], 0x5140), h01 = __byte_perm(e.v[u][0][w], e.v[u][1][w], 0x7362);
                    const uint32_t l23 = __byte_perm(e.v[u][2][w], e.v[u][3][w], 0x5140), h23 = __byte_perm(e.v[u][2][w], e.v[u][3][w], 0x7362);
                    uint32_t b0[4], b1[4];
                    widen4(l01, b0[0], b0[1]), widen4(h01, b0[2], b0[3]);
                    widen4(l23, b1[0], b1[1]), widen4(h23, b1[2], b1[3]);
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
                            if constexpr (PARTS == 1) mma(o[mt][4 * w + n], a[0][mt], b0[n], b1[n]);
                            else mma_two(o[mt][4 * w + n], a[0][mt], a[1][mt], b0[n], b1[n], ratio);
                }
            }
        }

        // ---- the warps' sums ----
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float y = l[mt][half];
                y += __shfl_xor_sync(0xffffffffu, y, 1);
                y += __shfl_xor_sync(0xffffffffu, y, 2);
                if (q4 == 0) s_ml[warp * RT + mt * 16 + half * 8 + g] = make_float2(m[mt][half], y);
            }
        __syncthreads();
        float M[MT][2], Ls[MT][2];
        vref *= 1.f / kLift;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int r = mt * 16 + half * 8 + g;
                float2 y[kWarps];
                float mm = -INFINITY, ll = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) y[w] = s_ml[w * RT + r], mm = fmaxf(mm, y[w].x);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) ll += mm == -INFINITY ? 0.f : y[w].y * ex2(y[w].x - mm);
                M[mt][half] = mm, Ls[mt][half] = ll;
                const float f = mm == -INFINITY ? 0.f : ex2(m[mt][half] - mm) * vref;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        s_o[(((warp * MT + mt) * NT + n) * 4 + 2 * half + i) * 32 + lane] = o[mt][n][2 * half + i] * f;
            }
        __syncthreads();
        // each warp has a quarter of the column tiles: NT / 4 neighbouring columns of the output
        const bool whole = sg.whole();
        const int64_t slot = sg.slot();
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int r = mt * 16 + half * 8 + g;
                if (r >= rows) continue;
                const int R = row0 + r;
                const int64_t at = (int64_t)(rq.first + R / p.G) * p.Hq + h * p.G + R % p.G;
                const float inv = Ls[mt][half] > 0.f ? 1.f / Ls[mt][half] : Ls[mt][half] == 0.f ? 0.f : NAN;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float y[NT / 4];
#pragma unroll
                    for (int n = 0; n < NT / 4; ++n) {
                        y[n] = 0.f;
#pragma unroll
                        for (int w = 0; w < kWarps; ++w)
                            y[n] += s_o[(((w * MT + mt) * NT + warp * (NT / 4) + n) * 4 + 2 * half + i) * 32 + lane];
                    }
                    const int col = D / 8 * (2 * q4 + i) + warp * (NT / 4);
                    if (whole) {
                        T* to = static_cast<T*>(p.o) + at * D + col;
                        if constexpr (sizeof(T) == 2 && NT / 4 >= 2) {
#pragma unroll
                            for (int n = 0; n < NT / 4; n += 2)
                                *reinterpret_cast<__nv_bfloat162*>(to + n) = __floats2bfloat162_rn(y[n] * inv, y[n + 1] * inv);
                        } else {
#pragma unroll
                            for (int n = 0; n < NT / 4; ++n) put(to + n, y[n] * inv);
                        }
                    } else {
                        float* to = p.part_o + (slot * RT + r) * D + col;
#pragma unroll
                        for (int n = 0; n < NT / 4; ++n) to[n] = y[n];
                    }
                }
                if (warp == 0 && q4 == 0) {
                    if (!whole) p.part_ml[slot * RT + r] = make_float2(M[mt][half], Ls[mt][half]);
                    else if (p.lse)
                        p.lse[at] = Ls[mt][half] == 0.f ? -INFINITY : (M[mt][half] + log2f(Ls[mt][half])) * 0.6931471805599453f;
                }
            }
        __syncthreads();
    }
}

// The joins are launched while the kernel that makes the parts still runs, and wait for it here; every CTA does, so that what
// follows in the stream waits for it too.
__device__ __forceinline__ void kernel_before_done() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A CTA adds up the parts of one row of a cut item, four warps sharing them.
template <int D, typename T, int RT>
__global__ void __launch_bounds__(128) paged_join_kernel(const __grid_constant__ PagedParams p) {
    constexpr int N = D / 32, W = 4;
    __shared__ float s_acc[W][D], s_l[W];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.x, c0 = blockIdx.y;
    kernel_before_done();
    const Cut cut = p.cuts[c0 + 1];
    if (r >= cut.rows) return;
    const int c1 = cut.last;
    auto slot = [&](int c) { return (int64_t)2 * c + (c == c0); };
    float m = -INFINITY;
    for (int c = c0 + lane; c <= c1; c += 32) m = fmaxf(m, p.part_ml[slot(c) * RT + r].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float acc[N] = {}, l = 0.f;
#pragma unroll 4
    for (int c = c0 + warp; c <= c1; c += W) {
        const float2 ml = p.part_ml[slot(c) * RT + r];
        const float* a = p.part_o + (slot(c) * RT + r) * D + lane * N;
        float y[N];
#pragma unroll
        for (int k = 0; k < N; ++k) y[k] = a[k];
        const float f = m == -INFINITY ? 0.f : ex2(ml.x - m);
        l += ml.y * f;
#pragma unroll
        for (int k = 0; k < N; ++k) acc[k] += f * y[k];
    }
#pragma unroll
    for (int k = 0; k < N; ++k) s_acc[warp][lane * N + k] = acc[k];
    if (lane == 0) s_l[warp] = l;
    __syncthreads();
    const int d = threadIdx.x, R = cut.row0 + r;
    l = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) l += s_l[w];
    const int64_t at = (int64_t)(cut.first + R / p.G) * p.Hq + cut.h * p.G + R % p.G;
    if (d < D) {
        float y = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) y += s_acc[w][d];
        put(static_cast<T*>(p.o) + at * D + d, y * (l > 0.f ? 1.f / l : l == 0.f ? 0.f : NAN));
    }
    if (d == 0 && p.lse) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// The same for tiles of many rows and few parts: a CTA takes 8 rows, a warp two of them (with 32, 16, 8 rows a CTA a prompt of 8192 took 478,
// 468, 466 us, 16 requests with one of 300 tokens 56, 46, 40).
constexpr int kJoinRows = 8;
template <int D, typename T, int RT>
__global__ void __launch_bounds__(128) paged_join_rows_kernel(const __grid_constant__ PagedParams p) {
    constexpr int N = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c0 = blockIdx.y;
    kernel_before_done();
    const Cut cut = p.cuts[c0 + 1];
    const int c1 = cut.last, end = min((int)(blockIdx.x + 1) * kJoinRows, cut.rows);
#pragma unroll 2
    for (int r = blockIdx.x * kJoinRows + warp; r < end; r += 4) {
        const int R = cut.row0 + r;
        float m = -INFINITY;
        for (int c = c0; c <= c1; ++c) m = fmaxf(m, p.part_ml[(2 * (int64_t)c + (c == c0)) * RT + r].x);
        float acc[N] = {}, l = 0.f;
#pragma unroll 2
        for (int c = c0; c <= c1; ++c) {
            const int64_t at = (2 * (int64_t)c + (c == c0)) * RT + r;
            const float2 ml = p.part_ml[at];
            const float f = m == -INFINITY ? 0.f : ex2(ml.x - m);
            l += ml.y * f;
#pragma unroll
            for (int k = 0; k < N; ++k) acc[k] += f * p.part_o[at * D + lane * N + k];
        }
        const int64_t at = (int64_t)(cut.first + R / p.G) * p.Hq + cut.h * p.G + R % p.G;
        const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : NAN;
#pragma unroll
        for (int k = 0; k < N; ++k) put(static_cast<T*>(p.o) + at * D + lane * N + k, acc[k] * inv);
        if (lane == 0 && p.lse) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
}

template <int D, typename T, int MT>
cudaError_t launch(const PagedParams& p, cudaStream_t s) {
    using F = Cfg<D, T, MT>;
    static std::atomic<int> optin[kMaxOptinDevices];
    const cudaError_t e = smem_optin(reinterpret_cast<const void*>(paged_kernel<D, T, MT>), F::kSmem, optin);
    if (e != cudaSuccess) return e;
    paged_kernel<D, T, MT><<<p.ctas, kWarps * 32, F::kSmem, s>>>(p);
    return cudaGetLastError();
}
template <int D, typename T>
cudaError_t join(const PagedParams& p, int tile_rows, cudaStream_t s) {
    const int64_t all = std::min<int64_t>((int64_t)p.t.max_new * p.G, p.max_rows), rows = std::min<int64_t>(all, tile_rows);
    // Large tiles: a CTA a row costs 2 us for about 2432 rows (16 CTAs a multiprocessor), cut or not; a warp for 2 rows takes
    // 1.5 us a row and 0.3 us a part.  (1 x 40 rows x 2 heads on 100 k tokens, 76 parts: 207 us by warps, 44 by rows.)
    const int64_t items = (all + tile_rows - 1) / tile_rows * p.t.B * p.c.Hkv, parts = p.ctas / items + 1;
    const bool by_row = tile_rows <= 32 || rows * p.ctas < 3650 + 730 * parts;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(by_row ? rows : (rows + kJoinRows - 1) / kJoinRows), p.ctas - 1), cfg.blockDim = dim3(128), cfg.stream = s;
    cfg.attrs = &attr, cfg.numAttrs = 1;
    if (tile_rows == 16) return cudaLaunchKernelEx(&cfg, paged_join_kernel<D, T, 16>, p);
    if constexpr (sizeof(T) == 4 || D == 32) {
        if (tile_rows == 32) return cudaLaunchKernelEx(&cfg, paged_join_kernel<D, T, 32>, p);
    } else {
        if (by_row) return cudaLaunchKernelEx(&cfg, paged_join_kernel<D, T, kTcRows>, p);
        return cudaLaunchKernelEx(&cfg, paged_join_rows_kernel<D, T, kTcRows>, p);
    }
    return cudaErrorInvalidValue;
}
template <typename F>
cudaError_t by_type(int D, bool bf16, F&& f) {
    switch (D * 2 + bf16) {
        case 64: return f(std::integral_constant<int, 32>(), 0.f);
        case 65: return f(std::integral_constant<int, 32>(), __nv_bfloat16());
        case 128: return f(std::integral_constant<int, 64>(), 0.f);
        case 129: return f(std::integral_constant<int, 64>(), __nv_bfloat16());
        case 256: return f(std::integral_constant<int, 128>(), 0.f);
        default: return f(std::integral_constant<int, 128>(), __nv_bfloat16());
    }
}

}  // namespace

cudaError_t launch_paged(const PagedParams& p, int D, bool bf16, int tiles, cudaStream_t s) {
    return by_type(D, bf16, [&](auto d, auto t) {
        // (bf16 of width 64 and 128 with more than 16 rows runs on the tensor cores)
        if constexpr (sizeof(t) == 4 || d() == 32)
            if (tiles == 2) return launch<d(), decltype(t), 2>(p, s);
        return tiles == 1 ? launch<d(), decltype(t), 1>(p, s) : cudaErrorInvalidValue;
    });
}

cudaError_t launch_paged_join(const PagedParams& p, int D, bool bf16, int tile_rows, cudaStream_t s) {
    return by_type(D, bf16, [&](auto d, auto t) { return join<d(), decltype(t)>(p, tile_rows, s); });
}

}  // namespace cache
}  // namespace gdn
