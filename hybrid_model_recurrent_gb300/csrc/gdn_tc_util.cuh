// gdn_tc_util.cuh - what the tensor-core kernels of gdn_hybrid.h share: bounded waits, the issue of products, packing.
#pragma once

#include <cuda_bf16.h>

#include "gdn_chunk_tc.cuh"

namespace gdn {
namespace tcu {

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
// the same for a warp, which agrees on the outcome
__device__ __forceinline__ bool warp_wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint64_t limit) {
    return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag, limit));
}

// One lane of a whole warp, always the same.  The warps that issue products run their loops as whole warps and branch on
// this only around the instructions themselves: the operand descriptors then stay in uniform registers, where the
// instruction takes them from.  A loop of one lane alone moves each of them there anew, and a product took 2 to 3 times
// its 65 cycles.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// A tile of 128 rows as two 64-column blocks of [128][128 B], 128-byte swizzle, and the start of its 16-wide step i:
// K-major (the 64 columns of a block are 4 steps of 32 bytes), or rows as the product's K (a step is 16 rows).
constexpr uint32_t kBlock = 16384;
__device__ __forceinline__ uint64_t tile_desc(uint32_t saddr, bool rows_are_k) {
    return rows_are_k ? tc::sdesc(saddr, kBlock, 1024) : tc::sdesc(saddr, 16, 1024);
}
// (the address field counts 16 bytes and never carries out: shared memory ends below 2^18)
__device__ __forceinline__ uint64_t cols_step(uint64_t desc, int i) { return desc + (uint64_t)(((i >> 2) * kBlock + (i & 3) * 32) >> 4); }
__device__ __forceinline__ uint64_t rows_step(uint64_t desc, int i) { return desc + (uint64_t)(i * 2048 >> 4); }

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 32 bytes of one row in one store (`wide`: the address is 32-byte aligned), else in two: a thread that holds a row fills
// whole sectors only with the former
__device__ __forceinline__ void store32(void* p, const uint32_t (&x)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]),
                     "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(x[4], x[5], x[6], x[7]);
    }
}

}  // namespace tcu
}  // namespace gdn
