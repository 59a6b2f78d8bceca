// gdn_linear.cuh - linear attention with a decay for each head: job tables and launchers shared by the
// kernels (gdn_linear.cu: every size and type, and the single-token step; gdn_linear_tc.cu: tensor cores) and
// the host side (gdn_hybrid_api.cu).
//
//     S_t = alpha_h S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t,   S in R^{d_v x d_k}
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn {
namespace lin {

constexpr int kMaxJobs = 384;    // jobs per launch (the host splits larger batches)
constexpr int kMaxCkpts = 1536;  // checkpoints per launch

// One scan over a contiguous token range, the same for all heads.
struct Job {
    int64_t tok_begin;    // stream row of the first token
    const float* s0;      // [H, dv, dk] initial state, nullptr = zeros
    float* s_final;       // [H, dv, dk] state after the last token, or nullptr
    int32_t len;          // tokens
    int32_t ck_begin;     // first entry of the launch's checkpoint table
    int32_t ck_count;
    int32_t pad_;
};
struct Ckpt {
    int32_t pos;    // 1-based token position within the job
    int32_t slot;   // destination in ckpt_states
};

struct Params {
    CUtensorMap tm_q, tm_k, tm_v, tm_o;   // tensor-core kernel only: [T, heads, d], box (64, 1, 128), 128-byte swizzle
    const void* q;                  // [T] rows of `q_stride` elements
    const void* k;
    const void* v;
    int64_t q_stride, k_stride, v_stride;
    const float* alpha;             // [H]
    void* o;                        // [T, H, dv], nullptr: no readout
    float* ckpt_states;             // [slots, H, dv, dk]
    unsigned int* status;
    unsigned long long wait_limit_ns;
    float scale;
    int32_t H, rep;                 // heads; heads that share one query / key head
    int32_t dv;
    int32_t rows_per_cta;           // gdn_linear.cu: state rows of a CTA
    int32_t n_jobs;
    int32_t stall_after;            // testing hook: stop issuing input copies after this many chunks (-1: off)
    int32_t pad_;
    Job jobs[kMaxJobs];
    Ckpt ckpts[kMaxCkpts];
};
static_assert(sizeof(Params) <= 32764, "kernel parameter block");

// Split scans: their segments' own states are chained into the segments' initial states.
struct Chain {
    const float* s0;   // initial state of the scan, nullptr = zeros
    int32_t slot;      // of the scan's first segment
    int32_t n;         // segments whose own state is there (all but the last)
};
struct ChainParams {
    float* states;        // [slots][H, dv, dk]: in: own state of a segment (from zero); out: initial state of the next
    const float* alpha;
    int32_t H, state;     // state = dv * dk
    int32_t n_scans;
    int32_t seg_len;      // tokens of each of those segments
    Chain scans[kMaxJobs];
};

struct StepParams {
    const void* q;
    const void* k;
    const void* v;
    int64_t q_stride, k_stride, v_stride;
    const float* alpha;
    float* states;
    const int32_t* slots;   // nullptr: slot b
    void* o;
    int64_t num_slots;
    float scale;
    int32_t B, H, rep, dv;
};

// rows of the state that one warp of the FP32-pipe kernels holds
constexpr int kWarpRows = 16;

cudaError_t launch_simt(const Params& p, int dk, bool in_bf16, bool out_bf16, cudaStream_t stream);
// d_k, d_v of 64 or 128, bf16 in and out (gdn_linear_tc.cu)
cudaError_t launch_tc(const Params& p, int dk, cudaStream_t stream);
cudaError_t launch_chain(const ChainParams& p, cudaStream_t stream);
cudaError_t launch_step(const StepParams& p, int dk, bool in_bf16, bool out_bf16, cudaStream_t stream);

}  // namespace lin
}  // namespace gdn
