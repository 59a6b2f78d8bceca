/*
 * gdn_hybrid.h - C ABI of the serving operators for the other layers of a hybrid model:
 * linear attention with a decay for each head (prompts and single tokens) and full
 * attention for a batch that shares a long prefix.
 *
 * They stand beside the Gated DeltaNet scan of gdn_scan.h and keep its conventions:
 * packed token streams, fp32 states [.., H, d_v, d_k] (key index fastest), 1-based
 * checkpoint positions, caller-owned buffers, a 256-byte workspace with the sticky device
 * status word (gdn_read_status), work enqueued on `stream`, host arrays read before the
 * call returns, and invalid arguments rejected on the host before anything is enqueued.
 * (The pages that gdn_scan.h cites have no counterpart of these operators: they name the
 * full-attention layers and their prefix KV, and recurrent layers other than the delta
 * rule, without defining them.)
 *
 * All values are expected to be finite.  An infinity or NaN spreads to what it takes part
 * in, and, in the linear prefill with d_k, d_v in {64, 128} and bf16 inputs (products of
 * whole tiles), also to the other tokens of its own sequence within the same 128-token
 * tile; in the attention, from a value of a request's tail also to that request's queries
 * that come before it.  Nothing outside a sequence's own tokens, or past a request's tail
 * length, is ever taken into a result.
 */
#ifndef GDN_HYBRID_H
#define GDN_HYBRID_H

#include "gdn_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Linear attention with a decay for each head:
 *
 *     S_t = alpha_h S_{t-1} + v_t k_t^T,     o_t = scale * S_t q_t
 *
 * A stream's rows are `*_stride` elements apart (0: packed) with the heads and the widths
 * contiguous inside a row, so that q, k and v may be slices of one projection's output.
 * Head h reads query and key head h / (num_heads / num_qk_heads).
 */
typedef struct gdn_linear_problem {
    int32_t num_seqs;            /* B >= 1                                              */
    int32_t num_heads;           /* H >= 1: heads of v, o and the states                */
    int32_t num_qk_heads;        /* heads of q and k; divides num_heads                 */
    int32_t d_k;                 /* 32, 64 or 128                                       */
    int32_t d_v;                 /* 32, 64 or 128                                       */
    const int64_t* cu_seqlens;   /* host [B+1] (unused by gdn_linear_step: may be NULL) */
    gdn_dtype qkv_dtype;         /* dtype of q, k, v                                    */
    gdn_dtype out_dtype;         /* dtype of o (rounded to nearest even)                */
    float scale;                 /* of the readout                                      */
    int64_t q_stride;            /* elements between tokens; 0 = num_qk_heads * d_k     */
    int64_t k_stride;            /* 0 = num_qk_heads * d_k                              */
    int64_t v_stride;            /* 0 = num_heads * d_v                                 */
} gdn_linear_problem;

/*
 * Prefill (the chunked form), with the checkpoints of gdn_prefill_ckpt and forks.
 *
 *  q, k         device [T, num_qk_heads, d_k]; q may be NULL when o is NULL
 *  v            device [T, H, d_v]
 *               (base addresses 16-byte aligned, row strides a multiple of 16 bytes)
 *  alpha        device [H] fp32 in [0, 1]: alpha_h (0: a token sees only itself)
 *  S0           device [slots, H, d_v, d_k] fp32, or NULL for zero initial states
 *  s0_index     host [B]: the slot of S0 that sequence b starts from, -1 for a zero state
 *               (several sequences may start from one slot: a fork of a cached prefix);
 *               NULL: slot b
 *  s0_slots     slots of S0 (bound of s0_index; with s0_index NULL at least B)
 *  o            device [T, H, d_v] out_dtype, packed, or NULL
 *  S_final      device [B, H, d_v, d_k] fp32
 *  ckpt_pos, cu_ckpt, ckpt_states   as gdn_prefill_ckpt; fewer than 2^23 in all.  A sequence
 *               with more than 1536 takes several launches in a row, and is taken in a call of
 *               at most 256 sequences (else GDN_ERR_UNSUPPORTED: give it a call of its own)
 *  scratch      device, 16-byte aligned, at least gdn_linear_scratch_bytes(p) bytes
 *               (may be NULL when that is 0): partial states of a call whose few long
 *               scans are split along the tokens
 *
 * S0 may not overlap S_final or ckpt_states.
 */
size_t gdn_linear_scratch_bytes(const gdn_linear_problem* p);

gdn_status gdn_linear_prefill(const gdn_linear_problem* p, const void* q, const void* k, const void* v,
                              const float* alpha, const float* S0, const int32_t* s0_index, int64_t s0_slots,
                              void* o, float* S_final, const int64_t* ckpt_pos, const int64_t* cu_ckpt,
                              float* ckpt_states, void* scratch, size_t scratch_bytes, void* workspace,
                              size_t ws_bytes, gdn_stream_t stream);

/*
 * One token a request (the recurrent form), the states updated in place.
 *
 *  q, k, v      device, one row a request (p->num_seqs rows)
 *  states       device [num_slots, H, d_v, d_k] fp32
 *  slots        device int32 [B]: the slot of each request, or NULL for slot b (then
 *               num_slots >= B).  A negative or out-of-range slot marks a padding row: its
 *               output is zero and no state is touched.  Two requests of one call must not
 *               share a slot (their updates would race).
 *  o            device [B, H, d_v] out_dtype, packed
 *
 * Nothing is read from the device on the host, so the call can be captured into a graph.
 */
gdn_status gdn_linear_step(const gdn_linear_problem* p, const void* q, const void* k, const void* v,
                           const float* alpha, float* states, int64_t num_slots, const int32_t* slots, void* o,
                           gdn_stream_t stream);

/*
 * Attention for a batch that shares a long prefix.  Request b has num_queries query tokens,
 * the last tokens of its own tail; query i attends to the whole prefix and to the tail's
 * tokens 0 .. tail_len[b] - num_queries + i:
 *
 *     x_j = softmax_scale (q_i . k_j),  o_i = sum_j e^{x_j} v_j / sum_j e^{x_j},
 *     lse_i = log sum_j e^{x_j}
 *
 * The prefix's part is computed once for all: the query rows of every request are stacked
 * against one read of the prefix keys and values, split along the prefix when there are
 * few rows, and joined with the tails' parts by their maxima and sums.  A row that sees
 * nothing (no prefix, empty tail) gives o = 0 and lse = -infinity.
 *
 *  num_q_heads, num_kv_heads   num_kv_heads divides num_q_heads; head h reads key/value
 *               head h / (num_q_heads / num_kv_heads)
 *  head_dim     32, 64 or 128
 *  softmax_scale  any sign; softmax_scale * log2 e finite in fp32
 *  prefix_len   P >= 0;  tail_cap  tokens a request's tail buffer holds, >= 0
 *  max_tail     host bound of tail_len (0 .. tail_cap); tail_len values above it are
 *               taken as max_tail, negative ones as 0
 *  *_stride     in elements, 0 = packed ([B, n, Hq, D], [P, Hkv, D], [B, cap, Hkv, D]);
 *               multiples of 16 bytes
 *  q            device [B, n, Hq, D]
 *  k_prefix, v_prefix  device [P, Hkv, D] (strides for the token and the head)
 *  k_tail, v_tail      device [B, cap, Hkv, D] (strides for the request, token and head);
 *               what lies past tail_len is never taken into a result
 *  tail_len     device int32 [B]; may be NULL when max_tail = 0
 *  o            device [B, n, Hq, D], dtype, packed
 *  lse          device [B, n, Hq] fp32, or NULL
 *  scratch      device, 32-byte aligned, gdn_prefix_scratch_bytes(p) bytes (partial sums)
 *
 * Nothing is read from the device on the host, so the call can be captured into a graph.
 */
typedef struct gdn_prefix_problem {
    int32_t batch;               /* B >= 1 */
    int32_t num_queries;         /* n >= 1: query tokens of each request */
    int32_t num_q_heads;
    int32_t num_kv_heads;
    int32_t head_dim;
    gdn_dtype dtype;             /* of q, k, v and o */
    int64_t prefix_len;
    int64_t tail_cap;
    int64_t max_tail;
    float softmax_scale;
    int64_t q_stride_b, q_stride_n, q_stride_h;
    int64_t kp_stride_t, kp_stride_h, vp_stride_t, vp_stride_h;
    int64_t kt_stride_b, kt_stride_t, kt_stride_h, vt_stride_b, vt_stride_t, vt_stride_h;
} gdn_prefix_problem;

size_t gdn_prefix_scratch_bytes(const gdn_prefix_problem* p);

gdn_status gdn_prefix_attention(const gdn_prefix_problem* p, const void* q, const void* k_prefix,
                                const void* v_prefix, const void* k_tail, const void* v_tail,
                                const int32_t* tail_len, void* o, float* lse, void* scratch,
                                size_t scratch_bytes, void* workspace, size_t ws_bytes, gdn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_HYBRID_H */
