/*
 * mm_experts.h -- C ABI of the operators for experts of a caller's own form (another activation, one
 * product only, 32-bit results) and for the step from gradients to an optimizer, in the same library
 * as the fused layer (mm.h) and the operators around it (mm_ops.h):
 *
 *   mm_expert_table      the stable order of a selection's slots by expert;
 *   mm_expert_dispatch   the tokens' rows in that order;
 *   mm_grouped_mm_*      each expert's rows times its matrix, ragged sizes, and the gradients;
 *   mm_expert_combine_*  a token's weighted sum of its slots' rows, and its gradients;
 *   mm_grad_norm         the norm of many tensors together;
 *   mm_grad_clip         the tensors scaled down to a largest norm.
 *
 * The rules of mm_ops.h hold here too: row-major contiguous device memory, every buffer (workspaces
 * included) belongs to the caller, nothing is allocated, all work is enqueued on `stream` and nothing
 * synchronises with the host. Host-side checks return an error before anything is enqueued. Host
 * threads may call concurrently on different workspaces. Pointers are aligned to their element; 16-byte
 * alignment where a function says so. Sums and products are held in 32 bits or more; every output is
 * rounded once to its type. Repeats give the same bits.
 */
#ifndef MM_EXPERTS_H_
#define MM_EXPERTS_H_

#include "mm_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Version of this header's functions and structs. */
int mm_experts_version(void);

/* ---- the order of a selection -------------------------------------------------------------
 *
 * Slots s = t K + k of topk_ids int32 [T, K], sorted by expert, equal ones by s:
 *   offsets[e]      int32 [E + 1]  slots with an id below e (of those with an expert)
 *   row_of_slot[s]  int32 [T, K]   place of slot s in the order
 *   slot_of_row[r]  int32 [T K]    slot at place r
 * An id outside [0, E) is a slot without an expert: row_of_slot is -1 there, and as many places of
 * slot_of_row behind offsets[E] are -1. These are mm_forward's tables without their padding.
 * Sizes: T >= 0, 1 <= E <= 1024, 1 <= K <= 16, T K < 2^31 - 2^16, 1 <= H <= 2^20. */
typedef struct mm_expert_desc {
  int64_t T, H;
  int32_t E, K;
  int32_t type; /* MM_BF16 or MM_FP32: of x, rows, y and their gradients */
} mm_expert_desc;

/* Bytes of workspace of mm_expert_table (0: unsupported sizes). Needs no initialisation; up to 2048
 * slots use none (NULL). H and type of the descriptor are not used by the two. */
size_t mm_expert_table_workspace_size(const mm_expert_desc* d);

mm_status mm_expert_table(const mm_expert_desc* d, const int32_t* topk_ids, int32_t* offsets,
                          int32_t* row_of_slot, int32_t* slot_of_row, void* workspace,
                          size_t workspace_bytes, void* stream);

/* rows[r] = x[slot_of_row[r] / K] (x [T, H], rows [T K, H]); rows behind offsets[E] are zero. offsets
 * and row_of_slot are mm_expert_table's; places outside [0, T K) are not written. */
mm_status mm_expert_dispatch(const mm_expert_desc* d, const void* x, const int32_t* offsets,
                             const int32_t* row_of_slot, void* rows, void* stream);

/* y[t] = sum_k w[t,k] rows[row_of_slot[t,k]], k ascending, over the slots with an expert (a token
 * without one gets zeros). w fp32 [T, K], or NULL: 1 (the gradient of mm_expert_dispatch). */
mm_status mm_expert_combine(const mm_expert_desc* d, const void* rows, const int32_t* row_of_slot,
                            const float* weights, void* y, void* stream);

/* d_rows[r] = w[s] dy[t], zero behind offsets[E]; d_weights[t,k] = <dy[t], rows[r]> (fp32 [T, K], zero
 * for a slot without an expert; NULL: not wanted, and rows may be NULL too). */
mm_status mm_expert_combine_backward(const mm_expert_desc* d, const void* dy, const void* rows,
                                     const int32_t* offsets, const int32_t* row_of_slot,
                                     const float* weights, void* d_rows, float* d_weights,
                                     void* stream);

/* ---- grouped products ---------------------------------------------------------------------
 *
 *   out[r]      = rows[r] W[e]                 offsets[e] <= r < offsets[e + 1]
 *   d_weight[e] = rows_e^T d_out_e             summed over the expert's rows (zero without rows)
 *
 * rows bf16 [R, K], W bf16 [E, K, N] or, `transposed`, [E, N, K] (as a linear layer keeps it), offsets
 * int32 [E + 1]: rising, from 0 on, at most R. Rows in no expert's range (before the first, behind the
 * last) have no part, whatever they hold; they are zero in `out`. The gradient of `rows` is
 * mm_grouped_mm of d_out with K and N exchanged and `transposed` negated. Offsets that fall, start below
 * 0 or end above R make every element of the output NaN; no row outside [0, R) is touched.
 * Sizes: 0 <= R < 2^30, 1 <= E <= 1024, K and N multiples of 8 up to 65536. rows, W, out, d_out and
 * d_weight 16-byte aligned. out_type (MM_BF16 or MM_FP32): of `out`, or of d_weight.
 * Device waits are bounded; what a wait that runs out (a failing device) leaves without a result is
 * NaN, and the caller's status word, if there is one, says so. */
#define MM_GROUPED_SINGLE_CTA 0x1u /* flags: one CTA per tile */
#define MM_GROUPED_CTA_PAIRS 0x2u  /* flags: tiles shared by two CTAs. Without either flag the form goes
                                      by the sizes; results are the same bit for bit. */
/* flags, a test hook for the failure path: the first CTA withholds its first sum, and device waits are
 * bounded by 50 ms instead of 2 s. The call ends with NaN where results are missing. */
#define MM_GROUPED_TEST_STALL 0x80000000u
typedef struct mm_grouped_desc {
  int64_t R, K, N;
  int32_t E;
  int32_t transposed;
  int32_t out_type;
  uint32_t flags;
} mm_grouped_desc;

/* Bytes of workspace (0: unsupported sizes). Need no initialisation; one call at a time may use them.
 * They depend on the current device's number of SMs. Where mm_grouped_mm's is 256, it uses none
 * (NULL); where it uses some, it is more. */
size_t mm_grouped_mm_workspace_size(const mm_grouped_desc* d);
size_t mm_grouped_weight_grad_workspace_size(const mm_grouped_desc* d);

mm_status mm_grouped_mm(const mm_grouped_desc* d, const void* rows, const void* weight,
                        const int32_t* offsets, void* out, void* workspace, size_t workspace_bytes,
                        void* stream);

/* accumulate: the sums are added to what d_weight holds (in 32 bits, one rounding); experts without
 * rows keep theirs. d_weight has W's layout. */
mm_status mm_grouped_mm_weight_grad(const mm_grouped_desc* d, const void* rows, const void* d_out,
                                    const int32_t* offsets, void* d_weight, int accumulate,
                                    void* workspace, size_t workspace_bytes, void* stream);

/* The same with a status: int32 [2] in device memory, zero before its first call and the caller's to read
 * and to set back; any number of calls may share it (NULL: none). The first wait that runs out sets
 * status[0] to MM_ERR_TIMEOUT and status[1] to what was awaited (1: a free stage for operands, 2: a free
 * accumulator, 3: operands, 4: the next tile, 5: a free place for one, 6: a sum), plus 256 times the
 * number of the CTA; later ones leave both. It costs nothing where no wait runs out. */
mm_status mm_grouped_mm_ex(const mm_grouped_desc* d, const void* rows, const void* weight,
                           const int32_t* offsets, void* out, void* workspace, size_t workspace_bytes,
                           int32_t* status, void* stream);
mm_status mm_grouped_mm_weight_grad_ex(const mm_grouped_desc* d, const void* rows, const void* d_out,
                                       const int32_t* offsets, void* d_weight, int accumulate,
                                       void* workspace, size_t workspace_bytes, int32_t* status,
                                       void* stream);

/* ---- the norm of many tensors, and clipping -----------------------------------------------
 *
 *   norm = sqrt(sum over all tensors of the squares of their elements)
 *   out  = min(1, max_norm / (norm + eps)) * data
 * Squares are summed in 32 bits over at most 64 elements (in 64 bits where they would leave the range
 * of 32), further in 64 bits: the norm is right for elements of any size. norm is fp32 (infinite where
 * it is above that type). A NaN among the elements makes the norm and with it all of `out` NaN, an
 * infinity makes the finite elements 0, as the formula has it. */
typedef struct mm_tensor_ref {
  const void* data;
  void* out;         /* mm_grad_clip: where the scaled elements go; may be `data` itself */
  int64_t count;     /* elements, contiguous; 0: data and out may be NULL */
  int32_t type;      /* MM_BF16 or MM_FP32 */
  int32_t out_type;  /* the same; of data and out that are one: equal to type */
} mm_tensor_ref;

/* Bytes of workspace for n tensors (0: unsupported). Needs no initialisation. */
size_t mm_grad_workspace_size(int64_t n);

/* `tensors`: n descriptions in host memory, read before the call returns. 0 <= n < 2^20. No tensor
 * overlaps an `out` other than its own. */
mm_status mm_grad_norm(int64_t n, const mm_tensor_ref* tensors, float* norm, void* workspace,
                       size_t workspace_bytes, void* stream);
mm_status mm_grad_clip(int64_t n, const mm_tensor_ref* tensors, double max_norm, double eps, float* norm,
                       void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MM_EXPERTS_H_ */
