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
 *   mm_grad_scale        the tensors scaled down to a largest norm.
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

/* ---- grouped products ---------------------------------------------------------------------
 *
 *   out[r]      = rows[r] W[e]                 offsets[e] <= r < offsets[e + 1]
 *   d_weight[e] = rows_e^T d_out_e             summed over the expert's rows (zero without rows)
 *
 * rows bf16 [R, K], W bf16 [E, K, N] or, `transposed`, [E, N, K] (as a linear layer keeps it), offsets
 * int32 [E + 1]: rising, from 0 on, at most R. Rows in no expert's range (before the first, behind the
 * last) are not read; they are zero in `out`. The gradient of `rows` is mm_grouped_mm of d_out with K
 * and N exchanged and `transposed` negated. Offsets that fall, start below 0 or end above R make every
 * element of the output NaN; no row outside [0, R) is touched.
 * Sizes: 0 <= R < 2^31, 1 <= E <= 1024, K and N multiples of 8 up to 65536. rows, W, out, d_out and
 * d_weight 16-byte aligned. out_type (MM_BF16 or MM_FP32): of `out`, or of d_weight.
 * Device waits are bounded; what a wait that runs out (a failing device) leaves without a result is
 * NaN. */
#define MM_GROUPED_SINGLE_CTA 0x1u /* flags: one CTA per tile */
#define MM_GROUPED_CTA_PAIRS 0x2u  /* flags: tiles shared by two CTAs. Without either flag the form goes
                                      by the sizes; results are the same bit for bit. */
typedef struct mm_grouped_desc {
  int64_t R, K, N;
  int32_t E;
  int32_t transposed;
  int32_t out_type;
  uint32_t flags;
} mm_grouped_desc;

/* Bytes of workspace that mm_grouped_mm and mm_grouped_mm_weight_grad need (0: unsupported sizes).
 * Needs no initialisation; one call at a time may use it. */
size_t mm_grouped_workspace_size(const mm_grouped_desc* d);

mm_status mm_grouped_mm(const mm_grouped_desc* d, const void* rows, const void* weight,
                        const int32_t* offsets, void* out, void* workspace, size_t workspace_bytes,
                        void* stream);

/* accumulate: the sums are added to what d_weight holds (in 32 bits, one rounding); experts without
 * rows keep theirs. d_weight has W's layout. */
mm_status mm_grouped_mm_weight_grad(const mm_grouped_desc* d, const void* rows, const void* d_out,
                                    const int32_t* offsets, void* d_weight, int accumulate,
                                    void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MM_EXPERTS_H_ */
