/*
 * fa_gb300_serve.h — C ABI of the serving operators next to fa_gb300.h, in
 * the same library: attention over packed prompts with grouped heads, and a
 * paged cache of keys and values held in 4 bits (storing, loading, and the
 * attention of new tokens over it).
 *
 * Conventions are those of fa_gb300.h: device pointers on the current
 * device unless said otherwise, asynchronous on `stream`, a status code
 * (enum fa_status) returned; a negative status is an error found before
 * launch, with nothing launched and the outputs untouched.  In addition:
 *   - T is a number of tokens; [T][heads][d] tensors have their heads
 *     contiguous within a token, and tokens q_stride (k_stride, v_stride)
 *     elements apart, so that q, k and v may be views of one fused
 *     projection's output.  A stride is at least heads * d and a multiple of
 *     8.  Outputs are contiguous.
 *   - Hq is a multiple of Hkv; query head h reads KV head h / (Hq / Hkv), and
 *     Hq / Hkv <= 128.
 *   - These operators allocate no device memory.  What they need beyond
 *     their operands is the caller's `workspace` (device, 256-byte aligned,
 *     at least as large as the matching ..._workspace call says; NULL where
 *     that is 0), used only by the work of that call: calls that may overlap
 *     on the GPU, replays of captured graphs among them, need workspaces of
 *     their own.  Its contents need no initial value and mean nothing after.
 *   - Every call can be captured into a graph.  Arguments read on the host
 *     (sizes, seq_lens) are then fixed in the graph.
 */
#ifndef FA_GB300_SERVE_H
#define FA_GB300_SERVE_H

#include <stddef.h>

#include "fa_gb300.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * fa_fwd_packed — attention over packed prompts.
 *
 *   q       : bf16 [T][Hq][d], token stride q_stride.
 *   k, v    : bf16 [T][Hkv][d], token strides k_stride, v_stride.
 *   o       : bf16 [T][Hq][d], contiguous; written.
 *   lse     : fp32 [Hq][T]; written with each row's natural-log logsumexp.
 *   seq_lens: HOST array of n_seqs lengths, each >= 0; their sum is at most
 *             T.  Sequence i holds the seq_lens[i] tokens after those of the
 *             sequences before it, and its tokens attend to it alone.  Tokens
 *             behind the last sequence are neither read into a result nor
 *             written (their rows of o and lse stay as they were).
 *   d       : 64 or 128.  T <= 2^30.
 *   causal  : 1 = a token sees its sequence up to itself; 0 = all of it.
 *   scale   : as for fa_fwd.
 *
 * A row whose visible scores are all -inf gets O = 0 and LSE = -inf.  P is
 * rounded to bf16 before P.V, every sum is fp32, O is rounded once.  Whatever
 * lies in the tensors outside a sequence, NaN and infinities included, does
 * not reach its results.  One launch per 1024 sequences, with a memset of the
 * workspace's counters before it where items are split between CTAs.
 * Results do not depend on timing: two calls give the same bits.
 *
 * Returns FA_OK (also when there is no token to do), FA_ERR_INVALID_ARG,
 * FA_ERR_NULL, FA_ERR_ALIGN (q, k, v, o 16 bytes, lse 4, workspace 256),
 * FA_ERR_ALIAS, FA_ERR_SCRATCH (workspace_bytes too small), FA_ERR_DEVICE or
 * FA_ERR_LAUNCH.
 */
int fa_fwd_packed(const void* q, const void* k, const void* v, void* o, float* lse, const int* seq_lens,
                  int n_seqs, int T, int Hq, int Hkv, int d, long long q_stride, long long k_stride,
                  long long v_stride, int causal, float scale, void* workspace, size_t workspace_bytes,
                  void* stream);

/* The workspace fa_fwd_packed needs for these sizes on the current device, in
 * bytes (0 where no item is split).  Errors as fa_fwd_packed's for the sizes. */
int fa_fwd_packed_workspace(const int* seq_lens, int n_seqs, int T, int Hq, int Hkv, int d, int causal,
                            size_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_SERVE_H */
