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
 * A row whose visible scores are all -inf gets O = 0 and LSE = -inf, whatever
 * V holds.  (In any other row NaN or an infinity in the value of a visible key
 * whose score is -inf may reach O or not: 0 * NaN in a product, or left out
 * with a part of weight 0.)  P is rounded to bf16 before P.V, every sum is
 * fp32, O is rounded once.  What a row does not see, other sequences and
 * (causal) later tokens, does not reach it even where that holds NaN or
 * infinities.  One launch per 1024 sequences, with a memset of the workspace's
 * counters before it where items are split between CTAs.
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

/*
 * The paged 4-bit cache.  16 consecutive elements of one head of one token
 * share an e4m3 scale s = e4m3(amax / (6 g)); an element's 4-bit code is the
 * e2m1 value nearest to x / (s g) (ties to the even code) and stands for
 * code * s * g, where g is k_scale or v_scale, the tensor's own scale: a power
 * of two (2^-40 to 2^40) chosen by the caller, 1 for values between about
 * 0.01 and 2688 in magnitude.  A block holding a NaN or an infinity reads back
 * as NaN; |x| above 2688 g saturates.
 *
 *   cache     : uint8 [num_pages][Hkv][page_size / 16 groups][18 d], 16-byte
 *               aligned; a group is 16 tokens of one head:
 *               [K codes 16 x d/2][K scales 16 x d/16][V codes][V scales], the
 *               even element of a code byte in its low four bits.  page_size
 *               is a power of two from 16 to 1024.
 *   page_table: int32 [n_seqs][max_pages], device.  Token x of sequence i
 *               lies in page page_table[i][x / page_size].  Entries past a
 *               sequence's tokens are not read.
 *   seq_lens  : int32 [n_seqs], device.
 *   errors    : one int32, device, or NULL.  A call sets FA_KV4_BAD_PAGE or
 *               FA_KV4_BAD_POSITION (bits) in it where it met a page id
 *               outside [0, num_pages), or a length or position that is
 *               negative or past max_pages * page_size, and never clears it.
 *               Such tokens are skipped: not stored, loaded as zeros, not
 *               attended to.  A length is taken as within that range.
 * Tables and lengths are read by the kernels, so a captured call follows them.
 */
#define FA_KV4_BAD_PAGE 1
#define FA_KV4_BAD_POSITION 2

/*
 * fa_kv4_store — quantises new keys and values into the cache.
 *
 *   k, v       : bf16 [T][Hkv][d], token strides k_stride, v_stride.
 *   cu_seqlens : int32 [n_seqs + 1], device, not decreasing: sequence i brings
 *                tokens cu_seqlens[i] .. cu_seqlens[i+1] - 1 of k and v.
 *   seq_lens   : the sequences' lengths with these tokens: they become the
 *                last cu_seqlens[i+1] - cu_seqlens[i] of the sequence.
 * Tokens of k and v outside all sequences are ignored; no other byte of the
 * cache is written.  Two sequences must not bring tokens for the same place
 * (a page shared by two sequences is copied before one of them writes to it).
 * One launch.  Errors: FA_ERR_INVALID_ARG, FA_ERR_NULL, FA_ERR_ALIGN (k, v,
 * cache 16 bytes, the rest 4), FA_ERR_ALIAS, FA_ERR_DEVICE, FA_ERR_LAUNCH.
 */
int fa_kv4_store(const void* k, const void* v, void* cache, const int* page_table, const int* seq_lens,
                 const int* cu_seqlens, int T, int n_seqs, int max_pages, int num_pages, int page_size, int Hkv,
                 int d, long long k_stride, long long v_stride, float k_scale, float v_scale, int* errors,
                 void* stream);

/*
 * fa_kv4_load — reads keys and values of cached tokens back as bf16 (exact:
 * bf16 holds every value the cache stands for).  The tokens are those that a
 * fa_kv4_store with the same tables would write: the last
 * cu_seqlens[i+1] - cu_seqlens[i] of sequence i's seq_lens[i].
 *
 *   k, v : bf16 [T][Hkv][d], contiguous; written.  Tokens outside all
 *          sequences are left as they were.
 * One launch.  Errors as fa_kv4_store's.
 */
int fa_kv4_load(const void* cache, const int* page_table, const int* seq_lens, const int* cu_seqlens, void* k,
                void* v, int T, int n_seqs, int max_pages, int num_pages, int page_size, int Hkv, int d,
                float k_scale, float v_scale, int* errors, void* stream);

/*
 * fa_kv4_attention — attention of each sequence's Lq newest tokens over its
 * cached keys and values (those tokens' own included: store first).
 *
 *   q   : bf16 [n_seqs * Lq][Hq][d], token stride q_stride; row i * Lq + j is
 *         the token at position seq_lens[i] - Lq + j, which sees positions up
 *         to its own.
 *   o   : bf16 [n_seqs * Lq][Hq][d], contiguous; written.
 *   lse : fp32 [Hq][n_seqs * Lq]; written.
 *   scale : as for fa_fwd; k_scale and v_scale as for the store.  scale *
 *         k_scale stays within fp32's range.
 * A row that sees no key (a position below 0, an empty sequence) gets O = 0
 * and LSE = -inf.  Scores, sums and O are fp32; P is rounded to f16 before
 * P.V; O is rounded once.  One launch, and a second that merges the parts of
 * sequences cut between CTAs where max_pages * page_size is over 512.
 * Results do not depend on timing: two calls give the same bits.
 *
 * Errors: as fa_kv4_store's, and FA_ERR_SCRATCH (workspace too small).
 */
int fa_kv4_attention(const void* q, const void* cache, const int* page_table, const int* seq_lens, void* o,
                     float* lse, int n_seqs, int Lq, int Hq, int Hkv, int d, int max_pages, int num_pages,
                     int page_size, long long q_stride, float scale, float k_scale, float v_scale, int* errors,
                     void* workspace, size_t workspace_bytes, void* stream);

/* The workspace fa_kv4_attention needs for these sizes on the current device, in bytes. */
int fa_kv4_attention_workspace(int n_seqs, int Lq, int Hq, int Hkv, int d, int max_pages, int page_size,
                               size_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_SERVE_H */
