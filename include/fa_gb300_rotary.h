/*
 * fa_gb300_rotary.h — C ABI of rotary positions, next to fa_gb300.h and
 * fa_gb300_serve.h and in the same library: turning queries and keys (and
 * their gradients), and appending new keys and values to the paged 4-bit cache
 * with the turn on the way.
 *
 * Conventions are those of fa_gb300_serve.h.  In addition:
 *   - The first rot_dim elements of a head are rot_dim / 2 pairs: elements i
 *     and i + rot_dim / 2 (interleaved = 0) or 2 i and 2 i + 1 (1).  rot_dim is
 *     a multiple of 16 up to d; elements past it are copied.
 *   - turns: int64 [rot_dim / 2], device: pair i turns by turns[i] / 2^64 of a
 *     whole turn a position (an angle of f radians is f / (2 pi) of a turn).
 *     The angle at position p is 2 pi frac(p turns[i] / 2^64): exact but for
 *     turns' last bit, for every 32-bit position, negative ones included.
 *   - magnitude (finite, above 0) multiplies cos and sin, as scalings for long
 *     contexts want; 1 otherwise.
 *   - a' = magnitude (a cos - b sin), b' = magnitude (a sin + b cos), in fp32,
 *     rounded to bf16 once.
 */
#ifndef FA_GB300_ROTARY_H
#define FA_GB300_ROTARY_H

#include "fa_gb300_serve.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * fa_rotate — turns q and k by their positions.
 *
 *   q, k         : bf16, element (b, n, h, e) at b * batch + n * token + h *
 *                  head stride + e; 0 <= b < B, 0 <= n < N, h < Hq (Hk).  k and
 *                  k_out are NULL where Hk is 0.
 *   q_out, k_out : bf16, written; strides of their own.  An output is its own
 *                  input with the same strides (in place) or shares no element
 *                  with any input; outputs share none.
 *   strides      : HOST array of 12: (batch, token, head) of q, k, q_out and
 *                  k_out, in elements, each a multiple of 8 up to 2^40; an output's
 *                  elements lie at places of their own.
 *   positions    : int32, device; token (b, n)'s is positions[b * position_stride
 *                  + n].  NULL: n.  position_stride is 0 (the same for every
 *                  b) or at least N.
 *   backward     : 1 = turn the other way: the gradients of the inputs from
 *                  those of the outputs.
 * One launch.  B <= 65535, B * N <= 2^30.  Returns FA_OK (also when there is
 * nothing to do), FA_ERR_INVALID_ARG, FA_ERR_NULL, FA_ERR_ALIGN (q, k, q_out, k_out 16
 * bytes, turns 8, positions 4), FA_ERR_ALIAS, FA_ERR_DEVICE or FA_ERR_LAUNCH.
 */
int fa_rotate(const void* q, const void* k, void* q_out, void* k_out, const int* positions, const long long* turns,
              int B, int N, int Hq, int Hk, int d, int rot_dim, int interleaved, float magnitude, int backward,
              const long long* strides, long long position_stride, void* stream);

/*
 * fa_kv4_append — fa_rotate of new queries and keys and fa_kv4_store of the
 * keys and values in one launch.
 *
 *   q, k, v   : bf16 [T][Hq][d] and [T][Hkv][d], token strides q_stride, k_stride, v_stride;
 *               Hq = 0 (q and q_out NULL) leaves q out.
 *   q_out     : bf16 [T][Hq][d], contiguous; written.
 *   k_out     : bf16 [T][Hkv][d], contiguous; written with the turned keys.  NULL:
 *               they are not wanted.
 *   positions : int32 [T], device: the positions to turn by.  NULL: each
 *               token's place in its sequence.
 * cache, page_table, seq_lens, cu_seqlens, k_scale, v_scale and errors are as
 * for fa_kv4_store, and so is what is stored: the turned key is rounded to bf16
 * (correctly, but for a chance of about 2^-30 an element) and then to 4 bits.
 * Rows of q_out and k_out of tokens outside all sequences are left as they
 * were; a token that is not stored (`errors`) is turned all the same.
 * One launch.  Errors as fa_kv4_store's.
 */
int fa_kv4_append(const void* q, const void* k, const void* v, void* q_out, void* k_out, void* cache,
                  const int* page_table, const int* seq_lens, const int* cu_seqlens, const int* positions,
                  const long long* turns, int T, int n_seqs, int max_pages, int num_pages, int page_size, int Hq,
                  int Hkv, int d, int rot_dim, int interleaved, float magnitude, long long q_stride,
                  long long k_stride, long long v_stride, float k_scale, float v_scale, int* errors, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_ROTARY_H */
