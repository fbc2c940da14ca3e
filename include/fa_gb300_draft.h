/*
 * fa_gb300_draft.h — C ABI of drafted tokens, next to fa_gb300_serve.h and in
 * the same library: attention of a tree of drafted tokens over the paged 4-bit
 * cache, their verification against the target's probabilities, and keeping the
 * accepted ones in the cache.
 *
 * Conventions are those of fa_gb300_serve.h.  In addition:
 *   - A tree has n_nodes places, 1 to 64, the same for every sequence of a
 *     call, with parents int32 [n_seqs][n_nodes], device: node i's parent is a
 *     node before it, or -1, the context itself.  Any other value (-2, say)
 *     means that there is no node in this place, so that smaller trees fit; nor
 *     is there one below such a place.
 *   - In the cache the places are the last n_nodes positions of the sequence
 *     (seq_lens counts them), node i's at seq_lens - n_nodes + i whatever its
 *     depth; what comes before them is the context.  A place at a position
 *     below 0 has no node.
 *   - FA_KV4_BAD_TREE is set in `errors` where a parent does not come before
 *     its child.
 */
#ifndef FA_GB300_DRAFT_H
#define FA_GB300_DRAFT_H

#include "fa_gb300_serve.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FA_KV4_BAD_TREE 4

/*
 * fa_kv4_tree_attention — as fa_kv4_attention for the nodes of a tree: node i
 * sees the whole context and the nodes on its line from the context, itself
 * included (their keys and values are in the cache: store or append first).
 *
 *   q : bf16 [n_seqs * n_nodes][Hq][d], token stride q_stride; row
 *       s * n_nodes + i is node i of sequence s.
 *   o, lse : as fa_kv4_attention's.  A place without a node gets O = 0 and
 *       LSE = -inf, whatever q holds there.
 * Everything else is as for fa_kv4_attention.  How a call is divided goes by the
 * table's width, max_pages: small trees over short contexts are quickest (by a
 * tenth to a fifth) under a table not much wider than the longest sequence.
 */
int fa_kv4_tree_attention(const void* q, const void* cache, const int* page_table, const int* seq_lens,
                          const int* parents, void* o, float* lse, int n_seqs, int n_nodes, int Hq, int Hkv, int d,
                          int max_pages, int num_pages, int page_size, long long q_stride, float scale, float k_scale,
                          float v_scale, int* errors, void* workspace, size_t workspace_bytes, void* stream);

/* The workspace fa_kv4_tree_attention needs for these sizes on the current device, in bytes. */
int fa_kv4_tree_attention_workspace(int n_seqs, int n_nodes, int Hq, int Hkv, int d, int max_pages, int page_size,
                                    size_t* bytes);

/*
 * fa_verify_tree — which drafted tokens are kept, and the token after them, so
 * that what comes out is distributed as the target model's own sampling.
 *
 * Node 0 (parent -1) holds the token that the context ends with, already
 * decided; the others are drafts.  From node 0 on, with r = p, the target's
 * distribution after the node (softmax of its logits / temperature), the
 * node's children are tried in order: child j with token x is accepted where
 *
 *     uniforms[j] q(x) < r(x),
 *
 * q being the draft's distribution that the children were drawn from, and the
 * walk goes on from it; else r becomes max(r - q, 0), normalised (as it was,
 * where nothing would be left).  Where no child is accepted, the next token is
 * drawn from r: the first one whose running sum of r exceeds uniforms[0].
 * Without draft_probs a child is a token given, not drawn: q is 1 at its
 * token, so that it is accepted where uniforms[j] < r(x), and r loses it otherwise.
 *
 *   logits      : bf16 (logits_fp32 = 0) or fp32 (1) [n_seqs * n_nodes][V], rows logits_stride
 *                 elements apart (at least V): row s * n_nodes + i holds the
 *                 target's after node i.  -inf is a token that cannot come; NaN counts
 *                 as -inf, +inf as the largest finite value.
 *   tokens      : int32 [n_seqs][n_nodes].  A node whose token is outside
 *                 [0, V) is passed over; node 0's is not looked at.
 *   parents     : int32 [n_seqs][n_nodes].  A node that node 0 does not lead to is not looked at.
 *   uniforms    : fp32 [n_seqs][n_nodes], random numbers from [0, 1); others are taken as its ends (NaN as 0).
 *   draft_probs : fp32 [n_seqs * n_nodes][V], rows draft_stride elements apart: row s *
 *                 n_nodes + i holds the distribution that node i's children
 *                 were drawn from (not read where it has none); or NULL.
 *   temperature : of all sequences; above 0; or 0, the target's likeliest token (the lowest of equals) with
 *                 probability 1.
 *   path        : int32 [n_seqs][n_nodes]; written: the kept nodes in order, node 0 first,
 *                 then -1.
 *   n_kept      : int32 [n_seqs]; written.  Next to n_kept - 1 accepted drafts
 *                 this counts node 0; 0 where there is no node 0 (parents[0] is not
 *                 -1), with next_token -1.
 *   next_token  : int32 [n_seqs]; written.  -1 where every logit of the row is -inf.
 *
 * Probabilities are taken to 2^-44 of a row's largest (exponentials right to 2^-29,
 * sums in 64-bit integers): where a running sum passes a random number hardly
 * ever depends on roundings, and never on how the work is divided.  A drawn child's
 * own r(x) is taken as it is down to 2^-126 of the largest, and as 0 below.
 * V <= 2^18.  One launch.  Errors: FA_ERR_INVALID_ARG, FA_ERR_NULL, FA_ERR_ALIGN (each
 * pointer to its element's size), FA_ERR_ALIAS, FA_ERR_DEVICE, FA_ERR_LAUNCH.
 */
int fa_verify_tree(const void* logits, int logits_fp32, const int* tokens, const int* parents, const float* uniforms,
                   const float* draft_probs, int* path, int* n_kept, int* next_token, int n_seqs, int n_nodes, int V,
                   long long logits_stride, long long draft_stride, float temperature, void* stream);

/*
 * fa_kv4_keep — moves the kept nodes' keys and values to the first places of
 * the tree, in order: what is cached at seq_lens[s] - n_nodes + path[s][j] goes
 * to seq_lens[s] - n_nodes + j, for j < n_kept[s], all read before any is
 * written.  No other byte of the cache changes.
 *
 *   path, n_kept : as fa_verify_tree writes them.
 *   new_lens     : int32 [n_seqs]; written: seq_lens - n_nodes + n_kept, at least 0.
 * An entry of path outside [0, n_nodes) and positions and pages as in
 * fa_kv4_store set bits in `errors` and are skipped; n_kept is taken as within
 * [0, n_nodes].  Two sequences must not share the pages that the places lie in.
 * One launch.  Errors as fa_kv4_store's.
 */
int fa_kv4_keep(void* cache, const int* page_table, const int* seq_lens, const int* path, const int* n_kept,
                int* new_lens, int n_seqs, int n_nodes, int max_pages, int num_pages, int page_size, int Hkv, int d,
                int* errors, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_DRAFT_H */
