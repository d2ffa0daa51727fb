/*
 * svattn.h -- C ABI of the attention that reads the caches of svkv.h, in the
 * same library as specverify.h (libspecverify.so): a drafted token tree over
 * a paged cache, the newest tokens over a sink + ring cache, and whole
 * prompts under the same window.
 *
 * Sources (page title and section):
 *   猜想解码 (Speculative Decoding) 全景, 考点3 (tree attention verifies
 *     several branches in one forward pass: a drafted token sees the context
 *     and the tokens on its own path) and 考点1 (gamma + 1 tokens at once);
 *   deferred speculative decoding page (lqnn.cn), "环形上下文与注意力沉淀机制"
 *     (S persistent sink slots, the last W positions in a ring, Slot(pos) =
 *     pos for pos < S, else S + ((pos - S) mod W));
 *   vllm-ascend draft KV sliding-window page (cf-1.com), "block table 的裁剪方式"
 *     (the draft model attends over a windowed block table).
 *
 * What all three compute, per query row (request, token, query head h):
 *   out = sum_t p_t v_t,  p = softmax over the visible t of scale * (q . k_t)
 *   with keys and values of KV head h / (Hq / Hkv).
 * The products run on the tensor cores in the storage type; scores, the
 * softmax's running maximum and sum, and the output's sums are 32-bit floats.
 * The softmax weights are rounded once to the storage type for the product
 * with v (half a step of that type each; in 16-bit IEEE floats, whose smallest
 * values are coarser, such errors of all the keys that the sizes allow add up
 * to half a step of the largest weight at most, up to 2^28 keys), and the
 * output once at the end.
 *
 * Conventions as in specverify.h: caller-owned device buffers (row-major,
 * contiguous) of the current device, calls enqueued on `stream` (a
 * cudaStream_t, NULL = legacy default stream), host-detectable errors returned
 * (SV_ERR_* codes), data errors OR-ed into *dev_status (may be NULL), nothing
 * traps.
 *   dtype: SV_BF16, or SV_F16 (16-bit IEEE floats); SV_F32 is SV_ERR_DTYPE.
 *   Hq a multiple of Hkv with Hq / Hkv <= 128; D a multiple of 8 in [8, 128];
 *   scale > 0, and scale * log2(e) finite; all 16-bit buffers aligned to 16 bytes, int32 ones
 *   to 4.  `out` overlaps no input.
 *   A NaN or infinity in a visible key or value reaches rows of its own
 *   request (sequence) only, there also rows that do not see it; cache
 *   entries that no row of the request sees are never used, whatever they
 *   hold (stale pages, unfilled slots, slots that left the window).
 *   workspace: sv_attn_workspace_bytes() bytes, 256-byte aligned; its
 *   contents need no preparation and nothing is kept in it between calls.
 *   Calls that may overlap on the GPU need separate workspaces.
 *   SV_ST_TIMEOUT in *dev_status: an internal wait gave up, and the contents
 *   of `out` are void.
 */
#ifndef SVATTN_H
#define SVATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* storage type of the attention calls, besides SV_BF16 of specverify.h */
enum { SV_F16 = 2 };

/* Bytes of workspace for sv_tree_attn with N nodes, or sv_ring_attn with
 * R = N tokens, of any batch; 0 for sizes those calls refuse. */
size_t sv_attn_workspace_bytes(int N, int Hq, int Hkv, int D);

/*
 * Attention of the N nodes of a drafted tree over a paged cache, per request
 * b: node n sees the cache positions 0 .. seq_lens[b] - 1, itself and its
 * ancestors.  The tree is that of sv_tree_verify (node 0 = the last emitted
 * token, parent[b][0] == -1, 0 <= parent[b][n] < n); parent == NULL is a
 * chain (each node below the one before it: gamma + 1 tokens of a plain
 * draft, or one token with N == 1).
 *   q, out         [B][N][Hq][D]
 *   k_pages, v_pages [num_pages][LH][page_size][D]  (LH = layers * kv heads)
 *   block_table    [B][cols] int32: position t is in page
 *                  block_table[b][t / page_size], row t mod page_size
 *   seq_lens       [B] int32, in [0, cols * page_size], at most 2^31 - 1024
 *   k_new, v_new   [B][LH][N][D]: the tree's own entries
 * The call attends for one layer: rows head0 .. head0 + Hkv - 1 of LH.
 * Requires page_size a multiple of 8 in [8, 65536], 1 <= N <= 256,
 * 0 <= head0, head0 + Hkv <= LH, B * LH < 2^31, B <= 65535.  sv_window_block_table's
 * outputs are a block_table and seq_lens of this call (the draft model's
 * window).
 * A request with a length outside its range (SV_ST_BAD_LENGTH), a malformed
 * parent array (SV_ST_BAD_TOKEN) or a page of its length outside
 * [0, num_pages) (SV_ST_BAD_PAGE) gets zeros.
 */
int sv_tree_attn(int dtype, const void* q, const void* k_pages, const void* v_pages,
                 const int32_t* block_table, const int32_t* seq_lens, const void* k_new,
                 const void* v_new, const int32_t* parent, float scale, int B, int N, int Hq,
                 int Hkv, int D, int num_pages, int LH, int head0, int page_size, int cols,
                 void* out, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                 void* stream);

/*
 * Attention of the newest R tokens (R = gamma + 1, or 1) over the sink + ring
 * cache of sv_kv_commit, per request b: token j stands at position
 * p = pos[b] + j and sees the positions t <= p with t < sink or
 * t > p - window: cache entries below pos[b], and staged entries 0 .. j.
 *   q, out         [B][R][Hq][D]
 *   k_pool, v_pool [B][LH][sink + window][D]
 *   k_new, v_new   [B][LH][R][D]: the staged entries (as sv_kv_commit takes them)
 *   pos            [B] int32: committed positions; the cache is only read
 * Requires 1 <= R <= 64, window >= R, sink >= 0, sink + window <= 2^31 - 1024,
 * B * LH < 2^31, 0 <= head0, head0 + Hkv <= LH and B <= 65535.
 * A position outside [0, 2^31 - R) gives zeros and SV_ST_BAD_LENGTH.
 */
int sv_ring_attn(int dtype, const void* q, const void* k_pool, const void* v_pool,
                 const int32_t* pos, const void* k_new, const void* v_new, float scale, int B,
                 int R, int Hq, int Hkv, int D, int LH, int head0, int sink, int window,
                 void* out, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                 void* stream);

/*
 * Attention of whole prompts, packed one after another: token i of a
 * sequence sees its tokens t <= i with t < sink or t > i - window (window >=
 * the longest sequence: plain causal attention).
 *   q, out     [T][Hq][D];  k, v [T][Hkv][D]
 *   cu_seqlens [B + 1] int32, non-decreasing: sequence b holds the rows
 *              cu_seqlens[b] .. cu_seqlens[b + 1] - 1 (none: an empty sequence)
 * Rows of `out` in no sequence are left as they were.  A sequence whose
 * bounds are not 0 <= cu_seqlens[b] <= cu_seqlens[b + 1] <= T is skipped
 * (SV_ST_BAD_LENGTH); where such bounds give rows to two sequences, those rows
 * and the ones of later sequences are not defined.
 * Requires T <= 2^31 - 512, sink >= 0, window >= 1, B <= 65535.  No workspace.
 */
int sv_prompt_attn(int dtype, const void* q, const void* k, const void* v,
                   const int32_t* cu_seqlens, float scale, int B, int T, int Hq, int Hkv, int D,
                   int sink, int window, void* out, int32_t* dev_status, void* stream);

/*
 * Failure-handling test aid, as sv_test_withhold_slot: while enabled, one of
 * the slots of block 0 of the next attention calls never counts as filled, so
 * that the waits for it run out after their one-second limit (SV_ST_TIMEOUT).
 * No fault, trap or endless wait is involved.  Not thread-safe.  Returns SV_OK.
 */
int sv_attn_test_withhold(int enable);

#ifdef __cplusplus
}
#endif

#endif /* SVATTN_H */
