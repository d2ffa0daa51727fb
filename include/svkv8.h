/*
 * svkv8.h -- C ABI of a paged cache held in 8 bits, in the same library as
 * specverify.h (libspecverify.so): writing it (packed tokens with the
 * rotation of svrope.h on the way, or a verified path of staged ones) and the
 * attention that reads it.
 *
 * Sources: as for svkv.h and svattn.h (the paged cache and its tree
 * attention); 猜想解码 (Speculative Decoding) 全景, 考点5 names reduced-precision
 * storage without a form, so the form is this library's:
 *
 *   k_pages, v_pages  [num_pages][LH][page_size][D] bytes, e4m3 (4 exponent
 *                     and 3 mantissa bits, largest value 448, no infinity)
 *   k_scales, v_scales [num_pages][LH][page_size / block] bytes s: 2^(s - 127)
 *                     (an exponent alone; 255 is NaN), one for each `block`
 *                     tokens of a page and row
 *   value = e4m3 * 2^(s - 127)
 *
 * Powers of two: the format floats, so its relative step is the same whatever
 * the scale; such a scale makes the values exact in 16 bits, and raising it
 * (below) exact down to the subnormal steps.
 *
 * Writing, per block of tokens and row: with a the largest size of its new
 * entries, e = the smallest exponent with a <= 448 * 2^e, at least the block's
 * own exponent when it holds entries of the request already, and within
 * [-117, 119] for bf16, [-15, 7] for fp16 (where every value of the cache is
 * exact in that type).  New entries are stored as e4m3(x * 2^-e), rounded to
 * nearest even, at most 448 in size; when e is above the block's own, its
 * older entries become e4m3(y * 2^(e_own - e)).  What is not finite is stored
 * as NaN and leaves the scale to the others.  A block whose first position is
 * new starts anew.
 *
 * Conventions as in svrope.h.  D a multiple of 16 in [16, 128]; block 8, 16,
 * 32, 64 or 128, page_size a multiple of it; pages aligned to 16 bytes.
 */
#ifndef SVKV8_H
#define SVKV8_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/*
 * sv_page_append into 8-bit pages (no queries, no packed keys): packed tokens
 * k, v [T][Hkv][D] of dtype SV_BF16 or SV_F16, keys rotated on the way when
 * table is not NULL, in 32 bits, and rounded once, to 8 bits.  Arguments,
 * requirements and faults as for sv_page_append; of a request that is not
 * appended also the block that holds its length keeps its values.
 */
int sv_page_append8(int dtype, const void* k, long long k_stride, const void* v,
                    long long v_stride, void* k_pages, void* v_pages, void* k_scales,
                    void* v_scales, const int32_t* block_table, const int32_t* seq_lens,
                    const int32_t* cu_seqlens, const float* table, int rows, int rot,
                    int interleaved, const int32_t* positions, int B, int T, int Hkv, int D,
                    int num_pages, int LH, int head0, int page_size, int block, int cols,
                    int32_t* out_seq_lens, int32_t* dev_status, void* stream);

/*
 * sv_page_commit into 8-bit pages: the verified path's staged entries
 * k_new, v_new [B][LH][N][D] (SV_BF16 or SV_F16) of every row.  nodes,
 * num_accepted, lengths (also in place) and faults as for sv_page_commit.
 * Requires 1 <= N <= 2^20, LH <= 2^31 - 1, B <= 65535.
 */
int sv_page_commit8(int dtype, void* k_pages, void* v_pages, void* k_scales, void* v_scales,
                    const void* k_new, const void* v_new, const int32_t* block_table,
                    const int32_t* seq_lens, const int32_t* nodes, const int32_t* num_accepted,
                    int B, int LH, int N, int D, int num_pages, int page_size, int block, int cols,
                    int32_t* out_seq_lens, int32_t* dev_status, void* stream);

/*
 * sv_tree_attn over 8-bit pages: queries, output and the tree's own staged
 * entries are of dtype.  Requirements and faults as for sv_tree_attn.
 * Values, cached and staged, are used exactly (a value that dtype cannot hold
 * exactly, through a scale outside the range above, counts as NaN).  The
 * softmax weights are rounded as by sv_tree_attn, whatever the values' sizes;
 * the sums of their products with values are kept such that they stay finite
 * for any values that dtype has, in steps of 2^-104 at most.
 * Cached keys are used exactly; queries and staged keys are split into 8-bit
 * terms (two for bf16, three for fp16) whose sums are off by up to 2^-17 of
 * the largest value of a query row, or of eight staged keys (nodes 8 i .. 8 i
 * + 7, whoever sees them): the scores have the errors of that.  A staged key
 * that is not finite gives NaN to the rows that see its node.
 * The terms are kept in the workspace, of sv_attn8_workspace_bytes() bytes.  A
 * batch of which they take more than 256 MiB goes in parts, one after another.
 * Which cache: 8 bits halve it always, and the time less often.  64 requests
 * over 2000 to 9000 entries, 8 KV heads of 128, bf16, us in 8 and in 16 bits,
 * by rows of a KV head (N * Hq / Hkv): 4 179 and 208, 16 182 and 209, 32 236
 * and 213, 88 248 and 227, 244 441 and 298; pages of 8 entries, 16 rows, 244
 * and 396.  Over contexts below some 1000 entries 16 bits are faster.
 */
/* Bytes of workspace for sv_tree_attn8 with up to B requests: beside
 * sv_attn_workspace_bytes() 256 MiB at most, or what one request takes; 0 for
 * sizes that it refuses. */
size_t sv_attn8_workspace_bytes(int B, int N, int Hq, int Hkv, int D);

int sv_tree_attn8(int dtype, const void* q, const void* k_pages, const void* v_pages,
                  const void* k_scales, const void* v_scales, const int32_t* block_table,
                  const int32_t* seq_lens, const void* k_new, const void* v_new,
                  const int32_t* parent, float scale, int B, int N, int Hq, int Hkv, int D,
                  int num_pages, int LH, int head0, int page_size, int block, int cols, void* out,
                  void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SVKV8_H */
