/*
 * svrope.h -- C ABI of rotary positions and of appending rotated keys to the
 * paged cache of svkv.h, in the same library as specverify.h
 * (libspecverify.so).
 *
 * Source (page title and section): deferred speculative decoding page
 * (lqnn.cn), "环形上下文与注意力沉淀机制" (rotary positions of cached keys) and
 * "C++ 环形 KV 缓存管理内核实现" (append to a preallocated pool); the paged
 * cache is that of sv_page_commit.
 *
 * Rotation of a head's first `rot` dimensions at position p, with the angles
 * p * w_i, i < rot / 2:
 *   y_a = x_a cos(p w_i) - x_b sin(p w_i)
 *   y_b = x_b cos(p w_i) + x_a sin(p w_i)
 *   half layout (interleaved == 0): a = i, b = i + rot / 2
 *   interleaved layout:             a = 2 i, b = 2 i + 1
 * The other dimensions stay.  Products and sums are 32-bit floats, each
 * rounded by itself (no multiply-add: the result does not depend on which
 * product one would keep exact); y is rounded once to the storage type.
 *
 * Conventions as in specverify.h: caller-owned device buffers of the current
 * device, calls enqueued on `stream` (a cudaStream_t, NULL = legacy default
 * stream), host-detectable errors returned (SV_ERR_* codes), data errors
 * OR-ed into *dev_status (may be NULL), nothing traps.
 *   dtype: SV_BF16 or SV_F16 (svattn.h).
 *   Packed tokens: x of T tokens, H heads and D dimensions has token t, head h
 *   at x + t * stride + h * D elements (stride >= H * D: a slice of a wider
 *   row, such as a fused projection's output, is taken as it is).
 *   D a multiple of 8 in [8, 256]; strides multiples of 8 elements; 16-bit
 *   buffers and tables aligned to 16 bytes, int32 ones to 4.
 *   rot even, in [2, D]; a table has `rows` rows [2][rot / 2] of 32-bit
 *   floats: cosines, then sines, of the positions 0 .. rows - 1.
 */
#ifndef SVROPE_H
#define SVROPE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* how sv_rope_table scales the rates w_i = base^(-2 i / rot) for contexts
 * `factor` times the `original` one */
enum {
  SV_ROPE_NONE = 0,   /* w_i */
  SV_ROPE_LINEAR = 1, /* w_i / factor (positions divided) */
  SV_ROPE_BASE = 2,   /* w_i of the base times factor^(rot / (rot - 2)); rot > 2 */
  SV_ROPE_RAMP = 3,   /* by pair: with d(t) = rot ln(original / (2 pi t)) / (2 ln base), the pair
                         that turns t times over the original context, lo = max(floor(d(high)), 0),
                         hi = min(ceil(d(low)), rot - 1) (0.001 more if equal) and r = (i - lo) /
                         (hi - lo) kept in [0, 1]: w_i (1 - r) + w_i / factor r */
  SV_ROPE_WAVE = 4    /* by wavelength: with t = original w_i / (2 pi) turns over the original
                         context and s = (t - low) / (high - low) kept in [0, 1]:
                         w_i s + w_i / factor (1 - s) */
};

/*
 * The table of positions first .. first + rows - 1: gain * cos(p w_i) and
 * gain * sin(p w_i).  The functions are 32-bit ones, off by less than 2^-22 of
 * the gain.  The rates are 64-bit floats by the formulas above, each with the
 * roundings of its own computation, about 2^-49 of it: the angle p w_i is off
 * by that part of itself (2^-32 at position 131072, 2^-18 at 2^31, with
 * w_i = 1) and loses nothing more, as whole turns fall off exactly.
 * Requires rows >= 0, first >= 0, first + rows <= 2^31 - 1, rot even in
 * [2, 256], base > 1, factor > 0, gain finite; RAMP and WAVE: original >= 1,
 * 0 < low < high.  A rate, or the base of SV_ROPE_BASE, that no 64-bit float
 * holds is refused.
 */
int sv_rope_table(int scaling, double base, double factor, int original, double low, double high,
                  double gain, int rot, int first, int rows, float* table, void* stream);

/*
 * Rotate queries and keys of T packed tokens at positions[t].  k may be NULL
 * (Hk 0).  q_out and k_out may be q and k themselves (with the same stride),
 * else they overlap no input.  Tokens whose position is outside [0, rows) are
 * left out (their output rows stay) and SV_ST_BAD_LENGTH is reported.
 * Requires T >= 0, 1 <= Hq <= 65535 and 0 <= Hk <= 65535.
 */
int sv_rope(int dtype, const void* q, long long q_stride, const void* k, long long k_stride,
            const int32_t* positions, const float* table, int rows, int rot, int interleaved,
            int T, int Hq, int Hk, int D, void* q_out, long long q_out_stride, void* k_out,
            long long k_out_stride, int32_t* dev_status, void* stream);

/*
 * Append packed tokens to the pages of a cache, the keys rotated on the way,
 * per request b with n = cu_seqlens[b + 1] - cu_seqlens[b] tokens: token j's
 * keys and values go to position seq_lens[b] + j, page
 * block_table[b][position / page_size], row position mod page_size, of rows
 * head0 .. head0 + Hkv - 1 of LH; out_seq_lens[b] = seq_lens[b] + n.
 *   k, v [T][Hkv][D] packed with strides; k_pages, v_pages
 *   [num_pages][LH][page_size][D]; block_table [B][cols]; seq_lens [B];
 *   cu_seqlens [B + 1], non-decreasing (none: an empty request).
 *   table == NULL: no rotation (rot, rows and interleaved are not looked at).
 *   positions [T] (may be NULL: a token's position in the cache): where its
 *   key is rotated to; a tree's nodes, whose positions follow their depth.
 *   q (may be NULL, Hq 0): queries of the same tokens, rotated to q_out in
 *   the same call.  k_out (may be NULL): the rotated keys packed, too.  Both
 *   may be q and k themselves.  (The staged entries [B][LH][N][D] of
 *   sv_tree_attn and sv_page_commit are pages of N rows: num_pages = B,
 *   cols = 1, block_table[b][0] = b, seq_lens[b] = 0.)
 *   out_seq_lens (may be NULL) overlaps no input: the other layers' calls
 *   still need the old lengths.
 * A request is not appended, out_seq_lens[b] = seq_lens[b], when its bounds
 * are not 0 <= cu_seqlens[b] <= cu_seqlens[b + 1] <= T, its length is
 * negative, the tokens do not fit the table's cols * page_size positions or
 * 2^31 - 1, a rotation's position is outside [0, rows) (SV_ST_BAD_LENGTH) or
 * a page in use outside [0, num_pages) (SV_ST_BAD_PAGE); what lies behind its
 * length in its pages, and its rows of q_out and k_out, are then not defined.
 * Rows of packed outputs in no request are left as they were.  Where bounds
 * decrease, which tokens of the requests around them are appended is not
 * defined.  No two requests may write one page.
 * Requires T >= 0, B <= 65535, page_size, cols, num_pages, LH >= 1,
 * 0 <= head0, head0 + Hkv <= LH, 1 <= Hkv and Hq <= 65535, and as for sv_rope.
 */
int sv_page_append(int dtype, const void* k, long long k_stride, const void* v,
                   long long v_stride, void* k_pages, void* v_pages, const int32_t* block_table,
                   const int32_t* seq_lens, const int32_t* cu_seqlens, const float* table,
                   int rows, int rot, int interleaved, const int32_t* positions, const void* q,
                   long long q_stride, void* q_out, long long q_out_stride, void* k_out,
                   long long k_out_stride, int B, int T, int Hq, int Hkv, int D, int num_pages,
                   int LH, int head0, int page_size, int cols, int32_t* out_seq_lens,
                   int32_t* dev_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SVROPE_H */
