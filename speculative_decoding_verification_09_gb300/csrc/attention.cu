// attention.cu -- C ABI of the attention over the caches (see include/svattn.h
// for the operations, layouts and error behaviour; the kernels are in
// attention.cuh).

#include "attention.cuh"
#include "svkv8.h"

namespace {

using namespace svattn;

constexpr float LOG2E = 1.44269504088896341f;

int g_withhold = 0;  // failure-handling test (sv_attn_test_withhold)

// -------------------------------------------------------------- host side

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// A map of 8-bit elements: dims[0] innermost, strides of dims 1.. in elements.
bool make_map8(CUtensorMap* m, const void* p, int rank, const uint64_t* dims,
               const uint64_t* strides, const uint32_t* box, CUtensorMapSwizzle swizzle) {
  cuuint64_t bytes[4];
  cuuint32_t one[5] = {1, 1, 1, 1, 1};
  for (int i = 0; i + 1 < rank; ++i) bytes[i] = strides[i];
  return encode_tiled()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, cuuint32_t(rank), const_cast<void*>(p),
                        dims, bytes, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A map of 16-bit elements: dims[0] innermost, strides of dims 1.. in elements.
bool make_map(CUtensorMap* m, int dtype, const void* p, int rank, const uint64_t* dims,
              const uint64_t* strides, const uint32_t* box) {
  cuuint64_t bytes[4];
  cuuint32_t one[5] = {1, 1, 1, 1, 1};
  for (int i = 0; i + 1 < rank; ++i) bytes[i] = strides[i] * 2;
  return encode_tiled()(m, dtype == SV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                            : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                        cuuint32_t(rank), const_cast<void*>(p), dims, bytes, box, one,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The layout for items of `rows` rows (see Smem): columns of the turned
// products, or 0 for a row per lane with one (128) or two (256) tiles.
Layout layout_of(int N, int G) {
  const int rows = N * G;
  if (rows <= 16) return {16, 16};
  if (rows <= 32) return {32, 32};
  return {0, N <= TILE / G ? TILE : 2 * TILE};
}

size_t workspace_for(int N, int G, int D) {
  const size_t rows = layout_of(N, G).rows, dp = D > 64 ? 128 : 64;
  return size_t(MAX_CTAS) * (2 * rows * (dp * 4 + 8) + sizeof(int4));
}

// Requests that a call over 8-bit pages takes at a time: as many as MOST_SPACE8 bytes hold of
// what is made of them, so that a workspace for both kinds of cache is bounded whatever the
// batch.  (32 heads of 128: 512 requests of 64 nodes over 500 to 2000 entries 1044 us in two parts
// and 1018 in one; 1194 in eight of 64 MiB.)
constexpr size_t MOST_SPACE8 = 256 << 20, TERMS8 = 3;  // (terms of fp16; bf16 has two)
int requests_at_once(int B, int N, int Hq, int Hkv, int D) {
  const size_t one = TERMS8 * N * (size_t(Hq) + Hkv) * D + size_t(4) * N * Hq +
                     size_t(Hkv) * ((N + TILE - 1) / TILE) * 16 * 4;
  const size_t n = MOST_SPACE8 / one;
  return n < 1 ? 1 : n < size_t(B) ? int(n) : B;
}

// What the first kernel of a call over 8-bit pages leaves for the second, behind the partials:
// the queries' and staged keys' terms, and their powers of two (of B requests at a time).
struct Space8 {
  size_t q8, k8, qf, kf, all;
};
Space8 space_for8(int B, int N, int Hq, int Hkv, int D) {
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  const size_t tokens = size_t(B) * N;
  Space8 s;
  s.q8 = up(workspace_for(N, Hq / Hkv, D));
  s.k8 = s.q8 + up(TERMS8 * tokens * Hq * D);
  s.qf = s.k8 + up(TERMS8 * tokens * Hkv * D);
  s.kf = s.qf + up(4 * tokens * Hq);
  s.all = s.kf + up(size_t(B) * Hkv * ((N + TILE - 1) / TILE) * 16 * 4);
  return s;
}

// q and k_new of 8-bit calls come in `prep`.
int launch(AttnParams& A, int dtype, const void* q, const void* k, const void* v,
           const void* k_new, const void* v_new, void* workspace, void* stream,
           Prep8* prep = nullptr) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      sms < 1 || !encode_tiled())
    return SV_ERR_CUDA;
  const int ctas = sms < MAX_CTAS ? sms : MAX_CTAS;
  A.G = A.Hq / A.Hkv;
  A.tpt = TILE / A.G;
  A.withhold = g_withhold;
  if (dtype == SV_F16 || A.k_scales) {
    // the keys that a row may see, times a weight's error of 2^-(25 + lift): below 2^-11 (fp16);
    // times a weight of up to 2^(MOST_BF16 + lift): 1 at most (bf16)
    const long long window = (long long)A.sink + A.window;
    const long long keys = A.kind == TREE   ? (long long)A.cols * A.page + A.N
                           : A.kind == RING ? window + A.N
                                            : (window < A.T ? window : A.T);
    int lift = 0;
    while (lift < MOST_LIFT && keys >> (14 + lift)) ++lift;
    A.lift = float(lift);
    if (dtype == SV_BF16) {
      lift = 0;
      while (lift < 31 && keys >> lift) ++lift;  // (a length is below 2^31)
      A.lift = -MOST_BF16 - float(lift);
    }
  }
  const uint64_t D = A.D, tokens = A.kind == PROMPT ? uint64_t(A.T) : uint64_t(A.B) * A.N;
  const uint32_t q_tok = uint32_t(
      A.tpt < (A.kind == PROMPT ? A.T : A.N) ? A.tpt : (A.kind == PROMPT ? A.T : A.N));
  A.q_rows = int(q_tok) * A.G;
  if (prep) {
    const Space8 s = space_for8(A.B, A.N, A.Hq, A.Hkv, A.D);
    unsigned char* const w = static_cast<unsigned char*>(workspace);
    const uint64_t terms = dtype == SV_BF16 ? TERMS_OF<true> : TERMS_OF<false>;
    prep->q8 = w + s.q8;
    prep->k8 = w + s.k8;
    prep->qf = reinterpret_cast<float*>(w + s.qf);
    prep->kf = reinterpret_cast<float*>(w + s.kf);
    A.qf = prep->qf;
    A.kf = prep->kf;
    const uint32_t dp = A.D > 64 ? 128 : 64;
    const CUtensorMapSwizzle swizzle =
        A.D > 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    const uint64_t qd[5] = {D, uint64_t(A.G), uint64_t(A.Hkv), tokens, terms};
    const uint64_t qs[4] = {D, D * A.G, D * A.Hq, D * A.Hq * tokens};
    const uint32_t qb[5] = {dp, uint32_t(A.G), 1, q_tok, 1};
    const uint64_t kd[3] = {D, uint64_t(A.N), uint64_t(A.B) * A.Hkv * terms};
    const uint64_t ks[2] = {D, D * A.N};
    const uint32_t kb[3] = {dp, TILE, 1};
    if (!make_map8(&A.mq, prep->q8, 5, qd, qs, qb, swizzle) ||
        !make_map8(&A.mkn, prep->k8, 3, kd, ks, kb, swizzle))
      return SV_ERR_CUDA;
  } else {
    const uint64_t dims[4] = {D, uint64_t(A.G), uint64_t(A.Hkv), tokens};
    const uint64_t str[3] = {D, D * A.G, D * A.Hq};
    const uint32_t box[4] = {64, uint32_t(A.G), 1, q_tok};
    if (!make_map(&A.mq, dtype, q, 4, dims, str, box)) return SV_ERR_CUDA;
  }
  if (A.kind == TREE) {
    A.box = TILE;
    while (A.page % A.box) A.box /= 2;
    const uint64_t dims[4] = {D, uint64_t(A.page), uint64_t(A.LH), uint64_t(A.num_pages)};
    const uint64_t str[3] = {D, D * A.page, D * A.page * A.LH};
    const uint32_t box[4] = {A.k_scales ? (A.D > 64 ? 128u : 64u) : 64u, uint32_t(A.box), 1, 1};
    // (keys go to products as they are; values are read by threads)
    if (A.k_scales ? !make_map8(&A.mk, k, 4, dims, str, box,
                                A.D > 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B) ||
                         !make_map8(&A.mv, v, 4, dims, str, box, CU_TENSOR_MAP_SWIZZLE_NONE)
                   : !make_map(&A.mk, dtype, k, 4, dims, str, box) ||
                         !make_map(&A.mv, dtype, v, 4, dims, str, box))
      return SV_ERR_CUDA;
  } else if (A.kind == RING) {
    const uint64_t C = uint64_t(A.sink) + A.window;
    const uint64_t dims[3] = {D, C, uint64_t(A.B) * A.LH};
    const uint64_t str[2] = {D, D * C};
    const uint32_t box[3] = {64, TILE, 1};
    if (!make_map(&A.mk, dtype, k, 3, dims, str, box) ||
        !make_map(&A.mv, dtype, v, 3, dims, str, box))
      return SV_ERR_CUDA;
  } else {
    const uint64_t dims[3] = {D, uint64_t(A.Hkv), uint64_t(A.T)};
    const uint64_t str[2] = {D, D * A.Hkv};
    const uint32_t box[3] = {64, 1, TILE};
    if (!make_map(&A.mk, dtype, k, 3, dims, str, box) ||
        !make_map(&A.mv, dtype, v, 3, dims, str, box))
      return SV_ERR_CUDA;
    A.mkn = A.mk;
    A.mvn = A.mv;
  }
  Layout lay;
  int grid = ctas;
  if (A.kind != PROMPT) {
    const uint64_t dims[3] = {D, uint64_t(A.N), uint64_t(A.B) * A.LH};
    const uint64_t str[2] = {D, D * A.N};
    const uint32_t box[3] = {64, TILE, 1};
    if ((!A.k_scales && !make_map(&A.mkn, dtype, k_new, 3, dims, str, box)) ||
        !make_map(&A.mvn, dtype, v_new, 3, dims, str, box))
      return SV_ERR_CUDA;
    lay = layout_of(A.N, A.G);
    const int tpi = lay.rows == 2 * TILE ? 2 * A.tpt : A.tpt;
    A.MT = (A.N + tpi - 1) / tpi;
    // Items are not cut, and not joined, when they have few tiles: a cut item's partials
    // and the join cost more than runs that differ by up to an item, the more so the
    // more rows an item has; unless they are too few to keep the SMs' loads going.  (8 KV
    // heads of 128, lengths up to 8 times apart, inputs from HBM, us cut and whole.
    // 4 rows, 3 tiles: 16 items 12.5 and 10.9, 1280 49.0 and 45.6; 5 tiles: 16 items 13.1
    // and 13.6 (pages of 16: 13.4 and 16.4), 80 15.9 and 14.5; 8 tiles: 80 16.8 and 16.8,
    // 1280 69.0 and 71.8, but with 32 rows 83.2 and 78.8.  200 rows, 8 tiles: 16 items
    // 19.4 and 20.9, 80 29.1 and 24.6; 12 tiles: 320 66.3 and 61.9, 1280 196 and 188.)
    const long long entries = A.kind == TREE ? (long long)A.cols * A.page
                                             : (long long)A.sink + A.window;
    const long long most = (entries + TILE - 1) / TILE + (A.N + TILE - 1) / TILE;
    const long long items = (long long)A.B * A.Hkv * A.MT;
    // The kernel decides by the batch's longest request, and the join, which then finds
    // nothing to do, is launched unless no request of this cache can be longer.  (Tables of
    // 32768 positions, by their extent and by the lengths, of 893: 160 requests of 200 rows
    // 212 us and 168, 10 such requests 28.5 and 24.6.)
    A.whole_tiles = 2 * items >= ctas ? (lay.nq == 0 ? 12 : items >= 8LL * ctas ? 8 : 5) : 3;
    A.join = most > A.whole_tiles;
    const size_t rows = lay.rows, dp = A.D > 64 ? 128 : 64;
    unsigned char* w = static_cast<unsigned char*>(workspace);
    A.part_o = reinterpret_cast<float*>(w);
    A.part_ml = reinterpret_cast<float2*>(w + size_t(MAX_CTAS) * 2 * rows * dp * 4);
    A.desc = reinterpret_cast<int4*>(w + size_t(MAX_CTAS) * 2 * rows * (dp * 4 + 8));
  } else {
    // Two query tiles per item when that leaves every SM an item, else one: half the
    // work per item, for twice the loads of keys.  (Enough items: 24 ragged prompts
    // 90 us in pairs, 108 singly; 8192 tokens 321 and 380.)
    lay = {0, (long long)A.Hkv * (A.T / (2 * A.tpt)) >= ctas ? 2 * TILE : TILE};
    const int tpi = lay.rows == 2 * TILE ? 2 * A.tpt : A.tpt;
    // an upper bound: every sequence that holds a token adds at most one part item
    const long long items = (long long)A.Hkv * (A.T / tpi + (A.B < A.T ? A.B : A.T));
    if (items > 0x7fffffff) return SV_ERR_INVALID_ARG;
    grid = int(items);
    A.MT = 1;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (A.k_scales)
    return (dtype == SV_BF16 ? launch8_bf16 : launch8_f16)(A, *prep, lay, dev, grid, ctas, st);
  return (dtype == SV_BF16 ? launch_bf16 : launch_f16)(A, lay, dev, grid, ctas, st);
}

bool misaligned(const void* p, unsigned a) {
  return (reinterpret_cast<uintptr_t>(p) % a) != 0;
}

// Finite and positive, also in base-2 units.
bool bad_scale(float scale) { return !(scale > 0.0f) || !isfinite(scale * LOG2E); }

bool bad_heads(int Hq, int Hkv, int D) {
  return Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq / Hkv > MAX_GROUP || D < 8 || D > MAX_D ||
         D % 8 != 0;
}

}  // namespace

extern "C" {

int sv_attn_test_withhold(int enable) {
  g_withhold = enable ? 1 : 0;
  return SV_OK;
}

size_t sv_attn_workspace_bytes(int N, int Hq, int Hkv, int D) {
  if (N < 1 || N > MAX_N || bad_heads(Hq, Hkv, D)) return 0;
  return workspace_for(N, Hq / Hkv, D);
}

int sv_tree_attn(int dtype, const void* q, const void* k_pages, const void* v_pages,
                 const int32_t* block_table, const int32_t* seq_lens, const void* k_new,
                 const void* v_new, const int32_t* parent, float scale, int B, int N, int Hq,
                 int Hkv, int D, int num_pages, int LH, int head0, int page_size, int cols,
                 void* out, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                 void* stream) {
  if (dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_DTYPE;
  if (B < 0 || B > 65535 || N < 1 || N > MAX_N || bad_heads(Hq, Hkv, D) || num_pages < 1 ||
      LH < 1 || head0 < 0 || head0 > LH - Hkv || page_size < 8 || page_size > 65536 ||
      page_size % 8 != 0 || cols < 1 || (long long)B * LH > 0x7fffffffLL || bad_scale(scale))
    return SV_ERR_INVALID_ARG;
  if (B == 0) return SV_OK;
  if (!q || !k_pages || !v_pages || !block_table || !seq_lens || !k_new || !v_new || !out)
    return SV_ERR_INVALID_ARG;
  if (misaligned(q, 16) || misaligned(k_pages, 16) || misaligned(v_pages, 16) ||
      misaligned(k_new, 16) || misaligned(v_new, 16) || misaligned(out, 16) ||
      misaligned(block_table, 4) || misaligned(seq_lens, 4) || misaligned(parent, 4) ||
      misaligned(dev_status, 4))
    return SV_ERR_INVALID_ARG;
  if (!workspace || misaligned(workspace, 256) ||
      workspace_bytes < sv_attn_workspace_bytes(N, Hq, Hkv, D))
    return SV_ERR_WORKSPACE;
  AttnParams A = {};
  A.kind = TREE;
  A.table = block_table;
  A.lens = seq_lens;
  A.parent = parent;
  A.out = static_cast<uint16_t*>(out);
  A.status = dev_status;
  A.c = scale * LOG2E;
  A.B = B; A.N = N; A.Hq = Hq; A.Hkv = Hkv; A.D = D;
  A.LH = LH; A.head0 = head0; A.num_pages = num_pages; A.page = page_size; A.cols = cols;
  return launch(A, dtype, q, k_pages, v_pages, k_new, v_new, workspace, stream);
}

size_t sv_attn8_workspace_bytes(int B, int N, int Hq, int Hkv, int D) {
  if (B < 0 || B > 65535 || N < 1 || N > MAX_N || bad_heads(Hq, Hkv, D) || D % 16 != 0) return 0;
  return space_for8(requests_at_once(B, N, Hq, Hkv, D), N, Hq, Hkv, D).all;
}

int sv_tree_attn8(int dtype, const void* q, const void* k_pages, const void* v_pages,
                  const void* k_scales, const void* v_scales, const int32_t* block_table,
                  const int32_t* seq_lens, const void* k_new, const void* v_new,
                  const int32_t* parent, float scale, int B, int N, int Hq, int Hkv, int D,
                  int num_pages, int LH, int head0, int page_size, int block, int cols, void* out,
                  void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  if (dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_DTYPE;
  int block_log = 3;
  while (block_log < 7 && 1 << block_log != block) ++block_log;
  if (B < 0 || B > 65535 || N < 1 || N > MAX_N || bad_heads(Hq, Hkv, D) || D % 16 != 0 ||
      num_pages < 1 || LH < 1 || head0 < 0 || head0 > LH - Hkv || page_size < 8 ||
      page_size > 65536 || 1 << block_log != block || page_size % block != 0 || cols < 1 ||
      (long long)B * LH > 0x7fffffffLL || bad_scale(scale))
    return SV_ERR_INVALID_ARG;
  if (B == 0) return SV_OK;
  if (!q || !k_pages || !v_pages || !k_scales || !v_scales || !block_table || !seq_lens ||
      !k_new || !v_new || !out)
    return SV_ERR_INVALID_ARG;
  if (misaligned(q, 16) || misaligned(k_pages, 16) || misaligned(v_pages, 16) ||
      misaligned(k_new, 16) || misaligned(v_new, 16) || misaligned(out, 16) ||
      misaligned(block_table, 4) || misaligned(seq_lens, 4) || misaligned(parent, 4) ||
      misaligned(dev_status, 4))
    return SV_ERR_INVALID_ARG;
  if (!workspace || misaligned(workspace, 256) ||
      workspace_bytes < sv_attn8_workspace_bytes(B, N, Hq, Hkv, D))
    return SV_ERR_WORKSPACE;
  // parts of equal size, one after another
  const int most = requests_at_once(B, N, Hq, Hkv, D), parts = (B + most - 1) / most;
  for (int part = 0; part < parts; ++part) {
    const int b0 = int((long long)B * part / parts), b1 = int((long long)B * (part + 1) / parts);
    const size_t rows = size_t(b0) * N * Hq * D, staged = size_t(b0) * LH * N * D;
    AttnParams A = {};
    A.kind = TREE;
    A.table = block_table + size_t(b0) * cols;
    A.lens = seq_lens + b0;
    A.parent = parent ? parent + size_t(b0) * N : nullptr;
    A.out = static_cast<uint16_t*>(out) + rows;
    A.status = dev_status;
    A.k_scales = static_cast<const uint8_t*>(k_scales);
    A.v_scales = static_cast<const uint8_t*>(v_scales);
    A.block_log = block_log;
    A.c = scale * LOG2E;
    A.B = b1 - b0; A.N = N; A.Hq = Hq; A.Hkv = Hkv; A.D = D;
    A.LH = LH; A.head0 = head0; A.num_pages = num_pages; A.page = page_size; A.cols = cols;
    Prep8 P = {};
    P.q = static_cast<const uint16_t*>(q) + rows;
    P.k_new = static_cast<const uint16_t*>(k_new) + staged;
    P.B = A.B; P.N = N; P.Hq = Hq; P.Hkv = Hkv; P.D = D; P.LH = LH; P.head0 = head0;
    const int rc = launch(A, dtype, nullptr, k_pages, v_pages, nullptr,
                          static_cast<const uint16_t*>(v_new) + staged, workspace, stream, &P);
    if (rc != SV_OK) return rc;
  }
  return SV_OK;
}

int sv_ring_attn(int dtype, const void* q, const void* k_pool, const void* v_pool,
                 const int32_t* pos, const void* k_new, const void* v_new, float scale, int B,
                 int R, int Hq, int Hkv, int D, int LH, int head0, int sink, int window,
                 void* out, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                 void* stream) {
  if (dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_DTYPE;
  if (B < 0 || B > 65535 || R < 1 || R > MAX_R || bad_heads(Hq, Hkv, D) || LH < 1 || head0 < 0 ||
      head0 > LH - Hkv || (long long)B * LH > 0x7fffffffLL || sink < 0 || window < R ||
      (long long)sink + window > MAX_KEYS || bad_scale(scale))
    return SV_ERR_INVALID_ARG;
  if (B == 0) return SV_OK;
  if (!q || !k_pool || !v_pool || !pos || !k_new || !v_new || !out) return SV_ERR_INVALID_ARG;
  if (misaligned(q, 16) || misaligned(k_pool, 16) || misaligned(v_pool, 16) ||
      misaligned(k_new, 16) || misaligned(v_new, 16) || misaligned(out, 16) ||
      misaligned(pos, 4) || misaligned(dev_status, 4))
    return SV_ERR_INVALID_ARG;
  if (!workspace || misaligned(workspace, 256) ||
      workspace_bytes < sv_attn_workspace_bytes(R, Hq, Hkv, D))
    return SV_ERR_WORKSPACE;
  AttnParams A = {};
  A.kind = RING;
  A.lens = pos;
  A.out = static_cast<uint16_t*>(out);
  A.status = dev_status;
  A.c = scale * LOG2E;
  A.B = B; A.N = R; A.Hq = Hq; A.Hkv = Hkv; A.D = D;
  A.LH = LH; A.head0 = head0; A.sink = sink; A.window = window;
  return launch(A, dtype, q, k_pool, v_pool, k_new, v_new, workspace, stream);
}

int sv_prompt_attn(int dtype, const void* q, const void* k, const void* v,
                   const int32_t* cu_seqlens, float scale, int B, int T, int Hq, int Hkv, int D,
                   int sink, int window, void* out, int32_t* dev_status, void* stream) {
  if (dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_DTYPE;
  if (B < 0 || B > 65535 || T < 0 || T > 0x7fffffff - 511 || bad_heads(Hq, Hkv, D) || sink < 0 ||
      window < 1 || bad_scale(scale))
    return SV_ERR_INVALID_ARG;
  if (B == 0 || T == 0) return SV_OK;
  if (!q || !k || !v || !cu_seqlens || !out) return SV_ERR_INVALID_ARG;
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(out, 16) ||
      misaligned(cu_seqlens, 4) || misaligned(dev_status, 4))
    return SV_ERR_INVALID_ARG;
  AttnParams A = {};
  A.kind = PROMPT;
  A.lens = cu_seqlens;
  A.out = static_cast<uint16_t*>(out);
  A.status = dev_status;
  A.c = scale * LOG2E;
  A.B = B; A.T = T; A.Hq = Hq; A.Hkv = Hkv; A.D = D;
  A.sink = sink; A.window = window;
  return launch(A, dtype, q, k, v, nullptr, nullptr, nullptr, stream);
}

}  // extern "C"
