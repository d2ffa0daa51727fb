// attention.cu -- sm_103a kernels and C ABI of the attention over the caches
// (see include/svattn.h for the operations, layouts and error behaviour).

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "specverify.h"
#include "svattn.h"
#include "svkv.h"

namespace {

enum Kind { TREE = 0, RING = 1, PROMPT = 2 };

constexpr int MAX_N = 256;     // tree nodes
constexpr int MAX_R = 64;      // staged tokens of the ring call
constexpr int MAX_GROUP = 128; // query heads per KV head
constexpr int MAX_D = 128;

struct AttnParams {
  int kind, dtype;
  const uint16_t* q;
  const uint16_t* k;      // pages, pool or packed prompt
  const uint16_t* v;
  const uint16_t* k_new;  // staged entries (TREE, RING)
  const uint16_t* v_new;
  const int32_t* table;
  const int32_t* lens;    // seq_lens, pos or cu_seqlens
  const int32_t* parent;
  uint16_t* out;
  int32_t* status;
  float scale;
  int B, N, Hq, Hkv, D, G;
  int LH, head0, num_pages, page, cols, sink, window, T;
};

__device__ __forceinline__ void set_status(int32_t* status, int bits) {
  if (status && bits) atomicOr(status, bits);
}

__device__ __forceinline__ float load16(const uint16_t* p, int dtype) {
  const uint16_t x = __ldg(p);
  return dtype == SV_BF16 ? __uint_as_float(unsigned(x) << 16)
                          : __half2float(__ushort_as_half(x));
}
__device__ __forceinline__ uint16_t round16(float x, int dtype) {
  return dtype == SV_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x))
                          : __half_as_ushort(__float2half_rn(x));
}

// One warp per query row: the running maximum and sum of the softmax over the
// visible keys one after another, lane l holding dimensions 4 l .. 4 l + 3.
__global__ void __launch_bounds__(128) sv_attn_plain(const AttnParams A) {
  const int lane = int(threadIdx.x) & 31;
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const long long rows = A.kind == PROMPT ? (long long)A.T * A.Hq : (long long)A.B * A.N * A.Hq;
  if (row >= rows) return;
  const int h = int(row % A.Hq), kvh = h / A.G;
  const long long tok = row / A.Hq;
  int b, n;             // request and its node / token
  long long len, base = 0;  // cache entries; first packed row (PROMPT)
  int bad = 0;
  if (A.kind == PROMPT) {
    b = -1;
    for (int i = lane; i < A.B; i += 32) {
      const int lo = __ldg(A.lens + i), hi = __ldg(A.lens + i + 1);
      if (lo < 0 || hi < lo || hi > A.T) bad = SV_ST_BAD_LENGTH;
      else if (tok >= lo && tok < hi) b = i;
    }
    b = __reduce_max_sync(0xffffffffu, b);
    set_status(A.status, bad);
    bad = 0;  // other sequences' bounds
    if (b < 0) return;
    base = __ldg(A.lens + b);
    n = int(tok - base);
    len = n + 1;
  } else {
    b = int(tok / A.N);
    n = int(tok % A.N);
    len = __ldg(A.lens + b);
    if (len < 0 || (A.kind == TREE ? len > (long long)A.cols * A.page : len >= 0x7fffffffLL - A.N + 1))
      bad = SV_ST_BAD_LENGTH;
    if (A.kind == TREE && !bad) {
      if (A.parent)
        for (int i = lane; i < A.N; i += 32) {
          const int p = __ldg(A.parent + (size_t)b * A.N + i);
          if (i == 0 ? p != -1 : (p < 0 || p >= i)) bad |= SV_ST_BAD_TOKEN;
        }
      for (int c = lane; c < (len + A.page - 1) / A.page; c += 32) {
        const int p = __ldg(A.table + (size_t)b * A.cols + c);
        if (p < 0 || p >= A.num_pages) bad |= SV_ST_BAD_PAGE;
      }
      bad = __reduce_or_sync(0xffffffffu, bad);
    }
    set_status(A.status, lane == 0 ? bad : 0);
  }
  const int d0 = lane * 4;
  const bool has = d0 < A.D;
  float q[4] = {0, 0, 0, 0}, o[4] = {0, 0, 0, 0};
  if (has)
    for (int i = 0; i < 4; ++i) q[i] = load16(A.q + row * A.D + d0 + i, A.dtype);
  float m = -INFINITY, l = 0;
  auto take = [&](const uint16_t* kr, const uint16_t* vr) {
    float s = 0;
    if (has)
      for (int i = 0; i < 4; ++i) s += q[i] * load16(kr + d0 + i, A.dtype);
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= A.scale;
    const float m2 = fmaxf(m, s), f = __expf(m - m2), p = __expf(s - m2);
    l = l * f + p;
    if (has)
      for (int i = 0; i < 4; ++i) o[i] = o[i] * f + p * load16(vr + d0 + i, A.dtype);
    m = m2;
  };
  if (!bad && A.kind == PROMPT) {
    for (long long t = 0; t <= n; ++t) {
      if (t >= A.sink && t <= (long long)n - A.window) { t = (long long)n - A.window; continue; }
      const size_t r = ((size_t)(base + t) * A.Hkv + kvh) * A.D;
      take(A.k + r, A.v + r);
    }
  } else if (!bad) {
    if (A.kind == TREE) {
      for (long long t = 0; t < len; ++t) {
        const int p = __ldg(A.table + (size_t)b * A.cols + t / A.page);
        const size_t r = (((size_t)p * A.LH + A.head0 + kvh) * A.page + t % A.page) * A.D;
        take(A.k + r, A.v + r);
      }
    } else {
      const long long C = (long long)A.sink + A.window, lo = len + n - A.window;
      for (long long t = 0; t < len; ++t) {
        if (t >= A.sink && t <= lo) { t = lo; continue; }
        const long long slot = t < A.sink ? t : A.sink + (t - A.sink) % A.window;
        const size_t r = (((size_t)b * A.LH + A.head0 + kvh) * C + slot) * A.D;
        take(A.k + r, A.v + r);
      }
    }
    for (int i = n; i >= 0;) {
      const size_t r = (((size_t)b * A.LH + A.head0 + kvh) * A.N + i) * A.D;
      take(A.k_new + r, A.v_new + r);
      i = A.parent ? __ldg(A.parent + (size_t)b * A.N + i) : i - 1;
    }
  }
  if (has)
    for (int i = 0; i < 4; ++i)
      A.out[row * A.D + d0 + i] = bad ? 0 : round16(o[i] / l, A.dtype);
}

bool misaligned(const void* p, unsigned a) {
  return (reinterpret_cast<uintptr_t>(p) % a) != 0;
}

bool bad_heads(int Hq, int Hkv, int D) {
  return Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq / Hkv > MAX_GROUP || D < 8 || D > MAX_D ||
         D % 8 != 0;
}

int launch_plain(const AttnParams& A, void* stream) {
  const long long rows = A.kind == PROMPT ? (long long)A.T * A.Hq : (long long)A.B * A.N * A.Hq;
  sv_attn_plain<<<unsigned((rows + 3) / 4), 128, 0, static_cast<cudaStream_t>(stream)>>>(A);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t sv_attn_workspace_bytes(int N, int Hq, int Hkv, int D) {
  if (N < 1 || N > MAX_N || bad_heads(Hq, Hkv, D)) return 0;
  return 256;
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
      page_size % 8 != 0 || cols < 1 || !isfinite(scale) || !(scale > 0.0f))
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
  A.dtype = dtype;
  A.q = static_cast<const uint16_t*>(q);
  A.k = static_cast<const uint16_t*>(k_pages);
  A.v = static_cast<const uint16_t*>(v_pages);
  A.k_new = static_cast<const uint16_t*>(k_new);
  A.v_new = static_cast<const uint16_t*>(v_new);
  A.table = block_table;
  A.lens = seq_lens;
  A.parent = parent;
  A.out = static_cast<uint16_t*>(out);
  A.status = dev_status;
  A.scale = scale;
  A.B = B; A.N = N; A.Hq = Hq; A.Hkv = Hkv; A.D = D; A.G = Hq / Hkv;
  A.LH = LH; A.head0 = head0; A.num_pages = num_pages; A.page = page_size; A.cols = cols;
  return launch_plain(A, stream);
}

int sv_ring_attn(int dtype, const void* q, const void* k_pool, const void* v_pool,
                 const int32_t* pos, const void* k_new, const void* v_new, float scale, int B,
                 int R, int Hq, int Hkv, int D, int LH, int head0, int sink, int window,
                 void* out, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                 void* stream) {
  if (dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_DTYPE;
  if (B < 0 || B > 65535 || R < 1 || R > MAX_R || bad_heads(Hq, Hkv, D) || LH < 1 || head0 < 0 ||
      head0 > LH - Hkv || (long long)B * LH > 0x7fffffffLL || sink < 0 || window < R ||
      (long long)sink + window > 0x7fffffffLL || !isfinite(scale) || !(scale > 0.0f))
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
  A.dtype = dtype;
  A.q = static_cast<const uint16_t*>(q);
  A.k = static_cast<const uint16_t*>(k_pool);
  A.v = static_cast<const uint16_t*>(v_pool);
  A.k_new = static_cast<const uint16_t*>(k_new);
  A.v_new = static_cast<const uint16_t*>(v_new);
  A.lens = pos;
  A.out = static_cast<uint16_t*>(out);
  A.status = dev_status;
  A.scale = scale;
  A.B = B; A.N = R; A.Hq = Hq; A.Hkv = Hkv; A.D = D; A.G = Hq / Hkv;
  A.LH = LH; A.head0 = head0; A.sink = sink; A.window = window;
  return launch_plain(A, stream);
}

int sv_prompt_attn(int dtype, const void* q, const void* k, const void* v,
                   const int32_t* cu_seqlens, float scale, int B, int T, int Hq, int Hkv, int D,
                   int sink, int window, void* out, int32_t* dev_status, void* stream) {
  if (dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_DTYPE;
  if (B < 0 || B > 65535 || T < 0 || T > 0x7fffffff - 511 || bad_heads(Hq, Hkv, D) || sink < 0 ||
      window < 1 || !isfinite(scale) || !(scale > 0.0f))
    return SV_ERR_INVALID_ARG;
  if (B == 0 || T == 0) return SV_OK;
  if (!q || !k || !v || !cu_seqlens || !out) return SV_ERR_INVALID_ARG;
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(out, 16) ||
      misaligned(cu_seqlens, 4) || misaligned(dev_status, 4))
    return SV_ERR_INVALID_ARG;
  AttnParams A = {};
  A.kind = PROMPT;
  A.dtype = dtype;
  A.q = static_cast<const uint16_t*>(q);
  A.k = static_cast<const uint16_t*>(k);
  A.v = static_cast<const uint16_t*>(v);
  A.lens = cu_seqlens;
  A.out = static_cast<uint16_t*>(out);
  A.status = dev_status;
  A.scale = scale;
  A.B = B; A.T = T; A.Hq = Hq; A.Hkv = Hkv; A.D = D; A.G = Hq / Hkv;
  A.sink = sink; A.window = window;
  return launch_plain(A, stream);
}

}  // extern "C"
