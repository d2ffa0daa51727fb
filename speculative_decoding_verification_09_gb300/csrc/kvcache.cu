// kvcache.cu -- sm_103a kernels and C ABI of the KV-cache steps around
// verification (see include/svkv.h for the operations, layouts and error
// behaviour):
//
//   sv_kv_commit           copy kernel (one 2-D grid: request x span of the
//                          request's staged vectors) + position update
//   sv_kv_fill             one copy kernel (request x span of its kept vectors)
//   sv_page_commit         copy kernel (rows x entries x request), and a length
//                          update when the lengths are updated in place
//   sv_kv_valid_slots      one thread per (request, slot index)
//   sv_window_block_table  one thread per (request, clone column)
//
// The ring slot formula and the valid-slot order follow the deferred
// speculative decoding page, sections "环形上下文与注意力沉淀机制" and
// "C++ 环形 KV 缓存管理内核实现"; the window arithmetic follows the vllm-ascend
// draft KV sliding-window page, sections "窗口数学" and "block table 的裁剪方式".
//
// All are memory-bound gathers and scatters of whole 16-byte vectors (the
// commits and the fill) or of int32 words (the maps); the commits move only
// the accepted entries: rejected drafts are never written.

#include <cuda_runtime.h>
#include <stdint.h>

#include "specverify.h"
#include "svkv.h"

namespace {

constexpr int KV_THREADS = 256;
constexpr int KV_UNROLL = 4;     // 16-byte vectors in flight per thread
constexpr int KV_MAX_R = 64;     // staged entries per request
constexpr int KV_MAX_NVEC = 512; // 16-byte vectors per KV row (8 KB rows)
constexpr int MAP_THREADS = 128;

// n / d for 0 <= n < 2^31 and 1 <= d <= 512 as (n * ceil(2^40 / d)) >> 40: the
// multiplier's excess over 2^40 / d is below 1, so the product's excess over
// n * 2^40 / d stays below 2^31 / 2^40 <= 1 / d, less than the distance from
// n / d to the next integer.
unsigned long long div_magic(int d) { return ((1ull << 40) + unsigned(d) - 1) / unsigned(d); }
__device__ __forceinline__ int div_by(int n, unsigned long long m) {
  return int((unsigned long long)(unsigned)n * m >> 40);
}

__device__ __forceinline__ void allow_next_kernel() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_previous_kernel() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void set_status(int32_t* status, int bits) {
  if (status && bits) atomicOr(status, bits);
}

// Slot(pos) of a cache with `sink` persistent slots and a ring of `window`.
__device__ __host__ __forceinline__ long long ring_slot(long long pos, int sink, int window) {
  return pos < sink ? pos : sink + (pos - sink) % window;
}

struct KvParams {
  unsigned char* k_pool;
  unsigned char* v_pool;
  const unsigned char* k_new;
  const unsigned char* v_new;
  const int32_t* num_accepted;
  int32_t* pos;
  int32_t* status;
  int B, LH, R, nvec, sink, window;  // nvec: 16-byte vectors per row
  int per_req;                       // LH * R * nvec, staged vectors per request
  unsigned long long m_nvec, m_R;    // division multipliers (div_magic)
};

// Copy of the accepted entries.  Request b = blockIdx.y; the CTAs of a
// request stride over its staged vectors f = (lh * R + j) * nvec + q, which
// are contiguous in k_new / v_new; entry j <= k goes to row (b, lh) of the
// pools at slot Slot(pos + j).  KV_UNROLL vectors of K and of V per thread
// are loaded before any is stored.
__global__ void __launch_bounds__(KV_THREADS) sv_kv_copy(const KvParams K) {
  __shared__ int slot_of[KV_MAX_R];  // Slot(pos + j) of the committed entries
  allow_next_kernel();  // the position update waits for this grid's completion
  const int b = int(blockIdx.y);
  const int k = __ldg(K.num_accepted + b);
  const int p = __ldg(K.pos + b);
  if (k < 0 || k >= K.R || p < 0 || p > 0x7fffffff - K.R) return;  // dropped or invalid
  if (int(threadIdx.x) <= k)
    slot_of[threadIdx.x] = int(ring_slot((long long)p + threadIdx.x, K.sink, K.window));
  __syncthreads();
  const int C = K.sink + K.window;
  const uint4* kn = reinterpret_cast<const uint4*>(K.k_new) + size_t(b) * K.per_req;
  const uint4* vn = reinterpret_cast<const uint4*>(K.v_new) + size_t(b) * K.per_req;
  uint4* kp = reinterpret_cast<uint4*>(K.k_pool);
  uint4* vp = reinterpret_cast<uint4*>(K.v_pool);
  const int stride = int(gridDim.x) * KV_THREADS;
  for (int f0 = int(blockIdx.x) * KV_THREADS + int(threadIdx.x); f0 < K.per_req;
       f0 += stride * KV_UNROLL) {
    uint4 kv[KV_UNROLL], vv[KV_UNROLL];
    size_t dst[KV_UNROLL];
    bool use[KV_UNROLL];
#pragma unroll
    for (int u = 0; u < KV_UNROLL; ++u) {
      const int f = f0 + u * stride;
      const int row = div_by(f, K.m_nvec), q = f - row * K.nvec;
      const int lh = div_by(row, K.m_R), j = row - lh * K.R;
      use[u] = f < K.per_req && j <= k;
      dst[u] = use[u] ? ((size_t(b) * K.LH + lh) * C + size_t(slot_of[j])) * K.nvec + q : 0;
      if (use[u]) {
        kv[u] = __ldg(kn + f);
        vv[u] = __ldg(vn + f);
      }
    }
#pragma unroll
    for (int u = 0; u < KV_UNROLL; ++u) {
      if (use[u]) {
        kp[dst[u]] = kv[u];
        vp[dst[u]] = vv[u];
      }
    }
  }
}

// Position update after the copy: pos[b] += k + 1 for a committed request.
__global__ void __launch_bounds__(KV_THREADS) sv_kv_advance(const KvParams K) {
  const int b = int(blockIdx.x) * KV_THREADS + int(threadIdx.x);
  int k = 0, p = 0;
  if (b < K.B) {  // inputs of this call, read before the wait
    k = __ldg(K.num_accepted + b);
  }
  wait_previous_kernel();  // the copy kernel has read every position
  if (b >= K.B) return;
  p = K.pos[b];
  if (k >= K.R || p < 0 || p > 0x7fffffff - K.R) {  // the position would overflow
    set_status(K.status, SV_ST_BAD_LENGTH);
    return;
  }
  if (k >= 0) K.pos[b] = p + k + 1;
}

struct FillParams {
  const uint4* k;
  const uint4* v;
  const int32_t* cu;
  uint4* k_pool;
  uint4* v_pool;
  int32_t* pos;
  int32_t* status;
  int T, Hkv, LH, head0, nvec, sink, window;
  unsigned long long m_nvec;  // division multiplier of nvec
};

// Prompt entries to their ring slots.  Sequence b = blockIdx.y; its CTAs
// share the vectors f = (slot * Hkv + h) * nvec + q of the slots that a
// prompt of n tokens leaves filled.  Slot s holds position s below the sinks
// and the newest position on it above, so every slot is written once, and a
// token's heads are read as one contiguous run.
__global__ void __launch_bounds__(KV_THREADS) sv_kv_fill_copy(const FillParams K) {
  const int b = int(blockIdx.y);
  const long long lo = __ldg(K.cu + b), hi = __ldg(K.cu + b + 1);
  if (lo < 0 || hi < lo || hi > K.T) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_status(K.status, SV_ST_BAD_LENGTH);
    return;
  }
  const int n = int(hi - lo);
  if (blockIdx.x == 0 && threadIdx.x == 0) K.pos[b] = n;
  const long long C = (long long)K.sink + K.window;
  const int filled = n < C ? n : int(C);
  const int total = filled * K.Hkv * K.nvec;  // <= 2^30, checked on the host
  const int stride = int(gridDim.x) * KV_THREADS;  // KV_UNROLL strides cover every total
  const int f0 = int(blockIdx.x) * KV_THREADS + int(threadIdx.x);
  uint4 kv[KV_UNROLL], vv[KV_UNROLL];
  size_t dst[KV_UNROLL];
#pragma unroll
  for (int u = 0; u < KV_UNROLL; ++u) {
    const int f = f0 + u * stride;
    if (f >= total) break;
    const int row = div_by(f, K.m_nvec), q = f - row * K.nvec;
    const int slot = row / K.Hkv, h = row - slot * K.Hkv;
    int p = slot;
    if (slot >= K.sink) p += (n - 1 - slot) / K.window * K.window;
    const size_t src = (size_t(lo + p) * K.Hkv + h) * K.nvec + q;
    dst[u] = ((size_t(b) * K.LH + K.head0 + h) * size_t(C) + slot) * K.nvec + q;
    kv[u] = __ldg(K.k + src);
    vv[u] = __ldg(K.v + src);
  }
#pragma unroll
  for (int u = 0; u < KV_UNROLL; ++u) {
    if (f0 + u * stride >= total) break;
    K.k_pool[dst[u]] = kv[u];
    K.v_pool[dst[u]] = vv[u];
  }
}

constexpr int PC_ROWS = 16;     // layer/head rows per CTA
constexpr int PC_ENTRIES = 64;  // path entries per CTA and pass
constexpr int PC_SPANS = 64;    // CTAs along the entries

struct PageParams {
  uint4* k_pages;
  uint4* v_pages;
  const uint4* k_new;
  const uint4* v_new;
  const int32_t* table;
  const int32_t* seq_lens;
  const int32_t* nodes;
  const int32_t* num_accepted;
  int32_t* out_seq_lens;
  int32_t* status;
  int B, LH, N, nvec, num_pages, page, cols;
  unsigned long long m_nvec;
};

// The status bits of request b's commit of k + 1 entries at `len`, agreed on by
// the whole CTA (every CTA of the request finds the same).
__device__ int page_commit_faults(const PageParams& K, int b, int k, long long len) {
  int bad = 0;
  if (k >= K.N || len < 0 || len + k + 1 > (long long)K.cols * K.page ||
      len + k + 1 > 0x7fffffffLL) {
    bad = SV_ST_BAD_LENGTH;
  } else {
    if (K.nodes)
      for (int j = int(threadIdx.x); j < k; j += KV_THREADS) {
        const int n = __ldg(K.nodes + size_t(b) * K.N + j);
        if (n < 0 || n >= K.N) bad |= SV_ST_BAD_TOKEN;
      }
    const int c0 = int(len / K.page), c1 = int((len + k) / K.page);
    for (int c = c0 + int(threadIdx.x); c <= c1; c += KV_THREADS) {
      const int pg = __ldg(K.table + size_t(b) * K.cols + c);
      if (pg < 0 || pg >= K.num_pages) bad |= SV_ST_BAD_PAGE;
    }
  }
  const int tok = __syncthreads_or(bad & SV_ST_BAD_TOKEN);
  const int pg = __syncthreads_or(bad & SV_ST_BAD_PAGE);
  return (bad & SV_ST_BAD_LENGTH) | (tok ? SV_ST_BAD_TOKEN : 0) | (pg ? SV_ST_BAD_PAGE : 0);
}

// Path entries into pages: PC_ROWS rows x PC_ENTRIES entries of request
// blockIdx.y per CTA and pass (passes of gridDim.z spans), KV_UNROLL vectors of
// K and of V per thread loaded before any is stored.  IN_PLACE: the lengths
// are updated by the next kernel instead, after every CTA has read them.
template <bool IN_PLACE>
__global__ void __launch_bounds__(KV_THREADS) sv_page_copy(const PageParams K) {
  __shared__ size_t dst_of[PC_ENTRIES];  // first row of the entry's page position
  __shared__ int src_of[PC_ENTRIES];     // its staged entry
  if (IN_PLACE) allow_next_kernel();
  const int b = int(blockIdx.y);
  const int k = __ldg(K.num_accepted + b);
  const long long len = __ldg(K.seq_lens + b);
  const int first = int(blockIdx.z) * PC_ENTRIES;
  const bool writer = blockIdx.x == 0 && blockIdx.z == 0;
  if (!writer && first > k) return;
  // One pass holds every entry of a short path: then the thread of an entry checks
  // what it needs anyway, its node read beside the count and the length.  (One
  // path of 32 rows: 11.4 us with a check of its own, 9.4 so, launch included; 64
  // paths of 384 rows: 21.7 and 20.6.)
  const bool short_path = K.N <= PC_ENTRIES;
  int bad = 0;
  if (short_path) {
    const int j = int(threadIdx.x);
    const int node = K.nodes && j > 0 && j < K.N ? __ldg(K.nodes + size_t(b) * K.N + j - 1) : j;
    if (k >= K.N || len < 0 || len + k + 1 > (long long)K.cols * K.page ||
        len + k + 1 > 0x7fffffffLL) {
      bad = k < 0 ? 0 : SV_ST_BAD_LENGTH;
    } else if (j <= k) {
      const unsigned at = unsigned(len) + unsigned(j), col = at / unsigned(K.page);
      const int pg = __ldg(K.table + size_t(b) * K.cols + col);
      if (node < 0 || node >= K.N) bad |= SV_ST_BAD_TOKEN;
      if (pg < 0 || pg >= K.num_pages) bad |= SV_ST_BAD_PAGE;
      dst_of[j] = size_t(pg) * K.LH * K.page + (at - col * unsigned(K.page));
      src_of[j] = node;
    }
    const int tok = __syncthreads_or(bad & SV_ST_BAD_TOKEN);
    const int pg = __syncthreads_or(bad & SV_ST_BAD_PAGE);
    bad = (bad & SV_ST_BAD_LENGTH) | (tok ? SV_ST_BAD_TOKEN : 0) | (pg ? SV_ST_BAD_PAGE : 0);
  } else if (k >= 0) {
    bad = page_commit_faults(K, b, k, len);
  }
  if (writer && threadIdx.x == 0 && !IN_PLACE) {
    K.out_seq_lens[b] = int32_t(k < 0 || bad ? len : len + k + 1);
    set_status(K.status, bad);
  }
  if (k < 0 || bad) return;
  const int r0 = int(blockIdx.x) * PC_ROWS, rows = min(PC_ROWS, K.LH - r0);
  for (int j0 = first; j0 <= k; j0 += int(gridDim.z) * PC_ENTRIES) {
    const int cnt = min(PC_ENTRIES, k + 1 - j0);
    if (!short_path && int(threadIdx.x) < cnt) {
      const int j = j0 + int(threadIdx.x);
      const long long at = len + j;
      const int pg = __ldg(K.table + size_t(b) * K.cols + at / K.page);
      dst_of[threadIdx.x] = size_t(pg) * K.LH * K.page + size_t(at % K.page);
      src_of[threadIdx.x] = K.nodes && j > 0 ? __ldg(K.nodes + size_t(b) * K.N + j - 1) : j;
    }
    __syncthreads();
    const int total = cnt * PC_ROWS * K.nvec;  // <= 64 * 16 * 512
    for (int f0 = int(threadIdx.x); f0 < total; f0 += KV_THREADS * KV_UNROLL) {
      uint4 kv[KV_UNROLL], vv[KV_UNROLL];
      size_t dst[KV_UNROLL];
      bool use[KV_UNROLL];
#pragma unroll
      for (int u = 0; u < KV_UNROLL; ++u) {
        const int f = f0 + u * KV_THREADS;
        const int row = div_by(f, K.m_nvec), q = f - row * K.nvec;
        const int r = row % PC_ROWS, j = row / PC_ROWS;
        use[u] = f < total && r < rows;
        dst[u] = 0;
        if (use[u]) {
          const size_t src = ((size_t(b) * K.LH + r0 + r) * K.N + src_of[j]) * K.nvec + q;
          dst[u] = (dst_of[j] + size_t(r0 + r) * K.page) * K.nvec + q;
          kv[u] = __ldg(K.k_new + src);
          vv[u] = __ldg(K.v_new + src);
        }
      }
#pragma unroll
      for (int u = 0; u < KV_UNROLL; ++u) {
        if (use[u]) {
          K.k_pages[dst[u]] = kv[u];
          K.v_pages[dst[u]] = vv[u];
        }
      }
    }
    __syncthreads();  // the entries' places are used up
  }
}

// Lengths updated in place after the copy: one CTA per request, as its CTAs
// of the copy judged it.
__global__ void __launch_bounds__(KV_THREADS) sv_page_advance(const PageParams K) {
  const int b = int(blockIdx.x);
  wait_previous_kernel();
  const int k = __ldg(K.num_accepted + b);
  const long long len = K.seq_lens[b];
  if (k < 0) return;
  const int bad = page_commit_faults(K, b, k, len);
  if (threadIdx.x != 0) return;
  if (bad) set_status(K.status, bad);
  else K.out_seq_lens[b] = int32_t(len + k + 1);
}

// Valid slots of request blockIdx.y, entries j = blockIdx.x * MAP_THREADS + tid.
__global__ void __launch_bounds__(MAP_THREADS) sv_kv_slots(const int32_t* pos, int sink,
                                                           int window, int32_t* out_slots,
                                                           int32_t* out_len, int32_t* status) {
  const int b = int(blockIdx.y);
  const int C = sink + window;
  const int j = int(blockIdx.x) * MAP_THREADS + int(threadIdx.x);
  const long long p = __ldg(pos + b);
  const long long n = p < 0 ? 0 : (p < C ? p : C);
  if (j < C) {
    long long slot = -1;
    if (j < n) {
      if (p <= C) slot = j;
      else if (j < sink) slot = j;
      else slot = ring_slot(p - window + (j - sink), sink, window);
    }
    out_slots[size_t(b) * C + j] = int32_t(slot);
  }
  if (j == 0) {
    out_len[b] = int32_t(n);
    if (p < 0) set_status(status, SV_ST_BAD_LENGTH);
  }
}

// The window arithmetic of one sequence length: start block and the number
// of blocks the windowed length needs; false for a negative length.
__device__ __host__ __forceinline__ bool window_of(long long s, int W, int blk, int K,
                                                  long long& start, long long& needed) {
  if (s < 0) return false;
  long long lo = s + K - W;
  if (lo < 0) lo = 0;
  start = (lo / blk) * blk;
  needed = (s - start + blk - 1) / blk;
  return true;
}

// Clone column j = blockIdx.x * MAP_THREADS + tid of request blockIdx.y.
__global__ void __launch_bounds__(MAP_THREADS) sv_window_table(
    const int32_t* seq_lens, const int32_t* table, int full_cols, int W, int blk, int K,
    int cols, int32_t* out_seq, int32_t* out_table, int32_t* out_start_block, int32_t* status) {
  const int b = int(blockIdx.y);
  const int j = int(blockIdx.x) * MAP_THREADS + int(threadIdx.x);
  const long long s = __ldg(seq_lens + b);
  long long start = 0, needed = 0;
  const bool ok = window_of(s, W, blk, K, start, needed);
  const long long sb = start / blk;
  if (j < cols) {
    int32_t v = 0;
    const long long col = sb + j;
    if (ok && j < needed && col < full_cols) v = __ldg(table + size_t(b) * full_cols + col);
    out_table[size_t(b) * cols + j] = v;
  }
  if (j == 0) {
    out_seq[b] = ok ? int32_t(s - start) : 0;
    if (out_start_block) out_start_block[b] = ok ? int32_t(sb) : 0;
    if (!ok) set_status(status, SV_ST_BAD_LENGTH);
  }
}

int window_cols(int W, int blk) {
  if (W < 1 || blk < 1) return -1;
  const long long page = (long long)W / blk + 1;
  const long long bound = ((long long)W + 2LL * blk - 2) / blk;  // ceil((W + b - 1) / b)
  const long long c = page > bound ? page : bound;
  return c > 0x7fffffffLL ? -1 : int(c);
}

bool misaligned(const void* p, unsigned a) {
  return (reinterpret_cast<uintptr_t>(p) % a) != 0;
}

}  // namespace

extern "C" {

int sv_kv_commit(void* k_pool, void* v_pool, const void* k_new, const void* v_new,
                 const int32_t* num_accepted, int32_t* pos, int B, int LH, int R, int row_bytes,
                 int sink, int window, int32_t* dev_status, void* stream) {
  if (B < 0 || LH < 1 || R < 1 || R > KV_MAX_R || row_bytes < 16 || (row_bytes % 16) != 0 ||
      row_bytes / 16 > KV_MAX_NVEC || sink < 0 || window < R ||
      (long long)sink + window > 0x7fffffffLL)
    return SV_ERR_INVALID_ARG;
  if (B == 0) return SV_OK;
  if (!k_pool || !v_pool || !k_new || !v_new || !num_accepted || !pos) return SV_ERR_INVALID_ARG;
  if (misaligned(k_pool, 16) || misaligned(v_pool, 16) || misaligned(k_new, 16) ||
      misaligned(v_new, 16) || misaligned(num_accepted, 4) || misaligned(pos, 4) ||
      (dev_status && misaligned(dev_status, 4)))
    return SV_ERR_INVALID_ARG;
  const long long per_req = (long long)LH * R * (row_bytes / 16);
  if (per_req > (1LL << 30) || B > 65535) return SV_ERR_INVALID_ARG;  // int indexing inside
  KvParams K;
  K.k_pool = static_cast<unsigned char*>(k_pool);
  K.v_pool = static_cast<unsigned char*>(v_pool);
  K.k_new = static_cast<const unsigned char*>(k_new);
  K.v_new = static_cast<const unsigned char*>(v_new);
  K.num_accepted = num_accepted;
  K.pos = pos;
  K.status = dev_status;
  K.B = B; K.LH = LH; K.R = R; K.nvec = row_bytes / 16;
  K.sink = sink; K.window = window;
  K.per_req = int(per_req);
  K.m_nvec = div_magic(K.nvec);
  K.m_R = div_magic(R);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // CTAs per request: enough for KV_UNROLL vectors per thread per pass
  const long long per_cta = (long long)KV_THREADS * KV_UNROLL;
  const unsigned gx = unsigned((per_req + per_cta - 1) / per_cta);
  sv_kv_copy<<<dim3(gx, unsigned(B)), KV_THREADS, 0, st>>>(K);
  if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((B + KV_THREADS - 1) / KV_THREADS));
  cfg.blockDim = dim3(KV_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, sv_kv_advance, K) != cudaSuccess) return SV_ERR_CUDA;
  return SV_OK;
}

int sv_kv_fill(const void* k, const void* v, const int32_t* cu_seqlens, void* k_pool,
               void* v_pool, int32_t* pos, int B, int T, int Hkv, int LH, int head0,
               int row_bytes, int sink, int window, int32_t* dev_status, void* stream) {
  if (B < 0 || B > 65535 || T < 0 || Hkv < 1 || LH < 1 || head0 < 0 || head0 > LH - Hkv ||
      row_bytes < 16 || (row_bytes % 16) != 0 || row_bytes / 16 > KV_MAX_NVEC || sink < 0 ||
      window < 1 || (long long)sink + window > 0x7fffffffLL)
    return SV_ERR_INVALID_ARG;
  if (B == 0) return SV_OK;
  if (!cu_seqlens || !k_pool || !v_pool || !pos || (T > 0 && (!k || !v)))
    return SV_ERR_INVALID_ARG;
  if (misaligned(k_pool, 16) || misaligned(v_pool, 16) || misaligned(k, 16) ||
      misaligned(v, 16) || misaligned(cu_seqlens, 4) || misaligned(pos, 4) ||
      (dev_status && misaligned(dev_status, 4)))
    return SV_ERR_INVALID_ARG;
  const long long C = (long long)sink + window;
  const long long slots = T < C ? T : C;
  const int nvec = row_bytes / 16;
  if (slots * Hkv > (1LL << 30) / nvec) return SV_ERR_INVALID_ARG;  // int indexing inside
  const long long most = slots * Hkv * nvec;
  FillParams K;
  K.k = static_cast<const uint4*>(k);
  K.v = static_cast<const uint4*>(v);
  K.cu = cu_seqlens;
  K.k_pool = static_cast<uint4*>(k_pool);
  K.v_pool = static_cast<uint4*>(v_pool);
  K.pos = pos;
  K.status = dev_status;
  K.T = T; K.Hkv = Hkv; K.LH = LH; K.head0 = head0; K.nvec = nvec;
  K.sink = sink; K.window = window;
  K.m_nvec = div_magic(nvec);
  const long long per_cta = (long long)KV_THREADS * KV_UNROLL;
  const unsigned gx = unsigned(most > per_cta ? (most + per_cta - 1) / per_cta : 1);
  sv_kv_fill_copy<<<dim3(gx, unsigned(B)), KV_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(K);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

int sv_page_commit(void* k_pages, void* v_pages, const void* k_new, const void* v_new,
                   const int32_t* block_table, const int32_t* seq_lens, const int32_t* nodes,
                   const int32_t* num_accepted, int B, int LH, int N, int row_bytes,
                   int num_pages, int page_size, int cols, int32_t* out_seq_lens,
                   int32_t* dev_status, void* stream) {
  if (B < 0 || B > 65535 || LH < 1 || N < 1 || N > (1 << 20) || row_bytes < 16 ||
      (row_bytes % 16) != 0 || row_bytes / 16 > KV_MAX_NVEC || num_pages < 1 || page_size < 1 ||
      cols < 1)
    return SV_ERR_INVALID_ARG;
  if (B == 0) return SV_OK;
  if (!k_pages || !v_pages || !k_new || !v_new || !block_table || !seq_lens || !num_accepted ||
      !out_seq_lens)
    return SV_ERR_INVALID_ARG;
  if (misaligned(k_pages, 16) || misaligned(v_pages, 16) || misaligned(k_new, 16) ||
      misaligned(v_new, 16) || misaligned(block_table, 4) || misaligned(seq_lens, 4) ||
      misaligned(nodes, 4) || misaligned(num_accepted, 4) || misaligned(out_seq_lens, 4) ||
      (dev_status && misaligned(dev_status, 4)))
    return SV_ERR_INVALID_ARG;
  const bool in_place = out_seq_lens == seq_lens;
  if (!in_place && out_seq_lens < seq_lens + B && seq_lens < out_seq_lens + B)
    return SV_ERR_INVALID_ARG;  // shifted against each other: neither in place nor apart
  const long long gx = ((long long)LH + PC_ROWS - 1) / PC_ROWS;
  PageParams K;
  K.k_pages = static_cast<uint4*>(k_pages);
  K.v_pages = static_cast<uint4*>(v_pages);
  K.k_new = static_cast<const uint4*>(k_new);
  K.v_new = static_cast<const uint4*>(v_new);
  K.table = block_table;
  K.seq_lens = seq_lens;
  K.nodes = nodes;
  K.num_accepted = num_accepted;
  K.out_seq_lens = out_seq_lens;
  K.status = dev_status;
  K.B = B; K.LH = LH; K.N = N; K.nvec = row_bytes / 16;
  K.num_pages = num_pages; K.page = page_size; K.cols = cols;
  K.m_nvec = div_magic(K.nvec);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int spans = (N + PC_ENTRIES - 1) / PC_ENTRIES;
  const dim3 grid(unsigned(gx), unsigned(B), unsigned(spans < PC_SPANS ? spans : PC_SPANS));
  if (!in_place) {
    sv_page_copy<false><<<grid, KV_THREADS, 0, st>>>(K);
    return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
  }
  sv_page_copy<true><<<grid, KV_THREADS, 0, st>>>(K);
  if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(B));
  cfg.blockDim = dim3(KV_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sv_page_advance, K) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

int sv_kv_valid_slots(const int32_t* pos, int B, int sink, int window, int32_t* out_slots,
                      int32_t* out_len, int32_t* dev_status, void* stream) {
  if (B < 0 || sink < 0 || window < 1 || (long long)sink + window > 0x7fffffffLL)
    return SV_ERR_INVALID_ARG;
  if (B == 0) return SV_OK;
  if (!pos || !out_slots || !out_len || B > 65535) return SV_ERR_INVALID_ARG;
  if (misaligned(pos, 4) || misaligned(out_slots, 4) || misaligned(out_len, 4) ||
      (dev_status && misaligned(dev_status, 4)))
    return SV_ERR_INVALID_ARG;
  const int C = sink + window;
  sv_kv_slots<<<dim3(unsigned((C + MAP_THREADS - 1) / MAP_THREADS), unsigned(B)), MAP_THREADS,
                 0, static_cast<cudaStream_t>(stream)>>>(pos, sink, window, out_slots, out_len,
                                                         dev_status);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

int sv_window_cols(int window, int block_size) { return window_cols(window, block_size); }

int sv_window_block_table(const int32_t* seq_lens, const int32_t* block_table, int B,
                          int full_cols, int window, int block_size, int future_offset,
                          int32_t* out_seq_lens, int32_t* out_block_table,
                          int32_t* out_start_block, int32_t* dev_status, void* stream) {
  const int cols = window_cols(window, block_size);
  if (B < 0 || full_cols < 1 || cols < 1 || future_offset < 0) return SV_ERR_INVALID_ARG;
  if (B == 0) return SV_OK;
  if (!seq_lens || !block_table || !out_seq_lens || !out_block_table || B > 65535)
    return SV_ERR_INVALID_ARG;
  if (misaligned(seq_lens, 4) || misaligned(block_table, 4) || misaligned(out_seq_lens, 4) ||
      misaligned(out_block_table, 4) || (out_start_block && misaligned(out_start_block, 4)) ||
      (dev_status && misaligned(dev_status, 4)))
    return SV_ERR_INVALID_ARG;
  sv_window_table<<<dim3(unsigned((cols + MAP_THREADS - 1) / MAP_THREADS), unsigned(B)),
                    MAP_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(
      seq_lens, block_table, full_cols, window, block_size, future_offset, cols, out_seq_lens,
      out_block_table, out_start_block, dev_status);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

int sv_window_seq_lens_host(const int32_t* seq_lens, int n, int window, int block_size,
                            int future_offset, int32_t* out) {
  if (n < 0 || window < 1 || block_size < 1 || future_offset < 0) return SV_ERR_INVALID_ARG;
  if (n > 0 && (!seq_lens || !out)) return SV_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    long long start = 0, needed = 0;
    const long long s = seq_lens[i];
    out[i] = window_of(s, window, block_size, future_offset, start, needed) ? int32_t(s - start)
                                                                            : 0;
  }
  return SV_OK;
}

}  // extern "C"
