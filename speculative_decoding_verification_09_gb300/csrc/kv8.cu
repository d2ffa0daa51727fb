// kv8.cu -- sm_103a kernels and C ABI of writing the 8-bit paged cache (see
// include/svkv8.h for the operations, layouts and errors):
//
//   sv_kv8_append   packed tokens, keys rotated on the way
//   sv_kv8_commit   a verified path's staged entries
//   sv_kv8_advance  lengths of a commit that are updated in place
//
// A unit is the new entries of one block of tokens and one row: they share a
// scale, so all of them have to be seen before any is stored.  A CTA holds a unit in
// registers, sixteen dimensions of a token's key and of its value per thread, finds
// both largest sizes, and rounds.  Every byte is moved once (a block's older entries
// only when its scale rises); what bounds it is HBM for prompts, and for single
// tokens the latency of the loads that depend on one another: bounds, length, page,
// scale.

#include "rope.cuh"
#include "svkv8.h"

namespace {

using namespace svrope;

constexpr int MAX_UNIT_THREADS = 1024;  // 128 tokens of 128 dimensions

__device__ __forceinline__ void allow_next_kernel() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_previous_kernel() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// 2^e, from -126 on; a factor that small leaves nothing of an 8-bit value.
__device__ __forceinline__ float power(int e) { return __int_as_float((max(e, -126) + 127) << 23); }

// The smallest e with a <= 448 * 2^e = 1.75 * 2^(e + 8), for finite a >= 0, in [least, most].
__device__ __forceinline__ int exponent_for(float a, int least, int most) {
  const int x = __float_as_int(a);
  const int e = (x >> 23) - 127 - 8 + ((x & 0x7fffff) > 0x600000);
  return min(max(e, least), most);  // (zero and subnormal sizes: below every `least`)
}

// Four values to e4m3: nearest even, at most 448 in size, NaN kept.
__device__ __forceinline__ uint32_t to_bytes(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return uint32_t(lo) | uint32_t(hi) << 16;
}
// Four e4m3 values times f, rounded again.
__device__ __forceinline__ uint32_t again(uint32_t w, float f) {
  float2 v[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(w >> (16 * i))));
    v[i] = widen<false>(h);
  }
  return to_bytes(v[0].x * f, v[0].y * f, v[1].x * f, v[1].y * f);
}

// What is not finite becomes NaN; the largest size of the rest, as bits.
__device__ __forceinline__ uint32_t largest(float (&x)[8], uint32_t most) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = __float_as_uint(x[i]) & 0x7fffffffu;
    if (a >= 0x7f800000u) x[i] = __int_as_float(0x7fffffff);
    else most = max(most, a);
  }
  return most;
}

struct Pools {
  unsigned char* k_pages;
  unsigned char* v_pages;
  unsigned char* k_scales;
  unsigned char* v_scales;
  int LH, page, block, D;
  int least, most;  // exponents
  int chunks;       // D / 16
};

// The unit of one CTA: new entries in rows `off` .. off + count - 1 of the block of `page`
// (a valid one) that begins at its row `at`, row `row` of LH.  `src` gives the thread's
// entry of the block: pointers to its key and value, and the row of angles (or null).
template <bool BF, class Source>
__device__ __forceinline__ void write_unit(const Pools& P, int page, int row, int at, int off,
                                           int count, int rot, bool inter, const Source& src) {
  __shared__ uint32_t most_of[2][MAX_UNIT_THREADS / 32];
  const int tid = int(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int r = tid / P.chunks, c = tid - r * P.chunks;
  const bool mine = r >= off && r < off + count, older = r < off;
  const size_t line = (size_t(page) * P.LH + row) * P.page + at;  // the block's first token
  const size_t scale_at = line / P.block;
  int own_k = -1000, own_v = -1000;  // the block's exponents, when it holds entries
  if (off) {
    own_k = int(P.k_scales[scale_at]) - 127;
    own_v = int(P.v_scales[scale_at]) - 127;
  }
  const bool vec = rot % 16 == 0, turned = 8 * c < rot / 2;
  const int d0 = vec && turned && !inter ? 8 * c : 16 * c;
  const int d1 = vec && turned && !inter ? d0 + rot / 2 : d0 + 8;
  float ka[8], kb[8], va[8], vb[8];
  if (mine) {
    const uint16_t *k, *v;
    const float* angles;
    src(r - off, k, v, angles);
    uint4 u, w;
    if (vec) {
      u = *reinterpret_cast<const uint4*>(k + d0);
      w = *reinterpret_cast<const uint4*>(k + d1);
    }
    const uint4 x = *reinterpret_cast<const uint4*>(v + 16 * c);
    const uint4 y = *reinterpret_cast<const uint4*>(v + 16 * c + 8);
    if (vec) {
      split<BF>(u, w, inter || !turned, ka, kb);
      if (turned) turn8(ka, kb, angles, rot, c);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int pair = 8 * c + e;
        ka[e] = widen1<BF>(k[first_of(pair, rot, inter)]);
        kb[e] = widen1<BF>(k[second_of(pair, rot, inter)]);
        if (pair < rot / 2) turn(ka[e], kb[e], __ldg(angles + pair), __ldg(angles + rot / 2 + pair));
      }
    }
    split<BF>(x, y, true, va, vb);
  }
  uint32_t mk = 0, mv = 0;
  if (mine) {
    mk = largest(kb, largest(ka, 0));
    mv = largest(vb, largest(va, 0));
  }
  mk = __reduce_max_sync(0xffffffffu, mk);
  mv = __reduce_max_sync(0xffffffffu, mv);
  if (lane == 0) {
    most_of[0][warp] = mk;
    most_of[1][warp] = mv;
  }
  __syncthreads();
  const int warps = int(blockDim.x) >> 5;
  mk = __reduce_max_sync(0xffffffffu, lane < warps ? most_of[0][lane] : 0);
  mv = __reduce_max_sync(0xffffffffu, lane < warps ? most_of[1][lane] : 0);
  __syncthreads();  // (before the next unit's)
  const int ek = max(exponent_for(__uint_as_float(mk), P.least, P.most), own_k);
  const int ev = max(exponent_for(__uint_as_float(mv), P.least, P.most), own_v);
  unsigned char* const kp = P.k_pages + (line + r) * P.D;
  unsigned char* const vp = P.v_pages + (line + r) * P.D;
  if (mine) {
    const float fk = power(-ek), fv = power(-ev);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      ka[e] *= fk;
      kb[e] *= fk;
      va[e] *= fv;
      vb[e] *= fv;
    }
    if (vec && turned && !inter) {
      *reinterpret_cast<uint2*>(kp + d0) =
          make_uint2(to_bytes(ka[0], ka[1], ka[2], ka[3]), to_bytes(ka[4], ka[5], ka[6], ka[7]));
      *reinterpret_cast<uint2*>(kp + d1) =
          make_uint2(to_bytes(kb[0], kb[1], kb[2], kb[3]), to_bytes(kb[4], kb[5], kb[6], kb[7]));
    } else if (vec) {
      *reinterpret_cast<uint4*>(kp + 16 * c) =
          make_uint4(to_bytes(ka[0], kb[0], ka[1], kb[1]), to_bytes(ka[2], kb[2], ka[3], kb[3]),
                     to_bytes(ka[4], kb[4], ka[5], kb[5]), to_bytes(ka[6], kb[6], ka[7], kb[7]));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int pair = 8 * c + e;
        const uint32_t w = to_bytes(ka[e], kb[e], 0.0f, 0.0f);
        kp[first_of(pair, rot, inter)] = uint8_t(w);
        kp[second_of(pair, rot, inter)] = uint8_t(w >> 8);
      }
    }
    *reinterpret_cast<uint4*>(vp + 16 * c) =
        make_uint4(to_bytes(va[0], vb[0], va[1], vb[1]), to_bytes(va[2], vb[2], va[3], vb[3]),
                   to_bytes(va[4], vb[4], va[5], vb[5]), to_bytes(va[6], vb[6], va[7], vb[7]));
  } else if (older) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int by = i ? own_v - ev : own_k - ek;
      uint4* const p = reinterpret_cast<uint4*>((i ? vp : kp) + 16 * c);
      if (by < 0) {
        const float f = power(by);
        const uint4 w = *p;
        *p = make_uint4(again(w.x, f), again(w.y, f), again(w.z, f), again(w.w, f));
      }
    }
  }
  if (tid == 0) {
    P.k_scales[scale_at] = uint8_t(ek + 127);
    P.v_scales[scale_at] = uint8_t(ev + 127);
  }
}

// -------------------------------------------------------------- packed tokens

struct AppendParams {
  Appended A;
  Pools P;
  const uint16_t* k;
  const uint16_t* v;
  const float* angles;
  long long ks, vs;
  int Hkv, head0, rot;
  int tokens;      // per CTA, whose units are those that begin among them
  int token_ctas;  // CTAs behind them settle the requests (of head 0)
  bool inter;
};

template <bool BF>
__global__ void __launch_bounds__(MAX_UNIT_THREADS) sv_kv8_append(
    const __grid_constant__ AppendParams R) {
  const Appended& A = R.A;
  const int tid = int(threadIdx.x), h = int(blockIdx.y);
  if (int(blockIdx.x) >= R.token_ctas) {
    const int warps = int(blockDim.x) >> 5;
    const int b = (int(blockIdx.x) - R.token_ctas) * warps + (tid >> 5);
    if (h == 0 && b < A.B) settle(A, b);
    return;
  }
  const int t0 = int(blockIdx.x) * R.tokens, t1 = min(t0 + R.tokens, A.T);
  const int r = tid / R.P.chunks;
  for (int t = t0; t < t1;) {
    int b, lo, hi;
    if (!request_of(A, t, b, lo, hi)) {  // no request's row: the next one may be
      ++t;
      continue;
    }
    const int len = __ldg(A.lens + b), n = hi - lo;
    if (!fits(A, len, n)) {
      t = hi;
      continue;
    }
    // the first unit that begins at t or behind it
    int j = t - lo;
    const int into = (len + j) % R.P.block;
    if (j > 0 && into) j += R.P.block - into;
    if (j >= n || lo + j >= t1) {
      t = j >= n ? hi : t1;
      continue;
    }
    const int at = len + j, off = at % R.P.block, count = min(R.P.block - off, n - j);
    t = lo + j + count;
    const int col = at / A.page;
    const int pg = __ldg(A.table + size_t(b) * A.cols + col);
    bool ok = pg >= 0 && pg < A.num_pages;
    if (off) {  // a block that holds entries stays as it is unless all of the request is right
      ok = !__syncthreads_or(faults_of(A, b, lo, n, len, tid, int(blockDim.x)));
    } else if (A.rows) {
      int p = 0;
      if (r < count) p = A.positions ? __ldg(A.positions + lo + j + r) : at + r;
      ok = !__syncthreads_or(p < 0 || p >= A.rows) && ok;
    }
    if (!ok) continue;
    write_unit<BF>(R.P, pg, R.head0 + h, at - off - col * A.page, off, count, R.rot, R.inter,
                   [&](int i, const uint16_t*& k, const uint16_t*& v, const float*& angles) {
                     const long long token = lo + j + i;
                     k = R.k + token * R.ks + (long long)h * R.P.D;
                     v = R.v + token * R.vs + (long long)h * R.P.D;
                     const int p = A.rows && A.positions ? __ldg(A.positions + token) : at + i;
                     angles = R.angles + (long long)(A.rows ? p : 0) * R.rot;
                   });
  }
}

// -------------------------------------------------------------- verified paths

struct CommitParams {
  Pools P;
  const uint16_t* k_new;
  const uint16_t* v_new;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* nodes;
  const int32_t* num_accepted;
  int32_t* out_lens;
  int32_t* status;
  int B, N, num_pages, cols;
};

// The status bits of request b's commit of k + 1 entries at `len`, agreed on by the CTA.
__device__ __forceinline__ int commit_faults(const CommitParams& R, int b, int k, int len) {
  int bad = 0;
  if (k >= R.N || len < 0 || (long long)len + k + 1 > (long long)R.cols * R.P.page ||
      (long long)len + k + 1 > 0x7fffffffLL) {
    bad = SV_ST_BAD_LENGTH;
  } else {
    if (R.nodes)
      for (int j = int(threadIdx.x); j < k; j += int(blockDim.x)) {
        const int n = __ldg(R.nodes + size_t(b) * R.N + j);
        if (n < 0 || n >= R.N) bad |= SV_ST_BAD_TOKEN;
      }
    const int c0 = len / R.P.page, c1 = (len + k) / R.P.page;
    for (int c = c0 + int(threadIdx.x); c <= c1; c += int(blockDim.x)) {
      const int pg = __ldg(R.table + size_t(b) * R.cols + c);
      if (pg < 0 || pg >= R.num_pages) bad |= SV_ST_BAD_PAGE;
    }
  }
  const int tok = __syncthreads_or(bad & SV_ST_BAD_TOKEN);
  const int pg = __syncthreads_or(bad & SV_ST_BAD_PAGE);
  return (bad & SV_ST_BAD_LENGTH) | (tok ? SV_ST_BAD_TOKEN : 0) | (pg ? SV_ST_BAD_PAGE : 0);
}

// Unit blockIdx.y (and every gridDim.y-th from there) of the path of request blockIdx.z, row
// blockIdx.x.  IN_PLACE: the lengths are updated by the next kernel instead.
template <bool BF, bool IN_PLACE>
__global__ void __launch_bounds__(MAX_UNIT_THREADS) sv_kv8_commit(
    const __grid_constant__ CommitParams R) {
  if (IN_PLACE) allow_next_kernel();
  const int b = int(blockIdx.z), row = int(blockIdx.x);
  const int k = __ldg(R.num_accepted + b), len = __ldg(R.lens + b);
  const int block = R.P.block;
  const bool writer = row == 0 && blockIdx.y == 0;
  // (entries of the units before this CTA's first)
  const long long before =
      blockIdx.y == 0 || len < 0 ? 0 : (long long)blockIdx.y * block - len % block;
  if (!writer && before > k) return;
  const int bad = k >= 0 ? commit_faults(R, b, k, len) : 0;
  if (writer && threadIdx.x == 0 && !IN_PLACE) {
    R.out_lens[b] = k < 0 || bad ? len : len + k + 1;
    set_status(R.status, bad);
  }
  if (k < 0 || bad) return;
  for (long long j0 = before; j0 <= k; j0 += (long long)gridDim.y * block - (j0 ? 0 : len % block)) {
    const int j = int(j0), at = len + j, off = at % block;
    const int count = min(block - off, k + 1 - j), col = at / R.P.page;
    const int pg = __ldg(R.table + size_t(b) * R.cols + col);
    write_unit<BF>(R.P, pg, row, at - off - col * R.P.page, off, count, 0, false,
                   [&](int i, const uint16_t*& kp, const uint16_t*& vp, const float*& angles) {
                     const int e = j + i;
                     const int node =
                         R.nodes && e > 0 ? __ldg(R.nodes + size_t(b) * R.N + e - 1) : e;
                     const size_t from = ((size_t(b) * R.P.LH + row) * R.N + node) * R.P.D;
                     kp = R.k_new + from;
                     vp = R.v_new + from;
                     angles = nullptr;
                   });
  }
}

// Lengths updated in place after the commit: one CTA per request, as its CTAs judged it.
__global__ void __launch_bounds__(128) sv_kv8_advance(const __grid_constant__ CommitParams R) {
  const int b = int(blockIdx.x);
  wait_previous_kernel();
  const int k = __ldg(R.num_accepted + b), len = R.lens[b];
  if (k < 0) return;
  const int bad = commit_faults(R, b, k, len);
  if (threadIdx.x != 0) return;
  if (bad) set_status(R.status, bad);
  else R.out_lens[b] = len + k + 1;
}

bool bad_pools(int D, int page_size, int block) {
  return D < 16 || D > 128 || D % 16 != 0 ||
         (block != 8 && block != 16 && block != 32 && block != 64 && block != 128) ||
         page_size < 1 || page_size % block != 0;
}
void set_pools(Pools& P, int dtype, void* kp, void* vp, void* ks, void* vs, int LH, int page,
               int block, int D) {
  P.k_pages = static_cast<unsigned char*>(kp);
  P.v_pages = static_cast<unsigned char*>(vp);
  P.k_scales = static_cast<unsigned char*>(ks);
  P.v_scales = static_cast<unsigned char*>(vs);
  P.LH = LH; P.page = page; P.block = block; P.D = D;
  P.least = dtype == SV_BF16 ? -117 : -15;
  P.most = dtype == SV_BF16 ? 119 : 7;
  P.chunks = D / 16;
}
int unit_threads(const Pools& P) { return (P.block * P.chunks + 31) / 32 * 32; }

}  // namespace

extern "C" {

int sv_page_append8(int dtype, const void* k, long long k_stride, const void* v,
                    long long v_stride, void* k_pages, void* v_pages, void* k_scales,
                    void* v_scales, const int32_t* block_table, const int32_t* seq_lens,
                    const int32_t* cu_seqlens, const float* table, int rows, int rot,
                    int interleaved, const int32_t* positions, int B, int T, int Hkv, int D,
                    int num_pages, int LH, int head0, int page_size, int block, int cols,
                    int32_t* out_seq_lens, int32_t* dev_status, void* stream) {
  if (dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_DTYPE;
  if (B < 0 || B > 65535 || T < 0 || Hkv < 1 || Hkv > 65535 || bad_pools(D, page_size, block) ||
      bad_rotation(table, rows, rot, D) || num_pages < 1 || LH < 1 || head0 < 0 ||
      head0 > LH - Hkv || cols < 1 || bad_stride(k_stride, Hkv, D) || bad_stride(v_stride, Hkv, D))
    return SV_ERR_INVALID_ARG;
  if (B == 0) return SV_OK;
  if (!k_pages || !v_pages || !k_scales || !v_scales || !block_table || !seq_lens ||
      !cu_seqlens || (T > 0 && (!k || !v)))
    return SV_ERR_INVALID_ARG;
  if (misaligned(k, 16) || misaligned(v, 16) || misaligned(k_pages, 16) ||
      misaligned(v_pages, 16) || misaligned(block_table, 4) || misaligned(seq_lens, 4) ||
      misaligned(cu_seqlens, 4) || misaligned(positions, 4) || misaligned(out_seq_lens, 4) ||
      misaligned(dev_status, 4))
    return SV_ERR_INVALID_ARG;
  if (out_seq_lens && out_seq_lens < seq_lens + B && seq_lens < out_seq_lens + B)
    return SV_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    return SV_ERR_CUDA;
  AppendParams R = {};
  R.A = {block_table, seq_lens, cu_seqlens, positions, out_seq_lens, dev_status,
         B, T, cols, page_size, num_pages, table ? rows : 0};
  set_pools(R.P, dtype, k_pages, v_pages, k_scales, v_scales, LH, page_size, block, D);
  R.k = static_cast<const uint16_t*>(k);
  R.v = static_cast<const uint16_t*>(v);
  R.angles = table;
  R.ks = k_stride; R.vs = v_stride;
  R.Hkv = Hkv; R.head0 = head0; R.rot = table ? rot : 0;
  R.inter = interleaved != 0;
  const int threads = unit_threads(R.P);
  // A CTA per token when that is a few CTAs per SM (single tokens: every unit at once), else
  // one per block's worth of tokens (a prompt's CTAs have one unit each).
  R.tokens = (long long)T * Hkv <= 16LL * sms ? 1 : block;
  R.token_ctas = int(((long long)T + R.tokens - 1) / R.tokens);
  const long long grid = R.token_ctas + ((long long)B + threads / 32 - 1) / (threads / 32);
  if (grid > 0x7fffffffLL) return SV_ERR_INVALID_ARG;
  const dim3 g(static_cast<unsigned>(grid), static_cast<unsigned>(Hkv));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == SV_BF16) sv_kv8_append<true><<<g, threads, 0, st>>>(R);
  else sv_kv8_append<false><<<g, threads, 0, st>>>(R);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

int sv_page_commit8(int dtype, void* k_pages, void* v_pages, void* k_scales, void* v_scales,
                    const void* k_new, const void* v_new, const int32_t* block_table,
                    const int32_t* seq_lens, const int32_t* nodes, const int32_t* num_accepted,
                    int B, int LH, int N, int D, int num_pages, int page_size, int block, int cols,
                    int32_t* out_seq_lens, int32_t* dev_status, void* stream) {
  if (dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_DTYPE;
  if (B < 0 || B > 65535 || LH < 1 || N < 1 || N > (1 << 20) || bad_pools(D, page_size, block) ||
      num_pages < 1 || cols < 1)
    return SV_ERR_INVALID_ARG;
  if (B == 0) return SV_OK;
  if (!k_pages || !v_pages || !k_scales || !v_scales || !k_new || !v_new || !block_table ||
      !seq_lens || !num_accepted || !out_seq_lens)
    return SV_ERR_INVALID_ARG;
  if (misaligned(k_pages, 16) || misaligned(v_pages, 16) || misaligned(k_new, 16) ||
      misaligned(v_new, 16) || misaligned(block_table, 4) || misaligned(seq_lens, 4) ||
      misaligned(nodes, 4) || misaligned(num_accepted, 4) || misaligned(out_seq_lens, 4) ||
      misaligned(dev_status, 4))
    return SV_ERR_INVALID_ARG;
  const bool in_place = out_seq_lens == seq_lens;
  if (!in_place && out_seq_lens < seq_lens + B && seq_lens < out_seq_lens + B)
    return SV_ERR_INVALID_ARG;  // shifted against each other: neither in place nor apart
  CommitParams R = {};
  set_pools(R.P, dtype, k_pages, v_pages, k_scales, v_scales, LH, page_size, block, D);
  R.k_new = static_cast<const uint16_t*>(k_new);
  R.v_new = static_cast<const uint16_t*>(v_new);
  R.table = block_table;
  R.lens = seq_lens;
  R.nodes = nodes;
  R.num_accepted = num_accepted;
  R.out_lens = out_seq_lens;
  R.status = dev_status;
  R.B = B; R.N = N; R.num_pages = num_pages; R.cols = cols;
  const int threads = unit_threads(R.P);
  const int units = (N - 1 + block - 1) / block + 1;  // of a path of N entries, wherever it begins
  const dim3 g(static_cast<unsigned>(LH), static_cast<unsigned>(units < 64 ? units : 64),
               static_cast<unsigned>(B));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = dtype == SV_BF16;
  if (!in_place) {
    if (bf) sv_kv8_commit<true, false><<<g, threads, 0, st>>>(R);
    else sv_kv8_commit<false, false><<<g, threads, 0, st>>>(R);
    return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
  }
  if (bf) sv_kv8_commit<true, true><<<g, threads, 0, st>>>(R);
  else sv_kv8_commit<false, true><<<g, threads, 0, st>>>(R);
  if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(B));
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sv_kv8_advance, R) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // extern "C"
