// rope.cuh -- what the kernels that take packed tokens share: 16-bit values, the
// rotation of eight pairs, the request that a token belongs to, and the check of
// a request that is to be appended (see include/svrope.h and include/svkv8.h).
#ifndef SV_ROPE_CUH
#define SV_ROPE_CUH

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "specverify.h"
#include "svattn.h"
#include "svkv.h"

namespace svrope {

__device__ __forceinline__ void set_status(int32_t* status, int bits) {
  if (status && bits) atomicOr(status, bits);
}

// Two 16-bit values of a word in 32 bits, and back (rounded to nearest even).
template <bool BF>
__device__ __forceinline__ float2 widen(uint32_t w) {
  if (BF) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  __half2 h;
  memcpy(&h, &w, 4);
  return __half22float2(h);
}
template <bool BF>
__device__ __forceinline__ float widen1(uint16_t w) {
  return widen<BF>(w).x;
}
template <bool BF>
__device__ __forceinline__ uint32_t narrow(float lo, float hi) {
  uint32_t r;
  if (BF) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A head's dimensions are taken in chunks of eight pairs; pair s < rot / 2 is rotated,
// and the pairs behind them are the neighbours 2 s, 2 s + 1, which stay.
__device__ __forceinline__ int first_of(int s, int rot, bool inter) {
  return s < rot / 2 && !inter ? s : 2 * s;
}
__device__ __forceinline__ int second_of(int s, int rot, bool inter) {
  return s < rot / 2 && !inter ? s + rot / 2 : 2 * s + 1;
}

// The rotation, every product and sum rounded by itself.
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float lo = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = lo;
}

// Eight pairs from two 16-byte vectors: the first members in u and the second in v
// (half layout), or neighbours, four pairs in each.
template <bool BF>
__device__ __forceinline__ void split(const uint4& u, const uint4& v, bool inter, float (&a)[8],
                                      float (&b)[8]) {
  const uint32_t x[4] = {u.x, u.y, u.z, u.w}, y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = widen<BF>(x[i]), q = widen<BF>(y[i]);
    if (inter) {
      a[i] = p.x;
      b[i] = p.y;
      a[4 + i] = q.x;
      b[4 + i] = q.y;
    } else {
      a[2 * i] = p.x;
      a[2 * i + 1] = p.y;
      b[2 * i] = q.x;
      b[2 * i + 1] = q.y;
    }
  }
}
template <bool BF>
__device__ __forceinline__ void merge(const float (&a)[8], const float (&b)[8], bool inter,
                                      uint4& u, uint4& v) {
  uint32_t x[4], y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = inter ? narrow<BF>(a[i], b[i]) : narrow<BF>(a[2 * i], a[2 * i + 1]);
    y[i] = inter ? narrow<BF>(a[4 + i], b[4 + i]) : narrow<BF>(b[2 * i], b[2 * i + 1]);
  }
  u = make_uint4(x[0], x[1], x[2], x[3]);
  v = make_uint4(y[0], y[1], y[2], y[3]);
}
// Eight pairs turned by their cosines and sines.
struct Turns { float4 c0, c1, s0, s1; };
__device__ __forceinline__ void turn8(float (&a)[8], float (&b)[8], const Turns& w) {
  turn(a[0], b[0], w.c0.x, w.s0.x);
  turn(a[1], b[1], w.c0.y, w.s0.y);
  turn(a[2], b[2], w.c0.z, w.s0.z);
  turn(a[3], b[3], w.c0.w, w.s0.w);
  turn(a[4], b[4], w.c1.x, w.s1.x);
  turn(a[5], b[5], w.c1.y, w.s1.y);
  turn(a[6], b[6], w.c1.z, w.s1.z);
  turn(a[7], b[7], w.c1.w, w.s1.w);
}
// Those of pairs p .. p + 3 and q .. q + 3 in a table's row (cosines, then sines; 16-byte
// aligned there).
__device__ __forceinline__ Turns turns(const float* row, int rot, int p, int q) {
  const float* const s = row + rot / 2;
  return {__ldg(reinterpret_cast<const float4*>(row + p)),
          __ldg(reinterpret_cast<const float4*>(row + q)),
          __ldg(reinterpret_cast<const float4*>(s + p)),
          __ldg(reinterpret_cast<const float4*>(s + q))};
}

// The packed tokens of an append and where they go.
struct Appended {
  const int32_t* table;      // block table [B][cols]
  const int32_t* lens;
  const int32_t* cu;
  const int32_t* positions;  // or null
  int32_t* out_lens;         // or null
  int32_t* status;
  int B, T, cols, page, num_pages, rows;  // rows: of the rotation's table; 0: no rotation
};

// The request that holds packed token t, found by a whole warp (a step takes 32 bounds):
// the number of bounds cu[1 ..] at or below t.  False when none does; whatever the bounds
// hold, only cu[0 .. B] is read.
__device__ __forceinline__ bool request_of(const Appended& A, int t, int& b, int& lo, int& hi) {
  const int lane = int(threadIdx.x) & 31;
  int at = 0, n = A.B;  // the answer is in at .. at + n
  while (n > 0) {
    const int step = (n + 31) / 32, i = (lane + 1) * step;
    const bool below = i <= n && __ldg(A.cu + at + i) <= t;
    const int k = __popc(__ballot_sync(0xffffffffu, below));
    at += k * step;
    n = min(step - 1, n - k * step);
  }
  if (at >= A.B) return false;
  b = at;
  lo = __ldg(A.cu + at);
  hi = __ldg(A.cu + at + 1);
  return lo >= 0 && lo <= t && t < hi && hi <= A.T;
}

// Whether n tokens behind `len` entries fit.
__device__ __forceinline__ bool fits(const Appended& A, int len, int n) {
  const long long end = (long long)len + n;
  return len >= 0 && end <= (long long)A.cols * A.page && end <= 0x7fffffffLL;
}

// Faults of request b's n tokens from packed token lo on (pages in use, positions),
// looked for by `threads` threads, of which this is number `i`: each gets its own part.
__device__ __forceinline__ int faults_of(const Appended& A, int b, int lo, int n, int len, int i,
                                         int threads) {
  if (n == 0) return 0;
  if (!fits(A, len, n)) return SV_ST_BAD_LENGTH;
  int bad = 0;
  if (A.rows) {
    if (!A.positions) {
      if ((long long)len + n > A.rows) bad = SV_ST_BAD_LENGTH;
    } else {
      for (int j = i; j < n; j += threads) {
        const int p = __ldg(A.positions + lo + j);
        if (p < 0 || p >= A.rows) bad = SV_ST_BAD_LENGTH;
      }
    }
  }
  const int c0 = len / A.page, c1 = (len + n - 1) / A.page;
  for (int c = c0 + i; c <= c1; c += threads) {
    const int pg = __ldg(A.table + size_t(b) * A.cols + c);
    if (pg < 0 || pg >= A.num_pages) bad |= SV_ST_BAD_PAGE;
  }
  return bad;
}

// One request's new length and faults, by a warp.
__device__ __forceinline__ void settle(const Appended& A, int b) {
  const int lane = int(threadIdx.x) & 31;
  const int lo = __ldg(A.cu + b), hi = __ldg(A.cu + b + 1), len = __ldg(A.lens + b);
  int bad = SV_ST_BAD_LENGTH;
  if (lo >= 0 && lo <= hi && hi <= A.T) bad = faults_of(A, b, lo, hi - lo, len, lane, 32);
  bad = __reduce_or_sync(0xffffffffu, unsigned(bad));
  if (lane == 0) {
    if (A.out_lens) A.out_lens[b] = bad ? len : len + (hi - lo);
    set_status(A.status, bad);
  }
}

inline bool misaligned(const void* p, unsigned a) {
  return (reinterpret_cast<uintptr_t>(p) % a) != 0;
}
// A packed tensor's stride: a multiple of 8 elements that holds H heads.
inline bool bad_stride(long long stride, int H, int D) {
  return stride % 8 != 0 || stride < (long long)H * D || stride > (1LL << 40);
}
inline bool bad_rotation(const float* table, int rows, int rot, int D) {
  return table && (misaligned(table, 16) || rows < 1 || rot < 2 || rot > D || rot % 2 != 0);
}

}  // namespace svrope

#endif  // SV_ROPE_CUH
