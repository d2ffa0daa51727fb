// kv8.cu -- sm_103a kernels and C ABI of writing the 8-bit paged cache (see
// include/svkv8.h for the operations, layouts and errors):
//
//   sv_kv8_append   packed tokens, keys rotated on the way
//   sv_kv8_commit   a verified path's staged entries
//   sv_kv8_advance  lengths of a commit that are updated in place
//
// A unit is the new entries of one block of tokens and one row: they share a
// scale, so all of them have to be seen before any is stored.  A CTA takes the units of one
// block and several rows, as many at once as two pieces per thread hold (a piece: sixteen
// dimensions of a token's key and of its value), finds each row's largest sizes, and rounds;
// the next rows' pieces are on their way to shared memory meanwhile.  Every byte is moved once
// (a block's older entries only when its scale rises); what bounds it is HBM and the
// instructions for prompts, and for single tokens and short paths the latency of the loads
// that depend on one another: bounds, length, page, entries.  (64 paths of 4 entries, 384 rows:
// 25 us; 101 with a CTA per unit, most of whose threads had no entry.  32 ragged prompts of 8
// heads, 86,000 tokens: 103 us, 5.2 TB/s, and 116 with the angles loaded again for every head;
// the registers leave an SM sixteen warps.)

#include <atomic>

#include "rope.cuh"
#include "svkv8.h"

namespace {

using namespace svrope;

constexpr int PIECES = 2;           // of a thread at a time
constexpr int MAX_THREADS = 512;    // a block of 128 tokens of 128 dimensions is 1024 pieces
constexpr int MAX_ROWS = 256;       // of a CTA

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

// The largest size of x and m, or NaN when either has one.
__device__ __forceinline__ float largest(const float (&x)[8], float m) {
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(x[i]), "f"(x[i + 1]));
  return m;
}
// That of sixteen 16-bit values.
template <bool BF>
__device__ __forceinline__ float largest(const uint4& a, const uint4& b) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t x = w[i] & 0x7fff7fffu;
    if (BF) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(x));
    else asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(m) : "r"(x));
  }
  const float2 f = widen<BF>(m);
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(f.x), "f"(f.y));
  return r;
}
// Where some are not finite: those become NaN, and the largest size of the rest.
__device__ __forceinline__ float largest_finite(float (&x)[8], float m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (fabsf(x[i]) <= 3.402823466e38f) m = fmaxf(m, fabsf(x[i]));
    else x[i] = __int_as_float(0x7fffffff);
  }
  return m;
}
__device__ __forceinline__ bool finite(float m) { return m <= 3.402823466e38f; }

__device__ __forceinline__ void copy_async(uint4* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   uint32_t(__cvta_generic_to_shared(to))), "l"(from) : "memory");
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

// A row's largest sizes, as bits, and the block's own exponents, when it holds entries.
struct RowState { uint32_t k, v; int own_k, own_v; };
struct Shared {
  RowState state[MAX_ROWS];
  uint4 pieces[];  // [two stages and the angles][piece][part of four][thread]
};
size_t shared_bytes(int threads, bool angles) {
  return sizeof(Shared) + size_t((angles ? 3 : 2) * PIECES * 4) * threads * 16;
}

__device__ __forceinline__ int exponent_k(const Pools& P, const RowState& x) {
  return max(exponent_for(__uint_as_float(x.k), P.least, P.most), x.own_k);
}
__device__ __forceinline__ int exponent_v(const Pools& P, const RowState& x) {
  return max(exponent_for(__uint_as_float(x.v), P.least, P.most), x.own_v);
}

// Entry `e` of a unit: its key and value in the first row, and the row of angles (or null).
struct Entry {
  const uint16_t *k, *v;
  const float* angles;
};

// The units of rows row0 .. row0 + rows - 1 of LH for the block of `page` (a valid one) that
// begins at its row `at`: new entries in its rows off .. off + count - 1.  source(e): entry e;
// the next row's lies k_row, v_row elements behind.
template <bool BF, bool VEC, class Source>
__device__ __forceinline__ void write_rows(const Pools& P, Shared& S, int page, int row0, int rows,
                                           int at, int off, int count, int rot, bool inter,
                                           long long k_row, long long v_row, const Source& source) {
  const int tid = int(threadIdx.x), threads = int(blockDim.x);
  const int per_row = count * P.chunks, at_once = min(rows, max(1, PIECES * threads / per_row));
  const size_t first = (size_t(page) * P.LH + row0) * P.page + at;  // the first row's block
  // where this thread's pieces lie: row of those at once, offset of an entry's dimensions, its
  // source.  (n / d as n * ceil(2^22 / d) >> 22: right while n * d < 2^22; both are 1024 at most.)
  const uint32_t by_row = ((1u << 22) + per_row - 1) / per_row;
  const uint32_t by_chunk = ((1u << 22) + P.chunks - 1) / P.chunks;
  int row[PIECES], chunk[PIECES], at_dim[PIECES];
  Entry entry[PIECES];
#pragma unroll
  for (int u = 0; u < PIECES; ++u) {
    const int f = tid + u * threads;
    row[u] = int(uint32_t(f) * by_row >> 22);
    const int rest = f - row[u] * per_row, e = int(uint32_t(rest) * by_chunk >> 22);
    chunk[u] = rest - e * P.chunks;
    at_dim[u] = (off + e) * P.D;
    if (row[u] < at_once) entry[u] = source(e);
    else row[u] = MAX_ROWS;  // never used
  }
  auto fetch = [&](int r0, int stage) {
#pragma unroll
    for (int u = 0; u < PIECES; ++u) {
      if (r0 + row[u] >= rows) continue;
      uint4* const to = S.pieces + (stage * PIECES + u) * 4 * threads + tid;
      const int c = chunk[u];
      if (VEC) {
        const bool halves = !inter && 8 * c < rot / 2;
        const uint16_t* const k = entry[u].k + (r0 + row[u]) * k_row + (halves ? 8 : 16) * c;
        copy_async(to, k);
        copy_async(to + threads, k + (halves ? rot / 2 : 8));
      }
      const uint16_t* const v = entry[u].v + (r0 + row[u]) * v_row + 16 * c;
      copy_async(to + 2 * threads, v);
      copy_async(to + 3 * threads, v + 8);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // (an entry's angles are those of every row)
  uint4* const held = S.pieces + 2 * PIECES * 4 * threads + tid;
  if (VEC && rot) {
#pragma unroll
    for (int u = 0; u < PIECES; ++u)
      if (row[u] < at_once && 8 * chunk[u] < rot / 2) {
        const float* const c = entry[u].angles + 8 * chunk[u];
        copy_async(held + u * 4 * threads, c);
        copy_async(held + (u * 4 + 1) * threads, c + 4);
        copy_async(held + (u * 4 + 2) * threads, c + rot / 2);
        copy_async(held + (u * 4 + 3) * threads, c + rot / 2 + 4);
      }
  }
  fetch(0, 0);
  __syncthreads();  // (the states of the units before these are used up)
  for (int r = tid; r < rows; r += threads) {
    RowState x = {0, 0, -1000, -1000};
    if (off) {
      const size_t s = (first + size_t(r) * P.page) / P.block;
      x.own_k = int(P.k_scales[s]) - 127;
      x.own_v = int(P.v_scales[s]) - 127;
    }
    S.state[r] = x;
  }
  __syncthreads();
  for (int r0 = 0, stage = 0; r0 < rows; r0 += at_once, stage ^= 1) {
    if (r0 + at_once < rows) {
      fetch(r0 + at_once, stage ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    float ka[PIECES][8], kb[PIECES][8];
#pragma unroll
    for (int u = 0; u < PIECES; ++u) {
      float mk = 0.0f, mv = 0.0f;
      if (r0 + row[u] < rows) {
        uint4* const from = S.pieces + (stage * PIECES + u) * 4 * threads + tid;
        const int c = chunk[u];
        if (VEC) {
          const bool turned = 8 * c < rot / 2;
          split<BF>(from[0], from[threads], inter || !turned, ka[u], kb[u]);
          if (turned) {
            const float4* const w = reinterpret_cast<const float4*>(held + u * 4 * threads);
            turn8(ka[u], kb[u], {w[0], w[threads], w[2 * threads], w[3 * threads]});
          }
        } else {
          const uint16_t* const k = entry[u].k + (r0 + row[u]) * k_row;
          const float* const angles = entry[u].angles;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int pair = e * P.chunks + c;
            ka[u][e] = widen1<BF>(k[first_of(pair, rot, inter)]);
            kb[u][e] = widen1<BF>(k[second_of(pair, rot, inter)]);
            if (pair < rot / 2)
              turn(ka[u][e], kb[u][e], __ldg(angles + pair), __ldg(angles + rot / 2 + pair));
          }
        }
        mk = largest(kb[u], largest(ka[u], 0.0f));
        if (!finite(mk)) mk = largest_finite(kb[u], largest_finite(ka[u], 0.0f));
        const uint4 va = from[2 * threads], vb = from[3 * threads];
        mv = largest<BF>(va, vb);
        if (!finite(mv)) {
          float x[8], y[8];
          split<BF>(va, vb, true, x, y);
          mv = largest_finite(y, largest_finite(x, 0.0f));
          merge<BF>(x, y, true, from[2 * threads], from[3 * threads]);
        }
      }
      if (per_row % 32 == 0) {  // the warp's pieces are of one row
        const uint32_t a = __reduce_max_sync(0xffffffffu, __float_as_uint(mk));
        const uint32_t b = __reduce_max_sync(0xffffffffu, __float_as_uint(mv));
        if (r0 + row[u] < rows && (tid & 31) == 0) {
          atomicMax(&S.state[r0 + row[u]].k, a);
          atomicMax(&S.state[r0 + row[u]].v, b);
        }
      } else if (r0 + row[u] < rows) {
        atomicMax(&S.state[r0 + row[u]].k, __float_as_uint(mk));
        atomicMax(&S.state[r0 + row[u]].v, __float_as_uint(mv));
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < PIECES; ++u) {
      if (r0 + row[u] >= rows) continue;
      const RowState x = S.state[r0 + row[u]];
      const float fk = power(-exponent_k(P, x)), fv = power(-exponent_v(P, x));
      const size_t to = (first + size_t(r0 + row[u]) * P.page) * P.D + at_dim[u];
      unsigned char* const kp = P.k_pages + to;
      const int c = chunk[u];
      const bool turned = 8 * c < rot / 2;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ka[u][e] *= fk;
        kb[u][e] *= fk;
      }
      const auto& a = ka[u];
      const auto& b = kb[u];
      if (VEC && turned && !inter) {
        *reinterpret_cast<uint2*>(kp + 8 * c) =
            make_uint2(to_bytes(a[0], a[1], a[2], a[3]), to_bytes(a[4], a[5], a[6], a[7]));
        *reinterpret_cast<uint2*>(kp + 8 * c + rot / 2) =
            make_uint2(to_bytes(b[0], b[1], b[2], b[3]), to_bytes(b[4], b[5], b[6], b[7]));
      } else if (VEC) {
        *reinterpret_cast<uint4*>(kp + 16 * c) =
            make_uint4(to_bytes(a[0], b[0], a[1], b[1]), to_bytes(a[2], b[2], a[3], b[3]),
                       to_bytes(a[4], b[4], a[5], b[5]), to_bytes(a[6], b[6], a[7], b[7]));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int pair = e * P.chunks + c;
          const uint32_t w = to_bytes(a[e], b[e], 0.0f, 0.0f);
          kp[first_of(pair, rot, inter)] = uint8_t(w);
          kp[second_of(pair, rot, inter)] = uint8_t(w >> 8);
        }
      }
      float y[8], z[8];
      const uint4* const from = S.pieces + (stage * PIECES + u) * 4 * threads + tid;
      split<BF>(from[2 * threads], from[3 * threads], true, y, z);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] *= fv;
        z[e] *= fv;
      }
      *reinterpret_cast<uint4*>(P.v_pages + to + 16 * c) =
          make_uint4(to_bytes(y[0], z[0], y[1], z[1]), to_bytes(y[2], z[2], y[3], z[3]),
                     to_bytes(y[4], z[4], y[5], z[5]), to_bytes(y[6], z[6], y[7], z[7]));
    }
  }
  // the rows' scales, and older entries of those whose scale has risen
  for (int r = tid; r < rows; r += threads) {
    const RowState x = S.state[r];
    const size_t s = (first + size_t(r) * P.page) / P.block;
    P.k_scales[s] = uint8_t(exponent_k(P, x) + 127);
    P.v_scales[s] = uint8_t(exponent_v(P, x) + 127);
  }
  for (int r = tid >> 5; off && r < rows; r += threads >> 5) {
    const RowState x = S.state[r];
    const int k_by = x.own_k - exponent_k(P, x), v_by = x.own_v - exponent_v(P, x);
    const size_t to = (first + size_t(r) * P.page) * P.D;
    for (int f = tid & 31; (k_by | v_by) && f < off * P.chunks; f += 32) {
      uint4* const k = reinterpret_cast<uint4*>(P.k_pages + to) + f;
      uint4* const v = reinterpret_cast<uint4*>(P.v_pages + to) + f;
      uint4 a, b;
      if (k_by) a = *k;
      if (v_by) b = *v;
      const float g = power(k_by), h = power(v_by);
      if (k_by) *k = make_uint4(again(a.x, g), again(a.y, g), again(a.z, g), again(a.w, g));
      if (v_by) *v = make_uint4(again(b.x, h), again(b.y, h), again(b.z, h), again(b.w, h));
    }
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
  int heads;       // of a CTA
  int tokens;      // per CTA, whose units are those that begin among them
  int token_ctas;  // CTAs behind them settle the requests (of the first heads)
  bool inter;
};

template <bool BF, bool VEC>
__global__ void __launch_bounds__(MAX_THREADS) sv_kv8_append(
    const __grid_constant__ AppendParams R) {
  extern __shared__ __align__(16) unsigned char smem[];
  Shared& S = *reinterpret_cast<Shared*>(smem);
  const Appended& A = R.A;
  const int tid = int(threadIdx.x), h = int(blockIdx.y) * R.heads;
  if (int(blockIdx.x) >= R.token_ctas) {
    const int warps = int(blockDim.x) >> 5;
    const int b = (int(blockIdx.x) - R.token_ctas) * warps + (tid >> 5);
    if (h == 0 && b < A.B) settle(A, b);
    return;
  }
  const int t0 = int(blockIdx.x) * R.tokens, t1 = t0 + min(R.tokens, A.T - t0);
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
      if (tid < count) p = A.positions ? __ldg(A.positions + lo + j + tid) : at + tid;
      ok = !__syncthreads_or(p < 0 || p >= A.rows) && ok;
    }
    if (!ok) continue;
    const long long token = lo + j;
    write_rows<BF, VEC>(R.P, S, pg, R.head0 + h, min(R.heads, R.Hkv - h), at - off - col * A.page,
                   off, count, R.rot, R.inter, R.P.D, R.P.D, [&](int e) {
                     const int p = A.rows && A.positions ? __ldg(A.positions + token + e) : at + e;
                     return Entry{R.k + (token + e) * R.ks + (long long)h * R.P.D,
                                  R.v + (token + e) * R.vs + (long long)h * R.P.D,
                                  R.angles + (long long)(A.rows ? p : 0) * R.rot};
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
  int rows;  // of a CTA
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

// Block blockIdx.y (and every gridDim.y-th from there) of the path of request blockIdx.z, rows
// from blockIdx.x * R.rows on.  IN_PLACE: the lengths are updated by the next kernel instead.
template <bool BF, bool IN_PLACE>
__global__ void __launch_bounds__(MAX_THREADS) sv_kv8_commit(
    const __grid_constant__ CommitParams R) {
  extern __shared__ __align__(16) unsigned char smem[];
  Shared& S = *reinterpret_cast<Shared*>(smem);
  if (IN_PLACE) allow_next_kernel();
  const int b = int(blockIdx.z), row = int(blockIdx.x) * R.rows;
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
  for (long long j0 = before; j0 <= k;
       j0 += (long long)gridDim.y * block - (j0 ? 0 : len % block)) {
    const int j = int(j0), at = len + j, off = at % block;
    const int count = min(block - off, k + 1 - j), col = at / R.P.page;
    const int pg = __ldg(R.table + size_t(b) * R.cols + col);
    const long long next = (long long)R.N * R.P.D;
    write_rows<BF, true>(R.P, S, pg, row, min(R.rows, R.P.LH - row), at - off - col * R.P.page,
                   off, count, 0, false, next, next, [&](int i) {
                     const int e = j + i;
                     const int node =
                         R.nodes && e > 0 ? __ldg(R.nodes + size_t(b) * R.N + e - 1) : e;
                     const size_t from = ((size_t(b) * R.P.LH + row) * R.N + node) * R.P.D;
                     return Entry{R.k_new + from, R.v_new + from, nullptr};
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
// Threads of a CTA: a row's pieces fit twice, if it is a whole block's.
int threads_for(const Pools& P) {
  return P.block * P.chunks <= PIECES * 128 ? 128 : P.block * P.chunks <= PIECES * 256 ? 256 : 512;
}
// Rows of a CTA: enough CTAs for `per_sm` on every SM, if there is work for them.  Otherwise
// 1024 threads' worth, twice what an SM holds.  (Eight CTAs per SM whatever their size: paths of
// 34 requests, 65 rows, blocks of 128: 28.3 us for 12.6; 25,000 tokens of prompts, 8 heads of
// 96, blocks of 128: 71 for 50.)
int rows_for(long long units, int rows, long long sms, int per_sm) {
  const long long n = (units * rows + per_sm * sms / 2) / (per_sm * sms);
  const int most = rows < MAX_ROWS ? rows : MAX_ROWS;
  return int(n < 1 ? 1 : n < most ? n : most);
}
template <auto KERNEL, class Params>
int start(dim3 grid, int threads, bool angles, cudaStream_t st, const Params& R) {
  const size_t bytes = shared_bytes(threads, angles);
  if (bytes > 48 * 1024) {
    // the kernel's shared-memory limit, raised once per device (ordinals past 63: every time)
    static std::atomic<uint64_t> raised{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SV_ERR_CUDA;
    const uint64_t mark = dev < 64 ? uint64_t(1) << dev : 0;
    if (!(raised.load(std::memory_order_acquire) & mark)) {
      if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               int(shared_bytes(MAX_THREADS, true))) != cudaSuccess)
        return SV_ERR_CUDA;
      raised.fetch_or(mark, std::memory_order_release);
    }
  }
  KERNEL<<<grid, threads, bytes, st>>>(R);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}
int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return sms;
}

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
  const int sms = sm_count();
  if (sms < 1) return SV_ERR_CUDA;
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
  const int threads = threads_for(R.P);
  // A CTA per token when that is a few CTAs per SM or most units are far shorter than a block
  // (single tokens: every unit at once), else one per block's worth of tokens (a prompt's CTAs
  // have one unit each).  (8 heads.  One token each of 1024 requests, blocks of 16: 9.9 us, and
  // 55 in CTAs of 16 tokens, one unit after another; 12 tokens each of 256, blocks of 32: 16.2
  // and 26.9; 30 tokens each of 64: 18.2 and 15.4.)
  R.tokens = (long long)T * Hkv <= 16LL * sms || 2LL * T < (long long)B * block ? 1 : block;
  R.token_ctas = int(((long long)T + R.tokens - 1) / R.tokens);
  const long long grid = R.token_ctas + ((long long)B + threads / 32 - 1) / (threads / 32);
  if (grid > 0x7fffffffLL) return SV_ERR_INVALID_ARG;
  // Heads of a single token are few pieces: two CTAs per SM, whose heads pass at once, beat more
  // CTAs.  (64 tokens of 32 heads 5.0 us, 7.8 with four per SM; 512 of 8 heads 5.7 and 8.9.)
  R.heads = rows_for(R.token_ctas, Hkv, sms, R.tokens == 1 ? 2 : 1024 / threads);
  const dim3 g(static_cast<unsigned>(grid), static_cast<unsigned>((Hkv + R.heads - 1) / R.heads));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = dtype == SV_BF16;
  const bool vec = R.rot % 16 == 0, angles = R.rot != 0 && vec;
  if (vec)
    return bf ? start<sv_kv8_append<true, true>>(g, threads, angles, st, R)
              : start<sv_kv8_append<false, true>>(g, threads, angles, st, R);
  return bf ? start<sv_kv8_append<true, false>>(g, threads, angles, st, R)
            : start<sv_kv8_append<false, false>>(g, threads, angles, st, R);
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
  const int sms = sm_count();
  if (sms < 1) return SV_ERR_CUDA;
  const int threads = threads_for(R.P);
  R.rows = rows_for(B, LH, sms, 1024 / threads);
  const int units = (N - 1 + block - 1) / block + 1;  // of a path of N entries, wherever it begins
  // A path's units one after another, unless there are too few CTAs otherwise: most paths have
  // one or two, whatever N, and the CTAs that find none cost 1 us of 30 (64 paths of 4 entries out
  // of 22 nodes, 384 rows).
  const long long ctas = (long long)B * ((LH + R.rows - 1) / R.rows), y = 8LL * sms / ctas;
  const dim3 g(static_cast<unsigned>((LH + R.rows - 1) / R.rows),
               static_cast<unsigned>(y < 1 ? 1 : y < units ? y : units), static_cast<unsigned>(B));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf = dtype == SV_BF16;
  if (!in_place)
    return bf ? start<sv_kv8_commit<true, false>>(g, threads, false, st, R)
              : start<sv_kv8_commit<false, false>>(g, threads, false, st, R);
  const int rc = bf ? start<sv_kv8_commit<true, true>>(g, threads, false, st, R)
                    : start<sv_kv8_commit<false, true>>(g, threads, false, st, R);
  if (rc != SV_OK) return rc;
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
