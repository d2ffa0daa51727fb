// rope.cu -- sm_103a kernels and C ABI of rotary positions and of appending to
// the paged cache (see include/svrope.h for the operations, layouts and errors):
//
//   sv_rope_angles  the table: one thread per angle
//   sv_rope_tokens  packed tokens: each thread turns eight pairs of a head at a
//                   time and writes them to every place they go (queries' and keys'
//                   packed outputs, pages), or carries values to their pages
//
// Both move every byte once and are bound by that, or by their latency.

#include <math.h>

#include "rope.cuh"
#include "svrope.h"

namespace {

using namespace svrope;

constexpr int THREADS = 256;
constexpr int MAX_ROT = 256;
constexpr int MAX_TOKENS = 32;   // tokens of a CTA
constexpr int UNROLL = 2;        // chunks of a thread that are loaded before any is stored

// -------------------------------------------------------------- the table

struct AngleParams {
  float* table;
  int half, first, rows;
  float gain;
  uint64_t turn[MAX_ROT / 2];  // the angle of one position, in 2^-64 turns
};

// Position p's angle is p * turn modulo 2^64: whole turns fall off the integer product
// without a rounding, however far p is.  (64-bit floats would do, but GB300 has few units
// for them.)  The upper 32 bits, as a signed part of a turn, are split into a 32-bit float
// and a rest d, and the functions at the float are moved on by the rest:
// cos(x + d) = cos x - d sin x to within d^2 / 2 < 2^-47.
__global__ void __launch_bounds__(THREADS) sv_rope_angles(const __grid_constant__ AngleParams R) {
  const long long total = (long long)R.rows * R.half;
  const long long stride = (long long)gridDim.x * THREADS;
  for (long long f = (long long)blockIdx.x * THREADS + threadIdx.x; f < total; f += stride) {
    const int p = int(f / R.half), i = int(f - (long long)p * R.half);
    const int h = int(uint64_t(uint32_t(R.first + p)) * R.turn[i] >> 32);
    const float x = __int2float_rn(h);
    const float d = float((long long)h - (long long)x) * 1.46291807926715968e-9f;  // 2 pi / 2^32
    float s, c;
    sincospif(x * 0x1p-31f, &s, &c);
    float* const row = R.table + size_t(p) * 2 * R.half;
    row[i] = fmaf(-s, d, c) * R.gain;
    row[R.half + i] = fmaf(c, d, s) * R.gain;
  }
}

// -------------------------------------------------------------- packed tokens

struct TokenParams {
  Appended A;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* q_out;
  uint16_t* k_out;
  uint16_t* k_pages;
  uint16_t* v_pages;
  const float* angles;
  long long qs, ks, vs, qos, kos;  // strides
  int Hq, Hk, Hv, D, rot, LH, head0;
  int tokens;      // per CTA
  int token_ctas;  // the CTAs behind them settle the requests
  int chunks;      // of a head
  unsigned long long m_chunks, m_heads;
  bool inter, pages;
};

// n / d as n * ceil(2^40 / d) >> 40: right while n * d < 2^40 (n < 2^22 and d < 2^18 here).
unsigned long long div_magic(int d) { return ((1ull << 40) + unsigned(d) - 1) / unsigned(d); }
__device__ __forceinline__ int div_by(int n, unsigned long long m) {
  return int((unsigned long long)(unsigned)n * m >> 40);
}

struct Chunk {
  uint4 u, v;
  const uint16_t* src;
  uint16_t* dst[2];
  int c, pos;
  bool on, rotates, turned;  // its row is rotated, and this chunk of it
};

// VEC: the rotated part is a multiple of 16 dimensions, and a chunk two 16-byte vectors;
// otherwise a chunk's values are moved one by one.
template <bool BF, bool VEC>
__global__ void __launch_bounds__(THREADS) sv_rope_tokens(const __grid_constant__ TokenParams R) {
  __shared__ int pos_of[MAX_TOKENS];          // where a token is rotated to; -1: left out
  __shared__ long long page_of[MAX_TOKENS];   // its page's first row, and its row there
  const int tid = int(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  if (int(blockIdx.x) >= R.token_ctas) {
    const int b = (int(blockIdx.x) - R.token_ctas) * (THREADS / 32) + warp;
    if (b < R.A.B) settle(R.A, b);
    return;
  }
  const int t0 = int(blockIdx.x) * R.tokens, count = min(R.tokens, R.A.T - t0);
  for (int i = warp; i < count; i += THREADS / 32) {
    int pos = -1;
    long long where = 0;
    if (R.pages) {
      int b, lo, hi;
      if (request_of(R.A, t0 + i, b, lo, hi)) {
        const int len = __ldg(R.A.lens + b);
        if (fits(R.A, len, t0 + i - lo + 1)) {
          const int at = len + (t0 + i - lo), col = at / R.A.page;
          const int pg = __ldg(R.A.table + size_t(b) * R.A.cols + col);
          const int p = R.A.rows && R.A.positions ? __ldg(R.A.positions + t0 + i) : at;
          if (pg >= 0 && pg < R.A.num_pages && p >= 0 && (!R.A.rows || p < R.A.rows)) {
            pos = p;
            where = (long long)pg * R.LH * R.A.page + (at - col * R.A.page);
          }
        }
      }
    } else {
      const int p = __ldg(R.A.positions + t0 + i);
      if (p >= 0 && p < R.A.rows) pos = p;
      else if (lane == 0) set_status(R.A.status, SV_ST_BAD_LENGTH);
    }
    if (lane == 0) {
      pos_of[i] = pos;
      page_of[i] = where;
    }
  }
  __syncthreads();
  const int heads = R.Hq + R.Hk + R.Hv, total = count * heads * R.chunks;
  for (int f0 = tid; f0 < total; f0 += THREADS * UNROLL) {
    Chunk x[UNROLL];
#pragma unroll
    for (int n = 0; n < UNROLL; ++n) {
      Chunk& k = x[n];
      const int f = f0 + n * THREADS;
      const int row = div_by(f, R.m_chunks), i = div_by(row, R.m_heads);
      int h = row - i * heads;
      k.c = f - row * R.chunks;
      k.on = f < total;
      k.pos = k.on ? pos_of[i] : -1;
      k.on = k.pos >= 0;
      k.dst[0] = k.dst[1] = nullptr;
      k.rotates = true;
      if (!k.on) continue;
      const long long t = t0 + i;
      if (h < R.Hq) {
        k.src = R.q + t * R.qs + (long long)h * R.D;
        k.dst[0] = R.q_out + t * R.qos + (long long)h * R.D;
      } else {
        h -= R.Hq;
        const bool is_v = h >= R.Hk;
        if (is_v) h -= R.Hk;
        k.src = is_v ? R.v + t * R.vs + (long long)h * R.D : R.k + t * R.ks + (long long)h * R.D;
        k.rotates = !is_v;
        if (!is_v && R.k_out) k.dst[0] = R.k_out + t * R.kos + (long long)h * R.D;
        if (R.pages)
          k.dst[1] = (is_v ? R.v_pages : R.k_pages) +
                     (page_of[i] + (long long)(R.head0 + h) * R.A.page) * R.D;
      }
      k.turned = k.rotates && 8 * k.c < R.rot / 2;
      if (VEC) {
        const int a = k.turned && !R.inter ? 8 * k.c : 16 * k.c;
        const int b = k.turned && !R.inter ? a + R.rot / 2 : a + 8;
        k.u = *reinterpret_cast<const uint4*>(k.src + a);
        k.v = b < R.D ? *reinterpret_cast<const uint4*>(k.src + b) : make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int n = 0; n < UNROLL; ++n) {
      Chunk& k = x[n];
      if (!k.on) continue;
      const float* const angles = R.angles + (long long)k.pos * R.rot;
      if (VEC) {
        if (k.turned) {
          float a[8], b[8];
          split<BF>(k.u, k.v, R.inter, a, b);
          turn8(a, b, angles, R.rot, k.c);
          merge<BF>(a, b, R.inter, k.u, k.v);
        }
        const int a = k.turned && !R.inter ? 8 * k.c : 16 * k.c;
        const int b = k.turned && !R.inter ? a + R.rot / 2 : a + 8;
#pragma unroll
        for (int d = 0; d < 2; ++d)
          if (k.dst[d]) {
            *reinterpret_cast<uint4*>(k.dst[d] + a) = k.u;
            if (b < R.D) *reinterpret_cast<uint4*>(k.dst[d] + b) = k.v;
          }
      } else {
        for (int e = 0; e < 8; ++e) {
          const int pair = 8 * k.c + e;
          if (pair >= R.D / 2) break;
          const int a = first_of(pair, R.rot, R.inter), b = second_of(pair, R.rot, R.inter);
          uint16_t u = k.src[a], v = k.src[b];
          if (k.rotates && pair < R.rot / 2) {
            float y = widen1<BF>(u), z = widen1<BF>(v);
            turn(y, z, __ldg(angles + pair), __ldg(angles + R.rot / 2 + pair));
            const uint32_t w = narrow<BF>(y, z);
            u = uint16_t(w);
            v = uint16_t(w >> 16);
          }
#pragma unroll
          for (int d = 0; d < 2; ++d)
            if (k.dst[d]) {
              k.dst[d][a] = u;
              k.dst[d][b] = v;
            }
        }
      }
    }
  }
}

template <bool BF>
void launch_tokens(const TokenParams& R, bool vec, int grid, cudaStream_t st) {
  if (vec) sv_rope_tokens<BF, true><<<grid, THREADS, 0, st>>>(R);
  else sv_rope_tokens<BF, false><<<grid, THREADS, 0, st>>>(R);
}

int run_tokens(TokenParams& R, int dtype, void* stream) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    return SV_ERR_CUDA;
  R.chunks = (R.D + 15) / 16;
  const int heads = R.Hq + R.Hk + R.Hv, per_token = heads * R.chunks;
  R.m_chunks = div_magic(R.chunks);
  R.m_heads = div_magic(heads);
  // Two rounds of two chunks per thread, as long as that leaves every SM two CTAs.
  int tokens = 4 * THREADS / per_token;
  tokens = tokens < R.A.T / (2 * sms) ? tokens : R.A.T / (2 * sms);
  R.tokens = tokens < 1 ? 1 : tokens > MAX_TOKENS ? MAX_TOKENS : tokens;
  R.token_ctas = (R.A.T + R.tokens - 1) / R.tokens;
  const long long grid =
      R.token_ctas + (R.pages ? (R.A.B + THREADS / 32 - 1) / (THREADS / 32) : 0);
  if (grid > 0x7fffffff) return SV_ERR_INVALID_ARG;
  const bool vec = R.rot % 16 == 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == SV_BF16) launch_tokens<true>(R, vec, int(grid), st);
  else launch_tokens<false>(R, vec, int(grid), st);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

bool bad_width(int D) { return D < 8 || D > MAX_ROT || D % 8 != 0; }

}  // namespace

extern "C" {

int sv_rope_table(int scaling, double base, double factor, int original, double low, double high,
                  double gain, int rot, int first, int rows, float* table, void* stream) {
  if (scaling < SV_ROPE_NONE || scaling > SV_ROPE_WAVE || !(base > 1.0) || !isfinite(base) ||
      !(factor > 0.0) || !isfinite(factor) || !isfinite(gain) || !isfinite(float(gain)) ||
      rot < 2 || rot > MAX_ROT || rot % 2 != 0 || first < 0 || rows < 0 ||
      (long long)first + rows > 0x7fffffffLL || (scaling == SV_ROPE_BASE && rot == 2))
    return SV_ERR_INVALID_ARG;
  if (scaling >= SV_ROPE_RAMP &&
      (original < 1 || !(low > 0.0) || !(high > low) || !isfinite(high)))
    return SV_ERR_INVALID_ARG;
  if (rows == 0) return SV_OK;
  if (!table || misaligned(table, 16)) return SV_ERR_INVALID_ARG;
  constexpr double TWO_PI = 6.283185307179586476925286766559;
  if (scaling == SV_ROPE_BASE) base *= pow(factor, double(rot) / (rot - 2));
  double lo = 0.0, hi = 0.0;
  if (scaling == SV_ROPE_RAMP) {
    lo = floor(rot * log(original / (TWO_PI * high)) / (2.0 * log(base)));
    hi = ceil(rot * log(original / (TWO_PI * low)) / (2.0 * log(base)));
    if (lo < 0.0) lo = 0.0;
    if (hi > rot - 1) hi = rot - 1;
    if (hi == lo) hi += 0.001;
  }
  AngleParams R;
  R.table = table;
  R.half = rot / 2;
  R.first = first;
  R.rows = rows;
  R.gain = float(gain);
  for (int i = 0; i < R.half; ++i) {
    double w = pow(base, -2.0 * i / rot);
    if (scaling == SV_ROPE_LINEAR) {
      w /= factor;
    } else if (scaling == SV_ROPE_RAMP) {
      const double r = fmin(fmax((i - lo) / (hi - lo), 0.0), 1.0);
      w = w * (1.0 - r) + w / factor * r;
    } else if (scaling == SV_ROPE_WAVE) {
      const double s = fmin(fmax((original * w / TWO_PI - low) / (high - low), 0.0), 1.0);
      w = w * s + w / factor * (1.0 - s);
    }
    const double turns = w / TWO_PI;  // whole turns of one position leave nothing behind
    R.turn[i] = uint64_t(ldexp(turns - floor(turns), 63)) << 1;
  }
  const long long total = (long long)rows * R.half, most = 1 << 20;
  const long long grid = (total + THREADS - 1) / THREADS;
  sv_rope_angles<<<unsigned(grid < most ? grid : most), THREADS, 0,
                   static_cast<cudaStream_t>(stream)>>>(R);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

int sv_rope(int dtype, const void* q, long long q_stride, const void* k, long long k_stride,
            const int32_t* positions, const float* table, int rows, int rot, int interleaved,
            int T, int Hq, int Hk, int D, void* q_out, long long q_out_stride, void* k_out,
            long long k_out_stride, int32_t* dev_status, void* stream) {
  if (dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_DTYPE;
  if (T < 0 || Hq < 1 || Hq > 65535 || Hk < 0 || Hk > 65535 || bad_width(D) || !table ||
      bad_rotation(table, rows, rot, D) || bad_stride(q_stride, Hq, D) ||
      bad_stride(q_out_stride, Hq, D) ||
      (Hk > 0 && (bad_stride(k_stride, Hk, D) || bad_stride(k_out_stride, Hk, D))))
    return SV_ERR_INVALID_ARG;
  if (T == 0) return SV_OK;
  if (!q || !q_out || !positions || (Hk > 0 && (!k || !k_out))) return SV_ERR_INVALID_ARG;
  if (Hk == 0) k = k_out = nullptr;
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(q_out, 16) || misaligned(k_out, 16) ||
      misaligned(positions, 4) || misaligned(dev_status, 4) ||
      (q == q_out && q_stride != q_out_stride) || (k && k == k_out && k_stride != k_out_stride))
    return SV_ERR_INVALID_ARG;
  TokenParams R = {};
  R.A.positions = positions;
  R.A.status = dev_status;
  R.A.T = T;
  R.A.rows = rows;
  R.q = static_cast<const uint16_t*>(q);
  R.k = static_cast<const uint16_t*>(k);
  R.q_out = static_cast<uint16_t*>(q_out);
  R.k_out = static_cast<uint16_t*>(k_out);
  R.angles = table;
  R.qs = q_stride; R.ks = k_stride; R.qos = q_out_stride; R.kos = k_out_stride;
  R.Hq = Hq; R.Hk = Hk; R.D = D; R.rot = rot; R.inter = interleaved != 0;
  return run_tokens(R, dtype, stream);
}

int sv_page_append(int dtype, const void* k, long long k_stride, const void* v,
                   long long v_stride, void* k_pages, void* v_pages, const int32_t* block_table,
                   const int32_t* seq_lens, const int32_t* cu_seqlens, const float* table,
                   int rows, int rot, int interleaved, const int32_t* positions, const void* q,
                   long long q_stride, void* q_out, long long q_out_stride, void* k_out,
                   long long k_out_stride, int B, int T, int Hq, int Hkv, int D, int num_pages,
                   int LH, int head0, int page_size, int cols, int32_t* out_seq_lens,
                   int32_t* dev_status, void* stream) {
  if (dtype != SV_BF16 && dtype != SV_F16) return SV_ERR_DTYPE;
  if (B < 0 || B > 65535 || T < 0 || Hq < 0 || Hq > 65535 || Hkv < 1 || Hkv > 65535 ||
      bad_width(D) || bad_rotation(table, rows, rot, D) || num_pages < 1 || LH < 1 || head0 < 0 ||
      head0 > LH - Hkv || page_size < 1 || cols < 1 || bad_stride(k_stride, Hkv, D) ||
      bad_stride(v_stride, Hkv, D) || (k_out && bad_stride(k_out_stride, Hkv, D)) ||
      (Hq > 0 && (!table || bad_stride(q_stride, Hq, D) || bad_stride(q_out_stride, Hq, D))))
    return SV_ERR_INVALID_ARG;
  if (Hq == 0) q = q_out = nullptr;
  if (B == 0) return SV_OK;
  if (!k_pages || !v_pages || !block_table || !seq_lens || !cu_seqlens ||
      (T > 0 && (!k || !v || (Hq > 0 && (!q || !q_out)))))
    return SV_ERR_INVALID_ARG;
  if (misaligned(k, 16) || misaligned(v, 16) || misaligned(q, 16) || misaligned(k_pages, 16) ||
      misaligned(v_pages, 16) || misaligned(q_out, 16) || misaligned(k_out, 16) ||
      misaligned(block_table, 4) || misaligned(seq_lens, 4) || misaligned(cu_seqlens, 4) ||
      misaligned(positions, 4) || misaligned(out_seq_lens, 4) || misaligned(dev_status, 4) ||
      (q && q == q_out && q_stride != q_out_stride) ||
      (k && k == k_out && k_stride != k_out_stride))
    return SV_ERR_INVALID_ARG;
  if (out_seq_lens && out_seq_lens < seq_lens + B && seq_lens < out_seq_lens + B)
    return SV_ERR_INVALID_ARG;
  TokenParams R = {};
  R.A = {block_table, seq_lens, cu_seqlens, positions, out_seq_lens, dev_status,
         B, T, cols, page_size, num_pages, table ? rows : 0};
  R.q = static_cast<const uint16_t*>(q);
  R.k = static_cast<const uint16_t*>(k);
  R.v = static_cast<const uint16_t*>(v);
  R.q_out = static_cast<uint16_t*>(q_out);
  R.k_out = static_cast<uint16_t*>(k_out);
  R.k_pages = static_cast<uint16_t*>(k_pages);
  R.v_pages = static_cast<uint16_t*>(v_pages);
  R.angles = table;
  R.qs = q_stride; R.ks = k_stride; R.vs = v_stride; R.qos = q_out_stride; R.kos = k_out_stride;
  R.Hq = Hq; R.Hk = Hkv; R.Hv = Hkv; R.D = D; R.rot = table ? rot : 0;
  R.LH = LH; R.head0 = head0;
  R.inter = interleaved != 0;
  R.pages = true;
  return run_tokens(R, dtype, stream);
}

}  // extern "C"
