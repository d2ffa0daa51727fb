// rope.cu -- sm_103a kernels and C ABI of rotary positions and of appending to
// the paged cache (see include/svrope.h for the operations, layouts and errors):
//
//   sv_rope_angles  the table: a thread takes one pair's angle at several positions
//   sv_rope_tokens  packed tokens: a thread takes the same eight pairs of several
//                   heads of a token, turns them by the same angles and writes them
//                   to every place they go (queries' and keys' packed outputs,
//                   pages), or carries values to their pages
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
  int passes;  // rows of a thread
  float gain;
  uint64_t turn[MAX_ROT / 2];  // the angle of one position, in 2^-64 turns
};

// Position p's angle is p * turn modulo 2^64: whole turns fall off the integer product
// without a rounding, however far p is.  (64-bit floats would do, but GB300 has few units
// for them.)  Its upper 32 bits are split into the nearest quarter turn and a rest x of at
// most pi / 4 to either side, where the Taylor polynomials of sine (to x^9) and cosine (to
// x^10) are off by less than 2^-29; the roundings of x and of the sums add up to 2^-23.
// What bounds it is the instructions until the table outgrows L2.  (131072 positions of 64
// pairs: 67 us with a division per angle and sincospif, whose reduction has nothing left to
// do here, 15 with a pair per thread, 11.4 with four, 5.9 TB/s.)
// V neighbouring pairs of a thread, stored as one vector: four where the pairs can be cut so.
template <int V>
__global__ void __launch_bounds__(THREADS) sv_rope_angles(const __grid_constant__ AngleParams R) {
  const int lanes = R.half / V, at_once = THREADS / lanes, r = int(threadIdx.x) / lanes;
  const int i = (int(threadIdx.x) - r * lanes) * V;
  if (r >= at_once) return;
  const long long p0 = (long long)blockIdx.x * R.passes * at_once + r;
  uint64_t angle[V], step[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    angle[v] = R.turn[i + v] * uint64_t(R.first + p0);
    step[v] = R.turn[i + v] * unsigned(at_once);
  }
  float* out = R.table + size_t(p0) * 2 * R.half + i;
#pragma unroll 1
  for (int n = 0; n < R.passes && p0 + n * at_once < R.rows; ++n) {
    float cs[V], sn[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t h = uint32_t(angle[v] >> 32), quarter = h + 0x20000000u;
      const float x =
          float(int(h - (quarter & 0xc0000000u))) * 1.46291807926715968e-9f;  // 2 pi / 2^32
      const float y = x * x;
      float s = fmaf(y, 1.0f / 362880, -1.0f / 5040);
      s = fmaf(y, s, 1.0f / 120);
      s = fmaf(y, s, -1.0f / 6);
      s = fmaf(x * y, s, x);
      float c = fmaf(y, -1.0f / 3628800, 1.0f / 40320);
      c = fmaf(y, c, -1.0f / 720);
      c = fmaf(y, c, 1.0f / 24);
      c = fmaf(y, c, -0.5f);
      c = fmaf(y, c, 1.0f);
      // a quarter turn more: (c, s) becomes (-s, c)
      const bool odd = quarter & 0x40000000u;
      const uint32_t low = quarter & 0x80000000u, high = low ^ (quarter << 1 & 0x80000000u);
      cs[v] = __uint_as_float(__float_as_uint(odd ? s : c) ^ high) * R.gain;
      sn[v] = __uint_as_float(__float_as_uint(odd ? c : s) ^ low) * R.gain;
      angle[v] += step[v];
    }
    if constexpr (V == 4) {
      *reinterpret_cast<float4*>(out) = make_float4(cs[0], cs[1], cs[2], cs[3]);
      *reinterpret_cast<float4*>(out + R.half) = make_float4(sn[0], sn[1], sn[2], sn[3]);
    } else {
      out[0] = cs[0];
      out[R.half] = sn[0];
    }
    out += size_t(at_once) * 2 * R.half;
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
  int lanes;       // the heads of a token that are taken at once
  bool inter, pages;
};

// A chunk is sixteen dimensions of a head, two vectors of eight: eight pairs that are turned,
// or what is not.  VEC: the rotated part is a multiple of 16 dimensions, and a chunk two 16-byte
// vectors half the head (or half the part) apart, so that neighbouring threads' vectors are
// neighbours; otherwise a chunk's values are moved one by one.
//
// The first heads are loaded before it is known where they go: bounds, length, page and angles
// are a chain of four loads, the latency of a decoding step.
template <bool BF, bool VEC>
__global__ void __launch_bounds__(THREADS, 4) sv_rope_tokens(
    const __grid_constant__ TokenParams R) {
  __shared__ int pos_of[MAX_TOKENS];          // where a token is rotated to; -1: left out
  __shared__ long long page_of[MAX_TOKENS];   // its page's first row, and its row there
  const int tid = int(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  if (int(blockIdx.x) >= R.token_ctas) {
    const int b = (int(blockIdx.x) - R.token_ctas) * (THREADS / 32) + warp;
    if (b < R.A.B) settle(R.A, b);
    return;
  }
  const int t0 = int(blockIdx.x) * R.tokens, count = min(R.tokens, R.A.T - t0);
  const int slot = tid / R.chunks, c = tid - slot * R.chunks;
  const int i = slot / R.lanes, h0 = slot - i * R.lanes;
  const int keys = R.Hq, values = R.Hq + R.Hk, heads = values + R.Hv;
  const bool active = i < count;
  const long long t = unsigned(t0) + unsigned(i);
  bool turned = 8 * c < R.rot / 2;  // (half layout)
  int a, b;                         // where the vectors lie in a head
  if (turned && !R.inter) {
    a = 8 * c;
    b = a + R.rot / 2;
  } else {
    const int skip = R.inter ? 0 : R.rot, vectors = (R.D - skip) / 8;
    a = 8 * c + skip / 2;
    b = a + (vectors + 1) / 2 * 8;
  }
  const bool second = b < R.D, turned_b = !R.inter || b < R.rot;
  if (R.inter) turned = a < R.rot;
  uint4 u[UNROLL], v[UNROLL];
  auto source = [&](int h) {
    return h < keys ? R.q + t * R.qs + (long long)h * R.D
           : h < values ? R.k + t * R.ks + (long long)(h - keys) * R.D
                        : R.v + t * R.vs + (long long)(h - values) * R.D;
  };
  auto load = [&](int first) {
#pragma unroll
    for (int n = 0; n < UNROLL; ++n) {
      const int h = first + n * R.lanes;
      if (h < heads) {
        const uint16_t* const src = source(h);
        u[n] = *reinterpret_cast<const uint4*>(src + a);
        v[n] = second ? *reinterpret_cast<const uint4*>(src + b) : make_uint4(0, 0, 0, 0);
      }
    }
  };
  if (VEC && active) load(h0);
  int pos = -1;
  long long where = 0;
  if (R.pages) {
    for (int j = warp; j < count; j += THREADS / 32) {
      int r, lo, hi, to = -1;
      long long row = 0;
      if (request_of(R.A, t0 + j, r, lo, hi)) {
        const int len = __ldg(R.A.lens + r);
        if (fits(R.A, len, t0 + j - lo + 1)) {
          const int at = len + (t0 + j - lo), col = at / R.A.page;
          const int pg = __ldg(R.A.table + size_t(r) * R.A.cols + col);
          const int p = R.A.rows && R.A.positions ? __ldg(R.A.positions + t0 + j) : at;
          if (pg >= 0 && pg < R.A.num_pages && p >= 0 && (!R.A.rows || p < R.A.rows)) {
            to = p;
            row = (long long)pg * R.LH * R.A.page + (at - col * R.A.page);
          }
        }
      }
      if (lane == 0) {
        pos_of[j] = to;
        page_of[j] = row;
      }
    }
    __syncthreads();
    if (active) {
      pos = pos_of[i];
      where = page_of[i];
    }
  } else if (active) {
    pos = __ldg(R.A.positions + t);
    if (pos < 0 || pos >= R.A.rows) {
      pos = -1;
      if (c == 0 && h0 == 0) set_status(R.A.status, SV_ST_BAD_LENGTH);
    }
  }
  if (pos < 0) return;
  const float* const angles = R.angles + (long long)pos * R.rot;
  Turns w = {};
  if (VEC && turned)
    w = turns(angles, R.rot, R.inter ? a / 2 : a, !R.inter ? a + 4 : turned_b ? b / 2 : a / 2);
  for (int first = h0; first < heads;) {
#pragma unroll
    for (int n = 0; n < UNROLL; ++n) {
      const int h = first + n * R.lanes;
      if (h >= heads) break;
      uint16_t *packed = nullptr, *paged = nullptr;
      if (h < keys) {
        packed = R.q_out + t * R.qos + (long long)h * R.D;
      } else {
        const bool is_v = h >= values;
        const int g = h - (is_v ? values : keys);
        if (!is_v && R.k_out) packed = R.k_out + t * R.kos + (long long)g * R.D;
        if (R.pages)
          paged = (is_v ? R.v_pages : R.k_pages) +
                  (where + (long long)(R.head0 + g) * R.A.page) * R.D;
      }
      if (VEC) {
        if (turned && h < values) {
          float x[8], y[8];
          const uint4 rest = v[n];
          split<BF>(u[n], v[n], R.inter, x, y);
          turn8(x, y, w);
          merge<BF>(x, y, R.inter, u[n], v[n]);
          if (!turned_b) v[n] = rest;
        }
        if (packed) {
          *reinterpret_cast<uint4*>(packed + a) = u[n];
          if (second) *reinterpret_cast<uint4*>(packed + b) = v[n];
        }
        if (paged) {
          *reinterpret_cast<uint4*>(paged + a) = u[n];
          if (second) *reinterpret_cast<uint4*>(paged + b) = v[n];
        }
      } else {
        // (neighbouring threads' pairs are neighbours: 2048 tokens of 40 heads of 96, 24 rotated,
        // 18 us; 41 with eight neighbouring pairs of a thread)
        const uint16_t* const src = source(h);
        for (int e = 0; e < 8; ++e) {
          const int pair = e * R.chunks + c;
          if (pair >= R.D / 2) break;
          const int d0 = first_of(pair, R.rot, R.inter), d1 = second_of(pair, R.rot, R.inter);
          uint16_t x = src[d0], y = src[d1];
          if (h < values && pair < R.rot / 2) {
            float f = widen1<BF>(x), g = widen1<BF>(y);
            turn(f, g, __ldg(angles + pair), __ldg(angles + R.rot / 2 + pair));
            const uint32_t z = narrow<BF>(f, g);
            x = uint16_t(z);
            y = uint16_t(z >> 16);
          }
          if (packed) {
            packed[d0] = x;
            packed[d1] = y;
          }
          if (paged) {
            paged[d0] = x;
            paged[d1] = y;
          }
        }
      }
    }
    first += UNROLL * R.lanes;
    if (VEC && first < heads) load(first);
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
  const int heads = R.Hq + R.Hk + R.Hv, slots = THREADS / R.chunks;
  // Four heads per thread, as long as that leaves every SM two CTAs.  (Two at once: 17800 tokens
  // of 48 heads 77 us, 96 when all four are loaded first, whose registers halve the CTAs of an SM.)
  int tokens = 4 * slots / heads;
  tokens = tokens < R.A.T / (2 * sms) ? tokens : R.A.T / (2 * sms);
  tokens = tokens < slots ? tokens : slots;
  R.tokens = tokens < 1 ? 1 : tokens > MAX_TOKENS ? MAX_TOKENS : tokens;
  R.lanes = slots / R.tokens;
  R.token_ctas = int(((long long)R.A.T + R.tokens - 1) / R.tokens);
  const long long grid =
      (long long)R.token_ctas + (R.pages ? (R.A.B + THREADS / 32 - 1) / (THREADS / 32) : 0);
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
  constexpr double TWO_PI = 6.283185307179586476925286766559;
  if (scaling == SV_ROPE_BASE) base *= pow(factor, double(rot) / (rot - 2));
  if (!(base > 0.0) || !isfinite(base)) return SV_ERR_INVALID_ARG;
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
  for (int i = 0; i < R.half; ++i) {  // (a rate that is not finite would have no turn)
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
    if (!isfinite(w)) return SV_ERR_INVALID_ARG;
    const double turns = w / TWO_PI;  // whole turns of one position leave nothing behind
    R.turn[i] = uint64_t(ldexp(turns - floor(turns), 63)) << 1;
  }
  if (rows == 0) return SV_OK;
  if (!table || misaligned(table, 16)) return SV_ERR_INVALID_ARG;
  // Sixteen rows per thread, as long as that leaves some CTAs for every SM.
  const bool vec = R.half % 4 == 0;
  const int at_once = THREADS / (vec ? R.half / 4 : R.half), passes = rows / at_once / 1024;
  R.passes = passes < 1 ? 1 : passes > 16 ? 16 : passes;
  const long long per_cta = (long long)at_once * R.passes, grid = (rows + per_cta - 1) / per_cta;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (vec) sv_rope_angles<4><<<unsigned(grid), THREADS, 0, st>>>(R);
  else sv_rope_angles<1><<<unsigned(grid), THREADS, 0, st>>>(R);
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
