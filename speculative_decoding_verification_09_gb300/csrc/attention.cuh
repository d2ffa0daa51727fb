// attention.cuh -- sm_103a kernels of the attention over the caches (the calls
// are in attention.cu, the operations in include/svattn.h).
//
//   sv_attn       per query row, over its visible keys t in tiles of 128:
//                   s_t = scale q . k_t,  m = max s,  l = sum exp(s_t - m),
//                   O = sum exp(s_t - m) v_t,  out = O / l
//                 in one pass: a tile's weights use the maximum so far, and O and l
//                 are rescaled when it has risen (exactly: exp(m_old - m_new))
//   sv_attn_join  the same sum over parts: m = max m_i, l = sum l_i exp(m_i - m),
//                 O = sum O_i exp(m_i - m)
//
// What bounds them.  Tokens over a cache (trees, the ring): the cache is read
// once, 4 D bytes per key and KV head, and the products are small beside it: HBM,
// as long as a key tile's chain of products and softmax (about 1 us) hides under
// its 64 KB (1.5 us of an SM's share).  Hence two streams of key tiles per SM, so
// that one's products run under the other's softmax, copies five to twelve stages
// ahead, and runs of equal length whatever the requests' lengths.  64 requests of
// 22 nodes over 2000 to 9000 tokens (1.39 GB): 225 us, 6.2 TB/s, 0.91 of the
// measured copy bandwidth.  Prompts: 4 D flops per pair of tokens and query head;
// the tensor cores are busy 0.61 of the time, and each of the two tiles of queries
// that share an SM is a chain: scores, softmax, the weights' product, the next
// scores (which take the weights' place).  8192 tokens under a window of 4096, 32
// heads of 128: 319 us, 1.29 PFLOP/s, 0.67 of the measured bf16 rate.
#ifndef SV_ATTENTION_CUH
#define SV_ATTENTION_CUH

#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "specverify.h"
#include "svattn.h"
#include "svkv.h"

namespace svattn {

enum Kind { TREE = 0, RING = 1, PROMPT = 2 };

constexpr int MAX_N = 256;      // tree nodes
constexpr int MAX_R = 64;       // staged tokens of the ring call
constexpr int MAX_GROUP = 128;  // query heads per KV head
constexpr int MAX_D = 128;
constexpr int MAX_KEYS = 0x7fffffff - 1023;  // cache entries: a tile more fits an int

constexpr int ITEM_COST = 2;    // an item's fixed cost in tiles (1 to 3: within 2 %)
constexpr int TILE = 128;       // query rows of a tile, and keys of a tile
constexpr int THREADS = 384;    // two softmax warpgroups, and one with a copy and a product warp
// Registers: launched with 168 a thread (64512 a CTA); the softmax warpgroups
// hold up to 128 scores a thread and take over what the third does not need.
// (Ragged prompts: 107 us with 208 / 88, 101 with 216 / 72, 132 with 184 / 136.)
constexpr int SOFTMAX_REGS = 216, OTHER_REGS = 72;
static_assert(256 * SOFTMAX_REGS + 128 * OTHER_REGS <= THREADS * 168, "register split");
constexpr int COPY_WARP = 8, MMA_WARP = 9, PLAN_WARP = 10;
constexpr int MAX_CTAS = 152;   // one per SM
constexpr unsigned long long WAIT_LIMIT_NS = 1000000000ull;
constexpr uint32_t SUSPEND_HINT_NS = 20000;
// A row's running maximum is raised only when a score would get a weight above 2^most,
// and has the weight 2^lift when it is; until the next time weights of up to 2^most are
// summed, which 32-bit sums hold as exactly as those below 1, and the output tile needs
// no rescaling.  bf16 weights are as exact at any size: no lift (8192 tokens: 325 us with
// a `most` of 8, 314 with 12).  fp16 ones end at 2^16 and get steps of 2^-24 below 2^-14:
// a weight is off by up to 2^-(25 + lift) of the largest one, and the launch chooses the
// lift by the number of keys so that all of them together stay below half a step of the
// type.  (Ragged prompts: 89.6 us with 0 and 14, 90.1 with 4 and 15, 93.0 with 8 and 15.)
constexpr float MOST_BF16 = 14.0f, MOST_F16 = 15.0f;
constexpr int MOST_LIFT = 14;

struct AttnParams {
  CUtensorMap mq, mk, mv, mkn, mvn;  // queries, cache (or prompt) K and V, staged K and V
  uint16_t* out;
  const int32_t* table;
  const int32_t* lens;    // seq_lens, pos or cu_seqlens
  const int32_t* parent;
  int32_t* status;
  float* part_o;          // partial outputs  [2 * CTAs][rows][DP / 4] x 4, columns outermost
  float2* part_ml;        // their maxima and sums [2 * CTAs][rows]
  int4* desc;             // [CTAs] what each CTA's first and last segments are (DESC_*)
  float c;                // scale * log2(e)
  float lift;             // fp16: weight of a row's maximum (log2)
  int kind;
  int B, N, Hq, Hkv, D, G;
  int LH, head0, num_pages, page, cols, sink, window, T;
  int box;                // page rows of one copy
  int tpt;                // tokens per query tile, floor(128 / G)
  int q_rows;             // rows of one query copy
  int MT;                 // items per KV head (TREE, RING)
  int whole_tiles;        // no item is cut when none has more tiles than this (TREE, RING)
  int join;               // and some may have, by the cache's extent
  int withhold;           // failure-handling test: CTA 0's second stage never fills
};

__device__ __forceinline__ void set_status(int32_t* status, int bits) {
  if (status && bits) atomicOr(status, bits);
}
__device__ __forceinline__ unsigned long long globaltimer() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void mbar_init(uint32_t bar, unsigned count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The same by one lane of a warp, without a branch that would split it.
__device__ __forceinline__ void mbar_arrive_if(uint32_t bar, bool on) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %1, 0;\n"
      " @p mbarrier.arrive.shared::cta.b64 _, [%0];\n}" ::"r"(bar), "r"(uint32_t(on))
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_tx(uint32_t bar, unsigned bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(SUSPEND_HINT_NS)
      : "memory");
  return ok != 0;
}
// Whether the phase has ended, without a wait.
__device__ __forceinline__ bool mbar_test(uint32_t bar, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait for a phase: false once the CTA gave up, or after one second,
// which reports SV_ST_TIMEOUT and makes the CTA's other waits give up too.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, unsigned parity, int32_t* status,
                                          volatile int* abort) {
  if (mbar_try(bar, parity)) return true;
  const unsigned long long t0 = globaltimer();
  for (;;) {
    if (mbar_try(bar, parity)) return true;
    if (*abort) return false;
    if (globaltimer() - t0 > WAIT_LIMIT_NS) {
      *abort = 1;
      set_status(status, SV_ST_TIMEOUT);
      return false;
    }
  }
}
// The same for a wait as long as an item: the second counts from the last change of
// `moving`'s phase, of a barrier that turns while the CTA gets on.  (Only for the plan,
// which is ahead: with the longer loop in every wait, 64 trees 224 -> 238 us.)
__device__ __forceinline__ bool mbar_wait_moving(uint32_t bar, unsigned parity, uint32_t moving,
                                                 int32_t* status, volatile int* abort) {
  unsigned long long t0 = globaltimer();
  bool phase = mbar_test(moving, 0);
  for (;;) {
    if (mbar_try(bar, parity)) return true;
    if (*abort) return false;
    if (mbar_test(moving, 0) != phase) {
      phase = !phase;
      t0 = globaltimer();
    }
    if (globaltimer() - t0 > WAIT_LIMIT_NS) {
      *abort = 1;
      set_status(status, SV_ST_TIMEOUT);
      return false;
    }
  }
}
// A wait by a whole warp, all lanes of which get one answer.
__device__ __forceinline__ bool warp_wait(uint32_t bar, unsigned parity, int32_t* status,
                                          volatile int* abort) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, status, abort)) != 0;
}

// Tiled copies global -> shared; a row past a map's extent arrives as zeros.
// The innermost coordinate is 0 or 64 elements: 16-byte boundaries.
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x,
                                       int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst), "l"(m), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x,
                                       int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst), "l"(m), "r"(bar), "r"(x), "r"(y),
      "r"(z), "r"(w)
      : "memory");
}

// Tensor-core products.  Tiles lie in shared memory as 64-element (128-byte)
// wide blocks of 128 rows in the 128-byte swizzle, one block after another.
// A descriptor's low word has the address; the high word is a constant of the
// operand's order, so that only the low words have to be moved for a product.
// K-major operand (queries, keys): rows 128 bytes apart, 8-row groups 1024.
constexpr uint32_t DESC_HI = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_rows(uint32_t addr) { return (addr >> 4) | (1u << 16); }
// MN-major operand (values: the 64 dimensions of a block are contiguous):
// 8-key groups 1024 bytes apart, 64-dimension blocks `blocks` bytes.  (0: a
// head of at most 64 dimensions taken twice to make up the 128 rows of V^T;
// the second half of O^T is not read.)
__device__ __forceinline__ uint32_t desc_cols(uint32_t addr, uint32_t blocks) {
  return (addr >> 4) | (blocks >> 4 << 16);
}
__device__ __forceinline__ uint32_t instr_desc(int bf16, bool a_cols, bool b_cols, int n) {
  return (1u << 4) | (uint32_t(bf16) << 7) | (uint32_t(bf16) << 10) | (a_cols ? 1u << 15 : 0u) |
         (b_cols ? 1u << 16 : 0u) | (uint32_t(n >> 3) << 17) | (uint32_t(TILE >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.u32 p, %4, 0;\n"
      " mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}" ::"r"(d), "r"(a), "r"(b),
      "r"(idesc), "r"(accumulate), "n"(DESC_HI)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 db;\n setp.ne.u32 p, %4, 0;\n mov.b64 db, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}" ::"r"(d), "r"(a), "r"(b),
      "r"(idesc), "r"(accumulate), "n"(DESC_HI)
      : "memory");
}
// One lane of the (converged) warp: the form in which the compiler knows that a
// single thread issues, and keeps the products' descriptors in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}"
               : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void tc_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// Tensor-memory loads, stores and their waits are instructions of a whole, converged
// warp.  What stands before them may go by lane (mask bits found along a tree path,
// output stores, one lane's arrival at a barrier), and the language promises no
// convergence after that: hence a warp sync in each of them, but for those (<false>) that
// stand behind one with nothing that goes by lane in between: a pair's tile has eleven,
// and 8192 tokens take 334 us with a sync in each, 319 with the two that it needs.
template <bool SYNC = true>
__device__ __forceinline__ void tm_wait_st() {
  if (SYNC) __syncwarp();
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// 32 columns of the warp's 32 lanes, one row per thread.
template <bool SYNC = true>
__device__ __forceinline__ void tm_ld32(uint32_t addr, uint32_t (&r)[32]) {
  if (SYNC) __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
      "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
// Waits for the warp's TMEM loads; passing the registers through keeps their
// uses behind the wait.
#define TM_REGS(r)                                                                              \
  "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),           \
      "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),   \
      "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]),             \
      "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]),             \
      "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
template <bool SYNC = true>
__device__ __forceinline__ void tm_wait_ld(uint32_t (&r)[32]) {
  if (SYNC) __syncwarp();
  asm volatile("tcgen05.wait::ld.sync.aligned;" : TM_REGS(r)::"memory");
}
__device__ __forceinline__ void tm_loaded(uint32_t (&r)[32]) {  // after tm_wait_ld
  asm volatile("" : TM_REGS(r)::"memory");
}
__device__ __forceinline__ void tm_st32(uint32_t addr, const uint32_t (&r)[32]) {
  __syncwarp();
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, "
      "%21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tm_ld8(uint32_t addr, uint32_t (&r)[8]) {
  __syncwarp();
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                      "=r"(r[6]), "=r"(r[7])
               : "r"(addr));
}
__device__ __forceinline__ void tm_ld16(uint32_t addr, uint32_t (&r)[16]) {
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                      "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                      "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(addr));
}
template <bool SYNC = true>
__device__ __forceinline__ void tm_st16(uint32_t addr, const uint32_t (&r)[16]) {
  if (SYNC) __syncwarp();
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                      "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
                      "r"(r[13]), "r"(r[14]), "r"(r[15])
               : "memory");
}
template <int N>
__device__ __forceinline__ void tm_ldn(uint32_t addr, uint32_t (&r)[N]) {
  if constexpr (N == 8) tm_ld8(addr, r);
  else if constexpr (N == 16) tm_ld16(addr, r);
  else tm_ld32(addr, r);
}
template <int N>
__device__ __forceinline__ void tm_stn(uint32_t addr, const uint32_t (&r)[N]) {
  if constexpr (N == 16) tm_st16(addr, r);
  else tm_st32(addr, r);
}
template <int N>
__device__ __forceinline__ void tm_loadedn(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i])::"memory");
}
template <int N>
__device__ __forceinline__ void tm_waitn(uint32_t (&r)[N]) {
  __syncwarp();
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  tm_loadedn<N>(r);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two 32-bit multiply-adds, or additions, in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mov.b64 c, {%6, %7};\n fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
template <bool BF>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  uint32_t r;
  if (BF) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void group_sync(int id, int n) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
__device__ __forceinline__ int group_or(int id, int n, int x) {
  int r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.s32 p, %3, 0;\n"
      " barrier.cta.red.or.pred q, %1, %2, p;\n selp.s32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"(id), "r"(n), "r"(x)
      : "memory");
  return r;
}

// -------------------------------------------------------------- what a CTA works on

__device__ __forceinline__ int tiles_of(int n) { return (n + TILE - 1) / TILE; }

// A segment: key tiles j0 .. j0 + n - 1 of the nt tiles of an item.  An item is
// the query rows of one KV head that share the tiles: tokens mt * tokens(item)
// on of request b, with the Hq / Hkv query heads of h.
struct Seg {
  int b, h, mt, j0, n, nt;
  int len;    // cache entries (TREE, RING; 0 when bad), or tokens of the sequence
  int bad;    // SV_ST_BAD_LENGTH for a length outside its range
  int ring;   // RING: the ring slot after the newest entry, which holds the oldest; -1: none
  int full;   // and whether it does
  int start;  // first packed row (PROMPT)
  // PROMPT: `near` tiles over the sinks that have left the window (of every
  // token of the item), then tiles from key `first` to the last token's
  int near, first, last;
};

// Tile j of a segment's item: its first key (of the cache, the staged entries or
// the sequence) and its keys.
struct Keys { int k0, n; bool staged; };
template <bool PR>
__device__ __forceinline__ Keys keys_of(const AttnParams& A, const Seg& s, int j) {
  if (PR) {
    if (j < s.near) return {j * TILE, min(TILE, A.sink - j * TILE), false};
    const int k0 = s.first + (j - s.near) * TILE;
    return {k0, min(TILE, s.last + 1 - k0), false};
  }
  const int ct = tiles_of(s.len);
  if (j < ct) return {j * TILE, min(TILE, s.len - j * TILE), false};
  return {(j - ct) * TILE, min(TILE, A.N - (j - ct) * TILE), true};
}
// The products take keys in sixteens.
__device__ __forceinline__ int width_of(const Keys& k) { return (k.n + 15) & ~15; }

// Cache entries of request b (0 with `bad` set for a length out of range).
__device__ __forceinline__ int cache_len(const AttnParams& A, int b, int& bad, int& pos) {
  const long long n = __ldg(A.lens + b);
  pos = int(n);
  if (A.kind == TREE) {
    bad = n < 0 || n > (long long)A.cols * A.page || n > MAX_KEYS ? SV_ST_BAD_LENGTH : 0;
    return bad ? 0 : int(n);
  }
  bad = n < 0 || n > 0x7fffffffLL - A.N ? SV_ST_BAD_LENGTH : 0;
  const long long C = (long long)A.sink + A.window;
  return bad ? 0 : int(n < C ? n : C);
}

// The segments of a CTA, in order, found by a whole warp.
// TREE and RING: the tiles of all items, in the order request, KV head, item of
// the head, are cut into equal runs, one per CTA; an item cut by a run's end is
// joined by the second kernel, or (whole) is taken by the CTA of its first
// tile.  An item counts ITEM_COST tiles more than it has
// (its queries, output and first tile's latency).
// PROMPT: whole items, one per CTA of the grid; a CTA that is done takes over
// the next one that has not been launched.  A sequence's last tokens (whose
// items are the longest) come first.
template <bool PAIR, bool PR>
struct Cursor;

template <bool PAIR>
struct Cursor<PAIR, false> {
  int b, item, j, nt, len, bad, pos;
  bool whole;      // items are not cut
  long long left;  // tiles of the run ahead

  __device__ void open(const AttnParams& A, int b0, long long at, long long count, bool w) {
    whole = w;
    left = count;
    if (count <= 0) return;
    b = b0;
    len = cache_len(A, b, bad, pos);
    nt = tiles_of(len) + tiles_of(A.N);
    const int cost = nt + ITEM_COST;
    item = at >> 32 ? int(at / cost) : int(uint32_t(at) / uint32_t(cost));
    j = int(at - (long long)item * cost);
    if (whole && j > 0) {  // an earlier CTA's item
      left -= cost - j;
      step(A);
    }
  }
  __device__ void step(const AttnParams& A) {  // to the next item
    j = 0;
    if (++item == A.MT * A.Hkv) {
      item = 0;
      if (left <= 0) return;
      ++b;
      len = cache_len(A, b, bad, pos);
      nt = tiles_of(len) + tiles_of(A.N);
    }
  }
  __device__ bool next(const AttnParams& A, Seg& s) {
    for (;;) {
      if (left <= 0) return false;
      if (j >= nt) {  // the item's fixed cost, counted behind its tiles
        left -= nt + ITEM_COST - j;
        step(A);
        continue;
      }
      s.b = b;
      s.h = item / A.MT;
      s.mt = item - s.h * A.MT;
      s.j0 = j;
      s.n = whole || left >= nt - j ? nt - j : int(left);
      s.nt = nt;
      s.len = len;
      s.bad = bad;
      s.ring = -1;
      s.full = 0;
      if (A.kind == RING && !bad && pos > A.sink) {
        s.ring = (pos - A.sink) % A.window;
        s.full = pos - A.sink >= A.window;
      }
      j += s.n;
      left -= s.n;
      return true;
    }
  }
};

template <bool PAIR>
struct Cursor<PAIR, true> {
  long long cum, incl;        // items before the 32 sequences, and up to the lane's
  int wb, w_start, w_len;     // the 32 sequences from wb on, one per lane

  __device__ void load_window(const AttnParams& A, bool report) {
    const int lane = int(threadIdx.x) & 31, s = wb + lane;
    w_start = w_len = 0;
    if (s < A.B) {
      const long long lo = __ldg(A.lens + s), hi = __ldg(A.lens + s + 1);
      if (lo < 0 || hi < lo || hi > A.T) {
        if (report) set_status(A.status, SV_ST_BAD_LENGTH);
      } else {
        w_start = int(lo);
        w_len = int(hi - lo);
      }
    }
    const int tpi = PAIR ? 2 * A.tpt : A.tpt;
    incl = (long long)((w_len + tpi - 1) / tpi) * A.Hkv;
    for (int x = 1; x < 32; x <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, x);
      if (lane >= x) incl += y;
    }
  }
  __device__ void open(const AttnParams& A, bool report) {
    cum = 0;
    wb = 0;
    load_window(A, report);
  }
  // Item i; false past the last.  The search goes on from the item before, and anew when
  // i lies before that one's sequences: in which order blocks are taken over is not
  // promised.
  __device__ bool item(const AttnParams& A, long long i, Seg& s, bool report) {
    if (i < cum) open(A, report);
    for (;;) {
      const long long total = __shfl_sync(0xffffffffu, incl, 31);
      if (i < cum + total) break;
      cum += total;
      wb += 32;
      if (wb >= A.B) {
        incl = 0;  // nothing in the windows past the last
        return false;
      }
      load_window(A, report);
    }
    const unsigned hit = __ballot_sync(0xffffffffu, i < cum + incl);
    const int src = __ffs(int(hit)) - 1;
    const long long before = src ? __shfl_sync(0xffffffffu, incl, src - 1) : 0;
    s.b = wb + src;
    s.start = __shfl_sync(0xffffffffu, w_start, src);
    s.len = __shfl_sync(0xffffffffu, w_len, src);
    const int tpi = PAIR ? 2 * A.tpt : A.tpt;
    const long long r = i - cum - before;
    const int back = r >> 32 ? int(r / A.Hkv) : int(uint32_t(r) / uint32_t(A.Hkv));
    s.h = int(r - (long long)back * A.Hkv);
    s.mt = (s.len + tpi - 1) / tpi - 1 - back;
    s.bad = 0;
    s.j0 = 0;
    const int q0 = s.mt * tpi, q1 = min(q0 + tpi, s.len) - 1;
    s.first = max(0, q0 - A.window + 1);  // (window >= 1: no overflow)
    s.last = q1;
    if (A.sink >= s.first) s.first = 0;
    s.near = s.first ? tiles_of(A.sink) : 0;
    s.n = s.nt = s.near + tiles_of(q1 + 1 - s.first);
    return true;
  }
};

// Copies of a segment in the order in which the product warp takes them.
// PAIR (two query tiles, every key tile used by both): K0 V0 K1 V1 ...
// otherwise (one query tile, even and odd key tiles in two streams, so that
// one stream's product runs under the other's softmax): K0 K1 V0 K2 V1 ...
template <bool PAIR>
__device__ __forceinline__ int k_order(int j) { return PAIR ? 2 * j : (j ? 2 * j - 1 : 0); }
template <bool PAIR>
__device__ __forceinline__ int v_order(int j, int n) {
  return PAIR ? 2 * j + 1 : (j < n - 1 ? 2 * j + 2 : 2 * n - 1);
}

// Bits a .. b - 1 of the 32 keys from k0 on.
__device__ __forceinline__ uint32_t span(int a, int b, int k0) {
  a = max(a - k0, 0);
  b = min(b - k0, 32);
  if (a >= b) return 0;
  return (0xffffffffu >> (32 - b)) & (0xffffffffu << a);
}

// The three layouts of an item's products, by the rows (tokens x query heads of
// a KV head) that share its keys:
//   NQ == 0, PAIR: more than 128 rows.  Two tiles of 128 rows; S = Q K^T has a
//     row per TMEM lane, every key tile serves both.
//   NQ == 0, !PAIR: 33 to 128 rows.  One such tile, in two streams.
//   NQ > 0: at most NQ rows.  The products are turned over, S^T = K Q^T and
//     O^T = V^T P^T, so that the lanes hold keys (dimensions) and the few rows
//     are columns: every thread has work however few the rows are, and the
//     products cost less.  (1024 requests of 12 rows per item: 444 us with a row
//     per lane, 260 so, when both were first built.  Later: 64 requests of 5000, 24 rows
//     of 128 dimensions, 207 us so and 215 with a row per lane, 32 rows 210 and 217;
//     but 64 rows, for which a warp agrees on 64 maxima, 258 and 218.)
constexpr int CTRL_BYTES = 3 * 1024;  // what 227 KB leave beside seven tiles of 32 KB
template <int DP, int NQ>
struct Smem {
  static constexpr int BYTES = TILE * DP * 2;                    // a tile of keys or values
  static constexpr int Q_BYTES = (NQ ? NQ : TILE) * DP * 2;      // a tile of queries
  static constexpr int P_BYTES = NQ * TILE * 2;                  // weights of a stream (NQ > 0)
  static constexpr int P_AT = 2 * Q_BYTES;
  static constexpr int STAGE_AT = P_AT + 2 * P_BYTES;
  static constexpr int FIT = (229376 - STAGE_AT) / BYTES;
  static constexpr int STAGES = FIT < 12 ? FIT : 12;
  static constexpr int CTRL = STAGE_AT + STAGES * BYTES;         // offset of the control part
  static constexpr int TOTAL = CTRL + CTRL_BYTES;
};
template <bool V>
struct Yes { static constexpr bool value = V; };
template <int NQ, class A, class B>
struct Either { using T = A; };
template <class A, class B>
struct Either<0, A, B> { using T = B; };
constexpr int SEGS = 4;        // segments planned ahead
constexpr int PROMPT_SEGS = 2; // of prompts, whose CTAs take items as they finish others
template <bool PAIR>
struct Exchange {              // NQ == 0: softmax state exchanged between the streams
  float2 ml[2][PAIR ? 1 : TILE];
};
template <int NQ>
struct Few {                   // NQ > 0, per stream and column
  uint32_t sees[2][NQ];            // columns that see a staged entry
  alignas(16) float nmc[2][NQ];    // the lift less the running maximum, in base-2 units; -inf: none yet
  alignas(16) float fac[2][NQ];    // rescaling, and at the end the streams' shares
  float sums[8][NQ];               // per warp, at the end
};
template <int NQ, bool PAIR>
struct Ctrl {
  // barriers: stages filled and free, queries, scores, weights (a pair's first half, all),
  // output complete, segments planned and taken, the end after a wait gave up, another item
  unsigned long long full[12], empty[12], q_full[2], q_empty[2], s_full[2], p_half[2], p_full[2],
      o_full[2], seg_full[SEGS], seg_empty[SEGS], drain, next_full;
  alignas(16) uint4 next;    // PROMPT: the answer to a request for another item
  Seg seg[SEGS];
  long long start_at;
  int start_b, abort;
  uint32_t tmem;
  uint8_t parent[2][NQ ? NQ : PAIR ? MAX_N : TILE];  // one copy per softmax warpgroup
  union {
    typename Either<NQ, Few<NQ>, Exchange<PAIR>>::T x;
    struct { long long sum[THREADS / 32]; int most[THREADS / 32]; } scan;
  };
  unsigned long long out_at[NQ ? NQ : 1];  // NQ > 0: elements from an item's output to a column's
};
static_assert(sizeof(Ctrl<0, true>) <= CTRL_BYTES && sizeof(Ctrl<0, false>) <= CTRL_BYTES &&
                  sizeof(Ctrl<16, false>) <= CTRL_BYTES && sizeof(Ctrl<32, false>) <= CTRL_BYTES,
              "control part");

// desc[cta]: x = flags, y = item (of its request) and z = request of the first segment
constexpr int DESC_THROUGH = 1 << 29;  // the first segment starts inside its item and runs to
                                       // the CTA's end without finishing it
constexpr int DESC_OUT = 1 << 28;      // the last segment leaves its item unfinished
constexpr int DESC_LAST1 = 1 << 27;    // the last segment's partials are in slot 1

// The largest of N values, in eight chains of three-operand maxima.
template <int N, class F>
__device__ __forceinline__ float max_of(F v) {
  float a[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) a[k] = v(k);
#pragma unroll
  for (int i = 8; i + 16 <= N; i += 16)
#pragma unroll
    for (int k = 0; k < 8; ++k) a[k] = fmaxf(fmaxf(a[k], v(i + 2 * k)), v(i + 2 * k + 1));
#pragma unroll
  for (int k = 0; k < 8; ++k) a[k] = fmaxf(a[k], v(N - 8 + k));  // (N mod 16 is 0: the last eight)
  return fmaxf(fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3])),
               fmaxf(fmaxf(a[4], a[5]), fmaxf(a[6], a[7])));
}

// A step of a 4 x 4 transposition between lanes: the lane without bit x keeps
// `a` and gets its partner's `a` as its `b`; the other the reverse.
__device__ __forceinline__ void swap_pieces(uint4& a, uint4& b, int x, int lane) {
  const bool up = lane & x;
  uint4 give = up ? a : b;
  give.x = __shfl_xor_sync(0xffffffffu, give.x, x);
  give.y = __shfl_xor_sync(0xffffffffu, give.y, x);
  give.z = __shfl_xor_sync(0xffffffffu, give.z, x);
  give.w = __shfl_xor_sync(0xffffffffu, give.w, x);
  if (up) a = give;
  else b = give;
}

// Sums of the columns over a warp's 32 lanes: lane i gets column i's (i mod 16's
// with 16 columns) in v[0].
template <int NQ>
__device__ __forceinline__ void sum_columns(float* v, int lane) {
#pragma unroll
  for (int x = NQ / 2; x; x >>= 1) {
    const bool up = lane & x;
#pragma unroll
    for (int i = 0; i < x; ++i) {
      const float give = up ? v[i] : v[i + x], keep = up ? v[i + x] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, x);
    }
  }
  if (NQ == 16) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 16);
}

// One tile's softmax with keys on the lanes: thread `key` takes its key's
// scores of all NQ columns (S^T, TMEM columns from ts), adds their weights to
// lq and stores them, rounded, as column `key` of P (a K-major operand of two
// 64-key blocks in the 128-byte swizzle).  `sees`: the columns that see the
// key.  All keys of a tile use one maximum per column; it is raised, the sums
// and O (columns from to) rescaled, when a weight would exceed 2^most.
template <int NQ, bool BF>
__device__ __forceinline__ void softmax_few(const AttnParams& A, Ctrl<NQ, false>& C, int st,
                                            int key, uint32_t ts, uint32_t to, uint32_t sees,
                                            bool masked, bool started, bool& unset, float* lq,
                                            unsigned char* pbuf) {
  constexpr float MOST = BF ? MOST_BF16 : MOST_F16;
  const float lift = BF ? 0.0f : A.lift;
  const int lane = key & 31, warp = key >> 5;
  float* const nmc = C.x.nmc[st];
  const float2 c2 = make_float2(A.c, A.c);
  uint32_t r[NQ];
  auto load = [&] {
    tm_ldn<NQ>(ts, r);
    tm_waitn<NQ>(r);
    if (masked) {
#pragma unroll
      for (int q = 0; q < NQ; ++q)
        if (!(sees >> q & 1)) r[q] = 0xff800000u;
    }
  };
  // the weights' exponents in place of the scores, and the largest
  auto exponents = [&] {
    float over = -INFINITY;
#pragma unroll
    for (int q = 0; q < NQ; q += 4) {
      const float4 n = *reinterpret_cast<const float4*>(nmc + q);
      const float2 a = fma2(make_float2(__uint_as_float(r[q]), __uint_as_float(r[q + 1])),
                            c2, make_float2(n.x, n.y));
      const float2 b =
          fma2(make_float2(__uint_as_float(r[q + 2]), __uint_as_float(r[q + 3])), c2,
               make_float2(n.z, n.w));
      r[q] = __float_as_uint(a.x);
      r[q + 1] = __float_as_uint(a.y);
      r[q + 2] = __float_as_uint(b.x);
      r[q + 3] = __float_as_uint(b.y);
      over = fmaxf(over, fmaxf(fmaxf(a.x, a.y), fmaxf(b.x, b.y)));
    }
    return over;
  };
  load();
  bool raise = !started || unset;
  if (!raise) {
    raise = group_or(1 + st, TILE, exponents() > MOST);
    __syncwarp();
    if (raise) load();
  }
  if (raise) {
    float* const wmax = reinterpret_cast<float*>(pbuf);  // [warp][NQ]; P is free until stored
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      float t;
      asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;"
                   : "=f"(t)
                   : "f"(__uint_as_float(r[q])));
      if (lane == q) wmax[warp * NQ + q] = t;
    }
    group_sync(1 + st, TILE);
    int none = 0;
    if (key < NQ) {
      const float t = fmaxf(fmaxf(wmax[key], wmax[NQ + key]),
                            fmaxf(wmax[2 * NQ + key], wmax[3 * NQ + key])) * A.c;
      float old = started ? -nmc[key] : INFINITY, f = 1.0f;
      if (old == INFINITY) {
        if (t > -INFINITY) old = t - lift;
      } else if (t - old > MOST) {
        f = ex2(old - (t - lift));
        old = t - lift;
      }
      nmc[key] = -old;
      C.x.fac[st][key] = f;
      none = old == INFINITY;
    }
    unset = group_or(1 + st, TILE, none);
    __syncwarp();
    if (started) {
#pragma unroll
      for (int q = 0; q < NQ; ++q) lq[q] *= C.x.fac[st][q];
      uint32_t o[NQ];
      tm_ldn<NQ>(to, o);
      tm_waitn<NQ>(o);
#pragma unroll
      for (int q = 0; q < NQ; ++q)
        o[q] = __float_as_uint(__uint_as_float(o[q]) * C.x.fac[st][q]);
      tm_stn<NQ>(to, o);
      tm_wait_st();
    }
    exponents();
  }
  // key k of row q: block k / 64, byte (k % 64) * 2 of the 128-byte row, its
  // 16-byte piece exchanged with that of q % 8
  unsigned char* const prow = pbuf + (key >> 6) * (NQ * 128) + (key & 7) * 2;
  const int piece = (key & 63) >> 3;
#pragma unroll
  for (int q = 0; q < NQ; q += 2) {
    const float2 p =
        make_float2(ex2(__uint_as_float(r[q])), ex2(__uint_as_float(r[q + 1])));
    const float2 l = add2(make_float2(lq[q], lq[q + 1]), p);
    lq[q] = l.x;
    lq[q + 1] = l.y;
    const uint32_t w = pack16<BF>(p.x, p.y);
    *reinterpret_cast<uint16_t*>(prow + q * 128 + ((piece ^ (q & 7)) << 4)) = uint16_t(w);
    *reinterpret_cast<uint16_t*>(prow + (q + 1) * 128 + ((piece ^ ((q + 1) & 7)) << 4)) =
        uint16_t(w >> 16);
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// The attention kernel, one CTA per SM.  Warps:
//   plan      the segments, a few ahead, with the loads and divisions they take
//   copy      queries and key and value tiles by TMA into a ring of stages
//   products  one thread: S and O += P V on the tensor cores (S, P and O in TMEM;
//             the turned layout's P in shared memory), and the waits before them
//   softmax   two warpgroups, one per stream.  A row per lane: the maximum and sum
//             of a row in its thread, P over S as 16-bit weights.  Keys on the
//             lanes: a maximum per column, agreed on by the warpgroup.
// The weights are rounded once to the storage type (half a step each); their sum
// l is taken before that, in 32 bits.
template <int DP, int NQ, bool PAIR, bool PR, bool BF>
__global__ void __launch_bounds__(THREADS, 1) sv_attn(const __grid_constant__ AttnParams A) {
  static_assert(!(NQ && (PAIR || PR)), "few rows make one tile, and prompts have many");
  using SM = Smem<DP, NQ>;
  constexpr int STAGES = SM::STAGES, BYTES = SM::BYTES, HALVES = DP / 64;
  constexpr int ROWS = NQ ? NQ : PAIR ? 2 * TILE : TILE;
  constexpr int TM_COLS = NQ ? 256 : 512;               // TMEM: S of both streams, then O
  constexpr int S_COLS = NQ ? 64 : 128, O_AT = TM_COLS / 2;
  extern __shared__ __align__(1024) unsigned char smem[];
  Ctrl<NQ, PAIR>& C = *reinterpret_cast<Ctrl<NQ, PAIR>*>(smem + SM::CTRL);
  const uint32_t base = smem_addr(smem);
  const int tid = int(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  auto bar = [&](unsigned long long* p) { return smem_addr(p); };

  // ---- set-up: barriers, TMEM, and where this CTA's run of tiles starts
  if (tid == 0) {
    for (int i = 0; i < STAGES; ++i) {
      // (withheld: one arrival too many, and every wait for that stage runs out)
      mbar_init(bar(&C.full[i]), A.withhold && blockIdx.x == 0 && i == 1 ? 2 : 1);
      mbar_init(bar(&C.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(&C.q_full[i]), 1);
      mbar_init(bar(&C.q_empty[i]), 1);
      mbar_init(bar(&C.s_full[i]), 1);
      mbar_init(bar(&C.p_half[i]), 4);
      mbar_init(bar(&C.p_full[i]), 4);
      mbar_init(bar(&C.o_full[i]), 1);
    }
    for (int i = 0; i < SEGS; ++i) {
      mbar_init(bar(&C.seg_full[i]), 1);
      mbar_init(bar(&C.seg_empty[i]), COPY_WARP + 2);  // every warp that reads it
    }
    mbar_init(bar(&C.drain), 1);
    mbar_init(bar(&C.next_full), 1);
    C.abort = 0;
    C.start_b = 0;
    C.start_at = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == MMA_WARP) {
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&C.tmem)),
                 "n"(TM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (NQ) {
    if (tid < NQ) C.out_at[tid] = ((unsigned long long)(tid / A.G) * A.Hq + tid % A.G) * A.D;
    // columns past the item's rows: finite, and never used
    for (int i = tid; i < SM::P_AT / 16; i += THREADS)
      reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  long long run = 0;  // tiles of this CTA (TREE, RING)
  bool whole_items = false;
  if (!PR) {
    // thread t sums requests t * per .. of the batch
    const int per = (A.B + THREADS - 1) / THREADS;
    const int b0 = min(tid * per, A.B), b1 = min(b0 + per, A.B);
    const long long items = (long long)A.MT * A.Hkv;
    long long mine = 0;
    int bad, pos, most = 0;
    for (int b = b0; b < b1; ++b) {
      const int nt = tiles_of(cache_len(A, b, bad, pos)) + tiles_of(A.N);
      mine += items * (nt + ITEM_COST);
      most = max(most, nt);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    long long incl = mine;
    for (int x = 1; x < 32; x <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, x);
      if (lane >= x) incl += y;
    }
    if (lane == 31) {
      C.scan.sum[warp] = incl;
      C.scan.most[warp] = most;
    }
    __syncthreads();
    long long total = 0, before = incl - mine;
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) before += C.scan.sum[w];
      total += C.scan.sum[w];
      most = max(most, C.scan.most[w]);
    }
    whole_items = most <= A.whole_tiles;
    const long long ctas = min((long long)gridDim.x, total), c = blockIdx.x;
    const long long each = total / ctas, more = total - each * ctas;
    const long long lo = c < ctas ? c * each + min(c, more) : total;
    const long long hi = c < ctas ? lo + each + (c < more) : total;
    run = hi - lo;
    if (run > 0 && lo >= before && lo < before + mine) {
      long long at = before;
      for (int b = b0; b < b1; ++b) {
        const long long t =
            items * (tiles_of(cache_len(A, b, bad, pos)) + tiles_of(A.N) + ITEM_COST);
        if (lo < at + t) {
          C.start_b = b;
          C.start_at = lo - at;
          break;
        }
        at += t;
      }
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  // the join may be launched now: its blocks find room when this grid's CTAs
  // leave, and wait for the last of them before they read anything
  if (!PR && A.join) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = C.tmem;
  const int start_b = C.start_b;
  const long long start_at = C.start_at;
  volatile int* abort = &C.abort;
  // the planned segments: a ring, read by every other role's warps
  constexpr int AHEAD = PR ? PROMPT_SEGS : SEGS;
  auto seg_wait = [&](int i) {
    return warp_wait(bar(&C.seg_full[i % AHEAD]), (i / AHEAD) & 1, A.status, abort);
  };
  auto seg_done = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(&C.seg_empty[i % AHEAD]));
  };

  if (warp < 8) {
    __syncwarp();
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SOFTMAX_REGS));
    // ------------------------------------------------------------ softmax
    const int st = warp >> 2;             // the stream of this warpgroup
    const int row = tid & (TILE - 1);     // query row of the tile, and key of a value tile
    const int rt = row / A.G, rg = row - rt * A.G;
    const uint32_t lanes = uint32_t(warp & 3) << 21;  // this warp's TMEM lanes
    const uint32_t ts = tmem + lanes + st * S_COLS, to = tmem + lanes + O_AT + st * S_COLS;
    uint32_t idx = 0;
    int segs = 0, parent_b = -1, parent_bad = 0;
    unsigned s_use = 0, o_use[2] = {0, 0};
    bool ok = true;
    int d_flags = 0, d_item = 0, d_b = 0;
    for (;;) {
      // The warps go on, or stop after a wait that gave up, together; and (two
      // streams over one O) both have read O before either lets it be overwritten.
      ok = ok && seg_wait(segs);
      if (group_or(PAIR ? 1 + st : 3, PAIR ? TILE : 2 * TILE, !ok)) break;
      tc_after();
      const Seg& s = C.seg[segs % AHEAD];
      const int n = s.n;
      if (n == 0) break;
      const int tpi = PAIR ? 2 * A.tpt : A.tpt;
      const int tok = s.mt * tpi + (PAIR ? st * A.tpt : 0) + rt;  // this row's token
      const int tokens = PR ? s.len : A.N;
      const bool active = rt < A.tpt && tok < tokens;
      const bool warp_active = __any_sync(0xffffffffu, active);
      const int ct = tiles_of(s.len);
      int bad = s.bad;
      if (!PR && A.kind == TREE) {
        // pages in use by this segment, and the parent array
        int pages_bad = 0;
        const int t1 = min(s.len, (s.j0 + n) * TILE);
        if (s.j0 * TILE < t1)
          for (int c = s.j0 * TILE / A.page + row; c <= (t1 - 1) / A.page; c += TILE) {
            const int pg = __ldg(A.table + size_t(s.b) * A.cols + c);
            pages_bad |= pg < 0 || pg >= A.num_pages;
          }
        if (A.parent && s.b != parent_b && s.j0 + n > ct) {
          if constexpr (NQ > 0)
            if (row < NQ) C.x.sees[st][row] = 0;
          int wrong = 0;
          for (int i = row; i < A.N; i += TILE) {
            const int p = __ldg(A.parent + size_t(s.b) * A.N + i);
            const bool w = i == 0 ? p != -1 : (p < 0 || p >= i);
            wrong |= w;
            C.parent[st][i] = uint8_t(w || i == 0 ? 0 : p);
          }
          parent_bad = group_or(1 + st, TILE, wrong) ? SV_ST_BAD_TOKEN : 0;
          parent_b = s.b;
          if constexpr (NQ > 0) {  // column `row` sees its token and those above it
            if (row < A.N * A.G)
              for (int i = row / A.G;; i = C.parent[st][i]) {
                atomicOr(&C.x.sees[st][i], 1u << row);
                if (i == 0) break;
              }
            group_sync(1 + st, TILE);
          }
        }
        if (group_or(1 + st, TILE, pages_bad)) bad |= SV_ST_BAD_PAGE;
        if (s.j0 + n > ct && A.parent) bad |= parent_bad;
      }
      if (bad && tid == 0) set_status(A.status, bad);
      const int ring_at = PR ? -1 : s.ring;
      const bool ring_full = !PR && s.full;
      const int q0 = s.mt * tpi, q1 = min(q0 + tpi, tokens) - 1;  // the item's tokens
      const int w0 = q0 + (PAIR ? st * A.tpt : 0), w1 = min(w0 + A.tpt, tokens) - 1;  // the tile's

      const float lift = BF ? 0.0f : A.lift, raise = BF ? MOST_BF16 : MOST_F16 - A.lift;
      float m = -INFINITY, l = 0.0f;
      float lq[NQ ? NQ : 1];  // NQ > 0: this key's share of the columns' sums
      bool unset = true;      // NQ > 0: a column has seen nothing yet
#pragma unroll
      for (int q = 0; q < NQ; ++q) lq[q] = 0.0f;
      int done = 0;
      for (int jj = PAIR ? 0 : st; jj < n; jj += PAIR ? 1 : 2, ++done) {
        const int j = s.j0 + jj;
        const Keys ky = keys_of<PR>(A, s, j);
        const int k0 = ky.k0, w = width_of(ky);
        // does the tile need a mask, and value rows that no query of the item sees
        // (among the w that the products take) zeroed?
        bool masked = NQ == 0 ? (w & 31) != 0 : false, clean = ky.n < w, dead = row >= ky.n;
        if (PR) {
          masked |= clean;
          if (j >= s.near) masked |= k0 + w - 1 > w0 || (k0 <= w1 - A.window && k0 + w > A.sink);
        } else if (ky.staged) {
          masked = true;
          clean = dead = false;  // (rows past the staged entries arrived as zeros)
        } else {
          masked |= k0 + (NQ ? TILE : w) > s.len;
          if (ring_at >= 0) {
            const int a = A.sink + ring_at, e = ring_at + A.N - A.window;
            masked |= (k0 < a + A.N && k0 + w > a) || (e > 0 && k0 < A.sink + e && k0 + w > A.sink);
            if (ring_full) {
              clean |= a >= k0 && a < k0 + w;
              dead |= k0 + row == a;
            }
          }
        }
        dead = dead && row < w;
        // (With keys on the lanes the warps meet at barriers within a tile: after a
        // wait that gave up they walk the rest of the segment's tiles together.)
        ok = ok && warp_wait(bar(&C.s_full[st]), s_use & 1, A.status, abort);
        if (NQ == 0 && !ok) break;
        ++s_use;
        tc_after();
        // (The scores' keys have arrived, and so has every copy before them, among
        // them the last one into this tile's stage: its phase is the next.)
        if (clean && (!PAIR || st == 0)) {
          const uint32_t u = idx + v_order<PAIR>(jj, n);
          ok = ok && warp_wait(bar(&C.full[u % STAGES]), (u / STAGES) & 1, A.status, abort);
          if (NQ == 0 && !ok) break;
          if (ok && dead) {
            uint4* v =
                reinterpret_cast<uint4*>(smem + SM::STAGE_AT + (u % STAGES) * BYTES + row * 128);
#pragma unroll
            for (int x = 0; x < HALVES; ++x)
#pragma unroll
              for (int i = 0; i < 8; ++i) v[x * 1024 + i] = make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
        auto half_done = [&] {  // PAIR: the weights of the tile's first 64 keys are stored
          if (!PAIR) return;
          tm_wait_st<false>();
          tc_before();
          __syncwarp();
          mbar_arrive_if(bar(&C.p_half[st]), lane == 0);
        };
        if constexpr (NQ > 0) {
          // one key per thread, all rows
          uint32_t sees = ~0u;
          if (masked) {
            const int k = k0 + row;
            if (!ky.staged) {
              if (k >= s.len) {
                sees = 0;
              } else if (ring_at >= 0 && k >= A.sink) {
                int v = k - A.sink - ring_at;  // tokens that still have the slot in their window
                if (v < 0) v += A.window;
                if (v < A.N) sees = (1u << (v * A.G)) - 1;
              }
            } else if (k >= A.N) {
              sees = 0;
            } else {
              sees = A.parent ? C.x.sees[st][k] : ~0u << (k * A.G);
            }
          }
          softmax_few<NQ, BF>(A, C, st, row, ts, to, sees, masked, done > 0, unset, lq,
                          smem + SM::P_AT + st * SM::P_BYTES);
        } else if (!warp_active) {
          __syncwarp();
          half_done();
        } else {
          // the tile's keys that this row sees, 32 to a word
          auto visible = [&](uint32_t (&see)[4]) {
            if (PR) {
              // near tiles: the sinks; others: the window, and the sinks when they adjoin it
              const int lo = j < s.near ? 0 : tok - A.window + 1;
              const int hi = j < s.near ? A.sink : tok + 1, sk = min(A.sink, tok + 1);
#pragma unroll
              for (int x = 0; x < 4; ++x)
                see[x] = span(lo, hi, k0 + 32 * x) | span(0, sk, k0 + 32 * x);
            } else if (!ky.staged) {
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                see[x] = span(0, s.len, k0 + 32 * x);
                if (ring_at >= 0)
                  see[x] &= ~(span(A.sink + ring_at, A.sink + min(ring_at + tok + 1, A.window),
                                   k0 + 32 * x) |
                              span(A.sink, A.sink + ring_at + tok + 1 - A.window, k0 + 32 * x));
              }
            } else if (A.parent) {
#pragma unroll
              for (int x = 0; x < 4; ++x) see[x] = 0;
              for (int i = active ? tok : 0;; i = C.parent[st][i]) {
                const int y = i - k0;
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  if (y >= 32 * x && y < 32 * x + 32) see[x] |= 1u << (y & 31);
                if (i == 0) break;
              }
            } else {
#pragma unroll
              for (int x = 0; x < 4; ++x) see[x] = span(0, tok + 1, k0 + 32 * x);
            }
          };
          // the row's maximum, raised to mt when that is far above it, and O and l with it
          auto raise_to = [&](float mt) {
            if (done == 0) {
              m = mt;
            } else {
              const bool rise = active && (mt - m) * A.c > raise;  // (-inf before: always)
              if (__any_sync(0xffffffffu, rise)) {
                const float f = rise ? ex2((m - mt) * A.c) : 1.0f;
                if (rise) m = mt;
                l *= f;
#pragma unroll 1
                for (int x = 0; x < DP / 32; ++x) {
                  uint32_t o[32];
                  tm_ld32(to + x * 32, o);
                  tm_wait_ld(o);
#pragma unroll
                  for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                  tm_st32(to + x * 32, o);
                }
              }
            }
          };
          if constexpr (PAIR) {
            uint32_t r[4][32];
            __syncwarp();
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (x * 32 < w) tm_ld32<false>(ts + x * 32, r[x]);
            tm_wait_ld<false>(r[0]);
            tm_loaded(r[1]);
            tm_loaded(r[2]);
            tm_loaded(r[3]);
            if (masked) {
              uint32_t see[4];
              visible(see);
              // (columns past the tile's width hold an earlier tile's)
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                see[x] &= span(0, w, 32 * x);
                if (x * 32 < w && !__all_sync(0xffffffffu, see[x] == 0xffffffffu)) {
#pragma unroll
                  for (int i = 0; i < 32; ++i)
                    if (!(see[x] >> i & 1)) r[x][i] = 0xff800000u;
                }
              }
            }
            float mt;
            if (w == TILE) {
              mt = max_of<128>([&](int i) { return __uint_as_float(r[i >> 5][i & 31]); });
            } else {
              mt = -INFINITY;
#pragma unroll
              for (int x = 0; x < 4; ++x)
                if (x * 32 < w)
                  mt = fmaxf(mt, max_of<32>([&](int i) { return __uint_as_float(r[x][i]); }));
            }
            raise_to(mt);
            const float nm = m == -INFINITY ? 0.0f : lift - m * A.c;
            const float2 c2 = make_float2(A.c, A.c), mc2 = make_float2(nm, nm);
            float2 sum[4] = {};
            uint32_t pw[16];
            auto chunk = [&](int x) {  // the weights of 32 keys
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float2 e = fma2(make_float2(__uint_as_float(r[x][2 * i]),
                                                  __uint_as_float(r[x][2 * i + 1])), c2, mc2);
                const float2 p = make_float2(ex2(e.x), ex2(e.y));
                sum[i & 3] = add2(sum[i & 3], p);
                pw[i] = pack16<BF>(p.x, p.y);
              }
            };
            // the products with the first 64 keys' values start under the others' weights
            // (One copy for all widths, fewer instructions to fetch: a second one for whole
            // tiles took 1280 items of 16 tiles from 222 us to 244, 8192 tokens to 318 as now.)
            __syncwarp();
            chunk(0);
            tm_st16<false>(ts, pw);
            if (w > 32) {
              chunk(1);
              tm_st16<false>(ts + 16, pw);
            }
            half_done();
            if (w > 64) {
              chunk(2);
              tm_st16<false>(ts + 32, pw);
            }
            if (w > 96) {
              chunk(3);
              tm_st16<false>(ts + 48, pw);
            }
            sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
            l += sum[0].x + sum[0].y;
          } else {
            // One tile of rows: 64 scores at a time, the maximum of the tile's second half,
            // then of its first, whose weights follow from registers; the second half is
            // loaded again behind them.  (64 requests of 88 rows: 243 us, and 266 with all
            // scores in registers as below, which spills; a pair's 8192 tokens take 372 us
            // by halves and 334 as below.)
            uint32_t r0[32], r1[32], see[4] = {~0u, ~0u, ~0u, ~0u};
            if (masked) {
              visible(see);
              // (columns past the tile's width hold an earlier tile's)
#pragma unroll
              for (int x = 0; x < 4; ++x) see[x] &= span(0, w, 32 * x);
            }
            auto hide = [&](uint32_t (&r)[32], uint32_t bits) {
              if (masked && !__all_sync(0xffffffffu, bits == 0xffffffffu)) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (!(bits >> i & 1)) r[i] = 0xff800000u;
              }
            };
            auto two = [&](int x) {  // chunks x and x + 1, and their maximum
              tm_ld32(ts + x * 32, r0);
              if ((x + 1) * 32 < w) tm_ld32(ts + x * 32 + 32, r1);
              tm_wait_ld(r0);
              tm_loaded(r1);
              hide(r0, see[x]);
              float t = max_of<32>([&](int i) { return __uint_as_float(r0[i]); });
              if ((x + 1) * 32 < w) {
                hide(r1, see[x + 1]);
                t = fmaxf(t, max_of<32>([&](int i) { return __uint_as_float(r1[i]); }));
              }
              return t;
            };
            float mt = w > 64 ? two(2) : -INFINITY;
            mt = fmaxf(mt, two(0));
            raise_to(mt);
            const float nm = m == -INFINITY ? 0.0f : lift - m * A.c;
            const float2 c2 = make_float2(A.c, A.c), mc2 = make_float2(nm, nm);
            float2 sum[4] = {};
            auto weights = [&](int x, uint32_t (&r)[32]) {  // of 32 keys
              uint32_t pw[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float2 e = fma2(
                    make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), c2, mc2);
                const float2 p = make_float2(ex2(e.x), ex2(e.y));
                sum[i & 3] = add2(sum[i & 3], p);
                pw[i] = pack16<BF>(p.x, p.y);
              }
              tm_st16(ts + x * 16, pw);
            };
            // (P's columns lie over scores of the first half only; a pair's products
            // with the first half's values start under the second's weights)
            weights(0, r0);
            if (w > 64) tm_ld32(ts + 64, r0);
            if (w > 32) weights(1, r1);
            half_done();
            if (w > 64) {
              tm_wait_ld(r0);
              hide(r0, see[2]);
              if (w > 96) tm_ld32(ts + 96, r1);
              weights(2, r0);
              if (w > 96) {
                tm_wait_ld(r1);
                hide(r1, see[3]);
                weights(3, r1);
              }
            }
            sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
            l += sum[0].x + sum[0].y;
          }
          tm_wait_st<false>();
        }
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(&C.p_full[st]));
      }

      // ---- the segment's end: the output rows, or their partials
      const bool whole = n == s.nt;
      const int slot = segs == 0 ? 0 : 1;
      const size_t part = (size_t(blockIdx.x) * 2 + slot) * ROWS + (PAIR ? st * TILE : 0) + row;
      const size_t token_row = PR ? size_t(s.start) + tok : size_t(s.b) * A.N + tok;
      uint16_t* const orow = A.out + (token_row * A.Hq + s.h * A.G + rg) * A.D;
      float4* const prow = reinterpret_cast<float4*>(A.part_o);
      const size_t pcol0 = (size_t(blockIdx.x) * 2 + slot) * (DP / 4);
      const unsigned rows_on = __ballot_sync(0xffffffffu, active);
      auto put = [&](const float (&v)[32], int col) {  // 32 columns from col on
        if (whole) {
          // Four lanes exchange their rows' 16-byte pieces, so that they write
          // 64 bytes of one row at a time instead of 16 of four.
          uint4 u[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            u[i].x = pack16<BF>(v[8 * i], v[8 * i + 1]);
            u[i].y = pack16<BF>(v[8 * i + 2], v[8 * i + 3]);
            u[i].z = pack16<BF>(v[8 * i + 4], v[8 * i + 5]);
            u[i].w = pack16<BF>(v[8 * i + 6], v[8 * i + 7]);
          }
          swap_pieces(u[0], u[1], 1, lane);
          swap_pieces(u[2], u[3], 1, lane);
          swap_pieces(u[0], u[2], 2, lane);
          swap_pieces(u[1], u[3], 2, lane);
          const int c = col + (lane & 3) * 8;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int from = (lane & 28) + i;
            uint16_t* const o = reinterpret_cast<uint16_t*>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(orow), from));
            if ((rows_on >> from & 1) && c < A.D)
              *reinterpret_cast<uint4*>(o + c) = bad ? make_uint4(0, 0, 0, 0) : u[i];
          }
        } else if (active) {
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            prow[(pcol0 + (col + i) / 4) * ROWS + (PAIR ? st * TILE : 0) + row] =
                make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
      };
      // (Loops that are not unrolled below, and where the maximum is raised: less code is
      // faster where it runs once an item, most so among much data, which looks like the
      // cost of fetching it, though that was not measured by itself.
      // 1280 items of 200 rows and 16 tiles: 291 us unrolled, 244 not; 64 trees of 88 rows
      // over 2000 to 9000: 231 and 225.)
      if constexpr (NQ > 0) {
        // sums over the keys: 32 lanes here, the four warps and two streams below
        sum_columns<NQ>(lq, lane);
        if (lane < NQ) C.x.sums[warp][lane] = lq[0];
        group_sync(3, 2 * TILE);
        if (tid < NQ) {
          float l0 = 0.0f, l1 = 0.0f;
          for (int w = 0; w < 4; ++w) {
            l0 += C.x.sums[w][tid];
            l1 += C.x.sums[4 + w][tid];
          }
          float a = -C.x.nmc[0][tid], b = n > 1 ? -C.x.nmc[1][tid] : INFINITY;
          if (a == INFINITY) a = -INFINITY;  // nothing seen
          if (b == INFINITY) b = -INFINITY;
          const float mm = fmaxf(a, b), mu = mm == -INFINITY ? 0.0f : mm;
          float f0 = ex2(a - mu), f1 = ex2(b - mu);
          const float ll = l0 * f0 + (n > 1 ? l1 * f1 : 0.0f);
          if (whole) {
            f0 /= ll;
            f1 /= ll;
          }
          C.x.fac[0][tid] = f0;
          C.x.fac[1][tid] = f1;
          if (!whole)
            A.part_ml[(size_t(blockIdx.x) * 2 + slot) * NQ + tid] =
                make_float2(mm, bad ? -1.0f : ll);
        }
        for (int x = 0; x < 2; ++x) {
          if (x >= n) break;
          ok = ok && warp_wait(bar(&C.o_full[x]), o_use[x] & 1, A.status, abort);
          ++o_use[x];
        }
        tc_after();
        group_sync(3, 2 * TILE);
        __syncwarp();
        if (ok) {
          constexpr int HALF = NQ / 2;  // columns of this warpgroup
          const int q0 = st * HALF;
          uint32_t o0[HALF], o1[HALF];
          tm_ldn<HALF>(tmem + lanes + O_AT + q0, o0);
          if (n > 1) tm_ldn<HALF>(tmem + lanes + O_AT + S_COLS + q0, o1);
          tm_waitn<HALF>(o0);
          if (n > 1) tm_loadedn<HALF>(o1);
#pragma unroll
          for (int q = 0; q < HALF; ++q) {
            float v = __uint_as_float(o0[q]) * C.x.fac[0][q0 + q];
            if (n > 1) v = fmaf(__uint_as_float(o1[q]), C.x.fac[1][q0 + q], v);
            o0[q] = __float_as_uint(v);
          }
          if (!whole) {
            float* const to_part =
                A.part_o + ((size_t(blockIdx.x) * 2 + slot) * NQ + q0) * DP + row;
            if (row < DP) {
#pragma unroll
              for (int q = 0; q < HALF; ++q) to_part[q * DP] = __uint_as_float(o0[q]);
            }
          } else if (row < A.D) {
            // (column q is token q / G, head q mod G of the group)
            const int rows = A.N * A.G - q0;
            uint16_t* const o = A.out + (size_t(s.b) * A.N * A.Hq + size_t(s.h) * A.G) * A.D + row;
#pragma unroll
            for (int q = 0; q < HALF; ++q)
              if (q < rows)
                o[C.out_at[q0 + q]] = bad ? 0 : uint16_t(pack16<BF>(__uint_as_float(o0[q]), 0.0f));
          }
        }
        tc_before();
      } else if (PAIR) {
        ok = ok && warp_wait(bar(&C.o_full[st]), o_use[st] & 1, A.status, abort);
        ++o_use[st];
        tc_after();
        if (ok && warp_active) {
          const float f = whole ? 1.0f / l : 1.0f;
#pragma unroll 1
          for (int x = 0; x < DP / 32; ++x) {
            uint32_t o[32];
            float v[32];
            tm_ld32(to + x * 32, o);
            tm_wait_ld(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(o[i]) * f;
            put(v, x * 32);
          }
          if (!whole && active) A.part_ml[part] = make_float2(m * A.c, bad ? -1.0f : l);
        }
        tc_before();
      } else {
        // join the two streams; warpgroup st takes half of the columns
        C.x.ml[st][row] = make_float2(m, l);
        for (int x = 0; x < 2; ++x) {
          if (x >= n) break;
          ok = ok && warp_wait(bar(&C.o_full[x]), o_use[x] & 1, A.status, abort);
          ++o_use[x];
        }
        tc_after();
        group_sync(3, 2 * TILE);
        __syncwarp();
        if (ok && warp_active) {
          const float2 a = C.x.ml[0][row], b = C.x.ml[1][row];
          const float mm = fmaxf(a.x, b.x);
          const float mu = mm == -INFINITY ? 0.0f : mm;
          float f0 = ex2((a.x - mu) * A.c), f1 = ex2((b.x - mu) * A.c);
          const float ll = a.y * f0 + (n > 1 ? b.y * f1 : 0.0f);
          if (whole) {
            f0 /= ll;
            f1 /= ll;
          }
          const uint32_t t0 = tmem + lanes + O_AT;
#pragma unroll 1
          for (int x = 0; x < DP / 64; ++x) {
            const int col = st * (DP / 2) + x * 32;
            uint32_t o[32];
            float v[32];
            tm_ld32(t0 + col, o);
            tm_wait_ld(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(o[i]) * f0;
            if (n > 1) {
              tm_ld32(t0 + S_COLS + col, o);
              tm_wait_ld(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = fmaf(__uint_as_float(o[i]), f1, v[i]);
            }
            put(v, col);
          }
          if (!whole && st == 0 && active)
            A.part_ml[part] = make_float2(mm * A.c, bad ? -1.0f : ll);
        }
        tc_before();
      }
      if (segs == 0) {
        d_item = s.h * A.MT + s.mt;
        d_b = s.b;
        if (s.j0 > 0 && s.j0 + n < s.nt) d_flags |= DESC_THROUGH;
      } else {
        d_flags |= DESC_LAST1;
      }
      d_flags = s.j0 + n < s.nt ? d_flags | DESC_OUT : d_flags & ~DESC_OUT;
      idx += 2 * n;
      seg_done(segs);
      ++segs;
    }
    if (!PR && A.join && tid == 0) A.desc[blockIdx.x] = make_int4(d_flags, d_item, d_b, 0);
  } else {
    __syncwarp();
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(OTHER_REGS));
  if (warp == PLAN_WARP) {
    // ------------------------------------------------------------ the plan
    Cursor<PAIR, PR> cur;
    Seg s;
    auto plan = [&](int i, bool more) {  // segment i, or the end
      // (the segment that stood there ends: until then its tiles pass through the stages)
      if (i >= AHEAD &&
          !__all_sync(0xffffffffu,
                      mbar_wait_moving(bar(&C.seg_empty[i % AHEAD]), (i / AHEAD - 1) & 1,
                                       bar(&C.empty[0]), A.status, abort)))
        return false;
      if (lane == 0) {
        if (!more) s.n = 0;
        C.seg[i % AHEAD] = s;
        mbar_arrive(bar(&C.seg_full[i % AHEAD]));
      }
      __syncwarp();
      return more;
    };
    if constexpr (PR) {
      bool report = blockIdx.x == 0;  // bad bounds are reported by the CTA of item 0
      cur.open(A, report);
      long long i = blockIdx.x;
      int seg_count = 0;
      for (int k = 0;; ++k) {
        // another item is asked for before this one is planned
        if (lane == 0) {
          mbar_arrive_tx(bar(&C.next_full), 16);
          asm volatile(
              "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 "
              "[%0], [%1];" ::"r"(smem_addr(&C.next)),
              "r"(bar(&C.next_full))
              : "memory");
        }
        __syncwarp();
        const bool have = cur.item(A, i, s, report);  // (none past the last sequence)
        const bool go = !have || plan(seg_count, true);
        if (have) ++seg_count;
        if (!warp_wait(bar(&C.next_full), k & 1, A.status, abort)) {
          const unsigned long long t0 = globaltimer();  // the answer lands before the CTA ends
          while (!mbar_try(bar(&C.next_full), k & 1) && globaltimer() - t0 < WAIT_LIMIT_NS) {
          }
          break;
        }
        uint32_t x, got;
        asm volatile(
            "{\n .reg .pred p;\n .reg .b128 r;\n .reg .b32 y, z;\n ld.shared.b128 r, [%2];\n"
            " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n"
            " selp.u32 %1, 1, 0, p;\n mov.u32 %0, 0;\n"
            " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n}"
            : "=r"(x), "=r"(got)
            : "r"(smem_addr(&C.next))
            : "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (!got || !go) break;
        i = x;
        if (i == 0) {
          report = true;
          cur.open(A, true);
        }
      }
      if (report) cur.item(A, 0x7fffffffffffffffll, s, true);  // the other sequences' bounds
      plan(seg_count, false);
    } else {
      cur.open(A, start_b, start_at, run, whole_items);
      int k = 0;
      while (plan(k, cur.next(A, s))) ++k;
    }
  } else if (warp == COPY_WARP) {
    // ------------------------------------------------------------ copies
    // One thread, or (pages) a warp with a lane per box of page rows.
    auto copies = [&](auto solo) {
      constexpr bool SOLO = decltype(solo)::value;
      const bool lead = SOLO || lane == 0;
      auto wait = [&](uint32_t bar, unsigned parity) {
        return SOLO ? mbar_wait(bar, parity, A.status, abort)
                    : warp_wait(bar, parity, A.status, abort);
      };
      auto together = [&] {
        if (!SOLO) __syncwarp();
      };
      uint32_t st = 0, lap = 0, idx = 0;  // stage, times around the ring, copies
      int segs = 0;
      bool ok = true;
      for (;;) {
        ok = wait(bar(&C.seg_full[segs % AHEAD]), (segs / AHEAD) & 1);
        if (!ok) break;
        const Seg s = C.seg[segs % AHEAD];
        if (s.n == 0) break;
        together();
        if (lead) mbar_arrive(bar(&C.seg_empty[segs % AHEAD]));
        const int slot = PAIR ? 0 : segs & 1;
        const int use = PAIR ? segs : segs >> 1;
        ok = wait(bar(&C.q_empty[slot]), (use & 1) ^ 1);  // (passes before the first use)
        if (!ok) break;
        if (lead) {
          const uint32_t fb = bar(&C.q_full[slot]);
          mbar_arrive_tx(fb, (PAIR ? 2 : 1) * A.q_rows * DP * 2);
          const int tok = PR ? s.start : s.b * A.N;
          for (int q = 0; q < (PAIR ? 2 : 1); ++q)
            for (int x = 0; x < HALVES; ++x)
              tma_4d(base + (PAIR ? q : slot) * SM::Q_BYTES + x * (SM::Q_BYTES / HALVES), &A.mq,
                     fb, x * 64, 0, s.h, tok + (s.mt * (PAIR ? 2 : 1) + q) * A.tpt);
        }
        together();
        ++segs;
        const int plane = PR ? s.h : s.b * A.LH + A.head0 + s.h;
        auto tile = [&](int jj, bool is_v) {
          const uint32_t fb = bar(&C.full[st]);
          const uint32_t dst = base + SM::STAGE_AT + st * BYTES;
          if (!wait(bar(&C.empty[st]), (lap & 1) ^ 1)) return false;
          const Keys ky = keys_of<PR>(A, s, s.j0 + jj);
          if (SOLO || ky.staged) {
            if (lead) {
              const CUtensorMap* const m = !PR && ky.staged ? (is_v ? &A.mvn : &A.mkn)
                                                            : (is_v ? &A.mv : &A.mk);
              mbar_arrive_tx(fb, BYTES);
#pragma unroll
              for (int x = 0; x < HALVES; ++x) {
                if (PR) tma_3d(dst + x * 16384, m, fb, x * 64, plane, s.start + ky.k0);
                else tma_3d(dst + x * 16384, m, fb, x * 64, ky.k0, plane);
              }
            }
          } else {
            // a page outside the pool is read as page 0 (the softmax warps report it
            // and drop the result)
            const int boxes = (ky.n + A.box - 1) / A.box;
            if (lead) mbar_arrive_tx(fb, boxes * A.box * DP * 2);
            __syncwarp();
            if (lane < boxes) {
              const int t = ky.k0 + lane * A.box;
              const int col = t / A.page;
              int pg = __ldg(A.table + size_t(s.b) * A.cols + col);
              if (pg < 0 || pg >= A.num_pages) pg = 0;
#pragma unroll
              for (int x = 0; x < HALVES; ++x)
                tma_4d(dst + x * 16384 + lane * A.box * 128, is_v ? &A.mv : &A.mk, fb, x * 64,
                       t - col * A.page, A.head0 + s.h, pg);
            }
          }
          together();
          ++idx;
          if (++st == STAGES) {
            st = 0;
            ++lap;
          }
          return true;
        };
        constexpr int LAG = PAIR ? 0 : 1;
        for (int i = 0; ok && i < s.n + LAG; ++i) {
          if (i < s.n) ok = tile(i, false);
          if (ok && i >= LAG) ok = tile(i - LAG, true);
        }
        if (!ok) break;
      }
      if (*abort) {  // the copies in flight land before the CTA ends
        const unsigned long long t0 = globaltimer();
        for (uint32_t u = idx > STAGES ? idx - STAGES : 0; u < idx; ++u)
          while (!mbar_try(bar(&C.full[u % STAGES]), (u / STAGES) & 1) &&
                 globaltimer() - t0 < WAIT_LIMIT_NS) {
          }
        for (int u = max(0, segs - (PAIR ? 1 : 2)); u < segs; ++u)
          while (!mbar_try(bar(&C.q_full[PAIR ? 0 : u & 1]), (PAIR ? u : u >> 1) & 1) &&
                 globaltimer() - t0 < WAIT_LIMIT_NS) {
          }
      }
    };
    if (PR || A.kind == RING) {
      if (elect_one()) copies(Yes<true>());
      __syncwarp();
    } else {
      copies(Yes<false>());
    }
  } else if (warp == MMA_WARP) {
    // ------------------------------------------------------------ products
    uint32_t idx = 0;
    int segs = 0;
    unsigned p_use[2] = {0, 0};
    // (the turned products: N = NQ, and V^T is an operand whose dimensions are contiguous)
    const uint32_t id_s = instr_desc(BF, false, false, NQ);  // (0: the tile's width goes there)
    const uint32_t id_o = instr_desc(BF, NQ > 0, NQ == 0, NQ ? NQ : DP);
    bool ok = true;
    auto full = [&](uint32_t u) {
      if (!mbar_wait(bar(&C.full[u % STAGES]), (u / STAGES) & 1, A.status, abort)) return false;
      tc_after();
      return true;
    };
    auto scores = [&](int st, int q, uint32_t u, int w) {  // S[st] = Q[q] K^T, or K Q[q]^T
      const uint32_t qa = desc_rows(base + q * SM::Q_BYTES);
      const uint32_t ka = desc_rows(base + SM::STAGE_AT + (u % STAGES) * BYTES);
#pragma unroll
      for (int k = 0; k < DP / 16; ++k) {
        if (k * 16 >= A.D) break;  // (the rest of the tiles is zeros)
        const uint32_t dq = qa + (((k / 4) * (SM::Q_BYTES / HALVES) + (k % 4) * 32) >> 4);
        const uint32_t dk = ka + (((k / 4) * 16384 + (k % 4) * 32) >> 4);
        mma_ss(tmem + st * S_COLS, NQ ? dk : dq, NQ ? dq : dk,
               NQ ? id_s : id_s | uint32_t(w >> 3) << 17, k > 0);
      }
      mma_commit(bar(&C.s_full[st]));
    };
    // O[st] (+)= P[st] V, or V^T P[st]^T, over sixteens k0 .. k1 - 1 of the tile's keys
    auto values = [&](int st, uint32_t u, int w, bool more, int k0, int k1) {
      const uint32_t va = desc_cols(base + SM::STAGE_AT + (u % STAGES) * BYTES,
                                    NQ && DP == 64 ? 0 : 16384);
      const uint32_t pa = desc_rows(base + SM::P_AT + st * SM::P_BYTES);
#pragma unroll
      for (int k = k0; k < k1; ++k) {
        if (k * 16 >= w) break;
        const uint32_t dv = va + ((k * 2048) >> 4);
        const uint32_t dp = pa + (((k / 4) * (NQ * 128) + (k % 4) * 32) >> 4);
        if (NQ) mma_ss(tmem + O_AT + st * S_COLS, dv, dp, id_o, more || k > 0);
        else mma_ts(tmem + O_AT + st * S_COLS, tmem + st * S_COLS + k * 8, dv, id_o, more || k > 0);
      }
    };
    auto first_half = [&](int st, uint32_t uv, int w, bool more) {
      if (!PAIR) return true;
      if (!mbar_wait(bar(&C.p_half[st]), p_use[st] & 1, A.status, abort)) return false;
      tc_after();
      values(st, uv, w, more, 0, 4);
      return true;
    };
    // One thread from here on: the waits, too, are its own.
    if (elect_one()) {
    while (ok) {
      ok = mbar_wait(bar(&C.seg_full[segs % AHEAD]), (segs / AHEAD) & 1, A.status, abort);
      if (!ok) break;
      const Seg s = C.seg[segs % AHEAD];
      if (s.n == 0) break;
      mbar_arrive(bar(&C.seg_empty[segs % AHEAD]));
      const int slot = PAIR ? 0 : segs & 1;
      const int use = PAIR ? segs : segs >> 1;
      ok = mbar_wait(bar(&C.q_full[slot]), use & 1, A.status, abort);
      const int n = s.n;
      const uint32_t u0 = idx;
      auto width = [&](int j) { return width_of(keys_of<PR>(A, s, s.j0 + j)); };
      if (PAIR) {
        int w = width(0);
        ok = ok && full(u0);
        if (ok) {
          scores(0, 0, u0, w);
          scores(1, 1, u0, w);
          mma_commit(bar(&C.empty[u0 % STAGES]));
          if (n == 1) mma_commit(bar(&C.q_empty[0]));
        }
        for (int j = 0; ok && j < n; ++j) {
          const uint32_t uv = u0 + v_order<true>(j, n), uk = u0 + k_order<true>(j + 1);
          const bool more = j + 1 < n;
          const int w2 = more ? width(j + 1) : 0;
          ok = full(uv) && (!more || full(uk));
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            ok = ok && first_half(st, uv, w, j > 0) &&
                 mbar_wait(bar(&C.p_full[st]), p_use[st] & 1, A.status, abort);
            ++p_use[st];
            if (!ok) break;
            tc_after();
            {
              values(st, uv, w, true, 4, 8);
              if (st == 1) mma_commit(bar(&C.empty[uv % STAGES]));
              if (more) {
                scores(st, st, uk, w2);
                if (st == 1) {
                  mma_commit(bar(&C.empty[uk % STAGES]));
                  if (j + 2 == n) mma_commit(bar(&C.q_empty[0]));
                }
              } else {
                mma_commit(bar(&C.o_full[st]));
              }
            }
            }
          w = w2;
        }
      } else {
        for (int j = 0; ok && j < 2 && j < n; ++j) {
          const uint32_t uk = u0 + k_order<false>(j);
          const int w = width(j);
          ok = full(uk);
          if (ok) {
            scores(j, slot, uk, w);
            mma_commit(bar(&C.empty[uk % STAGES]));
            if (j + 1 == n) mma_commit(bar(&C.q_empty[slot]));
          }
        }
        for (int j = 0; ok && j < n; ++j) {
          const int st = j & 1;
          const uint32_t uv = u0 + v_order<false>(j, n), uk = u0 + k_order<false>(j + 2);
          const bool more = j + 2 < n;
          const int w = width(j), w2 = more ? width(j + 2) : 0;
          ok = full(uv) && (!more || full(uk)) &&
               mbar_wait(bar(&C.p_full[st]), p_use[st] & 1, A.status, abort);
          ++p_use[st];
          if (!ok) break;
          tc_after();
          {
            values(st, uv, w, j >= 2, 0, 8);
            mma_commit(bar(&C.empty[uv % STAGES]));
            if (more) {
              scores(st, slot, uk, w2);
              mma_commit(bar(&C.empty[uk % STAGES]));
              if (j + 3 == n) mma_commit(bar(&C.q_empty[slot]));
            } else {
              mma_commit(bar(&C.o_full[st]));
            }
          }
        }
      }
      idx += 2 * n;
      ++segs;
    }
    if (!ok) {  // the products in flight end before TMEM is freed
      mma_commit(bar(&C.drain));
      const unsigned long long t0 = globaltimer();
      while (!mbar_try(bar(&C.drain), 0) && globaltimer() - t0 < WAIT_LIMIT_NS) {
      }
    }
    }
    __syncwarp();
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == MMA_WARP) {
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "n"(TM_COLS)
                 : "memory");
  }
}

// Join of the items that the CTAs' runs cut, from the parts' maxima, sums and
// outputs.  A warp takes one unit of a cut item at a time: one row's columns, a
// lane each four of them (NQ > 0), or 32 rows' 16 columns, a lane each a row.  It
// is bound by the latency of its loads, so what the CTAs were about is read once
// per block, and the parts' values are loaded four parts at a time.
constexpr int JOIN_WARPS = 8, JOIN_BLOCKS = 4;  // blocks per SM
template <int DP, int NQ, bool PAIR, bool BF>
__global__ void __launch_bounds__(JOIN_WARPS * 32) sv_attn_join(const __grid_constant__ AttnParams A,
                                                               int ctas) {
  constexpr int ROWS = NQ ? NQ : PAIR ? 2 * TILE : TILE;
  constexpr int VECS = NQ ? 1 : 4;  // four-column pieces per lane
  __shared__ int4 desc[MAX_CTAS];
  __shared__ int2 cuts[MAX_CTAS];   // (first CTA of the item, CTAs of it)
  __shared__ int found_s[JOIN_WARPS];
  const int tid = int(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  static_assert(MAX_CTAS <= JOIN_WARPS * 32, "one thread per CTA of the main kernel");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (tid < ctas) desc[tid] = A.desc[tid];
  __syncthreads();
  // The cut items, in the order of their first CTAs (every block has to find
  // the same list).  CTA c holds an item's first part when its last segment is
  // cut and did not itself begin inside the item.
  int parts = 0;
  if (tid + 1 < ctas) {
    const int x = desc[tid].x;
    if ((x & DESC_OUT) && !(x & DESC_THROUGH)) {
      int e = tid + 1;
      while (e + 1 < ctas && (desc[e].x & DESC_THROUGH)) ++e;
      parts = e - tid + 1;
    }
  }
  const unsigned found = __ballot_sync(0xffffffffu, parts != 0);
  if (lane == 0) found_s[warp] = __popc(found);
  __syncthreads();
  int at = __popc(found & ((1u << lane) - 1)), count = 0;
  for (int w = 0; w < JOIN_WARPS; ++w) {
    if (w < warp) at += found_s[w];
    count += found_s[w];
  }
  if (parts) cuts[at] = make_int2(tid, parts);
  __syncthreads();
  const int row_groups = (min(A.tpt, A.N) * A.G + 31) / 32;
  const int per_item = NQ ? A.N * A.G : row_groups * (PAIR ? 2 : 1) * (DP / 16);
  const int units = count * per_item;
  const float4* const src = reinterpret_cast<const float4*>(A.part_o);
  // neighbouring units on different SMs
  for (int u = int(blockIdx.x + gridDim.x * warp); u < units; u += int(gridDim.x) * JOIN_WARPS) {
    const int2 cut = cuts[u / per_item];
    const int w = u % per_item;
    const int cg = w % (DP / 16), rgp = w / (DP / 16);
    const int st = PAIR ? rgp / row_groups : 0;
    const int row = NQ ? w : (rgp % row_groups) * 32 + lane;
    const int4 d1 = desc[cut.x + 1];  // its first segment is of this item
    const int item = d1.y, b = d1.z;
    const int h = item / A.MT, mt = item - h * A.MT;
    const int rt = row / A.G, rg = row - rt * A.G;
    const int tok = mt * (PAIR ? 2 : 1) * A.tpt + st * A.tpt + rt;
    if (NQ ? lane >= DP / 4 : row >= TILE || rt >= A.tpt || tok >= A.N) continue;
    const size_t s0 = size_t(cut.x) * 2 + (desc[cut.x].x & DESC_LAST1 ? 1 : 0);
    float m = -INFINITY, l = 0.0f;
    bool bad = false;
    float4 acc[VECS];
#pragma unroll
    for (int i = 0; i < VECS; ++i) acc[i] = make_float4(0, 0, 0, 0);
    constexpr int AT_ONCE = 4;
    for (int p0 = 0; p0 < cut.y; p0 += AT_ONCE) {
      float2 ml[AT_ONCE];
      float4 o[AT_ONCE][VECS];
#pragma unroll
      for (int k = 0; k < AT_ONCE; ++k) {
        ml[k] = make_float2(-INFINITY, 0.0f);
        if (p0 + k < cut.y) {
          const size_t s = p0 + k ? size_t(cut.x + p0 + k) * 2 : s0;
          ml[k] = A.part_ml[s * ROWS + st * TILE + row];
#pragma unroll
          for (int i = 0; i < VECS; ++i)
            o[k][i] = NQ ? src[(s * ROWS + row) * (DP / 4) + lane]
                         : src[(s * (DP / 4) + cg * 4 + i) * ROWS + st * TILE + row];
        }
      }
      float m2 = m;
#pragma unroll
      for (int k = 0; k < AT_ONCE; ++k) m2 = fmaxf(m2, ml[k].x);
      const float mu = m2 == -INFINITY ? 0.0f : m2, f = ex2(m - mu);
      m = m2;
      l *= f;
#pragma unroll
      for (int i = 0; i < VECS; ++i) {
        acc[i].x *= f;
        acc[i].y *= f;
        acc[i].z *= f;
        acc[i].w *= f;
      }
#pragma unroll
      for (int k = 0; k < AT_ONCE; ++k)
        if (p0 + k < cut.y) {
          const float g = ex2(ml[k].x - mu);
          bad |= ml[k].y == -1.0f;
          l += ml[k].y * g;
#pragma unroll
          for (int i = 0; i < VECS; ++i) {
            acc[i].x += o[k][i].x * g;
            acc[i].y += o[k][i].y * g;
            acc[i].z += o[k][i].z * g;
            acc[i].w += o[k][i].w * g;
          }
        }
    }
    const float f = 1.0f / l;
    uint16_t* const o = A.out + ((size_t(b) * A.N + tok) * A.Hq + h * A.G + rg) * A.D;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int col = NQ ? lane * 4 : cg * 16 + i * 4;
      uint2 x = make_uint2(pack16<BF>(acc[i].x * f, acc[i].y * f),
                           pack16<BF>(acc[i].z * f, acc[i].w * f));
      if (bad) x = make_uint2(0, 0);
      if (col < A.D) *reinterpret_cast<uint2*>(o + col) = x;
    }
  }
}

// -------------------------------------------------------------- launches

// Columns of the turned products, or 0 for a row per lane; rows of an item.
struct Layout { int nq, rows; };

template <int DP, int NQ, bool PAIR, bool PR, bool BF>
int launch_as(const AttnParams& A, int device, int grid, int ctas, cudaStream_t st) {
  // the kernel's shared-memory limit, raised once per device (ordinals past 63: every time)
  static std::atomic<uint64_t> raised{0};
  const uint64_t mark = device < 64 ? uint64_t(1) << device : 0;
  if (!(raised.load(std::memory_order_acquire) & mark)) {
    if (cudaFuncSetAttribute(sv_attn<DP, NQ, PAIR, PR, BF>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (Smem<DP, NQ>::TOTAL)) != cudaSuccess)
      return SV_ERR_CUDA;
    raised.fetch_or(mark, std::memory_order_release);
  }
  sv_attn<DP, NQ, PAIR, PR, BF><<<grid, THREADS, (Smem<DP, NQ>::TOTAL), st>>>(A);
  if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  if (PR || !A.join) return SV_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(JOIN_BLOCKS * ctas));
  cfg.blockDim = dim3(JOIN_WARPS * 32);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sv_attn_join<DP, NQ, PAIR, BF>, A, ctas) == cudaSuccess ? SV_OK
                                                                                : SV_ERR_CUDA;
}

template <int DP, bool BF>
int launch_dp(const AttnParams& A, Layout l, int device, int grid, int ctas, cudaStream_t st) {
  if (A.kind == PROMPT)
    return l.rows == TILE ? launch_as<DP, 0, false, true, BF>(A, device, grid, ctas, st)
                          : launch_as<DP, 0, true, true, BF>(A, device, grid, ctas, st);
  if (l.nq == 16) return launch_as<DP, 16, false, false, BF>(A, device, grid, ctas, st);
  if (l.nq == 32) return launch_as<DP, 32, false, false, BF>(A, device, grid, ctas, st);
  if (l.rows == TILE) return launch_as<DP, 0, false, false, BF>(A, device, grid, ctas, st);
  return launch_as<DP, 0, true, false, BF>(A, device, grid, ctas, st);
}

// One translation unit per storage type (attn_bf16.cu, attn_f16.cu), compiled
// side by side.
int launch_bf16(const AttnParams& A, Layout l, int device, int grid, int ctas, cudaStream_t st);
int launch_f16(const AttnParams& A, Layout l, int device, int grid, int ctas, cudaStream_t st);

}  // namespace svattn

#endif  // SV_ATTENTION_CUH
