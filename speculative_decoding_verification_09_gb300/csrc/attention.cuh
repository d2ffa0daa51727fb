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
//
// Over 8-bit pages (Q8; include/svkv8.h) the cache is half as long, and a tile's chain
// holds the keys' powers of two and values' widening besides.  Few rows are bound by the
// widening (64 requests of 4 tokens, 16 rows: 182 us in bf16, 4.2 TB/s; 208 over 16 bits), more
// rows by the softmax and by how many roles' code an SM has to fetch: 22 nodes, 88 rows 248 us
// (225 over 16 bits).
//   sv_attn8_prep  before it: queries and staged keys as 8-bit terms
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
constexpr int THREADS8 = 512;   // and (8-bit caches) one that widens the values
// Registers: launched with 168 a thread (64512 a CTA); the softmax warpgroups
// hold up to 128 scores a thread and take over what the third does not need.
// (Ragged prompts: 107 us with 208 / 88, 101 with 216 / 72, 132 with 184 / 136.)
constexpr int SOFTMAX_REGS = 216, OTHER_REGS = 72;
static_assert(256 * SOFTMAX_REGS + 128 * OTHER_REGS <= THREADS * 168, "register split");
// With 8-bit caches the launch has 128 a thread (65536 a CTA), and a row per lane takes
// more than few rows do.
template <int NQ, bool Q8>
struct Regs {
  static constexpr int SOFTMAX = !Q8 ? SOFTMAX_REGS : NQ == 32 ? 160 : 144;
  static constexpr int OTHER = !Q8 ? OTHER_REGS : NQ == 32 ? 96 : 112;
  static_assert(!Q8 || 256 * SOFTMAX + 256 * OTHER <= THREADS8 * 128,
                "register split");
};
constexpr int COPY_WARP = 8, MMA_WARP = 9, PLAN_WARP = 10;
// 8-bit caches: 8 to 11 widen, and one other role beside each.  A warp's place goes by its
// number modulo 4, so every quarter of the SM has one that widens.  (64 requests of 4 nodes, bf16,
// 182 us, and 198 with two of them on each of two quarters; 22 nodes 248 and 264.)
constexpr int WIDEN_WARPS = 4;
constexpr int COPY8_WARP = 12, MMA8_WARP = 13, PLAN8_WARP = 14, SCALE_WARP = 15;
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
// (bf16 over 8-bit caches: the launch takes a lift below 0, at which the weights of a row add up
// to 1 at most, so that sums of weights times values as large as the type's stay finite.)

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
  float lift;             // weight of a row's maximum (log2; bf16 over 16 bits: 0)
  int kind;
  int B, N, Hq, Hkv, D, G;
  int LH, head0, num_pages, page, cols, sink, window, T;
  int box;                // page rows of one copy
  int tpt;                // tokens per query tile, floor(128 / G)
  int q_rows;             // rows of one query copy
  int MT;                 // items per KV head (TREE, RING)
  int whole_tiles;        // no item is cut when none has more tiles than this (TREE, RING)
  int join;               // and some may have, by the cache's extent
  int withhold;           // failure-handling test: one of CTA 0's stages never fills
  // 8-bit caches (mq: the queries' terms, mkn: the staged keys'): the blocks' scales
  // [num_pages][LH][page / block], and powers of two that the first kernel found, of the queries'
  // rows [B][N][Hq] and of the staged keys, eight at a time [B][Hkv][tiles][16]
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  const float* qf;
  const float* kf;
  int block_log;          // log2 of the tokens of a block
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

__device__ __forceinline__ void tma_5d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x,
                                       int y, int z, int w, int v) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst), "l"(m), "r"(bar), "r"(x), "r"(y),
      "r"(z), "r"(w), "r"(v)
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
// Products of 8-bit operands (e4m3), K-major tiles of DP bytes a row in the swizzle of that
// width; 32 dimensions a product.
template <int DP>
__device__ __forceinline__ void mma8_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                        uint32_t accumulate) {
  constexpr uint32_t HI = DP == 128 ? DESC_HI : (512 >> 4) | (1u << 14) | (4u << 29);
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.u32 p, %4, 0;\n"
      " mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n}" ::"r"(d), "r"(a), "r"(b),
      "r"(idesc), "r"(accumulate), "n"(HI)
      : "memory");
}
__device__ __forceinline__ uint32_t instr_desc8(int n) {  // 32-bit sums
  return (1u << 4) | (uint32_t(n >> 3) << 17) | (uint32_t(TILE >> 4) << 24);
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
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mul.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
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
// (8-bit caches: the staged tiles come first, since what is made of them takes longest.)
template <bool PR, bool Q8 = false>
__device__ __forceinline__ Keys keys_of(const AttnParams& A, const Seg& s, int j) {
  if (Q8) {
    const int ts = tiles_of(A.N);
    if (j < ts) return {j * TILE, min(TILE, A.N - j * TILE), true};
    return {(j - ts) * TILE, min(TILE, s.len - (j - ts) * TILE), false};
  }
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

// 8-bit caches: bytes have a ring for keys (TERMS stages for a staged tile's) and one for values,
// filled in the order K_i V_i, and the 16-bit ring has all values of a segment, whose first
// tiles are the staged ones.
__device__ __forceinline__ int staged_of(const AttnParams& A, const Seg& s) {
  return min(max(tiles_of(A.N) - s.j0, 0), s.n);
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
constexpr int CTRL8_BYTES = 1536;  // more of it with 8-bit caches
// 8-bit caches (Q8).  Keys stay bytes: scores are products of e4m3 with e4m3, the queries
// split into TERMS such terms whose sum is theirs exactly (4 bits of a mantissa each; see
// split_terms).  Values arrive as bytes, too, and the widening warps fill the 16-bit stages
// that their products read, times their power of two: a cache's exponents are those at which
// the storage type has every value exactly, so weights and sums are those of the 16-bit
// caches.  (The powers of two in the weights instead, relative to the largest so far, save the
// widening half of its instructions, but a value that a row gives no weight then decides how
// many bits the others' weights have.)  Few 16-bit stages are enough, since they are filled
// from shared memory; the bytes' stages cover the copies' latency.
template <bool BF>
constexpr int TERMS_OF = BF ? 2 : 3;
template <int DP, int NQ, int TERMS = 0, bool PAIR = false>  // TERMS: 0 for 16-bit caches
struct Smem {
  static constexpr bool Q8 = TERMS > 0;
  static constexpr int BYTES = TILE * DP * 2;                    // a tile of keys or values
  static constexpr int TERM = (NQ ? NQ : TILE) * DP;             // a term of a tile of queries
  static constexpr int Q_BYTES = TERM * (Q8 ? TERMS : 2);        // a tile of queries
  static constexpr int P_BYTES = NQ * TILE * 2;                  // weights of a stream (NQ > 0)
  // the next segment's queries have a place of their own, but for three terms of 128 rows of
  // 128 dimensions, beside which three stages of bytes would remain
  static constexpr int Q_SLOTS = TERMS == 3 && NQ == 0 && DP == 128 && !PAIR ? 1 : 2;
  static constexpr int P_AT = Q_SLOTS * Q_BYTES;
  static constexpr int STAGE_AT = P_AT + 2 * P_BYTES;
  static constexpr int ROOM = 232448 - CTRL_BYTES - (Q8 ? CTRL8_BYTES : 0);
  static constexpr int FIT = (ROOM - STAGE_AT) / BYTES;
  static constexpr int STAGES = Q8 ? (DP == 128 ? 2 : 3) : FIT < 12 ? FIT : 12;
  static constexpr int RAW = TILE * DP;                          // a tile of bytes
  static constexpr int RAW_AT = STAGE_AT + STAGES * BYTES;
  static constexpr int RAW_FIT = (ROOM - RAW_AT) / RAW;
  static constexpr int RAWS = !Q8 ? 0 : RAW_FIT < 12 - STAGES ? RAW_FIT : 12 - STAGES;
  static constexpr int RAW_K = (RAWS + 1) / 2, RAW_V = RAWS / 2;  // keys' stages, then values'
  static constexpr int CTRL = RAW_AT + RAWS * RAW;               // offset of the control part
  static constexpr int TOTAL = CTRL + CTRL_BYTES + (Q8 ? CTRL8_BYTES : 0);
  static_assert(!Q8 || RAWS >= 3, "bytes on their way");
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
  // barriers: stages filled and free (16-bit ones, then those of bytes), queries, scores, weights (a pair's first half, all),
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
    struct { long long sum[THREADS8 / 32]; int most[THREADS8 / 32]; } scan;
  };
  unsigned long long out_at[NQ ? NQ : 1];  // NQ > 0: elements from an item's output to a column's
};
static_assert(sizeof(Ctrl<0, true>) <= CTRL_BYTES && sizeof(Ctrl<0, false>) <= CTRL_BYTES &&
                  sizeof(Ctrl<16, false>) <= CTRL_BYTES && sizeof(Ctrl<32, false>) <= CTRL_BYTES,
              "control part");

// The control part's rest with 8-bit caches.  A tile's powers of two, eight keys at a time: of
// the keys in 32 bits, of the values in the storage type, twice in a word.
struct Tile8 {
  alignas(16) float kf[16];
  uint32_t vf[16];
};
constexpr int SCALES = 8;        // cached tiles whose scales are read ahead
template <int NQ>
struct Ctrl8 {
  unsigned long long full[SCALES], empty[SCALES];
  Tile8 tile[SCALES];
  alignas(16) float qf[2][NQ ? NQ : 1];  // the columns' powers of two, per stream
};
static_assert(sizeof(Ctrl8<0>) <= CTRL8_BYTES && sizeof(Ctrl8<32>) <= CTRL8_BYTES, "control part");
__device__ __forceinline__ float power(int e) { return __int_as_float((e + 127) << 23); }

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
// Q8: the scores are taken in base-2 units, times the powers of two of the key (kf) and of the
// columns (qf).
template <int NQ, bool BF, bool Q8>
__device__ __forceinline__ void softmax_few(const AttnParams& A, Ctrl<NQ, false>& C, int st,
                                            int key, uint32_t ts, uint32_t to, uint32_t sees,
                                            bool masked, bool started, bool& unset, float* lq,
                                            unsigned char* pbuf, const float* kf,
                                            const float* qf) {
  const float lift = BF && !Q8 ? 0.0f : A.lift, unit = Q8 ? 1.0f : A.c;
  const float heaviest = !BF ? MOST_F16 : Q8 ? MOST_BF16 + lift : MOST_BF16;
  const float kc = Q8 ? A.c * kf[key >> 3] : 0.0f;
  const int lane = key & 31, warp = key >> 5;
  float* const nmc = C.x.nmc[st];
  const float2 c2 = make_float2(A.c, A.c);
  uint32_t r[NQ];
  auto load = [&] {
    tm_ldn<NQ>(ts, r);
    tm_waitn<NQ>(r);
    if (Q8) {
      const float2 k2 = make_float2(kc, kc);
#pragma unroll
      for (int q = 0; q < NQ; q += 4) {
        const float4 f = *reinterpret_cast<const float4*>(qf + q);
        const float2 a = mul2(make_float2(__uint_as_float(r[q]), __uint_as_float(r[q + 1])),
                              mul2(make_float2(f.x, f.y), k2));
        const float2 b = mul2(make_float2(__uint_as_float(r[q + 2]), __uint_as_float(r[q + 3])),
                              mul2(make_float2(f.z, f.w), k2));
        r[q] = __float_as_uint(a.x);
        r[q + 1] = __float_as_uint(a.y);
        r[q + 2] = __float_as_uint(b.x);
        r[q + 3] = __float_as_uint(b.y);
      }
    }
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
      const float2 u = make_float2(__uint_as_float(r[q]), __uint_as_float(r[q + 1]));
      const float2 v = make_float2(__uint_as_float(r[q + 2]), __uint_as_float(r[q + 3]));
      const float2 a = Q8 ? add2(u, make_float2(n.x, n.y)) : fma2(u, c2, make_float2(n.x, n.y));
      const float2 b = Q8 ? add2(v, make_float2(n.z, n.w)) : fma2(v, c2, make_float2(n.z, n.w));
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
    raise = group_or(1 + st, TILE, exponents() > heaviest);
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
                            fmaxf(wmax[2 * NQ + key], wmax[3 * NQ + key])) * unit;
      float old = started ? -nmc[key] : INFINITY, f = 1.0f;
      if (old == INFINITY) {
        if (t > -INFINITY) old = t - lift;
      } else if (t - old > heaviest) {
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

// Four e4m3 values to the storage type, times a power of two (twice in `by`) at which it has
// them exactly; a NaN stays one.  (e4m3 goes to 16-bit floats by way of fp16, and to bf16 by way of
// 32 bits.)
template <bool BF>
__device__ __forceinline__ uint2 widen4(uint32_t w, uint32_t by) {
  uint2 r;
  asm("{\n .reg .b16 u, v;\n mov.b32 {u, v}, %2;\n"
      " cvt.rn.f16x2.e4m3x2 %0, u;\n cvt.rn.f16x2.e4m3x2 %1, v;\n}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(w));
  auto times = [&](uint32_t h) {
    if (BF) {
      asm("{\n .reg .b16 u, v;\n .reg .f32 a, b;\n mov.b32 {u, v}, %0;\n cvt.f32.f16 a, u;\n"
          " cvt.f32.f16 b, v;\n cvt.rn.bf16x2.f32 %0, b, a;\n mul.rn.bf16x2 %0, %0, %1;\n}"
          : "+r"(h)
          : "r"(by));
    } else {
      asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h) : "r"(by));
    }
    return h;
  };
  r.x = times(r.x);
  r.y = times(r.y);
  return r;
}

// A value's terms in e4m3: x = t1 + t2 (+ t3), each the rest rounded to nearest (8 values, in
// fp16, of a thread; 8 bytes a term).  A rounding leaves at most 1/16 of a value, and of 8 bits of a
// mantissa (bf16) what is left has at most 4, so two terms are exact, of 11 (fp16) three; but
// for what falls below the format's last step, 2^-9 where the largest value of the rows that
// share a power of two is 224 or more: half a step is 2^-17 of that value at most.
template <int TERMS>
__device__ __forceinline__ void split_terms(const uint4& x, uint2 (&out)[TERMS]) {
  uint32_t h[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int t = 0; t < TERMS; ++t) {
    uint16_t p[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(p[k]) : "r"(h[k]));
      if (t + 1 < TERMS)  // (exact: the rest is a multiple of the value's last step)
        asm("{\n .reg .b32 y;\n cvt.rn.f16x2.e4m3x2 y, %1;\n sub.rn.f16x2 %0, %0, y;\n}"
            : "+r"(h[k])
            : "h"(p[k]));
    }
    out[t] = make_uint2(uint32_t(p[0]) | uint32_t(p[1]) << 16, uint32_t(p[2]) | uint32_t(p[3]) << 16);
  }
}
// Eight 16-bit values times `by`, a power of two that makes them 448 at most, in fp16: exact
// down to its smallest steps, 2^-33 of the largest.  What is not finite becomes NaN.
template <bool BF>
__device__ __forceinline__ uint4 to_half(const uint4& u, float by) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
    float lo, hi;
    if (BF) {
      lo = __uint_as_float(w << 16);
      hi = __uint_as_float(w & 0xffff0000u);
    } else {
      asm("{\n .reg .b16 u, v;\n mov.b32 {u, v}, %2;\n cvt.f32.f16 %0, u;\n cvt.f32.f16 %1, v;\n}"
          : "=f"(lo), "=f"(hi)
          : "r"(w));
    }
    r[i] = pack16<false>(fmaf(lo, by, lo - lo), fmaf(hi, by, hi - hi));
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}
// The largest size among eight 16-bit values, as 32-bit float bits (of a NaN, a NaN's or more);
// FINITE: among those that are.
template <bool BF, bool FINITE = false>
__device__ __forceinline__ uint32_t size_of(const uint4& u) {
  uint4 x = {u.x & 0x7fff7fffu, u.y & 0x7fff7fffu, u.z & 0x7fff7fffu, u.w & 0x7fff7fffu};
  if (FINITE) {
    auto kept = [](uint32_t w) {
      constexpr uint32_t LOW = BF ? 0x7f80u : 0x7c00u;  // an infinity's bits
      return ((w & 0xffffu) < LOW ? w & 0xffffu : 0u) | (w >> 16 < LOW ? w & 0xffff0000u : 0u);
    };
    x = {kept(x.x), kept(x.y), kept(x.z), kept(x.w)};
  }
  uint32_t m = __vmaxu2(__vmaxu2(x.x, x.y), __vmaxu2(x.z, x.w));
  m = max(m & 0xffffu, m >> 16);
  if (BF) return m << 16;
  float f;
  asm("{\n .reg .b16 u, v;\n mov.b32 {u, v}, %1;\n cvt.f32.f16 %0, u;\n}" : "=f"(f) : "r"(m));
  return __float_as_uint(f) & 0x7fffffffu;
}
// The smallest e with a <= 448 * 2^e (a size's bits), kept in the bytes' range; NOT_FINITE for
// what is not: then the power of two is NaN, whatever the terms are.
constexpr int NOT_FINITE = 127;
__device__ __forceinline__ int exponent_over(uint32_t a) {
  const int e = int(a >> 23) - 127 - 8 + ((a & 0x7fffff) > 0x600000);
  return a >= 0x7f800000u ? NOT_FINITE : min(max(e, -117), 119);
}
__device__ __forceinline__ float power_or_nan(int e) {
  return e == NOT_FINITE ? __int_as_float(0x7fffffff) : power(e);
}

// The copies of a call over 8-bit pages, by a warp with a lane per box of page rows: a
// segment's query terms, its staged tiles' keys' terms, then its cached tiles' keys and values.
// Little is done per tile (pages' numbers are read a tile ahead, places found without a
// division), since a single warp gets an instruction about every ten cycles here (64 trees of 22
// nodes: 289 us with the loop of the 16-bit caches, whose tiles are twice as long, 242 so).
template <int DP, int NQ, bool PAIR, bool BF>
__device__ __forceinline__ void copy_bytes(const AttnParams& A, Ctrl<NQ, PAIR>& C,
                                           unsigned char* smem, volatile int* abort) {
  constexpr int TERMS = TERMS_OF<BF>;
  using SM = Smem<DP, NQ, TERMS, PAIR>;
  constexpr bool TURNS = !PAIR && SM::Q_SLOTS == 2;
  const int lane = int(threadIdx.x) & 31, boxes = TILE / A.box;
  const uint32_t raw = smem_addr(smem) + SM::RAW_AT;
  const int cols = TILE / A.page, rows = TILE - cols * A.page;  // from a tile to the next
  uint32_t k_at = 0, v_at = 0;  // copies of keys and of values
  int segs = 0;
  bool ok = true;
  auto wait = [&](unsigned long long* b, uint32_t parity) {
    ok = ok && warp_wait(smem_addr(b), parity, A.status, abort);
    return ok;
  };
  // the next stage of keys, waited for
  auto key_stage = [&](uint32_t& fb) {
    const uint32_t st = k_at % SM::RAW_K;
    if (!wait(&C.empty[SM::STAGES + st], ((k_at / SM::RAW_K) & 1) ^ 1)) return 0u;
    ++k_at;
    fb = smem_addr(&C.full[SM::STAGES + st]);
    return raw + st * SM::RAW;
  };
  for (;; ++segs) {
    if (!wait(&C.seg_full[segs % SEGS], (segs / SEGS) & 1)) break;
    const Seg s = C.seg[segs % SEGS];
    if (s.n == 0) break;
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&C.seg_empty[segs % SEGS]));
    const int ts = tiles_of(A.N), g = staged_of(A, s), first = s.j0 + g - ts, n = s.n - g;
    // the first cached tile's place of this lane's box, and its page
    int t = first * TILE + lane * A.box, col = t / A.page, row = t - col * A.page, page = 0;
    const int32_t* const table = A.table + size_t(s.b) * A.cols;
    if (n > 0 && lane < boxes && t < s.len) page = __ldg(table + col);
    // (passes before the first use)
    const int slot = TURNS ? segs & 1 : 0;
    if (!wait(&C.q_empty[slot], ((TURNS ? segs >> 1 : segs) & 1) ^ 1)) break;
    if (lane == 0) {
      const uint32_t fb = smem_addr(&C.q_full[slot]);
      mbar_arrive_tx(fb, (PAIR ? 2 : 1) * A.q_rows * DP * TERMS);
#pragma unroll 1
      for (int q = 0; q < (PAIR ? 2 : 1) * TERMS; ++q)
        tma_5d(smem_addr(smem) + (PAIR ? q / TERMS : slot) * SM::Q_BYTES + q % TERMS * SM::TERM, &A.mq,
               fb, 0, 0, s.h, s.b * A.N + (s.mt * (PAIR ? 2 : 1) + q / TERMS) * A.tpt, q % TERMS);
    }
    __syncwarp();
#pragma unroll 1
    for (int i = 0; i < g * TERMS; ++i) {
      uint32_t fb = 0;
      const uint32_t dst = key_stage(fb);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_tx(fb, SM::RAW);
        tma_3d(dst, &A.mkn, fb, 0, (s.j0 + i / TERMS) * TILE, (i % TERMS * A.B + s.b) * A.Hkv + s.h);
      }
      __syncwarp();
    }
#pragma unroll 1
    for (int i = 0; ok && i < n; ++i) {
      // a page outside the pool is read as page 0 (the softmax warps report it and drop the result)
      const int pg = page < 0 || page >= A.num_pages ? 0 : page, r = row;
      const int here = min(boxes, (s.len - (first + i) * TILE + A.box - 1) / A.box);
      t += TILE;
      col += cols;
      row += rows;
      if (row >= A.page) {
        row -= A.page;
        ++col;
      }
      if (i + 1 < n && lane < boxes && t < s.len) page = __ldg(table + col);
      uint32_t fb = 0;
      const uint32_t dst = key_stage(fb);
      if (!ok) break;
      if (lane == 0) mbar_arrive_tx(fb, here * A.box * DP);
      __syncwarp();
      if (lane < here) tma_4d(dst + lane * A.box * DP, &A.mk, fb, 0, r, A.head0 + s.h, pg);
      const uint32_t st = SM::RAW_K + v_at % SM::RAW_V;
      if (!wait(&C.empty[SM::STAGES + st], ((v_at / SM::RAW_V) & 1) ^ 1)) break;
      ++v_at;
      fb = smem_addr(&C.full[SM::STAGES + st]);
      if (lane == 0) mbar_arrive_tx(fb, here * A.box * DP);
      __syncwarp();
      if (lane < here)
        tma_4d(raw + st * SM::RAW + lane * A.box * DP, &A.mv, fb, 0, r, A.head0 + s.h, pg);
      __syncwarp();
    }
    if (!ok) break;
  }
  if (*abort) {  // the copies in flight land before the CTA ends
    const unsigned long long t0 = globaltimer();
    auto land = [&](uint32_t at, unsigned long long* full, uint32_t count) {
      for (uint32_t u = at > count ? at - count : 0; u < at; ++u)
        while (!mbar_try(smem_addr(full + u % count), (u / count) & 1) &&
               globaltimer() - t0 < WAIT_LIMIT_NS) {
        }
    };
    land(k_at, C.full + SM::STAGES, SM::RAW_K);
    land(v_at, C.full + SM::STAGES + SM::RAW_K, SM::RAW_V);
    for (int u = max(0, segs - (TURNS ? 2 : 1)); u <= segs; ++u)
      while (!mbar_try(smem_addr(&C.q_full[TURNS ? u & 1 : 0]), (TURNS ? u >> 1 : u) & 1) &&
             globaltimer() - t0 < WAIT_LIMIT_NS) {
      }
  }
}

// The widening warps: a segment's values, tile by tile, to the storage type.  Cached ones from
// bytes: a thread takes 16, 16 dimensions of a token, and writes two 16-byte pieces of a
// 64-dimension block in the 128-byte swizzle; lanes of a row's two blocks write their pieces in
// opposite order, so that eight lanes fall on eight pieces.  Staged ones are copied as they are.
template <int DP, int NQ, bool PAIR, bool BF>
__device__ __forceinline__ void widen_tiles(const AttnParams& A, Ctrl<NQ, PAIR>& C, Ctrl8<NQ>& C8,
                                            unsigned char* smem, volatile int* abort) {
  using SM = Smem<DP, NQ, TERMS_OF<BF>, PAIR>;
  constexpr int STAGES = SM::STAGES;
  constexpr int PER_ROW = DP / 16;                            // threads of a row
  constexpr int ROWS = 32 * WIDEN_WARPS / PER_ROW;            // rows of a step
  // Steps at once: few rows are bound by this loop's chains (4 nodes, bf16: 182 us with four, 194
  // with one), the others by how much code an SM has to fetch (8 nodes: 262 and 235; 22 nodes: 275
  // and 248).
  constexpr int STEPS = TILE / ROWS, BATCH = NQ == 16 ? 4 : 1;
  static_assert(STEPS % BATCH == 0, "whole rounds");
  const int lane = int(threadIdx.x) & 31;
  const int tid = int(threadIdx.x) & (32 * WIDEN_WARPS - 1), warp = tid >> 5;
  const int row0 = tid / PER_ROW, dim = tid % PER_ROW * 16;
  uint32_t out = 0, raw0 = 0;  // 16-bit stages (tiles), and stages of bytes, so far
  bool ok = true;
  auto wait = [&](unsigned long long* b, uint32_t parity) {
    ok = ok && warp_wait(smem_addr(b), parity, A.status, abort);
  };
  for (int segs = 0;; ++segs) {
    wait(&C.seg_full[segs % SEGS], (segs / SEGS) & 1);
    if (!ok) break;
    const Seg s = C.seg[segs % SEGS];
    if (s.n == 0) break;
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&C.seg_empty[segs % SEGS]));
#pragma unroll 1
    for (int j = 0; j < s.n; ++j, ++out) {
      const Keys ky = keys_of<false, true>(A, s, s.j0 + j);
      const uint32_t st = out % STAGES, rs = SM::RAW_K + raw0 % SM::RAW_V, sc = out % SCALES;
      unsigned char* const dst = smem + SM::STAGE_AT + st * SM::BYTES;
      wait(&C.empty[st], ((out / STAGES) & 1) ^ 1);
      wait(&C8.full[sc], (out / SCALES) & 1);
      if (!ky.staged) wait(&C.full[STAGES + rs], (raw0 / SM::RAW_V) & 1);
      if (!ok) break;
      if (ky.staged) {
        if (lane == 0) {
          const uint32_t fb = smem_addr(&C.full[st]);
          mbar_arrive(smem_addr(&C8.empty[sc]));
          if (warp == 0) {
            mbar_arrive_tx(fb, SM::BYTES);
            for (int x = 0; x < DP / 64; ++x)
              tma_3d(smem_addr(dst) + x * 16384, &A.mvn, fb, x * 64, ky.k0,
                     s.b * A.LH + A.head0 + s.h);
          } else {
            mbar_arrive(fb);
          }
        }
        __syncwarp();
        continue;
      }
      // a row's 16 dimensions of the tile
      auto put = [&](int row, const uint4& lo, const uint4& hi) {
        unsigned char* const line = dst + (dim >> 6) * 16384 + row * 128;
        const int at = dim >> 3 & 7, swap = dim >> 6;
        *reinterpret_cast<uint4*>(line + (((at + swap) ^ (row & 7)) << 4)) = swap ? hi : lo;
        *reinterpret_cast<uint4*>(line + (((at + 1 - swap) ^ (row & 7)) << 4)) = swap ? lo : hi;
      };
      const unsigned char* const src = smem + SM::RAW_AT + rs * SM::RAW + tid * 16;
#pragma unroll 1
      for (int g = 0; g < STEPS; g += BATCH) {
        uint4 b[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
          b[i] = *reinterpret_cast<const uint4*>(src + (g + i) * (32 * WIDEN_WARPS * 16));
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          const int row = row0 + (g + i) * ROWS;
          const uint32_t by = C8.tile[sc].vf[row >> 3];
          const uint2 p = widen4<BF>(b[i].x, by), q = widen4<BF>(b[i].y, by);
          const uint2 y = widen4<BF>(b[i].z, by), z = widen4<BF>(b[i].w, by);
          put(row, make_uint4(p.x, p.y, q.x, q.y), make_uint4(y.x, y.y, z.x, z.y));
        }
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_addr(&C.empty[STAGES + rs]));
        mbar_arrive(smem_addr(&C8.empty[sc]));
      }
      ++raw0;
      // behind the entries: whatever the bytes are, weights of 0 take zeros
      const int w = width_of(ky);
      if (ky.n < w) {
#pragma unroll 1
        for (int row = row0; row < w; row += ROWS)
          if (row >= ky.n) put(row, make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0));
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&C.full[st]));
    }
    if (!ok) break;
  }
  if (*abort) {  // a staged copy in flight lands before the CTA ends
    const unsigned long long t0 = globaltimer();
    for (uint32_t u = out > STAGES ? out - STAGES : 0; u < out; ++u)
      while (!mbar_try(smem_addr(&C.full[u % STAGES]), (u / STAGES) & 1) &&
             globaltimer() - t0 < WAIT_LIMIT_NS) {
      }
  }
}

// The scales of every segment's tiles, as powers of two of eight tokens each, up to SCALES
// tiles ahead: staged ones as the first kernel left them, cached ones as many tiles at once
// as their blocks fill lanes, since the loads of a page's number and then of its scales take
// longer than a tile does.
template <int NQ, bool PAIR, bool BF>
__device__ __forceinline__ void read_scales(const AttnParams& A, Ctrl<NQ, PAIR>& C, Ctrl8<NQ>& C8,
                                            volatile int* abort) {
  const int lane = int(threadIdx.x) & 31;
  const int log = 7 - A.block_log, blocks = 1 << log;  // of a tile
  const int mine = lane >> log, block = lane & (blocks - 1), per_page = A.page >> A.block_log;
  const int at_once = min(32 >> log, 4), rep = 1 << (A.block_log - 3);
  uint32_t tiles = 0;
  bool ok = true;
  for (int segs = 0; ok; ++segs) {
    ok = warp_wait(smem_addr(&C.seg_full[segs % SEGS]), (segs / SEGS) & 1, A.status, abort);
    if (!ok) break;
    const Seg s = C.seg[segs % SEGS];
    if (s.n == 0) break;
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&C.seg_empty[segs % SEGS]));
    const int g = staged_of(A, s), ts = tiles_of(A.N);
#pragma unroll 1
    for (int j = 0; ok && j < s.n;) {
      const int count = j < g ? 1 : min(at_once, s.n - j);
      int k = 0, v = 0;  // (blocks behind the entries: any)
      bool nan = false;
      float staged = 0.0f;
      if (j < g) {
        if (lane < 16)
          staged = __ldcg(A.kf + ((size_t(s.b) * A.Hkv + s.h) * ts + s.j0 + j) * 16 + lane);
      } else {
        const int t = (s.j0 + j - ts + mine) * TILE + (block << A.block_log);
        if (mine < count && t < s.len) {
          const int col = t / A.page;
          int pg = __ldg(A.table + size_t(s.b) * A.cols + col);
          if (pg < 0 || pg >= A.num_pages) pg = 0;  // (reported, and its result dropped, elsewhere)
          const size_t at = (size_t(pg) * A.LH + A.head0 + s.h) * per_page +
                            ((t - col * A.page) >> A.block_log);
          k = int(__ldg(A.k_scales + at)) - 127;
          v = int(__ldg(A.v_scales + at)) - 127;
          // exponents at which dtype does not hold every value: NaN
          const int lo = BF ? -117 : -15, hi = BF ? 119 : 7;
          nan = k < lo || k > hi || v < lo || v > hi;
          if (nan) k = v = 0;
        }
      }
      const float kf = power(k);
      uint32_t vf = nan ? 0x7fffu : BF ? uint32_t(v + 127) << 7 : v < -14 ? 0x200u : uint32_t(v + 15) << 10;
      vf |= vf << 16;
#pragma unroll 1
      for (int x = 0; x < count; ++x, ++tiles) {
        const uint32_t sc = tiles % SCALES;
        ok = warp_wait(smem_addr(&C8.empty[sc]), ((tiles / SCALES) & 1) ^ 1, A.status, abort);
        if (!ok) break;
        Tile8& t8 = C8.tile[sc];
        if (j < g) {
          if (lane < 16) t8.kf[lane] = staged;
        } else if (mine == x) {
#pragma unroll 1
          for (int i = block * rep; i < block * rep + rep; ++i) {
            t8.kf[i] = kf;
            t8.vf[i] = vf;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&C8.full[sc]));
      }
      j += count;
    }
  }
}

// -------------------------------------------------------------- queries and staged entries

// What the kernel before the attention over 8-bit pages makes of the queries and the staged
// keys, so that they arrive there by copies like everything else: the terms of both and their
// powers of two.  (Made by the attention kernel's own warps first: 6 us more per item, in which
// the tiles waited.)
struct Prep8 {
  const uint16_t* q;
  const uint16_t* k_new;
  uint8_t* q8;    // [TERMS][B][N][Hq][D]
  uint8_t* k8;    // [TERMS][B][Hkv][N][D]
  float* qf;      // [B][N][Hq]
  float* kf;      // [B][Hkv][tiles][16]
  int B, N, Hq, Hkv, D, LH, head0;
};
constexpr int PREP_THREADS = 128, PREP_ROWS = 64;  // query rows of a CTA
inline long long prep8_blocks(const Prep8& P) {
  return (long long)P.B * P.Hkv * ((P.N + TILE - 1) / TILE) +
         ((long long)P.B * P.N * P.Hq + PREP_ROWS - 1) / PREP_ROWS;
}

// The first B * Hkv * tiles CTAs a staged tile each, eight keys of which share a power of two;
// the others PREP_ROWS query rows.  A thread takes 16 dimensions of a row.
template <int DP, bool BF>
__global__ void __launch_bounds__(PREP_THREADS) sv_attn8_prep(const __grid_constant__ Prep8 P) {
  constexpr int TERMS = TERMS_OF<BF>, PER_ROW = DP / 16, WARP_ROWS = 32 / PER_ROW;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = int(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int dim = lane % PER_ROW * 16, lane_row = lane / PER_ROW;
  struct Row { uint4 lo, hi; };
  auto fetch = [&](const uint16_t* src, bool on) {  // zeros where there is nothing
    Row r = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (on && dim < P.D) {
      r.lo = __ldg(reinterpret_cast<const uint4*>(src + dim));
      r.hi = __ldg(reinterpret_cast<const uint4*>(src + dim) + 1);
    }
    return r;
  };
  auto size = [](const Row& r) { return max(size_of<BF>(r.lo), size_of<BF>(r.hi)); };
  auto terms = [&](const Row& u, int e, uint8_t* to, size_t stride) {
    const float by = power(-min(e, 119));
    uint2 lo[TERMS], hi[TERMS];
    split_terms<TERMS>(to_half<BF>(u.lo, by), lo);
    split_terms<TERMS>(to_half<BF>(u.hi, by), hi);
#pragma unroll
    for (int t = 0; t < TERMS; ++t)
      *reinterpret_cast<uint4*>(to + t * stride + dim) = make_uint4(lo[t].x, lo[t].y, hi[t].x, hi[t].y);
  };
  const int ts = tiles_of(P.N);
  const long long staged = (long long)P.B * P.Hkv * ts;
  if (blockIdx.x < staged) {
    const int tile = int(blockIdx.x) % ts, bh = int(blockIdx.x) / ts, b = bh / P.Hkv, h = bh - b * P.Hkv;
    const int k0 = tile * TILE, n = min(TILE, P.N - k0);
    const size_t from = ((size_t(b) * P.LH + P.head0 + h) * P.N + k0) * P.D;
    const size_t to = (size_t(bh) * P.N + k0) * P.D, stride = size_t(P.B) * P.Hkv * P.N * P.D;
    for (int g = warp; g < 16; g += PREP_THREADS / 32) {
      constexpr int V = 8 / WARP_ROWS;  // rows of a lane
      Row k[V];
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int row = g * 8 + i * WARP_ROWS + lane_row;
        k[i] = fetch(P.k_new + from + size_t(row) * P.D, row < n);
        most = max(most, size(k[i]));
      }
      int e = exponent_over(__reduce_max_sync(0xffffffffu, most));
      if (e == NOT_FINITE) {  // (those become NaN by themselves, and the others keep their bits)
        most = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
          most = max(most, max(size_of<BF, true>(k[i].lo), size_of<BF, true>(k[i].hi)));
        e = exponent_over(__reduce_max_sync(0xffffffffu, most));
      }
      if (lane == 0) P.kf[size_t(blockIdx.x) * 16 + g] = power(e);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int row = g * 8 + i * WARP_ROWS + lane_row;
        if (row < n && dim < P.D) terms(k[i], e, P.k8 + to + size_t(row) * P.D, stride);
      }
    }
    return;
  }
  const long long rows = (long long)P.B * P.N * P.Hq, r0 = (blockIdx.x - staged) * PREP_ROWS;
#pragma unroll
  for (int i = 0; i < PREP_ROWS / (4 * WARP_ROWS); ++i) {
    const long long r = r0 + (i * 4 + warp) * WARP_ROWS + lane_row;
    const Row u = fetch(P.q + r * P.D, r < rows);
    uint32_t most = size(u);
#pragma unroll
    for (int k = 1; k < PER_ROW; k *= 2)  // (a row's lanes are neighbours)
      most = max(most, __shfl_xor_sync(0xffffffffu, most, k));
    const int e = exponent_over(most);
    if (r < rows && dim < P.D) terms(u, e, P.q8 + r * P.D, size_t(rows) * P.D);
    if (r < rows && dim == 0) P.qf[r] = power_or_nan(e);
  }
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
// 8-bit caches (Q8) add
//   widen     four warps: cached values from bytes to the storage type
//   scales    the blocks' powers of two, a few tiles ahead
template <int DP, int NQ, bool PAIR, bool PR, bool BF, bool Q8 = false>
__global__ void __launch_bounds__(Q8 ? THREADS8 : THREADS, 1)
    sv_attn(const __grid_constant__ AttnParams A) {
  static_assert(!(NQ && (PAIR || PR)), "few rows make one tile, and prompts have many");
  static_assert(!(Q8 && PR), "8-bit entries are in pages");
  constexpr int TERMS = Q8 ? TERMS_OF<BF> : 0;
  using SM = Smem<DP, NQ, TERMS, PAIR>;
  constexpr int NT = Q8 ? THREADS8 : THREADS;
  constexpr int STAGES = SM::STAGES, BYTES = SM::BYTES, HALVES = DP / 64;
  constexpr int ROWS = NQ ? NQ : PAIR ? 2 * TILE : TILE;
  constexpr int TM_COLS = NQ ? 256 : 512;               // TMEM: S of both streams, then O
  constexpr int S_COLS = NQ ? 64 : 128, O_AT = TM_COLS / 2;
  extern __shared__ __align__(1024) unsigned char smem[];
  Ctrl<NQ, PAIR>& C = *reinterpret_cast<Ctrl<NQ, PAIR>*>(smem + SM::CTRL);
  Ctrl8<NQ>& C8 = *reinterpret_cast<Ctrl8<NQ>*>(smem + SM::CTRL + (Q8 ? CTRL_BYTES : 0));  // Q8
  const uint32_t base = smem_addr(smem);
  const int tid = int(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  auto bar = [&](unsigned long long* p) { return smem_addr(p); };

  // ---- set-up: barriers, TMEM, and where this CTA's run of tiles starts
  if (tid == 0) {
    for (int i = 0; i < STAGES; ++i) {
      // (withheld: one arrival too many, and every wait for that stage runs out)
      const int arrivals = Q8 ? WIDEN_WARPS : 1;
      const bool withheld = A.withhold && blockIdx.x == 0 && i == (Q8 ? 0 : 1);
      mbar_init(bar(&C.full[i]), withheld ? arrivals + 1 : arrivals);
      mbar_init(bar(&C.empty[i]), 1);
    }
    if (Q8) {
      for (int i = STAGES; i < STAGES + SM::RAWS; ++i) {
        mbar_init(bar(&C.full[i]), 1);
        mbar_init(bar(&C.empty[i]), i < STAGES + SM::RAW_K ? 1 : WIDEN_WARPS);
      }
      for (int i = 0; i < SCALES; ++i) {
        mbar_init(bar(&C8.full[i]), 1);
        mbar_init(bar(&C8.empty[i]), (PAIR ? 8 : 4) + WIDEN_WARPS);
      }
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
      mbar_init(bar(&C.seg_empty[i]), 8 + 2 + (Q8 ? WIDEN_WARPS + 1 : 0));  // its readers
    }
    mbar_init(bar(&C.drain), 1);
    mbar_init(bar(&C.next_full), 1);
    C.abort = 0;
    C.start_b = 0;
    C.start_at = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == (Q8 ? MMA8_WARP : MMA_WARP)) {
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
    for (int i = tid; i < SM::P_AT / 16; i += NT)
      reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  long long run = 0;  // tiles of this CTA (TREE, RING)
  bool whole_items = false;
  if (!PR) {
    // thread t sums requests t * per .. of the batch
    const int per = (A.B + NT - 1) / NT;
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
    for (int w = 0; w < NT / 32; ++w) {
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
  // (the first kernel of a call over 8-bit pages: its outputs are there from here on, for copies and
  // ordinary loads; it may have run beside this one, which read-only loads do not allow)
  if (Q8) asm volatile("griddepcontrol.wait;" ::: "memory");
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
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Regs<NQ, Q8>::SOFTMAX));
    // ------------------------------------------------------------ softmax
    const int st = warp >> 2;             // the stream of this warpgroup
    const int row = tid & (TILE - 1);     // query row of the tile, and key of a value tile
    const int rt = row / A.G, rg = row - rt * A.G;
    const uint32_t lanes = uint32_t(warp & 3) << 21;  // this warp's TMEM lanes
    const uint32_t ts = tmem + lanes + st * S_COLS, to = tmem + lanes + O_AT + st * S_COLS;
    uint32_t idx = 0, tiles8 = 0;  // (Q8: tiles before the segment)
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
      const int staged = Q8 ? staged_of(A, s) : 0;  // (the first tiles)
      // the segment's cached tiles, of the request's, and whether it has staged ones
      const int c0 = Q8 ? max(s.j0 - tiles_of(A.N), 0) : s.j0;
      const int c1 = Q8 ? s.j0 + n - tiles_of(A.N) : s.j0 + n;
      const bool has_staged = Q8 ? staged > 0 : s.j0 + n > ct;
      float qf = 1.0f;  // Q8: the row's power of two
      if (Q8) {
        const int r = NQ ? row : rt, t = NQ ? row / A.G : tok;  // (column `row` is of token row / G)
        const bool on = NQ ? row < A.N * A.G : active;
        if (on)
          qf = __ldcg(A.qf + (size_t(s.b) * A.N + t) * A.Hq + s.h * A.G + (NQ ? row - t * A.G : rg));
        if (NQ && r < NQ) C8.qf[st][row] = qf;
      }
      int bad = s.bad;
      if (!PR && (Q8 || A.kind == TREE)) {
        // pages in use by this segment, and the parent array
        int pages_bad = 0;
        const int t1 = min(s.len, c1 * TILE);
        if (c0 * TILE < t1)
          for (int c = c0 * TILE / A.page + row; c <= (t1 - 1) / A.page; c += TILE) {
            const int pg = __ldg(A.table + size_t(s.b) * A.cols + c);
            pages_bad |= pg < 0 || pg >= A.num_pages;
          }
        if (A.parent && s.b != parent_b && has_staged) {
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
        if (has_staged && A.parent) bad |= parent_bad;
      }
      if (bad && tid == 0) set_status(A.status, bad);
      const int ring_at = PR || Q8 ? -1 : s.ring;  // (8-bit entries are in pages)
      const bool ring_full = !PR && !Q8 && s.full;
      const int q0 = s.mt * tpi, q1 = min(q0 + tpi, tokens) - 1;  // the item's tokens
      const int w0 = q0 + (PAIR ? st * A.tpt : 0), w1 = min(w0 + A.tpt, tokens) - 1;  // the tile's

      const float lift = BF && !Q8 ? 0.0f : A.lift, raise = BF ? MOST_BF16 : MOST_F16 - A.lift;
      const float unit = Q8 ? 1.0f : A.c;  // of the maxima, in base-2 units
      float m = -INFINITY, l = 0.0f;
      float lq[NQ ? NQ : 1];  // NQ > 0: this key's share of the columns' sums
      bool unset = true;      // NQ > 0: a column has seen nothing yet
#pragma unroll
      for (int q = 0; q < NQ; ++q) lq[q] = 0.0f;
      int done = 0;
      for (int jj = PAIR ? 0 : st; jj < n; jj += PAIR ? 1 : 2, ++done) {
        const int j = s.j0 + jj;
        const Keys ky = keys_of<PR, Q8>(A, s, j);
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
        if (Q8) clean = false;  // (the widening warps' rows behind the entries are zeros)
        // (With keys on the lanes the warps meet at barriers within a tile: after a
        // wait that gave up they walk the rest of the segment's tiles together.)
        ok = ok && warp_wait(bar(&C.s_full[st]), s_use & 1, A.status, abort);
        if (NQ == 0 && !ok) break;
        ++s_use;
        tc_after();
        // Q8: the tile's powers of two
        const Tile8* t8 = nullptr;
        const uint32_t tile8 = tiles8 + jj, sc = tile8 % SCALES;
        if (Q8) {
          t8 = &C8.tile[sc];
          ok = ok && warp_wait(bar(&C8.full[sc]), (tile8 / SCALES) & 1, A.status, abort);
          if (NQ == 0 && !ok) break;
        }
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
          softmax_few<NQ, BF, Q8>(A, C, st, row, ts, to, sees, masked, done > 0, unset, lq,
                                  smem + SM::P_AT + st * SM::P_BYTES,
                                  t8->kf, C8.qf[st]);
        } else if (!warp_active) {
          __syncwarp();
          half_done();
        } else {
          // Q8: what the scores of eight keys are multiplied by
          float qc = 0.0f, spoilt = 0.0f;
          if (Q8) {
            qc = A.c * qf;
            spoilt = qc - qc;  // NaN with the row's power of two, else 0
          }
          auto factors = [&](int x) {  // (not 0: hidden scores stay at -infinity)
            const float4 k = *reinterpret_cast<const float4*>(t8->kf + 4 * x);
            return make_float4(fmaxf(qc * k.x, 1e-37f), fmaxf(qc * k.y, 1e-37f),
                               fmaxf(qc * k.z, 1e-37f), fmaxf(qc * k.w, 1e-37f));
          };
          auto most = [&](int x, uint32_t (&r)[32]) {  // the largest of 32 scores
            const float4 f = factors(x);
            float t[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              auto v = [&](int i) { return __uint_as_float(r[8 * g + i]); };
              t[g] = fmaxf(fmaxf(fmaxf(v(0), v(1)), v(2)),
                           fmaxf(fmaxf(fmaxf(v(3), v(4)), v(5)), fmaxf(v(6), v(7))));
            }
            return fmaxf(fmaxf(t[0] * f.x, t[1] * f.y), fmaxf(t[2] * f.z, t[3] * f.w));
          };
          // the weights of 32 keys, and their sum
          auto weigh = [&](int x, const uint32_t (&r)[32], float nm, uint32_t (&pw)[16],
                           float2 (&sum)[4]) {
            const float4 f = factors(x);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const float fg = g == 0 ? f.x : g == 1 ? f.y : g == 2 ? f.z : f.w;
#pragma unroll
              for (int i = 4 * g; i < 4 * g + 4; ++i) {
                const float2 e = fma2(
                    make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])),
                    make_float2(fg, fg), make_float2(nm, nm));
                const float2 p = make_float2(ex2(e.x), ex2(e.y));
                sum[i & 3] = add2(sum[i & 3], p);
                pw[i] = pack16<BF>(p.x, p.y);
              }
            }
          };
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
              const bool rise = active && (mt - m) * unit > raise;  // (-inf before: always)
              if (__any_sync(0xffffffffu, rise)) {
                const float f = rise ? ex2((m - mt) * unit) : 1.0f;
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
          if constexpr (Q8) {
            // 32 scores at a time, for the maximum and again for the weights, in loops that are
            // not unrolled: with the powers of two the code of a whole tile is longer than what
            // is fetched in time (64 trees of 88 rows: 447 us unrolled, 344 so).
            uint32_t see[4] = {~0u, ~0u, ~0u, ~0u};
            if (masked) {
              visible(see);
#pragma unroll
              for (int x = 0; x < 4; ++x) see[x] &= span(0, w, 32 * x);
            }
            auto scores = [&](int x, uint32_t (&r)[32]) {
              tm_ld32(ts + x * 32, r);
              tm_wait_ld(r);
              if (masked) {
                const uint32_t bits = x == 0 ? see[0] : x == 1 ? see[1] : x == 2 ? see[2] : see[3];
                if (!__all_sync(0xffffffffu, bits == 0xffffffffu)) {
#pragma unroll
                  for (int i = 0; i < 32; ++i)
                    if (!(bits >> i & 1)) r[i] = 0xff800000u;
                }
              }
            };
            float mt = -INFINITY;
#pragma unroll 1
            for (int x = 0; x * 32 < w; ++x) {
              uint32_t r[32];
              scores(x, r);
              mt = fmaxf(mt, most(x, r));
            }
            raise_to(mt);
            const float nm = (m == -INFINITY ? 0.0f : lift - m) + spoilt;
            float2 sum[4] = {};
#pragma unroll 1
            for (int x = 0; x * 32 < w; ++x) {  // (P's columns lie over scores that are done with)
              uint32_t r[32], pw[16];
              scores(x, r);
              weigh(x, r, nm, pw, sum);
              tm_st16(ts + x * 16, pw);
              if (x == 1) half_done();
            }
            if (w <= 32) {
              __syncwarp();
              half_done();
            }
            sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
            l += sum[0].x + sum[0].y;
            __syncwarp();
          } else if constexpr (PAIR) {
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
        if (lane == 0) {
          mbar_arrive(bar(&C.p_full[st]));
          if (Q8) mbar_arrive(bar(&C8.empty[sc]));
        }
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
          if (!whole && active)
            A.part_ml[part] = make_float2(m * unit, bad ? -1.0f : l);
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
          float f0 = ex2((a.x - mu) * unit), f1 = ex2((b.x - mu) * unit);
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
            A.part_ml[part] = make_float2(mm * unit, bad ? -1.0f : ll);
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
      tiles8 += n;
      seg_done(segs);
      ++segs;
    }
    if (!PR && A.join && tid == 0) A.desc[blockIdx.x] = make_int4(d_flags, d_item, d_b, 0);
  } else {
    __syncwarp();
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<NQ, Q8>::OTHER));
  if (Q8 && warp < 8 + WIDEN_WARPS) {
    if constexpr (Q8) widen_tiles<DP, NQ, PAIR, BF>(A, C, C8, smem, abort);
  } else if (warp == (Q8 ? PLAN8_WARP : PLAN_WARP)) {
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
  } else if (warp == (Q8 ? COPY8_WARP : COPY_WARP)) {
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
    if constexpr (Q8) {
      copy_bytes<DP, NQ, PAIR, BF>(A, C, smem, abort);
    } else if (PR || A.kind == RING) {
      if (elect_one()) copies(Yes<true>());
      __syncwarp();
    } else {
      copies(Yes<false>());
    }
  } else if (Q8 && warp == SCALE_WARP) {
    if constexpr (Q8) read_scales<NQ, PAIR, BF>(A, C, C8, abort);
  } else if (warp == (Q8 ? MMA8_WARP : MMA_WARP)) {
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
    if constexpr (Q8) {
      const uint32_t id_8 = instr_desc8(NQ);  // (0: the tile's width goes there)
      uint32_t raw0 = 0;                      // stages of keys before the segment
      while (ok) {
        ok = mbar_wait(bar(&C.seg_full[segs % AHEAD]), (segs / AHEAD) & 1, A.status, abort);
        if (!ok) break;
        const Seg s = C.seg[segs % AHEAD];
        if (s.n == 0) break;
        mbar_arrive(bar(&C.seg_empty[segs % AHEAD]));
        constexpr bool TURNS = !PAIR && SM::Q_SLOTS == 2;
        const int slot = TURNS ? segs & 1 : 0, use = TURNS ? segs >> 1 : segs;
        ok = mbar_wait(bar(&C.q_full[slot]), use & 1, A.status, abort);
        tc_after();
        const int n = s.n, g = staged_of(A, s);
        // (tiles are whole but for the staged and the last cached ones)
        auto width = [&](int j) {
          return j >= g && j + 1 < n ? TILE : width_of(keys_of<PR, Q8>(A, s, s.j0 + j));
        };
        // S[st] (+)= the terms of query tile q with the term of keys at `ka`
        auto term = [&](int st, int q, uint32_t ka, int w, bool more) {
          const uint32_t id = NQ ? id_8 : id_8 | uint32_t(w >> 3) << 17;
          const uint32_t dk = desc_rows(ka), dq = desc_rows(base + q * SM::Q_BYTES);
#pragma unroll
          for (int t = 0; t < TERMS; ++t)
#pragma unroll
            for (int k = 0; k < DP / 32; ++k) {
              if (k * 32 >= A.D) break;
              const uint32_t a = dq + ((t * SM::TERM + k * 32) >> 4), b = dk + ((k * 32) >> 4);
              mma8_ss<DP>(tmem + st * S_COLS, NQ ? b : a, NQ ? a : b, id, more || t > 0 || k > 0);
            }
        };
        // One copy of the scores' code: step j first finishes tile j - AHEAD8's values.
        constexpr int AHEAD8 = PAIR ? 1 : 2;
#pragma unroll 1
        for (int i = 0; ok && i < n + AHEAD8; ++i) {
          const int j = i - AHEAD8;  // the tile whose weights are next
          const bool raw = i >= g && i < n;
          const uint32_t ku = raw0 + (i < g ? i * TERMS : g * TERMS + i - g), ks = ku % SM::RAW_K;
          auto raw_here = [&](uint32_t u) {
            if (!mbar_wait(bar(&C.full[STAGES + u % SM::RAW_K]), (u / SM::RAW_K) & 1, A.status, abort))
              return false;
            tc_after();
            return true;
          };
          const uint32_t uv = idx + j;
          const int w = width(j);
          if (j >= 0) ok = full(uv);
          if (raw) ok = ok && raw_here(ku);
#pragma unroll
          for (int x = 0; x < (PAIR ? 2 : 1); ++x) {
            const int st = PAIR ? x : i & 1;
            if (j >= 0) {
              ok = ok && first_half(st, uv, w, j > 0) &&
                   mbar_wait(bar(&C.p_full[st]), p_use[st] & 1, A.status, abort);
              ++p_use[st];
              if (!ok) break;
              tc_after();
              values(st, uv, w, PAIR || j >= 2, PAIR ? 4 : 0, 8);
              if (!PAIR || x == 1) mma_commit(bar(&C.empty[uv % STAGES]));
              if (i >= n) mma_commit(bar(&C.o_full[st]));
            }
            if (ok && raw) {
              term(st, PAIR ? x : slot, base + SM::RAW_AT + ks * SM::RAW, width(i), false);
              mma_commit(bar(&C.s_full[st]));
              if (!PAIR || x == 1) mma_commit(bar(&C.empty[STAGES + ks]));
            }
          }
          if (i < g) {  // a staged tile, by its keys' terms (pairs: for both query tiles)
            const int st = PAIR ? 0 : i & 1;
#pragma unroll 1
            for (int y = 0; ok && y < TERMS; ++y) {
              const uint32_t u = ku + y, at = base + SM::RAW_AT + u % SM::RAW_K * SM::RAW;
              ok = raw_here(u);
              if (!ok) break;
#pragma unroll 1
              for (int x = 0; x < (PAIR ? 2 : 1); ++x)
                term(st + x, PAIR ? x : slot, at, width(i), y > 0);
              mma_commit(bar(&C.empty[STAGES + u % SM::RAW_K]));
            }
            mma_commit(bar(&C.s_full[st]));
            if (PAIR) mma_commit(bar(&C.s_full[st + 1]));
          }
          if (ok && i + 1 == n) mma_commit(bar(&C.q_empty[slot]));  // (queries done with)
        }
        idx += n;
        raw0 += n - g + TERMS * g;
        ++segs;
      }
    }
    while (!Q8 && ok) {
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
  if (warp == (Q8 ? MMA8_WARP : MMA_WARP)) {
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

template <int DP, int NQ, bool PAIR, bool PR, bool BF, bool Q8 = false>
int launch_as(const AttnParams& A, int device, int grid, int ctas, cudaStream_t st) {
  // the kernel's shared-memory limit, raised once per device (ordinals past 63: every time)
  static std::atomic<uint64_t> raised{0};
  const uint64_t mark = device < 64 ? uint64_t(1) << device : 0;
  if (!(raised.load(std::memory_order_acquire) & mark)) {
    if (cudaFuncSetAttribute(sv_attn<DP, NQ, PAIR, PR, BF, Q8>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (Smem<DP, NQ, Q8 ? TERMS_OF<BF> : 0, PAIR>::TOTAL)) != cudaSuccess)
      return SV_ERR_CUDA;
    raised.fetch_or(mark, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (Q8) {  // (sets up beside the kernel that splits the queries)
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(THREADS8);
    cfg.dynamicSmemBytes = Smem<DP, NQ, Q8 ? TERMS_OF<BF> : 0, PAIR>::TOTAL;
    if (cudaLaunchKernelEx(&cfg, sv_attn<DP, NQ, PAIR, PR, BF, Q8>, A) != cudaSuccess)
      return SV_ERR_CUDA;
    cfg.dynamicSmemBytes = 0;
  } else {
    sv_attn<DP, NQ, PAIR, PR, BF, Q8><<<grid, THREADS, (Smem<DP, NQ>::TOTAL), st>>>(A);
    if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  }
  if (PR || !A.join) return SV_OK;
  cfg.gridDim = dim3(unsigned(JOIN_BLOCKS * ctas));
  cfg.blockDim = dim3(JOIN_WARPS * 32);
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

// The same over an 8-bit cache.
template <int DP, bool BF>
int launch_dp8(const AttnParams& A, const Prep8& P, Layout l, int device, int grid, int ctas,
               cudaStream_t st) {
  const long long blocks = prep8_blocks(P);
  if (blocks > 0x7fffffffLL) return SV_ERR_INVALID_ARG;
  sv_attn8_prep<DP, BF><<<unsigned(blocks), PREP_THREADS, 0, st>>>(P);
  if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  if (l.nq == 16) return launch_as<DP, 16, false, false, BF, true>(A, device, grid, ctas, st);
  if (l.nq == 32) return launch_as<DP, 32, false, false, BF, true>(A, device, grid, ctas, st);
  if (l.rows == TILE) return launch_as<DP, 0, false, false, BF, true>(A, device, grid, ctas, st);
  return launch_as<DP, 0, true, false, BF, true>(A, device, grid, ctas, st);
}

// One translation unit per storage type and cache (attn_bf16.cu, attn_f16.cu, attn8_bf16.cu,
// attn8_f16.cu), compiled side by side.
int launch_bf16(const AttnParams& A, Layout l, int device, int grid, int ctas, cudaStream_t st);
int launch_f16(const AttnParams& A, Layout l, int device, int grid, int ctas, cudaStream_t st);
int launch8_bf16(const AttnParams& A, const Prep8& P, Layout l, int device, int grid, int ctas,
                 cudaStream_t st);
int launch8_f16(const AttnParams& A, const Prep8& P, Layout l, int device, int grid, int ctas,
                cudaStream_t st);

}  // namespace svattn

#endif  // SV_ATTENTION_CUH
