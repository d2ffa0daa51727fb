// attn_plan_probe.cu -- asks the attention kernels' plan of prompt items (Cursor of
// attention.cuh) for items in a given order and writes down what it answers.  Built
// and called by test_gpu_attn_plan.py.

#include "attention.cuh"

namespace {

template <bool PAIR>
__global__ void probe(svattn::AttnParams A, const long long* ids, int n, int32_t* out) {
  svattn::Cursor<PAIR, true> cur;
  svattn::Seg s = {};
  cur.open(A, false);
  for (int k = 0; k < n; ++k) {
    const bool have = cur.item(A, ids[k], s, false);
    if (threadIdx.x == 0) {
      int32_t* const o = out + 5 * k;
      o[0] = have;
      o[1] = s.b;
      o[2] = s.h;
      o[3] = s.mt;
      o[4] = s.nt;
    }
  }
}

}  // namespace

extern "C" int plan_items(const int32_t* cu, int B, int T, int Hkv, int tpt, int pair, int sink,
                          int window, const long long* ids, int n, int32_t* out, void* stream) {
  svattn::AttnParams A = {};
  A.kind = svattn::PROMPT;
  A.lens = cu;
  A.B = B; A.T = T; A.Hkv = Hkv; A.tpt = tpt; A.sink = sink; A.window = window;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (pair) probe<true><<<1, 32, 0, st>>>(A, ids, n, out);
  else probe<false><<<1, 32, 0, st>>>(A, ids, n, out);
  return int(cudaGetLastError());
}
