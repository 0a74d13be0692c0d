// Causal attention over packed prompts: o_i = sum_{j <= i} softmax_j(scale q_i . k_j) v_j.
// One warp per (token, query head).
#include "attn_common.cuh"

namespace gdn {

namespace {

// The sequence that holds token t, as [start, start + i], or start = -1: the entries of a
// malformed table are clamped to [0, T] and raised to the largest entry before them, so
// the first entry that passes t ends the sequence.
__device__ int seq_start(const int32_t* cu, int N, int T, int t) {
  if (!cu) return 0;
  int last = min(max(cu[0], 0), T);
  if (t < last) return -1;
  for (int n = 1; n <= N; ++n) {
    const int e = max(last, min(max(cu[n], 0), T));
    if (t < e) return last;
    last = e;
  }
  return -1;
}

template <int D>
__global__ void __launch_bounds__(128) prefill_rows_kernel(AttnParams p) {
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.cu && p.status) {
    int last = 0;
    for (int n = 0; n <= p.N; ++n) {
      if (p.cu[n] < last || p.cu[n] > p.T) set_status(p.status, GDN_DEV_BAD_CU_SEQLENS);
      last = max(last, p.cu[n]);
    }
  }
  if (w >= (int64_t)p.T * p.H) return;
  const int t = (int)(w / p.H), h = (int)(w % p.H);
  const int start = seq_start(p.cu, p.N, p.T, t);
  if (start < 0) return;
  const size_t kv = ((size_t)start * p.Hk + h / p.G) * D, step = (size_t)p.Hk * D;
  float o[D / 32], lse;
  attn_row<D>(p.q + (size_t)w * D, t - start + 1, p.scale,
              [&](int j) { return p.k + kv + j * step; },
              [&](int j) { return p.v + kv + j * step; }, o, lse);
  store_row<D>(p.out, p.out_bf16, (size_t)w, o);
  if (p.lse && (threadIdx.x & 31) == 0) p.lse[w] = lse;
}

}  // namespace

bool launch_attn_prefill(const AttnParams& p, cudaStream_t s) {
  const int64_t blocks = ((int64_t)p.T * p.H + 3) / 4;
  if (p.D == 128) prefill_rows_kernel<128><<<(unsigned)blocks, 128, 0, s>>>(p);
  else prefill_rows_kernel<64><<<(unsigned)blocks, 128, 0, s>>>(p);
  return cudaPeekAtLastError() == cudaSuccess;
}

}  // namespace gdn
