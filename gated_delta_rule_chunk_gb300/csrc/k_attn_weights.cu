// The weight that a prompt's rows give its keys: w_j = sum over the rows i >= j of the window and
// the query heads of the group of exp(scale q_i . k_j - lse_i). One warp per key and key head.
#include "attn_common.cuh"

namespace gdn {

namespace {

template <int D>
__global__ void __launch_bounds__(128) prefill_weights_kernel(const AttnWeightsParams p) {
  constexpr int E = D / 32;
  const uint32_t item = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, t = item / p.Hk, hk = item - t * p.Hk;
  pdl_wait();
  if (t >= p.T) return;
  // entries clamped to [0, T] and raised to the largest before them
  int n = 0, b = 0, e = p.T;
  if (p.cu) {
    e = min(max(p.cu[0], 0), p.T);
    for (n = 0; n < p.N; ++n) {
      b = e;
      e = max(b, min(p.cu[n + 1], p.T));
      if (item == 0 && lane == 0 && (p.cu[n] < (n ? p.cu[n - 1] : 0) || p.cu[n + 1] < p.cu[n] ||
                                     p.cu[n + 1] > p.T))
        set_status(p.status, GDN_DEV_BAD_CU_SEQLENS);
      if (item != 0 && b <= t && t < e) break;
    }
    if (item == 0)
      for (n = 0, e = min(max(p.cu[0], 0), p.T); n < p.N; ++n) {
        b = e;
        e = max(b, min(p.cu[n + 1], p.T));
        if (b <= t && t < e) break;
      }
    if (n == p.N) return;
  }
  const int j = t - b;
  if ((j >> p.page_shift) >= p.max_pages) {
    if (lane == 0) set_status(p.status, GDN_DEV_BAD_LENGTH);
    return;
  }
  const int page = p.table[(size_t)n * p.max_pages + (j >> p.page_shift)];
  if (page < 0 || page >= p.n_pages) {
    if (lane == 0) set_status(p.status, GDN_DEV_BAD_PAGE_TABLE);
    return;
  }
  float k[E], sum = 0.f;
  for (int x = 0; x < E; ++x)
    k[x] = __bfloat162float(p.k[((size_t)t * p.Hk + hk) * D + lane * E + x]);
  const int first = p.window ? max(t, e - p.window) : t;
  for (int i = first; i < e; ++i)
    for (int g = 0; g < p.G; ++g) {
      const size_t row = (size_t)i * p.H + hk * p.G + g;
      float s = 0.f;
      for (int x = 0; x < E; ++x) s += k[x] * __bfloat162float(p.q[row * D + lane * E + x]);
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      sum += expf(s * p.scale - p.lse[row]);
    }
  if (lane == 0)
    p.weights[(((size_t)page * p.Hk + hk) << p.page_shift) + (j & (p.page - 1))] = sum;
}

}  // namespace

size_t attn_prefill_weights_workspace(int T, int N, int H, int Hk, int D) { return 256; }

bool launch_attn_prefill_weights(const AttnWeightsParams& p, void* workspace, cudaStream_t s) {
  const auto kernel = p.D == 128 ? prefill_weights_kernel<128> : prefill_weights_kernel<64>;
  const int64_t blocks = ((int64_t)p.T * p.Hk + 3) / 4;
  return launch_pdl(kernel, dim3((unsigned)blocks), dim3(128), 0, s, p) == cudaSuccess;
}

}  // namespace gdn
