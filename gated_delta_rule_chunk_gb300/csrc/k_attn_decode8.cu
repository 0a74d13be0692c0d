// Decode attention over a cache in 8 bits, and the weight that each key gets: one warp per row
// with a running maximum, then one warp per key.
#include "attn_common.cuh"
#include "e4m3.cuh"

namespace gdn {

namespace {

// Row of sequence n's key j in the cache, -1 where its page does not exist.
__device__ __forceinline__ int64_t cache_row(const AttnParams& p, int n, int hk, int j) {
  const int page = p.table[(size_t)(j < p.common ? 0 : n) * p.max_pages + (j >> p.page_shift)];
  if (page < 0 || page >= p.n_pages) {
    set_status(p.status, GDN_DEV_BAD_PAGE_TABLE);
    return -1;
  }
  return ((((int64_t)page * p.Hk + hk) << p.page_shift) + (j & (p.page - 1)));
}

template <int D, bool k8>
__device__ __forceinline__ void load_key(const __nv_bfloat16* x, const float* scale, int64_t row,
                                         float (&y)[D / 32]) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  for (int e = 0; e < E; ++e) y[e] = 0.f;
  if (row < 0) return;
  for (int e = 0; e < E; ++e) {
    if constexpr (k8)
      y[e] = e4m3x2_to_float2(reinterpret_cast<const uint8_t*>(x)[row * D + lane * E + e]).x *
             scale[row / kBlock8];
    else
      y[e] = __bfloat162float(x[row * D + lane * E + e]);
  }
}

template <int D, bool k8>
__global__ void __launch_bounds__(128) rows_kernel(const AttnParams p, float* lse) {
  constexpr int E = D / 32;
  const uint32_t at = blockIdx.x * 4 + (threadIdx.x >> 5);  // (n, i, h)
  const int lane = threadIdx.x & 31;
  pdl_wait();
  if (at >= (uint32_t)(p.T * p.H)) return;
  const int t = at / p.H, h = at - t * p.H, n = t / p.nq, hk = h / p.G;
  if (lane == 0 && (p.kv_lens[n] < 0 || p.kv_lens[n] > (p.max_pages << p.page_shift)))
    set_status(p.status, GDN_DEV_BAD_LENGTH);
  const int keys = keys_seen(p, n, t - n * p.nq);
  float q[E], o[E] = {}, m = -INFINITY, l = 0.f, x[E];
  for (int e = 0; e < E; ++e) q[e] = __bfloat162float(p.q[(size_t)at * D + lane * E + e]);
  for (int j = 0; j < keys; ++j) {
    const int64_t row = cache_row(p, n, hk, j);
    load_key<D, k8>(p.k, p.ks, row, x);
    float s = 0.f;
    for (int e = 0; e < E; ++e) s += q[e] * x[e];
    for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
    s *= p.scale;
    const float mn = fmaxf(m, s), f = m == mn ? 1.f : expf(m - mn), w = expf(s - mn);
    load_key<D, k8>(p.v, p.vs, row, x);
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + w * x[e];
    l = l * f + w;
    m = mn;
  }
  for (int e = 0; e < E; ++e) o[e] = l == 0.f ? 0.f : o[e] / l;
  store_row<D>(p.out, p.out_bf16, at, o);
  if (lane == 0) {
    const float y = l == 0.f ? -INFINITY : m + logf(l);
    if (p.lse) p.lse[at] = y;
    lse[at] = y;
  }
}

template <int D, bool k8>
__global__ void __launch_bounds__(128) weights_kernel(const AttnParams p, const float* lse) {
  constexpr int E = D / 32;
  const int n = blockIdx.y / p.Hk, hk = blockIdx.y - n * p.Hk, lane = threadIdx.x & 31;
  pdl_wait();
  const int len = seq_len(p, n);
  for (int j = blockIdx.x * 4 + (threadIdx.x >> 5); j < len; j += gridDim.x * 4) {
    const int64_t row = cache_row(p, n, hk, j);
    if (row < 0) continue;
    float x[E], sum = 0.f;
    load_key<D, k8>(p.k, p.ks, row, x);
    for (int i = max(0, j - (len - p.nq)); i < p.nq; ++i)
      for (int g = 0; g < p.G; ++g) {
        const size_t at = (size_t)(n * p.nq + i) * p.H + hk * p.G + g;
        float s = 0.f;
        for (int e = 0; e < E; ++e) s += __bfloat162float(p.q[at * D + lane * E + e]) * x[e];
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        sum += expf(s * p.scale - lse[at]);
      }
    if (lane == 0) {
      if (j >= len - p.nq) p.weights[row] = sum;
      else atomicAdd(p.weights + row, sum);
    }
  }
}

template <int D, bool k8>
bool launch(const AttnParams& p, float* lse, cudaStream_t s) {
  const size_t rows = (size_t)p.T * p.H;
  if (launch_pdl(rows_kernel<D, k8>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, s, p, lse) !=
      cudaSuccess)
    return false;
  if (!p.weights) return true;
  return launch_pdl(weights_kernel<D, k8>, dim3(64, (unsigned)(p.N * p.Hk)), dim3(128), 0, s, p,
                    lse) == cudaSuccess;
}

}  // namespace

size_t attn_decode_cache_workspace(int T, int N, int H, int Hk, int D, int64_t max_keys, bool weights) {
  return align_up(sizeof(float) * (size_t)T * H + 1, 256);
}

bool launch_attn_decode_cache(const AttnParams& p, void* workspace, cudaStream_t s) {
  float* lse = static_cast<float*>(workspace);
  if (p.ks) return p.D == 128 ? launch<128, true>(p, lse, s) : launch<64, true>(p, lse, s);
  return p.D == 128 ? launch<128, false>(p, lse, s) : launch<64, false>(p, lse, s);
}

}  // namespace gdn
