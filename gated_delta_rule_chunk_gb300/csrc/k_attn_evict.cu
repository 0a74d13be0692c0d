// Eviction: the tokens of a sequence that stay (select_kernel), and their copies (move_kernel).
//
// The choice is per sequence and key head: the k = keep - recent largest weights among the first
// len - recent tokens, of equal ones those of lower index. A CTA finds the k-th largest weight by
// its bits, 8 at a time from the top (a histogram of the values that agree so far, then the bin in
// which the k-th lies), and goes through the tokens once more in their order: larger ones stay,
// and of the equal ones the first that are still wanted.
//
// The copies are rows of 64 to 256 bytes from anywhere to consecutive places. A warp takes 16
// places of K or of V, all rows loaded side by side.
#include "attn_common.cuh"
#include "e4m3.cuh"

namespace gdn {

namespace {

constexpr int kSelect = 512;
constexpr int kMoveWarps = 4;

// Bits whose unsigned order is that of the numbers; NaN above all, both zeros the same.
__device__ __forceinline__ uint32_t order_bits(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int evict_len(const AttnEvictParams& p, int n) {
  return min(max(p.kv_lens[n], 0), p.max_pages << p.page_shift);
}

__global__ void __launch_bounds__(kSelect) select_kernel(const AttnEvictParams p) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t found[2];
  __shared__ uint32_t sums[2][kSelect / 32];
  const int n = blockIdx.x / p.Hk, hk = blockIdx.x - n * p.Hk;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  const int len = evict_len(p, n);
  if (tid == 0 && hk == 0 && p.kv_lens[n] != len) set_status(p.status, GDN_DEV_BAD_LENGTH);
  int32_t* kept = p.kept + (size_t)blockIdx.x * p.keep;
  const int stay = min(len, p.keep);
  for (int i = stay + tid; i < p.keep; i += kSelect) kept[i] = -1;
  if (len <= p.keep) {
    for (int i = tid; i < len; i += kSelect) kept[i] = i;
    return;
  }
  const int M = len - p.recent, k = p.keep - p.recent;
  for (int i = tid; i < p.recent; i += kSelect) kept[k + i] = M + i;
  if (k == 0) return;
  auto bits = [&](int i) -> uint32_t {
    const int page = p.table[(size_t)n * p.max_pages + (i >> p.page_shift)];
    if (page < 0 || page >= p.n_pages) return order_bits(0.f);
    return order_bits(p.weights[(((size_t)page * p.Hk + hk) << p.page_shift) + (i & (p.page - 1))]);
  };
  uint32_t prefix = 0, want = k;  // want: of the values that agree with prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kSelect) hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < M; i += kSelect) {
      const uint32_t u = bits(i);
      if (shift == 24 || (u >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(&hist[(u >> shift) & 255], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t above = 0;
      int bin = 255;
      while (above + hist[bin] < want) above += hist[bin--];
      found[0] = bin;
      found[1] = above;
    }
    __syncthreads();
    prefix |= found[0] << shift;
    want -= found[1];
    __syncthreads();
  }
  uint32_t out = 0, equal = 0;  // so far
  for (int i0 = 0; i0 < M; i0 += kSelect) {
    const int i = i0 + tid;
    const uint32_t u = i < M ? bits(i) : 0;
    const bool more = i < M && u > prefix, same = i < M && u == prefix;
    const uint32_t ms = __ballot_sync(0xffffffffu, same), lower = (1u << lane) - 1;
    const uint32_t mm = __ballot_sync(0xffffffffu, more);
    if (lane == 0) {
      sums[0][warp] = __popc(ms);
      sums[1][warp] = __popc(mm);
    }
    __syncthreads();
    uint32_t s_before = 0, m_before = 0, s_all = 0, m_all = 0;
    for (int w = 0; w < kSelect / 32; ++w) {
      if (w < warp) {
        s_before += sums[0][w];
        m_before += sums[1][w];
      }
      s_all += sums[0][w];
      m_all += sums[1][w];
    }
    const uint32_t s_rank = equal + s_before + __popc(ms & lower);
    const uint32_t s_taken = min(s_rank, want);  // equal ones before this that stay
    if (more || (same && s_rank < want)) kept[out + m_before + __popc(mm & lower) + s_taken] = i;
    out += m_all;
    equal += s_all;
    __syncthreads();
  }
}

// `out` above counts the larger ones only; the equal ones that stay come in by s_taken.

template <int kRow, bool k8>
__global__ void __launch_bounds__(kMoveWarps * 32) move_kernel(const AttnEvictParams p) {
  constexpr int L = kRow / 16, kAtOnce = 32 / L, kPasses = kBlock8 / kAtOnce;
  const int lane = threadIdx.x & 31;
  const uint32_t item = blockIdx.x * kMoveWarps + (threadIdx.x >> 5);
  const uint32_t blocks = (p.keep + kBlock8 - 1) / kBlock8;
  const bool is_v = item & 1;
  const uint32_t head = (item >> 1) / blocks;  // (n, hk)
  const int j0 = ((item >> 1) - head * blocks) * kBlock8;
  pdl_wait();
  if (head >= (uint32_t)(p.N * p.Hk)) return;
  const int n = head / p.Hk, hk = head - n * p.Hk;
  if (hk == 0 && j0 == 0 && !is_v && lane == 0) {
    const int len = evict_len(p, n);
    p.new_lens[n] = min(len, p.keep);
  }
  // one lane a token
  int src = -1;
  if (lane < kBlock8 && j0 + lane < p.keep) src = p.kept[(size_t)head * p.keep + j0 + lane];
  const uint32_t there = __ballot_sync(0xffffffffu, src >= 0);
  if (there == 0) return;
  const int rows = __popc(there);  // the places that are taken come first
  int64_t from = -1;
  if (src >= 0) {
    const int page = p.table[(size_t)n * p.max_pages + (src >> p.page_shift)];
    if (page >= 0 && page < p.n_pages)
      from = ((((int64_t)page * p.Hk + hk) << p.page_shift) + (src & (p.page - 1)));
  }
  const int to_page = p.new_table[(size_t)n * p.new_max + (j0 >> p.page_shift)];
  const bool to_ok = to_page >= 0 && to_page < p.n_pages;
  if (lane == 0 && !to_ok) set_status(p.status, GDN_DEV_BAD_PAGE_TABLE);
  if (src >= 0 && from < 0) set_status(p.status, GDN_DEV_BAD_PAGE_TABLE);
  if (!to_ok) return;
  const int64_t to = (((int64_t)to_page * p.Hk + hk) << p.page_shift) + (j0 & (p.page - 1));
  char* cache = is_v ? p.vc : p.kc;
  const int r0 = lane / L, col = (lane % L) * 16;
  uint4 x[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = i * kAtOnce + r0;
    const int64_t at = __shfl_sync(0xffffffffu, from, r);
    x[i] = make_uint4(0, 0, 0, 0);
    if (r < rows && at >= 0) x[i] = *reinterpret_cast<const uint4*>(cache + at * kRow + col);
  }
  if (!is_v) {
    float w = 0.f;
    if (from >= 0) w = p.weights[from];
    if (src >= 0) p.weights[to + lane] = w;
  }
  if constexpr (k8) {
    float* scales = is_v ? p.vs : p.ks;
    float s = 0.f;
    if (from >= 0) s = scales[from / kBlock8];
    float most = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    if (lane == 0) scales[to / kBlock8] = most;
    const float ratio = s == most ? 1.f : s / most;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const float f = __shfl_sync(0xffffffffu, ratio, i * kAtOnce + r0);
      if (f == 1.f) continue;
      uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 a = e4m3x2_to_float2(u[j] & 0xFFFF), b = e4m3x2_to_float2(u[j] >> 16);
        u[j] = to_e4m3x2(a.x * f, a.y * f) | to_e4m3x2(b.x * f, b.y * f) << 16;
      }
      x[i] = make_uint4(u[0], u[1], u[2], u[3]);
    }
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = i * kAtOnce + r0;
    if (r < rows) *reinterpret_cast<uint4*>(cache + (to + r) * kRow + col) = x[i];
  }
}

}  // namespace

bool launch_attn_evict(const AttnEvictParams& p, cudaStream_t s) {
  if (launch_pdl(select_kernel, dim3((unsigned)(p.N * p.Hk)), dim3(kSelect), 0, s, p) != cudaSuccess)
    return false;
  const int64_t items = (int64_t)p.N * p.Hk * ((p.keep + kBlock8 - 1) / kBlock8) * 2;
  const dim3 grid((unsigned)((items + kMoveWarps - 1) / kMoveWarps)), block(kMoveWarps * 32);
  const auto kernel = p.ks ? (p.D == 128 ? move_kernel<128, true> : move_kernel<64, true>)
                           : (p.D == 128 ? move_kernel<256, false> : move_kernel<128, false>);
  return launch_pdl(kernel, grid, block, 0, s, p) == cudaSuccess;
}

}  // namespace gdn
