// Eviction: the tokens of a sequence that stay (select_kernel), and their copies (move_kernel).
//
// The choice is per sequence and key head: the k = keep - recent largest weights among the first
// len - recent tokens, of equal ones those of lower index. A CTA holds the weights in registers, as
// integers of the same order, and finds the k-th largest bit by bit from the top: a bit is set where
// at least k values reach the number with it, from the first bit in which the values differ on. A
// round is a comparison a value and one barrier, and the rounds end early once exactly k values
// reach the number. A lane holds few consecutive tokens and the next lane the next ones, so that
// the places in the result, from scans over a warp's lanes, are close together where they are
// written at once: larger values stay, and of those equal to the k-th the first that are still
// wanted. Bound: latency, of the loads (page, then weights), the rounds and the writes, a few
// microseconds each (one sequence of 16383 in 8 bits, four heads, the whole call: 16 consecutive
// tokens a lane 17.4 us, 4 and the rounds' first bit from the ends 16.4). A histogram of 8 bits a
// pass took ten times as long as the rounds, as weights share their exponents and most of a
// warp's additions went to one counter.
// Rows longer than the registers of a CTA hold (kSelect * 32 tokens) are read again each round, 8
// bits a round (select_long_row).
//
// The copies are rows of 64 to 256 bytes from anywhere to consecutive places. A warp takes 16
// places of K or of V, all rows loaded side by side. Measured (GB300): 64 sequences of up to 4096
// tokens cut to 1024, bf16, 80 us (5.6 TB/s), of which the copies alone take 65; one of 16383 cut to 4001
// 16.2, in 8 bits 16.7.
#include "attn_common.cuh"
#include "e4m3.cuh"

namespace gdn {

namespace {

constexpr int kSelect = 1024;  // threads of a selection
constexpr int kList = 512;      // values that one warp goes on with
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

// What a selection does before it looks at weights: the lists of sequences that stay whole, the
// last tokens. Returns whether there is nothing left to do.
__device__ __forceinline__ bool easy_part(const AttnEvictParams& p, int n, int hk, int32_t* kept, int& M,
                                          int& k) {
  const int tid = threadIdx.x, step = blockDim.x, len = evict_len(p, n);
  if (tid == 0 && hk == 0 && p.kv_lens[n] != len) set_status(p.status, GDN_DEV_BAD_LENGTH);
  for (int i = min(len, p.keep) + tid; i < p.keep; i += step) kept[i] = -1;
  if (len <= p.keep) {
    for (int i = tid; i < len; i += step) kept[i] = i;
    return true;
  }
  M = len - p.recent;
  k = p.keep - p.recent;
  for (int i = tid; i < p.recent; i += step) kept[k + i] = M + i;
  return k == 0;
}

// The k largest of the first M weights of a row, which kT threads hold, E each.
template <int E, int kT>
__device__ __forceinline__ void select_row(const AttnEvictParams& p, int n, int hk, int32_t* kept, int M,
                                           int k, bool wide) {
  __shared__ uint32_t counts[2][32], ends[2][32], list[kList], listed, found[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) listed = 0;
  // (8 values: 8 consecutive ones, one lookup; 64 sequences of up to 4096 80.0 us, with 4 80.7.)
  // This thread's tokens: V from i0 + 32 V c on, for each c; 0 stands for what is past the end (no
  // weight's bits are 0). Pages are looked up side by side, then weights.
  constexpr int V = E == 8 ? 8 : 4, C = E / V;
  const int i0 = warp * E * 32 + lane * V;
  uint32_t u[E];
  int page[C];
  float4 x[E / 4];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = i0 + c * 32 * V;
    page[c] = -1;
    if (i < M) page[c] = p.table[(size_t)n * p.max_pages + (i >> p.page_shift)];
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const float* w = p.weights + ((((int64_t)page[c] * p.Hk + hk) << p.page_shift) +
                                  ((i0 + c * 32 * V) & (p.page - 1)));
    if (i0 + c * 32 * V < M && (page[c] < 0 || page[c] >= p.n_pages)) set_status(p.status, GDN_DEV_BAD_PAGE_TABLE);
#pragma unroll
    for (int e = 0; e < V / 4; ++e) {
      x[c * V / 4 + e] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (page[c] >= 0 && page[c] < p.n_pages) {
        if (wide) x[c * V / 4 + e] = reinterpret_cast<const float4*>(w)[e];
        else x[c * V / 4 + e] = make_float4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < E; e += 4) {
    const int i = i0 + e / V * 32 * V + e % V;
    u[e] = i < M ? order_bits(x[e / 4].x) : 0;
    u[e + 1] = i + 1 < M ? order_bits(x[e / 4].y) : 0;
    u[e + 2] = i + 2 < M ? order_bits(x[e / 4].z) : 0;
    u[e + 3] = i + 3 < M ? order_bits(x[e / 4].w) : 0;
  }
  // Sum of a value over the CTA.
  auto total = [&](uint32_t x, int buf) -> uint32_t {
    x = __reduce_add_sync(0xffffffffu, x);
    if (lane == 0) counts[buf][warp] = x;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, lane < kT / 32 ? counts[buf][lane] : 0);
  };
  // The k-th largest value lies in [top, top + 2^bit); `above` values lie above that, `reach` from
  // top on.
  uint32_t above = 0, reach = M, least = ~0u, most = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    most = max(most, u[e]);
    least = min(least, u[e] - 1);  // (past the end: the largest)
  }
  most = __reduce_max_sync(0xffffffffu, most);
  least = __reduce_min_sync(0xffffffffu, least);
  if (lane == 0) {
    ends[0][warp] = most;
    ends[1][warp] = least;
  }
  __syncthreads();
  most = __reduce_max_sync(0xffffffffu, lane < kT / 32 ? ends[0][lane] : 0);
  least = __reduce_min_sync(0xffffffffu, lane < kT / 32 ? ends[1][lane] : ~0u) + 1;
  // The bits above the first one in which the ends differ are known.
  int bit = 32 - __clz(most ^ least);
  uint32_t top = bit < 32 ? most >> bit << bit : 0;
  while (bit > 0 && reach != (uint32_t)k && reach - above > kList) {
    const uint32_t next = top + (1u << --bit);
    uint32_t c = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) c += u[e] >= next;
    c = total(c, bit & 1);
    if (c >= (uint32_t)k) {
      top = next;
      reach = c;
    } else {
      above = c;
    }
  }
  if (bit > 0 && reach != (uint32_t)k) {
    // Few are left: one warp goes on with them, without barriers.
    __syncthreads();
    const uint32_t last = top + ((bit < 32 ? 1u << bit : 0u) - 1);
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (u[e] >= top && u[e] <= last && u[e] != 0) list[atomicAdd(&listed, 1u)] = u[e];
    __syncthreads();
    if (warp == 0) {
      uint32_t x[kList / 32];
#pragma unroll
      for (int i = 0; i < kList / 32; ++i) x[i] = i * 32 + lane < (int)listed ? list[i * 32 + lane] : 0;
      while (bit > 0 && reach != (uint32_t)k) {
        const uint32_t next = top + (1u << --bit);
        uint32_t c = 0;
#pragma unroll
        for (int i = 0; i < kList / 32; ++i) c += x[i] >= next;
        c = above + __reduce_add_sync(0xffffffffu, c);
        if (c >= (uint32_t)k) {
          top = next;
          reach = c;
        }
      }
      if (lane == 0) {
        found[0] = top;
        found[1] = reach;
      }
    }
    __syncthreads();
    top = found[0];
    reach = found[1];
  }
  const bool exact = reach == (uint32_t)k;  // k values reach it
  // Where exactly k values reach it, all of them stay; else the larger ones and the first equal ones.
  // Places by scans over the lanes of a warp, of four c's at once: a byte each, 128 at most (one c: up
  // to 256, in all bits).
  constexpr int Q = (C + 3) / 4;
  constexpr uint32_t kField = C == 1 ? ~0u : 255;
  uint32_t more[Q] = {}, same[Q] = {}, m_inc[Q], s_inc[Q], m_all[Q], s_all[Q], m_sum = 0, s_sum = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const uint32_t one = 1u << (e / V % 4 * 8);
    more[e / V / 4] += (exact ? u[e] >= top : u[e] > top) ? one : 0;
    same[e / V / 4] += !exact && u[e] == top ? one : 0;
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    m_inc[q] = more[q];
    s_inc[q] = same[q];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t a = __shfl_up_sync(0xffffffffu, m_inc[q], o);
      const uint32_t b = __shfl_up_sync(0xffffffffu, s_inc[q], o);
      if (lane >= o) {
        m_inc[q] += a;
        s_inc[q] += b;
      }
    }
    m_all[q] = __shfl_sync(0xffffffffu, m_inc[q], 31);
    s_all[q] = __shfl_sync(0xffffffffu, s_inc[q], 31);
#pragma unroll
    for (int b = 0; b < (C == 1 ? 8 : 32); b += 8) {
      m_sum += m_all[q] >> b & kField;
      s_sum += s_all[q] >> b & kField;
    }
  }
  __syncthreads();
  if (lane == 0) {
    counts[0][warp] = m_sum;
    counts[1][warp] = s_sum;
  }
  __syncthreads();
  const uint32_t mw = lane < kT / 32 ? counts[0][lane] : 0, sw = lane < kT / 32 ? counts[1][lane] : 0;
  const uint32_t want = k - __reduce_add_sync(0xffffffffu, mw);  // of the equal ones
  uint32_t m_base = __reduce_add_sync(0xffffffffu, lane < warp ? mw : 0);
  uint32_t s_base = __reduce_add_sync(0xffffffffu, lane < warp ? sw : 0);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int q = c / 4, b = c % 4 * 8;
    uint32_t m_at = m_base + (m_inc[q] >> b & kField) - (more[q] >> b & kField);
    uint32_t s_at = s_base + (s_inc[q] >> b & kField) - (same[q] >> b & kField);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const uint32_t x = u[c * V + e];
      const bool is_more = exact ? x >= top : x > top, is_same = !exact && x == top;
      if (is_more || (is_same && s_at < want)) kept[m_at + min(s_at, want)] = i0 + c * 32 * V + e;
      m_at += is_more;
      s_at += is_same;
    }
    m_base += m_all[q] >> b & kField;
    s_base += s_all[q] >> b & kField;
  }
}

template <int E, int kT>
__global__ void __launch_bounds__(kT, E == 32 ? 1 : (E == 8 ? 1536 : 1024) / kT)
select_kernel(const AttnEvictParams p, bool wide) {
  const int n = blockIdx.x / p.Hk, hk = blockIdx.x - n * p.Hk;
  pdl_wait();
  pdl_release();
  int32_t* kept = p.kept + (size_t)blockIdx.x * p.keep;
  int M, k;
  if (!easy_part(p, n, hk, kept, M, k)) select_row<E, kT>(p, n, hk, kept, M, k, wide);
}

// The same for a row of any length, whose weights are read again each round.
__device__ __forceinline__ void select_long_row(const AttnEvictParams& p, int n, int hk, int32_t* kept, int M,
                                                int k) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t found[2];
  __shared__ uint32_t sums[2][kSelect / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto bits = [&](int i) -> uint32_t {
    const int page = p.table[(size_t)n * p.max_pages + (i >> p.page_shift)];
    if (page < 0 || page >= p.n_pages) {
      set_status(p.status, GDN_DEV_BAD_PAGE_TABLE);
      return order_bits(0.f);
    }
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

// For a table wider than registers hold: what a row takes goes by its own length, which the host does
// not know. (With a table of 131072 tokens: 64 sequences of up to 600 cut to 256 33.5 us, all of them by
// select_long_row 49.5; 64 of up to 4096 cut to 1024 91.2 and 125.6; one of 16383 16.8 and 63.6; two of
// 30000 28.7 and 104.8. Two of 50000 to 100000 take 270.)
__global__ void __launch_bounds__(kSelect) select_any_kernel(const AttnEvictParams p, bool wide) {
  const int n = blockIdx.x / p.Hk, hk = blockIdx.x - n * p.Hk;
  pdl_wait();
  pdl_release();
  int32_t* kept = p.kept + (size_t)blockIdx.x * p.keep;
  int M, k;
  if (easy_part(p, n, hk, kept, M, k)) return;
  if (M <= 8 * kSelect) select_row<8, kSelect>(p, n, hk, kept, M, k, wide);
  else if (M <= 16 * kSelect) select_row<16, kSelect>(p, n, hk, kept, M, k, wide);
  else if (M <= 32 * kSelect) select_row<32, kSelect>(p, n, hk, kept, M, k, wide);
  else select_long_row(p, n, hk, kept, M, k);
}

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
  // The smallest form that the table's rows fit: registers are read once, and more CTAs fit an SM. 16
  // values a thread where that makes a row 512 threads (32 sequences of 8000 cut to 256 in 8 bits 22.3
  // us, 8 values and 1024 threads 25.2), 8 below (64 sequences of up to 4096 cut to 1024 80.0 us, 16
  // values and 256 threads 80.8; two of 2000 cut to 256 10.2 us, 16 and 128 threads 10.5).
  const dim3 rows((unsigned)(p.N * p.Hk));
  const int64_t most = (int64_t)p.max_pages * p.page;
  const bool wide = ((uintptr_t)p.weights & 15) == 0;
  const cudaError_t e =
      most <= 2048    ? launch_pdl(select_kernel<8, 256>, rows, dim3(256), 0, s, p, wide)
      : most <= 4096  ? launch_pdl(select_kernel<8, 512>, rows, dim3(512), 0, s, p, wide)
      : most <= 8192  ? launch_pdl(select_kernel<16, 512>, rows, dim3(512), 0, s, p, wide)
      : most <= 16384 ? launch_pdl(select_kernel<16, 1024>, rows, dim3(1024), 0, s, p, wide)
      : most <= 32768 ? launch_pdl(select_kernel<32, 1024>, rows, dim3(1024), 0, s, p, wide)
                      : launch_pdl(select_any_kernel, rows, dim3(kSelect), 0, s, p, wide);
  if (e != cudaSuccess) return false;
  const int64_t items = (int64_t)p.N * p.Hk * ((p.keep + kBlock8 - 1) / kBlock8) * 2;
  const dim3 grid((unsigned)((items + kMoveWarps - 1) / kMoveWarps)), block(kMoveWarps * 32);
  const auto kernel = p.ks ? (p.D == 128 ? move_kernel<128, true> : move_kernel<64, true>)
                           : (p.D == 128 ? move_kernel<256, false> : move_kernel<128, false>);
  return launch_pdl(kernel, grid, block, 0, s, p) == cudaSuccess;
}

}  // namespace gdn
