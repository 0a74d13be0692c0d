// Keys and values into a cache in 8 bits, a scale for each 16 tokens and key head.
//
// Per block of 16 tokens: s = the least power of two, 2^-100 or more, with max|x| <= 448 s;
// elements are held as x / s rounded once to e4m3. Multiplying by a power of two is exact, so the
// scale costs no rounding of its own, and an e4m3 number loses nothing by a scale up to twice as
// large as it might be (it is a floating number; only what lies below 2^-6 s does). That is also
// what lets a block take more tokens later: where a new token needs a larger scale, the elements
// that are there are multiplied by a power of two and rounded again, exact but for those that
// become subnormal.
//
// A warp takes one (block, key head, k or v): all of its rows (4 KB in bf16 at D = 128) are loaded
// side by side and kept as they are (32 registers a lane), their maximum is a few shuffles away,
// and the rounded rows are stored from the registers; a block that holds earlier tokens reads its
// scale meanwhile, and those tokens' rows only where the scale grows. The first row of each block
// stands for it: a warp looks through `span` consecutive rows of the call for such rows, 16 for
// prompts, where that is one or two blocks, and one for steps. Bound: the loads that depend on one
// another (cu_seqlens, kv_lens, then the rows and the page), so the search for a sequence looks at
// 32 entries at a time. Measured (GB300): 8 ragged prompts of up to 2048 tokens, 8 heads of 128 (46 MB),
// 8.6 us where they are in L2 from the call before (with the rows turned to 32 bits as loaded and half the
// warps an SM 26.9), 11.2 from HBM (4.1 TB/s); in 32 bits 13.5 (L2); 64 single tokens 2.8 us.
#include "attn_common.cuh"
#include "e4m3.cuh"

namespace gdn {

namespace {

constexpr int kWarps = 4;
constexpr uint32_t kLargest = 0x7F7FFFFFu;  // bits of the largest finite number

// Sequence n of row t and its rows [b, e), which are rows of the call; n = -1 outside every sequence
// and in one that passes the call's rows. By a whole warp.
__device__ __forceinline__ int warp_find_seq(const AttnAppend8Params& p, int t, int& b, int& e) {
  if (!p.cu) {
    b = 0;
    e = p.T;
    return 0;
  }
  const int lane = threadIdx.x & 31;
  // In a step the sequence is the row's number; looked at beside the first part of the search.
  const int guess = min(t, p.N - 1);
  const int gb = p.cu[guess], ge = p.cu[guess + 1];
  int lo = 0, count = p.N + 1;  // the last entry <= t is one of [lo, lo + count)
  while (true) {
    const int step = (count + 31) / 32, at = lo + min(lane * step, count - 1);
    const uint32_t below = __ballot_sync(0xffffffffu, lane * step < count && p.cu[at] <= t);
    if (gb >= 0 && gb <= t && t < ge && ge <= p.T) {
      b = gb;
      e = ge;
      return guess;
    }
    if (below == 0) return -1;
    const int j = 31 - __clz(below);
    lo += j * step;
    count = min(step, count - j * step);
    if (count == 1) break;
  }
  if (lo >= p.N) return -1;
  b = p.cu[lo];
  e = p.cu[lo + 1];
  return b <= t && t < e && b >= 0 && e <= p.T ? lo : -1;
}

// 8 elements of a row as they were loaded.
template <bool kBf16>
struct Run {
  uint32_t w[kBf16 ? 4 : 8];
  __device__ __forceinline__ void load(const void* x, size_t at) {
    const uint4* v = reinterpret_cast<const uint4*>(static_cast<const char*>(x) + at * (kBf16 ? 2 : 4));
    *reinterpret_cast<uint4*>(w) = __ldcs(v);
    if constexpr (!kBf16) *reinterpret_cast<uint4*>(w + 4) = __ldcs(v + 1);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (uint32_t& x : w) x = 0;
  }
  // bits of element i in 32 bits
  __device__ __forceinline__ uint32_t bits(int i) const {
    if constexpr (kBf16) return i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16;
    else return w[i];
  }
};

template <int D, bool kBf16>
__global__ void __launch_bounds__(kWarps * 32, kBf16 ? 7 : 5)
append8_kernel(const AttnAppend8Params p) {
  constexpr int L = D / 8, kAtOnce = 32 / L, kPasses = kBlock8 / kAtOnce;
  const uint32_t item = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const bool is_v = item & 1;
  const uint32_t group = (item >> 1) / p.Hk;
  const int hk = (item >> 1) - group * p.Hk;
  pdl_wait();
  if (p.status && p.cu && blockIdx.x == 0)
    for (int i = threadIdx.x; i <= p.N; i += kWarps * 32)
      if (p.cu[i] < (i ? p.cu[i - 1] : 0) || p.cu[i] > p.T)
        set_status(p.status, GDN_DEV_BAD_CU_SEQLENS);
  if ((uint64_t)group * p.span >= (uint64_t)p.T) return;

  const void* x = is_v ? p.v : p.k;
  uint8_t* cache = is_v ? p.vc : p.kc;
  float* scales = is_v ? p.vs : p.ks;
  const int r0 = lane / L, col = (lane % L) * 8;
  int t = (int)(group * p.span), b = 0, e = 0;
  const int t_end = min(t + p.span, p.T);
  // The group's rows are on their way while its sequence and place are looked up, a line a lane.
  constexpr int kLine = 128 / (kBf16 ? 2 : 4), kLines = D / kLine;  // of a row
  for (int i = lane; i < (t_end - t) * kLines; i += 32)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(x) +
        (((size_t)(t + i / kLines) * p.Hk + hk) * D + i % kLines * kLine) * (kBf16 ? 2 : 4)));
  int n = warp_find_seq(p, t, b, e);
  while (t < t_end) {
    if (n < 0 || t >= e) {
      if (n < 0) {  // (only with cu) before the first sequence, or behind the last
        if (t >= p.cu[p.N]) return;
        t = max(t + 1, min(p.cu[0], t_end));
      }
      if (t < t_end) n = warp_find_seq(p, t, b, e);
      continue;
    }
    const int64_t at = p.kv_lens ? (int64_t)p.kv_lens[n] - (e - t) : t - b;
    const int in_block = (int)(at & (kBlock8 - 1));
    const int rows = min(kBlock8 - in_block, e - t), t0 = t;
    t += rows;
    if (t0 != b && in_block != 0) continue;  // another warp's block
    if (at < 0 || (at >> p.page_shift) >= p.max_pages) {
      if (lane == 0) set_status(p.status, GDN_DEV_BAD_LENGTH);
      continue;
    }
    const int held = in_block;  // earlier tokens in the block
    const int page = p.table[(size_t)n * p.max_pages + (at >> p.page_shift)];
    Run<kBf16> y[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = i * kAtOnce + r0;
      if (r < rows) y[i].load(x, ((size_t)(t0 + r) * p.Hk + hk) * D + col);
      else y[i].zero();
    }
    if (page < 0 || page >= p.n_pages) {
      if (lane == 0) set_status(p.status, GDN_DEV_BAD_PAGE_TABLE);
      continue;
    }
    const size_t row = ((((size_t)page * p.Hk + hk) << p.page_shift) + (at & (p.page - 1)));
    const size_t block = row / kBlock8;
    float old = 0.f;
    if (held) old = scales[block];
    uint32_t top = 0;  // the largest |x|; its bits are in the order of the values
    if constexpr (kBf16) {
      uint32_t two = 0;  // of even and odd elements
#pragma unroll
      for (int i = 0; i < kPasses; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) two = __vmaxu2(two, y[i].w[j] & 0x7FFF7FFFu);
      top = max(two << 16, two & 0xFFFF0000u);
    } else {
#pragma unroll
      for (int i = 0; i < kPasses; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, y[i].w[j] & 0x7FFFFFFFu);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    // What is seldom (infinities, NaN, a scale that is no power of two) goes through the rows once
    // more, from memory, so that the code for it stays small.
    const bool finite = top <= kLargest;
    if (!finite) {
      top = 0;  // of the finite ones
#pragma unroll 1
      for (int r = r0; r < rows; r += kAtOnce) {
        Run<kBf16> z;
        z.load(x, ((size_t)(t0 + r) * p.Hk + hk) * D + col);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t a = z.bits(j) & 0x7FFFFFFFu;
          top = max(top, a <= kLargest ? a : 0u);
        }
      }
      top = __reduce_max_sync(0xffffffffu, top);
    }
    // 448 = 1.75 * 2^8
    const int ex = max((int)(top >> 23) - 127 - 8 + ((top & 0x7FFFFFu) > 0x600000u), -100);
    const float need = __uint_as_float((uint32_t)(ex + 127) << 23);
    const float s = fmaxf(need, old);
    const bool power = (__float_as_uint(s) & 0x7FFFFFu) == 0;
    const float inv = 1.0f / s;  // exact for a power of two
    uint8_t* dst = cache + row * D + col;
    if (finite && power) {
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int r = i * kAtOnce + r0;
        uint32_t z[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          z[j] = finite_to_e4m3x2(__uint_as_float(y[i].bits(2 * j)) * inv,
                                  __uint_as_float(y[i].bits(2 * j + 1)) * inv);
        if (r < rows)
          *reinterpret_cast<uint2*>(dst + (size_t)r * D) = make_uint2(z[0] | z[1] << 16, z[2] | z[3] << 16);
      }
    } else {
#pragma unroll 1
      for (int r = r0; r < rows; r += kAtOnce) {
        Run<kBf16> v;
        v.load(x, ((size_t)(t0 + r) * p.Hk + hk) * D + col);
        uint32_t z[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          z[j] = to_e4m3x2(__uint_as_float(v.bits(2 * j)) / s, __uint_as_float(v.bits(2 * j + 1)) / s);
        *reinterpret_cast<uint2*>(dst + (size_t)r * D) = make_uint2(z[0] | z[1] << 16, z[2] | z[3] << 16);
      }
    }
    if (s != old || !held) {
      if (lane == 0) scales[block] = s;
      // the tokens that were there, to the new scale
      const float ratio = old * inv;
      for (int r = r0; r < held; r += kAtOnce) {
        uint2* w = reinterpret_cast<uint2*>(dst - (size_t)(in_block - r) * D);
        const uint2 u = *w;
        uint32_t z[4] = {u.x & 0xFFFF, u.x >> 16, u.y & 0xFFFF, u.y >> 16};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = e4m3x2_to_float2(z[j]);
          z[j] = to_e4m3x2(f.x * ratio, f.y * ratio);
        }
        *w = make_uint2(z[0] | z[1] << 16, z[2] | z[3] << 16);
      }
    }
  }
}

template <int D>
bool launch(const AttnAppend8Params& p, cudaStream_t s) {
  const int64_t groups = ((int64_t)p.T + p.span - 1) / p.span;
  const int64_t blocks = (groups * p.Hk * 2 + kWarps - 1) / kWarps;
  if (blocks >= (int64_t)1 << 31) return false;
  const auto kernel = p.in_bf16 ? append8_kernel<D, true> : append8_kernel<D, false>;
  return launch_pdl(kernel, dim3((unsigned)blocks), dim3(kWarps * 32), 0, s, p) == cudaSuccess;
}

}  // namespace

bool launch_attn_append8(const AttnAppend8Params& params, cudaStream_t s) {
  AttnAppend8Params p = params;
  p.span = p.T <= 2 * (int64_t)p.N ? 1 : kBlock8;
  return p.D == 128 ? launch<128>(p, s) : launch<64>(p, s);
}

}  // namespace gdn
