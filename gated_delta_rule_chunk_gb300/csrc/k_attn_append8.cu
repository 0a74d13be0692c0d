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
// side by side, their maximum is a few shuffles away, and the rounded rows are stored from the
// registers; a block that holds earlier tokens reads its scale meanwhile, and those tokens' rows
// only where the scale grows. A warp finds its block from the rows of the call: the first row of
// each block stands for it.
#include "attn_common.cuh"
#include "e4m3.cuh"

namespace gdn {

namespace {

constexpr int kWarps = 4;
constexpr uint32_t kLargest = 0x7F7FFFFFu;  // bits of the largest finite number

template <int D, bool kBf16>
__global__ void __launch_bounds__(kWarps * 32) append8_kernel(const AttnAppend8Params p) {
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

  // The rows of this group that are the first of a block, one lane a row.
  const int t = (int)(group * p.span) + lane;
  int n = -1, b = 0, e = 0;
  int64_t pos = 0;
  if (lane < p.span && t < p.T) n = find_seq(p.cu, p.N, p.T, t, b, e);
  if (n >= 0) pos = p.kv_lens ? (int64_t)p.kv_lens[n] - (e - t) : t - b;
  uint32_t firsts = __ballot_sync(0xffffffffu, n >= 0 && (t == b || (pos & (kBlock8 - 1)) == 0));

  const void* x = is_v ? p.v : p.k;
  uint8_t* cache = is_v ? p.vc : p.kc;
  float* scales = is_v ? p.vs : p.ks;
  const int r0 = lane / L, col = (lane % L) * 8;
  while (firsts) {
    const int src = __ffs(firsts) - 1;
    firsts &= firsts - 1;
    const int t0 = __shfl_sync(0xffffffffu, t, src), n0 = __shfl_sync(0xffffffffu, n, src);
    const int b0 = __shfl_sync(0xffffffffu, b, src), e0 = __shfl_sync(0xffffffffu, e, src);
    const int64_t at = __shfl_sync(0xffffffffu, pos, src);
    if (at < 0 || (at >> p.page_shift) >= p.max_pages) {
      if (lane == 0) set_status(p.status, GDN_DEV_BAD_LENGTH);
      continue;
    }
    const int in_block = (int)(at & (kBlock8 - 1));
    const int rows = min(kBlock8 - in_block, e0 - t0);
    const int held = t0 == b0 ? in_block : 0;
    const int page = p.table[(size_t)n0 * p.max_pages + (at >> p.page_shift)];

    float y[kPasses][8];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = i * kAtOnce + r0;
#pragma unroll
      for (int j = 0; j < 8; ++j) y[i][j] = 0.f;
      if (r >= rows) continue;
      const size_t from = ((size_t)(t0 + r) * p.Hk + hk) * D + col;
      if constexpr (kBf16) {
        const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(x) + from);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[i][2 * j] = __uint_as_float(u[j] << 16);
          y[i][2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
        }
      } else {
        const float4* w = reinterpret_cast<const float4*>(static_cast<const float*>(x) + from);
        *reinterpret_cast<float4*>(y[i]) = w[0];
        *reinterpret_cast<float4*>(y[i] + 4) = w[1];
      }
    }
    if (page < 0 || page >= p.n_pages) {
      if (lane == 0) set_status(p.status, GDN_DEV_BAD_PAGE_TABLE);
      continue;
    }
    const size_t row = ((((size_t)page * p.Hk + hk) << p.page_shift) + (at & (p.page - 1)));
    const size_t block = row / kBlock8;
    float old = 0.f;
    if (held) old = scales[block];
    uint32_t top = 0;  // the largest finite |x|; its bits are in the order of the values
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t a = __float_as_uint(y[i][j]) & 0x7FFFFFFFu;
        top = max(top, a <= kLargest ? a : 0u);
      }
    top = __reduce_max_sync(0xffffffffu, top);
    // 448 = 1.75 * 2^8
    const int ex = max((int)(top >> 23) - 127 - 8 + ((top & 0x7FFFFFu) > 0x600000u), -100);
    const float need = __uint_as_float((uint32_t)(ex + 127) << 23);
    const float s = fmaxf(need, old);
    const bool power = (__float_as_uint(s) & 0x7FFFFFu) == 0;
    const float inv = 1.0f / s;  // exact for a power of two
    uint8_t* dst = cache + row * D + col;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = i * kAtOnce + r0;
      if (r >= rows) continue;
      uint32_t z[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = y[i][2 * j], c = y[i][2 * j + 1];
        z[j] = power ? to_e4m3x2(a * inv, c * inv) : to_e4m3x2(a / s, c / s);
      }
      *reinterpret_cast<uint2*>(dst + (size_t)r * D) = make_uint2(z[0] | z[1] << 16, z[2] | z[3] << 16);
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
