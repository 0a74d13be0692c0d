// Front end of a softmax-attention layer: projection output -> q, k, v, with k and v
// appended to the paged cache in the same pass.
//
// Per (token, head) of q and k: y = x / sqrt(mean x^2 + eps) * w, then each rotated pair
// (a, b) becomes (a cos - b sin, b cos + a sin) with the table's row of the token's
// position; fp32 throughout and one rounding at the store (a rounding between norm and
// rotation would double the error of a bf16 result). v is copied.
//
// D / 8 lanes hold one head row, 8 elements each (16-byte loads and stores), so the norm's
// sum is a few shuffles; a pair's other half is 8-element aligned (rot % 16 == 0), hence one
// shuffle away (half layout) or in the same lane (interleaved). A lane group takes R heads
// of one token, all loaded before anything waits, with one lookup of the token's sequence,
// position and page and one load of its cos/sin row. Bound: HBM for long prompts; latency
// (cu_seqlens -> kv_lens -> page table and rotary row -> store, x loaded meanwhile) for a
// decode step.
#include "attn_common.cuh"

namespace gdn {

namespace {

constexpr int kThreads = 128;

template <bool kBf16>
__device__ __forceinline__ void load8(const void* x, size_t at, float (&y)[8]) {
  if constexpr (kBf16) {
    const uint4 r = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(x) + at);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
      y[2 * i] = f.x;
      y[2 * i + 1] = f.y;
    }
  } else {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
    const float4 a = f[0], b = f[1];
    y[0] = a.x; y[1] = a.y; y[2] = a.z; y[3] = a.w;
    y[4] = b.x; y[5] = b.y; y[6] = b.z; y[7] = b.w;
  }
}

template <bool kBf16>
__device__ __forceinline__ void store8(void* x, size_t at, const float (&y)[8]) {
  if constexpr (kBf16) {
    uint4 r;
    uint32_t* w = &r.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(x) + at) = r;
  } else {
    float4* f = reinterpret_cast<float4*>(static_cast<float*>(x) + at);
    f[0] = make_float4(y[0], y[1], y[2], y[3]);
    f[1] = make_float4(y[4], y[5], y[6], y[7]);
  }
}

// Sequence n of token t and its [cu[n], cu[n + 1]); n = -1 outside every sequence. The guess
// n = t is right in a decode step (one token each), where it saves the search's loads.
__device__ __forceinline__ int find_seq(const int32_t* cu, int N, int T, int t, int& b, int& e) {
  if (!cu) {
    b = 0;
    e = T;
    return 0;
  }
  int n = min(t, N - 1);
  b = cu[n];
  e = cu[n + 1];
  if (b <= t && t < e) return n;
  int lo = 0, hi = N;  // the last entry <= t lies in [lo, hi]
  while (lo < hi) {
    const int m = (lo + hi + 1) >> 1;
    if (cu[m] <= t) lo = m;
    else hi = m - 1;
  }
  if (lo >= N) return -1;
  b = cu[lo];
  e = cu[lo + 1];
  return b <= t && t < e && b >= 0 && e <= T ? lo : -1;
}

template <int D, bool kInBf16, bool kOutBf16, int R>
__global__ void __launch_bounds__(kThreads) attn_front_kernel(AttnFrontParams p) {
  constexpr int L = D / 8;  // lanes of a head row
  const int heads = p.H + 2 * p.Hk, chunks = (heads + R - 1) / R;
  const int64_t item = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / L;
  const int lane = threadIdx.x % L;
  const int64_t t64 = item / chunks;
  const int h0 = (int)(item % chunks) * R;
  bool live = t64 < p.T;
  const int t = live ? (int)t64 : 0;

  float y[R][8];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (live && h0 + r < heads) {
      load8<kInBf16>(p.x, ((size_t)t * heads + h0 + r) * D + lane * 8, y[r]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[r][i] = 0.f;
    }
  }

  if (p.status && p.cu && blockIdx.x == 0)
    for (int i = threadIdx.x; i <= p.N; i += kThreads)
      if (p.cu[i] < (i ? p.cu[i - 1] : 0) || p.cu[i] > p.T)
        set_status(p.status, GDN_DEV_BAD_CU_SEQLENS);

  int b = 0, e = 0;
  const int n = find_seq(p.cu, p.N, p.T, t, b, e);
  live = live && n >= 0;
  int64_t pos = 0;
  if (live) pos = p.kv_lens ? (int64_t)p.kv_lens[n] - (e - t) : t - b;

  size_t slot = 0;  // row of key head 0 in the cache; key head h is at slot + h * page
  bool append = false;
  if (live && p.kc) {
    if (pos < 0 || (pos >> p.page_shift) >= p.max_pages) {
      set_status(p.status, GDN_DEV_BAD_LENGTH);
    } else {
      const int pg = p.table[(size_t)n * p.max_pages + (pos >> p.page_shift)];
      append = pg >= 0 && pg < p.n_pages;
      if (!append) set_status(p.status, GDN_DEV_BAD_PAGE_TABLE);
      slot = (((size_t)pg * p.Hk) << p.page_shift) + (pos & (p.page - 1));
    }
  }

  // cos and sin of this lane's elements: 8 of each (half layout) or 4 (interleaved)
  float c[8], s[8];
  const bool turns = live && lane * 8 < p.rot && h0 < p.H + p.Hk;
  const int half = p.rot >> 1, pair = half >> 3;  // lanes of one half
  if (turns) {
    if (pos < 0 || pos >= p.max_pos) {
      set_status(p.status, GDN_DEV_BAD_LENGTH);
      pos = pos < 0 ? 0 : p.max_pos - 1;
    }
    const float* row = p.rope + (size_t)pos * p.rot;
    if (p.interleaved) {
      const float4 a = *reinterpret_cast<const float4*>(row + lane * 4);
      const float4 d = *reinterpret_cast<const float4*>(row + half + lane * 4);
      c[0] = c[1] = a.x; c[2] = c[3] = a.y; c[4] = c[5] = a.z; c[6] = c[7] = a.w;
      s[0] = s[1] = d.x; s[2] = s[3] = d.y; s[4] = s[5] = d.z; s[6] = s[7] = d.w;
    } else {
      const int f = (lane < pair ? lane : lane - pair) * 8;
      load8<false>(row, f, c);
      load8<false>(row, half + f, s);
    }
  }

#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int h = h0 + r;
    const bool is_q = h < p.H, is_k = !is_q && h < p.H + p.Hk;
    const float* w = is_q ? p.qw : is_k ? p.kw : nullptr;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += y[r][i] * y[r][i];
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (w) {
      const float norm = 1.0f / sqrtf(ss * (1.0f / D) + p.eps);
      float wv[8];
      load8<false>(w, lane * 8, wv);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[r][i] *= norm * wv[i];
    }
    float z[8];  // the other halves of this lane's pairs
    const int src = lane < pair ? lane + pair : lane - pair;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float far = __shfl_sync(0xffffffffu, y[r][i], src & (L - 1), L);
      z[i] = p.interleaved ? y[r][i ^ 1] : far;
    }
    if (turns && (is_q || is_k)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool first = p.interleaved ? (i & 1) == 0 : lane < pair;
        z[i] = y[r][i] * c[i] + (first ? -z[i] : z[i]) * s[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) y[r][i] = z[i];
    }
    if (!live || h >= heads) continue;
    if (is_q) {
      store8<kOutBf16>(p.q, ((size_t)t * p.H + h) * D + lane * 8, y[r]);
    } else {
      const int hk = is_k ? h - p.H : h - p.H - p.Hk;
      void* dense = is_k ? p.k : p.v;
      if (dense) store8<kOutBf16>(dense, ((size_t)t * p.Hk + hk) * D + lane * 8, y[r]);
      if (append)
        store8<kOutBf16>(is_k ? p.kc : p.vc,
                         (slot + ((size_t)hk << p.page_shift)) * D + lane * 8, y[r]);
    }
  }
}

template <int D, bool kInBf16, bool kOutBf16>
bool launch(const AttnFrontParams& p, cudaStream_t s) {
  const int heads = p.H + 2 * p.Hk, per_block = kThreads / (D / 8);
  const int64_t rows = (int64_t)p.T * heads;
  // One head per lane group while that leaves SMs idle (a decode step: the fewer steps in a
  // row the better), four when there is work for all of them.
  const bool wide = rows >= 8 * 152 * 16;
  const int64_t items = wide ? (int64_t)p.T * ((heads + 3) / 4) : rows;
  const int64_t blocks = (items + per_block - 1) / per_block;
  if (wide) attn_front_kernel<D, kInBf16, kOutBf16, 4><<<(unsigned)blocks, kThreads, 0, s>>>(p);
  else attn_front_kernel<D, kInBf16, kOutBf16, 1><<<(unsigned)blocks, kThreads, 0, s>>>(p);
  return cudaPeekAtLastError() == cudaSuccess;
}

template <int D>
bool launch_d(const AttnFrontParams& p, cudaStream_t s) {
  if (p.in_bf16)
    return p.out_bf16 ? launch<D, true, true>(p, s) : launch<D, true, false>(p, s);
  return p.out_bf16 ? launch<D, false, true>(p, s) : launch<D, false, false>(p, s);
}

}  // namespace

bool launch_attn_front(const AttnFrontParams& p, cudaStream_t s) {
  if (p.T == 0) return true;
  return p.D == 128 ? launch_d<128>(p, s) : launch_d<64>(p, s);
}

}  // namespace gdn
