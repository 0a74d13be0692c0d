// Front end of a softmax-attention layer: projection output -> q, k, v, with k and v
// appended to the paged cache in the same pass.
//
// Per (token, head) of q and k: y = x / sqrt(mean x^2 + eps) * w, then each rotated pair
// (a, b) becomes (a cos - b sin, b cos + a sin) with the table's row of the token's
// position; fp32 throughout and one rounding at the store (a rounding between norm and
// rotation would double the error of a bf16 result). v is copied.
//
// D / 8 lanes hold one head row, each two runs of 4 elements, so that the norm's sum is a few
// shuffles and both halves of every rotated pair are in one lane: in the half layout the runs
// of a rotated lane l are [4l, 4l + 4) and [rot/2 + 4l, ..), elsewhere the lane's 8 elements
// (rot % 16 == 0). In both layouts the lane then needs the frequencies [4l, 4l + 4). A lane
// group takes R heads of one token, all loaded before anything waits, with one lookup of the
// token's sequence, position and page and one load of its cos/sin. Bound: HBM for long
// prompts; latency (cu_seqlens -> kv_lens -> page table and rotary row -> store, x loaded
// meanwhile) for a decode step. Measured (GB300): 8 prompts to 2048 in 32 bits 27.3 us (6.2 TB/s),
// 4096 tokens in bf16 with dense and cached k and v 12.1 us (3.9 TB/s: 8-byte accesses and their
// latency at 16 warps an SM), one token 2.3 us.
#include "attn_common.cuh"

namespace gdn {

namespace {

constexpr int kThreads = 128;

template <bool kBf16>
__device__ __forceinline__ void load4(const void* x, size_t at, float* y) {
  if constexpr (kBf16) {
    const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(x) + at);
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&r.y));
    y[0] = a.x; y[1] = a.y; y[2] = b.x; y[3] = b.y;
  } else {
    const float4 r = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
    y[0] = r.x; y[1] = r.y; y[2] = r.z; y[3] = r.w;
  }
}

template <bool kBf16>
__device__ __forceinline__ void store4(void* x, size_t at, const float* y) {
  if constexpr (kBf16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(y[0], y[1]), b = __floats2bfloat162_rn(y[2], y[3]);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(x) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(x) + at) = make_float4(y[0], y[1], y[2], y[3]);
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

// 1 / sqrt(x): rsqrtf is good to 2 ulp, one Newton step brings it to rounding (not from 0, the
// result for infinity, which the step would make NaN).
__device__ __forceinline__ float inv_sqrt(float x) {
  const float r = rsqrtf(x);
  return r == 0.f ? 0.f : r * (1.5f - 0.5f * x * r * r);
}

template <int D, bool kInBf16, bool kOutBf16, int R, bool kInter>
__global__ void __launch_bounds__(kThreads) attn_front_kernel(const AttnFrontParams p) {
  constexpr int L = D / 8;  // lanes of a head row
  // A token's chunks of R heads: first the query heads', then those of the keys and values, so
  // that a lane group's heads take one path.
  const uint32_t heads = p.H + 2 * p.Hk, q_chunks = (p.H + R - 1) / R;
  const uint32_t chunks = q_chunks + (2 * p.Hk + R - 1) / R;
  const uint32_t item = blockIdx.x * (kThreads / L) + threadIdx.x / L;
  const int lane = threadIdx.x % L;
  const uint32_t ti = item / chunks, chunk = item - ti * chunks;
  bool live = ti < (uint32_t)p.T;
  const int t = live ? (int)ti : 0;
  const bool is_q = chunk < q_chunks;
  const uint32_t h0 = is_q ? chunk * R : p.H + (chunk - q_chunks) * R;
  const int cnt = live ? min(R, (int)((is_q ? p.H : heads) - h0)) : 0;
  // this lane's elements: [e0, e0 + 4) and [e1, e1 + 4)
  const int half = p.rot >> 1;
  const bool turned = lane * 8 < p.rot, split = !kInter && turned;
  const int e0 = split ? 4 * lane : 8 * lane, e1 = split ? half + 4 * lane : 8 * lane + 4;
  pdl_wait();

  float y[R][8];
  const size_t src = ((size_t)t * heads + h0) * D;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (r < cnt) {
      load4<kInBf16>(p.x, src + r * D + e0, y[r]);
      load4<kInBf16>(p.x, src + r * D + e1, y[r] + 4);
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

  // cos and sin of this lane's pairs
  float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
  if (live && turned) {
    if (pos < 0 || pos >= p.max_pos) set_status(p.status, GDN_DEV_BAD_LENGTH);
    const int64_t row = pos < 0 ? 0 : pos < p.max_pos ? pos : p.max_pos - 1;
    load4<false>(p.rope, (size_t)row * p.rot + 4 * lane, c);
    load4<false>(p.rope, (size_t)row * p.rot + half + 4 * lane, s);
  }
  const float* weight = is_q ? p.qw : p.kw;
  float w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 1.f;
  if (weight) {
    load4<false>(weight, e0, w);
    load4<false>(weight, e1, w + 4);
  }
  // Factors of the norms, for all heads before anything depends on one (their shuffles overlap;
  // all lanes, as the sums cross the lanes of a group).
  const uint32_t k_end = p.H + p.Hk;
  auto normed = [&](int r) { return weight && h0 + r < k_end; };
  auto squares = [&](const float (&z)[8]) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += z[i] * z[i];
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    return ss;
  };
  float f[R];
  bool big = false;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float ss = squares(y[r]);
    big |= normed(r) && ss == INFINITY;
    f[r] = normed(r) ? inv_sqrt(ss * (1.0f / D) + p.eps) : 1.f;
  }
  // A sum past the largest number (elements from about 2^60): again with the row times 2^-70,
  // which leaves y as it is. The squares then stay below 2^116; what they lose at the lower end,
  // and eps, are nothing beside a sum of at least 2^-12 (for an eps below 2^90).
  if (__any_sync(0xffffffffu, big)) {
    constexpr float kDown = 1.0f / (1ull << 35) / (1ull << 35);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool down = normed(r) && f[r] == 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) y[r][i] *= down ? kDown : 1.f;
      const float ss = squares(y[r]);
      if (down) f[r] = inv_sqrt(ss * (1.0f / D));
    }
  }
  auto norm_turn = [&](float (&z)[8], const float (&w)[8], float f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] *= f * w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float& a = kInter ? z[2 * i] : z[i];
      float& d = kInter ? z[2 * i + 1] : z[4 + i];
      const float a0 = a;
      // (elsewhere as it is: a sin of 0 would make NaN of an infinity)
      a = turned ? a0 * c[i] - d * s[i] : a0;
      d = turned ? d * c[i] + a0 * s[i] : d;
    }
  };
  auto put = [&](void* dst, size_t at, const float (&z)[8]) {
    store4<kOutBf16>(dst, at + e0, z);
    store4<kOutBf16>(dst, at + e1, z + 4);
  };
  if (__all_sync(0xffffffffu, is_q)) {
    const size_t dst = ((size_t)t * p.H + h0) * D;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      norm_turn(y[r], w, f[r]);
      if (live && r < cnt) put(p.q, dst + r * D, y[r]);
    }
    return;
  }
  // Keys and values (and, in a warp that holds both kinds, queries).
  size_t slot = 0;  // row of key head 0 in the cache; key head h is at slot + h * page
  bool append = false;
  if (live && !is_q && p.kc) {
    if (pos < 0 || (pos >> p.page_shift) >= p.max_pages) {
      set_status(p.status, GDN_DEV_BAD_LENGTH);
    } else {
      const int pg = p.table[(size_t)n * p.max_pages + (pos >> p.page_shift)];
      append = pg >= 0 && pg < p.n_pages;
      if (!append) set_status(p.status, GDN_DEV_BAD_PAGE_TABLE);
      slot = (((size_t)pg * p.Hk) << p.page_shift) + (pos & (p.page - 1));
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const uint32_t h = h0 + r;
    float z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = y[r][i];
    norm_turn(z, w, f[r]);
    if (!live || r >= cnt) continue;
    if (is_q) {
      put(p.q, ((size_t)t * p.H + h) * D, z);
      continue;
    }
    const bool is_v = h >= k_end;
    if (is_v) {
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = y[r][i];
    }
    const uint32_t hk = is_v ? h - k_end : h - p.H;
    void* dense = is_v ? p.v : p.k;
    if (dense) put(dense, ((size_t)t * p.Hk + hk) * D, z);
    if (append) put(is_v ? p.vc : p.kc, (slot + ((size_t)hk << p.page_shift)) * D, z);
  }
}

template <int D, bool kInBf16, bool kOutBf16, bool kInter>
bool launch(const AttnFrontParams& p, cudaStream_t s) {
  const int per_block = kThreads / (D / 8);
  const int64_t rows = (int64_t)p.T * (p.H + 2 * p.Hk);
  // Two heads per lane group where there is work for all SMs, so that the lookups serve both
  // (4096 tokens x 20 heads: 12.1 us; one head 15.8 us, four 13.3 us, eight 15.1 us); one head
  // where there is not, as in a decode step.
  const bool wide = rows >= 8 * 152 * 16;
  const int64_t items = wide ? (int64_t)p.T * ((p.H + 1) / 2 + p.Hk) : rows;
  const int64_t blocks = (items + per_block - 1) / per_block;
  const auto kernel = wide ? attn_front_kernel<D, kInBf16, kOutBf16, 2, kInter>
                           : attn_front_kernel<D, kInBf16, kOutBf16, 1, kInter>;
  return launch_pdl(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s, p) == cudaSuccess;
}

template <int D, bool kInter>
bool launch_t(const AttnFrontParams& p, cudaStream_t s) {
  if (p.in_bf16)
    return p.out_bf16 ? launch<D, true, true, kInter>(p, s) : launch<D, true, false, kInter>(p, s);
  return p.out_bf16 ? launch<D, false, true, kInter>(p, s) : launch<D, false, false, kInter>(p, s);
}

template <int D>
bool launch_d(const AttnFrontParams& p, cudaStream_t s) {
  return p.interleaved ? launch_t<D, true>(p, s) : launch_t<D, false>(p, s);
}

}  // namespace

bool launch_attn_front(const AttnFrontParams& p, cudaStream_t s) {
  if (p.T == 0) return true;
  return p.D == 128 ? launch_d<128>(p, s) : launch_d<64>(p, s);
}

}  // namespace gdn
