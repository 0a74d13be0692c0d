// Shared definitions of the softmax-attention kernels (include/gdn_attn.h): launch
// parameters, the sequence lookup and the row-by-row attention that the tiled kernels
// are checked against.
#pragma once

#include "../../include/gdn_attn.h"
#include "gdn_common.cuh"

namespace gdn {

struct AttnFrontParams {
  int T, N, H, Hk, D, page, page_shift, n_pages, max_pages, rot, max_pos;
  const void* x;
  const float* qw;          // [D] or null
  const float* kw;          // [D] or null
  const float* rope;        // [max_pos, rot] or null
  const int32_t* cu;        // [N + 1] or null
  const int32_t* kv_lens;   // [N] or null
  const int32_t* table;     // [N, max_pages] or null
  void* q;
  void* k;                  // or null
  void* v;                  // or null
  void* kc;                 // or null
  void* vc;                 // or null
  int32_t* status;          // or null
  float eps;
  int in_bf16, out_bf16, interleaved;
};

struct AttnParams {
  int T, N, H, Hk, G, D;              // G = H / Hk
  int nq;                             // decode: tokens of each sequence
  int page, page_shift, n_pages, max_pages;
  int common;                         // decode: tokens whose pages are those of sequence 0
  int shared;                         // those of them that the prefix kernel takes (all or 0)
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;             // [T, Hk, D] or the cache
  const __nv_bfloat16* v;
  const int32_t* cu;                  // prefill: [N + 1] or null
  const int32_t* table;               // decode
  const int32_t* kv_lens;             // decode
  float scale;
  void* out;
  float* lse;                         // or null
  int32_t* status;                    // or null
  int out_bf16;
  int tiles;                          // prefill: row tiles of a work item, 1 or 2
};

// Testing hook (gdn_test_attn_prefix): a common prefix takes its own kernel at every size.
bool attn_prefix_always();
// Testing hook (gdn_test_attn_tiles): row tiles of a prompt's work items, 0: by the rule.
int attn_prefill_tiles();

bool launch_attn_front(const AttnFrontParams& p, cudaStream_t s);
bool launch_attn_prefill(const AttnParams& p, cudaStream_t s);
bool launch_attn_decode(const AttnParams& p, void* workspace, cudaStream_t s);
size_t attn_decode_workspace(int T, int N, int H, int Hk, int D);

// Decode: the keys of sequence n, and those that its new token i sees.
__device__ __forceinline__ int seq_len(const AttnParams& p, int n) {
  return min(max(p.kv_lens[n], 0), p.max_pages << p.page_shift);
}
__device__ __forceinline__ int keys_seen(const AttnParams& p, int n, int i) {
  return max(seq_len(p, n) - p.nq + i + 1, 0);
}

// Attention of one query row by one warp, in fp32 throughout: keys 32 at a time, one per
// lane for the scores, then the lanes own D / 32 output columns each. kp(j) and vp(j) give
// key j's rows, or null for a row of zeros. Nothing past n_keys is read.
template <int D, typename KP, typename VP>
__device__ void attn_row(const __nv_bfloat16* __restrict__ q, int n_keys, float scale, KP kp,
                         VP vp, float (&o)[D / 32], float& lse) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int j0 = 0; j0 < n_keys; j0 += 32) {
    const int j = j0 + lane;
    float s = -INFINITY;
    if (j < n_keys) {
      const __nv_bfloat16* kr = kp(j);
      float acc = 0.f;
      if (kr)
        for (int d = 0; d < D; ++d) acc += __bfloat162float(q[d]) * __bfloat162float(kr[d]);
      s = acc * scale;
    }
    float mt = s;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, x));
    const float mn = fmaxf(m, mt);
    const float ref = mn == -INFINITY ? 0.f : mn;  // no key with a weight yet
    const float c = expf(m - ref), w = expf(s - ref);
    m = mn;
    l = l * c + w;  // this lane's keys
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= c;
    const int cnt = min(32, n_keys - j0);
    for (int i = 0; i < cnt; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      const __nv_bfloat16* vr = vp(j0 + i);
      if (vr) {
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += wi * __bfloat162float(vr[lane * E + e]);
      }
    }
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  const float r = l == 0.f ? 0.f : 1.f / l;  // a row without keys: zeros
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] *= r;
  lse = l == 0.f ? -INFINITY : m + logf(l);
}

// One lane's D / 32 output columns of row `row` (a [rows, D] array).
template <int D>
__device__ __forceinline__ void store_row(void* out, bool bf16, size_t row,
                                          const float (&o)[D / 32]) {
  constexpr int E = D / 32;
  const size_t at = row * D + (threadIdx.x & 31) * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if (bf16) static_cast<__nv_bfloat16*>(out)[at + e] = __float2bfloat16_rn(o[e]);
    else static_cast<float*>(out)[at + e] = o[e];
  }
}

}  // namespace gdn
