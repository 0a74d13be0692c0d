// Shared definitions of the softmax-attention kernels (include/gdn_attn.h): launch
// parameters and the sequence lookup.
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
  uint32_t polls;                     // limit of an on-chip wait
  uint32_t stall;                     // testing hook: item + 1 that waits for what never happens, or 0
};

// Polls of an on-chip wait before it gives up.
constexpr uint32_t kAttnPolls = 1u << 22;
// Testing hook (gdn_test_attn_timeout): sets polls and stall where it is on.
void attn_test_timeout(AttnParams& p);
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
