// Causal attention over packed prompts: o_i = sum_{j <= i} softmax_j(scale q_i . k_j) v_j.
// The kernel and its design are in attn_tc.cuh.
#include "attn_tc.cuh"

namespace gdn {

namespace {

template <int D>
bool launch(const AttnParams& p, cudaStream_t s) {
  CUtensorMap tm_q, tm_k, tm_v;
  const int nt = kRows / p.G;
  const uint32_t box_q[3] = {64, (uint32_t)p.G, (uint32_t)nt}, box_kv[3] = {64, 1, kKeys};
  const uint64_t dim_q[3] = {D, (uint64_t)p.H, (uint64_t)p.T};
  const uint64_t dim_kv[3] = {D, (uint64_t)p.Hk, (uint64_t)p.T};
  const uint64_t str_q[2] = {D * 2, (uint64_t)p.H * D * 2}, str_kv[2] = {D * 2, (uint64_t)p.Hk * D * 2};
  if (!encode_bf16_tmap(&tm_q, p.q, 3, dim_q, str_q, box_q) ||
      !encode_bf16_tmap(&tm_k, p.k, 3, dim_kv, str_kv, box_kv) ||
      !encode_bf16_tmap(&tm_v, p.v, 3, dim_kv, str_kv, box_kv))
    return false;
  const auto kernel = attn_prompt_kernel<D>;
  constexpr int smem = AttnSmem<D>::kBytes;
  ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem);
  for (int n0 = 0; n0 < p.N; n0 += kAttnSeqs) {
    AttnParams a = p;
    a.N = min(kAttnSeqs, p.N - n0);
    a.cu = p.cu ? p.cu + n0 : nullptr;
    // at most this many pairs of row tiles, whatever the lengths
    const int64_t items = (((int64_t)p.T + 2 * nt - 1) / (2 * nt) + a.N - 1) * p.Hk;
    const int grid = (int)min((int64_t)num_sms(), items);
    kernel<<<grid, kAttnThreads, smem, s>>>(a, tm_q, tm_k, tm_v);
  }
  return cudaPeekAtLastError() == cudaSuccess;
}

}  // namespace

bool launch_attn_prefill(const AttnParams& p, cudaStream_t s) {
  return p.D == 128 ? launch<128>(p, s) : launch<64>(p, s);
}

}  // namespace gdn
