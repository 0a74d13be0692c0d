// Causal attention over packed prompts: o_i = sum_{j <= i} softmax_j(scale q_i . k_j) v_j.
// The kernel and its design are in attn_tc.cuh.
#include "attn_tc.cuh"

namespace gdn {

namespace {

template <int D>
bool launch(const AttnParams& p, cudaStream_t s) {
  CUtensorMap tm_k, tm_v;
  const uint32_t box[3] = {64, 1, kKeys};
  const uint64_t dim[3] = {D, (uint64_t)p.Hk, (uint64_t)p.T}, str[2] = {D * 2, (uint64_t)p.Hk * D * 2};
  if (!encode_bf16_tmap(&tm_k, p.k, 3, dim, str, box) ||
      !encode_bf16_tmap(&tm_v, p.v, 3, dim, str, box))
    return false;
  const int span = 2 * (kRows / p.G);
  for (int n0 = 0; n0 < p.N; n0 += kAttnSeqs) {
    AttnParams a = p;
    a.N = p.N - n0 < kAttnSeqs ? p.N - n0 : kAttnSeqs;
    a.cu = p.cu ? p.cu + n0 : nullptr;
    // at most this many pairs of row tiles, whatever the lengths
    const int64_t items = (((int64_t)p.T + span - 1) / span + a.N - 1) * p.Hk;
    if (!launch_attn_tc<D, false>(a, PrefixParts{}, tm_k, tm_v, items, s)) return false;
  }
  return cudaPeekAtLastError() == cudaSuccess;
}

}  // namespace

bool launch_attn_prefill(const AttnParams& p, cudaStream_t s) {
  return p.D == 128 ? launch<128>(p, s) : launch<64>(p, s);
}

}  // namespace gdn
