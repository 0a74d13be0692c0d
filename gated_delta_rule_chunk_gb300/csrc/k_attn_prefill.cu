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
  const int nt = kRows / p.G;
  for (int n0 = 0; n0 < p.N; n0 += kAttnSeqs) {
    AttnParams a = p;
    a.N = p.N - n0 < kAttnSeqs ? p.N - n0 : kAttnSeqs;
    a.cu = p.cu ? p.cu + n0 : nullptr;
    // at most this many work items, whatever the lengths
    auto items_of = [&](int span) { return (((int64_t)p.T + span - 1) / span + a.N - 1) * p.Hk; };
    // Row tiles of an item: two, whose steps overlap (2,600 cycles a step of both, one alone takes
    // about 2,000), but one where single tiles leave no SM more than one item, or two of long
    // prompts, as an SM's longest item is what counts there. Measured with one / two tiles an
    // item: 2 x 2010 tokens x 2 heads of 64 16.9 / 22.7 us, 75 tokens x 15 heads 7.4 / 8.8 (no
    // more than one item an SM); 960 x 20 heads 16.1 / 18.6, 9632 x 4 heads 76.8 / 83.1, but
    // 19 x 164 tokens x 8 heads 11.2 / 9.9 (two); 1785 x 5 x 8 heads 47.7 / 32.3 (four). The
    // lengths are on the device: half a tile a sequence stands for the ragged ends.
    const int64_t each = (int64_t)p.T >= 256 * (int64_t)p.N ? 2 : 1;
    const int64_t singles = (((int64_t)p.T + nt - 1) / nt + a.N / 2) * p.Hk;
    a.tiles = attn_prefill_tiles() ? attn_prefill_tiles() : singles <= each * num_sms() ? 1 : 2;
    const int64_t items = items_of(a.tiles * nt);
    if (!launch_attn_tc<D, false>(a, PrefixParts{}, tm_k, tm_v, items, s)) return false;
  }
  return cudaPeekAtLastError() == cudaSuccess;
}

}  // namespace

bool launch_attn_prefill(const AttnParams& p, cudaStream_t s) {
  return p.D == 128 ? launch<128>(p, s) : launch<64>(p, s);
}

}  // namespace gdn
