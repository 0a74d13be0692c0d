// Decode attention over the paged cache. One warp per (token, query head).
#include "attn_common.cuh"

namespace gdn {

namespace {

template <int D>
__global__ void __launch_bounds__(128) decode_rows_kernel(AttnParams p) {
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (w >= (int64_t)p.T * p.H) return;
  const int t = (int)(w / p.H), h = (int)(w % p.H), n = t / p.nq, i = t % p.nq, hk = h / p.G;
  const int len = p.kv_lens[n], cap = p.max_pages << p.page_shift;
  if (len < 0 || len > cap) set_status(p.status, GDN_DEV_BAD_LENGTH);
  const int n_keys = min(max(len, 0), cap) - p.nq + i + 1;
  auto row = [&](const __nv_bfloat16* base, int j) -> const __nv_bfloat16* {
    // the shared prefix's pages are those of the first sequence
    const int pg = p.table[(size_t)(j < p.shared ? 0 : n) * p.max_pages + (j >> p.page_shift)];
    if (pg < 0 || pg >= p.n_pages) {
      set_status(p.status, GDN_DEV_BAD_PAGE_TABLE);
      return nullptr;
    }
    return base + ((((size_t)pg * p.Hk + hk) << p.page_shift) + (j & (p.page - 1))) * D;
  };
  float o[D / 32], lse;
  attn_row<D>(p.q + (size_t)w * D, n_keys, p.scale, [&](int j) { return row(p.k, j); },
              [&](int j) { return row(p.v, j); }, o, lse);
  store_row<D>(p.out, p.out_bf16, (size_t)w, o);
  if (p.lse && (threadIdx.x & 31) == 0) p.lse[w] = lse;
}

}  // namespace

bool launch_attn_decode(const AttnParams& p, cudaStream_t s) {
  const int64_t blocks = ((int64_t)p.T * p.H + 3) / 4;
  if (p.D == 128) decode_rows_kernel<128><<<(unsigned)blocks, 128, 0, s>>>(p);
  else decode_rows_kernel<64><<<(unsigned)blocks, 128, 0, s>>>(p);
  return cudaPeekAtLastError() == cudaSuccess;
}

}  // namespace gdn
