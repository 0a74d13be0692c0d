// Host side of the attention part of the C ABI (include/gdn_attn.h): argument
// validation and launches. No allocation, no synchronization, no device reads.
#include <math.h>

#include <atomic>

#include "attn_common.cuh"

using namespace gdn;

namespace gdn {

static std::atomic<bool> g_prefix_always{false};
bool attn_prefix_always() { return g_prefix_always.load(std::memory_order_relaxed); }

static std::atomic<int> g_prefill_tiles{0};
int attn_prefill_tiles() { return g_prefill_tiles.load(std::memory_order_relaxed); }

static std::atomic<uint32_t> g_wait_polls{0}, g_wait_item{0};
void attn_test_timeout(AttnParams& p) {
  if (const uint32_t polls = g_wait_polls.load(std::memory_order_relaxed)) {
    p.polls = polls;
    p.stall = g_wait_item.load(std::memory_order_relaxed) + 1;
  }
}

}  // namespace gdn

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

int check_impl(const gdn_attn_desc* d) {
  if (!d) return GDN_ERR_NULL_ARG;
  if (d->T < 0 || d->N < 1 || d->H < 1 || d->Hk < 1 || d->H % d->Hk != 0) return GDN_ERR_BAD_SHAPE;
  if (d->page_size < 0 || d->n_pages < 0 || d->max_pages < 0 || d->rot_dim < 0 || d->max_pos < 0 ||
      d->rot_dim > d->D)
    return GDN_ERR_BAD_SHAPE;
  if (d->D != 64 && d->D != 128) return GDN_ERR_UNSUPPORTED;
  if (d->H / d->Hk > 64 || d->rot_dim % 16 != 0) return GDN_ERR_UNSUPPORTED;
  const int ps = d->page_size;
  if (ps != 0 && (ps < 16 || ps > 256 || (ps & (ps - 1)) != 0)) return GDN_ERR_UNSUPPORTED;
  const bool dt_ok = (d->in_dtype == GDN_F32 || d->in_dtype == GDN_BF16) &&
                     (d->out_dtype == GDN_F32 || d->out_dtype == GDN_BF16);
  if (!dt_ok || (d->flags & ~(uint32_t)GDN_ATTN_ROPE_INTERLEAVED)) return GDN_ERR_UNSUPPORTED;
  // Positions (with those of the tile that a sequence ends in) and row counts stay within 31
  // bits, grids within their limits (element offsets are 64-bit).
  if ((int64_t)d->T * (d->H + 2 * (int64_t)d->Hk) >= ((int64_t)1 << 31) ||
      (int64_t)d->max_pages * ps > ((int64_t)1 << 31) - 4096 ||
      (int64_t)d->n_pages * d->Hk * ps >= ((int64_t)1 << 34) || d->H > 65535 || d->N > 65535 * 16)
    return GDN_ERR_BAD_SHAPE;
  return GDN_OK;
}

int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

bool clear_status(int32_t* status, cudaStream_t s) {
  if (!aligned(status, 4)) return false;
  return !status || cudaMemsetAsync(status, 0, sizeof(int32_t), s) == cudaSuccess;
}

AttnParams attn_params(const gdn_attn_desc& d, const void* q, const void* k, const void* v,
                       float scale, void* out, float* lse) {
  AttnParams p{};
  p.T = d.T; p.N = d.N; p.H = d.H; p.Hk = d.Hk; p.G = d.H / d.Hk; p.D = d.D;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.scale = scale > 0.f ? scale : 1.0f / sqrtf((float)d.D);  // also NaN
  p.out = out; p.lse = lse; p.status = d.status;
  p.out_bf16 = d.out_dtype == GDN_BF16;
  p.polls = kAttnPolls;
  attn_test_timeout(p);
  return p;
}

}  // namespace

extern "C" {

void gdn_test_attn_prefix(int32_t always) {
  g_prefix_always.store(always != 0, std::memory_order_relaxed);
}

void gdn_test_attn_tiles(int32_t tiles) {
  g_prefill_tiles.store(tiles == 1 || tiles == 2 ? tiles : 0, std::memory_order_relaxed);
}

void gdn_test_attn_timeout(uint32_t polls, uint32_t item) {
  g_wait_item.store(item, std::memory_order_relaxed);
  g_wait_polls.store(polls, std::memory_order_relaxed);
}

int gdn_attn_check_desc(const gdn_attn_desc* desc) { return check_impl(desc); }

size_t gdn_attn_workspace_size(const gdn_attn_desc* desc) {
  if (check_impl(desc) != GDN_OK || desc->T % desc->N != 0) return 0;
  return attn_decode_workspace(desc->T, desc->N, desc->H, desc->Hk, desc->D);
}

int gdn_attn_front(const gdn_attn_desc* desc, const void* x, const float* q_weight,
                   const float* k_weight, const float* rope, const int32_t* cu_seqlens,
                   const int32_t* kv_lens, const int32_t* page_table, void* q, void* k, void* v,
                   void* k_cache, void* v_cache, cudaStream_t stream) {
  const int rc = check_impl(desc);
  if (rc != GDN_OK) return rc;
  const gdn_attn_desc& d = *desc;
  if (d.T == 0) return clear_status(d.status, stream) ? GDN_OK : GDN_ERR_LAUNCH_FAILED;
  if (!x || !q || (!k) != (!v) || (d.rot_dim > 0 && !rope)) return GDN_ERR_NULL_ARG;
  const bool cache = k_cache || v_cache || page_table;
  if (cache && (!k_cache || !v_cache || !page_table)) return GDN_ERR_NULL_ARG;
  if (cache && d.page_size == 0) return GDN_ERR_BAD_SHAPE;
  if (d.rot_dim > 0 && d.max_pos < 1) return GDN_ERR_BAD_SHAPE;
  if (!cu_seqlens && d.N != 1) return GDN_ERR_BAD_SHAPE;
  const void* ptrs16[] = {x, q_weight, k_weight, rope, q, k, v, k_cache, v_cache};
  for (const void* p : ptrs16)
    if (!aligned(p, 16)) return GDN_ERR_MISALIGNED;
  const void* ptrs4[] = {cu_seqlens, kv_lens, page_table, d.status};
  for (const void* p : ptrs4)
    if (!aligned(p, 4)) return GDN_ERR_MISALIGNED;
  AttnFrontParams p{};
  p.T = d.T; p.N = d.N; p.H = d.H; p.Hk = d.Hk; p.D = d.D;
  p.page = d.page_size; p.page_shift = log2_of(d.page_size);
  p.n_pages = d.n_pages; p.max_pages = d.max_pages; p.rot = d.rot_dim; p.max_pos = d.max_pos;
  p.x = x; p.qw = q_weight; p.kw = k_weight; p.rope = rope; p.cu = cu_seqlens;
  p.kv_lens = kv_lens; p.table = page_table;
  p.q = q; p.k = k; p.v = v; p.kc = k_cache; p.vc = v_cache; p.status = d.status;
  p.eps = d.norm_eps > 0.f ? d.norm_eps : 1e-6f;
  p.in_bf16 = d.in_dtype == GDN_BF16;
  p.out_bf16 = d.out_dtype == GDN_BF16;
  p.interleaved = (d.flags & GDN_ATTN_ROPE_INTERLEAVED) != 0;
  if (!clear_status(d.status, stream)) return GDN_ERR_LAUNCH_FAILED;
  if (!launch_attn_front(p, stream)) return GDN_ERR_LAUNCH_FAILED;
  return cudaPeekAtLastError() == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH_FAILED;
}

int gdn_attn_prefill(const gdn_attn_desc* desc, const void* q, const void* k, const void* v,
                     const int32_t* cu_seqlens, float scale, void* out, float* lse,
                     cudaStream_t stream) {
  const int rc = check_impl(desc);
  if (rc != GDN_OK) return rc;
  const gdn_attn_desc& d = *desc;
  if (d.in_dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  if (d.T == 0) return clear_status(d.status, stream) ? GDN_OK : GDN_ERR_LAUNCH_FAILED;
  if (!q || !k || !v || !out) return GDN_ERR_NULL_ARG;
  if (!cu_seqlens && d.N != 1) return GDN_ERR_BAD_SHAPE;
  const void* ptrs16[] = {q, k, v, out};
  for (const void* p : ptrs16)
    if (!aligned(p, 16)) return GDN_ERR_MISALIGNED;
  if (!aligned(cu_seqlens, 4) || !aligned(lse, 4) || !aligned(d.status, 4))
    return GDN_ERR_MISALIGNED;
  AttnParams p = attn_params(d, q, k, v, scale, out, lse);
  p.cu = cu_seqlens;
  if (!clear_status(d.status, stream)) return GDN_ERR_LAUNCH_FAILED;
  if (!launch_attn_prefill(p, stream)) return GDN_ERR_LAUNCH_FAILED;
  return cudaPeekAtLastError() == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH_FAILED;
}

int gdn_attn_decode(const gdn_attn_desc* desc, const void* q, const void* k_cache,
                    const void* v_cache, const int32_t* page_table, const int32_t* kv_lens,
                    int32_t shared_len, float scale, void* out, float* lse, cudaStream_t stream) {
  const int rc = check_impl(desc);
  if (rc != GDN_OK) return rc;
  const gdn_attn_desc& d = *desc;
  if (d.in_dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  if (d.T == 0) return clear_status(d.status, stream) ? GDN_OK : GDN_ERR_LAUNCH_FAILED;
  if (!q || !k_cache || !v_cache || !page_table || !kv_lens || !out || !d.workspace)
    return GDN_ERR_NULL_ARG;
  if (d.page_size == 0 || d.T % d.N != 0 || shared_len < 0 || shared_len % d.page_size != 0 ||
      shared_len > d.max_pages * d.page_size)
    return GDN_ERR_BAD_SHAPE;
  if ((int64_t)(d.T / d.N) * (d.H / d.Hk) > 64) return GDN_ERR_UNSUPPORTED;
  // 64-key units of all pairs are counted in 31 bits
  if ((int64_t)d.N * d.Hk * ((int64_t)d.max_pages * d.page_size / 64 + 4) >= ((int64_t)1 << 31))
    return GDN_ERR_BAD_SHAPE;
  const void* ptrs16[] = {q, k_cache, v_cache, out};
  for (const void* p : ptrs16)
    if (!aligned(p, 16)) return GDN_ERR_MISALIGNED;
  if (!aligned(page_table, 4) || !aligned(kv_lens, 4) || !aligned(lse, 4) ||
      !aligned(d.status, 4) || !aligned(d.workspace, 256))
    return GDN_ERR_MISALIGNED;
  if (d.workspace_bytes < gdn_attn_workspace_size(desc)) return GDN_ERR_WORKSPACE_TOO_SMALL;
  AttnParams p = attn_params(d, q, k_cache, v_cache, scale, out, lse);
  p.nq = d.T / d.N;
  p.page = d.page_size; p.page_shift = log2_of(d.page_size);
  p.n_pages = d.n_pages; p.max_pages = d.max_pages; p.common = shared_len;
  p.table = page_table; p.kv_lens = kv_lens;
  if (!clear_status(d.status, stream)) return GDN_ERR_LAUNCH_FAILED;
  if (!launch_attn_decode(p, d.workspace, stream)) return GDN_ERR_LAUNCH_FAILED;
  return cudaPeekAtLastError() == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH_FAILED;
}

}  // extern "C"
