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
void attn_test_timeout(uint32_t& polls, uint32_t& stall) {
  if (const uint32_t n = g_wait_polls.load(std::memory_order_relaxed)) {
    polls = n;
    stall = g_wait_item.load(std::memory_order_relaxed) + 1;
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
  attn_test_timeout(p.polls, p.stall);
  return p;
}

int front_impl(const gdn_attn_desc* desc, const void* x, const float* q_weight,
               const float* k_weight, const float* rope, const int32_t* cu_seqlens,
               const int32_t* kv_lens, const int32_t* positions, int32_t n_axes,
               const uint8_t* rope_axes, const int32_t* page_table, void* q, void* k, void* v,
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
  const void* ptrs4[] = {cu_seqlens, kv_lens, page_table, positions, rope_axes, d.status};
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
  p.positions = positions; p.n_axes = n_axes; p.axes = rope_axes;
  if (!clear_status(d.status, stream)) return GDN_ERR_LAUNCH_FAILED;
  if (!launch_attn_front(p, stream)) return GDN_ERR_LAUNCH_FAILED;
  return cudaPeekAtLastError() == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH_FAILED;
}

// Both decode calls; `cache`: the one whose cache may be in 8 bits and which takes weights.
int decode_impl(const gdn_attn_desc* desc, const void* q, const void* k_cache, const void* v_cache,
                const float* k_scale, const float* v_scale, const int32_t* page_table,
                const int32_t* kv_lens, int32_t shared_len, float scale, void* out, float* lse,
                float* weights, bool cache, cudaStream_t stream) {
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
  if ((!k_scale) != (!v_scale)) return GDN_ERR_NULL_ARG;
  if (weights && shared_len > 0) return GDN_ERR_UNSUPPORTED;
  // 64-key units of all pairs are counted in 31 bits
  if ((int64_t)d.N * d.Hk * ((int64_t)d.max_pages * d.page_size / 64 + 4) >= ((int64_t)1 << 31))
    return GDN_ERR_BAD_SHAPE;
  const void* ptrs16[] = {q, k_cache, v_cache, out};
  for (const void* p : ptrs16)
    if (!aligned(p, 16)) return GDN_ERR_MISALIGNED;
  const void* ptrs4[] = {page_table, kv_lens, lse, k_scale, v_scale, weights, d.status};
  for (const void* p : ptrs4)
    if (!aligned(p, 4)) return GDN_ERR_MISALIGNED;
  if (!aligned(d.workspace, 256)) return GDN_ERR_MISALIGNED;
  const size_t need = cache ? gdn_attn_decode_cache_workspace_size(desc, weights != nullptr)
                            : gdn_attn_workspace_size(desc);
  if (d.workspace_bytes < need) return GDN_ERR_WORKSPACE_TOO_SMALL;
  AttnParams p = attn_params(d, q, k_cache, v_cache, scale, out, lse);
  p.nq = d.T / d.N;
  p.page = d.page_size; p.page_shift = log2_of(d.page_size);
  p.n_pages = d.n_pages; p.max_pages = d.max_pages; p.common = shared_len;
  p.table = page_table; p.kv_lens = kv_lens;
  p.ks = k_scale; p.vs = v_scale; p.weights = weights;
  if (!clear_status(d.status, stream)) return GDN_ERR_LAUNCH_FAILED;
  if (!(k_scale ? launch_attn_decode8(p, d.workspace, stream)
                : launch_attn_decode(p, d.workspace, stream)))
    return GDN_ERR_LAUNCH_FAILED;
  return cudaPeekAtLastError() == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH_FAILED;
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
  return front_impl(desc, x, q_weight, k_weight, rope, cu_seqlens, kv_lens, nullptr, 0, nullptr,
                    page_table, q, k, v, k_cache, v_cache, stream);
}

int gdn_attn_front_axes(const gdn_attn_desc* desc, const void* x, const float* q_weight,
                        const float* k_weight, const float* rope, const int32_t* cu_seqlens,
                        const int32_t* kv_lens, const int32_t* positions, int32_t n_axes,
                        const uint8_t* rope_axes, const int32_t* page_table, void* q, void* k,
                        void* v, void* k_cache, void* v_cache, cudaStream_t stream) {
  const int rc = check_impl(desc);
  if (rc != GDN_OK) return rc;
  if (desc->rot_dim == 0 || n_axes < 1 || n_axes > 8) return GDN_ERR_BAD_SHAPE;
  if (desc->T > 0 && !positions) return GDN_ERR_NULL_ARG;
  return front_impl(desc, x, q_weight, k_weight, rope, cu_seqlens, kv_lens, positions, n_axes,
                    rope_axes, page_table, q, k, v, k_cache, v_cache, stream);
}

int gdn_attn_append8(const gdn_attn_desc* desc, const void* k, const void* v,
                     const int32_t* cu_seqlens, const int32_t* kv_lens, const int32_t* page_table,
                     void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                     cudaStream_t stream) {
  const int rc = check_impl(desc);
  if (rc != GDN_OK) return rc;
  const gdn_attn_desc& d = *desc;
  if (d.T == 0) return clear_status(d.status, stream) ? GDN_OK : GDN_ERR_LAUNCH_FAILED;
  if (!k || !v || !page_table || !k_cache || !v_cache || !k_scale || !v_scale)
    return GDN_ERR_NULL_ARG;
  if (d.page_size == 0 || (!cu_seqlens && d.N != 1)) return GDN_ERR_BAD_SHAPE;
  const void* ptrs16[] = {k, v, k_cache, v_cache};
  for (const void* p : ptrs16)
    if (!aligned(p, 16)) return GDN_ERR_MISALIGNED;
  const void* ptrs4[] = {cu_seqlens, kv_lens, page_table, k_scale, v_scale, d.status};
  for (const void* p : ptrs4)
    if (!aligned(p, 4)) return GDN_ERR_MISALIGNED;
  AttnAppend8Params p{};
  p.T = d.T; p.N = d.N; p.Hk = d.Hk; p.D = d.D;
  p.page = d.page_size; p.page_shift = log2_of(d.page_size);
  p.n_pages = d.n_pages; p.max_pages = d.max_pages;
  p.k = k; p.v = v; p.cu = cu_seqlens; p.kv_lens = kv_lens; p.table = page_table;
  p.kc = static_cast<uint8_t*>(k_cache); p.vc = static_cast<uint8_t*>(v_cache);
  p.ks = k_scale; p.vs = v_scale; p.status = d.status;
  p.in_bf16 = d.in_dtype == GDN_BF16;
  if (!clear_status(d.status, stream)) return GDN_ERR_LAUNCH_FAILED;
  if (!launch_attn_append8(p, stream)) return GDN_ERR_LAUNCH_FAILED;
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
  return decode_impl(desc, q, k_cache, v_cache, nullptr, nullptr, page_table, kv_lens, shared_len,
                     scale, out, lse, nullptr, false, stream);
}

int gdn_attn_decode_cache(const gdn_attn_desc* desc, const void* q, const void* k_cache,
                          const void* v_cache, const float* k_scale, const float* v_scale,
                          const int32_t* page_table, const int32_t* kv_lens, int32_t shared_len,
                          float scale, void* out, float* lse, float* weights, cudaStream_t stream) {
  return decode_impl(desc, q, k_cache, v_cache, k_scale, v_scale, page_table, kv_lens, shared_len,
                     scale, out, lse, weights, true, stream);
}

size_t gdn_attn_decode_cache_workspace_size(const gdn_attn_desc* desc, int32_t with_weights) {
  if (check_impl(desc) != GDN_OK || desc->T % desc->N != 0) return 0;
  return attn_decode_cache_workspace(desc->T, desc->N, desc->H, desc->Hk, desc->D,
                                     (int64_t)desc->max_pages * desc->page_size, with_weights != 0);
}

int gdn_attn_prefill_weights(const gdn_attn_desc* desc, const void* q, const void* k,
                             const float* lse, const int32_t* cu_seqlens,
                             const int32_t* page_table, int32_t window, float scale,
                             float* weights, cudaStream_t stream) {
  const int rc = check_impl(desc);
  if (rc != GDN_OK) return rc;
  const gdn_attn_desc& d = *desc;
  if (d.in_dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  if (d.T == 0) return clear_status(d.status, stream) ? GDN_OK : GDN_ERR_LAUNCH_FAILED;
  if (!q || !k || !lse || !page_table || !weights || !d.workspace) return GDN_ERR_NULL_ARG;
  if (d.page_size == 0 || (!cu_seqlens && d.N != 1) || window < 0) return GDN_ERR_BAD_SHAPE;
  if (scale > 0.f && scale < 0x1p-100f) return GDN_ERR_UNSUPPORTED;  // lse / scale is formed
  if (!aligned(q, 16) || !aligned(k, 16)) return GDN_ERR_MISALIGNED;
  const void* ptrs4[] = {lse, cu_seqlens, page_table, weights, d.status};
  for (const void* p : ptrs4)
    if (!aligned(p, 4)) return GDN_ERR_MISALIGNED;
  if (!aligned(d.workspace, 256)) return GDN_ERR_MISALIGNED;
  if (d.workspace_bytes < gdn_attn_prefill_weights_workspace_size(desc))
    return GDN_ERR_WORKSPACE_TOO_SMALL;
  AttnWeightsParams p{};
  p.T = d.T; p.N = d.N; p.H = d.H; p.Hk = d.Hk; p.G = d.H / d.Hk; p.D = d.D;
  p.page = d.page_size; p.page_shift = log2_of(d.page_size);
  p.n_pages = d.n_pages; p.max_pages = d.max_pages; p.window = window;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.lse = lse; p.cu = cu_seqlens; p.table = page_table;
  p.scale = scale > 0.f ? scale : 1.0f / sqrtf((float)d.D);  // also NaN
  p.weights = weights; p.status = d.status;
  p.polls = kAttnPolls;
  attn_test_timeout(p.polls, p.stall);
  if (!clear_status(d.status, stream)) return GDN_ERR_LAUNCH_FAILED;
  if (!launch_attn_prefill_weights(p, d.workspace, stream)) return GDN_ERR_LAUNCH_FAILED;
  return cudaPeekAtLastError() == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH_FAILED;
}

size_t gdn_attn_prefill_weights_workspace_size(const gdn_attn_desc* desc) {
  if (check_impl(desc) != GDN_OK) return 0;
  return attn_prefill_weights_workspace(desc->T, desc->N, desc->H, desc->Hk, desc->D);
}

int gdn_attn_evict(const gdn_attn_desc* desc, void* k_cache, void* v_cache, float* k_scale,
                   float* v_scale, float* weights, const int32_t* page_table,
                   const int32_t* kv_lens, const int32_t* new_table, int32_t new_max_pages,
                   int32_t keep, int32_t recent, int32_t* new_lens, int32_t* kept,
                   cudaStream_t stream) {
  const int rc = check_impl(desc);
  if (rc != GDN_OK) return rc;
  const gdn_attn_desc& d = *desc;
  if (!k_cache || !v_cache || (!k_scale) != (!v_scale) || !weights || !page_table || !kv_lens ||
      !new_table || !new_lens || !kept)
    return GDN_ERR_NULL_ARG;
  if (d.page_size == 0 || new_max_pages < 1 || keep < 1 || recent < 0 || recent > keep ||
      (int64_t)keep > (int64_t)new_max_pages * d.page_size ||
      (int64_t)d.N * d.Hk * ((int64_t)keep / kBlock8 + 1) >= ((int64_t)1 << 29))
    return GDN_ERR_BAD_SHAPE;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return GDN_ERR_MISALIGNED;
  const void* ptrs4[] = {k_scale, v_scale, weights, page_table, kv_lens,
                         new_table, new_lens, kept, d.status};
  for (const void* p : ptrs4)
    if (!aligned(p, 4)) return GDN_ERR_MISALIGNED;
  AttnEvictParams p{};
  p.N = d.N; p.Hk = d.Hk; p.D = d.D;
  p.page = d.page_size; p.page_shift = log2_of(d.page_size);
  p.n_pages = d.n_pages; p.max_pages = d.max_pages; p.new_max = new_max_pages;
  p.keep = keep; p.recent = recent;
  p.kc = static_cast<char*>(k_cache); p.vc = static_cast<char*>(v_cache);
  p.ks = k_scale; p.vs = v_scale; p.weights = weights;
  p.table = page_table; p.kv_lens = kv_lens; p.new_table = new_table;
  p.new_lens = new_lens; p.kept = kept; p.status = d.status;
  if (!clear_status(d.status, stream)) return GDN_ERR_LAUNCH_FAILED;
  if (!launch_attn_evict(p, stream)) return GDN_ERR_LAUNCH_FAILED;
  return cudaPeekAtLastError() == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH_FAILED;
}

}  // extern "C"
