/*
 * gdn_attn.h -- C ABI of libgdn, second part: the softmax-attention layers that
 * stand between gated-delta-rule layers in a hybrid stack (front end, causal
 * attention over packed prompts, decode attention over a paged cache).
 *
 * The operations (query head h reads key head h / (H / Hk)):
 *
 *   front     q, k <- rotate(norm(x_q), pos), rotate(norm(x_k), pos); v <- x_v
 *             norm(y) = y / sqrt(mean(y^2) + eps) * weight, per head
 *   prefill   o_i = sum_{j <= i} w_ij v_j,  w_i = softmax_j(scale * q_i . k_j)
 *   decode    the same for the last tokens of each sequence, over keys and values
 *             held in pages; the first shared_len tokens may be the same pages for
 *             all sequences and are then read once for all
 *
 * Conventions are those of gdn.h: device pointers owned by the caller, work
 * enqueued on `stream`, no allocation, no synchronization, nothing read back, so
 * that every call can be captured in a CUDA graph; a negative gdn_status for an
 * argument error (nothing is enqueued then), bits of a device status word
 * (gdn_dev_status) for what only the data reveals, which never faults.
 * Layouts are dense, row-major, innermost dimension last:
 *   x                 [T, (H + 2 Hk) * D]  projection output, channels q | k | v
 *   q, out            [T, H, D]            (decode: [N, n_q, H, D], T = N * n_q)
 *   k, v              [T, Hk, D]
 *   lse               [T, H] fp32          log of the softmax denominator, natural
 *                                          log, scale included; -inf for a row that
 *                                          sees no key
 *   k_cache, v_cache  [n_pages, Hk, page_size, D]
 *   page_table        [N, max_pages] int32: sequence n's token t is held by page
 *                     page_table[n, t / page_size] at row t % page_size
 *   kv_lens           [N] int32: tokens of each sequence in the cache, the call's
 *                     own tokens included (they are the last ones)
 *   cu_seqlens        [N + 1] int32 prefix sums of the call's new tokens, or NULL for
 *                     one sequence of T tokens
 *   rope              [max_pos, rot_dim] fp32: row p holds cos(p * f_i) for the
 *                     rot_dim / 2 frequencies f_i, then sin(p * f_i); a scaling rule
 *                     for long contexts is a choice of f_i (and of a factor on both)
 */
#ifndef GDN_ATTN_H_
#define GDN_ATTN_H_

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
  GDN_ATTN_ROPE_INTERLEAVED = 1u  /* rotate pairs (2i, 2i + 1); without it the pairs are
                                     (i, i + rot_dim / 2) */
};

/*
 * Problem descriptor. Fields:
 *   T            rows of x, q, k, v, out (0: the call does nothing and takes NULL tensors)
 *   N            sequences
 *   H, Hk        query heads and key heads; H a multiple of Hk, H / Hk <= 64
 *   D            head size, 64 or 128
 *   page_size    tokens per page: 16, 32, 64, 128 or 256 (0: no cache in the call)
 *   n_pages      pages in k_cache and v_cache
 *   max_pages    columns of page_table
 *   rot_dim      rotated elements at the start of each head: 0 or a multiple of 16, <= D
 *   max_pos      rows of rope
 *   in_dtype     gdn_dtype of x (front), q, k, v and the cache (prefill and decode:
 *                GDN_BF16 only)
 *   out_dtype    gdn_dtype of q, k, v and the cache (front), out (prefill, decode)
 *   flags        GDN_ATTN_* bits
 *   norm_eps     eps of the norms; <= 0 selects 1e-6
 *   status       one int32 of device memory, cleared by the call and then ORed with
 *                gdn_dev_status bits, or NULL
 *   workspace    device scratch of gdn_attn_workspace_size(desc) bytes for
 *                gdn_attn_decode, 256-byte aligned; it must not be used by another call
 *                that may run at the same time (the other two calls need none)
 */
typedef struct gdn_attn_desc {
  int32_t T;
  int32_t N;
  int32_t H;
  int32_t Hk;
  int32_t D;
  int32_t page_size;
  int32_t n_pages;
  int32_t max_pages;
  int32_t rot_dim;
  int32_t max_pos;
  int32_t in_dtype;
  int32_t out_dtype;
  uint32_t flags;
  float norm_eps;
  int32_t* status;
  void* workspace;
  size_t workspace_bytes;
} gdn_attn_desc;

/* Validate a descriptor's dimensions, dtypes and flags (host only; no pointer is looked at). */
int gdn_attn_check_desc(const gdn_attn_desc* desc);

/*
 * Bytes of workspace gdn_attn_decode needs for this descriptor: the partial results of a
 * long axis split over the GPU's SMs. 0 if the descriptor is invalid or T is not a
 * multiple of N. It depends on T, N, H, Hk and D, and on the current device, not on the
 * lengths, so a workspace serves every step of a batch.
 */
size_t gdn_attn_workspace_size(const gdn_attn_desc* desc);

/*
 * Front end: projection output to q, k, v.
 *   x            [T, (H + 2 Hk) * D] in in_dtype
 *   q_weight, k_weight  fp32 [D], the norms' weights; NULL: that norm is left out
 *   rope         the table above; NULL when rot_dim = 0
 *   kv_lens      [N]; token t of sequence n has position kv_lens[n] - len_n + t. NULL: t
 *   page_table, k_cache, v_cache  where k and v are appended; all NULL: not appended
 *   q            [T, H, D] in out_dtype
 *   k, v         [T, Hk, D] in out_dtype; both NULL: not written
 * Norm, rotation and their sums are fp32, rounded once to out_dtype; any finite row has a
 * finite norm, elements past the rotated ones are not touched by the rotation, and an infinite
 * element takes only its own head with it (where that is normed). Rows outside every
 * sequence are not written. A position past max_pos uses the table's last row
 * (GDN_DEV_BAD_LENGTH); a token whose place in the cache does not exist is not appended
 * (GDN_DEV_BAD_PAGE_TABLE for a page outside [0, n_pages), GDN_DEV_BAD_LENGTH for a
 * position outside the table). A malformed cu_seqlens (GDN_DEV_BAD_CU_SEQLENS) gives
 * in-bounds but otherwise undefined results. Two tokens at the same place: undefined.
 */
int gdn_attn_front(const gdn_attn_desc* desc, const void* x, const float* q_weight,
                   const float* k_weight, const float* rope, const int32_t* cu_seqlens,
                   const int32_t* kv_lens, const int32_t* page_table, void* q, void* k, void* v,
                   void* k_cache, void* v_cache, cudaStream_t stream);

/*
 * Causal attention of packed prompts over their own keys and values.
 *   q [T, H, D], k, v [T, Hk, D]  bf16
 *   scale        <= 0 or NaN selects 1/sqrt(D)
 *   out          [T, H, D] in out_dtype; rows outside every sequence are not written
 *   lse          [T, H] fp32 or NULL
 * Entries of a malformed cu_seqlens are clamped to [0, T] and raised to the largest entry
 * before them (GDN_DEV_BAD_CU_SEQLENS; past 1024 sequences, to the largest of their 1024). What a row does not see has no influence on it,
 * infinities and NaN included.
 */
int gdn_attn_prefill(const gdn_attn_desc* desc, const void* q, const void* k, const void* v,
                     const int32_t* cu_seqlens, float scale, void* out, float* lse,
                     cudaStream_t stream);

/*
 * Attention of the last n_q = T / N tokens of each sequence over the paged cache (n_q = 1:
 * decode; a few: speculative verification). n_q * H / Hk <= 64.
 *   q            [N, n_q, H, D] bf16
 *   kv_lens      [N]: row i of sequence n sees keys 0 .. kv_lens[n] - n_q + i; a sequence of
 *                length 0 (padding) gets zeros
 *   shared_len   the first shared_len tokens of every sequence are the same pages (a
 *                multiple of page_size; their columns are read from page_table's first row
 *                only), which are read once for all where that pays; 0: none. A sequence may be shorter than shared_len.
 *   scale, out, lse  as for gdn_attn_prefill ([N, n_q, H, D], [N, n_q, H])
 * A length outside [0, max_pages * page_size] is clamped (GDN_DEV_BAD_LENGTH); keys and
 * values of a page outside [0, n_pages) read as zeros (GDN_DEV_BAD_PAGE_TABLE). Rows of the
 * cache past a sequence's length have no influence, infinities and NaN included.
 */
int gdn_attn_decode(const gdn_attn_desc* desc, const void* q, const void* k_cache,
                    const void* v_cache, const int32_t* page_table, const int32_t* kv_lens,
                    int32_t shared_len, float scale, void* out, float* lse, cudaStream_t stream);

/*
 * Testing hook. gdn_attn_decode gives a common prefix its own pass only where that pays (many
 * sequences behind a long prefix); with always != 0 it does so at every size in the calls that
 * follow, so that tests can reach that path with small inputs. 0 (the default) turns it off.
 */
void gdn_test_attn_prefix(int32_t always);

/*
 * Testing hook. gdn_attn_prefill works on one or two tiles of rows at a time, by a rule on the
 * sizes; 1 or 2 fixes that for the calls that follow, 0 (the default) is the rule. Results are
 * the same bit for bit (where all values are finite).
 */
void gdn_test_attn_tiles(int32_t tiles);

/*
 * Testing hook. Every on-chip wait of gdn_attn_prefill and of a common prefix's own pass is
 * bounded. With polls > 0, that is the bound in the calls that follow, and what issues the
 * products waits, before a CTA's work item number `item`, for an event that never happens: the
 * wait runs out, GDN_DEV_TIMEOUT is in the status word, every warp leaves, the results of that
 * call are invalid, and copies and products in flight are still waited for (at the full bound)
 * before the kernel ends, so the device stays usable. 0 (the default) turns it off.
 */
void gdn_test_attn_timeout(uint32_t polls, uint32_t item);

#ifdef __cplusplus
}
#endif
#endif /* GDN_ATTN_H_ */
