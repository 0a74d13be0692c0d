// Attention of row tiles on the tensor cores (tcgen05), shared by the prompt kernel and the
// decode kernel's common-prefix part.
//
// Mathematics, per row with scores s_j = q . k_j: with any reference r,
//   o = sum_j 2^(c (s_j - r)) v_j / sum_j 2^(c (s_j - r)),   c = scale * log2(e),
// so the keys are taken 128 at a time with the running maximum as r. r is replaced only when
// the maximum has grown by more than kGrow (in powers of two): weights then stay below
// 2^kGrow, far inside fp32 and bf16, and the accumulator is rescaled a few times a row
// instead of once a tile. The weights are rounded to bf16 for the second product (an fp16
// weight would need an fp16 V); the denominator sums them in fp32 before that rounding.
//
// A row tile is 128 rows = floor(128 / G) tokens x the G query heads of one key head, so a
// key tile is read once for all heads of its group, and a causal tile's masked part is
// smaller. A CTA works on two row tiles (A, B) at a time against the same key tiles (on A alone
// where the prompts are too few to fill the GPU):
//   warps 0-3, 4-7  one thread per row of A, B: scores from TMEM, weights back to TMEM (over
//                   the scores), running sums, the output
//   warp 8          TMA loads: Q of both tiles, a ring of K and V tiles
//   warp 9          issues every MMA: S = Q K^T (both operands in shared memory),
//                   O += P V (P in TMEM). While A's rows are weighed, B's products run.
//   warp 10         hands out the work items (persistent CTAs, one per SM)
//   warps 12-15     V tiles with masked keys: rows past the sequence's end are zeroed, and
//                   so is a value that is not finite, because a weight of 0 would not remove
//                   it (0 * inf). The rows that do see one get it added to their result (no
//                   weight changes what it makes of it).
// TMEM: score buffers of 128 columns, then O_A and O_B of D. At D = 128 there is room for two
// buffers, one of A's and one of B's: a tile's next scores wait for its own P V, and the order
// of issue keeps them apart. At D = 64 there are three, taken in turn by the sequence of
// products (A and B of each key tile), so that the next scores are there before the row warps
// have weighed these; the products are short, and two warps issue them: warp 9 Q K^T, warp 11
// P V (one warp's issue took 1,200 cycles a product, twice the MMAs).
//
// Bound: at D = 128 the chain of a step (scores, weights, products; 2,600 cycles, 2,048 of them
// MMAs); short prompts by the start and the output of an item, about 2.3 steps. Measured
// (GB300): 16384 tokens x 32 heads 1.25 to 1.27 ms (1,740 TFLOP/s; 1.39 ms under the power limit),
// 4096 x 16 heads 51.3 us (1,340 TFLOP/s), 8 ragged prompts x 32 heads 62.5 us (963 TFLOP/s), 4001
// x 16 heads of 64 40.1 us (819 TFLOP/s).
#pragma once

#include <cuda.h>

#include <type_traits>

#include "attn_common.cuh"
#include "umma.cuh"
#include "warp_mma.cuh"

namespace gdn {

constexpr int kAttnThreads = 512;
constexpr int kRows = 128;           // rows of a tile
constexpr int kKeys = 128;           // keys of a tile
constexpr int kAttnSeqs = 1024;      // sequences of one launch
constexpr int kItems = 4;            // work items handed out ahead
constexpr float kGrow = 8.0f;

struct AttnItem {
  int base;        // first token (row of q) of the sequence (prefix: 0)
  int len;         // its tokens
  int tok;         // first token of tile A, from base
  int hk;
  int kv0;         // first key tile (prompts: 0)
  int nA, nB;      // key tiles of A and B (nB = 0: no tile B)
  int z;           // prefix: which split of the keys
  int mask0;       // first key tile that some row sees only in part
  int valid;
};

// The common prefix's part of a decode step: per split of its keys, the rows' unnormalised
// sums [splits][T][H][D], and their reference (in powers of two) and denominator.
struct PrefixParts {
  float* o;
  float2* ml;
  int splits, tiles;  // tiles: key tiles of the prefix
};

template <int D, bool kPrefix>
struct AttnSmem {
  static constexpr int kTile = 128 * D * 2;            // one Q, K or V tile
  // K and V tiles: 64-element halves of 128 rows each; a tile gathered from pages instead has
  // both halves of every 8 rows together, so that a page is one box of any height.
  static constexpr int kGroup = kPrefix ? D * 16 : 1024;    // bytes from 8 rows to the next
  static constexpr int kHalf = kPrefix ? 1024 : 128 * 128;  // ... from a half to the other
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kBufs = D == 128 ? 2 : 3;       // score buffers
  static constexpr int kQ = 0, kRing = 2 * kTile;
  static constexpr int kBounds = kRing + kStages * kTile;      // sanitized cu_seqlens, pairs
  static constexpr int kOutRow = 80;                           // 64 bytes of a row, padded
  static constexpr int kOut = kBounds + 8 * (kAttnSeqs + 4);   // 32 rows a row warp
  static constexpr int kBars = kOut + 8 * 32 * kOutRow;
  static constexpr int kBytes = kBars + 768 + 1024;            // + alignment of the tiles
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two fp32 FMAs / adds in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
      " mov.b64 z, {%6, %7};\n fma.rn.f32x2 w, x, y, z;\n mov.b64 {%0, %1}, w;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
      " add.rn.f32x2 w, x, y;\n mov.b64 {%0, %1}, w;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// The warp that issues the MMAs runs converged, and everything it issues is predicated on one
// lane, chosen once: then descriptors and addresses live in uniform registers and the loop is
// straight-line. (Issued from a `lane == 0` branch, every operand word takes a move, and a
// step's issue takes longer than its products: 5,000 cycles at D = 128 for 2,048 of MMAs.)
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p;
}
// The same value in all lanes, known as such to the compiler.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_or_sync(0xffffffffu, x); }

// D[tmem] (+)= A * B with A and B in shared memory; `el` != 0 in the issuing lane only.
__device__ __forceinline__ void mma_ss(uint32_t el, uint32_t d, uint32_t a_lo, uint32_t a_hi,
                                       uint32_t b_lo, uint32_t b_hi, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b64 a, b;\n setp.ne.b32 p, %6, 0;\n setp.ne.b32 e, %7, 0;\n"
      " mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %4};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc), "r"(el)
      : "memory");
}
// The same with A in TMEM: M x 16 bf16, two to a 32-bit column.
__device__ __forceinline__ void mma_ts(uint32_t el, uint32_t d, uint32_t a, uint32_t b_lo,
                                       uint32_t b_hi, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b64 b;\n setp.ne.b32 p, %5, 0;\n setp.ne.b32 e, %6, 0;\n"
      " mov.b64 b, {%2, %3};\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc), "r"(el)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t el, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
          smem_addr(bar)),
      "r"(el)
      : "memory");
}
__device__ __forceinline__ void arrive_one(uint32_t el, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n .reg .b64 st;\n setp.ne.b32 e, %1, 0;\n"
      " @e mbarrier.arrive.shared::cta.b64 st, [%0];\n}\n" ::"r"(smem_addr(bar)),
      "r"(el)
      : "memory");
}
__device__ __forceinline__ void tmem_st32u(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
      "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
      "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
      "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16};\n" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
      "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const void* tmap, int x, int y, int z, int w,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];\n" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void prefetch_tmap(const CUtensorMap* tm) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(tm)) : "memory");
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}

// Barriers of the attention kernel (all in shared memory).
template <int kStages, int kSet>
struct AttnBars {
  // A V tile with masked keys completes v_raw and, once the V warps are done, v_fixed, in
  // place of kv_full: so whoever waits on one of the three sees each of its phases.
  uint64_t kv_full[kStages], kv_empty[kStages], v_raw[kStages], v_fixed[kStages];
  // s_full, p_full, o_full: A's and B's scores, weights and products into O are complete (with
  // two score buffers, o_full: the item's last product). With three score buffers, all may hold tiles of one of them, and one side of a barrier be as
  // many tiles ahead of the other's wait: so A's and B's tiles each take the barriers in turn.
  // buf_empty: the product with the weights in a score buffer is complete.
  uint64_t q_full[2], q_empty[2], s_full[2][kSet], p_full[2][kSet], o_full[2][kSet];
  uint64_t o_empty[2], buf_empty[3];
  uint64_t idle[2];  // all products of an issuing warp are complete
  uint64_t item_full[kItems], item_empty[kItems];
  AttnItem item[kItems];
  uint32_t tmem;
  // Item number + 1 of the last item in this place with a value taken out of a V tile: the
  // ring holds V tiles of at most four items after the one whose rows are being written.
  int poison[8];
};

// A bounded wait. Once one has run out, the thread waits for nothing any more and goes on to its
// next item, where its warp leaves; the others' waits run out in turn, and the call's results are
// invalid. What must not happen is that a ring place is loaded again before its last copy has
// landed (a barrier that counts bytes would be armed twice): so the load warp stops at its first
// failure, and a place is not handed back (v_fixed, kv_empty, q_empty) by a thread that has given
// up. Copies and products in flight are waited for before the CTA ends. (Not to issue products
// after a failure would put a test into their stream: 4096 tokens 53.9 -> 70.5 us.)
struct Waiter {
  uint32_t limit;
  int32_t* status;
  __device__ Waiter(int32_t* s, uint32_t polls) : limit(polls), status(s) {}
  __device__ __forceinline__ bool ok() const { return limit != 0; }
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t phase) {
    if (mbar_try_wait(bar, phase & 1u)) return;
    for (uint32_t i = 0; i < limit; ++i)
      if (mbar_try_wait(bar, phase & 1u)) return;
    if (limit) set_status(status, GDN_DEV_TIMEOUT);
    limit = 0;
  }
};

// The work items of a batch of prompts, the ones with most keys first: pair i of a sequence
// is its tokens [i * span, (i + 1) * span); the pairs of all sequences are numbered by
// falling i, so that those that start last are the shortest. Called by one warp; each lane
// keeps the pair count of one sequence in a register (more sequences: in shared memory),
// because the first tile's loads wait for the first item.
struct PromptItems {
  const int* bounds;  // [N + 1] in shared memory
  const int* pairs;   // [N] in shared memory
  int N, span, Hk, mine, most, total;  // most: pairs of the longest sequence; total: items

  __device__ PromptItems(const int* bounds_, const int* pairs_, int N_, int span_, int Hk_)
      : bounds(bounds_), pairs(pairs_), N(N_), span(span_), Hk(Hk_) {
    const int lane = threadIdx.x & 31;
    mine = lane < N ? pairs[lane] : 0;
    int m = mine;
    for (int n = lane + 32; n < N; n += 32) m = max(m, pairs[n]);
    most = __reduce_max_sync(0xffffffffu, m);
    total = count(0) * Hk;
  }
  // pairs numbered i or higher, over all sequences
  __device__ int count(int i) const {
    int c = max(0, mine - i);
    for (int n = (threadIdx.x & 31) + 32; n < N; n += 32) c += max(0, pairs[n] - i);
    return __reduce_add_sync(0xffffffffu, c);
  }
  __device__ AttnItem get(int idx, int nt) const {
    AttnItem it{};
    if (idx >= total) return it;
    const int s = idx / Hk, lane = threadIdx.x & 31;
    int i, n = 0;
    if (N == 1) {
      i = most - 1 - s;
    } else {
      int lo = 0, hi = most - 1;  // the largest i with count(i) > s
      while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (count(m) > s) lo = m;
        else hi = m - 1;
      }
      i = lo;
      int r = s - count(i + 1);  // of the sequences that have a pair i, the r-th
      for (int n0 = 0; n0 < N; n0 += 32) {
        const bool has = n0 + lane < N && (n0 ? pairs[n0 + lane] : mine) > i;
        const uint32_t mask = __ballot_sync(0xffffffffu, has);
        const bool it_is = has && __popc(mask & ((1u << lane) - 1u)) == r;
        const uint32_t hit = __ballot_sync(0xffffffffu, it_is);
        if (hit) {
          n = n0 + __ffs(hit) - 1;
          break;
        }
        r -= __popc(mask);
      }
    }
    it.base = bounds[n];
    it.len = bounds[n + 1] - it.base;
    it.tok = i * span;
    it.hk = idx - s * Hk;
    it.nA = (min(it.tok + nt, it.len) + kKeys - 1) / kKeys;
    it.nB = span > nt && it.tok + nt < it.len ? (min(it.tok + 2 * nt, it.len) + kKeys - 1) / kKeys : 0;
    it.mask0 = (it.tok + 1) / kKeys;
    it.valid = 1;
    return it;
  }
};

// The work items of a common prefix: (pair of row tiles, key head, split of the keys).
struct PrefixItems {
  const AttnParams& p;
  const PrefixParts& x;
  int span, total;

  __device__ PrefixItems(const AttnParams& p_, const PrefixParts& x_, int span_)
      : p(p_), x(x_), span(span_) {
    total = (p.T + span - 1) / span * p.Hk * x.splits;
  }
  __device__ AttnItem get(int idx, int nt) const {
    AttnItem it{};
    if (idx >= total) return it;
    // The split runs fastest: CTAs that work at the same time read neighbouring keys.
    const uint32_t at = (uint32_t)idx / x.splits, pair = at / p.Hk, lane = threadIdx.x & 31;
    const int q = x.tiles / x.splits, rest = x.tiles - q * x.splits;  // the first have one more
    it.z = idx - at * x.splits;
    it.len = p.T;
    it.tok = pair * span;
    it.hk = at - pair * p.Hk;
    it.kv0 = it.z * q + min(it.z, rest);
    it.nA = q + (it.z < rest);
    it.nB = it.tok + nt < it.len ? it.nA : 0;
    // keys that every row of the pair sees: a sequence's first new token sees the fewest
    int lim = p.shared;
    const int last = min(it.tok + span, it.len) - 1;
    for (int n = it.tok / p.nq + lane; n <= last / p.nq; n += 32)
      lim = min(lim, keys_seen(p, n, 0));
    it.mask0 = max(__reduce_min_sync(0xffffffffu, lim) / kKeys - it.kv0, 0);
    it.valid = 1;
    return it;
  }
};

template <int D, bool kPrefix>
__global__ void __launch_bounds__(kAttnThreads, 1)
attn_tc_kernel(const AttnParams p, const PrefixParts parts,
               const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
               const __grid_constant__ CUtensorMap tm_v) {
  using S = AttnSmem<D, kPrefix>;
  constexpr int kStages = S::kStages, kBufs = S::kBufs;
  constexpr int kSet = kBufs == 2 ? 1 : kBufs;  // barriers of a kind for each of A and B
  extern __shared__ char smem_raw[];
  char* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  int* bounds = reinterpret_cast<int*>(smem + S::kBounds);
  int* pairs = bounds + kAttnSeqs + 4;  // pairs of row tiles of each sequence
  auto& B = *reinterpret_cast<AttnBars<kStages, kSet>*>(smem + S::kBars);
  static_assert(sizeof(AttnBars<kStages, kSet>) <= 768, "barrier area");
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int nt = kRows / p.G;  // tokens of a row tile
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&B.kv_full[i], 1);
      mbar_init(&B.kv_empty[i], 1);
      mbar_init(&B.v_raw[i], 1);
      mbar_init(&B.v_fixed[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B.q_full[i], 1);
      mbar_init(&B.q_empty[i], 1);
      mbar_init(&B.o_empty[i], 4);
      for (int x = 0; x < kSet; ++x) {
        mbar_init(&B.s_full[i][x], 1);
        mbar_init(&B.p_full[i][x], 4);
        mbar_init(&B.o_full[i][x], 1);
      }
    }
    for (int i = 0; i < 3; ++i) mbar_init(&B.buf_empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&B.idle[i], 1);
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&B.item_full[i], 1);
      mbar_init(&B.item_empty[i], kBufs == 2 ? 14 : 15);  // load, MMA, 8 row warps, 4 V warps
    }
    for (int i = 0; i < 8; ++i) B.poison[i] = 0;
    mbar_init_fence();
  }
  if (warp == 8) {
    tmem_alloc(&B.tmem, 512);
    tmem_relinquish();
    if (lane < 3) prefetch_tmap(lane == 0 ? &tm_q : lane == 1 ? &tm_k : &tm_v);
  }
  // All of the above needs nothing of the launch before this one in the stream.
  pdl_wait();
  if (kPrefix) pdl_release();  // the decode kernel needs nothing from here
  if (!kPrefix && warp == 10) {  // cu_seqlens, each entry clamped and raised to the largest before it
    const int span = p.tiles * nt;
    int carry = 0;
    bool bad = false;
    for (int n0 = 0; n0 <= p.N; n0 += 32) {
      const int n = n0 + lane;
      const int raw = n > p.N ? 0 : p.cu ? p.cu[n] : n ? p.T : 0;
      int e = min(max(raw, 0), p.T);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, e, o);
        if (lane >= o) e = max(e, x);
      }
      e = max(e, carry);
      int before = __shfl_up_sync(0xffffffffu, e, 1);
      if (lane == 0) before = n ? carry : e;
      if (n <= p.N) {
        bounds[n] = e;
        if (n) pairs[n - 1] = (e - before + span - 1) / span;
        bad |= raw != e;
      }
      carry = __shfl_sync(0xffffffffu, e, 31);
    }
    if (bad && blockIdx.x == 0) set_status(p.status, GDN_DEV_BAD_CU_SEQLENS);
    __syncwarp();
  }
  // A prefix's first item is found while TMEM is allocated, as its lookup waits for the sequences'
  // lengths (64 sequences behind 16384 keys, the whole call 55.0 -> 53.7 us). Prompts find
  // theirs from shared memory, later: there the same costs more code than it saves (20 short
  // prompts 13.3 -> 13.5 us).
  if (kPrefix && warp == 10) {
    const AttnItem it = PrefixItems(p, parts, 2 * nt).get((int)blockIdx.x, nt);
    if (lane == 0) B.item[0] = it;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B.tmem;
  Waiter wait(p.status, p.polls);
  // Whether any lane of this warp has seen the last item, or has given up.
  auto done = [&](const AttnItem& it) {
    return __any_sync(0xffffffffu, !it.valid || !wait.ok()) != 0;
  };

  // ------------------------------------------------------------------ rows
  if (warp < 8) {
    regs_inc<192>();
    const int X = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tO = tmem + lanes + kBufs * 128 + X * D;
    const float c = p.scale * 1.44269504088896340736f;
    const int rt = row / p.G, rh = row - rt * p.G;  // token and head of this row in the tile
    // the item's first product; products into O_X and tiles written before it
    uint32_t seq0 = 0, products = 0, written = 0;
    for (uint32_t k = 0;; ++k) {
      wait(&B.item_full[k % kItems], k / kItems);
      const AttnItem it = B.item[k % kItems];
      __syncwarp();
      if (lane == 0) mbar_arrive(&B.item_empty[k % kItems]);
      if (done(it)) break;
      const int n = X ? it.nB : it.nA;
      const uint32_t first = seq0;
      seq0 += it.nA + it.nB;
      if (n == 0) continue;
      const int tok = it.tok + X * nt + rt;
      const bool real = rt < nt && tok < it.len;
      const int last = min(tok, it.len - 1);
      // keys this row sees, from the item's first
      const int lim = kPrefix ? min(keys_seen(p, last / p.nq, last % p.nq), p.shared) - it.kv0 * kKeys
                              : last + 1;
      float ref = -INFINITY, l = 0.f;            // reference of the weights, their sum
      for (int j = 0; j < n; ++j) {
        // this tile's place among all products, and among those of X
        const uint32_t seq = first + j + (X ? min(j + 1, it.nA) : min(j, it.nB)), own = products + j;
        const uint32_t tS = tmem + lanes + (kBufs == 2 ? X : seq % kBufs) * 128;
        wait(&B.s_full[X][own % kSet], own / kSet);
        tc_fence_after();
        float s[128];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          tmem_ld32(tS + 32 * q, *reinterpret_cast<float(*)[32]>(&s[32 * q]));
        tmem_ld_wait();
        const int seen = lim - j * kKeys;
        if (__any_sync(0xffffffffu, seen < kKeys)) {
#pragma unroll
          for (int i = 0; i < 128; ++i) s[i] = i < seen ? s[i] : -INFINITY;
        }
        float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int i = 4; i < 128; i += 4) {
          m4[0] = fmaxf(m4[0], s[i]);
          m4[1] = fmaxf(m4[1], s[i + 1]);
          m4[2] = fmaxf(m4[2], s[i + 2]);
          m4[3] = fmaxf(m4[3], s[i + 3]);
        }
        const float m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        // A new reference where the maximum outgrew the old one (always in the first tile
        // that holds a key).
        const bool grown = m > ref && (m - ref) * c > kGrow;
        if (__any_sync(0xffffffffu, grown)) {
          const float f = grown ? ex2((ref - m) * c) : 1.f;  // 0 from -inf
          if (grown) ref = m;
          l *= f;
          if (j > 0) {
            // (in order of issue, the product of the tile before is complete when S is; three
            // buffers have S made before it)
            if (kBufs > 2) wait(&B.o_full[X][(own - 1) % kSet], (own - 1) / kSet);
            tc_fence_after();
#pragma unroll 1
            for (int q = 0; q < D; q += 16) {
              float o[16];
              tmem_ld16(tO + q, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= f;
              tmem_st16(tO + q, o);
            }
          }
        }
        const float nr = ref == -INFINITY ? 0.f : -ref * c;
        const float2 c2 = make_float2(c, c), r2 = make_float2(nr, nr);
        float2 l0 = make_float2(l, 0.f), l1 = make_float2(0.f, 0.f);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const int e = 64 * q + 2 * i;
            float2 a = fma2(make_float2(s[e], s[e + 1]), c2, r2);
            float2 b = fma2(make_float2(s[e + 2], s[e + 3]), c2, r2);
            a.x = ex2(a.x); a.y = ex2(a.y); b.x = ex2(b.x); b.y = ex2(b.y);
            l0 = add2(l0, a);
            l1 = add2(l1, b);
            w[i] = pack_bf16(a.x, a.y);
            w[i + 1] = pack_bf16(b.x, b.y);
          }
          tmem_st32u(tS + 32 * q, w);
        }
        l = (l0.x + l0.y) + (l1.x + l1.y);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.p_full[X][own % kSet]);
      }
      products += n;
      if (kBufs == 2) wait(&B.o_full[X][0], written);
      else wait(&B.o_full[X][(products - 1) % kSet], (products - 1) / kSet);
      ++written;
      tc_fence_after();
      int64_t at = (int64_t)(it.base + tok) * p.H + it.hk * p.G + rh;
      const int64_t part0 = kPrefix ? (int64_t)it.z * p.T * p.H : 0;  // the split's rows
      at += part0;
      const bool poison = *reinterpret_cast<volatile int*>(&B.poison[k & 7]) == (int)k + 1;
      // prefix: as they are, for the merge with the other splits; NaN stays NaN
      const float r = kPrefix ? 1.f : l == 0.f ? 0.f : 1.f / l;
      // A thread holds a whole row; stored from here, every 16 bytes of a warp's store would
      // fall into another line (4,000 cycles a pair of tiles). So 64 bytes a row at a time go
      // through shared memory, and four lanes write one row's. A rolled loop: this code is
      // fetched anew for every item.
      char* stage = smem + S::kOut + warp * (32 * S::kOutRow);
      int64_t to[4];  // the rows that this lane writes, -1: none
#pragma unroll
      for (int i = 0; i < 4; ++i)
        to[i] = __shfl_sync(0xffffffffu, real ? at : -1, i * 8 + (lane >> 2));
      const bool wide = kPrefix || !p.out_bf16;  // fp32 rows
      char* out = static_cast<char*>(kPrefix ? static_cast<void*>(parts.o) : p.out) + (lane & 3) * 16;
#pragma unroll 1
      for (int q = 0; q < D; q += wide ? 16 : 32) {
        float o[32];
        tmem_ld16(tO + q, *reinterpret_cast<float(*)[16]>(&o[0]));
        if (!wide) tmem_ld16(tO + q + 16, *reinterpret_cast<float(*)[16]>(&o[16]));
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4 y;
          if (wide)
            y = make_uint4(__float_as_uint(o[4 * i] * r), __float_as_uint(o[4 * i + 1] * r),
                           __float_as_uint(o[4 * i + 2] * r), __float_as_uint(o[4 * i + 3] * r));
          else
            y = make_uint4(pack_bf16(o[8 * i] * r, o[8 * i + 1] * r),
                           pack_bf16(o[8 * i + 2] * r, o[8 * i + 3] * r),
                           pack_bf16(o[8 * i + 4] * r, o[8 * i + 5] * r),
                           pack_bf16(o[8 * i + 6] * r, o[8 * i + 7] * r));
          *reinterpret_cast<uint4*>(stage + lane * S::kOutRow + i * 16) = y;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 z = *reinterpret_cast<const uint4*>(stage + (i * 8 + (lane >> 2)) * S::kOutRow +
                                                          (lane & 3) * 16);
          if (to[i] >= 0) {
            const int64_t byte = wide ? (to[i] * D + q) * 4 : (to[i] * D + q) * 2;
            *reinterpret_cast<uint4*>(out + byte) = z;
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&B.o_empty[X]);
      if constexpr (kPrefix) {
        if (real) parts.ml[at] = make_float2(ref * c, l);
      } else {
        if (real && p.lse) p.lse[at] = l == 0.f ? -INFINITY : ref * p.scale + logf(l);
      }
      if (poison) {  // values that were taken out of V tiles go to this warp's rows that see them
        __syncwarp();
        constexpr int E = D / 32;
        const int sees = real ? lim : 0;
        const int end = __reduce_max_sync(0xffffffffu, min(sees, n * kKeys));
#pragma unroll 1
        for (int key = kPrefix ? it.mask0 * kKeys : it.tok + 1; key < end; ++key) {
          const __nv_bfloat16* v = p.v + lane * E;
          if constexpr (kPrefix) {
            const int at_key = it.kv0 * kKeys + key, pg = p.table[at_key >> p.page_shift];
            if (pg < 0 || pg >= p.n_pages) continue;
            v += ((((size_t)pg * p.Hk + it.hk) << p.page_shift) + (at_key & (p.page - 1))) * D;
          } else {
            v += ((size_t)(it.base + key) * p.Hk + it.hk) * D;
          }
          float x[E];
          bool bad = false;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            x[e] = __bfloat162float(v[e]);
            bad |= !isfinite(x[e]);
          }
          if (!__any_sync(0xffffffffu, bad)) continue;
#pragma unroll 1
          for (int i = 0; i < 32; ++i) {
            const int64_t row = __shfl_sync(0xffffffffu, at, i);
            if (key >= __shfl_sync(0xffffffffu, sees, i)) continue;
#pragma unroll
            for (int e = 0; e < E; ++e) {
              if (isfinite(x[e])) continue;
              const int64_t to_e = row * D + lane * E + e;
              if (wide) {
                (kPrefix ? parts.o : static_cast<float*>(p.out))[to_e] += x[e];
              } else {
                __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.out) + to_e;
                *y = __float2bfloat16_rn(__bfloat162float(*y) + x[e]);
              }
            }
          }
        }
      }
    }
  } else if (warp < 12) {
    regs_dec<88>();
    // ---------------------------------------------------------------- loads
    if (warp == 8 && (kPrefix || lane == 0)) {
      uint32_t slot = 0, loads[2] = {0, 0};
      uint32_t kv_uses = 0, raw_uses = 0, is_raw = 0;  // per stage: uses (mod 2), the last one
      for (uint32_t k = 0;; ++k) {
        wait(&B.item_full[k % kItems], k / kItems);
        const AttnItem it = B.item[k % kItems];
        if constexpr (kPrefix) __syncwarp();
        if (lane == 0) mbar_arrive(&B.item_empty[k % kItems]);
        if (kPrefix ? done(it) : !it.valid || !wait.ok()) break;
        const int n = max(it.nA, it.nB);
        auto load_q = [&](int X) {
          if (X && it.nB == 0) return;
          wait(&B.q_empty[X], loads[X] + 1);
          if (!wait.ok()) return;
          ++loads[X];
          if (lane != 0) return;
          mbar_expect_tx(&B.q_full[X], (uint32_t)(nt * p.G * D * 2));
          for (int d = 0; d < D; d += 64)
            tma_load_3d(smem + S::kQ + X * S::kTile + d * 256, &tm_q, d, it.hk * p.G,
                        it.base + it.tok + X * nt, &B.q_full[X]);
        };
        // Page of this lane's part of key tile j (prefix): a tile is up to eight pages, one
        // lane each, or part of one; -1 past the prefix. Looked up a tile ahead.
        auto page_of = [&](int j) -> int {
          const int key = (it.kv0 + j) * kKeys + lane * min(p.page, kKeys);
          return lane * p.page < kKeys && key < p.shared ? p.table[key >> p.page_shift] : -1;
        };
        int page = 0;
        auto load_kv = [&](const CUtensorMap* tm, int j, bool raw) {
          const int st = slot % kStages;
          wait(&B.kv_empty[st], slot / kStages + 1);
          if (kPrefix ? __any_sync(0xffffffffu, !wait.ok()) : !wait.ok()) {
            wait.limit = 0;
            return;
          }
          ++slot;
          uint64_t* bar = raw ? &B.v_raw[st] : &B.kv_full[st];
          (raw ? raw_uses : kv_uses) ^= 1u << st;
          is_raw = (is_raw & ~(1u << st)) | ((uint32_t)raw << st);
          char* dst = smem + S::kRing + st * S::kTile;
          if constexpr (kPrefix) {
            const int key = (it.kv0 + j) * kKeys, box = min(p.page, kKeys);
            const int rows = min(kKeys, p.shared - key);
            if (lane == 0) mbar_expect_tx(bar, (uint32_t)(rows * D * 2));
            __syncwarp();
            if (lane * box < rows) {
              const bool ok = page >= 0 && page < p.n_pages;
              if (!ok) set_status(p.status, GDN_DEV_BAD_PAGE_TABLE);
              // a page that does not exist: past the tensor's end, which reads zeros
              const int64_t group = (((int64_t)(ok ? page : p.n_pages) * p.Hk + (ok ? it.hk : 0))
                                     << p.page_shift) + (ok ? key & (p.page - 1) : 0);
              tma_load_4d(dst + lane * box * D * 2, tm, 0, 0, 0, (int)(group >> 3), bar);
            }
          } else {
            mbar_expect_tx(bar, S::kTile);
            for (int d = 0; d < D; d += 64)
              tma_load_3d(dst + d * 256, tm, d, it.hk, it.base + j * kKeys, bar);
          }
        };
        load_q(0);
        if (kPrefix) page = page_of(0);
        load_kv(&tm_k, 0, false);
        load_q(1);
        for (int j = 0; j < n; ++j) {
          if (j > 0) load_kv(&tm_k, j, false);
          const int page_next = kPrefix && j + 1 < n ? page_of(j + 1) : 0;
          load_kv(&tm_v, j, j >= it.mask0);
          page = page_next;
        }
      }
      // Copies in flight end before the CTA does (all have been waited for already, unless someone
      // gave up).
      if (lane == 0) {
#pragma unroll 1
        for (uint32_t i = 0; i < kStages && i < slot; ++i) {
          const bool r = (is_raw >> i) & 1;
          mbar_wait(r ? &B.v_raw[i] : &B.kv_full[i], (((r ? raw_uses : kv_uses) >> i) & 1) ^ 1, kAttnPolls);
        }
#pragma unroll 1
        for (int X = 0; X < 2; ++X)
          if (loads[X]) mbar_wait(&B.q_full[X], (loads[X] - 1) & 1, kAttnPolls);
      }
    }
    // ---------------------------------------------------------------- products
    // Nothing that this warp issued is still running when TMEM is freed.
    auto finish = [&](uint32_t el, uint64_t* bar) {
      mma_commit(el, bar);
      if (!mbar_wait(bar, 0, kAttnPolls)) set_status(p.status, GDN_DEV_TIMEOUT);
    };
    if (kBufs == 2 && warp == 9) {
      constexpr uint32_t kIdS = idesc_bf16_f32(128, kKeys);
      constexpr uint32_t kIdO = idesc_bf16_f32(128, D, false, true);
      constexpr uint32_t kT = S::kTile >> 4;
      // descriptor words (sdesc_sw128): the low ones hold the address, the high ones the strides
      const uint64_t dQ = sdesc_sw128(smem_addr(smem + S::kQ), 16, 1024);
      const uint64_t dK = sdesc_sw128(smem_addr(smem + S::kRing), 16, S::kGroup);
      const uint64_t dV = sdesc_sw128(smem_addr(smem + S::kRing), S::kHalf, S::kGroup);
      const uint32_t q_lo = uniform((uint32_t)dQ), k_lo = uniform((uint32_t)dK),
                     v_lo = uniform((uint32_t)dV);
      constexpr uint32_t kHi = (1u << 14) | (2u << 29);
      constexpr uint32_t kQHi = kHi | (1024 >> 4), kKHi = kHi | (S::kGroup >> 4);
      const uint32_t el = elect_one(), tm = uniform(tmem);
      // parities to wait for, a bit per barrier
      uint32_t kvs = 0, fixes = 0, qs = 0, ps = 0, os = 3;

      auto wait_kv = [&](uint32_t st) {
        wait(&B.kv_full[st], kvs >> st);
        kvs ^= 1u << st;
      };
      auto wait_v = [&](uint32_t st, bool masked) {
        if (masked) {
          wait(&B.v_fixed[st], fixes >> st);
          fixes ^= 1u << st;
        } else {
          wait_kv(st);
        }
      };
      auto scores = [&](auto x, uint32_t st, bool last) {  // S_X = Q_X K^T
        constexpr int X = decltype(x)::value;
        tc_fence_after();
        const uint32_t b = k_lo + st * kT;
#pragma unroll
        for (int d = 0; d < D; d += 16)
          mma_ss(el, tm + X * 128, q_lo + X * kT + (((d >> 6) * 16384 + (d & 63) * 2) >> 4), kQHi,
                 b + (((d >> 6) * S::kHalf + (d & 63) * 2) >> 4), kKHi, kIdS, d > 0);
        mma_commit(el, &B.s_full[X][0]);
        if (last) mma_commit(wait.ok() ? el : 0u, &B.q_empty[X]);
      };
      auto weigh = [&](auto x, uint32_t st, bool first, bool last) {  // O_X (+)= P_X V
        constexpr int X = decltype(x)::value;
        wait(&B.p_full[X][0], ps >> X);
        ps ^= 1u << X;
        if (first) {
          wait(&B.o_empty[X], os >> X);
          os ^= 1u << X;
        }
        tc_fence_after();
        const uint32_t b = v_lo + st * kT;
#pragma unroll
        for (int t = 0; t < kKeys; t += 16)
          mma_ts(el, tm + kBufs * 128 + X * D, tm + X * 128 + (t >> 1), b + ((t >> 3) * S::kGroup >> 4),
                 kKHi, kIdO, t > 0 || !first);
        if (last) mma_commit(el, &B.o_full[X][0]);
      };
      auto wait_q = [&](int X) {
        wait(&B.q_full[X], qs >> X);
        qs ^= 1u << X;
      };
      // The fields of item k that count here (no tiles: the end).
      auto item = [&](uint32_t k, int& a, int& b, int& mask0) {
        wait(&B.item_full[k % kItems], k / kItems);
        if (p.stall == k + 1) wait(&B.idle[0], 0);
        const AttnItem& it = B.item[k % kItems];
        const bool ok = !done(it);
        a = (int)uniform(ok ? it.nA : 0);
        b = (int)uniform(ok ? it.nB : 0);
        mask0 = (int)uniform(it.mask0);
        arrive_one(el, &B.item_empty[k % kItems]);
      };
      constexpr std::integral_constant<int, 0> A{};
      constexpr std::integral_constant<int, 1> Bt{};
      int nA, nB, mask0;
      uint32_t kst = 0;  // ring place of the K tile at hand (its V tile is the next place)
      item(0, nA, nB, mask0);
      if (nA) {
        wait_q(0);
        wait_kv(0);
        scores(A, 0, nA == 1);
        if (nB) {
          wait_q(1);
          scores(Bt, 0, nB == 1);
        }
        mma_commit(wait.ok() ? el : 0u, &B.kv_empty[0]);
      }
      for (uint32_t k = 1; nA; ++k) {
        const int n = max(nA, nB);
        int a2 = 0, b2 = 0, m2 = 0;  // the next item
        wait_v(kst + 1, mask0 == 0);
        for (int j = 0; j < n; ++j) {
          const uint32_t vst = kst + 1, nst = kst + 2 == kStages ? 0 : kst + 2;
          const bool end = j == n - 1;
          if (end) item(k, a2, b2, m2);
          if (j < nA) weigh(A, vst, j == 0, j == nA - 1);
          const bool k_next = !end || a2;  // another K tile follows
          if (k_next) wait_kv(nst);
          if (j + 1 < nA) {
            scores(A, nst, j + 2 == nA);
          } else if (end && a2) {
            wait_q(0);
            scores(A, nst, a2 == 1);
          }
          if (!end) wait_v(nst + 1, j + 1 >= mask0);
          if (j < nB) weigh(Bt, vst, j == 0, j == nB - 1);
          mma_commit(wait.ok() ? el : 0u, &B.kv_empty[vst]);
          if (j + 1 < nB) {
            scores(Bt, nst, j + 2 == nB);
          } else if (end && b2) {
            wait_q(1);
            scores(Bt, nst, b2 == 1);
          }
          if (k_next) mma_commit(wait.ok() ? el : 0u, &B.kv_empty[nst]);
          kst = nst;
        }
        nA = a2;
        nB = b2;
        mask0 = m2;
      }
      finish(el, &B.idle[0]);
    }
    // Three score buffers: warp 9 issues Q K^T, warp 11 P V, in the same sequence.
    if (kBufs == 3 && (warp == 9 || warp == 11)) {
      constexpr uint32_t kT = S::kTile >> 4, kHi = (1u << 14) | (2u << 29);
      constexpr uint32_t kQHi = kHi | (1024 >> 4), kKHi = kHi | (S::kGroup >> 4);
      const uint32_t q_lo = uniform((uint32_t)sdesc_sw128(smem_addr(smem + S::kQ), 16, 1024));
      const uint32_t k_lo = uniform((uint32_t)sdesc_sw128(smem_addr(smem + S::kRing), 16, S::kGroup));
      const uint32_t v_lo =
          uniform((uint32_t)sdesc_sw128(smem_addr(smem + S::kRing), S::kHalf, S::kGroup));
      const uint32_t el = elect_one(), tm = uniform(tmem);
      const bool qk = warp == 9;
      uint32_t kvs = 0, fixes = 0;      // parities to wait for, a bit per ring place
      uint32_t qs = 0, os = 3;          // ... and for A and B
      uint32_t buf = 0, turn = 0;       // score buffer of the next product, times round
      uint32_t own[2] = {0, 0}, round[2] = {0, 0};  // barriers of A's, B's next tile, times round
      uint32_t st = qk ? 0 : 1;         // ring place of the key tile
      auto step = [&](auto x, int j, int n, bool first, bool end, bool masked) {
        constexpr int X = decltype(x)::value;
        if (qk) {
          wait(&B.buf_empty[buf], turn + 1);
          if (j == 0) {
            wait(&B.q_full[X], qs >> X);
            qs ^= 1u << X;
          }
          if (first) {
            wait(&B.kv_full[st], kvs >> st);
            kvs ^= 1u << st;
          }
          tc_fence_after();
          const uint32_t b = k_lo + st * kT;
#pragma unroll
          for (int d = 0; d < D; d += 16)
            mma_ss(el, tm + buf * 128, q_lo + X * kT + (((d >> 6) * 16384 + (d & 63) * 2) >> 4), kQHi,
                   b + (((d >> 6) * S::kHalf + (d & 63) * 2) >> 4), kKHi, idesc_bf16_f32(128, kKeys),
                   d > 0);
          mma_commit(el, &B.s_full[X][own[X]]);
          if (j == n - 1) mma_commit(wait.ok() ? el : 0u, &B.q_empty[X]);
        } else {
          if (first && masked) {
            wait(&B.v_fixed[st], fixes >> st);
            fixes ^= 1u << st;
          } else if (first) {
            wait(&B.kv_full[st], kvs >> st);
            kvs ^= 1u << st;
          }
          if (j == 0) {
            wait(&B.o_empty[X], os >> X);
            os ^= 1u << X;
          }
          wait(&B.p_full[X][own[X]], round[X]);
          tc_fence_after();
          const uint32_t b = v_lo + st * kT;
#pragma unroll
          for (int t = 0; t < kKeys; t += 16)
            mma_ts(el, tm + kBufs * 128 + X * D, tm + buf * 128 + (t >> 1),
                   b + ((t >> 3) * S::kGroup >> 4), kKHi, idesc_bf16_f32(128, D, false, true),
                   t > 0 || j > 0);
          mma_commit(el, &B.o_full[X][own[X]]);
          mma_commit(el, &B.buf_empty[buf]);
        }
        if (end) {  // the last product of this key tile
          mma_commit(wait.ok() ? el : 0u, &B.kv_empty[st]);
          st = st + 2 >= kStages ? st + 2 - kStages : st + 2;
        }
        if (++buf == kBufs) {
          buf = 0;
          ++turn;
        }
        if (++own[X] == kSet) {
          own[X] = 0;
          ++round[X];
        }
      };
      for (uint32_t k = 0;; ++k) {
        wait(&B.item_full[k % kItems], k / kItems);
        if (qk && p.stall == k + 1) wait(&B.idle[0], 0);
        const AttnItem& it = B.item[k % kItems];
        const bool ok = !done(it);
        const int nA = (int)uniform(ok ? it.nA : 0), nB = (int)uniform(ok ? it.nB : 0);
        const int mask0 = (int)uniform(it.mask0);
        arrive_one(el, &B.item_empty[k % kItems]);
        if (nA == 0) break;
        for (int j = 0; j < max(nA, nB); ++j) {
          if (j < nA) step(std::integral_constant<int, 0>{}, j, nA, true, j >= nB, j >= mask0);
          if (j < nB) step(std::integral_constant<int, 1>{}, j, nB, j >= nA, true, j >= mask0);
        }
      }
      finish(el, &B.idle[qk ? 0 : 1]);
    }
    // ---------------------------------------------------------------- work items
    if (warp == 10) {
      if (kPrefix && lane == 0) mbar_arrive(&B.item_full[0]);  // found above
      auto items = [&] {
        if constexpr (kPrefix) {
          return PrefixItems(p, parts, 2 * nt);
        } else {
          return PromptItems(bounds, pairs, p.N, p.tiles * nt, p.Hk);
        }
      }();
      const int grid = (int)gridDim.x, b = (int)blockIdx.x;
      const bool any = !kPrefix || B.item[0].valid;
      for (uint32_t k = kPrefix; any; ++k) {
        // every other round dealt backwards, which evens out the falling sizes
        const int64_t idx = (int64_t)k * grid + ((k & 1) ? grid - 1 - b : b);
        const AttnItem it = items.get((int)min(idx, (int64_t)items.total), nt);
        wait(&B.item_empty[k % kItems], k / kItems + 1);
        if (__any_sync(0xffffffffu, !wait.ok())) break;
        if (lane == 0) {
          B.item[k % kItems] = it;
          mbar_arrive(&B.item_full[k % kItems]);
        }
        __syncwarp();
        // a round dealt backwards may skip this CTA in the last, partial round only
        if (!it.valid) break;
      }
    }
    __syncwarp();
  } else {
    regs_dec<40>();
    // ---------------------------------------------------------------- V tiles with masked keys
    const int tid = threadIdx.x - 12 * 32;
    uint32_t base = 0, raws = 0;
    for (uint32_t k = 0;; ++k) {
      wait(&B.item_full[k % kItems], k / kItems);
      const AttnItem it = B.item[k % kItems];
      __syncwarp();
      if (lane == 0) mbar_arrive(&B.item_empty[k % kItems]);
      if (done(it)) break;
      const int n = max(it.nA, it.nB);
      for (int j = it.mask0; j < n; ++j) {
        const uint32_t st = (base + 2 * j + 1) % kStages;
        wait(&B.v_raw[st], raws >> st);
        raws ^= 1u << st;
        char* tile = smem + S::kRing + st * S::kTile;
        // rows of this tile inside the sequence, the prefix
        const int rows = (kPrefix ? p.shared : it.len) - (it.kv0 + j) * kKeys;
        // Prompts: keys up to the first row's own are seen by all rows of the item and stay as
        // they are. (A prefix's rows may end anywhere.) Rolled loops: unrolled, the code that
        // is fetched for every item costs more than they save (8 ragged prompts 64.6 against
        // 62.2 us).
        const int seen = kPrefix ? 0 : max(it.tok + 1 - j * kKeys, 0);
        bool found = false;
        auto look = [&](uint4* v, int row) {
          if (row >= rows) {
            *v = make_uint4(0, 0, 0, 0);
          } else {
            const uint4 x = *v;  // a bf16 exponent of all ones, in either half
            const uint32_t e = ((x.x & 0x7F807F80u) + 0x00800080u) |
                               ((x.y & 0x7F807F80u) + 0x00800080u) |
                               ((x.z & 0x7F807F80u) + 0x00800080u) |
                               ((x.w & 0x7F807F80u) + 0x00800080u);
            if (e & 0x80008000u) {
              found = true;
              uint16_t* y = reinterpret_cast<uint16_t*>(v);
#pragma unroll 1
              for (int i = 0; i < 8; ++i)
                if ((y[i] & 0x7F80) == 0x7F80) y[i] = 0;
            }
          }
        };
        uint4* v = reinterpret_cast<uint4*>(tile);
        if constexpr (kPrefix) {
#pragma unroll 1
          for (int i = tid; i < S::kTile / 16; i += 128) look(v + i, i / D * 8 + ((i >> 3) & 7));
        } else {
#pragma unroll 1
          for (int i = seen * 8 + tid; i < kKeys * 8; i += 128) {
#pragma unroll
            for (int h = 0; h < D / 64; ++h) look(v + h * kKeys * 8 + i, i >> 3);
          }
        }
        if (found) *reinterpret_cast<volatile int*>(&B.poison[k & 7]) = (int)k + 1;
        fence_async_smem();
        __syncwarp();
        if (lane == 0 && wait.ok()) mbar_arrive(&B.v_fixed[st]);
      }
      base += 2 * n;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

// One launch over the q rows [T, H, D]; the items' number bounds the grid.
template <int D, bool kPrefix>
bool launch_attn_tc(const AttnParams& p, const PrefixParts& parts, const CUtensorMap& tm_k,
                    const CUtensorMap& tm_v, int64_t items, cudaStream_t s) {
  const uint32_t box[3] = {64, (uint32_t)p.G, (uint32_t)(kRows / p.G)};
  const uint64_t dim[3] = {D, (uint64_t)p.H, (uint64_t)p.T}, str[2] = {D * 2, (uint64_t)p.H * D * 2};
  CUtensorMap tm_q;
  if (!encode_bf16_tmap(&tm_q, p.q, 3, dim, str, box)) return false;
  const auto kernel = attn_tc_kernel<D, kPrefix>;
  constexpr int smem = AttnSmem<D, kPrefix>::kBytes;
  ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem);
  const int64_t sms = num_sms();
  return launch_pdl(kernel, dim3((unsigned)(items < sms ? items : sms)), dim3(kAttnThreads), smem, s,
                    p, parts, tm_q, tm_k, tm_v) == cudaSuccess;
}

}  // namespace gdn
