// The weight that a prompt's rows give its keys: w_j = sum over the rows i >= j of the window and
// the query heads of the group of exp(scale q_i . k_j - lse_i), on the tensor cores.
//
// With the keys as the rows of the product, S^T = K Q^T, a key's scores are one lane of TMEM and
// its sum is one thread's: no exchange between threads, and no weights are stored. A step is 128
// query rows (tokens of one head) against a pair of key tiles, A and B, of 128 keys, so that a Q
// tile is read once for both: two M = 128, N = 128 products, 2 x 16384 exponentials.
//   warps 0-7, 8-15 two threads per key of A, B: 2^(c s) of 64 of its 128 columns each, summed in fp32,
//                   four partial sums a step. (With one thread a key, eight warps, the exponentials'
//                   latency shows: 405 cycles for 32 columns, 256 of them the unit's.)
//   warp 16         TMA loads: a pair's K tiles (two pairs), a ring of Q tiles
//   warp 17         issues the MMAs; a step's scores are in one of two TMEM buffers a tile
//   warp 18         the rows' -lse / scale as 16 more elements of the product's depth: three bf16 parts
//                   (24 bits) against ones, so that the scores come out as s - lse / scale. (Read by
//                   the threads instead, 128 values a step each, they took as much of shared memory's
//                   bandwidth as the products' operands, which take nearly all of it: 2,300 cycles
//                   a step.)
// The steps of all (sequence, key head, key pair) items form one list, and each SM takes an equal
// contiguous part of it: causal items are of any length, and one prompt is spread over the GPU. An
// item that spans CTAs leaves partial sums in the workspace, which reduce_kernel adds in the order
// of the rows, so that results do not depend on timing.
// Columns that a key does not count (rows before it or before the window, past the sequence's end)
// are selected away in the tiles that have any; a row there may hold anything.
//
// Bound: a step's operands take 1,152 cycles of shared memory (both of an N = 128 product come from
// there) and the Q tile that TMA writes there 256 more, its exponentials 1,024 of their unit, and what
// passes between warps is on the way from one to the other: 1,700 cycles a step measured. In front and
// behind stand the lookup of a CTA's part, its first tiles and the sums' merge, 9 us for any call. 4096
// tokens, 16 heads 37.1 us (0.93 PFLOP/s of the pairs seen), 8 ragged prompts 77.2; from the last 64 rows
// of each alone 12.9 and 23.9; a prompt of 100 9.4. Branches of masked tiles between the loads and the
// exponentials of unmasked ones cost 1 us of the first, 64-bit divisions and a binary search in the
// lookups 2. No gain: barriers of their own for the two tiles, three Q tiles, two warps that
// issue, all of a thread's columns loaded first.
#include "attn_tc.cuh"

namespace gdn {

namespace {

// Two fp32 products in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
      " mul.rn.f32x2 w, x, y;\n mov.b64 {%0, %1}, w;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Whether the phase with this parity is complete; does not wait.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t phase) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(phase)
      : "memory");
  return ok != 0;
}

constexpr int kTile = 128;        // keys of a tile, rows of a step
constexpr int kThreads = 19 * 32;
constexpr float kLog2e = 1.44269504088896340736f;

template <int D>
struct WeightsSmem {
  static constexpr int kBytesTile = kTile * D * 2;
  static constexpr int kStages = 2;                         // Q tiles
  static constexpr int kK = 0;                              // two pairs of K tiles
  static constexpr int kQ = 4 * kBytesTile;
  static constexpr int kLse = kQ + kStages * kBytesTile;    // [kStages][128 rows of 16], no swizzle
  static constexpr int kOnes = kLse + kStages * kTile * 32;
  static constexpr int kSums = kOnes + kTile * 32;          // [2][128], from the one half to the other
  static constexpr int kBars = kSums + 2 * kTile * 4;
  static constexpr int kBytes = kBars + 256 + 1024;         // + alignment of the tiles
};

// Step s uses the Q tile, the denominators and the score buffers s % 2: what it read is free, and
// its scores are there, when its products are complete (s_full).
struct WeightsBars {
  uint64_t k_full[2], k_empty[2], q_full[2], lse_full[2], s_full[2], s_empty[2];
  uint64_t sum_full[2], sum_empty[2], idle, never;
  uint32_t tmem;
};

// The workspace.
struct WeightsParts {
  int64_t* first;  // [N + 1] number of each sequence's first step
  int2* seq;       // [N] sanitized (first row, length)
  float* part;     // [2 * grid][256] an item's sums in a CTA: of its first item, of its last
};

// a / b of numbers that seldom need 64 bits, whose division takes several times as long.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// The last i in [0, count) with holds(i), which is true up to some i (and at 0); by a whole warp.
template <typename F>
__device__ __forceinline__ int last_of(int count, F holds) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  while (count > 1) {
    const int step = (count + 31) / 32;
    const bool yes = lane * step < count && (lane == 0 || holds(lo + lane * step));
    const int j = 31 - __clz(__ballot_sync(0xffffffffu, yes));
    lo += j * step;
    count = min(step, count - j * step);
  }
  return lo;
}

// Steps of a sequence: nt row tiles, of which the window begins in tile w.
struct Shape {
  int len, row0, nt, w;
  __device__ Shape(const AttnWeightsParams& p, int len_) : len(len_) {
    row0 = p.window > 0 && p.window < len ? len - p.window : 0;
    nt = (len + kTile - 1) / kTile;
    w = row0 / kTile;
  }
  __device__ int first_row_tile(int pair) const { return max(2 * pair, w); }
  // steps of one head in the pairs before `pair`
  __device__ int64_t before(int pair) const {
    const int k0 = (w + 1) / 2;
    if (pair <= k0) return (int64_t)pair * (nt - w);
    return (int64_t)k0 * (nt - w) + (int64_t)(pair - k0) * (nt - pair + 1 - k0);
  }
  __device__ int pairs() const { return (nt + 1) / 2; }
  // the pair that step u (of one key head, all its query heads) is in; by a whole warp
  __device__ int pair_of(int64_t u, int G) const {
    return last_of(pairs(), [&](int m) { return before(m) * G <= u; });
  }
};

// A place in the list of steps.
struct StepCursor {
  int n, hk, pair, rt, g;
  int base, end, next;  // rows of the sequence, and the next entry of cu_seqlens
  Shape shape;
  __device__ explicit StepCursor(const AttnWeightsParams& p) : shape(p, 0) {}
  __device__ int bound(const AttnWeightsParams& p, int i) const {
    return i <= p.N ? min(max(p.cu[i], 0), p.T) : p.T;
  }
  __device__ bool starts_item() const { return g == 0 && rt == shape.first_row_tile(pair); }
  // steps from here to the item's end
  __device__ uint32_t left(const AttnWeightsParams& p) const {
    return (uint32_t)(shape.nt - rt) * p.G - g;
  }
  __device__ void next_item(const AttnWeightsParams& p) {
    g = 0;
    if (++pair >= shape.pairs()) {
      pair = 0;
      if (++hk >= p.Hk) {
        hk = 0;
        do {
          if (++n >= p.N) return;
          base = end;
          end = max(base, next);
          next = bound(p, n + 2);
          shape = Shape(p, end - base);
        } while (shape.len == 0);
      }
    }
    rt = shape.first_row_tile(pair);
  }
  __device__ void advance(const AttnWeightsParams& p) {
    if (++g < p.G) return;
    g = 0;
    if (++rt >= shape.nt) next_item(p);
  }
};

__device__ __forceinline__ int64_t steps_of(const AttnWeightsParams& p, int len) {
  const Shape s(p, len);
  return s.before(s.pairs()) * p.G * p.Hk;
}

// The first of CTA blockIdx.x's steps and their number, found by a warp. The scribe writes what
// reduce_kernel needs.
__device__ __forceinline__ uint32_t find_steps(const AttnWeightsParams& p, const WeightsParts& w,
                                               StepCursor& at, bool scribe) {
  const int lane = threadIdx.x & 31;
  int64_t U = 0, u0 = -1, r = 0;
  uint32_t steps = 0;
  // The sequences 32 at a time, twice: for the number of steps, then for u0's sequence; a batch of
  // no more is looked at once.
#pragma unroll 1
  for (int n0 = 0, carry = 0;;) {
    const int n = n0 + lane;
    int b = 0, e = 0;
    if (n < p.N) {
      const int b_in = p.cu ? p.cu[n] : 0, e_in = p.cu ? p.cu[n + 1] : p.T;
      if (scribe && u0 < 0 && (b_in < 0 || e_in < b_in || e_in > p.T))
        set_status(p.status, GDN_DEV_BAD_CU_SEQLENS);
      b = min(max(b_in, 0), p.T);
      e = min(max(e_in, 0), p.T);
    }
    b = max(b, carry);  // raised to the largest entry before it
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, b, o);
      if (lane >= o) b = max(b, x);
    }
    e = n < p.N ? max(b, e) : b;
    const int64_t c = n < p.N ? steps_of(p, e - b) : 0;
    int64_t inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    const int64_t first = U + inc - c;
    const bool count = u0 < 0, last = n0 + 32 >= p.N;
    if (count && scribe && n < p.N) {
      w.first[n] = first;
      w.seq[n] = make_int2(b, e - b);
    }
    const int64_t after = U + __shfl_sync(0xffffffffu, inc, 31);
    if (count && last) {
      if (scribe && lane == 0) w.first[p.N] = after;
      const int64_t grid = min((int64_t)gridDim.x, after);
      if ((int64_t)blockIdx.x >= grid) return 0;
      u0 = quotient(after * blockIdx.x, grid);
      steps = (uint32_t)(quotient(after * (blockIdx.x + 1), grid) - u0);
    }
    if (!count || (last && p.N <= 32)) {
      const uint32_t hit = __ballot_sync(0xffffffffu, c > 0 && u0 >= first && u0 < first + c);
      if (hit) {
        const int src = __ffs(hit) - 1;
        at.n = n0 + src;
        at.base = __shfl_sync(0xffffffffu, b, src);
        at.end = __shfl_sync(0xffffffffu, e, src);
        r = u0 - __shfl_sync(0xffffffffu, first, src);
        break;
      }
    }
    U = last ? 0 : after;
    carry = last ? 0 : __shfl_sync(0xffffffffu, e, 31);
    n0 = last ? 0 : n0 + 32;
  }
  at.next = p.cu ? at.bound(p, at.n + 2) : p.T;
  at.shape = Shape(p, at.end - at.base);
  const int64_t head = at.shape.before(at.shape.pairs()) * p.G;
  at.hk = (int)quotient(r, head);
  r -= at.hk * head;
  at.pair = at.shape.pair_of(r, p.G);
  r -= at.shape.before(at.pair) * p.G;
  const int tile = (int)quotient(r, p.G);
  at.rt = at.shape.first_row_tile(at.pair) + tile;
  at.g = (int)(r - (int64_t)tile * p.G);
  return steps;
}

// Where the weight of key `key` of sequence n goes; null where its place does not exist.
__device__ __forceinline__ float* weight_at(const AttnWeightsParams& p, int n, int hk, int key) {
  if ((key >> p.page_shift) >= p.max_pages) {
    set_status(p.status, GDN_DEV_BAD_LENGTH);
    return nullptr;
  }
  const int page = p.table[(size_t)n * p.max_pages + (key >> p.page_shift)];
  if (page < 0 || page >= p.n_pages) {
    set_status(p.status, GDN_DEV_BAD_PAGE_TABLE);
    return nullptr;
  }
  return p.weights + ((((size_t)page * p.Hk + hk) << p.page_shift) + (key & (p.page - 1)));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
weights_tc_kernel(const AttnWeightsParams p, const WeightsParts parts,
                  const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k) {
  using S = WeightsSmem<D>;
  extern __shared__ char raw_smem[];
  char* smem = raw_smem + (-smem_u32(raw_smem) & 1023u);
  auto& B = *reinterpret_cast<WeightsBars*>(smem + S::kBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 17) {
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        for (uint64_t* one : {B.k_full, B.k_empty, B.q_full, B.lse_full, B.s_full}) mbar_init(one + i, 1);
        mbar_init(&B.s_empty[i], 16);
        mbar_init(&B.sum_full[i], 4);
        mbar_init(&B.sum_empty[i], 4);
      }
      mbar_init(&B.idle, 1);
      mbar_init(&B.never, 1);
      mbar_init_fence();
      prefetch_tmap(&tm_q);
      prefetch_tmap(&tm_k);
    }
    __syncwarp();
    tmem_alloc(&B.tmem, 512);
    tmem_relinquish();
  }
  // The operands of the denominators: element k of row r at (r / 8) 256 + (k / 8) 128 + (r % 8) 16 + 2 (k % 8)
  // bytes; the keys' side is three ones a row, the rows' side is written step by step.
  for (int i = threadIdx.x; i < 3 * kTile * 2; i += kThreads) {
    const bool ones = i >= 2 * kTile * 2 && (i >> 3 & 1) == 0;
    *reinterpret_cast<uint4*>(smem + S::kLse + i * 16) = ones ? make_uint4(0x3F803F80u, 0x3F80u, 0, 0)
                                                              : make_uint4(0, 0, 0, 0);
  }
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B.tmem;
  pdl_wait();
  pdl_release();
  StepCursor at(p);
  const uint32_t steps = find_steps(p, parts, at, blockIdx.x == 0 && warp == 0);
  Waiter wait(p.status, p.polls);
  // A warp gives up as one, at the next such point; up to it works on whatever is there.
  auto good = [&] {
    const bool ok = __all_sync(0xffffffffu, wait.ok());
    if (!ok) wait.limit = 0;
    return ok;
  };
  if (steps > 0 && warp < 16) {
    // ---------------------------------------------------------------- exponentials and sums
    const int X = warp >> 3, half = warp >> 2 & 1, of_tile = (warp & 3) * 32 + lane;
    float* other = reinterpret_cast<float*>(smem + S::kSums) + X * kTile + of_tile;
    const uint32_t t = tmem + ((uint32_t)((warp & 3) * 32) << 16) + X * 256 + half * 64;
    const float c = p.scale * kLog2e;
    const float2 c2 = make_float2(c, c);
    bool from_start = at.starts_item();
    uint32_t s = 0, items = 0;
    float v[2][16];
    bool loaded = false;  // v[0] is being loaded for step s
    for (uint32_t left = steps; left > 0;) {
      const Shape& q = at.shape;
      const int kt = 2 * at.pair + X, key = kt * kTile + of_tile;
      float sum = 0.f;
      bool ends = false;
      while (left > 0 && !ends) {
        float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};  // of a row tile's steps
        // Columns [lo, hi) of this half count for the key; [lo0, hi) for the warp's first key,
        // [lo1, hi) for its last.
        const int r0 = at.rt * kTile + half * 64;
        const int lo = max(key, q.row0) - r0, hi = at.rt >= kt && kt < q.nt ? q.len - r0 : INT_MIN;
        const int lo0 = max(key - lane, q.row0) - r0, lo1 = max(key - lane + 31, q.row0) - r0;
        auto all = [&](const float (&y)[16]) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 x = mul2(make_float2(y[2 * i], y[2 * i + 1]), c2);
            acc[i & 1] = add2(acc[i & 1], make_float2(ex2(x.x), ex2(x.y)));
          }
        };
        auto some = [&](const float (&y)[16], int c0) {
          if (c0 + 16 <= lo0 || c0 >= hi) return;
          if (c0 >= lo1 && c0 + 16 <= hi) return all(y);
          const uint32_t counts =
              (lo <= c0 ? 0xffffu : lo >= c0 + 16 ? 0u : 0xffffu << (lo - c0)) &
              (hi >= c0 + 16 ? 0xffffu : (1u << (hi - c0)) - 1);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float x = ex2(y[i] * c);
            float& a = i & 1 ? acc[i >> 1 & 1].y : acc[i >> 1 & 1].x;
            a += counts >> i & 1u ? x : 0.f;
          }
        };
        const uint32_t todo = min((uint32_t)(p.G - at.g), left), end = s + todo;
        auto step = [&](auto chunk) {
          const uint32_t b = s & 1;
          if (!loaded) {
            wait(&B.s_full[b], s >> 1);
            tc_fence_after();
            tmem_ld16(t + b * 128, v[0]);
          }
#pragma unroll
          for (int ch = 0; ch < 3; ++ch) {
            tmem_ld_wait();
            tmem_ld16(t + b * 128 + 16 * (ch + 1), v[(ch + 1) & 1]);
            chunk(v[ch & 1], 16 * ch);
          }
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&B.s_empty[b]);
          // The next step's first columns come while this one's last are worked on, where they are
          // there.
          loaded = s + 1 < steps &&
                   __all_sync(0xffffffffu, mbar_test(&B.s_full[b ^ 1], ((s + 1) >> 1) & 1));
          if (loaded) {
            tc_fence_after();
            tmem_ld16(t + (b ^ 1) * 128, v[0]);
          }
          chunk(v[1], 48);
        };
        // (all columns count: no branches between a step's loads and its exponentials)
        if (lo1 <= 0 && hi >= 64)
          for (; s < end; ++s) step([&](const float (&y)[16], int) { all(y); });
        else
          for (; s < end; ++s) step(some);
        sum += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
        left -= todo;
        at.g += (int)todo;
        if (at.g == p.G) {
          at.g = 0;
          ends = ++at.rt == q.nt;
        }
        if (!good()) break;
      }
      // The end of the item, or of the CTA's part of it.
      if (half == 1) {
        wait(&B.sum_empty[X], items + 1);
        *other = sum;
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.sum_full[X]);
      } else {
        wait(&B.sum_full[X], items);
        sum += *other;
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.sum_empty[X]);
        if (!ends || !from_start) {
          parts.part[(size_t)(2 * blockIdx.x + (items > 0)) * 256 + X * kTile + of_tile] = sum;
        } else if (key < q.len) {
          if (float* to = weight_at(p, at.n, at.hk, key)) *to = sum;
        }
      }
      if (!good()) break;
      ++items;
      from_start = true;
      if (ends) at.next_item(p);
    }
    tmem_ld_wait();  // (who gave up may have columns on the way)
  } else if (steps > 0 && warp == 16) {
    // ---------------------------------------------------------------- loads
    if (lane == 0) {
      uint32_t items = 0, in_item = 0, s = 0;  // in_item: steps to come of the item
      for (; s < steps; ++s, --in_item, at.advance(p)) {
        const uint32_t b = s & 1;
        if (in_item == 0) {
          const uint32_t k = items & 1;
          in_item = at.left(p);
          wait(&B.k_empty[k], (items >> 1) + 1);
          if (!wait.ok()) break;
          const bool two = 2 * at.pair + 1 < at.shape.nt;
          mbar_expect_tx(&B.k_full[k], S::kBytesTile * (two ? 2 : 1));
          for (int x = 0; x < (two ? 2 : 1); ++x)
            for (int d = 0; d < D; d += 64)
              tma_load_3d(smem + S::kK + (2 * k + x) * S::kBytesTile + d * 256, &tm_k, d, at.hk,
                          at.base + (2 * at.pair + x) * kTile, &B.k_full[k]);
          ++items;
        }
        wait(&B.s_full[b], (s >> 1) + 1);
        if (!wait.ok()) break;
        mbar_expect_tx(&B.q_full[b], S::kBytesTile);
        for (int d = 0; d < D; d += 64)
          tma_load_3d(smem + S::kQ + b * S::kBytesTile + d * 256, &tm_q, d, at.hk * p.G + at.g,
                      at.base + at.rt * kTile, &B.q_full[b]);
      }
      // Copies in flight end before the CTA does (all have been waited for already, unless someone
      // gave up).
      for (uint32_t i = 0; i < 2 && i < items; ++i)
        mbar_wait(&B.k_full[i], ((items - 1 - i) / 2) & 1, kAttnPolls);
      for (uint32_t i = 0; i < 2 && i < s; ++i)
        mbar_wait(&B.q_full[i], ((s - 1 - i) / 2) & 1, kAttnPolls);
    }
  } else if (steps > 0 && warp == 17) {
    // ---------------------------------------------------------------- products
    constexpr uint32_t kId = idesc_bf16_f32(128, kTile), kT = S::kBytesTile >> 4;
    constexpr uint32_t kHi = (1u << 14) | (2u << 29) | (1024 >> 4);
    constexpr uint32_t kFlat = (1u << 14) | (256 >> 4);  // no swizzle
    const uint32_t k_lo = uniform((uint32_t)sdesc_sw128(smem_addr(smem + S::kK), 16, 1024));
    const uint32_t q_lo = uniform((uint32_t)sdesc_sw128(smem_addr(smem + S::kQ), 16, 1024));
    const uint32_t ones_lo = uniform((uint32_t)sdesc_kmajor(smem_addr(smem + S::kOnes), 128, 256));
    const uint32_t lse_lo = uniform((uint32_t)sdesc_kmajor(smem_addr(smem + S::kLse), 128, 256));
    const uint32_t el = elect_one(), tm = uniform(tmem);
    // Straight-line, two steps at a time, so that operands are constants from uniform registers: with
    // the buffers as variables a step's issue took 1,300 cycles. Each wait costs about 100 even
    // where it need not, each commit 130: so one of each for both tiles.
    uint32_t left = steps, items = 0, in_item = 0, k_pair = k_lo;
    for (uint32_t turn = 0; left > 0; ++turn) {
#pragma unroll
      for (uint32_t b = 0; b < 2; ++b) {
        if (left == 0) break;
        if (in_item == 0) {
          in_item = at.left(p);
          at.next_item(p);
          wait(&B.k_full[items & 1], items >> 1);
          k_pair = uniform(k_lo + (items & 1) * 2 * kT);
        }
        wait(&B.q_full[b], turn);
        wait(&B.lse_full[b], turn);
        wait(&B.s_empty[b], turn + 1);
        if (p.stall && turn * 2 + b + 1 == p.stall) wait(&B.never, 0);  // testing hook
        tc_fence_after();
#pragma unroll
        for (uint32_t x = 0; x < 2; ++x) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const uint32_t off = (i >> 2) * (kTile * 128 >> 4) + (i & 3) * 2;
            mma_ss(el, tm + x * 256 + b * 128, k_pair + x * kT + off, kHi, q_lo + b * kT + off, kHi, kId,
                   i > 0);
          }
          mma_ss(el, tm + x * 256 + b * 128, ones_lo, kFlat, lse_lo + b * (kTile * 32 >> 4), kFlat, kId, 1);
        }
        mma_commit(el, &B.s_full[b]);
        if (--in_item == 0) {
          mma_commit(el, &B.k_empty[items & 1]);
          ++items;
        }
        --left;
      }
      if (!good()) break;
    }
    // Nothing that this warp issued is still running when TMEM is freed.
    mma_commit(el, &B.idle);
    if (!mbar_wait(&B.idle, 0, kAttnPolls)) set_status(p.status, GDN_DEV_TIMEOUT);
  } else if (steps > 0 && warp == 18) {
    // ---------------------------------------------------------------- the rows' denominators
    const float down = -1.0f / p.scale;
    float v[2][4];  // of the next two steps
    uint32_t fetched = 0;
    auto fetch = [&](float (&y)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = at.rt * kTile + i * 32 + lane;
        y[i] = 0.f;
        if (fetched < steps && row < at.shape.len)
          y[i] = p.lse[(size_t)(at.base + row) * p.H + at.hk * p.G + at.g];
      }
      if (fetched++ < steps) at.advance(p);
    };
    fetch(v[0]);
    fetch(v[1]);
    uint32_t left = steps;
    for (uint32_t turn = 0; left > 0; ++turn) {
#pragma unroll
      for (uint32_t b = 0; b < 2; ++b) {
        if (left == 0) break;
        wait(&B.s_full[b], turn + 1);
        if (!good()) {
          left = 0;
          break;
        }
        --left;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = i * 32 + lane;
          const float x = v[b][i] * down;
          const float hi = __bfloat162float(__float2bfloat16_rn(x));
          const float y = isfinite(hi) ? x - hi : 0.f, mid = __bfloat162float(__float2bfloat16_rn(y));
          *reinterpret_cast<uint4*>(smem + S::kLse + b * kTile * 32 + (r >> 3) * 256 + (r & 7) * 16) =
              make_uint4(pack_bf16(hi, mid), pack_bf16(y - mid, 0.f), 0, 0);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.lse_full[b]);
        fetch(v[b]);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 17) tmem_dealloc(tmem, 512);
}

// The sums of the items that span CTAs: block i those of the item that the end of CTA i's part cuts,
// if it began there.
__global__ void __launch_bounds__(256) reduce_kernel(const AttnWeightsParams p, const WeightsParts w) {
  pdl_wait();
  const int64_t U = w.first[p.N], grid = min((int64_t)gridDim.x + 1, U);
  const int64_t cta = blockIdx.x;
  if (cta + 1 >= grid) return;
  const int64_t u0 = quotient(U * cta, grid), cut = quotient(U * (cta + 1), grid);
  // the last sequence that begins at or before the cut
  const int n = last_of(p.N, [&](int m) { return w.first[m] <= cut; });
  const Shape s(p, w.seq[n].y);
  const int64_t head = s.before(s.pairs()) * p.G, r = cut - w.first[n];
  const int hk = (int)quotient(r, head), pair = s.pair_of(r - hk * head, p.G);
  const int64_t first = w.first[n] + hk * head + s.before(pair) * p.G;
  const int64_t last = w.first[n] + hk * head + s.before(pair + 1) * p.G;
  if (first >= cut || first < u0) return;
  // The CTAs up to the one with the item's last step (U i / grid < last), eight parts at a time.
  const int64_t end = quotient(last * grid - 1, U);
  float sum = w.part[(2 * cta + (first == u0 ? 0 : 1)) * 256 + threadIdx.x];
  for (int64_t i = cta + 1; i <= end; i += 8) {
    float x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = i + k <= end ? w.part[2 * (i + k) * 256 + threadIdx.x] : 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += x[k];
  }
  const int key = pair * 256 + threadIdx.x;
  if (key >= s.len) return;
  if (float* to = weight_at(p, n, hk, key)) *to = sum;
}

struct WeightsLayout {
  size_t first, seq, part, total;
};
WeightsLayout layout(int N) {
  WeightsLayout L{};
  L.seq = align_up(sizeof(int64_t) * ((size_t)N + 1), 256);
  L.part = align_up(L.seq + sizeof(int2) * N, 256);
  L.total = L.part + sizeof(float) * 512 * num_sms();
  return L;
}

template <int D>
bool launch(const AttnWeightsParams& p, void* workspace, cudaStream_t s) {
  const WeightsLayout L = layout(p.N);
  char* ws = static_cast<char*>(workspace);
  const WeightsParts w{reinterpret_cast<int64_t*>(ws), reinterpret_cast<int2*>(ws + L.seq),
                       reinterpret_cast<float*>(ws + L.part)};
  const uint32_t box[3] = {64, 1, kTile};
  const uint64_t dim_q[3] = {D, (uint64_t)p.H, (uint64_t)p.T}, str_q[2] = {D * 2, (uint64_t)p.H * D * 2};
  const uint64_t dim_k[3] = {D, (uint64_t)p.Hk, (uint64_t)p.T}, str_k[2] = {D * 2, (uint64_t)p.Hk * D * 2};
  CUtensorMap tm_q, tm_k;
  if (!encode_bf16_tmap(&tm_q, p.q, 3, dim_q, str_q, box) ||
      !encode_bf16_tmap(&tm_k, p.k, 3, dim_k, str_k, box))
    return false;
  constexpr int smem = WeightsSmem<D>::kBytes;
  ensure_smem_limit(reinterpret_cast<const void*>(weights_tc_kernel<D>), smem);
  const int grid = num_sms();
  if (launch_pdl(weights_tc_kernel<D>, dim3(grid), dim3(kThreads), smem, s, p, w, tm_q, tm_k) !=
      cudaSuccess)
    return false;
  return grid == 1 ||
         launch_pdl(reduce_kernel, dim3(grid - 1), dim3(256), 0, s, p, w) == cudaSuccess;
}

}  // namespace

size_t attn_prefill_weights_workspace(int T, int N, int H, int Hk, int D) { return layout(N).total; }

bool launch_attn_prefill_weights(const AttnWeightsParams& p, void* workspace, cudaStream_t s) {
  return p.D == 128 ? launch<128>(p, workspace, s) : launch<64>(p, workspace, s);
}

}  // namespace gdn
