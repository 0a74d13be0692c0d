// Decode attention over the paged cache in 8 bits: as k_attn_decode.cu (the same list of units,
// equal parts of it, merge of the parts), with half the bytes to read.
//
// Mathematics: with the scales a_j of the keys and b_j of the values (of 16 tokens each), q' = 2^-x q
// the row's queries in fp16 (x: by the row's largest element), e4m3 keys k and values v in fp16,
//   t_j = c 2^x a_j (q' . k_j),  c = scale * log2(e);   l = sum_j 2^(t_j - r),
//   o = sum_j 2^(t_j + log2 b_j - r') v_j;              out = 2^(r' - r) o / l.
// r' is set to 2^7 below the largest b_j 2^(t_j) so far, and again when outgrown by 2^8; r to the
// largest t_j (of the lane's own keys), and again when outgrown by 2^40. With a reference of their
// own the weights of the second product lie between 2^7 and 2^15 where they are largest, whatever
// the scales are, and keep fp16's 11 bits down to 2^-21 of that. Both products are fp16 MMAs
// (m16n8k16), exact but for their fp32 sums: e4m3 is a part of fp16.
//
// Keys and values are the MMAs' 16-row operand and the queries their 8 columns (S^T = K Q^T, then
// O^T = V^T P^T): a decode step seldom has more than 8 rows for a key head, and with the queries as
// rows half of each MMA, and of each lane's registers and exponentials, was for nothing.
//
// Bound: reading; to get there, the instructions that a key takes, of which the conversions (one a
// pair of elements) are the first part. 64 sequences of up to 8192 keys: bf16's cp.async and 16-key
// blocks 143 us; 32 keys at a time, so that the ring's bookkeeping serves twice as many, 120; three
// CTAs an SM in place of two 109; e4m3 MMAs on split queries and weights, which sm_103a makes of
// fp16 ones, 104. The blocks come by TMA, two copies issued by one lane, laid out for ldmatrix by the
// tensor map's swizzle. Rows of a block past the sequence's end come along: their scores are masked,
// and their values, which a weight of 0 would not remove where they are NaN, are made 0 in the
// registers (the second half of a block that is past the end is not looked at: its page is not loaded).
// Measured (GB300): 64 sequences of up to 8192 keys 89 us (6.0 TB/s, the second kernel included), one
// of 8191 keys 10.7 us, two of 20 and 40 keys 6.5 us.
#include "attn_decode.cuh"
#include "e4m3.cuh"

namespace gdn {

namespace {

constexpr int kBlk = 32;    // keys of a warp's block
constexpr int kUnit = kWarps * kBlk;
constexpr float kApart = 40.f;  // how far the denominators' reference may fall behind

template <int D, int RN>
struct Smem8 {
  static constexpr int kHalf = kBlk * D;     // a K or V block
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kScales = kWarps * kStages * kStage;                // float4 a stage
  static constexpr int kMerge = kScales + kWarps * kStages * 16;
  static constexpr int kMl = kMerge + (RN == 3 ? 3 : 1) * kMergeBytes;
  static constexpr int kBars = kMl + kWarps * RN * 8 * 8;
  static constexpr int kBytes = kBars + (kWarps * kStages + 1) * 8 + 1024;  // + alignment
};

// 16-byte piece c of row r of D bytes, as TMA's swizzle of rows of that size has it.
template <int D>
__device__ __forceinline__ uint32_t piece(int r, int c) {
  if constexpr (D == 64) return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
  return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
}

__device__ __forceinline__ uint32_t max_finite(uint32_t m, uint32_t bits) {
  bits &= 0x7FFFFFFFu;
  return max(m, bits < 0x7F800000u ? bits : 0u);
}

// Bytes of e4m3: the top bits of those that are NaN; the bytes with 0 in the place of NaN.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t x) {
  return ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}
__device__ __forceinline__ uint32_t without_nan(uint32_t x) {
  return x & ~((nan_bytes(x) >> 7) * 0xFFu);
}

__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap* tm, int row, int z,
                                          uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(0), "r"(row), "r"(z), "r"(bar), "l"(policy)
      : "memory");
}

// RN tiles of 8 query rows a warp, WM warps for a pair's rows.
template <int D, int RN, int WM, bool kScores>
__global__ void __launch_bounds__(kWarps * 32, RN == 3 ? 2 : kDecode8Ctas)
decode8_kernel(const AttnParams p, const DecodeParts w, const __grid_constant__ CUtensorMap tm_k,
               const __grid_constant__ CUtensorMap tm_v) {
  using S = Smem8<D, RN>;
  constexpr int kSt = S::kStages, E = D / 16, TM = 8 * RN;
  extern __shared__ char raw_smem[];
  char* smem = raw_smem + (-smem_u32(raw_smem) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int kg = warp / WM, mt = warp % WM;  // key group, row tile
  const int R = p.nq * p.G;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBars);  // [kWarps][kSt], one for the test
  if (tid == 0) {
    for (int i = 0; i <= kWarps * kSt; ++i) mbar_init(bars + i, 1);
    mbar_init_fence();
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  __syncthreads();
  pdl_wait();
  pdl_release();
  int u1;
  Cursor<kUnit> cur;
  if (!find_units(p, w, cur, u1)) return;
  Cursor<kUnit> ahead = cur;  // what is loaded next

  // ---- loads: this warp's block of unit `ahead`, into ring place `st`. Even and odd lanes hold the
  // pages of its two halves.
  const uint32_t ring = smem_u32(smem) + warp * kSt * S::kStage;
  auto page_of = [&]() -> int {
    const int key = ahead.key() + warp * kBlk + (lane & 1) * kBlock8;
    if (key >= ahead.len) return -1;
    return p.table[(size_t)(key < p.common ? 0 : ahead.n) * p.max_pages + (key >> p.page_shift)];
  };
  int page = page_of();
  uint64_t once;  // read once: leaves L2 first
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
  Waiter wait(p.status, p.polls);
  uint32_t phases = 0;  // bit b * kSt + st: of the next wait for the group's block b
  uint32_t loading = 0;  // bit st: this warp's block is being loaded
  auto load_next = [&](int st) {
    if (ahead.u < u1) {
      const int key = ahead.key() + warp * kBlk;
      if (key < ahead.len && wait.ok()) {
        const bool ok = page >= 0 && page < p.n_pages;
        const bool second = key + kBlock8 < ahead.len;
        const bool there = (lane & 1) == 0 || second;
        if (!ok && there && lane < 2) set_status(p.status, GDN_DEV_BAD_PAGE_TABLE);
        // (a page that does not exist: rows outside the tensor, which are zeros, and scales of 0)
        const int z = ok ? page * p.Hk + ahead.hk : max(p.n_pages * p.Hk, 1);
        const int z1 = __shfl_sync(0xffffffffu, z, 1);
        const int row = key & (p.page - 1);
        if (lane < 4) {
          const float* x = lane < 2 ? p.ks : p.vs;
          const bool get = ok && there;
          const size_t at = (((size_t)z << p.page_shift) + row) / kBlock8;
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(
                           smem_u32(smem) + S::kScales + (warp * kSt + st) * 16 + lane * 4),
                       "l"(get ? x + at + (p.page > kBlock8 ? lane & 1 : 0) : x), "r"(get ? 4 : 0));
        }
        if (lane == 0) {
          const uint32_t bar = smem_u32(bars + warp * kSt + st), dst = ring + st * S::kStage;
          const int boxes = p.page > kBlock8 || !second ? 1 : 2;
          const uint32_t bytes = p.page > kBlock8 ? S::kStage : boxes * S::kStage / 2;
          mbar_expect_tx(bars + warp * kSt + st, bytes);
          load_rows(dst, &tm_k, row, z, bar, once);
          load_rows(dst + S::kHalf, &tm_v, row, z, bar, once);
          if (boxes == 2) {
            load_rows(dst + S::kHalf / 2, &tm_k, row, z1, bar, once);
            load_rows(dst + S::kHalf / 2 * 3, &tm_v, row, z1, bar, once);
          }
        }
        loading |= 1u << st;
      }
      ahead.next(p);
      if (ahead.u < u1) page = page_of();  // used a step later
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kSt - 1; ++i) load_next(i);

  const float c = p.scale * 1.44269504088896340736f;
  const int g = lane >> 2, cq = (lane & 3) * 2;
  const int row0 = mt * TM + cq;  // this thread's rows in the sums: row0 + 8 n + x
  uint32_t qf[RN][E][2];          // row mt * TM + 8 n + g
  float qc[RN][2];                // what a row's products are multiplied with
  float o[RN][E][4];              // columns 16 e + 2 g + (i >> 1), row x = i & 1
  float refv[RN][2], ref[RN][2], l[RN][2];  // ref and l: of this thread's keys alone
  int lim_off[RN][2];  // keys past len that the row does not see: lim = len - lim_off
#pragma unroll
  for (int n = 0; n < RN; ++n)
#pragma unroll
    for (int x = 0; x < 2; ++x) lim_off[n][x] = p.nq - 1 - min((row0 + 8 * n + x) / p.G, p.nq - 1);
  // This warp's rows of the queries of the pair at `cur`, in fp16: times a power of two, by the
  // row's largest element, that puts it below 2^15; elements are then exact down to 2^-29 of it, and
  // below that off by 2^-40 of it at most (in rows whose largest is below 2^-86, off by 2^-125). Row k of the MMAs' operand is element 4 (k / 2) + k % 2 of
  // 16, row 8 + k the one 2 further on: so a lane's 4 bytes of a key are two of its operands.
  auto load_q = [&] {
#pragma unroll
    for (int n = 0; n < RN; ++n) {
      const int r = mt * TM + 8 * n + g;
      const __nv_bfloat16* q =
          p.q + ((size_t)(cur.n * p.nq + r / p.G) * p.H + cur.hk * p.G + r % p.G) * D + 2 * cq;
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint2 y = r < R ? *reinterpret_cast<const uint2*>(q + e * 16) : make_uint2(0, 0);
        qf[n][e][0] = y.x;
        qf[n][e][1] = y.y;
        top = max_finite(max_finite(max_finite(max_finite(top, y.x << 16), y.x & 0xFFFF0000u), y.y << 16),
                         y.y & 0xFFFF0000u);
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int ex = max((int)(top >> 23) - 127 - 14, -100);
      const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
      const float up = c * __uint_as_float((uint32_t)(127 + ex) << 23);
      qc[n][0] = __shfl_sync(0xffffffffu, up, cq * 4);
      qc[n][1] = __shfl_sync(0xffffffffu, up, cq * 4 + 4);
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          qf[n][e][i] = pack_f16(__uint_as_float(qf[n][e][i] << 16) * down,
                                 __uint_as_float(qf[n][e][i] & 0xFFFF0000u) * down);
    }
  };
  auto reset = [&] {
#pragma unroll
    for (int n = 0; n < RN; ++n) {
      ref[n][0] = ref[n][1] = refv[n][0] = refv[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[n][e][0] = o[n][e][1] = o[n][e][2] = o[n][e][3] = 0.f;
    }
  };
  load_q();
  reset();
  int seg_chunk = cur.chunk;  // first chunk of this pair in this CTA
  bool seg_first = true;      // the pair's part begins at the CTA's first unit
  int st = 0;
  uint32_t steps = 0;

  while (cur.u < u1) {
    load_next((st + kSt - 1) % kSt);
    cp_async_wait<kSt - 1>();
    if constexpr (WM == 1) __syncwarp();
    else named_sync(1 + kg, WM * 32);
    if (p.stall && ++steps == p.stall) wait(bars + kWarps * kSt, 0);  // testing hook: never arrives
#pragma unroll 1
    for (int b = 0; b < WM; ++b) {
      const int blk = kg * WM + b, key0 = cur.key() + blk * kBlk;
      if (key0 >= cur.len) break;
      const uint32_t bit = b * kSt + st;
      wait(bars + blk * kSt + st, phases >> bit);
      if (!__all_sync(0xffffffffu, wait.ok())) wait.limit = 0;  // a warp gives up as one
      if (wait.ok()) {
        phases ^= 1u << bit;
        if (blk == warp) loading &= ~(1u << st);
      }
      const uint32_t kb = smem_u32(smem) + (blk * kSt + st) * S::kStage, vb = kb + S::kHalf;
      // scores of the keys 16 h + g + 8 (i >> 1) and the rows row0 + 8 n + (i & 1)
      float s[RN][2][4] = {};
#pragma unroll
      for (int e = 0; e < E; e += 2)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t f[4];
          ldsm_x4_addr(f, kb + piece<D>(h * 16 + (lane & 15), e + (lane >> 4)));
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            uint32_t a[4];
            e4m3x4_to_f16x4(f[2 * z], a[0], a[2]);
            e4m3x4_to_f16x4(f[2 * z + 1], a[1], a[3]);
#pragma unroll
            for (int n = 0; n < RN; ++n) mma_f16(s[n][h], a, qf[n][e + z][0], qf[n][e + z][1]);
          }
        }
      const float4 scale = *reinterpret_cast<const float4*>(smem + S::kScales + (blk * kSt + st) * 16);
      const float lv[2] = {log2f(scale.z), log2f(scale.w)};
      const bool part = key0 + kBlk > cur.len - (p.nq - 1);  // some row does not see all
      bool any = false;  // a reference is outgrown
      float top[RN][2], mine[RN][2];
#pragma unroll
      for (int n = 0; n < RN; ++n) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[n][h][i] *= qc[n][i & 1] * (h ? scale.y : scale.x);
        if (part) {  // (after the scales, which may be 0)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (key0 + h * 16 + (i >> 1) * 8 + g >= cur.len - lim_off[n][i & 1]) s[n][h][i] = -INFINITY;
        }
        if constexpr (kScores) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (row0 + 8 * n + x >= R) continue;
            float* to = w.scores +
                        ((size_t)(cur.n * p.Hk + cur.hk) * R + row0 + 8 * n + x) * w.keys + key0 + g;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (h && key0 + kBlock8 >= cur.len) continue;  // (it may lie past the table)
              to[h * 16] = s[n][h][x];
              to[h * 16 + 8] = s[n][h][2 + x];
            }
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float m0 = fmaxf(s[n][0][x], s[n][0][2 + x]), m1 = fmaxf(s[n][1][x], s[n][1][2 + x]);
          // (a key that is not seen weighs nothing, whatever its block's scale is)
          top[n][x] = fmaxf(m0 == -INFINITY ? m0 : m0 + lv[0], m1 == -INFINITY ? m1 : m1 + lv[1]) - 7.f;
          mine[n][x] = fmaxf(m0, m1);
          any |= (top[n][x] > refv[n][x] && top[n][x] - refv[n][x] > kGrow) ||
                 (mine[n][x] > ref[n][x] && mine[n][x] - ref[n][x] > kApart);
        }
      }
      if (__any_sync(0xffffffffu, any)) {
#pragma unroll
        for (int n = 0; n < RN; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float m = top[n][x];
#pragma unroll
            for (int y = 4; y < 32; y <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, y));
            if (m > refv[n][x] && m - refv[n][x] > kGrow) {
              const float f = ex2(refv[n][x] - m);
              refv[n][x] = m;
#pragma unroll
              for (int e = 0; e < E; ++e) {
                o[n][e][x] *= f;
                o[n][e][2 + x] *= f;
              }
            }
            if (mine[n][x] > ref[n][x] && mine[n][x] - ref[n][x] > kApart) {
              l[n][x] *= ex2(ref[n][x] - mine[n][x]);
              ref[n][x] = mine[n][x];
            }
          }
      }
      // A value scale that is not finite, in a half that some row may not see: its weight there is 0
      // and not that scale's (-inf + NaN, -inf + inf). A branch, as seldom taken.
      const bool odd = part && !(fmaxf(lv[0], lv[1]) < INFINITY && lv[0] == lv[0] && lv[1] == lv[1]);
      uint32_t pf[RN][2][2];  // the weights as the MMAs' operand: [half][8 keys]
#pragma unroll
      for (int n = 0; n < RN; ++n) {
        float r[2], v[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {  // (-inf: nothing seen so far)
          r[x] = ref[n][x] == -INFINITY ? 0.f : ref[n][x];
          v[x] = refv[n][x] == -INFINITY ? 0.f : refv[n][x];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            l[n][i & 1] += ex2(s[n][h][i] - r[i & 1]);
            y[i] = ex2(s[n][h][i] + (lv[h] - v[i & 1]));
          }
          if (odd) {
            asm volatile("");
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (s[n][h][i] == -INFINITY) y[i] = 0.f;
          }
          pf[n][h][0] = transpose_8x8(pack_f16(y[0], y[1]));
          pf[n][h][1] = transpose_8x8(pack_f16(y[2], y[3]));
        }
      }
      // A value that a weight of 0 would not remove: in any key of the halves that are used (the
      // second one may not have been loaded), and in one that some row sees.
      const int halves = key0 + kBlock8 < cur.len ? 2 : 1;
      bool bad = false, seen = false;
      if (part) {
#pragma unroll 4
        for (int i = lane; i < halves * (S::kHalf / 32); i += 32) {
          const uint4 x = *reinterpret_cast<const uint4*>(smem + (vb - smem_u32(smem)) + i * 16);
          const bool nan = (nan_bytes(x.x) | nan_bytes(x.y) | nan_bytes(x.z) | nan_bytes(x.w)) != 0;
          bad |= nan;
          seen |= nan && key0 + i / (D / 16) < cur.len;
        }
        bad = __any_sync(0xffffffffu, bad);
        seen = __any_sync(0xffffffffu, seen);
      }
      // Pairs of elements of 8 keys come transposed as one matrix: the even elements are the
      // operand's first 8 rows, the odd ones its last 8.
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h >= halves) break;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          uint32_t f[4];
          ldsm_x4_t_addr(f, vb + piece<D>(h * 16 + (lane & 15), e + (lane >> 4)));
          if (bad) {
            asm volatile("");  // a branch: as selects this is a third of the loop's instructions
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = without_nan(f[i]);
          }
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            uint32_t a[4];
            e4m3x4_to_f16x4(__byte_perm(f[2 * z], 0, 0x3120), a[0], a[1]);
            e4m3x4_to_f16x4(__byte_perm(f[2 * z + 1], 0, 0x3120), a[2], a[3]);
#pragma unroll
            for (int n = 0; n < RN; ++n) mma_f16(o[n][e + z], a, pf[n][h][0], pf[n][h][1]);
          }
        }
      }
      if (seen) {  // NaN to the rows that see it, whatever its weight
#pragma unroll 1
        for (int j = 0; j < kBlk && key0 + j < cur.len; ++j) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const uint32_t nan = nan_bytes(*reinterpret_cast<const uint16_t*>(
                smem + (vb - smem_u32(smem)) + piece<D>(j, e) + g * 2));
#pragma unroll
            for (int n = 0; n < RN; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if ((nan >> (i >> 1) * 8 & 0x80u) && key0 + j < cur.len - lim_off[n][i & 1]) o[n][e][i] = NAN;
          }
        }
      }
    }
    if constexpr (WM == 1) __syncwarp();
    else named_sync(1 + kg, WM * 32);
    st = (st + 1) % kSt;

    const Cursor<kUnit> was = cur;
    cur.next(p);
    if (cur.u < u1 && cur.n == was.n && cur.hk == was.hk) continue;

    // ---- the end of a pair's part
    if (cur.u < u1) load_q();  // the next pair's queries arrive meanwhile
    const bool whole = seg_chunk == cur.kOwn && was.chunk == was.chunks - 1;
    float2* ml = reinterpret_cast<float2*>(smem + S::kMl);
    constexpr int kCols = RN == 2 ? 32 : 64;
    finish_part<D, WM, TM, kCols, kScores, 1>(
        p, w, reinterpret_cast<float*>(smem + S::kMerge), ml,
        [&] {
#pragma unroll
          for (int n = 0; n < RN; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float m = ref[n][x];
#pragma unroll
              for (int z = 4; z < 32; z <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, z));
              float y = l[n][x];
              if (ref[n][x] != -INFINITY) y *= ex2(ref[n][x] - m);
#pragma unroll
              for (int z = 4; z < 32; z <<= 1) y += __shfl_xor_sync(0xffffffffu, y, z);
              if (g == 0) ml[kg * TM * WM + row0 + 8 * n + x] = make_float2(m, y);
            }
        },
        [&](float* buf, int q, auto most) {
#pragma unroll
          for (int n = 0; n < RN; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int row = row0 + 8 * n + x;
              const float m = most(row);
              // in two factors: a scale may take their product past fp32 where the sum is not
              const float f = m == -INFINITY ? 0.f : ex2(0.5f * (refv[n][x] - m));
#pragma unroll
              for (int e = 0; e < kCols / 16; ++e) {
                const float* y = o[n][kCols / 16 * q + e];
                *reinterpret_cast<float2*>(buf + (kg * TM * WM + row) * kCols +
                                           ((e * 16 + g * 2) ^ ((row & 3) * 8))) =
                    make_float2(y[x] * f * f, y[2 + x] * f * f);
              }
            }
        },
        was.n, was.hk, whole, 2 * blockIdx.x + (seg_first ? 0 : 1));
    __syncthreads();
    reset();
    seg_chunk = cur.chunk;
    seg_first = false;
  }
  // After a wait that ran out, copies may still be under way.
  if (!wait.ok()) {
    Waiter rest(p.status, kAttnPolls);
    for (int i = 0; i < kSt; ++i)
      if (loading >> i & 1u) rest(bars + warp * kSt + i, phases >> (mt * kSt + i));
  }
}

template <int D, bool kScores>
bool launch(AttnParams p, void* workspace, cudaStream_t s) {
  const int64_t keys = (int64_t)p.max_pages * p.page;
  const DecodeLayout L = layout(p.T, p.N, p.H, p.Hk, D, kScores ? keys : 0, kDecode8Ctas);
  DecodeParts w = parts_of(L, workspace);
  p.shared = 0;
  // no more CTAs than units there can be
  const int64_t most = (int64_t)p.N * p.Hk * ((keys + kUnit - 1) / kUnit);
  const int R = p.nq * p.G;
  const bool by24 = (R > 16 && R <= 24) || (R > 32 && R <= 48);  // rows a warp, see below
  const int full = by24 ? L.grid / kDecode8Ctas * 2 : L.grid;
  w.grid = (int)(most < full ? (most > 0 ? most : 1) : full);
  if (kScores) {
    w.lse2 = reinterpret_cast<float*>(static_cast<char*>(workspace) + L.lse2);
    w.scores = reinterpret_cast<float*>(static_cast<char*>(workspace) + L.scores);
    w.keys = keys;
  }
  // A box is as many rows of one page and key head as a block has, or a page of 16.
  const uint64_t rows = (uint64_t)p.n_pages * p.Hk;
  const uint64_t dim[3] = {D, (uint64_t)p.page, rows > 0 ? rows : 1};
  const uint64_t str[2] = {D, (uint64_t)p.page * D};
  const uint32_t box[3] = {D, (uint32_t)(p.page < kBlk ? p.page : kBlk), 1};
  CUtensorMap tm_k, tm_v;
  if (!encode_u8_tmap(&tm_k, p.k, 3, dim, str, box) || !encode_u8_tmap(&tm_v, p.v, 3, dim, str, box))
    return false;
  auto go = [&](auto kernel, int smem) {
    ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem);
    return launch_pdl(kernel, dim3(w.grid), dim3(kWarps * 32), smem, s, p, w, tm_k, tm_v) == cudaSuccess;
  };
  // (More than 16 rows: warps with 24 each where that leaves fewer rows empty, with the registers of
  // two CTAs an SM in place of three; else several with 16, which convert the same keys. 24 a warp and
  // 16, us, 64 sequences of 2000 to 4000 keys, 8 key heads: head size 128, 24 rows 147.4 and 164.0, 40 rows
  // 234.5 and 281.6; head size 64, 24 rows 108.0 and 115.3, 40 rows 177.2 and 197.2. Four of 4000 to 8000,
  // 4 key heads, head size 64, 40 rows: 22.7 and 23.9. One of 8000: head size 128, 40 rows 20.8 and 23.3;
  // head size 64, 24 rows 12.7 and 13.4, but 33 to 48 rows 17.6 to 17.9 and 16.5 to 17.4, the rule's one
  // point on the wrong side: which batches come next to it the host cannot see. One warp with 32
  // rows has too few registers for its sums: 96 sequences, 32 rows, 30 us and 52 with 407 to 814 keys
  // of head size 128, 86 and 162 with 4000 to 8000 of 64.)
  const bool ok = R <= 8    ? go(decode8_kernel<D, 1, 1, kScores>, Smem8<D, 1>::kBytes)
                  : R <= 16 ? go(decode8_kernel<D, 2, 1, kScores>, Smem8<D, 2>::kBytes)
                  : by24 && R <= 24 ? go(decode8_kernel<D, 3, 1, kScores>, Smem8<D, 3>::kBytes)
                  : R <= 32 ? go(decode8_kernel<D, 2, 2, kScores>, Smem8<D, 2>::kBytes)
                  : by24    ? go(decode8_kernel<D, 3, 2, kScores>, Smem8<D, 3>::kBytes)
                            : go(decode8_kernel<D, 2, 4, kScores>, Smem8<D, 2>::kBytes);
  return ok && launch_rest<D, kUnit, kScores>(p, w, s);
}

}  // namespace

bool launch_attn_decode8(const AttnParams& p, void* workspace, cudaStream_t s) {
  if (p.weights)
    return p.D == 128 ? launch<128, true>(p, workspace, s) : launch<64, true>(p, workspace, s);
  return p.D == 128 ? launch<128, false>(p, workspace, s) : launch<64, false>(p, workspace, s);
}

}  // namespace gdn
