// Decode attention over the paged cache: the last nq tokens of each sequence against all of
// its keys and values, R = nq * G <= 64 query rows per (sequence, key head).
//
// Bound: every key and value is read once from HBM for R rows, a few flops a byte, so the
// kernel is built around keeping reads in flight. The keys of all (sequence, key head) pairs
// are cut into units of 64; the units form one list, and the persistent CTAs (two per SM)
// take equal contiguous parts of it, so that any mix of lengths is balanced and one long
// sequence is spread over the whole GPU. Each warp copies 16-key blocks of K and V (one page
// each; 4 KB at D = 128) with cp.async through a ring of its own that runs across the ends
// of sequences, and multiplies with m16n8k16 MMAs: 16 rows are all that a decode step has,
// an eighth of a tcgen05 tile, and the MMAs take a few per cent of the time.
//
// Rows of a pair: WM warps hold 16 rows each and share their key blocks (a named barrier per
// ring step), 4 / WM groups of warps split the keys. At the end of a pair the groups' results
// are merged in shared memory; a pair that lies in one CTA is finished there, the parts of
// the others go to the workspace (fp32 sums, reference and denominator) and are merged in a
// fixed order by combine_kernel, so results do not depend on timing.
//
// Weights are 2^(c s - ref) with c = scale * log2(e) and ref a running maximum that is
// replaced when outgrown by 2^8, as in attn_tc.cuh; rounded to bf16 for the second product,
// summed in fp32 before that. Where the keys' weights are wanted as well, the second product takes the
// weights in two parts of 8 bits each (twice its MMAs), so that the output is as good as those weights
// are. 64 sequences of up to 4096 keys, bf16 outputs, 2-norm of the error against 64 bits: rounded 2.3e-3
// (87.0 us), in two parts 1.66e-3 (87.5 us), all of it the output's own rounding; 8 x 4 tokens 22.6 and 23.7.
//
// Measured (GB300): 64 sequences of up to 8192 keys 148.5 to 153 us (6.8 TB/s), one of 8191 keys
// 10.1 to 10.7 us, 64 behind 16384 shared keys 53 to 58 us; with weights, 64 of up to 4096 keys 88 us.
#include "attn_decode.cuh"

namespace gdn {

namespace {

constexpr int kUnit = 64;   // keys of a unit
constexpr int kBlk = 16;    // keys of a warp's block

template <int D>
struct DecodeSmem {
  static constexpr int kRow = D * 2;                 // bytes of a key
  static constexpr int kStage = 2 * kBlk * kRow;     // a K and a V block
  // 64 KB of ring per CTA, half of it in flight. More only makes every other read (a row of
  // the queries, a page number) wait longer in a saturated memory system: with 96 KB, 64
  // sequences of up to 8192 keys took 163.4 us, with 64 KB 159.0 us.
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kMerge = kWarps * kStages * kStage;
  static constexpr int kMl = kMerge + 2 * kMergeBytes;
  static constexpr int kBytes = kMl + kWarps * 16 * 8;
};

// 16-byte piece c of row r, spread over the banks for ldmatrix.
template <int D>
__device__ __forceinline__ uint32_t piece(int r, int c) {
  return (uint32_t)(r * D * 2 + ((c ^ (r & 7)) << 4));
}

// Two weights as a first part of 8 bits, cut, and a rest of 8 more: off by 2^-16 of the weight. Both
// parts of a weight that is not 0 are above 0 (by 2^-126, where there is no rest), so that an infinite
// value times them is that infinity.
__device__ __forceinline__ void split_weights(float x0, float x1, uint32_t& first, uint32_t& rest) {
  const uint32_t u0 = __float_as_uint(x0) & 0xFFFF0000u, u1 = __float_as_uint(x1) & 0xFFFF0000u;
  first = __byte_perm(u0, u1, 0x7632);
  auto left = [](float x, uint32_t u) { return fminf(fmaxf(x - __uint_as_float(u), 0x1p-126f), x); };
  rest = pack_bf16(left(x0, u0), left(x1, u1));
}

template <int D, int WM, bool kScores>
__global__ void __launch_bounds__(kWarps * 32, 2)
decode_kernel(const AttnParams p, const DecodeParts w) {
  using S = DecodeSmem<D>;
  constexpr int kSt = S::kStages, E = D / 16;
  extern __shared__ __align__(128) char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int kg = warp / WM, mt = warp % WM;  // key group, row tile
  const int R = p.nq * p.G;
  // With a prefix kernel before this one in the stream nothing of it is needed here, and it
  // has waited for what came before; this kernel then only ends after it.
  if (p.shared == 0) pdl_wait();
  pdl_release();

  int u1;
  Cursor<kUnit> cur;
  if (!find_units(p, w, cur, u1)) {
    pdl_wait();
    return;
  }
  Cursor<kUnit> ahead = cur;  // what is loaded next

  // ---- loads: this warp's block of unit `ahead`, into ring place `st`
  const uint32_t ring = smem_u32(smem) + warp * kSt * S::kStage;
  auto page_of = [&]() -> int {
    const int key = p.shared + ahead.key() + warp * kBlk;
    if (key >= ahead.len) return -1;
    return p.table[(size_t)(key < p.common ? 0 : ahead.n) * p.max_pages + (key >> p.page_shift)];
  };
  int page = page_of();
  // Keys and values are read once, so they leave L2 first: what stays is what is read again,
  // above all the prefix's parts (with 64 sequences behind a prefix, 73.7 -> 65.7 us).
  uint64_t once;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
  auto load_next = [&](int st) {
    if (ahead.u < u1) {
      const int key = p.shared + ahead.key() + warp * kBlk;
      if (key < ahead.len) {
        const bool ok = page >= 0 && page < p.n_pages;
        if (!ok && lane == 0) set_status(p.status, GDN_DEV_BAD_PAGE_TABLE);
        const size_t at = ((((size_t)(ok ? page : 0) * p.Hk + ahead.hk) << p.page_shift) +
                           (key & (p.page - 1))) * D;
        const int rows = ahead.len - key;  // rows past the end are not read, zeros stand for them
        const char* k = reinterpret_cast<const char*>(p.k + at);
        const char* v = reinterpret_cast<const char*>(p.v + at);
        const uint32_t dst = ring + st * S::kStage;
#pragma unroll
        for (int i = 0; i < kBlk * D / 8 / 32; ++i) {
          const int x = i * 32 + lane, r = x / (D / 8), c = x % (D / 8);
          const uint32_t n = ok && r < rows ? 16 : 0;
          asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;\n" ::"r"(
                           dst + piece<D>(r, c)),
                       "l"(n ? k + x * 16 : reinterpret_cast<const char*>(p.k)), "r"(n), "l"(once));
          asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;\n" ::"r"(
                           dst + kBlk * S::kRow + piece<D>(r, c)),
                       "l"(n ? v + x * 16 : reinterpret_cast<const char*>(p.v)), "r"(n), "l"(once));
        }
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
  const int row0 = mt * 16 + g;  // this thread's rows: row0, row0 + 8
  uint32_t qf[E][4];
  float o[2 * E][4], ref[2], l[2];
  int lim_off[2];  // keys past len that the row does not see: lim = len - lim_off
#pragma unroll
  for (int x = 0; x < 2; ++x) lim_off[x] = p.nq - 1 - min((row0 + 8 * x) / p.G, p.nq - 1);
  // This warp's rows of the queries of the pair at `cur`.
  auto load_q = [&] {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = row0 + 8 * x;
      const __nv_bfloat16* q =
          p.q + ((size_t)(cur.n * p.nq + r / p.G) * p.H + cur.hk * p.G + r % p.G) * D;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        qf[e][x] = r < R ? *reinterpret_cast<const uint32_t*>(q + e * 16 + cq) : 0u;
        qf[e][x + 2] = r < R ? *reinterpret_cast<const uint32_t*>(q + e * 16 + 8 + cq) : 0u;
      }
    }
  };
  auto reset = [&] {
    ref[0] = ref[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int e = 0; e < 2 * E; ++e) o[e][0] = o[e][1] = o[e][2] = o[e][3] = 0.f;
  };
  load_q();
  reset();
  int seg_chunk = cur.chunk;  // first chunk of this pair in this CTA
  bool seg_first = true;      // the pair's part begins at the CTA's first unit
  int st = 0;

  while (cur.u < u1) {
    load_next((st + kSt - 1) % kSt);
    cp_async_wait<kSt - 1>();
    if constexpr (WM == 1) __syncwarp();
    else named_sync(1 + kg, WM * 32);
#pragma unroll 1
    for (int b = 0; b < WM; ++b) {
      const int blk = kg * WM + b;
      const int key0 = p.shared + cur.key() + blk * kBlk;
      if (key0 >= cur.len) break;
      const uint32_t kb = smem_u32(smem) + (blk * kSt + st) * S::kStage;
      const uint32_t vb = kb + kBlk * S::kRow;
      float s[2][4] = {};
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int m = lane >> 3, r = (lane & 7) + (m >> 1) * 8;
        uint32_t f[4];
        ldsm_x4_addr(f, kb + piece<D>(r, 2 * e + (m & 1)));
        mma_bf16(s[0], qf[e], f[0], f[1]);
        mma_bf16(s[1], qf[e], f[2], f[3]);
      }
      const bool part = key0 + kBlk > cur.len - (p.nq - 1);  // some row does not see all
      if (part) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (key0 + t * 8 + cq + (x & 1) >= cur.len - lim_off[x >> 1]) s[t][x] = -INFINITY;
      }
      if constexpr (kScores) {
        float* to = w.scores + ((size_t)(cur.n * p.Hk + cur.hk) * R + row0) * w.keys + key0 + cq;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (row0 + 8 * x >= R) continue;
#pragma unroll
          for (int t = 0; t < 2; ++t)
            *reinterpret_cast<float2*>(to + 8 * x * w.keys + t * 8) =
                make_float2(s[t][2 * x] * c, s[t][2 * x + 1] * c);
        }
      }
      float mx[2] = {fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1])),
                     fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]))};
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 1));
        mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 2)) * c;
      }
      const bool grown0 = mx[0] > ref[0] && mx[0] - ref[0] > kGrow;
      const bool grown1 = mx[1] > ref[1] && mx[1] - ref[1] > kGrow;
      if (__any_sync(0xffffffffu, grown0 || grown1)) {
        const float f0 = grown0 ? ex2(ref[0] - mx[0]) : 1.f, f1 = grown1 ? ex2(ref[1] - mx[1]) : 1.f;
        if (grown0) ref[0] = mx[0];
        if (grown1) ref[1] = mx[1];
        l[0] *= f0;
        l[1] *= f1;
#pragma unroll
        for (int e = 0; e < 2 * E; ++e) {
          o[e][0] *= f0; o[e][1] *= f0; o[e][2] *= f1; o[e][3] *= f1;
        }
      }
      const float n0 = ref[0] == -INFINITY ? 0.f : -ref[0], n1 = ref[1] == -INFINITY ? 0.f : -ref[1];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int x = 0; x < 4; ++x) s[t][x] = ex2(fmaf(s[t][x], c, x < 2 ? n0 : n1));
        l[0] += s[t][0] + s[t][1];
        l[1] += s[t][2] + s[t][3];
      }
      uint32_t a[4], rest[4];  // rest: of weights in two parts
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float y0 = s[x >> 1][2 * (x & 1)], y1 = s[x >> 1][2 * (x & 1) + 1];
        if constexpr (kScores) split_weights(y0, y1, a[x], rest[x]);
        else a[x] = pack_bf16(y0, y1);
      }
      bool bad = false;  // a value that a weight of 0 would not remove
      if (part && p.nq > 1) {
        for (int i = lane; i < kBlk * S::kRow / 16; i += 32) {
          const uint4 x = *reinterpret_cast<const uint4*>(smem + (vb - smem_u32(smem)) + i * 16);
          const uint32_t e = ((x.x & 0x7F807F80u) + 0x00800080u) | ((x.y & 0x7F807F80u) + 0x00800080u) |
                             ((x.z & 0x7F807F80u) + 0x00800080u) | ((x.w & 0x7F807F80u) + 0x00800080u);
          bad |= (e & 0x80008000u) != 0;
        }
        bad = __any_sync(0xffffffffu, bad);
      }
      if (!bad) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int m = lane >> 3, r = (lane & 7) + (m & 1) * 8;
          uint32_t f[4];
          ldsm_x4_t_addr(f, vb + piece<D>(r, 2 * e + (m >> 1)));
          mma_bf16(o[2 * e], a, f[0], f[1]);
          mma_bf16(o[2 * e + 1], a, f[2], f[3]);
          if constexpr (kScores) {
            mma_bf16(o[2 * e], rest, f[0], f[1]);
            mma_bf16(o[2 * e + 1], rest, f[2], f[3]);
          }
        }
      } else {  // key by key, each row only over the keys that it sees
#pragma unroll
        for (int j = 0; j < kBlk; ++j) {
          const int from = (lane & ~3) | ((j & 7) >> 1);
          const float w0 = __shfl_sync(0xffffffffu, s[j >> 3][j & 1], from);
          const float w1 = __shfl_sync(0xffffffffu, s[j >> 3][2 + (j & 1)], from);
          const bool sees0 = key0 + j < cur.len - lim_off[0], sees1 = key0 + j < cur.len - lim_off[1];
#pragma unroll
          for (int e = 0; e < 2 * E; ++e) {
            const __nv_bfloat162 v2 = *reinterpret_cast<const __nv_bfloat162*>(
                smem + (vb - smem_u32(smem)) + piece<D>(j, e) + cq * 2);
            const float2 v = __bfloat1622float2(v2);
            if (sees0) { o[e][0] += w0 * v.x; o[e][1] += w0 * v.y; }
            if (sees1) { o[e][2] += w1 * v.x; o[e][3] += w1 * v.y; }
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

    // ---- the end of a pair's part: merge the key groups, finish or hand over
    if (cur.u < u1) load_q();  // the next pair's queries arrive meanwhile
    const bool whole = seg_chunk == cur.kOwn && was.chunk == was.chunks - 1;
    float2* ml = reinterpret_cast<float2*>(smem + S::kMl);
    float f[2];
    finish_part<D, WM, 16, 32, kScores, 2>(
        p, w, reinterpret_cast<float*>(smem + S::kMerge), ml,
        [&] {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
            l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
            if ((lane & 3) == 0) ml[kg * 16 * WM + row0 + 8 * x] = make_float2(ref[x], l[x]);
          }
        },
        [&](float* buf, int q, auto most) {
          if (q == 0) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float m = most(row0 + 8 * x);
              f[x] = m == -INFINITY ? 0.f : ex2(ref[x] - m);
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float* y = o[4 * q + e];
            float* dst = buf + (kg * 16 * WM + row0) * 32 + ((e ^ (row0 & 3)) * 8) + cq;
            *reinterpret_cast<float2*>(dst) = make_float2(y[0] * f[0], y[1] * f[0]);
            *reinterpret_cast<float2*>(dst + 8 * 32) = make_float2(y[2] * f[1], y[3] * f[1]);
          }
        },
        was.n, was.hk, whole, 2 * blockIdx.x + (seg_first ? 0 : 1));
    __syncthreads();
    reset();
    seg_chunk = cur.chunk;
    seg_first = false;
  }
  pdl_wait();
}

template <int D>
bool launch_prefix(const AttnParams& p, const PrefixParts& parts, cudaStream_t s) {
  // A page's rows of one key head, in groups of 8 rows with their 64-element halves apart.
  const uint32_t box[4] = {64, 8, D / 64, (uint32_t)(p.page < kKeys ? p.page : kKeys) / 8};
  const uint64_t dim[4] = {64, 8, D / 64, (uint64_t)p.n_pages * p.Hk * p.page / 8};
  const uint64_t str[3] = {D * 2, 128, D * 16};
  CUtensorMap tm_k, tm_v;
  if (!encode_bf16_tmap(&tm_k, p.k, 4, dim, str, box) ||
      !encode_bf16_tmap(&tm_v, p.v, 4, dim, str, box))
    return false;
  const int span = 2 * (kRows / p.G);
  return launch_attn_tc<D, true>(p, parts, tm_k, tm_v,
                                 ((int64_t)p.T + span - 1) / span * p.Hk * parts.splits, s);
}

template <int D, bool kScores>
bool launch(AttnParams p, void* workspace, cudaStream_t s) {
  const int64_t keys = (int64_t)p.max_pages * p.page;
  const DecodeLayout L = layout(p.T, p.N, p.H, p.Hk, D, kScores ? keys : 0);
  DecodeParts w = parts_of(L, workspace);
  w.prefix.tiles = (p.common + kKeys - 1) / kKeys;
  w.prefix.splits = L.splits < w.prefix.tiles ? L.splits : w.prefix.tiles;
  // The prefix kernel and the merge of its parts cost about 5 us; without them every sequence
  // reads the prefix's keys itself, mostly from L2, and with many query rows also multiplies
  // them in WM row tiles at warp-MMA speed. What counts is how many keys that is, of either head
  // size. Measured (GB300; thousands of keys read again, with / without the prefix kernel):
  // 84 17.7 / 14.3 us, 129 15.4 / 15.0, 172 27.3 / 24.7, 188 17.9 / 20.4, 224 17.7 / 21.5,
  // 429 17.4 / 29.9; D = 64: 157 20.9 / 20.7, 237 15.1 / 18.1, 396 15.6 / 24.1. One point is on
  // the wrong side of the rule: four row tiles behind a short prefix, 199, 24.3 / 20.8.
  const int R = p.nq * p.G, WM = R <= 16 ? 1 : R <= 32 ? 2 : 4;
  const int64_t again = (int64_t)(p.N - 1) * p.common * p.Hk * WM;
  p.shared = p.n_pages > 0 && p.N > 1 && (again >= 180000 || attn_prefix_always())
                 ? p.common : 0;
  if (p.shared > 0 && !launch_prefix<D>(p, w.prefix, s)) return false;
  // no more CTAs than units there can be
  const int64_t most = (int64_t)p.N * p.Hk * (((int64_t)p.max_pages * p.page + kUnit - 1) / kUnit);
  w.grid = (int)(most < L.grid ? (most > 0 ? most : 1) : L.grid);
  if (kScores) {
    w.lse2 = reinterpret_cast<float*>(static_cast<char*>(workspace) + L.lse2);
    w.scores = reinterpret_cast<float*>(static_cast<char*>(workspace) + L.scores);
    w.keys = keys;
  }
  const auto kernel = R <= 16   ? decode_kernel<D, 1, kScores>
                      : R <= 32 ? decode_kernel<D, 2, kScores>
                                : decode_kernel<D, 4, kScores>;
  constexpr int smem = DecodeSmem<D>::kBytes;
  ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem);
  return launch_pdl(kernel, dim3(w.grid), dim3(kWarps * 32), smem, s, p, w) == cudaSuccess &&
         launch_rest<D, kUnit, kScores>(p, w, s);
}

}  // namespace

size_t attn_decode_workspace(int T, int N, int H, int Hk, int D) {
  return layout(T, N, H, Hk, D).total;
}
size_t attn_decode_cache_workspace(int T, int N, int H, int Hk, int D, int64_t keys, bool weights) {
  return layout(T, N, H, Hk, D, weights ? keys : 0, kDecode8Ctas).total;
}

bool launch_attn_decode(const AttnParams& p, void* workspace, cudaStream_t s) {
  if (p.weights)
    return p.D == 128 ? launch<128, true>(p, workspace, s) : launch<64, true>(p, workspace, s);
  return p.D == 128 ? launch<128, false>(p, workspace, s) : launch<64, false>(p, workspace, s);
}

}  // namespace gdn
