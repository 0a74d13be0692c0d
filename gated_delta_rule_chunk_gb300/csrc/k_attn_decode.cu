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
// summed in fp32 before that.
//
// Measured (GB300): 64 sequences of up to 8192 keys 148.5 to 153 us (6.8 TB/s), one of 8191 keys
// 10.1 us, 64 behind 16384 shared keys 53 to 58 us.
#include "attn_tc.cuh"
#include "e4m3.cuh"

namespace gdn {

namespace {

constexpr int kUnit = 64;   // keys of a unit
// Units that a pair counts for beside its keys', for its queries, merge and results: without
// them the CTAs that get many short sequences end last (64 sequences of up to 8192 keys
// 155.4 us, with one 150.2, two 148.5, three 149.3; of up to 1024 behind a prefix 67.2, 61.3,
// 60.7, 59.7; the price: one sequence of 8191 keys 12.3 -> 12.9, as some CTAs get less).
constexpr int kPair = 2;
constexpr int kBlk = 16;    // keys of a warp's block
constexpr int kWarps = 4;

// The workspace: partial sums of pairs that span CTAs (two places per CTA: the part at its
// start, the part at its end), the unit numbers of the sequences.
struct DecodeParts {
  int32_t* first;      // [N + 1] unit number of each sequence's first unit
  float* lse2;         // [N, nq, H] log2 of the softmax denominators, where weights are wanted
  float* scores;       // [N * Hk][R][keys] scores in powers of two: of what a row sees, -inf else
  int64_t keys;        // max_pages * page
  float* part;         // [2 * grid][R][D]
  float2* part_ml;     // [2 * grid][R] reference (powers of two) and denominator
  float* own;          // [N * Hk][R][D] and [N * Hk][R]: pairs that lie in one CTA, when
  float2* own_ml;      // the prefix's part is still to be added
  int grid;
  PrefixParts prefix;
};

// Units of each pair of a sequence of `len` keys: its keys' and, before them, kPair for the
// pair itself.
__device__ __forceinline__ int chunks_of(const AttnParams& p, int len) {
  const int keys = len - p.shared;
  return keys > 0 ? kPair + (keys + kUnit - 1) / kUnit : 0;
}
// Equal parts of U units for `grid` CTAs (at most one a unit): CTA c's first unit, and the
// CTA of unit u. The parts that are one unit longer are spread evenly: with the first CTAs
// taking them, both CTAs of the same SMs do (64 sequences 159 -> 170 us).
__device__ __forceinline__ int unit_of(int c, int U, int grid) {
  if (U < 1 << 22) return (int)((uint32_t)c * (uint32_t)U / (uint32_t)grid);  // c < 1024
  return (int)((int64_t)c * U / grid);
}
__device__ __forceinline__ int cta_of(int u, int U, int grid) {
  if (U < 1 << 22) return (int)(((uint32_t)(u + 1) * grid - 1) / (uint32_t)U);
  return (int)((((int64_t)u + 1) * grid - 1) / U);
}

// A place in the unit list: unit u, `chunk` of a pair's. The units that stand for the pair
// itself are passed over.
struct Cursor {
  int u, n, hk, chunk, chunks, len;
  __device__ void load(const AttnParams& p) {
    len = seq_len(p, n);
    chunks = chunks_of(p, len);
  }
  __device__ void settle() {
    u += max(kPair - chunk, 0);
    chunk = max(chunk, kPair);
  }
  __device__ void next(const AttnParams& p) {
    ++u;
    if (++chunk < chunks) return;
    chunk = 0;
    settle();
    if (++hk < p.Hk) return;
    hk = 0;
    do {
      if (++n >= p.N) {
        chunks = len = 0;
        return;
      }
      load(p);
    } while (chunks == 0);
  }
  __device__ int key() const { return (chunk - kPair) * kUnit; }  // first key, past the prefix
};

template <int D, bool k8>
struct DecodeSmem {
  static constexpr int kRow = k8 ? D : D * 2;        // bytes of a key
  static constexpr int kScale = 2 * kBlk * kRow;     // in 8 bits: the scales of K and V
  static constexpr int kStage = kScale + (k8 ? 128 : 0);  // a K and a V block
  // 64 KB of ring per CTA, half of it in flight. More only makes every other read (a row of
  // the queries, a page number) wait longer in a saturated memory system: with 96 KB, 64
  // sequences of up to 8192 keys took 163.4 us, with 64 KB 159.0 us.
  static constexpr int kStages = (D == 128 ? 2 : 4) * (k8 ? 2 : 1);
  static constexpr int kMerge = kWarps * kStages * kStage;
  static constexpr int kMl = kMerge + 2 * kWarps * 16 * 32 * 4;
  static constexpr int kBytes = kMl + kWarps * 16 * 8;
};

// 16-byte piece c of row r (of kRow bytes), spread over the banks for ldmatrix.
template <int kRow>
__device__ __forceinline__ uint32_t piece(int r, int c) {
  if constexpr (kRow == 64) return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
  return (uint32_t)(r * kRow + ((c ^ (r & 7)) << 4));
}

__device__ __forceinline__ uint32_t max_abs(uint32_t m, uint32_t bits) {
  bits &= 0x7FFFFFFFu;
  return max(m, bits < 0x7F800000u ? bits : 0u);
}

// Bytes of e4m3 with 0 in the place of NaN.
__device__ __forceinline__ uint32_t without_nan(uint32_t x) {
  const uint32_t nan = ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  return x & ~((nan >> 7) * 0xFFu);
}

template <int D, int WM, bool k8, bool kScores>
__global__ void __launch_bounds__(kWarps * 32, 2)
decode_kernel(const AttnParams p, const DecodeParts w) {
  using S = DecodeSmem<D, k8>;
  constexpr int kRow = S::kRow, kPieces = kRow / 16;
  constexpr int kSt = S::kStages, WK = kWarps / WM, E = D / 16;
  extern __shared__ __align__(128) char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int kg = warp / WM, mt = warp % WM;  // key group, row tile
  const int R = p.nq * p.G;
  // With a prefix kernel before this one in the stream nothing of it is needed here, and it
  // has waited for what came before; this kernel then only ends after it.
  if (p.shared == 0) pdl_wait();
  pdl_release();

  // ---- the CTA's part of the unit list; each warp looks it up for itself
  int U = 0, len32 = 0;  // len32: of this lane's sequence among the first 32
  for (int n = lane; n < p.N; n += 32) {
    const int len = seq_len(p, n);
    if (n == lane) len32 = len;
    U += chunks_of(p, len);
    if (blockIdx.x == 0 && (p.kv_lens[n] < 0 || p.kv_lens[n] > (p.max_pages << p.page_shift)))
      set_status(p.status, GDN_DEV_BAD_LENGTH);
  }
  U = __reduce_add_sync(0xffffffffu, U) * p.Hk;
  const int grid = min((int)gridDim.x, U), b = (int)blockIdx.x;
  const int u0 = b < grid ? unit_of(b, U, grid) : U, u1 = b < grid ? unit_of(b + 1, U, grid) : U;
  Cursor cur{};
  const bool scribe = b == 0 && warp == 0;  // writes the sequences' first units
  int before = 0;
  for (int n0 = 0; n0 < p.N && (scribe || before * p.Hk <= u0); n0 += 32) {
    const int n = n0 + lane;
    const int len = n0 == 0 ? len32 : n < p.N ? seq_len(p, n) : 0;
    const int c = n < p.N ? chunks_of(p, len) : 0;
    int inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    const int at = (before + inc - c) * p.Hk;
    if (scribe && n < p.N) w.first[n] = at;
    const uint32_t hit = __ballot_sync(0xffffffffu, c > 0 && u0 >= at && u0 < at + c * p.Hk);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const int off = u0 - __shfl_sync(0xffffffffu, at, src), ch = __shfl_sync(0xffffffffu, c, src);
      cur.n = n0 + src;
      cur.hk = off / ch;
      cur.chunk = off % ch;
      cur.chunks = ch;
      cur.len = __shfl_sync(0xffffffffu, len, src);
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (scribe && lane == 0) w.first[p.N] = U;
  if (u0 < u1) {
    cur.u = u0;
    cur.settle();
  }
  if (u0 >= u1 || cur.u >= u1) {
    pdl_wait();
    return;
  }
  Cursor ahead = cur;  // what is loaded next

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
        const size_t row = (((size_t)(ok ? page : 0) * p.Hk + ahead.hk) << p.page_shift) +
                           (key & (p.page - 1));
        const int rows = ahead.len - key;  // rows past the end are not read, zeros stand for them
        const char* k = reinterpret_cast<const char*>(p.k) + row * kRow;
        const char* v = reinterpret_cast<const char*>(p.v) + row * kRow;
        const uint32_t dst = ring + st * S::kStage;
#pragma unroll
        for (int i = 0; i < kBlk * kPieces / 32; ++i) {
          const int x = i * 32 + lane, r = x / kPieces, c = x % kPieces;
          const uint32_t n = ok && r < rows ? 16 : 0;
          asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;\n" ::"r"(
                           dst + piece<kRow>(r, c)),
                       "l"(n ? k + x * 16 : reinterpret_cast<const char*>(p.k)), "r"(n), "l"(once));
          asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;\n" ::"r"(
                           dst + kBlk * kRow + piece<kRow>(r, c)),
                       "l"(n ? v + x * 16 : reinterpret_cast<const char*>(p.v)), "r"(n), "l"(once));
        }
        if constexpr (k8) {
          if (lane < 2) {  // (a page that does not exist: keys and values times 0)
            const float* x = lane ? p.vs : p.ks;
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst + S::kScale + lane * 4),
                         "l"(ok ? x + row / kBlk : x), "r"(ok ? 4 : 0));
          }
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
  auto pack_p = [](float lo, float hi) { return k8 ? pack_f16(lo, hi) : pack_bf16(lo, hi); };
  const int g = lane >> 2, cq = (lane & 3) * 2;
  const int row0 = mt * 16 + g;  // this thread's rows: row0, row0 + 8
  uint32_t qf[E][4];
  float o[2 * E][4], ref[2], l[2];
  float refv[2];  // 8 bits: the reference of the sums in o
  int lim_off[2];  // keys past len that the row does not see: lim = len - lim_off
#pragma unroll
  for (int x = 0; x < 2; ++x) lim_off[x] = p.nq - 1 - min((row0 + 8 * x) / p.G, p.nq - 1);
  // This warp's rows of the queries of the pair at `cur`. Over a cache in 8 bits they are fp16
  // like its keys: times a power of two, by the row's largest element, that puts it below 2^15;
  // elements are then exact down to 2^-29 of it, and below off by 2^-40 of it at most.
  float qc[2] = {c, c};  // what a row's scores are multiplied with
  auto load_q = [&] {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = row0 + 8 * x;
      const __nv_bfloat16* q =
          p.q + ((size_t)(cur.n * p.nq + r / p.G) * p.H + cur.hk * p.G + r % p.G) * D;
      if constexpr (k8) {
        // columns k of the MMAs are elements 4 (k / 2) + k % 2 of 16, columns 8 + k those 2 on
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint2 y = r < R ? *reinterpret_cast<const uint2*>(q + e * 16 + 2 * cq) : make_uint2(0, 0);
          qf[e][x] = y.x;
          qf[e][x + 2] = y.y;
          top = max_abs(max_abs(max_abs(max_abs(top, y.x << 16), y.x & 0xFFFF0000u), y.y << 16),
                        y.y & 0xFFFF0000u);
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = max((int)(top >> 23) - 127 - 14, -100);
        const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
        qc[x] = c * __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
          for (int y = x; y < 4; y += 2)
            qf[e][y] = pack_f16(__uint_as_float(qf[e][y] << 16) * down,
                                __uint_as_float(qf[e][y] & 0xFFFF0000u) * down);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          qf[e][x] = r < R ? *reinterpret_cast<const uint32_t*>(q + e * 16 + cq) : 0u;
          qf[e][x + 2] = r < R ? *reinterpret_cast<const uint32_t*>(q + e * 16 + 8 + cq) : 0u;
        }
      }
    }
  };
  auto reset = [&] {
    ref[0] = ref[1] = refv[0] = refv[1] = -INFINITY;
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
      const uint32_t vb = kb + kBlk * kRow;
      float s[2][4] = {};
      [[maybe_unused]] float sv = 0.f;  // 8 bits: the scale of the block's values
      const bool part = key0 + kBlk > cur.len - (p.nq - 1);  // some row does not see all
      if constexpr (k8) {
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const int m = lane >> 3, r = (lane & 7) + (m & 1) * 8;
          uint32_t f[4];
          ldsm_x4_addr(f, kb + piece<kRow>(r, e + (m >> 1)));
          mma_f16(s[0], qf[e], e4m3x2_to_f16x2(f[0]), e4m3x2_to_f16x2(f[0] >> 16));
          mma_f16(s[1], qf[e], e4m3x2_to_f16x2(f[1]), e4m3x2_to_f16x2(f[1] >> 16));
          mma_f16(s[0], qf[e + 1], e4m3x2_to_f16x2(f[2]), e4m3x2_to_f16x2(f[2] >> 16));
          mma_f16(s[1], qf[e + 1], e4m3x2_to_f16x2(f[3]), e4m3x2_to_f16x2(f[3] >> 16));
        }
        const float2 scale = *reinterpret_cast<const float2*>(smem + (kb - smem_u32(smem)) + S::kScale);
        sv = scale.y;
        const float c0 = qc[0] * scale.x, c1 = qc[1] * scale.x;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          s[t][0] *= c0; s[t][1] *= c0; s[t][2] *= c1; s[t][3] *= c1;
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int m = lane >> 3, r = (lane & 7) + (m >> 1) * 8;
          uint32_t f[4];
          ldsm_x4_addr(f, kb + piece<kRow>(r, 2 * e + (m & 1)));
          mma_bf16(s[0], qf[e], f[0], f[1]);
          mma_bf16(s[1], qf[e], f[2], f[3]);
        }
      }
      if (part) {  // (after the scales, which may be 0)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (key0 + t * 8 + cq + (x & 1) >= cur.len - lim_off[x >> 1]) s[t][x] = -INFINITY;
      }
      constexpr bool kInPowers = k8;  // the scores are in powers of two already
      const float cc = kInPowers ? 1.f : c;
      if constexpr (kScores) {
        float* to = w.scores + ((size_t)(cur.n * p.Hk + cur.hk) * R + row0) * w.keys + key0 + cq;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (row0 + 8 * x >= R) continue;
#pragma unroll
          for (int t = 0; t < 2; ++t)
            *reinterpret_cast<float2*>(to + 8 * x * w.keys + t * 8) =
                make_float2(s[t][2 * x] * cc, s[t][2 * x + 1] * cc);
        }
      }
      float mx[2] = {fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1])),
                     fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]))};
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 1));
        mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 2)) * cc;
      }
      const bool grown0 = mx[0] > ref[0] && mx[0] - ref[0] > kGrow;
      const bool grown1 = mx[1] > ref[1] && mx[1] - ref[1] > kGrow;
      if (__any_sync(0xffffffffu, grown0 || grown1)) {
        const float f0 = grown0 ? ex2(ref[0] - mx[0]) : 1.f, f1 = grown1 ? ex2(ref[1] - mx[1]) : 1.f;
        if (grown0) ref[0] = mx[0];
        if (grown1) ref[1] = mx[1];
        l[0] *= f0;
        l[1] *= f1;
        if constexpr (!k8) {
#pragma unroll
          for (int e = 0; e < 2 * E; ++e) {
            o[e][0] *= f0; o[e][1] *= f0; o[e][2] *= f1; o[e][3] *= f1;
          }
        }
      }
      [[maybe_unused]] float raw[2][4];
      if constexpr (k8) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int x = 0; x < 4; ++x) raw[t][x] = s[t][x];
      }
      const float n0 = ref[0] == -INFINITY ? 0.f : -ref[0], n1 = ref[1] == -INFINITY ? 0.f : -ref[1];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int x = 0; x < 4; ++x) s[t][x] = kInPowers ? ex2(s[t][x] + (x < 2 ? n0 : n1)) : ex2(fmaf(s[t][x], c, x < 2 ? n0 : n1));
        l[0] += s[t][0] + s[t][1];
        l[1] += s[t][2] + s[t][3];
      }
      if constexpr (k8) {
        // Weights times the values' scale, in fp16 like the values, against a reference of their
        // own: 2^7 where it is set, 2^15 at most; below 2^-24 they are subnormal, 2^-31 of the
        // largest. (One reference for both would leave fp16's range where scales differ.)
        const float lv = log2f(sv);
        float f[2];
        bool grown[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float top = mx[x] == -INFINITY ? -INFINITY : mx[x] + lv - 7.f;
          grown[x] = top > refv[x] && top - refv[x] > kGrow;
          f[x] = grown[x] ? ex2(refv[x] - top) : 1.f;
          if (grown[x]) refv[x] = top;
        }
        if (__any_sync(0xffffffffu, grown[0] || grown[1])) {
#pragma unroll
          for (int e = 0; e < 2 * E; ++e) {
            o[e][0] *= f[0]; o[e][1] *= f[0]; o[e][2] *= f[1]; o[e][3] *= f[1];
          }
        }
        // from the one reference to the other; nothing where a row sees none of the block, or its
        // scale is 0
        float far = 0.f;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const bool none = mx[x] == -INFINITY || refv[x] == -INFINITY;
          const float d = none ? -INFINITY : lv + ref[x] - refv[x];
          far = fmaxf(far, d);
          f[x] = ex2(d);
        }
        if (__any_sync(0xffffffffu, far > 100.f)) {
          // scores far below the largest with values as far above: f or the weight leaves fp32
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              s[t][x] = f[x >> 1] > 0.f ? ex2((raw[t][x] - refv[x >> 1]) + lv) : 0.f;
        } else {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            s[t][0] *= f[0]; s[t][1] *= f[0]; s[t][2] *= f[1]; s[t][3] *= f[1];
          }
        }
      }
      const uint32_t a[4] = {pack_p(s[0][0], s[0][1]), pack_p(s[0][2], s[0][3]),
                             pack_p(s[1][0], s[1][1]), pack_p(s[1][2], s[1][3])};
      bool bad = false;  // a value that a weight of 0 would not remove
      if (part && p.nq > 1) {
        for (int i = lane; i < kBlk * kPieces; i += 32) {
          const uint4 x = *reinterpret_cast<const uint4*>(smem + (vb - smem_u32(smem)) + i * 16);
          // the exponent's bits (8 bits: all but the sign) are ones
          constexpr uint32_t kBits = k8 ? 0x7F7F7F7Fu : 0x7F807F80u, kOne = k8 ? 0x01010101u : 0x00800080u;
          const uint32_t e = ((x.x & kBits) + kOne) | ((x.y & kBits) + kOne) |
                             ((x.z & kBits) + kOne) | ((x.w & kBits) + kOne);
          bad |= (e & (k8 ? 0x80808080u : 0x80008000u)) != 0;
        }
        bad = __any_sync(0xffffffffu, bad);
      }
      if (k8 || !bad) {
        if constexpr (k8) {
          // A pair of elements of 8 keys comes transposed as one matrix: its even elements are one
          // tile's columns, the odd ones the next tile's.
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const int m = lane >> 3, r = (lane & 7) + (m & 1) * 8;
            uint32_t f[4];
            ldsm_x4_t_addr(f, vb + piece<kRow>(r, e + (m >> 1)));
#pragma unroll
            for (int x = 0; x < 4; ++x) f[x] = __byte_perm(bad ? without_nan(f[x]) : f[x], 0, 0x3120);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              mma_f16(o[2 * (e + x)], a, e4m3x2_to_f16x2(f[2 * x]), e4m3x2_to_f16x2(f[2 * x + 1]));
              mma_f16(o[2 * (e + x) + 1], a, e4m3x2_to_f16x2(f[2 * x] >> 16),
                      e4m3x2_to_f16x2(f[2 * x + 1] >> 16));
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int m = lane >> 3, r = (lane & 7) + (m & 1) * 8;
            uint32_t f[4];
            ldsm_x4_t_addr(f, vb + piece<kRow>(r, 2 * e + (m >> 1)));
            mma_bf16(o[2 * e], a, f[0], f[1]);
            mma_bf16(o[2 * e + 1], a, f[2], f[3]);
          }
        }
      }
      if (bad && k8) {  // NaN to the rows that see it (with a weight of 0, too)
#pragma unroll 1
        for (int j = 0; j < kBlk; ++j) {
          const bool sees0 = key0 + j < cur.len - lim_off[0], sees1 = key0 + j < cur.len - lim_off[1];
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const uint32_t x = *reinterpret_cast<const uint32_t*>(
                smem + (vb - smem_u32(smem)) + piece<kRow>(j, e) + cq * 2);
            const uint32_t nan = ((x & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (!(nan >> (8 * i) & 0x80u)) continue;
              if (sees0) o[2 * e + (i & 1)][i >> 1] = NAN;
              if (sees1) o[2 * e + (i & 1)][2 + (i >> 1)] = NAN;
            }
          }
        }
      } else if (bad) {  // key by key, each row only over the keys that it sees
#pragma unroll
        for (int j = 0; j < kBlk; ++j) {
          const int from = (lane & ~3) | ((j & 7) >> 1);
          const float w0 = __shfl_sync(0xffffffffu, s[j >> 3][j & 1], from);
          const float w1 = __shfl_sync(0xffffffffu, s[j >> 3][2 + (j & 1)], from);
          const bool sees0 = key0 + j < cur.len - lim_off[0], sees1 = key0 + j < cur.len - lim_off[1];
#pragma unroll
          for (int e = 0; e < 2 * E; ++e) {
            const __nv_bfloat162 v2 = *reinterpret_cast<const __nv_bfloat162*>(
                smem + (vb - smem_u32(smem)) + piece<kRow>(j, e) + cq * 2);
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

    const Cursor was = cur;
    cur.next(p);
    if (cur.u < u1 && cur.n == was.n && cur.hk == was.hk) continue;

    // ---- the end of a pair's part: merge the key groups, finish or hand over
    if (cur.u < u1) load_q();  // the next pair's queries arrive meanwhile
    const bool whole = seg_chunk == kPair && was.chunk == was.chunks - 1;
    const int place = 2 * blockIdx.x + (seg_first ? 0 : 1);
    float2* ml = reinterpret_cast<float2*>(smem + S::kMl);  // [WK][16 WM]
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
      if ((lane & 3) == 0) ml[kg * 16 * WM + row0 + 8 * x] = make_float2(ref[x], l[x]);
    }
    __syncthreads();
    float f[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float m = -INFINITY;
#pragma unroll
      for (int k = 0; k < WK; ++k) m = fmaxf(m, ml[k * 16 * WM + row0 + 8 * x].x);
      f[x] = m == -INFINITY ? 0.f : ex2((k8 ? refv[x] : ref[x]) - m);
    }
    // 32 columns at a time through two buffers [WK][16 WM][32], one barrier a round: a buffer
    // is written again two rounds later, past a barrier that its readers have reached. 8-column
    // pieces are swapped by row, so that a warp's eight rows do not share banks.
#pragma unroll
    for (int q = 0; q < D / 32; ++q) {
      float* buf = reinterpret_cast<float*>(smem + S::kMerge) + (q & 1) * (kWarps * 16 * 32);
      if constexpr (k8) {  // 4 columns in a row: even and odd ones of two tiles
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float *y = o[4 * q + 2 * e], *z = o[4 * q + 2 * e + 1];
          const int col = e * 16 + cq * 2;
          float* dst = buf + (kg * 16 * WM + row0) * 32 + (col ^ ((row0 & 3) * 8));
          *reinterpret_cast<float4*>(dst) =
              make_float4(y[0] * f[0], z[0] * f[0], y[1] * f[0], z[1] * f[0]);
          *reinterpret_cast<float4*>(dst + 8 * 32) =
              make_float4(y[2] * f[1], z[2] * f[1], y[3] * f[1], z[3] * f[1]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float* y = o[4 * q + e];
          float* dst = buf + (kg * 16 * WM + row0) * 32 + ((e ^ (row0 & 3)) * 8) + cq;
          *reinterpret_cast<float2*>(dst) = make_float2(y[0] * f[0], y[1] * f[0]);
          *reinterpret_cast<float2*>(dst + 8 * 32) = make_float2(y[2] * f[1], y[3] * f[1]);
        }
      }
      __syncthreads();
#pragma unroll
      for (int z = 0; z < WM; ++z) {
        const int x = z * 128 + tid, r = x >> 3, col = (x & 7) * 4;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float m = -INFINITY, d = 0.f;
#pragma unroll
        for (int k = 0; k < WK; ++k) {
          const float4 y = *reinterpret_cast<const float4*>(buf + (k * 16 * WM + r) * 32 +
                                                              (col ^ ((r & 3) * 8)));
          acc.x += y.x; acc.y += y.y; acc.z += y.z; acc.w += y.w;
          m = fmaxf(m, ml[k * 16 * WM + r].x);
        }
#pragma unroll
        for (int k = 0; k < WK; ++k) {
          const float2 y = ml[k * 16 * WM + r];
          d += m == -INFINITY ? y.y : y.y * ex2(y.x - m);
        }
        if (r >= R) continue;
        if (whole && p.shared == 0) {
          const float inv = d == 0.f ? 0.f : 1.f / d;
          const size_t at = (size_t)(was.n * p.nq + r / p.G) * p.H + was.hk * p.G + r % p.G;
          if (p.out_bf16)
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at * D + q * 32 + col) =
                make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
          else
            *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at * D + q * 32 + col) =
                make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
          if ((p.lse || kScores) && q == 0 && col == 0) {
            const float lse2 = d == 0.f ? -INFINITY : m + log2f(d);
            if (p.lse) p.lse[at] = lse2 * 0.69314718055994530942f;
            if (kScores) w.lse2[at] = lse2;
          }
        } else {
          const size_t at = (size_t)(whole ? was.n * p.Hk + was.hk : place) * R + r;
          *reinterpret_cast<float4*>((whole ? w.own : w.part) + at * D + q * 32 + col) = acc;
          if (q == 0 && col == 0) (whole ? w.own_ml : w.part_ml)[at] = make_float2(m, d);
        }
      }
    }
    __syncthreads();
    reset();
    seg_chunk = cur.chunk;
    seg_first = false;
  }
  pdl_wait();
}

// The parts of a pair that spans CTAs, merged in the order of the keys; zeros for a row that
// saw no key. W warps a row take every W-th part; a CTA has W warps, or four with a row each.
template <int D, int W>
__global__ void __launch_bounds__(W == 1 ? 128 : W * 32)
combine_kernel(const AttnParams p, const DecodeParts w) {
  constexpr int E = D / 32;
  __shared__ float sh_o[W][D];
  __shared__ float2 sh_ml[W];
  const int warp = W == 1 ? 0 : threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t at = W == 1 ? blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;  // (n, i, h)
  if (at >= (uint32_t)(p.T * p.H)) return;
  const int t = (int)(at / (uint32_t)p.H), h = (int)at - t * p.H, n = t / p.nq, hk = h / p.G;
  const int R = p.nq * p.G, r = (t - n * p.nq) * p.G + h - hk * p.G;
  pdl_wait();
  const int U = w.first[p.N], b = w.first[n], c = (w.first[n + 1] - b) / p.Hk;
  const int ub = b + hk * c;  // the pair's units [ub, ub + c)
  const int grid = min(w.grid, U);
  int c0 = 0, parts = 0;
  if (c > 0) {
    c0 = cta_of(ub + kPair, U, grid);
    parts = cta_of(ub + c - 1, U, grid) - c0 + 1;
  }
  const int splits = p.shared > 0 ? w.prefix.splits : 0;
  if (parts == 1 && splits == 0) return;  // finished by its CTA
  // Part i's row: the prefix's splits, then the pair's parts. Only its first CTA can have begun
  // with another pair, so that the pair's part is the CTA's second.
  const int second = c > 0 && unit_of(c0, U, grid) < ub;
  auto row_of = [&](int i, const float2*& ml) -> const float* {
    const float* o;
    size_t row;
    if (i < splits) {
      row = (size_t)i * p.T * p.H + at;
      o = w.prefix.o;
      ml = w.prefix.ml;
    } else if (parts == 1) {
      row = (size_t)(n * p.Hk + hk) * R + r;
      o = w.own;
      ml = w.own_ml;
    } else {
      const int j = i - splits;
      row = (size_t)(2 * (c0 + j) + (j == 0 ? second : 0)) * R + r;
      o = w.part;
      ml = w.part_ml;
    }
    ml += row;
    return o + row * D;
  };
  // A warp takes every W-th part, kAtOnce of them loaded side by side (the row with its
  // reference and denominator, which all lanes read) before the first is used: what counts is
  // the number of round trips to L2 (one sequence of 8191 keys, eight warps, the whole call:
  // 4 at once 13.9 us, 6 12.5, 8 11.5, 10 10.4, 12 10.5).
  constexpr int kAtOnce = W == 8 ? 10 : 6;
  float m = -INFINITY, l = 0.f, o[E] = {};
#pragma unroll 1
  for (int i0 = warp; i0 < splits + parts; i0 += kAtOnce * W) {
    float2 ml[kAtOnce];
    float v[kAtOnce][E];
#pragma unroll
    for (int x = 0; x < kAtOnce; ++x) {
      ml[x] = make_float2(-INFINITY, 0.f);
      if (i0 + x * W < splits + parts) {
        const float2* q;
        const float* y = row_of(i0 + x * W, q);
        ml[x] = *q;
        if constexpr (E == 4)
          *reinterpret_cast<float4*>(v[x]) = *reinterpret_cast<const float4*>(y + lane * E);
        else
          *reinterpret_cast<float2*>(v[x]) = *reinterpret_cast<const float2*>(y + lane * E);
      }
    }
#pragma unroll
    for (int x = 0; x < kAtOnce; ++x) {
      if (ml[x].y == 0.f) continue;  // the row saw no key of this part (NaN is kept)
      const float mn = fmaxf(m, ml[x].x);
      const float f = m == mn ? 1.f : ex2(m - mn), fi = ml[x].x == mn ? 1.f : ex2(ml[x].x - mn);
      m = mn;
      l = l * f + ml[x].y * fi;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * f + v[x][e] * fi;
    }
  }
  if constexpr (W > 1) {
    if (lane == 0) sh_ml[warp] = make_float2(m, l);
#pragma unroll
    for (int e = 0; e < E; ++e) sh_o[warp][lane * E + e] = o[e];
    __syncthreads();
    if (warp != 0) return;
    m = sh_ml[0].x;
#pragma unroll
    for (int i = 1; i < W; ++i) m = fmaxf(m, sh_ml[i].x);
    l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if (sh_ml[i].y == 0.f) continue;
      const float f = sh_ml[i].x == m ? 1.f : ex2(sh_ml[i].x - m);
      l += sh_ml[i].y * f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] += sh_o[i][lane * E + e] * f;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] *= inv;
  store_row<D>(p.out, p.out_bf16, at, o);
  if (lane == 0 && (p.lse || w.lse2)) {
    const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
    if (p.lse) p.lse[at] = lse2 * 0.69314718055994530942f;
    if (w.lse2) w.lse2[at] = lse2;
  }
}

// The weight that each key gets: 2^(score - lse2) over the R rows of its pair, from the scores
// that decode_kernel left (a few bytes a key beside its K and V). Each warp takes an equal part
// of the units, two keys a lane.
__global__ void __launch_bounds__(256) weights_kernel(const AttnParams p, const DecodeParts w) {
  const int lane = threadIdx.x & 31, R = p.nq * p.G;
  pdl_wait();
  const int U = w.first[p.N], W = gridDim.x * 8, me = blockIdx.x * 8 + (threadIdx.x >> 5);
  int u = (int)((int64_t)me * U / W);
  const int u1 = (int)((int64_t)(me + 1) * U / W);
  int n = -1, at = 0, end = 0, c = 0, len = 0;  // the sequence of unit u and its units [at, end)
  for (; u < u1; ++u) {
    if (u >= end) {
      for (int n0 = n + 1; n0 < p.N; n0 += 32) {  // the first sequence that ends after u
        const uint32_t hit = __ballot_sync(0xffffffffu, n0 + lane < p.N && w.first[n0 + lane + 1] > u);
        if (hit) {
          n = n0 + __ffs(hit) - 1;
          break;
        }
      }
      at = w.first[n];
      end = w.first[n + 1];
      c = (end - at) / p.Hk;
      len = seq_len(p, n);
    }
    const int hk = (u - at) / c, chunk = (u - at) - hk * c - kPair;
    const int key = chunk * kUnit + 2 * lane;
    if (chunk < 0 || key >= len) continue;
    const int page = p.table[(size_t)n * p.max_pages + (key >> p.page_shift)];
    const float* x = w.scores + (size_t)(n * p.Hk + hk) * R * w.keys + key;
    const float* lse = w.lse2 + (size_t)n * p.nq * p.H + hk * p.G;
    float2 sum = make_float2(0.f, 0.f);
    int r = 0;
    for (int i = 0; i < p.nq; ++i)
      for (int g = 0; g < p.G; ++g, ++r) {
        const float2 y = *reinterpret_cast<const float2*>(x + (size_t)r * w.keys);
        const float l = lse[(size_t)i * p.H + g];
        // (a row that sees no key: -inf - -inf)
        sum.x += y.x == -INFINITY ? 0.f : ex2(y.x - l);
        sum.y += y.y == -INFINITY ? 0.f : ex2(y.y - l);
      }
    if (page < 0 || page >= p.n_pages) continue;
    float* to = p.weights + ((((size_t)page * p.Hk + hk) << p.page_shift) + (key & (p.page - 1)));
    const int fresh = len - p.nq;  // from here on keys are the call's own
    if (key >= fresh) to[0] = sum.x;
    else atomicAdd(to, sum.x);
    if (key + 1 < len) {
      if (key + 1 >= fresh) to[1] = sum.y;
      else atomicAdd(to + 1, sum.y);
    }
  }
}

struct DecodeLayout {
  size_t first, part, part_ml, own, own_ml, prefix, prefix_ml, lse2, scores, total;
  int grid, splits;  // splits: of the prefix's keys, at most
};

// keys: of the page table where weights are wanted, else 0
DecodeLayout layout(int T, int N, int H, int Hk, int D, int64_t keys = 0) {
  DecodeLayout L{};
  const int G = H / Hk, span = 2 * (kRows / G);
  const size_t R = (size_t)(T / N) * G, rows = (size_t)T * H;
  L.grid = 2 * num_sms();
  const int64_t pairs = (T > 0 ? ((int64_t)T + span - 1) / span : 1) * Hk;
  L.splits = pairs >= num_sms() ? 1 : (int)(num_sms() / pairs);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes, 256);
    return at;
  };
  L.first = take(sizeof(int32_t) * ((size_t)N + 1));
  L.part = take(sizeof(float) * 2 * L.grid * R * D);
  L.part_ml = take(sizeof(float2) * 2 * L.grid * R);
  L.own = take(sizeof(float) * rows * D);
  L.own_ml = take(sizeof(float2) * rows);
  L.prefix = take(sizeof(float) * L.splits * rows * D);
  L.prefix_ml = take(sizeof(float2) * L.splits * rows);
  L.lse2 = take(keys > 0 ? sizeof(float) * rows : 0);
  L.scores = take(sizeof(float) * rows * keys);
  L.total = o;
  return L;
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

template <int D, bool k8, bool kScores>
bool launch(AttnParams p, void* workspace, cudaStream_t s) {
  const int64_t keys = (int64_t)p.max_pages * p.page;
  const DecodeLayout L = layout(p.T, p.N, p.H, p.Hk, p.D, kScores ? keys : 0);
  char* ws = static_cast<char*>(workspace);
  DecodeParts w{};
  w.first = reinterpret_cast<int32_t*>(ws + L.first);
  w.part = reinterpret_cast<float*>(ws + L.part);
  w.part_ml = reinterpret_cast<float2*>(ws + L.part_ml);
  w.own = reinterpret_cast<float*>(ws + L.own);
  w.own_ml = reinterpret_cast<float2*>(ws + L.own_ml);
  w.prefix.o = reinterpret_cast<float*>(ws + L.prefix);
  w.prefix.ml = reinterpret_cast<float2*>(ws + L.prefix_ml);
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
  p.shared = !k8 && p.n_pages > 0 && p.N > 1 && (again >= 180000 || attn_prefix_always())
                 ? p.common : 0;
  if (p.shared > 0 && !launch_prefix<D>(p, w.prefix, s)) return false;
  // no more CTAs than units there can be
  const int64_t most = (int64_t)p.N * p.Hk * (((int64_t)p.max_pages * p.page + kUnit - 1) / kUnit);
  w.grid = (int)(most < L.grid ? (most > 0 ? most : 1) : L.grid);
  if (kScores) {
    w.lse2 = reinterpret_cast<float*>(ws + L.lse2);
    w.scores = reinterpret_cast<float*>(ws + L.scores);
    w.keys = keys;
  }
  const auto kernel = R <= 16   ? decode_kernel<D, 1, k8, kScores>
                      : R <= 32 ? decode_kernel<D, 2, k8, kScores>
                                : decode_kernel<D, 4, k8, kScores>;
  constexpr int smem = DecodeSmem<D, k8>::kBytes;
  ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem);
  // Warps of a merged row: eight while all their CTAs fit the GPU at once (a row has many
  // parts then: one sequence of 8191 keys 13.4 us with four, 12.5 with eight; 64 sequences,
  // 2048 rows, 157.0 with four, 159.6 with eight), four up to as many rows as those fit, one
  // beyond (64 sequences x 5 tokens x 64 heads behind 256 keys 46.7 us with four, 29.2 with one).
  const size_t rows = (size_t)p.T * p.H, sms = (size_t)num_sms();
  const int W = rows <= 8 * sms ? 8 : rows <= 32 * sms ? 4 : 1;
  const auto combine = W == 8 ? combine_kernel<D, 8> : W == 4 ? combine_kernel<D, 4> : combine_kernel<D, 1>;
  if (launch_pdl(kernel, dim3(w.grid), dim3(kWarps * 32), smem, s, p, w) != cudaSuccess ||
      launch_pdl(combine, dim3((unsigned)(W == 1 ? (rows + 3) / 4 : rows)), dim3(W == 8 ? 256 : 128), 0,
                 s, p, w) != cudaSuccess)
    return false;
  if (!kScores) return true;
  return launch_pdl(weights_kernel, dim3(2 * num_sms()), dim3(256), 0, s, p, w) == cudaSuccess;
}

}  // namespace

size_t attn_decode_workspace(int T, int N, int H, int Hk, int D) {
  return layout(T, N, H, Hk, D).total;
}
size_t attn_decode_cache_workspace(int T, int N, int H, int Hk, int D, int64_t keys, bool weights) {
  return layout(T, N, H, Hk, D, weights ? keys : 0).total;
}

bool launch_attn_decode(const AttnParams& p, void* workspace, cudaStream_t s) {
  return p.D == 128 ? launch<128, false, false>(p, workspace, s)
                    : launch<64, false, false>(p, workspace, s);
}

bool launch_attn_decode_cache(const AttnParams& p, void* workspace, cudaStream_t s) {
  if (!p.ks)
    return p.D == 128 ? launch<128, false, true>(p, workspace, s)
                      : launch<64, false, true>(p, workspace, s);
  if (p.weights)
    return p.D == 128 ? launch<128, true, true>(p, workspace, s)
                      : launch<64, true, true>(p, workspace, s);
  return p.D == 128 ? launch<128, true, false>(p, workspace, s)
                    : launch<64, true, false>(p, workspace, s);
}

}  // namespace gdn
