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

template <int D>
struct DecodeSmem {
  static constexpr int kRow = D * 2;                 // bytes of a key
  static constexpr int kStage = 2 * kBlk * kRow;     // a K and a V block
  // 64 KB of ring per CTA, half of it in flight. More only makes every other read (a row of
  // the queries, a page number) wait longer in a saturated memory system: with 96 KB, 64
  // sequences of up to 8192 keys took 163.4 us, with 64 KB 159.0 us.
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kMerge = kWarps * kStages * kStage;
  static constexpr int kMl = kMerge + 2 * kWarps * 16 * 32 * 4;
  static constexpr int kBytes = kMl + kWarps * 16 * 8;
};

// 16-byte piece c of row r, spread over the banks for ldmatrix.
template <int D>
__device__ __forceinline__ uint32_t piece(int r, int c) {
  return (uint32_t)(r * D * 2 + ((c ^ (r & 7)) << 4));
}

template <int D, int WM>
__global__ void __launch_bounds__(kWarps * 32, 2)
decode_kernel(const AttnParams p, const DecodeParts w) {
  using S = DecodeSmem<D>;
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
      const uint32_t a[4] = {pack_bf16(s[0][0], s[0][1]), pack_bf16(s[0][2], s[0][3]),
                             pack_bf16(s[1][0], s[1][1]), pack_bf16(s[1][2], s[1][3])};
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
      f[x] = m == -INFINITY ? 0.f : ex2(ref[x] - m);
    }
    // 32 columns at a time through two buffers [WK][16 WM][32], one barrier a round: a buffer
    // is written again two rounds later, past a barrier that its readers have reached. 8-column
    // pieces are swapped by row, so that a warp's eight rows do not share banks.
#pragma unroll
    for (int q = 0; q < D / 32; ++q) {
      float* buf = reinterpret_cast<float*>(smem + S::kMerge) + (q & 1) * (kWarps * 16 * 32);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float* y = o[4 * q + e];
        float* dst = buf + (kg * 16 * WM + row0) * 32 + ((e ^ (row0 & 3)) * 8) + cq;
        *reinterpret_cast<float2*>(dst) = make_float2(y[0] * f[0], y[1] * f[0]);
        *reinterpret_cast<float2*>(dst + 8 * 32) = make_float2(y[2] * f[1], y[3] * f[1]);
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
          if (p.lse && q == 0 && col == 0)
            p.lse[at] = d == 0.f ? -INFINITY : (m + log2f(d)) * 0.69314718055994530942f;
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
  if (p.lse && lane == 0)
    p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
}

struct DecodeLayout {
  size_t first, part, part_ml, own, own_ml, prefix, prefix_ml, total;
  int grid, splits;  // splits: of the prefix's keys, at most
};

DecodeLayout layout(int T, int N, int H, int Hk, int D) {
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

template <int D>
bool launch(AttnParams p, void* workspace, cudaStream_t s) {
  const DecodeLayout L = layout(p.T, p.N, p.H, p.Hk, D);
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
  p.shared = p.n_pages > 0 && p.N > 1 && (again >= 180000 || attn_prefix_always())
                 ? p.common : 0;
  if (p.shared > 0 && !launch_prefix<D>(p, w.prefix, s)) return false;
  // no more CTAs than units there can be
  const int64_t most = (int64_t)p.N * p.Hk * (((int64_t)p.max_pages * p.page + kUnit - 1) / kUnit);
  w.grid = (int)(most < L.grid ? (most > 0 ? most : 1) : L.grid);
  const auto kernel = R <= 16 ? decode_kernel<D, 1> : R <= 32 ? decode_kernel<D, 2> : decode_kernel<D, 4>;
  constexpr int smem = DecodeSmem<D>::kBytes;
  ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem);
  // Warps of a merged row: eight while all their CTAs fit the GPU at once (a row has many
  // parts then: one sequence of 8191 keys 13.4 us with four, 12.5 with eight; 64 sequences,
  // 2048 rows, 157.0 with four, 159.6 with eight), four up to as many rows as those fit, one
  // beyond (64 sequences x 5 tokens x 64 heads behind 256 keys 46.7 us with four, 29.2 with one).
  const size_t rows = (size_t)p.T * p.H, sms = (size_t)num_sms();
  const int W = rows <= 8 * sms ? 8 : rows <= 32 * sms ? 4 : 1;
  const auto combine = W == 8 ? combine_kernel<D, 8> : W == 4 ? combine_kernel<D, 4> : combine_kernel<D, 1>;
  return launch_pdl(kernel, dim3(w.grid), dim3(kWarps * 32), smem, s, p, w) == cudaSuccess &&
         launch_pdl(combine, dim3((unsigned)(W == 1 ? (rows + 3) / 4 : rows)), dim3(W == 8 ? 256 : 128), 0,
                    s, p, w) == cudaSuccess;
}

}  // namespace

size_t attn_decode_workspace(int T, int N, int H, int Hk, int D) {
  return layout(T, N, H, Hk, D).total;
}

bool launch_attn_decode(const AttnParams& p, void* workspace, cudaStream_t s) {
  return p.D == 128 ? launch<128>(p, workspace, s) : launch<64>(p, workspace, s);
}

}  // namespace gdn
