// Parts that the decode kernels share: the list of key units and a CTA's part of it, the merge of
// what several warps and CTAs computed for a row, the weights of the keys, the workspace. What is
// cut into units, and why, is in k_attn_decode.cu.
#pragma once

#include "attn_tc.cuh"

namespace gdn {

namespace {

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

// Units of each pair of a sequence of `len` keys: its keys' and, before them, kPair for the pair
// itself, for its queries, merge and results: without them the CTAs that get many short sequences
// end last (bf16, units of 64 keys: 64 sequences of up to 8192 keys 155.4 us, with one 150.2, two
// 148.5, three 149.3; of up to 1024 behind a prefix 67.2, 61.3, 60.7, 59.7; the price: one sequence
// of 8191 keys 12.3 -> 12.9, as some CTAs get less).
template <int kUnit>
constexpr int kPair = 128 / kUnit;
template <int kUnit>
__device__ __forceinline__ int chunks_of(const AttnParams& p, int len) {
  const int keys = len - p.shared;
  return keys > 0 ? kPair<kUnit> + (keys + kUnit - 1) / kUnit : 0;
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
template <int kUnit>
struct Cursor {
  static constexpr int kOwn = kPair<kUnit>;
  int u, n, hk, chunk, chunks, len;
  __device__ void load(const AttnParams& p) {
    len = seq_len(p, n);
    chunks = chunks_of<kUnit>(p, len);
  }
  __device__ void settle() {
    u += max(kOwn - chunk, 0);
    chunk = max(chunk, kOwn);
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
  __device__ int key() const { return (chunk - kOwn) * kUnit; }  // first key, past the prefix
};

// The part of CTA blockIdx.x of the unit list: cur at its first unit, the unit u1 after its last;
// whether it has any. Each warp looks it up for itself.
template <int kUnit>
__device__ __forceinline__ bool find_units(const AttnParams& p, const DecodeParts& w,
                                           Cursor<kUnit>& cur, int& u1) {
  const int lane = threadIdx.x & 31;
  int U = 0, len32 = 0;  // len32: of this lane's sequence among the first 32
  for (int n = lane; n < p.N; n += 32) {
    const int len = seq_len(p, n);
    if (n == lane) len32 = len;
    U += chunks_of<kUnit>(p, len);
    if (blockIdx.x == 0 && (p.kv_lens[n] < 0 || p.kv_lens[n] > (p.max_pages << p.page_shift)))
      set_status(p.status, GDN_DEV_BAD_LENGTH);
  }
  U = __reduce_add_sync(0xffffffffu, U) * p.Hk;
  const int grid = min((int)gridDim.x, U), b = (int)blockIdx.x;
  const int u0 = b < grid ? unit_of(b, U, grid) : U;
  u1 = b < grid ? unit_of(b + 1, U, grid) : U;
  cur = Cursor<kUnit>{};
  const bool scribe = b == 0 && threadIdx.x < 32;  // writes the sequences' first units
  int before = 0;
  for (int n0 = 0; n0 < p.N && (scribe || before * p.Hk <= u0); n0 += 32) {
    const int n = n0 + lane;
    const int len = n0 == 0 ? len32 : n < p.N ? seq_len(p, n) : 0;
    const int c = n < p.N ? chunks_of<kUnit>(p, len) : 0;
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
  return u0 < u1 && cur.u < u1;
}

// The end of a pair's part: its key groups' results merged in shared memory and finished, or handed
// over in place `place`. A warp has TM rows. stats() writes the reference and denominator of the
// warp's rows to ml [WK][TM WM]; put(buf, q, m) writes columns kCols q .. kCols (q + 1) - 1 of their sums,
// against the references m of all groups (m(row)), to buf [WK][TM WM][kCols], the 8-column pieces of 32
// columns swapped by row (piece e at e ^ (row & 3)), so that a warp's eight rows do not share banks.
// merge: kBufs such buffers.
constexpr int kMergeBytes = kWarps * 16 * 32 * 4;
template <int D, int WM, int TM, int kCols, bool kScores, int kBufs, typename Stats, typename Put>
__device__ __forceinline__ void finish_part(const AttnParams& p, const DecodeParts& w, float* merge,
                                            float2* ml, Stats stats, Put put, int n, int hk,
                                            bool whole, int place) {
  constexpr int WK = kWarps / WM, kQuads = kCols / 4;  // threads of a row
  constexpr int kTurns = TM * WM * kQuads / (kWarps * 32);
  const int tid = threadIdx.x, R = p.nq * p.G;
  stats();
  __syncthreads();
  auto most = [&](int row) {
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < WK; ++k) m = fmaxf(m, ml[k * TM * WM + row].x);
    return m;
  };
  // This thread's rows: z * 128 / kQuads + tid / kQuads.
  float m[kTurns], d[kTurns];
#pragma unroll
  for (int z = 0; z < kTurns; ++z) {
    const int r = (z * kWarps * 32 + tid) / kQuads;
    m[z] = most(r);
    d[z] = 0.f;
#pragma unroll
    for (int k = 0; k < WK; ++k) {
      const float2 y = ml[k * TM * WM + r];
      d[z] += m[z] == -INFINITY ? y.y : y.y * ex2(y.x - m[z]);
    }
  }
  // The buffers in turn, one barrier a round: a buffer is written again two rounds later, past a
  // barrier that its readers have reached (one buffer: past one of its own).
#pragma unroll
  for (int q = 0; q < D / kCols; ++q) {
    float* buf = merge + (kBufs == 2 ? q & 1 : 0) * (WK * TM * WM * kCols);
    if (kBufs == 1 && q > 0) __syncthreads();
    put(buf, q, most);
    __syncthreads();
#pragma unroll
    for (int z = 0; z < kTurns; ++z) {
      const int r = (z * kWarps * 32 + tid) / kQuads, col = tid % kQuads * 4;
      if (r >= R) continue;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < WK; ++k) {
        const float4 y = *reinterpret_cast<const float4*>(buf + (k * TM * WM + r) * kCols +
                                                            (col ^ ((r & 3) * 8)));
        acc.x += y.x; acc.y += y.y; acc.z += y.z; acc.w += y.w;
      }
      if (whole && p.shared == 0) {
        const float inv = d[z] == 0.f ? 0.f : 1.f / d[z];
        const size_t at = (size_t)(n * p.nq + r / p.G) * p.H + hk * p.G + r % p.G;
        if (p.out_bf16)
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at * D + q * kCols + col) =
              make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
        else
          *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at * D + q * kCols + col) =
              make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if ((p.lse || kScores) && q == 0 && col == 0) {
          const float lse2 = d[z] == 0.f ? -INFINITY : m[z] + log2f(d[z]);
          if (p.lse) p.lse[at] = lse2 * 0.69314718055994530942f;
          if (kScores) w.lse2[at] = lse2;
        }
      } else {
        const size_t at = (size_t)(whole ? n * p.Hk + hk : place) * R + r;
        *reinterpret_cast<float4*>((whole ? w.own : w.part) + at * D + q * kCols + col) = acc;
        if (q == 0 && col == 0) (whole ? w.own_ml : w.part_ml)[at] = make_float2(m[z], d[z]);
      }
    }
  }
}

// The parts of a pair that spans CTAs, merged in the order of the keys; zeros for a row that
// saw no key. W warps a row take every W-th part; a CTA has W warps, or four with a row each.
template <int D, int W, int kUnit>
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
    c0 = cta_of(ub + kPair<kUnit>, U, grid);
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
// that the decode kernel left (a few bytes a key beside its K and V). Each warp takes an equal part
// of the list of 64-key pieces, two keys a lane. Bound: latency, a chain of lookups (unit numbers,
// page, scores, weights) for a few pieces a warp, so the next piece's loads are issued before this
// one's are used; and the instructions of a piece: the rows' denominators are one load, handed out by
// shuffles, and a place in the list comes from the one before it. 64 sequences of up to 4096 keys,
// bf16: 87.5 us with weights, 79.5 without (a load for each row's denominator, divisions for each
// place: 5 us more); 8 x 4 tokens in 8 bits 23.6 and 17.4.
// kRows rows are loaded side by side.
template <int kUnit, int kRows>
__global__ void __launch_bounds__(256, 3) weights_kernel(const AttnParams p, const DecodeParts w) {
  constexpr int kPieces = kUnit / 64;
  const int lane = threadIdx.x & 31, R = p.nq * p.G;
  pdl_wait();
  const uint64_t U = (uint64_t)w.first[p.N] * kPieces, W = gridDim.x * 8;
  const uint64_t me = blockIdx.x * 8 + (threadIdx.x >> 5);
  const uint32_t z0 = (uint32_t)(me * U / W), z1 = (uint32_t)((me + 1) * U / W);
  // The last unit looked up, its sequence, whose units are [at, end), c a key head.
  int last = -2, n = -1, at = 0, end = 0, c = 1, len = 0, hk = 0, chunk = 0;
  // Rows lane and lane + 32 of a pair, whose denominators the lane holds for all.
  const int row0 = lane < R ? lane / p.G * p.H + lane % p.G : -1;
  const int row1 = lane + 32 < R ? (lane + 32) / p.G * p.H + (lane + 32) % p.G : -1;
  struct Piece {
    const float* x;  // this lane's first score
    float l0, l1;
    int n, hk, key, len, page;
    bool live;
    float2 y[kRows];
  };
  auto rows = [&](Piece& a, int r0) {
    const float* x = a.x + (size_t)r0 * w.keys;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      a.y[r] = make_float2(-INFINITY, -INFINITY);
      if (a.live && r0 + r < R) a.y[r] = __ldcs(reinterpret_cast<const float2*>(x));
      x += w.keys;
    }
  };
  auto begin = [&](Piece& a, uint32_t z) {
    const int u = (int)(z / kPieces);
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
      hk = (u - at) / c;
      chunk = (u - at) - hk * c - kPair<kUnit>;
    } else if (u != last && ++chunk == c - kPair<kUnit>) {
      chunk = -kPair<kUnit>;
      ++hk;
    }
    last = u;
    a.n = n;
    a.hk = hk;
    a.len = len;
    a.key = chunk * kUnit + (int)(z % kPieces) * 64 + 2 * lane;
    a.live = chunk >= 0 && a.key < len;
    a.page = -1;
    if (a.live) a.page = p.table[(size_t)n * p.max_pages + (a.key >> p.page_shift)];
    a.x = w.scores + (size_t)(n * p.Hk + hk) * R * w.keys + a.key;
    rows(a, 0);
    const float* lse = w.lse2 + (size_t)n * p.nq * p.H + hk * p.G;
    a.l0 = row0 >= 0 ? lse[row0] : 0.f;
    a.l1 = row1 >= 0 ? lse[row1] : 0.f;
  };
  auto finish = [&](Piece& a) {
    float2 sum = make_float2(0.f, 0.f);
    for (int r0 = 0; r0 < R; r0 += kRows) {
      if (r0 > 0) rows(a, r0);
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float l = __shfl_sync(0xffffffffu, r0 < 32 ? a.l0 : a.l1, (r0 + r) & 31);
        // (a row that sees no key: -inf - -inf)
        sum.x += a.y[r].x == -INFINITY ? 0.f : ex2(a.y[r].x - l);
        sum.y += a.y[r].y == -INFINITY ? 0.f : ex2(a.y[r].y - l);
      }
    }
    if (a.page < 0 || a.page >= p.n_pages) return;
    float* to = p.weights + ((((size_t)a.page * p.Hk + a.hk) << p.page_shift) + (a.key & (p.page - 1)));
    const int fresh = a.len - p.nq;  // from here on keys are the call's own
    if (a.key >= fresh) to[0] = sum.x;
    else atomicAdd(to, sum.x);
    if (a.key + 1 < a.len) {
      if (a.key + 1 >= fresh) to[1] = sum.y;
      else atomicAdd(to + 1, sum.y);
    }
  };
  if (z0 >= z1) return;
  Piece a, b;
  begin(a, z0);
  for (uint32_t z = z0;;) {
    if (z + 1 < z1) begin(b, z + 1);
    finish(a);
    if (++z >= z1) break;
    if (z + 1 < z1) begin(a, z + 1);
    finish(b);
    if (++z >= z1) break;
  }
}

struct DecodeLayout {
  size_t first, part, part_ml, own, own_ml, prefix, prefix_ml, lse2, scores, total;
  int grid, splits;  // splits: of the prefix's keys, at most
};

// keys: of the page table where weights are wanted, else 0; ctas: of an SM
DecodeLayout layout(int T, int N, int H, int Hk, int D, int64_t keys = 0, int ctas = 2) {
  DecodeLayout L{};
  const int G = H / Hk, span = 2 * (kRows / G);
  const size_t R = (size_t)(T / N) * G, rows = (size_t)T * H;
  L.grid = ctas * num_sms();
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

// The merge of the parts, and the weights of the keys where they are wanted.
template <int D, int kUnit, bool kScores>
bool launch_rest(const AttnParams& p, const DecodeParts& w, cudaStream_t s) {
  // Warps of a merged row: eight while all their CTAs fit the GPU at once (a row has many
  // parts then: one sequence of 8191 keys 13.4 us with four, 12.5 with eight; 64 sequences,
  // 2048 rows, 157.0 with four, 159.6 with eight), four up to as many rows as those fit, one
  // beyond (64 sequences x 5 tokens x 64 heads behind 256 keys 46.7 us with four, 29.2 with one).
  const size_t rows = (size_t)p.T * p.H, sms = (size_t)num_sms();
  const int W = rows <= 8 * sms ? 8 : rows <= 32 * sms ? 4 : 1;
  const auto combine = W == 8   ? combine_kernel<D, 8, kUnit>
                       : W == 4 ? combine_kernel<D, 4, kUnit>
                                : combine_kernel<D, 1, kUnit>;
  if (launch_pdl(combine, dim3((unsigned)(W == 1 ? (rows + 3) / 4 : rows)), dim3(W == 8 ? 256 : 128), 0,
                 s, p, w) != cudaSuccess)
    return false;
  if (!kScores) return true;
  const auto weights = p.nq * p.G <= 4 ? weights_kernel<kUnit, 4> : weights_kernel<kUnit, 8>;
  return launch_pdl(weights, dim3(3 * num_sms()), dim3(256), 0, s, p, w) == cudaSuccess;
}

// Where the parts are in the workspace.
DecodeParts parts_of(const DecodeLayout& L, void* workspace) {
  char* ws = static_cast<char*>(workspace);
  DecodeParts w{};
  w.first = reinterpret_cast<int32_t*>(ws + L.first);
  w.part = reinterpret_cast<float*>(ws + L.part);
  w.part_ml = reinterpret_cast<float2*>(ws + L.part_ml);
  w.own = reinterpret_cast<float*>(ws + L.own);
  w.own_ml = reinterpret_cast<float2*>(ws + L.own_ml);
  w.prefix.o = reinterpret_cast<float*>(ws + L.prefix);
  w.prefix.ml = reinterpret_cast<float2*>(ws + L.prefix_ml);
  return w;
}

}  // namespace

}  // namespace gdn
