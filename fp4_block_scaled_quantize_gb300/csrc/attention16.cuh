// attention16.cuh -- attention of one new token per sequence over a paged cache
// (sm_103a):  out = sum_j w_j v_j,  w = softmax_j(scale q . k_j).
//
// Bound: HBM, every key and value of the seen positions read once for each 8 NT
// query heads that share them (4 D bytes per position and key head); at 6.8 TB/s an SM moves 23 bytes a clock, so the
// 2 x 8 NT MMAs per 16 positions are cheap even on the m16n8k16 path, and no
// part of the cache needs to pass through shared memory.
//
// Mathematics.  Scores in binary32 (times scale log2 e), a running maximum m
// and sum l per query head with weights 2^(s - m).  m is moved only when a
// score passes it by more than 8 (weights stay below 2^8): most steps then
// need no reduction over lanes and no rescaling.  A weight enters its product
// with the values as two 16-bit parts (hi + lo, 2^-16 of it left out; f16:
// 2^-32 of the largest if that is more) and the sum l as it is, so rounding
// weights costs no accuracy; the products are summed in binary32.  A warp that
// meets a value that is not finite goes over its part again with hi alone, for
// the sums that are not finite; the others keep the first pass.
//
// Layout.  Query heads that share a key head are the 8 columns of an MMA (NT
// tiles of 8), positions or head elements its 16 rows:
//   S^T = K Q^T   lane (g, t) loads 16-byte pieces 32 i + 8 t of keys g, g + 8
//   O^T = V^T P^T lane (g, t) loads 16-byte pieces 64 i + 8 g of values
//                 2 t, 2 t + 1, 2 t + 8, 2 t + 9 and pairs positions by byte
//                 permutes; P^T is transposed in registers (movmatrix)
// The order of k within an MMA is free, so both operands come from global
// memory in whole 16-byte pieces, straight into registers: the keys of the
// next 16 positions are requested as soon as this step's are multiplied, the
// values likewise, and page numbers a step ahead of both.
//
// Split.  The tiles (16 or 32 positions) of all (sequence, key head, head
// group) rows form one list that the warps of the resident CTAs share out
// evenly, whatever the lengths.  A warp writes the rows it holds whole; what
// it holds of others (at most two) is joined with the neighbours' in shared
// memory, and a CTA leaves at most two partial rows (m, l, O) in the
// workspace.  A second, dependent launch joins those in CTA order, so results
// repeat exactly.  Short rows go to clusters instead, which join in their
// shared memory (cluster_of).
// Measured: 64 sequences of up to 16384 positions, 32 heads over 8 of 128,
// BF16: 313 - 324 us (97 - 101% of a copy's rate); one of 131071: 87 us (91%),
// 3 us of them the join; 96 windows of 1000, 16 heads of 64: 76 - 84 us (62 -
// 68%: loads a step ahead in registers, which 12 warps an SM do not cover; a
// quarter of the issue slots is used), with 4 first positions before each 80; one
// of 300: 6.3 us in a graph (by one CTA 8.5).
#pragma once
#include <cooperative_groups.h>

#include "attention.cuh"

namespace fp4 {

namespace {

namespace cg = cooperative_groups;

// Groups of 16 positions a warp takes a step: what it keeps in flight.  When
// this was chosen, heads of 64, 96 windows of 1000: 82 us, with one group 88;
// heads of 128, 64 sequences: 329 us, with two groups and two CTAs an SM 332.
constexpr int units_of(int dp) { return dp <= 64 ? 2 : 1; }
constexpr int tile_of(int dp) { return 16 * units_of(dp); }

// CTAs an SM holds at least, by the kernel's launch bounds.
constexpr int per_sm(int dp, int nt) { return nt == 1 && dp <= 128 ? 3 : 2; }

template <typename T, int DP, int NT, bool UNITS, bool SINKS>
__global__ void __launch_bounds__(kThreads, per_sm(DP, NT))
    k_attention(const __grid_constant__ AtParams a) {
  constexpr int kCols = 8 * NT, kKey = DP / 32, kVal = DP / 64, kUnits = units_of(DP);
  constexpr int kTile = 16 * kUnits;
  // wide heads: keys and values take turns in the same registers
  constexpr bool kTurns = DP > 128;
  extern __shared__ __align__(16) float smem[];
  __shared__ int64_t scan[kWarps + 2];
  // parts of rows that a warp began or ended with: [2 kWarps][kCols][DP + 8]
  // outputs, [2 kWarps][kCols] m, l, seen, 1, and whose they are
  constexpr int kParts = 2 * kWarps;
  float *const o_sh = smem;
  float4 *const st_sh = reinterpret_cast<float4 *>(smem + kParts * kCols * (DP + 8));
  float *const part = reinterpret_cast<float *>(st_sh + kParts * kCols);  // clusters: the CTA's partial row
  __shared__ int4 part_sh[kParts];  // sequence (-1: none), row, begins with it, ends with it
  const fp4_kv_cache &c = a.p.cache;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int D = c.head_dim, rows = c.kv_heads * a.groups;

  int64_t at, end, start;
  int s;
  dependent_wait();
  launch_dependents();
  if (lane < 2) part_sh[2 * warp + lane] = make_int4(-1, 0, 0, 0);
  __syncwarp();
  const int rank = a.direct ? blockIdx.x % a.direct : 0, mine_row = a.direct ? blockIdx.x / a.direct : 0;
  if (a.direct) {
    s = mine_row / rows;
    start = 0;
    const int tiles = span_of<SINKS>(a, s).tiles;
    at = (int64_t)(mine_row - s * rows) * tiles;
    end = at + (int64_t)tiles * (rank + 1) / a.direct;
    at += (int64_t)tiles * rank / a.direct;
  } else {
    const Found f = find<kThreads, SINKS>(a, rows, blockIdx.x, scan);
    s = f.seq;
    start = f.start;
    at = end = 0;
    if (blockIdx.x < f.ctas) {
      at = f.total * blockIdx.x / f.ctas;
      end = f.total * (blockIdx.x + 1) / f.ctas;
    }
  }
  // sequences that see nothing are in no slice: their rows are written here
  for (int e = a.direct ? s : blockIdx.x; e < c.seqs; e += a.direct ? c.seqs : a.ctas) {
    const int given = a.p.lengths[e];
    if (a.direct && (rank || mine_row != s * rows)) break;
    if (threadIdx.x == 0 && (given < 0 || given > (int64_t)c.seq_pages * c.page_size))
      raise_status(a.status, kStatusIndex);
    if (span_of<SINKS>(a, e).tiles) continue;
    const float zero[8] = {};
    for (int i = threadIdx.x; i < a.p.heads * (D / 8); i += kThreads) {
      const int head = i / (D / 8), d = 8 * (i % (D / 8));
      store8<T>(a, e, head, d, zero);
      if (a.p.lse && d == 0) a.p.lse[(int64_t)e * a.p.heads + head] = -INFINITY;
    }
  }

  // each warp takes a quarter of the slice, row by row, by itself
  {
    const int64_t n = end - at;
    end = at + n * (warp + 1) / kWarps;
    at += n * warp / kWarps;
  }
  bool bad = false;  // a page outside the cache was met: reported at the end, not in the loop's way
  while (at < end) {
    const Span sp = span_of<SINKS>(a, s);
    const int64_t mine = (int64_t)rows * sp.tiles;
    if (at >= start + mine) {  // on to the next sequence
      start += mine;
      ++s;
      continue;
    }
    const int row = (int)((at - start) / sp.tiles), tile0 = (int)(at - start - (int64_t)row * sp.tiles);
    const int tile1 = (int)min((int64_t)sp.tiles, tile0 + (end - at));
    const int kvh = row / a.groups, head0 = kvh * a.share + (row - kvh * a.groups) * kCols;
    const int heads = min(kCols, (kvh + 1) * a.share - head0);
    at += tile1 - tile0;

    // queries: heads past the group's repeat as zero
    uint4 q[NT][kKey];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < kKey; ++i) {
        const int d = 32 * i + 8 * t;
        q[n][i] = 8 * n + g < heads && d < D
                      ? load16(static_cast<const T *>(a.p.q) + s * a.p.q_seq + (head0 + 8 * n + g) * a.p.q_head + d)
                      : make_uint4(0, 0, 0, 0);
      }

    float m[NT][2], l[NT][2], o[NT][kVal][4][4];
    bool seen;
    const int32_t *table = c.table + s * c.table_stride;
    // Where the 16 positions of a unit lie.  UNITS (pages of whole units):
    // all on one page, the same for every lane.  Else lane i & 15 holds
    // position i's offsets in keys and values.  Bit i of on: position i is
    // seen and its page exists.
    struct Where {
      int64_t k, v;
      uint32_t on;
    };
    int page_next[kUnits];  // UNITS: page numbers a step ahead (their loads are not waited for)
    // position where a tile starts, and what of it and behind it is seen (SINKS are a
    // form of their own: one for both took up to 4.5% more without first positions,
    // one sequence of 4000 14.5 us for 13.9)
    const int stop = min(sp.len, sp.base + kTile * tile1);
    auto tile_at = [&](int tile, int &lo, int &hi) {
      if (!SINKS) {
        lo = sp.from, hi = stop;
        return sp.base + kTile * tile;
      }
      const int pos = sp.start(tile, kTile, lo, hi);
      if (tile >= tile1) hi = 0;
      return pos;
    };
    auto ask = [&](int tile) {
      int lo, hi;
      const int pos = tile_at(tile, lo, hi);
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const int first = pos + 16 * u;
        page_next[u] = -1;
        if (UNITS) {
          if (first < hi) page_next[u] = table[a.shift >= 0 ? first >> a.shift : first / c.page_size];
        } else {
          const int i = first + (lane & 15);
          if (i >= lo && i < hi) page_next[u] = table[i / c.page_size];
        }
      }
    };
    auto where = [&](Where (&w)[kUnits], int tile) {
      int lo, hi;
      const int pos = tile_at(tile, lo, hi);
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const int first = pos + 16 * u;
        const int page = page_next[u];
        const bool ok = page >= 0 && page < c.pages;
        if (UNITS) {
          const int place = a.shift >= 0 ? first & (c.page_size - 1) : first % c.page_size;
          w[u].k = (int64_t)page * c.k_page + (int64_t)place * c.k_place;
          w[u].v = (int64_t)page * c.v_page + (int64_t)place * c.v_place;
          w[u].on = 0xFFFFu;
          if (first < lo) w[u].on &= 0xFFFFu << (lo - first);  // base <= from < base + 16
          if (first + 16 > hi) w[u].on &= (1u << max(hi - first, 0)) - 1;
          if (!ok) {
            bad |= w[u].on != 0;
            w[u].on = 0;
          }
        } else {
          const int i = first + (lane & 15);
          const bool in = i >= lo && i < hi;
          bad |= in && !ok;
          const int place = i % c.page_size;
          w[u].k = (int64_t)page * c.k_page + (int64_t)place * c.k_place;
          w[u].v = (int64_t)page * c.v_page + (int64_t)place * c.v_place;
          w[u].on = __ballot_sync(~0u, in && ok) & 0xFFFFu;
        }
      }
    };
    const bool exact = D == DP;  // no head element is padding
    const T *const keys = static_cast<const T *>(c.k) + kvh * c.k_head + 8 * t;
    const T *const values = static_cast<const T *>(c.v) + kvh * c.v_head + 8 * g;
    uint4 key[kUnits][2][kKey], val[kUnits][4][kVal];
    Where now[kUnits], next[kUnits];
    // What is not seen is not read: zeros, which its zero weights then meet.
    auto load_keys = [&](const Where (&w)[kUnits]) {
#pragma unroll
      for (int u = 0; u < kUnits; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int i = g + 8 * h;
          const T *k = keys + (UNITS ? w[u].k + i * c.k_place : __shfl_sync(~0u, w[u].k, i));
          if (exact && w[u].on == 0xFFFFu) {
#pragma unroll
            for (int e = 0; e < kKey; ++e) key[u][h][e] = load16(k + 32 * e);
          } else {
            const bool on = w[u].on >> i & 1;
#pragma unroll
            for (int e = 0; e < kKey; ++e)
              key[u][h][e] = on && 32 * e + 8 * t < D ? load16(k + 32 * e) : make_uint4(0, 0, 0, 0);
          }
        }
    };
    auto load_values = [&](const Where (&w)[kUnits]) {
#pragma unroll
      for (int u = 0; u < kUnits; ++u)
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int i = 2 * t + (h & 1) + 8 * (h >> 1);
          const T *v = values + (UNITS ? w[u].v + i * c.v_place : __shfl_sync(~0u, w[u].v, i));
          if (exact && w[u].on == 0xFFFFu) {
#pragma unroll
            for (int e = 0; e < kVal; ++e) val[u][h][e] = load16(v + 64 * e);
          } else {
            const bool on = w[u].on >> i & 1;
#pragma unroll
            for (int e = 0; e < kVal; ++e)
              val[u][h][e] = on && 64 * e + 8 * g < D ? load16(v + 64 * e) : make_uint4(0, 0, 0, 0);
          }
        }
    };

    // A value that is not finite makes lo x value a NaN where hi x value is an
    // infinity: a warp with a sum that is not finite repeats its part without
    // lo, and takes from that pass what was not finite in the first.
    const int at_part = 2 * warp + (tile0 == 0);  // the warp's first row, or its last
    // the place of this row's part, outputs 64 i + 8 g ... of column 8 n + 2 t + e
    auto part_at = [&](int n, int e, int i) {
      int place = (at_part * kCols + 2 * t) * (DP + 8) + 8 * g;
      return reinterpret_cast<float4 *>(o_sh + place + (8 * n + e) * (DP + 8) + 64 * i);
    };
    for (bool both = true;; both = false) {
    seen = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.0f;
#pragma unroll
      for (int i = 0; i < kVal; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[n][i][j][0] = o[n][i][j][1] = o[n][i][j][2] = o[n][i][j][3] = 0.0f;
    }
    ask(tile0);
    where(now, tile0);
    ask(tile0 + 1);
    load_keys(now);
    if (!kTurns) load_values(now);
    for (int tile = tile0; tile < tile1; ++tile) {
      float sc[kUnits][NT][4];
#pragma unroll
      for (int u = 0; u < kUnits; ++u)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          sc[u][n][0] = sc[u][n][1] = sc[u][n][2] = sc[u][n][3] = 0.0f;
#pragma unroll
          for (int i = 0; i < kKey; ++i) {
            const uint4 &k0 = key[u][0][i], &k1 = key[u][1][i];
            mma(sc[u][n], k0.x, k1.x, k0.y, k1.y, q[n][i].x, q[n][i].y, T());
            mma(sc[u][n], k0.z, k1.z, k0.w, k1.w, q[n][i].z, q[n][i].w, T());
          }
        }
      where(next, tile + 1);
      ask(tile + 2);
      if (kTurns)
        load_values(now);
      else
        load_keys(next);
      // weights: lane (g, t) has positions g, g + 8 of heads 2 t, 2 t + 1
      float base[NT][2];
      bool passed = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          base[n][e] = m[n][e] == -INFINITY ? 0.0f : m[n][e];
          passed |= m[n][e] == -INFINITY;
        }
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        seen |= now[u].on != 0;
        const bool on0 = now[u].on >> g & 1, on1 = now[u].on >> (g + 8) & 1;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // (log2 of the weight; -inf: not seen)
            sc[u][n][e] = (e >> 1 ? on1 : on0) ? sc[u][n][e] * a.scale2 : -INFINITY;
            passed |= sc[u][n][e] > base[n][e & 1] + kSlack;
          }
      }
      if (__any_sync(~0u, passed)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = m[n][e];
#pragma unroll
            for (int u = 0; u < kUnits; ++u) top = fmaxf(top, fmaxf(sc[u][n][e], sc[u][n][2 + e]));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 4));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
            const float fade = ex2(m[n][e] - (top == -INFINITY ? 0.0f : top));
            m[n][e] = top;
            base[n][e] = top == -INFINITY ? 0.0f : top;
            l[n][e] *= fade;
#pragma unroll
            for (int i = 0; i < kVal; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                o[n][i][j][e] *= fade;
                o[n][i][j][2 + e] *= fade;
              }
          }
      }
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            w[e] = ex2(sc[u][n][e] - (base[n][e & 1] - lift<T>()));
            l[n][e & 1] += w[e];
          }
          if (!Bf16<T>::value && !both)  // a weight that f16 would round to zero still meets an infinity
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = w[e] > 0.0f ? fmaxf(w[e], 0x1p-24f) : w[e];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t p = pack<T>(w[2 * h], w[2 * h + 1]);
            const float2 r = unpack<T>(p);
            hi[n][h] = transpose8x8(p);
            lo[n][h] = transpose8x8(pack<T>(w[2 * h] - r.x, w[2 * h + 1] - r.y));
          }
        }
#pragma unroll
        for (int i = 0; i < kVal; ++i) {
          const uint32_t *v0 = reinterpret_cast<const uint32_t *>(&val[u][0][i]);
          const uint32_t *v1 = reinterpret_cast<const uint32_t *>(&val[u][1][i]);
          const uint32_t *v2 = reinterpret_cast<const uint32_t *>(&val[u][2][i]);
          const uint32_t *v3 = reinterpret_cast<const uint32_t *>(&val[u][3][i]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // rows g, g + 8: elements 2 j, 2 j + 1 of the lane's piece
            const uint32_t a0 = __byte_perm(v0[j], v1[j], 0x5410), a1 = __byte_perm(v0[j], v1[j], 0x7632);
            const uint32_t a2 = __byte_perm(v2[j], v3[j], 0x5410), a3 = __byte_perm(v2[j], v3[j], 0x7632);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma(o[n][i][j], a0, a1, a2, a3, hi[n][0], hi[n][1], T());
              if (both) mma(o[n][i][j], a0, a1, a2, a3, lo[n][0], lo[n][1], T());
            }
          }
        }
      }
      if (kTurns)
        load_keys(next);
      else
        load_values(next);
#pragma unroll
      for (int u = 0; u < kUnits; ++u) now[u] = next[u];
    }
    float worst = 0.0f;  // NaN if a sum is not finite
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < kVal; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) worst = fmaf(o[n][i][j][e], 0.0f, worst);
    if (__builtin_expect(both && !__any_sync(~0u, worst != 0.0f), 1)) break;
    // a lane's own values, so nothing has to be waited for
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < kVal; ++i) {
          float4 *const at = part_at(n, e, i);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float *const v[4] = {&o[n][i][2 * h][e], &o[n][i][2 * h][2 + e], &o[n][i][2 * h + 1][e],
                                 &o[n][i][2 * h + 1][2 + e]};
            if (both) {
              at[h] = make_float4(*v[0], *v[1], *v[2], *v[3]);
            } else {
              const float4 first = at[h];
              if (isfinite(first.x)) *v[0] = first.x;
              if (isfinite(first.y)) *v[1] = first.y;
              if (isfinite(first.z)) *v[2] = first.z;
              if (isfinite(first.w)) *v[3] = first.w;
            }
          }
        }
    if (!both) break;
    }

#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[n][e] += __shfl_xor_sync(~0u, l[n][e], 4);
        l[n][e] += __shfl_xor_sync(~0u, l[n][e], 8);
        l[n][e] += __shfl_xor_sync(~0u, l[n][e], 16);
      }
    if (tile0 == 0 && tile1 == sp.tiles) {  // the whole row
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = 8 * n + 2 * t + e;
          if (col >= heads) continue;
          const float w = seen ? 1.0f / l[n][e] : 0.0f;
#pragma unroll
          for (int i = 0; i < kVal; ++i) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v[2 * j] = o[n][i][j][e] * w;
              v[2 * j + 1] = o[n][i][j][2 + e] * w;
            }
            if (64 * i + 8 * g < D) store8<T>(a, s, head0 + col, 64 * i + 8 * g, v);
          }
          if (a.p.lse && g == 0) store_lse<T, false>(a, s, head0 + col, seen, m[n][e], l[n][e]);
        }
      continue;
    }
    if (lane == 0) part_sh[at_part] = make_int4(s, row, tile0 == 0, tile1 == sp.tiles);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = 8 * n + 2 * t + e;
        if (g == 0) st_sh[at_part * kCols + col] = make_float4(m[n][e], l[n][e], seen ? 1.0f : 0.0f, 1.0f);
#pragma unroll
        for (int i = 0; i < kVal; ++i) {
          part_at(n, e, i)[0] = make_float4(o[n][i][0][e], o[n][i][0][2 + e], o[n][i][1][e], o[n][i][1][2 + e]);
          part_at(n, e, i)[1] = make_float4(o[n][i][2][e], o[n][i][2][2 + e], o[n][i][3][e], o[n][i][3][2 + e]);
        }
      }
  }

  if (bad) raise_status(a.status, kStatusIndex);
  // join the warps' parts, row by row
  __syncthreads();
  const int4 mine = part_sh[lane % kParts];
  uint32_t there = __ballot_sync(~0u, mine.x >= 0) & ((1u << kParts) - 1);
  bool partial = false;
  while (there) {
    const int i0 = __ffs(there) - 1;
    const int s = __shfl_sync(~0u, mine.x, i0), row = __shfl_sync(~0u, mine.y, i0);
    const bool begins = __shfl_sync(~0u, mine.z, i0);
    const uint32_t parts = __ballot_sync(~0u, mine.x == s && mine.y == row) & there;
    const bool whole = begins && __shfl_sync(~0u, mine.w, 31 - __clz(parts));
    there &= ~parts;
    const int kvh = row / a.groups, head0 = kvh * a.share + (row - kvh * a.groups) * kCols;
    const int heads = min(kCols, (kvh + 1) * a.share - head0);
    float *slot = a.direct ? part : a.ws + (blockIdx.x * 2 + begins) * (int64_t)slot_floats(kCols, DP);
    partial = !whole;
    for (int item = threadIdx.x; item < heads * (DP / 8); item += kThreads) {
      const int col = item / (DP / 8), d = 8 * (item % (DP / 8));
      if (d >= D) continue;
      const Whole r = join_all<kParts, false>([&](int q, float4 &st, float4 &lo, float4 &hi) {
        if (!(parts >> q & 1)) return;
        const float *from = o_sh + (q * kCols + col) * (DP + 8) + d;
        st = st_sh[q * kCols + col];
        lo = *reinterpret_cast<const float4 *>(from);
        hi = *reinterpret_cast<const float4 *>(from + 4);
      });
      if (whole) {
        finish<T, false>(a, s, head0 + col, d, r.j, r.seen);
        continue;
      }
      const float *v = r.j.v;
      float *out = slot + col * DP + d;
      *reinterpret_cast<float4 *>(out) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4 *>(out + 4) = make_float4(v[4], v[5], v[6], v[7]);
      if (d == 0)
        *reinterpret_cast<float4 *>(slot + kCols * DP + col * 4) = make_float4(r.j.top, r.j.sum, r.seen ? 1.0f : 0.0f, 1.0f);
    }
  }
  if (a.direct < 2) return;

  // join the cluster's partial rows, an output piece a thread, in CTA order
  if (!partial)
    for (int i = threadIdx.x; i < slot_floats(kCols, DP); i += kThreads)
      part[i] = i >= kCols * DP && i % 4 == 0 ? -INFINITY : 0.0f;
  cg::this_cluster().sync();
  const int row = mine_row - s * rows, kvh = row / a.groups, head0 = kvh * a.share + (row - kvh * a.groups) * kCols;
  const int heads = min(kCols, (kvh + 1) * a.share - head0);
  for (int item = threadIdx.x * a.direct + rank; item < heads * (DP / 8); item += kThreads * a.direct) {
    const int col = item / (DP / 8), d = 8 * (item % (DP / 8));
    if (d >= D) continue;
    const Whole r = join_all<kCluster, false>([&](int q, float4 &st, float4 &lo, float4 &hi) {
      if (q >= a.direct) return;
      const float *from = cg::this_cluster().map_shared_rank(part, q);
      st = *reinterpret_cast<const float4 *>(from + kCols * DP + col * 4);
      lo = *reinterpret_cast<const float4 *>(from + col * DP + d);
      hi = *reinterpret_cast<const float4 *>(from + col * DP + d + 4);
    });
    if (r.there) finish<T, false>(a, s, head0 + col, d, r.j, r.seen);
  }
  cg::this_cluster().sync();  // nobody leaves while its part may be read
}

// CTAs (a cluster) that take a row of up to `reach` positions between them,
// joined in their shared memory: no workspace and no second launch.  0: equal
// slices.  As many as leave a warp two tiles (one, if each has an SM to
// itself) and are resident at once (7/8: clusters leave some places empty).  A row longer than the others keeps its
// CTAs to itself, so slices take over where they are as fast for equal rows.
// Measured, 32 heads over 8 of 128, us as clusters of 1, 2, 4, 8 / as slices:
//   1 sequence    of  200:  7.7,  7.1,  6.5,  6.2 /  7.1   (1000, 8: 8.0 / 8.6; 2000, 8: 10.9 / 10.6)
//   8 sequences   of  500: 15.1, 11.2, 10.8,   -  / 14.0   (1000, 4: 14.2 / 16.3; 2000, 4: 20.8 / 20.8)
//   16 sequences  of  500: 15.7, 14.0,   -     -  / 16.2   (1000, 2: 20.6 / 20.9; 128, 1: 7.4, 2: 8.8)
//   50 sequences  of  200: 13.7,   -     -     -  / 17.4   (500, 1: 23.1 / 27.2)
// Rows that fill the GPU more than once are left to slices earlier (64
// sequences of 512: 32 us, a CTA per row 38).
int cluster_of(int64_t rows, int64_t reach, int dp, int nt) {
  const int64_t sms = sm_count(), fit = sms * per_sm(dp, nt);
  int n = 1;
  while (n < kCluster && rows * 2 * n <= fit * 7 / 8 &&
         (rows * 2 * n <= sms ? n : 2 * n) * kWarps * tile_of(dp) < reach)
    n *= 2;
  const int64_t most = rows > fit ? 128 : n == kCluster ? 2048 : 384 * n;
  return reach <= most ? n : 0;
}

template <typename T, int DP, int NT, bool UNITS, bool SINKS>
fp4_status launch(AtParams a, cudaStream_t s) {
  constexpr int kMaxDev = 64;
  static std::atomic<int> occupancy[kMaxDev];
  constexpr int cols = 8 * NT;
  constexpr size_t smem = (2 * kWarps * cols * (DP + 8) + 8 * kWarps * cols) * sizeof(float);
  constexpr size_t part = slot_floats(cols, DP) * sizeof(float);
  auto kern = k_attention<T, DP, NT, UNITS, SINKS>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return FP4_ERR_CUDA;
  int per = occupancy[dev].load(std::memory_order_acquire);
  if (!per) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(smem + part)) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, kThreads, smem) != cudaSuccess || per < 1)
      return FP4_ERR_CUDA;
    occupancy[dev].store(per, std::memory_order_release);
  }
  const fp4_kv_cache &c = a.p.cache;
  a.tile = tile_of(DP);
  a.least = kWarps;
  a.bundle = 1;
  // no more CTAs than the table has tiles
  const int64_t rows = (int64_t)c.seqs * c.kv_heads * a.groups;
  const int64_t room = (int64_t)c.seq_pages * c.page_size;
  const int64_t most = (int64_t)sm_count() * (per < kPerSM ? per : kPerSM);
  const int64_t tiles = ceil_div(rows * ceil_div(room, a.tile), kWarps);
  if (rows > INT32_MAX) return FP4_ERR_SHAPE;
  const int64_t reach = (int64_t)a.p.window + 15 + ceil_div(a.p.sinks, a.tile) * a.tile;
  a.direct = cluster_of(rows, a.p.window && reach < room ? reach : room, DP, NT);
  if (!a.direct && !a.ws) return FP4_ERR_INVALID_ARG;  // (where rows of `room` have CTAs of their own, shorter ones do)
  a.ctas = (int)(a.direct ? rows * a.direct : tiles < most ? tiles : most);
  // Rows of their own may start early.  Equal slices may not: their CTAs would be
  // placed around those that still run, two on one SM and none on another
  // (64 sequences of up to 16384: 435 us for 317).
  if (a.direct) {
    const size_t bytes = smem + (a.direct > 1 ? part : 0);
    return launch_dependent_clusters(kern, a.direct, dim3((unsigned)a.ctas), dim3(kThreads), bytes, s, a) == cudaSuccess
               ? FP4_OK
               : FP4_ERR_CUDA;
  }
  kern<<<(unsigned)a.ctas, kThreads, smem, s>>>(a);
  if (cudaGetLastError() != cudaSuccess) return FP4_ERR_CUDA;
  if (a.ctas < 2) return FP4_OK;
  const cudaError_t e =
      rows * 4 <= a.ctas
          ? launch_dependent(k_attention_join<T, DP, NT, kWide, SINKS, false>, dim3((unsigned)rows), dim3(kWide), 0, s, a)
          : launch_dependent(k_attention_join<T, DP, NT, kNarrow, SINKS, false>, dim3((unsigned)a.ctas - 1), dim3(kNarrow), 0, s, a);
  return e == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

template <typename T, int DP, int NT, bool SINKS>
fp4_status launch_pages(const AtParams &a, cudaStream_t s) {
  return a.p.cache.page_size % 16 == 0 ? launch<T, DP, NT, true, SINKS>(a, s) : launch<T, DP, NT, false, SINKS>(a, s);
}

template <typename T, bool SINKS>
fp4_status launch_type(const AtParams &a, int nt, cudaStream_t s) {
  switch (dp_of(a.p.cache.head_dim)) {
    case 64: return nt == 1 ? launch_pages<T, 64, 1, SINKS>(a, s) : launch_pages<T, 64, 2, SINKS>(a, s);
    case 128: return nt == 1 ? launch_pages<T, 128, 1, SINKS>(a, s) : launch_pages<T, 128, 2, SINKS>(a, s);
    case 192: return launch_pages<T, 192, 1, SINKS>(a, s);
    default: return launch_pages<T, 256, 1, SINKS>(a, s);
  }
}

// Without first positions (SINKS false) the kernels are those that know of none.
template <bool SINKS>
fp4_status launch_attention(const fp4_attention_params &p, cudaStream_t s) {
  AtParams a{};
  a.p = p;
  a.status = status_word();
  if (!a.status) return FP4_ERR_CUDA;
  const fp4_kv_cache &c = p.cache;
  a.share = p.heads / c.kv_heads;
  const int nt = nt_of(a.share, dp_of(c.head_dim));
  a.groups = (a.share + 8 * nt - 1) / (8 * nt);
  a.shift = log2_or(c.page_size, -1);
  a.out16 = aligned16(p.out) && p.out_seq % 8 == 0 && p.out_head % 8 == 0;
  a.scale2 = p.scale * 1.44269504088896f;
  a.ws = static_cast<float *>(p.workspace);
  return c.type == FP4_BF16 ? launch_type<__nv_bfloat16, SINKS>(a, nt, s) : launch_type<__half, SINKS>(a, nt, s);
}

}  // namespace

}  // namespace fp4
