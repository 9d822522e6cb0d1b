// attention.cu -- attention of one new token per sequence over a paged cache
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
// quarter of the issue slots is used); one of 300: 6.3 us in a graph (by one CTA
// 8.5).
#include <cooperative_groups.h>

#include <cmath>

#include "serve.cuh"

namespace fp4 {

namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
// Groups of 16 positions a warp takes a step: what it keeps in flight.  When
// this was chosen, heads of 64, 96 windows of 1000: 82 us, with one group 88;
// heads of 128, 64 sequences: 329 us, with two groups and two CTAs an SM 332.
constexpr int units_of(int dp) { return dp <= 64 ? 2 : 1; }
constexpr int tile_of(int dp) { return 16 * units_of(dp); }
constexpr int kPerSM = 5;            // CTAs per SM at most (workspace bound)
constexpr int kCluster = 8;          // CTAs that take a row between them, at most
constexpr float kSlack = 8.0f;       // log2 by which scores may pass the maximum in use

struct AtParams {
  fp4_attention_params p;
  int groups;   // head groups of a key head: ceil(heads / kv_heads / (8 NT))
  int share;    // heads / kv_heads
  int tile;     // positions of a tile: 16 per unit
  int ctas;     // CTAs of the main kernel
  int direct;   // CTAs (a cluster) that take a row between them, or 0: equal slices
  int shift;    // log2 page_size, or -1: no power of two
  int out16;    // rows of out allow 16-byte stores
  float scale2; // scale * log2 e
  float *ws;    // [ctas][2] partial rows
  uint32_t *status;
};

// Partial row: 8 NT x DP outputs, then m, l, seen (1.0 or 0.0) and whether
// there is one (clusters) per head.
constexpr int slot_floats(int cols, int dp) { return cols * (dp + 3 + 1); }

__device__ __forceinline__ void mma(float *d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1, __nv_bfloat16) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma(float *d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1, __half) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <typename T>
struct Bf16 {
  static constexpr bool value = false;
};
template <>
struct Bf16<__nv_bfloat16> {
  static constexpr bool value = true;
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint4 load16(const void *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Weights are held 2^lift times as large: f16's smallest is 2^-24, and a long
// context may have most of its weight in small ones.
template <typename T>
__device__ __forceinline__ constexpr float lift() {
  return Bf16<T>::value ? 0.0f : 7.0f;
}

// Two values as a pair of T, and what the pair leaves of them.
template <typename T>
__device__ __forceinline__ uint32_t pack(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
template <typename T>
__device__ __forceinline__ float2 unpack(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack<__nv_bfloat16>(uint32_t w) {
  return make_float2(bf16_lo(w), bf16_hi(w));
}
template <>
__device__ __forceinline__ float2 unpack<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// What of a sequence is seen: positions [from, len); its tiles start at base.
struct Span {
  int from, len, base, tiles;
};
__device__ __forceinline__ Span span_of(const AtParams &a, int s) {
  const fp4_kv_cache &c = a.p.cache;
  const int64_t room = (int64_t)c.seq_pages * c.page_size;  // fits 32 bits
  const int given = a.p.lengths[s];
  Span r;
  r.len = given < 0 ? 0 : given > room ? (int)room : given;
  r.from = a.p.window && r.len > a.p.window ? r.len - a.p.window : 0;
  r.base = r.from & ~15;
  r.tiles = (r.len - r.base + a.tile - 1) / a.tile;
  return r;
}

// Prefix over the sequences: the sum of rows * tiles of all, and the sequence
// in which a slice of the list begins (or the sequence `which`).
struct Found {
  int64_t total, start;  // start: list index of the found sequence's first tile
  int64_t ctas;          // CTAs that share the list: a tile or more for each warp
  int seq;
};
template <int THREADS>
__device__ Found find(const AtParams &a, int rows, int64_t slice, int64_t *shared, int which = -1) {
  constexpr int kW = THREADS / 32;
  const int seqs = a.p.cache.seqs, per = (seqs + THREADS - 1) / THREADS;
  if (seqs <= 32) {  // each warp by itself
    const int lane = threadIdx.x & 31;
    const int64_t sum = lane < seqs ? (int64_t)rows * span_of(a, lane).tiles : 0;
    int64_t inc = sum;
    for (int o = 1; o < seqs; o <<= 1) {
      const int64_t v = __shfl_up_sync(~0u, inc, o);
      if (lane >= o) inc += v;
    }
    Found f;
    f.total = __shfl_sync(~0u, inc, seqs - 1);
    f.ctas = min((int64_t)a.ctas, (f.total + kWarps - 1) / kWarps);
    const int64_t x = slice < f.ctas ? f.total * slice / f.ctas : f.total;
    const uint32_t hit = __ballot_sync(~0u, which < 0 ? x >= inc - sum && x < inc : lane == which);
    f.seq = hit ? __ffs(hit) - 1 : seqs;
    f.start = hit ? __shfl_sync(~0u, inc - sum, f.seq) : f.total;
    return f;
  }
  const int s0 = threadIdx.x * per, s1 = min(s0 + per, seqs);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t sum = 0;
  for (int s = s0; s < s1; ++s) sum += (int64_t)rows * span_of(a, s).tiles;
  int64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(~0u, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) shared[warp] = inc;
  __syncthreads();
  int64_t before = inc - sum, total = 0;
#pragma unroll
  for (int w = 0; w < kW; ++w) {
    if (w < warp) before += shared[w];
    total += shared[w];
  }
  const int64_t ctas = min((int64_t)a.ctas, (total + kWarps - 1) / kWarps);
  const int64_t x = slice < ctas ? total * slice / ctas : total;
  if (which < 0 ? x >= before && x < before + sum : which >= s0 && which < s1) {  // one thread, if any
    int64_t at = before;
    for (int s = s0;; ++s) {
      const int64_t n = (int64_t)rows * span_of(a, s).tiles;
      if (which < 0 ? x < at + n : s == which) {
        shared[kW] = s;
        shared[kW + 1] = at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  Found f;
  f.total = total;
  f.ctas = ctas;
  const bool found = which >= 0 || slice < ctas;
  f.seq = found ? (int)shared[kW] : seqs;
  f.start = found ? shared[kW + 1] : total;
  return f;
}

// Eight outputs of a row, rounded once.
template <typename T>
__device__ __forceinline__ void store8(const AtParams &a, int s, int head, int d, const float *v) {
  T *out = static_cast<T *>(a.p.out) + s * a.p.out_seq + head * a.p.out_head + d;
  if (a.out16) {
    *reinterpret_cast<uint4 *>(out) = make_uint4(pack<T>(v[0], v[1]), pack<T>(v[2], v[3]),
                                                 pack<T>(v[4], v[5]), pack<T>(v[6], v[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = from_f32<T>(v[i]);
  }
}

// log sum exp of a row: m + log2 l in base 2.
template <typename T>
__device__ __forceinline__ void store_lse(const AtParams &a, int s, int head, bool seen, float m, float l) {
  a.p.lse[(int64_t)s * a.p.heads + head] =
      seen ? ((m == -INFINITY ? 0.0f : m) + log2f(l) - lift<T>()) * 0.693147180559945f : -INFINITY;
}

// Eight outputs of a row joined from parts, one for each bit of `parts`:
// m(i), l(i) are part i's statistics, add(i, w, v) adds w times its outputs.
struct Joined {
  float top, sum, v[8];
};
template <typename M, typename L, typename Add>
__device__ __forceinline__ Joined join(uint32_t parts, M m, L l, Add add) {
  Joined j;
  j.top = -INFINITY;
  j.sum = 0.0f;
  for (uint32_t p = parts; p; p &= p - 1) j.top = fmaxf(j.top, m(__ffs(p) - 1));
  const float base = j.top == -INFINITY ? 0.0f : j.top;
#pragma unroll
  for (int e = 0; e < 8; ++e) j.v[e] = 0.0f;
  for (uint32_t p = parts; p; p &= p - 1) {
    const int i = __ffs(p) - 1;
    const float w = ex2(m(i) - base);
    j.sum = fmaf(w, l(i), j.sum);
    add(i, w, j.v);
  }
  return j;
}
// The same of parts held side by side: get(q, st, lo, hi) reads part q (m, l,
// seen, 1 and the outputs) if there is one.  All are requested together.
struct Whole {
  Joined j;
  bool seen, there;
};
template <int N, typename Get>
__device__ __forceinline__ Whole join_all(Get get) {
  float4 st[N], lo[N], hi[N];
#pragma unroll
  for (int q = 0; q < N; ++q) {
    st[q] = make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
    lo[q] = hi[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    get(q, st[q], lo[q], hi[q]);
  }
  Whole r = {};
  r.j.top = -INFINITY;
#pragma unroll
  for (int q = 0; q < N; ++q) {
    r.j.top = fmaxf(r.j.top, st[q].x);
    r.seen |= st[q].z != 0.0f;
    r.there |= st[q].w != 0.0f;
  }
  const float base = r.j.top == -INFINITY ? 0.0f : r.j.top;
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const float w = ex2(st[q].x - base);
    r.j.sum = fmaf(w, st[q].y, r.j.sum);
    const float v[8] = {lo[q].x, lo[q].y, lo[q].z, lo[q].w, hi[q].x, hi[q].y, hi[q].z, hi[q].w};
#pragma unroll
    for (int e = 0; e < 8; ++e) r.j.v[e] = fmaf(w, v[e], r.j.v[e]);
  }
  return r;
}
// Writes the result of a row that saw something (seen) or nothing.
template <typename T>
__device__ __forceinline__ void finish(const AtParams &a, int s, int head, int d, Joined j, bool seen) {
  const float w = seen ? 1.0f / j.sum : 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) j.v[e] *= w;
  store8<T>(a, s, head, d, j.v);
  if (a.p.lse && d == 0) store_lse<T>(a, s, head, seen, j.top, j.sum);
}

// CTAs an SM holds at least, by the kernel's launch bounds.
constexpr int per_sm(int dp, int nt) { return nt == 1 && dp <= 128 ? 3 : 2; }

template <typename T, int DP, int NT, bool UNITS>
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
    const int tiles = span_of(a, s).tiles;
    at = (int64_t)(mine_row - s * rows) * tiles;
    end = at + (int64_t)tiles * (rank + 1) / a.direct;
    at += (int64_t)tiles * rank / a.direct;
  } else {
    const Found f = find<kThreads>(a, rows, blockIdx.x, scan);
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
    if (span_of(a, e).tiles) continue;
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
  while (at < end) {
    const Span sp = span_of(a, s);
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
    const int stop = min(sp.len, sp.base + kTile * tile1);
    // Where the 16 positions of a unit lie.  UNITS (pages of whole units):
    // all on one page, the same for every lane.  Else lane i & 15 holds
    // position i's offsets in keys and values.  Bit i of on: position i is
    // seen and its page exists.
    struct Where {
      int64_t k, v;
      uint32_t on;
    };
    int page_next[kUnits];  // UNITS: page numbers a step ahead (their loads are not waited for)
    auto ask = [&](int pos) {
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const int first = pos + 16 * u;
        page_next[u] = -1;
        if (UNITS) {
          if (first < stop) page_next[u] = table[a.shift >= 0 ? first >> a.shift : first / c.page_size];
        } else {
          const int i = first + (lane & 15);
          if (i >= sp.from && i < stop) page_next[u] = table[i / c.page_size];
        }
      }
    };
    auto where = [&](Where (&w)[kUnits], int pos) {
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
          if (first < sp.from) w[u].on &= 0xFFFFu << (sp.from - first);  // base <= from < base + 16
          if (first + 16 > stop) w[u].on &= (1u << max(stop - first, 0)) - 1;
          if (!ok) {
            if (w[u].on && lane == 0) raise_status(a.status, kStatusIndex);
            w[u].on = 0;
          }
        } else {
          const int i = first + (lane & 15);
          const bool in = i >= sp.from && i < stop;
          if (in && !ok && lane < 16) raise_status(a.status, kStatusIndex);
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
    int pos = sp.base + kTile * tile0;
    ask(pos);
    where(now, pos);
    ask(pos + kTile);
    load_keys(now);
    if (!kTurns) load_values(now);
    for (; pos < stop; pos += kTile) {
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
      where(next, pos + kTile);
      ask(pos + 2 * kTile);
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
          if (a.p.lse && g == 0) store_lse<T>(a, s, head0 + col, seen, m[n][e], l[n][e]);
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
      const Whole r = join_all<kParts>([&](int q, float4 &st, float4 &lo, float4 &hi) {
        if (!(parts >> q & 1)) return;
        const float *from = o_sh + (q * kCols + col) * (DP + 8) + d;
        st = st_sh[q * kCols + col];
        lo = *reinterpret_cast<const float4 *>(from);
        hi = *reinterpret_cast<const float4 *>(from + 4);
      });
      if (whole) {
        finish<T>(a, s, head0 + col, d, r.j, r.seen);
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
    const Whole r = join_all<kCluster>([&](int q, float4 &st, float4 &lo, float4 &hi) {
      if (q >= a.direct) return;
      const float *from = cg::this_cluster().map_shared_rank(part, q);
      st = *reinterpret_cast<const float4 *>(from + kCols * DP + col * 4);
      lo = *reinterpret_cast<const float4 *>(from + col * DP + d);
      hi = *reinterpret_cast<const float4 *>(from + col * DP + d + 4);
    });
    if (r.there) finish<T>(a, s, head0 + col, d, r.j, r.seen);
  }
  cg::this_cluster().sync();  // nobody leaves while its part may be read
}

// Joins partial rows.  Many rows are cut into few parts each: narrow CTAs, of
// which CTA c takes the row in which slice c + 1 begins, if it began in slice
// c (so every cut row has one).  Few rows are cut into many: wide CTAs, one
// for each row.  Which parts a row has follows from the lengths, which are read
// before the main grid is waited for: that grid is an ordinary launch, so what
// came before it on the stream is complete.  A CTA's threads take eight outputs each, in groups
// that walk every kGroups-th part four at a time; the first joins the groups.
constexpr int kNarrow = 128, kWide = 1024;
template <typename T, int DP, int NT, int THREADS>
__global__ void __launch_bounds__(THREADS) k_attention_join(const __grid_constant__ AtParams a) {
  constexpr int kCols = 8 * NT, kItems = kCols * DP / 8;
  constexpr int kGroups = THREADS < kItems ? 1 : THREADS / kItems;
  __shared__ int64_t scan[THREADS / 32 + 2];
  __shared__ float part_sh[kGroups][11][kItems];  // m, l, seen, eight outputs
  const fp4_kv_cache &c = a.p.cache;
  const int rows = c.kv_heads * a.groups, slice = blockIdx.x + 1;
  const Found f = THREADS == kNarrow ? find<THREADS>(a, rows, slice, scan)
                                     : find<THREADS>(a, rows, 0, scan, blockIdx.x / rows);
  int s = f.seq, row = 0, first = 0, parts = 1;
  if (s < c.seqs && span_of(a, s).tiles) {
    const int tiles = span_of(a, s).tiles;
    const int64_t at = f.total * slice / f.ctas;  // narrow: list index where the slice begins
    row = THREADS == kNarrow ? (int)((at - f.start) / tiles) : blockIdx.x - s * rows;
    const int64_t begin = f.start + (int64_t)row * tiles;
    first = (int)(((begin + 1) * f.ctas - 1) / f.total);  // the CTA whose slice holds the row's first tile
    parts = (int)(((begin + tiles) * f.ctas - 1) / f.total) - first + 1;
    if (THREADS == kNarrow && (begin == at || first != (int)blockIdx.x)) parts = 1;
  }
  dependent_wait();  // also where there is nothing to do: this grid ends after the main one
  launch_dependents();
  if (parts == 1) return;
  const int kvh = row / a.groups, head0 = kvh * a.share + (row - kvh * a.groups) * kCols;
  const int heads = min(kCols, (kvh + 1) * a.share - head0);
  const int group = THREADS < kItems ? 0 : threadIdx.x / kItems;
  for (int item = threadIdx.x % kItems; item < kItems; item += THREADS < kItems ? THREADS : kItems) {
    const int col = item / (DP / 8), d = 8 * (item % (DP / 8));
    if (group < kGroups) {
      float m = -INFINITY, l = 0.0f, any = 0.0f, v[8] = {};
      constexpr int kBatch = 4;
      for (int w0 = group; w0 < parts; w0 += kBatch * kGroups) {
        float4 st[kBatch], lo[kBatch], hi[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int w = w0 + i * kGroups;
          st[i] = make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
          lo[i] = hi[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (w >= parts) continue;
          const float *slot = a.ws + ((int64_t)(first + w) * 2 + (w == 0)) * slot_floats(kCols, DP);
          if (col < heads && d < c.head_dim) {  // what was written
            st[i] = *reinterpret_cast<const float4 *>(slot + kCols * DP + col * 4);
            lo[i] = *reinterpret_cast<const float4 *>(slot + col * DP + d);
            hi[i] = *reinterpret_cast<const float4 *>(slot + col * DP + d + 4);
          }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const float now = fmaxf(m, st[i].x), base = now == -INFINITY ? 0.0f : now;
          const float fo = ex2(m - base), fn = ex2(st[i].x - base);
          m = now;
          l = l * fo + st[i].y * fn;
          any = fmaxf(any, st[i].z);
          const float p[8] = {lo[i].x, lo[i].y, lo[i].z, lo[i].w, hi[i].x, hi[i].y, hi[i].z, hi[i].w};
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = v[e] * fo + p[e] * fn;
        }
      }
      part_sh[group][0][item] = m;
      part_sh[group][1][item] = l;
      part_sh[group][2][item] = any;
#pragma unroll
      for (int e = 0; e < 8; ++e) part_sh[group][3 + e][item] = v[e];
    }
    if (kGroups > 1) __syncthreads();  // (then the loop runs once, for every thread)
    if (group != 0 || col >= heads || d >= c.head_dim) continue;
    bool seen = false;
    for (int w = 0; w < kGroups; ++w) seen |= part_sh[w][2][item] != 0.0f;
    const Joined j = join(
        (1u << kGroups) - 1, [&](int w) { return part_sh[w][0][item]; },
        [&](int w) { return part_sh[w][1][item]; },
        [&](int w, float fw, float *v) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = fmaf(fw, part_sh[w][3 + e][item], v[e]);
        });
    finish<T>(a, s, head0 + col, d, j, seen);
  }
}

constexpr int dp_of(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : d <= 192 ? 192 : 256; }
// Two tiles of 8 heads where a key head serves more than 8, but not for wide
// heads: their queries and sums would not fit the registers.  Further heads are
// rows of their own, which read the same keys and values again, in part from
// L2 (32 sequences of 4000, one key head: of 256, 8 heads 31.6 us, 16 heads
// 42.6; of 128, 16 heads 23.2, 32 heads 29.9).
constexpr int nt_of(int share, int dp) { return share > 8 && dp <= 128 ? 2 : 1; }

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

template <typename T, int DP, int NT, bool UNITS>
fp4_status launch(AtParams a, cudaStream_t s) {
  constexpr int kMaxDev = 64;
  static std::atomic<int> occupancy[kMaxDev];
  constexpr int cols = 8 * NT;
  constexpr size_t smem = (2 * kWarps * cols * (DP + 8) + 8 * kWarps * cols) * sizeof(float);
  constexpr size_t part = slot_floats(cols, DP) * sizeof(float);
  auto kern = k_attention<T, DP, NT, UNITS>;
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
  // no more CTAs than the table has tiles
  const int64_t rows = (int64_t)c.seqs * c.kv_heads * a.groups;
  const int64_t room = (int64_t)c.seq_pages * c.page_size;
  const int64_t most = (int64_t)sm_count() * (per < kPerSM ? per : kPerSM);
  const int64_t tiles = ceil_div(rows * ceil_div(room, a.tile), kWarps);
  if (rows > INT32_MAX) return FP4_ERR_SHAPE;
  a.direct = cluster_of(rows, a.p.window && a.p.window < room - 15 ? a.p.window + 15 : room, DP, NT);
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
          ? launch_dependent(k_attention_join<T, DP, NT, kWide>, dim3((unsigned)rows), dim3(kWide), 0, s, a)
          : launch_dependent(k_attention_join<T, DP, NT, kNarrow>, dim3((unsigned)a.ctas - 1), dim3(kNarrow), 0, s, a);
  return e == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

template <typename T, int DP, int NT>
fp4_status launch_pages(const AtParams &a, cudaStream_t s) {
  return a.p.cache.page_size % 16 == 0 ? launch<T, DP, NT, true>(a, s) : launch<T, DP, NT, false>(a, s);
}

template <typename T>
fp4_status launch_type(const AtParams &a, int nt, cudaStream_t s) {
  switch (dp_of(a.p.cache.head_dim)) {
    case 64: return nt == 1 ? launch_pages<T, 64, 1>(a, s) : launch_pages<T, 64, 2>(a, s);
    case 128: return nt == 1 ? launch_pages<T, 128, 1>(a, s) : launch_pages<T, 128, 2>(a, s);
    case 192: return launch_pages<T, 192, 1>(a, s);
    default: return launch_pages<T, 256, 1>(a, s);
  }
}

}  // namespace

int64_t decode_attention_workspace(int64_t seqs, int64_t room, int heads, int kv_heads, int head_dim) {
  const int dp = dp_of(head_dim), nt = nt_of(heads / kv_heads, dp), cols = 8 * nt;
  if (cluster_of(seqs * kv_heads * ceil_div(heads / kv_heads, cols), room, dp, nt)) return 0;
  return (int64_t)sm_count() * kPerSM * 2 * slot_floats(cols, dp) * sizeof(float);
}

fp4_status launch_decode_attention(const fp4_attention_params &p, cudaStream_t s) {
  AtParams a{};
  a.p = p;
  a.status = status_word();
  if (!a.status) return FP4_ERR_CUDA;
  const fp4_kv_cache &c = p.cache;
  a.share = p.heads / c.kv_heads;
  const int nt = nt_of(a.share, dp_of(c.head_dim));
  a.groups = (a.share + 8 * nt - 1) / (8 * nt);
  a.shift = -1;
  if ((c.page_size & (c.page_size - 1)) == 0)
    for (a.shift = 0; (1 << a.shift) < c.page_size;) ++a.shift;
  a.out16 = aligned16(p.out) && p.out_seq % 8 == 0 && p.out_head % 8 == 0;
  a.scale2 = p.scale * 1.44269504088896f;
  a.ws = static_cast<float *>(p.workspace);
  return c.type == FP4_BF16 ? launch_type<__nv_bfloat16>(a, nt, s) : launch_type<__half>(a, nt, s);
}

}  // namespace fp4
