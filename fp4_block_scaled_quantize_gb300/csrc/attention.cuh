// attention.cuh -- what the attention kernels over a paged cache share
// (attention16.cuh: keys and values of 16 bits, attention8.cu: of 8): which
// positions are seen, the list of tiles that warps share out, the tensor-core
// and packing helpers, and the joins of partial rows.
#pragma once
#include <cmath>

#include "serve.cuh"

namespace fp4 {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kPerSM = 5;            // CTAs per SM at most (workspace bound)
constexpr int kCluster = 8;          // CTAs that take a row between them, at most
constexpr float kSlack = 8.0f;       // log2 by which scores may pass the maximum in use

struct AtParams {
  fp4_attention_params p;
  int groups;   // head groups of a key head: ceil(heads / kv_heads / (8 NT))
  int share;    // heads / kv_heads
  int tile;     // positions of a tile: 16 per unit
  int ctas;     // slices of the list of tiles: one for a CTA of the main kernel, or more
  int least;    // tiles of a slice, at least
  int bundle;   // rows whose tiles are one item of the list, worked on side by side
  int direct;   // CTAs (a cluster) that take a row between them, or 0: equal slices
  int shift;    // log2 page_size, or -1: no power of two (16 bits)
  int out16;    // rows of out allow 16-byte stores
  float scale2; // scale * log2 e
  float *ws;    // [ctas][2] partial rows
  uint32_t *status;
};

// Partial row: 8 NT x DP outputs relative to m, then m, l, seen (1.0 or 0.0) and
// whether there is one (clusters) per head.  Over codes the outputs are relative
// to a maximum of their own, mo (of scores with the values' exponents), which may
// lie as far from m as the exponents of binary32 reach: m, l, kThere or kSeen, mo.
constexpr float kThere = 1.0f, kSeen = 2.0f;
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

// What of a sequence is seen: positions [0, sinks) and [from, len), apart from
// each other (sinks is 0 where they meet, and without SINKS).  Its tiles are those
// of the first positions, then those of the others, which start at base.
struct Span {
  int from, len, base, sinks, first, tiles;  // first: tiles of the first positions
  // the seen positions [lo, hi) of tile i and the position where it starts
  __device__ __forceinline__ int start(int i, int tile, int &lo, int &hi) const {
    const bool early = i < first;
    lo = early ? 0 : from;
    hi = early ? sinks : len;
    return early ? i * tile : base + (i - first) * tile;
  }
};
template <bool SINKS>
__device__ __forceinline__ Span span_of(const AtParams &a, int s) {
  const fp4_kv_cache &c = a.p.cache;
  const int64_t room = (int64_t)c.seq_pages * c.page_size;  // fits 32 bits
  const int given = a.p.lengths[s];
  Span r;
  r.len = given < 0 ? 0 : given > room ? (int)room : given;
  r.from = a.p.window && r.len > a.p.window ? r.len - a.p.window : 0;
  r.sinks = SINKS ? a.p.sinks : 0;
  if (SINKS && r.from <= r.sinks) r.from = r.sinks = 0;
  r.base = r.from & ~15;
  r.first = SINKS ? (r.sinks + a.tile - 1) / a.tile : 0;
  r.tiles = r.first + (r.len - r.base + a.tile - 1) / a.tile;
  return r;
}

// Prefix over the sequences: the sum of rows * tiles of all, and the sequence
// in which a slice of the list begins (or the sequence `which`).
struct Found {
  int64_t total, start;  // start: list index of the found sequence's first tile
  int64_t ctas;          // slices that share the list
  int seq;
};
template <int THREADS, bool SINKS>
__device__ Found find(const AtParams &a, int rows, int64_t slice, int64_t *shared, int which = -1) {
  constexpr int kW = THREADS / 32;
  const int seqs = a.p.cache.seqs, per = (seqs + THREADS - 1) / THREADS;
  if (seqs <= 32) {  // each warp by itself
    const int lane = threadIdx.x & 31;
    const int64_t sum = lane < seqs ? (int64_t)rows * span_of<SINKS>(a, lane).tiles : 0;
    int64_t inc = sum;
    for (int o = 1; o < seqs; o <<= 1) {
      const int64_t v = __shfl_up_sync(~0u, inc, o);
      if (lane >= o) inc += v;
    }
    Found f;
    f.total = __shfl_sync(~0u, inc, seqs - 1);
    f.ctas = min((int64_t)a.ctas, (f.total + a.least - 1) / a.least);
    const int64_t x = slice < f.ctas ? f.total * slice / f.ctas : f.total;
    const uint32_t hit = __ballot_sync(~0u, which < 0 ? x >= inc - sum && x < inc : lane == which);
    f.seq = hit ? __ffs(hit) - 1 : seqs;
    f.start = hit ? __shfl_sync(~0u, inc - sum, f.seq) : f.total;
    return f;
  }
  const int s0 = threadIdx.x * per, s1 = min(s0 + per, seqs);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t sum = 0;
  for (int s = s0; s < s1; ++s) sum += (int64_t)rows * span_of<SINKS>(a, s).tiles;
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
  const int64_t ctas = min((int64_t)a.ctas, (total + a.least - 1) / a.least);
  const int64_t x = slice < ctas ? total * slice / ctas : total;
  if (which < 0 ? x >= before && x < before + sum : which >= s0 && which < s1) {  // one thread, if any
    int64_t at = before;
    for (int s = s0;; ++s) {
      const int64_t n = (int64_t)rows * span_of<SINKS>(a, s).tiles;
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

// log sum exp of a row: m + log2 l in base 2.  Scores that are all -inf have the
// sum 0 and give -inf; over codes, which are finite, it is the query that is not,
// and that is NaN.
template <typename T, bool CODES>
__device__ __forceinline__ void store_lse(const AtParams &a, int s, int head, bool seen, float m, float l) {
  if (CODES && l == 0.0f) l = NAN;
  a.p.lse[(int64_t)s * a.p.heads + head] =
      seen ? ((m == -INFINITY ? 0.0f : m) + log2f(l) - lift<T>()) * 0.693147180559945f : -INFINITY;
}

// v 2^x in two steps: x alone may pass binary32's exponents where the result does not.
__device__ __forceinline__ float shifted(float v, float half) { return v * half * half; }

// Eight outputs of a row joined from parts, one for each bit of `parts`: m(i),
// l(i) are part i's statistics, mo(i) what its outputs are relative to (CODES;
// else m), add(i, w, v) adds w times its outputs.
struct Joined {
  float top, topo, sum, v[8];
};
template <bool CODES, typename M, typename Mo, typename L, typename Add>
__device__ __forceinline__ Joined join(uint32_t parts, M m, Mo mo, L l, Add add) {
  Joined j;
  j.top = j.topo = -INFINITY;
  j.sum = 0.0f;
  for (uint32_t p = parts; p; p &= p - 1) {
    j.top = fmaxf(j.top, m(__ffs(p) - 1));
    if (CODES) j.topo = fmaxf(j.topo, mo(__ffs(p) - 1));
  }
  const float base = j.top == -INFINITY ? 0.0f : j.top, baseo = j.topo == -INFINITY ? 0.0f : j.topo;
#pragma unroll
  for (int e = 0; e < 8; ++e) j.v[e] = 0.0f;
  for (uint32_t p = parts; p; p &= p - 1) {
    const int i = __ffs(p) - 1;
    const float w = ex2(m(i) - base);
    j.sum = fmaf(w, l(i), j.sum);
    add(i, CODES ? ex2(mo(i) - baseo) : w, j.v);
  }
  return j;
}
// The same of parts held side by side: get(q, st, lo, hi) reads part q (its
// statistics and the outputs) if there is one.  All are requested together.
struct Whole {
  Joined j;
  bool seen, there;
};
template <int N, bool CODES, typename Get>
__device__ __forceinline__ Whole join_all(Get get) {
  float4 st[N], lo[N], hi[N];
#pragma unroll
  for (int q = 0; q < N; ++q) {
    st[q] = make_float4(-INFINITY, 0.0f, 0.0f, CODES ? -INFINITY : 0.0f);
    lo[q] = hi[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    get(q, st[q], lo[q], hi[q]);
  }
  Whole r = {};
  r.j.top = r.j.topo = -INFINITY;
#pragma unroll
  for (int q = 0; q < N; ++q) {
    r.j.top = fmaxf(r.j.top, st[q].x);
    if (CODES) r.j.topo = fmaxf(r.j.topo, st[q].w);
    r.seen |= CODES ? st[q].z == kSeen : st[q].z != 0.0f;
    r.there |= (CODES ? st[q].z : st[q].w) != 0.0f;
  }
  const float base = r.j.top == -INFINITY ? 0.0f : r.j.top, baseo = r.j.topo == -INFINITY ? 0.0f : r.j.topo;
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const float w = ex2(st[q].x - base), wo = CODES ? ex2(st[q].w - baseo) : w;
    r.j.sum = fmaf(w, st[q].y, r.j.sum);
    const float v[8] = {lo[q].x, lo[q].y, lo[q].z, lo[q].w, hi[q].x, hi[q].y, hi[q].z, hi[q].w};
#pragma unroll
    for (int e = 0; e < 8; ++e) r.j.v[e] = fmaf(wo, v[e], r.j.v[e]);
  }
  return r;
}
// sqrt 2^(topo - top), or 1 where there is no weight at all.
__device__ __forceinline__ float half_shift(float top, float topo) {
  return top == -INFINITY || topo == -INFINITY ? 1.0f : ex2(0.5f * (topo - top));
}
// Writes the result of a row that saw something (seen) or nothing.
template <typename T, bool CODES>
__device__ __forceinline__ void finish(const AtParams &a, int s, int head, int d, Joined j, bool seen) {
  const float w = seen ? 1.0f / j.sum : 0.0f, half = CODES ? half_shift(j.top, j.topo) : 1.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) j.v[e] = CODES ? shifted(j.v[e] * w, half) : j.v[e] * w;
  store8<T>(a, s, head, d, j.v);
  if (a.p.lse && d == 0) store_lse<T, CODES>(a, s, head, seen, j.top, j.sum);
}

// Joins partial rows.  Many rows are cut into few parts each: narrow CTAs, of
// which CTA c takes the row in which slice c + 1 begins, if it began in slice
// c (so every cut row has one).  Few rows are cut into many: wide CTAs, one
// for each row.  Which parts a row has follows from the lengths, which are read
// before the main grid is waited for: that grid is an ordinary launch, so what
// came before it on the stream is complete.  A CTA's threads take eight outputs each, in groups
// that walk every kGroups-th part some at a time; the first joins the groups.  The
// rows of a bundle have a CTA each.  Over codes, where a part has one number more,
// wide CTAs have half the threads (one sequence of 131071: 56.7 us with 6 parts at
// a time, 57.7 with 4; 1024 threads 57.8 with 2, 59.0 with 4 and spills), and narrow
// ones take two at a time (40 windows of 4096: 66.1 us, with 4 67.1, with 8 69.3).
constexpr int kNarrow = 128, kWide = 1024, kWide8 = 512;
template <typename T, int DP, int NT, int THREADS, bool SINKS, bool CODES>
__global__ void __launch_bounds__(THREADS) k_attention_join(const __grid_constant__ AtParams a) {
  constexpr int kCols = 8 * NT, kItems = kCols * DP / 8;
  constexpr int kGroups = THREADS < kItems ? 1 : THREADS / kItems;
  __shared__ int64_t scan[THREADS / 32 + 2];
  constexpr int kStats = CODES ? 4 : 3, kBatch = !CODES ? 4 : THREADS == kNarrow ? 2 : 6;  // parts at a time
  __shared__ float part_sh[kGroups][kStats + 8][kItems];  // m, l, seen, mo (CODES); eight outputs
  const fp4_kv_cache &c = a.p.cache;
  const int bundle = CODES ? a.bundle : 1;
  const int rows = c.kv_heads * a.groups / bundle, index = blockIdx.x / bundle, member = blockIdx.x % bundle;
  const int slice = index + 1;
  const Found f = THREADS == kNarrow ? find<THREADS, SINKS>(a, rows, slice, scan)
                                     : find<THREADS, SINKS>(a, rows, 0, scan, index / rows);
  int s = f.seq, row = 0, first = 0, parts = 1;
  if (s < c.seqs && span_of<SINKS>(a, s).tiles) {
    const int tiles = span_of<SINKS>(a, s).tiles;
    const int64_t at = f.total * slice / f.ctas;  // narrow: list index where the slice begins
    row = THREADS == kNarrow ? (int)((at - f.start) / tiles) : index - s * rows;
    const int64_t begin = f.start + (int64_t)row * tiles;
    first = (int)(((begin + 1) * f.ctas - 1) / f.total);  // the CTA whose slice holds the row's first tile
    parts = (int)(((begin + tiles) * f.ctas - 1) / f.total) - first + 1;
    if (THREADS == kNarrow && (begin == at || first != index)) parts = 1;
  }
  dependent_wait();  // also where there is nothing to do: this grid ends after the main one
  launch_dependents();
  if (parts == 1) return;
  row = row * bundle + member;
  const int kvh = row / a.groups, head0 = kvh * a.share + (row - kvh * a.groups) * kCols;
  const int heads = min(kCols, (kvh + 1) * a.share - head0);
  const int group = THREADS < kItems ? 0 : threadIdx.x / kItems;
  for (int item = threadIdx.x % kItems; item < kItems; item += THREADS < kItems ? THREADS : kItems) {
    const int col = item / (DP / 8), d = 8 * (item % (DP / 8));
    if (group < kGroups) {
      float m = -INFINITY, mo = -INFINITY, l = 0.0f, any = 0.0f, v[8] = {};
      for (int w0 = group; w0 < parts; w0 += kBatch * kGroups) {
        float4 st[kBatch], lo[kBatch], hi[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int w = w0 + i * kGroups;
          st[i] = make_float4(-INFINITY, 0.0f, 0.0f, CODES ? -INFINITY : 0.0f);
          lo[i] = hi[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (w >= parts) continue;
          const float *slot =
              a.ws + (((int64_t)(first + w) * 2 + (w == 0)) * bundle + member) * slot_floats(kCols, DP);
          if (col < heads && d < c.head_dim) {  // what was written
            st[i] = *reinterpret_cast<const float4 *>(slot + kCols * DP + col * 4);
            lo[i] = *reinterpret_cast<const float4 *>(slot + col * DP + d);
            hi[i] = *reinterpret_cast<const float4 *>(slot + col * DP + d + 4);
          }
        }
        if constexpr (CODES) {  // what was joined before moves once for the batch
          float now = m, nowo = mo;
#pragma unroll
          for (int i = 0; i < kBatch; ++i) now = fmaxf(now, st[i].x), nowo = fmaxf(nowo, st[i].w);
          const float base = now == -INFINITY ? 0.0f : now, baseo = nowo == -INFINITY ? 0.0f : nowo, fade = ex2(mo - baseo);
          l *= ex2(m - base);
          m = now;
          mo = nowo;
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= fade;
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const float w = ex2(st[i].w - baseo);
            l = fmaf(ex2(st[i].x - base), st[i].y, l);
            any = fmaxf(any, st[i].z);
            const float p[8] = {lo[i].x, lo[i].y, lo[i].z, lo[i].w, hi[i].x, hi[i].y, hi[i].z, hi[i].w};
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = fmaf(w, p[e], v[e]);
          }
        } else {
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
      }
      part_sh[group][0][item] = m;
      part_sh[group][1][item] = l;
      part_sh[group][2][item] = any;
      if (CODES) part_sh[group][kStats - 1][item] = mo;
#pragma unroll
      for (int e = 0; e < 8; ++e) part_sh[group][kStats + e][item] = v[e];
    }
    if (kGroups > 1) __syncthreads();  // (then the loop runs once, for every thread)
    if (group != 0 || col >= heads || d >= c.head_dim) continue;
    bool seen = false;
    for (int w = 0; w < kGroups; ++w) seen |= CODES ? part_sh[w][2][item] == kSeen : part_sh[w][2][item] != 0.0f;
    const Joined j = join<CODES>(
        (1u << kGroups) - 1, [&](int w) { return part_sh[w][0][item]; },
        [&](int w) { return part_sh[w][kStats - 1][item]; }, [&](int w) { return part_sh[w][1][item]; },
        [&](int w, float fw, float *v) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = fmaf(fw, part_sh[w][kStats + e][item], v[e]);
        });
    finish<T, CODES>(a, s, head0 + col, d, j, seen);
  }
}

constexpr int dp_of(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : d <= 192 ? 192 : 256; }
// Two tiles of 8 heads where a key head serves more than 8, but not for wide
// heads: their queries and sums would not fit the registers.  Further heads are
// rows of their own, which read the same keys and values again, in part from
// L2 (32 sequences of 4000, one key head: of 256, 8 heads 31.6 us, 16 heads
// 42.6; of 128, 16 heads 23.2, 32 heads 29.9).
constexpr int nt_of(int share, int dp) { return share > 8 && dp <= 128 ? 2 : 1; }

}  // namespace

}  // namespace fp4
