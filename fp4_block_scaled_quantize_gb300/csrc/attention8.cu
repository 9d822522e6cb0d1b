// attention8.cu -- attention of one new token per sequence over a paged cache
// of E4M3 codes with a power-of-two scale for each block of tokens and head
// (sm_103a):  out = sum_j w_j 2^ev_j cv_j,  w = softmax_j(scale q . 2^ek_j ck_j).
//
// Bound: HBM, 2 D bytes per position and key head, half of what 16 bits move,
// so twice the positions per time: at 6.8 TB/s an SM has 190 clocks for 16
// positions of a head of 128, which take ~320 instructions of a warp, 40% of its
// issue slots.
//
// Mathematics.  Codes become f16 exactly (one conversion a pair) and meet the
// queries, held in f16 times a power of two per head (exact down to 2^-38 of
// the head's largest element, 2^-31 for BF16's eight bits), in MMAs that sum in
// binary32.  A score is that sum times two powers of two and scale log2 e.  The
// values' scales go into the weights: with s_j the score in base 2 the sum l
// takes 2^(s_j - m), the product with the codes 2^(s_j + ev_j - mo), each with a
// running maximum of its own, so whatever the scales are, the terms that make
// the result are held to full precision; 2^(mo - m), which may pass binary32's
// exponents where the result does not, is applied at the very end, in two steps,
// and parts of a row are joined before it.  Both maxima are moved only when
// passed by more than 8.  A weight enters its
// product as two f16 parts (2^-22 of it left out, or 2^-32 of the largest).
//
// Loads.  Asynchronous 16-byte copies into a ring of shared memory that each
// warp fills for itself, kStages - 1 tiles ahead, across the rows of its slice;
// scales are requested with the copies and put beside them a step later.
//
// Split.  Short rows go to clusters, as in attention16.cuh.  Otherwise the warps of
// the resident CTAs share the list of all tiles out evenly; warps of a CTA take
// `bundle` (4, 2 or 1) neighbouring key heads over the same positions.  In a page
// with heads innermost a head's row of 128 bytes lies between others': copies
// alone reach 6.1 TB/s of rows that one warp takes by itself, 7.1 where two or
// more neighbours are in flight together.  What a warp has of a row that others
// share goes to the workspace, for the join of attention.cuh in a second,
// dependent launch, in slice order, so results repeat exactly.
// Measured in a graph, 32 heads over 8 of 128, BF16: 64 sequences of up to 16384
// positions 179 - 182 us (87 - 89% of a copy's rate; the kernel's copies without its
// work 174; pages of 24 183, of 8 188, of 20 in blocks of 4 192); one of 131071 57
// us (copies 56), of 65000 38, of 16000 20, so that some 15 us do not grow with the
// length, with or without the work; one of 300 7.0; 40 windows of 4096 with 20 first
// positions 65 - 67 (copies 63).  Heads of 64 (16, 64 sequences of 16384) 433 us for
// 317 at a copy's rate: as many instructions a position as heads of 128, half the
// bytes; of 256 333.  Query heads that need a second pass over a key head (32
// sequences of 4000): of 256, 8 heads 25.3, 16 heads 28.1.
//
// Layout is that of attention16.cuh:
//   S^T = K Q^T   lane (g, t) reads pieces 64 i + 16 t of keys g, g + 8
//   O^T = V^T P^T lane (g, t) reads pieces 128 i + 16 g (or 8 g) of values
//                 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#include <cooperative_groups.h>

#include "attention.cuh"

namespace fp4 {

namespace {

namespace cg = cooperative_groups;

struct At8Params {
  AtParams a;
  fp4_kv_scales s;
  Divisor page, block;
  int64_t k_step, v_step;  // from a lane's row to its next
  // strides in 32 bits (pages of whole units only)
  int k_page, k_place, v_page, v_place, ks_page, ks_block, vs_page, vs_block;
};

constexpr int kStages = 2;  // 3 - 6: slower, by up to a tenth
// CTAs an SM holds at most (workspace bound).  3 (160 registers): 177 us for 183
// with 64 sequences of up to 16384, but 76 for 67 with 40 windows of 4096, 60 for
// 57 with one of 131071.
constexpr int kPerSM8 = 2;
// CTAs an SM holds at least, by the kernel's launch bounds.
constexpr int per_sm8(int dp) { return dp <= 128 ? 2 : 1; }
constexpr float kNone = -3e38f;  // a running maximum before there is a score
constexpr float kLift = 7.0f;  // weights are held 2^7 times as large (f16's smallest is 2^-24)

// Groups of 16 positions a step.
constexpr int units8(int dp) { return dp <= 64 ? 4 : dp <= 128 ? 2 : 1; }

// The ring of a warp, a stage: keys, values, then per unit 32 floats (the keys'
// scales, the values' exponents) and the mask of what is seen.
constexpr int info_bytes = 40 * 4;
constexpr int unit_bytes(int dp) { return 32 * dp + info_bytes; }
constexpr int ring_bytes(int dp) { return kStages * units8(dp) * unit_bytes(dp); }
constexpr int part_bytes(int cols, int dp) { return cols * (dp + 8) * 4; }

__device__ __forceinline__ void copy16(uint32_t to, const void *from, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t to, const void *from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t shared_at(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// A stage's keys and values lie there by rows (positions) of DP bytes, in chunks
// of 16.  Eight neighbouring lanes copy 128 consecutive bytes of a row (DP 64: two
// rows of 64): where a lane copied the pieces that it reads itself, 4 rows to
// eight lanes, the copies ran at 2.5 TB/s.  Chunks change places so that both the
// copies and the reads meet all banks:
//   keys    chunk c of row r at c ^ 4 (r & 1)           read by rows g, chunks t
//   values  chunk c of row r at c ^ 2 ((r / 2) & 3)     read by rows 2 t, chunks g
// (rows of 192 bytes shift by half the banks by themselves; their last four
// chunks, and the values of DP 64, change places within four, and the latter's
// rows r and r + 4 share 128 bytes).
template <int DP>
struct Layout {
  static constexpr int kLanes = DP <= 64 ? 4 : DP <= 128 ? 8 : 16;  // of a row
  static constexpr int kRows = 32 / kLanes, kSteps = 16 / kRows;    // rows of a copy, copies of 16
  static __device__ __forceinline__ int row(int lane) {  // of a lane's keys and values in the first copy
    return DP == 64 ? (lane >> 3) + (lane & 4) : lane / kLanes;
  }
  static __device__ __forceinline__ int chunk(int lane) { return lane % kLanes; }
  // where copy j puts the chunk
  static __device__ __forceinline__ int key(int lane, int j) {
    const int r = row(lane) + kRows * j, c = chunk(lane);
    return r * DP + 16 * (DP % 128 == 0 ? c ^ 4 * (r & 1) : c);
  }
  static __device__ __forceinline__ int value(int lane, int j) {
    const int r = row(lane) + kRows * j, c = chunk(lane);
    if (DP == 64) return 128 * ((r & 3) | (r >> 3) << 2) + 64 * (r >> 2 & 1) + 16 * (c ^ (r & 2));
    return r * DP + 16 * (DP == 192 && c >= 8 ? c ^ (r & 2) : c ^ 2 * (r >> 1 & 3));
  }
  // where lane (g, t) finds piece i of key g (g + 8: 8 DP on)
  static __device__ __forceinline__ int key_at(int g, int t, int i) {
    return g * DP + 16 * (DP % 128 == 0 ? (4 * i + t) ^ 4 * (g & 1) : 4 * i + t);
  }
  // where it finds its piece of 16 bytes, i, of value 2 t + (h & 1) + 8 (h / 2)
  static __device__ __forceinline__ int value_at(int g, int t, int h, int i) {
    return (2 * t + (h & 1) + 8 * (h >> 1)) * DP + 128 * i + 16 * (g ^ 2 * t);
  }
  // and that of 8 bytes behind them
  static __device__ __forceinline__ int value8_at(int g, int t, int h) {
    const int in = 16 * (g >> 1 ^ 2 * (t & 1)) + 8 * (g & 1);
    return DP == 64 ? 256 * (t & 1) + 128 * (h & 1) + 512 * (h >> 1) + 64 * (t >> 1) + in
                    : (2 * t + (h & 1) + 8 * (h >> 1)) * DP + 128 + in;
  }
};

// What a warp has to know of a row that it works on: sequence, row, tiles of it
// in the slice, and whether it begins (1) and ends (2) there.
struct Row {
  int s, row, tiles, ends;
};
constexpr int kQueue = 8;  // rows between the copies and the work: kStages + 1 at most

// UNITS: pages of whole units of 16 places, strides below 2^31.
template <typename T, int DP, int NT, bool UNITS>
__global__ void __launch_bounds__(kThreads, per_sm8(DP)) k_attention8(const __grid_constant__ At8Params b) {
  constexpr int kCols = 8 * NT, kKey = DP / 64, kV16 = DP / 128, kV8 = DP / 64 % 2, kWords = DP / 32;
  constexpr int kUnits = units8(DP), kTile = 16 * kUnits;
  constexpr int kRows = Layout<DP>::kRows, kSteps = Layout<DP>::kSteps;
  const AtParams &a = b.a;
  extern __shared__ __align__(16) char smem8[];
  __shared__ int64_t scan[kWarps + 2];
  __shared__ bool part_sh[kWarps];  // clusters: whether a warp has a part of the row
  __shared__ Row queue_sh[kWarps][kQueue];
  const fp4_kv_cache &c = a.p.cache;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int D = c.head_dim, rows = c.kv_heads * a.groups / a.bundle;  // of the list, `bundle` rows in one
  // the warps' rings; m, l, seen, 1 of partial rows (clusters: their outputs take
  // the place of the rings); the partial row of a CTA of a cluster
  char *const ring = smem8 + warp * ring_bytes(DP);
  float4 *const st_sh = reinterpret_cast<float4 *>(smem8 + kWarps * ring_bytes(DP));
  float *const part = reinterpret_cast<float *>(st_sh + kWarps * kCols);
  auto part_of = [&](int p) { return reinterpret_cast<float *>(smem8 + p * ring_bytes(DP)); };

  int64_t at, end, start;
  int s;
  dependent_wait();
  launch_dependents();
  if (lane == 0) part_sh[warp] = false;
  const int rank = a.direct ? blockIdx.x % a.direct : 0, mine_row = a.direct ? blockIdx.x / a.direct : 0;
  if (a.direct) {
    s = mine_row / rows;
    start = 0;
    const int tiles = span_of<true>(a, s).tiles;
    at = (int64_t)(mine_row - s * rows) * tiles;
    end = at + (int64_t)tiles * (rank + 1) / a.direct;
    at += (int64_t)tiles * rank / a.direct;
  } else {
    // warps of a bundle share a slice
    const int subs = kWarps / a.bundle;
    const int64_t first = (int64_t)blockIdx.x * subs, slice = first + warp / a.bundle;
    const Found f = find<kThreads, true>(a, rows, first, scan);
    s = f.seq;
    start = f.start;
    at = end = 0;
    if (slice < f.ctas) {
      at = f.total * slice / f.ctas;
      end = f.total * (slice + 1) / f.ctas;
    }
  }
  // sequences that see nothing are in no slice: their rows are written here
  for (int e = a.direct ? s : blockIdx.x; e < c.seqs; e += a.direct ? c.seqs : gridDim.x) {
    const int given = a.p.lengths[e];
    if (a.direct && (rank || mine_row != s * rows)) break;
    if (threadIdx.x == 0 && (given < 0 || given > (int64_t)c.seq_pages * c.page_size))
      raise_status(a.status, kStatusIndex);
    if (span_of<true>(a, e).tiles) continue;
    const float zero[8] = {};
    for (int i = threadIdx.x; i < a.p.heads * (D / 8); i += kThreads) {
      const int head = i / (D / 8), d = 8 * (i % (D / 8));
      store8<T>(a, e, head, d, zero);
      if (a.p.lse && d == 0) a.p.lse[(int64_t)e * a.p.heads + head] = -INFINITY;
    }
  }

  if (a.direct) {  // a quarter of the CTA's tiles for each warp
    const int64_t n = end - at;
    end = at + n * (warp + 1) / kWarps;
    at += n * warp / kWarps;
  }
  Row *const queue = queue_sh[warp];
  // The tile that is copied next: position pos, tile `tile` of a row of which the
  // slice has those before tile1; where the row's keys, values (a lane's first
  // pieces), scales and page numbers are.
  // bad: a page outside the cache was met, reported at the end (a branch to it in
  // the loop makes loads in flight be waited for: 64 sequences of up to 16384 took
  // 233 us for 173).
  bool live = at < end, bad = false;
  Span sp = live ? span_of<true>(a, s) : Span{};
  int tile = 0, tile1 = 0, pos = 0, entered = 0;
  const int32_t *table = c.table;
  const char *keys = nullptr, *values = nullptr;
  const uint8_t *codes = nullptr;
  auto enter = [&] {  // on to the next row of the slice
    live = at < end;
    if (!live) return;
    while (at >= start + (int64_t)rows * sp.tiles) {
      start += (int64_t)rows * sp.tiles;
      sp = span_of<true>(a, ++s);
    }
    const int item = (int)((at - start) / sp.tiles), row = item * a.bundle + warp % a.bundle, kvh = row / a.groups;
    tile = (int)(at - start - (int64_t)item * sp.tiles);
    tile1 = (int)min((int64_t)sp.tiles, tile + (end - at));
    at += tile1 - tile;
    if (lane == 0)
      queue[entered % kQueue] = Row{s, row, tile1 - tile, (tile == 0 ? 1 : 0) | (tile1 == sp.tiles ? 2 : 0)};
    ++entered;
    int lo, hi;
    pos = sp.start(tile, kTile, lo, hi);
    table = c.table + s * c.table_stride;
    keys = static_cast<const char *>(c.k) + kvh * c.k_head;
    values = static_cast<const char *>(c.v) + kvh * c.v_head;
    if (UNITS) {  // (lanes behind the head's end copy nothing: an address inside it)
      const int in = 16 * Layout<DP>::chunk(lane) < D ? 16 * Layout<DP>::chunk(lane) : 0;
      keys += Layout<DP>::row(lane) * c.k_place + in;
      values += Layout<DP>::row(lane) * c.v_place + in;
    }
    codes = lane < 16 ? b.s.k_sf + kvh * b.s.k_head : b.s.v_sf + kvh * b.s.v_head;
  };
  auto advance = [&] {
    if (!live) return;
    if (++tile < tile1)
      pos = tile == sp.first ? sp.base : pos + kTile;
    else
      enter();
  };
  const int sf_page = lane < 16 ? b.ks_page : b.vs_page, sf_block = lane < 16 ? b.ks_block : b.vs_block;

  // page numbers a step ahead of the copies (their loads are not waited for).
  // UNITS (pages of whole units): one for a unit, else lane i & 15 has that of
  // position i.
  auto ask = [&](int (&page)[kUnits]) {
    const int lo = tile < sp.first ? 0 : sp.from, hi = live ? tile < sp.first ? sp.sinks : sp.len : 0;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int i = pos + 16 * u + (UNITS ? 0 : lane & 15);
      page[u] = -1;
      if (i < hi && (UNITS || i >= lo)) page[u] = table[over(i, b.page)];
    }
  };
  // Copies the next tile into a stage and requests its scales: lanes 0 - 15
  // those of the keys of 16 positions, lanes 16 - 31 those of the values.
  auto copy = [&](int stage, const int (&pages)[kUnits], uint32_t (&code)[kUnits], uint32_t (&on)[kUnits]) {
    const int lo = tile < sp.first ? 0 : sp.from, hi = live ? tile < sp.first ? sp.sinks : sp.len : 0;
    const uint32_t to0 = shared_at(ring) + stage * kUnits * unit_bytes(DP);
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const uint32_t to = to0 + u * unit_bytes(DP), tv = to + 16 * DP;
      const int first = pos + 16 * u, i = first + (lane & 15);
      int page = pages[u];
      const bool in = i >= lo && i < hi, ok = page >= 0 && page < c.pages;
      bad |= in && !ok;
      on[u] = __ballot_sync(~0u, in && ok) & 0xFFFFu;
      if (on[u] == 0 && UNITS) {  // nothing is seen: zeros
#pragma unroll
        for (int e = 0; e < DP / 16; ++e)
          *reinterpret_cast<uint4 *>(ring + (stage * kUnits + u) * unit_bytes(DP) + e * 512 + 16 * lane) = make_uint4(0, 0, 0, 0);
        code[u] = 0;
        continue;
      }
      const int place0 = (UNITS ? first : i) - over(UNITS ? first : i, b.page) * c.page_size;
      const int place = UNITS ? place0 + (lane & 15) : place0;
      code[u] = 0;
      if (in && ok) {
        const int blk = over(place, b.block);
        code[u] = UNITS ? codes[(int64_t)page * sf_page + (int64_t)blk * sf_block]
                        : codes[page * (lane < 16 ? b.s.k_page : b.s.v_page) + blk * (lane < 16 ? b.s.k_block : b.s.v_block)];
      }
      if (UNITS) {
        // every place of the unit is one of its page, so every address is inside the cache
        const char *const k = keys + (int64_t)page * b.k_page + (int64_t)place0 * b.k_place;
        const char *const v = values + (int64_t)page * b.v_page + (int64_t)place0 * b.v_place;
        if (on[u] == 0xFFFFu && D == DP) {
#pragma unroll
          for (int j = 0; j < kSteps; ++j)
            if (DP != 192 || Layout<DP>::chunk(lane) < 12) copy16(to + Layout<DP>::key(lane, j), k + j * b.k_step);
#pragma unroll
          for (int j = 0; j < kSteps; ++j)
            if (DP != 192 || Layout<DP>::chunk(lane) < 12) copy16(tv + Layout<DP>::value(lane, j), v + j * b.v_step);
        } else {
          const bool inside = 16 * Layout<DP>::chunk(lane) < D;
#pragma unroll
          for (int j = 0; j < kSteps; ++j) {
            const bool yes = inside && (on[u] >> (Layout<DP>::row(lane) + kRows * j) & 1);
            if (DP == 192 && Layout<DP>::chunk(lane) >= 12) continue;
            copy16(to + Layout<DP>::key(lane, j), k + j * b.k_step, yes);
            copy16(tv + Layout<DP>::value(lane, j), v + j * b.v_step, yes);
          }
        }
      } else {
        const int64_t k0 = (int64_t)page * c.k_page + (int64_t)place0 * c.k_place;
        const int64_t v0 = (int64_t)page * c.v_page + (int64_t)place0 * c.v_place;
        const char *const nothing = static_cast<const char *>(a.p.q);  // an address for copies of no bytes
        const int in = 16 * Layout<DP>::chunk(lane);
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
          const int row = Layout<DP>::row(lane) + kRows * j;
          const char *const k = keys + __shfl_sync(~0u, k0, row) + in, *const v = values + __shfl_sync(~0u, v0, row) + in;
          const bool yes = in < D && (on[u] >> row & 1);
          if (DP == 192 && Layout<DP>::chunk(lane) >= 12) continue;
          copy16(to + Layout<DP>::key(lane, j), yes ? k : nothing, yes);
          copy16(tv + Layout<DP>::value(lane, j), yes ? v : nothing, yes);
        }
      }
    }
    copies_commit();
  };
  // Puts the scales of a copied stage beside it.
  auto settle = [&](int stage, const uint32_t (&code)[kUnits], const uint32_t (&on)[kUnits]) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      float *info = reinterpret_cast<float *>(ring + (stage * kUnits + u) * unit_bytes(DP) + 32 * DP);
      const float e = code[u] == 255 ? NAN : (float)((int)code[u] - 127);
      const float v = __uint_as_float(code[u] ? code[u] << 23 : 0x00400000u);
      info[lane] = lane < 16 ? (code[u] == 255 ? NAN : v) : e;
      if (lane == 0) info[32] = __uint_as_float(on[u]);
    }
  };

  int page_next[kUnits];
  {
    int page[kStages - 1][kUnits];
    uint32_t code[kStages - 1][kUnits], on[kStages - 1][kUnits];
    enter();
    ask(page_next);
#pragma unroll
    for (int n = 0; n < kStages - 1; ++n) {
#pragma unroll
      for (int u = 0; u < kUnits; ++u) page[n][u] = page_next[u];
      copy(n, page[n], code[n], on[n]);
      advance();
      ask(page_next);
    }
#pragma unroll
    for (int n = 0; n < kStages - 1; ++n) settle(n, code[n], on[n]);
  }

  int stage = 0;
  for (int done = 0; done < entered; ++done) {
    __syncwarp();
    const Row mine = queue[done % kQueue];
    const int kvh = mine.row / a.groups, head0 = kvh * a.share + (mine.row - kvh * a.groups) * kCols;
    const int heads = min(kCols, (kvh + 1) * a.share - head0);

    // queries, times a power of two per head; heads past the group's repeat as zero
    uint32_t q[NT][kKey][8];
    float qs[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      uint4 raw[kKey][2];
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < kKey; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int d = 64 * i + 16 * t + 8 * h;
          raw[i][h] = 8 * n + g < heads && d < D
                          ? load16(static_cast<const T *>(a.p.q) + mine.s * a.p.q_seq + (head0 + 8 * n + g) * a.p.q_head + d)
                          : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {raw[i][h].x, raw[i][h].y, raw[i][h].z, raw[i][h].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 v = unpack<T>(w[j]);
            top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
          }
        }
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
      // 2^e times the largest is at least 2^14 and below 2^15
      const int e = top > 0.0f ? min(14 + 127 - (int)(__float_as_uint(top) >> 23), 126) : 0;
      const float f = __uint_as_float((uint32_t)(e + 127) << 23);
      const float back = a.scale2 * __uint_as_float((uint32_t)(127 - e) << 23);
      qs[n][0] = __shfl_sync(~0u, back, 8 * t);
      qs[n][1] = __shfl_sync(~0u, back, 8 * t + 4);
#pragma unroll
      for (int i = 0; i < kKey; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t w[4] = {raw[i][h].x, raw[i][h].y, raw[i][h].z, raw[i][h].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 v = unpack<T>(w[j]);
            q[n][i][4 * h + j] = pack<__half>(v.x * f, v.y * f);
          }
        }
    }

    float m[NT][2], mo[NT][2], l[NT][2], o[NT][2 * kWords][4];
    bool seen = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = mo[n][0] = mo[n][1] = kNone;
      l[n][0] = l[n][1] = 0.0f;
#pragma unroll
      for (int i = 0; i < 2 * kWords; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.0f;
    }

    for (int left = mine.tiles; left > 0; --left) {
      copies_wait<kStages - 2>();
      __syncwarp();  // the scales that other lanes put there
      uint32_t code_next[kUnits], on_next[kUnits];
      const int free = stage == 0 ? kStages - 1 : stage - 1;
      copy(free, page_next, code_next, on_next);
      advance();
      ask(page_next);

      const char *const here = ring + stage * kUnits * unit_bytes(DP);
      float sc[kUnits][NT][4], so[kUnits][NT][4];
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const char *const kp = here + u * unit_bytes(DP);
#pragma unroll
        for (int n = 0; n < NT; ++n) sc[u][n][0] = sc[u][n][1] = sc[u][n][2] = sc[u][n][3] = 0.0f;
#pragma unroll
        for (int i = 0; i < kKey; ++i) {
          const uint4 k0 = *reinterpret_cast<const uint4 *>(kp + Layout<DP>::key_at(g, t, i));
          const uint4 k1 = *reinterpret_cast<const uint4 *>(kp + Layout<DP>::key_at(g, t, i) + 8 * DP);
          const uint32_t x[4] = {k0.x, k0.y, k0.z, k0.w}, y[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t x0, x1, y0, y1;
            e4m3_halves(x[j], x0, x1);
            e4m3_halves(y[j], y0, y1);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma(sc[u][n], x0, y0, x1, y1, q[n][i][2 * j], q[n][i][2 * j + 1], __half());
          }
        }
      }
      // scores: lane (g, t) has positions g, g + 8 of heads 2 t, 2 t + 1
      bool passed = false;
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const float *info = reinterpret_cast<const float *>(here + u * unit_bytes(DP) + 32 * DP);
        const uint32_t on = __float_as_uint(info[32]);
        const float ks[2] = {info[g], info[g + 8]}, ve[2] = {info[16 + g], info[24 + g]};
        seen |= on != 0;
        const bool on0 = on >> g & 1, on1 = on >> (g + 8) & 1;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float qk[4] = {qs[n][0] * ks[0], qs[n][1] * ks[0], qs[n][0] * ks[1], qs[n][1] * ks[1]};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sc[u][n][e] = (e >> 1 ? on1 : on0) ? sc[u][n][e] * qk[e] : -INFINITY;
            so[u][n][e] = sc[u][n][e] + ve[e >> 1];
            passed |= sc[u][n][e] > m[n][e & 1] + kSlack || so[u][n][e] > mo[n][e & 1] + kSlack;
          }
        }
      }
      if (__any_sync(~0u, passed)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = m[n][e], topo = mo[n][e];
#pragma unroll
            for (int u = 0; u < kUnits; ++u) {
              top = fmaxf(top, fmaxf(sc[u][n][e], sc[u][n][2 + e]));
              topo = fmaxf(topo, fmaxf(so[u][n][e], so[u][n][2 + e]));
            }
#pragma unroll
            for (int x = 4; x <= 16; x <<= 1) {
              top = fmaxf(top, __shfl_xor_sync(~0u, top, x));
              topo = fmaxf(topo, __shfl_xor_sync(~0u, topo, x));
            }
            l[n][e] *= ex2(m[n][e] - top);
            const float fade = ex2(mo[n][e] - topo);
            m[n][e] = top;
            mo[n][e] = topo;
#pragma unroll
            for (int i = 0; i < 2 * kWords; ++i) {
              o[n][i][e] *= fade;
              o[n][i][2 + e] *= fade;
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
            l[n][e & 1] += ex2(sc[u][n][e] - m[n][e & 1]);
            w[e] = ex2(so[u][n][e] - (mo[n][e & 1] - kLift));
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t p = pack<__half>(w[2 * h], w[2 * h + 1]);
            const float2 r = unpack<__half>(p);
            hi[n][h] = transpose8x8(p);
            lo[n][h] = transpose8x8(pack<__half>(w[2 * h] - r.x, w[2 * h + 1] - r.y));
          }
        }
        const char *vp = here + u * unit_bytes(DP) + 16 * DP;
#pragma unroll
        for (int i = 0; i < kV16 + kV8; ++i) {
          uint32_t v[4][4];
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            if (i < kV16) {
              const uint4 w = *reinterpret_cast<const uint4 *>(vp + Layout<DP>::value_at(g, t, h, i));
              v[h][0] = w.x, v[h][1] = w.y, v[h][2] = w.z, v[h][3] = w.w;
            } else {
              const uint2 w = *reinterpret_cast<const uint2 *>(vp + Layout<DP>::value8_at(g, t, h));
              v[h][0] = w.x, v[h][1] = w.y;
            }
          }
#pragma unroll
          for (int j = 0; j < (i < kV16 ? 4 : 2); ++j)
#pragma unroll
            for (int p = 0; p < 2; ++p) {  // rows g, g + 8: elements 2 p, 2 p + 1 of the word
              uint32_t a0, a1, a2, a3;
              e4m3_halves(__byte_perm(v[0][j], v[1][j], p ? 0x7362 : 0x5140), a0, a1);
              e4m3_halves(__byte_perm(v[2][j], v[3][j], p ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                float *d = o[n][2 * (4 * i + j) + p];
                mma(d, a0, a1, a2, a3, hi[n][0], hi[n][1], __half());
                mma(d, a0, a1, a2, a3, lo[n][0], lo[n][1], __half());
              }
            }
        }
      }
      settle(free, code_next, on_next);
      stage = stage == kStages - 1 ? 0 : stage + 1;
    }

    // the row's outputs relative to mo, sums relative to m, both 2^lift<T>() times:
    // the result, or a partial row for the join (clusters: in this warp's ring,
    // which is done with)
    const bool whole = mine.ends == 3;
    const int pitch = a.direct ? DP + 8 : DP;
    float *outs = part_of(warp);
    float4 *stats = st_sh + warp * kCols;
    if (!whole && a.direct) {
      if (lane == 0) part_sh[warp] = true;
      copies_wait<0>();
      __syncwarp();
    } else if (!whole) {
      const int64_t slice = (int64_t)blockIdx.x * (kWarps / a.bundle) + warp / a.bundle;
      outs = a.ws + ((slice * 2 + (mine.ends & 1)) * a.bundle + warp % a.bundle) * slot_floats(kCols, DP);
      stats = reinterpret_cast<float4 *>(outs + kCols * DP);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[n][e] * exp2f(lift<T>());
        sum += __shfl_xor_sync(~0u, sum, 4);
        sum += __shfl_xor_sync(~0u, sum, 8);
        sum += __shfl_xor_sync(~0u, sum, 16);
        const int col = 8 * n + 2 * t + e;
        if (col >= heads) continue;
        // (no maximum: nothing seen, or sums that are NaN already)
        if (m[n][e] == kNone) m[n][e] = -INFINITY;
        if (mo[n][e] == kNone) mo[n][e] = -INFINITY;
        float w = exp2f(lift<T>() - kLift);
        const float half = whole ? half_shift(m[n][e], mo[n][e]) : 1.0f;
        if (whole) w = seen ? w / sum : 0.0f;
#pragma unroll
        for (int x = 0; x < kWords / 2; ++x) {
          const int d = x < 2 * kV16 ? 128 * (x / 2) + 16 * g + 8 * (x % 2) : 128 * kV16 + 8 * g;
          float v[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[2 * j] = shifted(o[n][4 * x + j][e] * w, half);
            v[2 * j + 1] = shifted(o[n][4 * x + j][2 + e] * w, half);
          }
          if (!whole) {
            float4 *to = reinterpret_cast<float4 *>(outs + col * pitch + d);
            to[0] = make_float4(v[0], v[1], v[2], v[3]);
            to[1] = make_float4(v[4], v[5], v[6], v[7]);
          } else if (d < D) {
            store8<T>(a, mine.s, head0 + col, d, v);
          }
        }
        if (g == 0) {
          if (!whole)
            stats[col] = make_float4(m[n][e], sum, seen ? kSeen : kThere, mo[n][e]);
          else if (a.p.lse)
            store_lse<T, true>(a, mine.s, head0 + col, seen, m[n][e], sum);
        }
      }
  }

  if (bad) raise_status(a.status, kStatusIndex);
  if (!a.direct) return;

  // join the warps' parts of the row
  copies_wait<0>();
  __syncthreads();
  const int row = mine_row - s * rows, kvh = row / a.groups, head0 = kvh * a.share + (row - kvh * a.groups) * kCols;
  const int heads = min(kCols, (kvh + 1) * a.share - head0);
  const uint32_t parts = __ballot_sync(~0u, part_sh[lane % kWarps]) & ((1u << kWarps) - 1);
  const bool partial = parts != 0 && a.direct > 1;
  if (parts)
    for (int item = threadIdx.x; item < heads * (DP / 8); item += kThreads) {
      const int col = item / (DP / 8), d = 8 * (item % (DP / 8));
      if (d >= D) continue;
      const Whole r = join_all<kWarps, true>([&](int q, float4 &st, float4 &lo, float4 &hi) {
        if (!(parts >> q & 1)) return;
        const float *from = part_of(q) + col * (DP + 8) + d;
        st = st_sh[q * kCols + col];
        lo = *reinterpret_cast<const float4 *>(from);
        hi = *reinterpret_cast<const float4 *>(from + 4);
      });
      if (a.direct == 1) {
        finish<T, true>(a, s, head0 + col, d, r.j, r.seen);
        continue;
      }
      const float *v = r.j.v;
      float *out = part + col * DP + d;
      *reinterpret_cast<float4 *>(out) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4 *>(out + 4) = make_float4(v[4], v[5], v[6], v[7]);
      if (d == 0)
        *reinterpret_cast<float4 *>(part + kCols * DP + col * 4) =
            make_float4(r.j.top, r.j.sum, r.seen ? kSeen : kThere, r.j.topo);
    }
  if (a.direct < 2) return;

  // join the cluster's partial rows, an output piece a thread, in CTA order
  if (!partial)
    for (int i = threadIdx.x; i < slot_floats(kCols, DP); i += kThreads)
      part[i] = i >= kCols * DP && (i % 4 == 0 || i % 4 == 3) ? -INFINITY : 0.0f;
  cg::this_cluster().sync();
  for (int item = threadIdx.x * a.direct + rank; item < heads * (DP / 8); item += kThreads * a.direct) {
    const int col = item / (DP / 8), d = 8 * (item % (DP / 8));
    if (d >= D) continue;
    const Whole r = join_all<kCluster, true>([&](int q, float4 &st, float4 &lo, float4 &hi) {
      if (q >= a.direct) return;
      const float *from = cg::this_cluster().map_shared_rank(part, q);
      st = *reinterpret_cast<const float4 *>(from + kCols * DP + col * 4);
      lo = *reinterpret_cast<const float4 *>(from + col * DP + d);
      hi = *reinterpret_cast<const float4 *>(from + col * DP + d + 4);
    });
    if (r.there) finish<T, true>(a, s, head0 + col, d, r.j, r.seen);
  }
  cg::this_cluster().sync();  // nobody leaves while its part may be read
}

// CTAs (a cluster) that take a row of up to `reach` positions between them, as
// in attention.cu; 0: equal slices.
int cluster_of(int64_t rows, int64_t reach, int dp, int nt) {
  const int64_t sms = sm_count(), fit = sms * per_sm8(dp);
  int n = 1;
  while (n < kCluster && rows * 2 * n <= fit * 7 / 8 &&
         (rows * 2 * n <= sms ? n : 2 * n) * kWarps * 16 * units8(dp) < reach)
    n *= 2;
  const int64_t most = rows > fit ? 128 : n == kCluster ? 2048 : 384 * n;
  return reach <= most ? n : 0;
}

template <typename T, int DP, int NT, bool UNITS>
fp4_status launch(At8Params b, cudaStream_t s) {
  constexpr int kMaxDev = 64;
  static std::atomic<int> occupancy[kMaxDev];
  constexpr int cols = 8 * NT;
  constexpr size_t smem = kWarps * (ring_bytes(DP) + cols * sizeof(float4));
  constexpr size_t part = slot_floats(cols, DP) * sizeof(float);
  static_assert(ring_bytes(DP) >= part_bytes(cols, DP), "a part takes the place of a ring");
  auto kern = k_attention8<T, DP, NT, UNITS>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return FP4_ERR_CUDA;
  int per = occupancy[dev].load(std::memory_order_acquire);
  if (!per) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(smem + part)) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, kThreads, smem) != cudaSuccess || per < 1)
      return FP4_ERR_CUDA;
    occupancy[dev].store(per, std::memory_order_release);
  }
  AtParams &a = b.a;
  const fp4_kv_cache &c = a.p.cache;
  a.tile = 16 * units8(DP);
  b.k_step = Layout<DP>::kRows * c.k_place;
  b.v_step = Layout<DP>::kRows * c.v_place;
  const int64_t rows = (int64_t)c.seqs * c.kv_heads * a.groups;
  const int64_t room = (int64_t)c.seq_pages * c.page_size;
  const int64_t most = (int64_t)sm_count() * (per < kPerSM8 ? per : kPerSM8);
  if (rows > INT32_MAX) return FP4_ERR_SHAPE;
  // by what a window and the first positions reach, but by slices only where the
  // workspace, which knows the table's room alone, has been asked for
  const int64_t reach = (int64_t)a.p.window + 15 + ceil_div(a.p.sinks, a.tile) * a.tile;
  const int by_room = cluster_of(rows, room, DP, NT);
  a.direct = a.p.window && reach < room ? cluster_of(rows, reach, DP, NT) : by_room;
  if (!a.direct) a.direct = by_room;
  if (!a.direct && !a.ws) return FP4_ERR_INVALID_ARG;
  const int each = c.kv_heads * a.groups;
  a.bundle = a.direct ? 1 : each % kWarps == 0 ? kWarps : each % 2 == 0 ? 2 : 1;
  a.least = 4;
  const int subs = kWarps / a.bundle;
  const int64_t want = ceil_div(rows / a.bundle * ceil_div(room, a.tile), subs);  // no more than the table has tiles
  const int64_t grid = a.direct ? rows * a.direct : want < most ? want : most;
  a.ctas = (int)grid * subs;
  if (a.direct) {
    const size_t bytes = smem + (a.direct > 1 ? part : 0);
    return launch_dependent_clusters(kern, a.direct, dim3((unsigned)grid), dim3(kThreads), bytes, s, b) == cudaSuccess
               ? FP4_OK
               : FP4_ERR_CUDA;
  }
  kern<<<(unsigned)grid, kThreads, smem, s>>>(b);  // (an ordinary launch, as in attention16.cuh)
  if (cudaGetLastError() != cudaSuccess) return FP4_ERR_CUDA;
  if (a.ctas < 2) return FP4_OK;
  const cudaError_t e =
      rows * 4 <= (int64_t)a.ctas * a.bundle
          ? launch_dependent(k_attention_join<T, DP, NT, kWide8, true, true>, dim3((unsigned)rows), dim3(kWide8), 0, s, a)
          : launch_dependent(k_attention_join<T, DP, NT, kNarrow, true, true>, dim3((unsigned)((a.ctas - 1) * a.bundle)), dim3(kNarrow), 0,
                             s, a);
  return e == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

template <typename T, int DP, int NT>
fp4_status launch_pages(const At8Params &b, cudaStream_t s) {
  const fp4_kv_cache &c = b.a.p.cache;
  const int64_t far = c.k_page | c.k_place | c.v_page | c.v_place | b.s.k_page | b.s.k_block | b.s.v_page | b.s.v_block;
  return c.page_size % 16 == 0 && far <= INT32_MAX ? launch<T, DP, NT, true>(b, s) : launch<T, DP, NT, false>(b, s);
}

template <typename T>
fp4_status launch_type(const At8Params &b, int nt, cudaStream_t s) {
  switch (dp_of(b.a.p.cache.head_dim)) {
    case 64: return nt == 1 ? launch_pages<T, 64, 1>(b, s) : launch_pages<T, 64, 2>(b, s);
    case 128: return nt == 1 ? launch_pages<T, 128, 1>(b, s) : launch_pages<T, 128, 2>(b, s);
    case 192: return launch_pages<T, 192, 1>(b, s);
    default: return launch_pages<T, 256, 1>(b, s);
  }
}

}  // namespace

int64_t decode_attention8_workspace(int64_t seqs, int64_t room, int heads, int kv_heads, int head_dim) {
  const int dp = dp_of(head_dim), nt = nt_of(heads / kv_heads, dp), cols = 8 * nt;
  if (cluster_of(seqs * kv_heads * ceil_div(heads / kv_heads, cols), room, dp, nt)) return 0;
  return (int64_t)sm_count() * kPerSM8 * kWarps * 2 * slot_floats(cols, dp) * sizeof(float);
}

fp4_status launch_decode_attention8(const fp4_attention8_params &p, cudaStream_t s) {
  At8Params b{};
  AtParams &a = b.a;
  a.p = p.base;
  b.s = p.scales;
  a.status = status_word();
  if (!a.status) return FP4_ERR_CUDA;
  const fp4_kv_cache &c = a.p.cache;
  a.share = a.p.heads / c.kv_heads;
  const int nt = nt_of(a.share, dp_of(c.head_dim));
  a.groups = (a.share + 8 * nt - 1) / (8 * nt);
  b.page = divisor(c.page_size);
  b.block = divisor(b.s.block);
  b.k_page = (int)c.k_page, b.k_place = (int)c.k_place, b.v_page = (int)c.v_page, b.v_place = (int)c.v_place;
  b.ks_page = (int)b.s.k_page, b.ks_block = (int)b.s.k_block, b.vs_page = (int)b.s.v_page, b.vs_block = (int)b.s.v_block;
  a.out16 = aligned16(a.p.out) && a.p.out_seq % 8 == 0 && a.p.out_head % 8 == 0;
  a.scale2 = a.p.scale * 1.44269504088896f;
  a.ws = static_cast<float *>(a.p.workspace);
  return c.type == FP4_BF16 ? launch_type<__nv_bfloat16>(b, nt, s) : launch_type<__half>(b, nt, s);
}

}  // namespace fp4
