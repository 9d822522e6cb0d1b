// matvec.cu -- y = x W^T for a few tokens, W a 4-bit copy with block scales,
// x in 16 bits (sm_103a):
//   y[m][n] = s_dec 2^shift[n] sum_b dec(sf[n][b]) sum_{k in b} e2m1(q[n][k]) x[m][k]
//
// Bound: HBM, 0.5 + 1/B bytes per weight read once.  At 6.8 TB/s an SM has
// 23 clocks, 90 issue slots, for every 16 x 64 weights, and two instructions a
// pair (decode, scale) already take 32 of them; so the rest of the arithmetic
// is the m16n8k16 f16 MMA with the weight as its 16-row operand and up to 8 NT
// tokens as columns.  (tcgen05 multiplies 4-bit weights as they lie only with
// activations of at most 8 bits: 16-bit ones would have to be split into parts,
// or the weights decoded into shared or tensor memory first.)
// Measured (131072 x 4096, NVFP4): 1 token 52.2 us (5.8 TB/s, 85% of a copy),
// 8 tokens 58.9 us (76%), 16 tokens 81 us (57%): instruction issue, about 480
// instructions for 32 x 256 weights and 8 tokens of which 304 decode, scale
// and multiply, at half an instruction a clock and scheduler.  4096 x 14336,
// 1 token: 11.3 us behind another of its kind (a dependent launch: barriers and
// parameters are set up while the kernel before drains; 13.1 without).
//
// Mathematics.  E2M1 has 2 significant bits, a block scale at most 4, so
// e2m1 * dec(sf) is exact in f16 for E4M3 (2^-10 .. 2,688) and times 2^-3 for
// UE5M3 (2^-21 .. 46,080).
// E8M0 scales span more than f16: per row and 256 columns they are taken
// relative to the largest of the eight (2^13 at most, exact 36 binades down)
// and the largest is applied in binary32.  A BF16 x is multiplied per token
// and 256 columns by the power of two that puts its largest magnitude in
// [2^15, 2^16): 8 significant bits stay exact in f16 for 32 binades below
// it.  Products are exact, the MMA adds 256 columns in binary32, and these
// sums are multiplied by the power(s) of two and added in binary32 with
// nearest rounding.
//
// Layout.  A warp takes 32 weight rows (16 above 8 tokens) and 256 columns a
// step.  The order of k within an MMA is free as long as both operands share
// it: lane (g, t) takes columns 64 t .. 64 t + 63 of rows g, g + 8, .. -- four
// 16-byte pieces of payload and the scale codes over 64 columns of each, whole
// loads and no exchange between lanes -- and each MMA four of its weights.  The
// payload comes as TMA boxes of 128 bytes a row in the 128-byte swizzle (rows
// g, g + 1 of a quarter-warp then read different banks), the scales as a box
// of their own (Words); x lies in shared memory as f16, the 16-byte pieces of
// 256 columns in the order (piece of the lane, t), so that four lanes read 64
// contiguous bytes, tokens 64 mod 128 bytes apart.
//
// Split.  One CTA of up to 16 warps per SM; each warp runs its own ring of 2
// to 4 stages with an mbarrier each, filled by its lane 0 as soon as a stage
// is in registers, so that 64 KB or more of weights are in flight per SM
// across tiles and before x is ready, and no warp waits for another inside a
// tile.  The CTA holds x for its K range; sk of its warps share a row tile
// along K, and a cluster of S CTAs splits K where x for all of it does not
// fit.  The parts are added in shared memory (over the cluster: distributed)
// in a fixed order.  A row pitch that is not a multiple of 16 bytes (K / 16
// odd) is no TMA stride: the ring is then filled by 8-byte cp.async.
#include <cooperative_groups.h>

#include "serve.cuh"
#include "tcgen05.cuh"

namespace fp4 {

namespace {

namespace cg = cooperative_groups;

constexpr int kStep = 256;             // columns a step
constexpr int kMaxDepth = 4;
constexpr int kMaxSmem = 227 * 1024;

constexpr int kMaxWarps = 16;
// Weight rows of a tile: two MMA row tiles share the loads of x; with two
// token tiles one, so that 16 warps have the registers and, beside twice the
// x, the shared memory (131072 x 4096, 16 tokens, when this was chosen: 95 us,
// with 32 rows and 12 warps 103; 81 now).
constexpr int rows_of(int nt) { return nt == 1 ? 32 : 16; }
constexpr int payload_of(int nt) { return rows_of(nt) * kStep / 2; }  // bytes of a stage

struct MvParams {
  CUtensorMap map;   // payload [N][K / 2], boxes of 8, 16 or 32 rows x 128 bytes
  CUtensorMap smap;  // scales, see Words
  MatvecJob j;
  int steps;         // ceil(K / 256)
  int tiles;         // of all rows, N rounded up to 128
  int warps;         // of a CTA
  int sk, S;         // warps and CTAs that share a tile along K
  int rounds;        // row tiles a warp takes, one after the other
  int clusters;
  int mc;            // tokens a CTA takes (blockIdx.y counts them off)
  int depth;         // stages of a warp's ring
  int words;         // how scales reach shared memory: Words
  int tma;           // payload by TMA: rows of whole 16 bytes
  uint32_t *status;
};

// 2^e as binary32, e in [-149, 127].
__device__ __forceinline__ float pow2(int e) {
  return __uint_as_float(e >= -126 ? (uint32_t)(e + 127) << 23 : 1u << (e + 149));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Both halves of a by the low (hi = false) or high half of s.
__device__ __forceinline__ uint32_t hmul2_by(uint32_t a, uint32_t s, bool hi) {
  const __half2 v = *reinterpret_cast<const __half2 *>(&s);
  const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), hi ? __high2half2(v) : __low2half2(v));
  return *reinterpret_cast<const uint32_t *>(&r);
}

// The four bytes of w as four f16 pairs (E2M1 -> f16, exact).
__device__ __forceinline__ void decode8(uint32_t w, uint32_t *h) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

__device__ __forceinline__ void mma(float *d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four bytes, of which the first `bytes` are read and the rest zero.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(on ? 8 : 0)
               : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x,
                                            int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
      "%4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// The lane's arrival, when its cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Scales of a stage in shared memory, and the rows of a tile.
//   kTiled: the tensor-core layout.  512-byte tiles hold 32 lines of 16 bytes,
//     the words of rows l, l + 32, l + 64, l + 96 of their 128 rows; so a
//     tile of weight rows is 4 (of 16 rows: 2) groups of 8 rows 32 apart, its
//     payload a TMA box for each, and its scales lie in 128 contiguous bytes
//     of each 64 (or, 32-element blocks, 128) columns: one box.  Lane (g, t)
//     finds its words in 16 bytes at 128 t + 16 g (t / 2 for 32-blocks).
//   kBoxed: plain rows with a pitch of whole 16 bytes: one box of the rows x
//     16 bytes (with 32-element blocks the 16 bytes that hold the step's 8);
//     word i of a lane at 128 i + 4 lane (row g + 8 i, word t).
//   kPieces: plain rows of any other pitch, by 4-byte cp.async: the whole words
//     that a row's bytes lie in, in the same places.  Where rows do not begin
//     with words, a lane's codes are cut out of two words as they are read,
//     and each row has one word more from 512 on.  (30000 x 2064, 1 token: 18.2
//     us; with byte loads, which a fill waited for, 35.1.)
enum Words { kTiled = 0, kBoxed = 1, kPieces = 2 };
// A kernel's MODE is kTiled or kBoxed with the payload by TMA, or kAny: tiled
// scales with the payload by copies, or pieces with either, as the parameters
// say.
constexpr int kAny = 2;
constexpr int words_of(int mode) { return mode == kAny ? 640 : 512; }  // scale bytes of a stage

// Fills a warp's stages one after the other.
template <int BLOCK, int MODE, int kRows>
struct Loader {
  static constexpr int kPayload = kRows * kStep / 2, kGroups = kRows / 8;
  int step, row0;        // of the next stage: row0 the tile's first row

  // kTiled: tile i of a 128-row group holds lines 8 (i % 4) ... of its words 0 .. 3
  // (16 rows: 0, 1, then 2, 3).
  static __device__ __forceinline__ int64_t first_row(int64_t tile, bool tiled) {
    if (!tiled) return tile * kRows;
    if (kRows == 32) return (tile >> 2) * 128 + (tile & 3) * 8;
    return (tile >> 3) * 128 + ((tile >> 2) & 1) * 64 + (tile & 3) * 8;
  }

  __device__ __forceinline__ void fill(const MvParams &p, uint32_t payload, uint32_t words,
                                       uint32_t bar, int lane) {
    const MatvecJob &j = p.j;
    const bool tiled = (MODE == kAny ? p.words : MODE) == kTiled, tma = MODE != kAny || p.tma;
    constexpr int kPer = kStep / BLOCK;  // scale bytes of a row and step
    if (lane == 0) {
      // full boxes count, whatever part of them lies outside
      const uint32_t bytes = (tma ? kPayload : 0) + (MODE == kBoxed ? kRows * 16 : tiled ? 32 * kPer : 0);
      if (MODE != kAny || bytes) tc::mbar_expect_tx(bar, bytes);
      if (tma) {
        if (MODE == kTiled) {
#pragma unroll
          for (int i = 0; i < kGroups; ++i)
            tc::tma_load_2d(payload + 1024 * i, &p.map, bar, step * (kStep / 2), row0 + 32 * i);
        } else {
          tc::tma_load_2d(payload, &p.map, bar, step * (kStep / 2), row0);
        }
      }
      if (tiled)
        tma_load_3d(words, &p.smap, bar, (row0 & 31) * 16, step * (kPer / 4), row0 >> 7);
      else if (MODE == kBoxed)
        tc::tma_load_2d(words, &p.smap, bar, step * kPer & ~15, row0);
    }
    ++step;
    if (MODE != kAny) return;
    if (!tma) {
      // 16 pieces of 8 bytes a row; lane: piece lane % 16 of every other row,
      // in the swizzled place the TMA would use
      const int half = (int)(j.K / 2), odd = lane >> 4, at = (step - 1) * (kStep / 2) + (lane & 15) * 8;
      const int rows = at < half ? (int)max((int64_t)0, min(j.N - row0 - odd, (int64_t)1024)) : 0;
      const uint8_t *from = j.q + (rows ? (int64_t)(row0 + odd) * half + at : 0);
      const uint32_t to = payload + odd * 128 + (lane & 1) * 8;
#pragma unroll
      for (int i = 0; i < kRows / 2; ++i) {
        const int r = tiled ? 32 * (i >> 2) + 2 * (i & 3) : 2 * i;  // and `odd`
        const bool on = r < rows;
        cp_async8(to + 256 * i + ((((lane & 15) >> 1) ^ odd ^ (2 * (i & 3))) << 4), from + (on ? r * half : 0), on);
      }
    }
    if (!tiled) {
      // offsets from the tile's first row, whose place is a multiple of 16; a
      // row's first word may begin in the row before
      const int blocks = (int)(j.K / BLOCK), first = (step - 1) * kPer;
      const int64_t begin = (int64_t)row0 * blocks;
      const int left = (int)max((int64_t)0, min(j.N * blocks - begin, (int64_t)kRows * blocks + 64));
      const uint8_t *from = j.sf + (left ? begin : 0);
      auto copy = [&](uint32_t dst, int at) {
        const int bytes = min(max(left - at, 0), 4);
        cp_async4(dst, from + (bytes ? at : 0), bytes);
      };
      int at = ((lane >> 2) * blocks & ~3) + first + (BLOCK == 16 ? 4 * (lane & 3) : 2 * (lane & 2));
#pragma unroll
      for (int i = 0; i < kGroups; ++i, at += 8 * blocks) copy(words + 128 * i + 4 * lane, at);
      if ((blocks & 3) && lane < kRows) copy(words + 512 + 4 * lane, (lane * blocks & ~3) + first + kPer);
    }
    cp_async_arrive(bar);
  }
};

// The f16 scales over 32 of the lane's 64 columns of one row, from the codes
// at the bottom of w: two blocks of 16 (low and high half), or one of 32.
template <int KIND, int BLOCK>
__device__ __forceinline__ uint32_t scale_pair(uint32_t w, int top) {
  if (KIND == kMXFP4) {
    // 2^(code - top + 13): f16 exponent field 28 + code - top, subnormal below 1
    const int e = 28 + (int)(w & 255u) - top;
    return (e >= 1 ? (uint32_t)e << 10 : e >= -9 ? 1u << (e + 9) : 0u) * 0x10001u;
  }
  if (BLOCK == 32) w = __byte_perm(w, 0, 0x4400);  // the one code twice
  if (KIND == kNVFP4) {
    uint32_t h;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(w));
    return h;
  }
  // E5M3 is the head of an f16; times 2^-3 to leave room for a product
  return hmul2(__byte_perm(w, 0, 0x1404) >> 1, 0x30003000u);
}

template <typename TX>
struct Is {
  static constexpr bool bf16 = false;
};
template <>
struct Is<__nv_bfloat16> {
  static constexpr bool bf16 = true;
};

// Eight BF16 values times the power of two that brings the largest of the
// warp's 256 into [2^15, 2^16), as f16; returns the exponent taken out.
__device__ __forceinline__ int normalize(uint32_t *w) {
  auto as2 = [](uint32_t v) { return *reinterpret_cast<const __nv_bfloat162 *>(&v); };
  const __nv_bfloat162 t = __hmax2(__hmax2(__habs2(as2(w[0])), __habs2(as2(w[1]))),
                                   __hmax2(__habs2(as2(w[2])), __habs2(as2(w[3]))));  // (passes over NaN)
  const uint32_t u = *reinterpret_cast<const uint32_t *>(&t);
  const uint32_t top = __reduce_max_sync(~0u, max(u & 0xFFFFu, u >> 16));
  // exponent of the largest finite magnitude (2^133 x subnormals: 1 + mantissa bits)
  const int f = (int)(top >> 7);
  const int e = f >= 255 ? 127 : f > 0 ? f - 127 : top ? (31 - __clz((int)top)) - 133 : 0;
  const int ex = e - 15;
  if (ex >= -127) {
    const float s = pow2(-ex);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const __half2 v = __floats2half2_rn(bf16_lo(w[q]) * s, bf16_hi(w[q]) * s);
      w[q] = *reinterpret_cast<const uint32_t *>(&v);
    }
  } else {  // binary32 does not hold 2^-ex: two factors
    const float s = pow2(-ex - 64), s2 = 0x1p64f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const __half2 v = __floats2half2_rn(bf16_lo(w[q]) * s * s2, bf16_hi(w[q]) * s * s2);
      w[q] = *reinterpret_cast<const uint32_t *>(&v);
    }
  }
  return ex;
}

// x[0 .. M) over steps [s0, s0 + n) as f16 into shared memory, and the power
// of two taken out of each (token, step); a warp per (token, step), eight
// elements a lane, eight (tokens, or steps of few tokens) requested together.
template <typename TX>
__device__ void prepare_x(const MatvecJob &j, int64_t m0, int M, int s0, int n, uint8_t *xs, int pitch,
                          float *sx, int cols, int warps) {
  const TX *x = static_cast<const TX *>(j.x) + m0 * j.xs;
  const bool vec = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && (M == 1 || j.xs % 8 == 0);
  const int warp = threadIdx.x >> 5, piece = threadIdx.x & 31;
  const int across = min(warps, n), deep = warps / across;  // warps along K, and along the tokens
  if (warp >= across * deep) return;
  constexpr int kBatch = 8;
  const bool few = M < kBatch * deep;
  const int dm = few ? 0 : deep, dc = few ? across : 0;  // from one of a batch to the next
  for (int c = warp % across; c < n; c += few ? kBatch * across : across) {
    for (int m = warp / across; m < M; m += few ? deep : kBatch * deep) {
      int k = (s0 + c) * kStep + piece * 8;
      const TX *from = x + m * j.xs + k;
      uint32_t w[kBatch][4];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        w[i][0] = w[i][1] = w[i][2] = w[i][3] = 0;
        // K is a multiple of 16: a piece is inside or outside
        if (m + i * dm < M && c + i * dc < n && k < (int)j.K) {
          if (vec) {
            const uint4 v = *reinterpret_cast<const uint4 *>(from);
            w[i][0] = v.x, w[i][1] = v.y, w[i][2] = v.z, w[i][3] = v.w;
          } else {
            const uint16_t *e = reinterpret_cast<const uint16_t *>(from);
#pragma unroll
            for (int q = 0; q < 4; ++q) w[i][q] = e[2 * q] | ((uint32_t)e[2 * q + 1] << 16);
          }
        }
        from += dm * j.xs + dc * kStep;
        k += dc * kStep;
      }
      // piece q of lane t (piece = 8 t + q) lies at 64 q + 16 t
      uint8_t *to = xs + m * pitch + c * 512 + (piece & 7) * 64 + (piece >> 3) * 16;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (m + i * dm >= M || c + i * dc >= n) break;
        int ex = 0;
        if (Is<TX>::bf16) ex = normalize(w[i]);
        *reinterpret_cast<uint4 *>(to) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
        to += dm * pitch + dc * 512;
        if (piece == 0) sx[(c + i * dc) * cols + m + i * dm] = pow2(ex);
      }
    }
  }
}

template <int KIND, int BLOCK, int MODE, typename TX, int NT>
__global__ void __launch_bounds__(32 * kMaxWarps, 1) k_matvec(const __grid_constant__ MvParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int kCols = 8 * NT, kRows = rows_of(NT), kPayload = payload_of(NT), kWords = words_of(MODE);
  constexpr int kPairs = kRows / 16, kGroups = kRows / 8;  // MMA row tiles; rows of a lane
  const int kWarps = p.warps;
  const MatvecJob &j = p.j;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int S = p.S, sk = p.sk, depth = p.depth;
  const int rank = blockIdx.x % S, cluster = blockIdx.x / S;
  const int64_t m0 = (int64_t)blockIdx.y * p.mc;
  const int M = (int)min((int64_t)p.mc, j.M - m0);
  // the CTA's steps, and the warp's share of them
  const int c0 = (int)((int64_t)p.steps * rank / S), c1 = (int)((int64_t)p.steps * (rank + 1) / S);
  const int kw = warp % sk, tw = warp / sk, group = kWarps / sk;
  const int n = c1 - c0;
  const int s0 = c0 + n * kw / sk, ns = c0 + n * (kw + 1) / sk - s0;
  const int pitch = n * 512 + 64;
  const int span = (p.steps + S - 1) / S;  // same on every CTA of the cluster
  uint8_t *ring = smem + warp * depth * kPayload;
  uint8_t *word_ring = smem + kWarps * depth * kPayload + warp * depth * kWords;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kWarps * depth * (kPayload + kWords)) + warp * kMaxDepth;
  float *sx = reinterpret_cast<float *>(smem + kWarps * depth * (kPayload + kWords) + kWarps * kMaxDepth * 8);
  float *parts = sx + span * kCols;  // [kWarps][kCols][kRows]
  uint8_t *xs = reinterpret_cast<uint8_t *>(parts + kWarps * kRows * kCols);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(xs + p.mc * (span * 512 + 64));
  const uint32_t ring_a = tc::smem_u32(ring), words_a = tc::smem_u32(word_ring), bars_a = tc::smem_u32(bars);

  // the warp's own ring: one arrival that expects the boxes of a stage, if it
  // has any, and in kAny 32 lanes' for their own copies
  const bool boxes = MODE != kAny || p.tma || p.words == kTiled;
  if (threadIdx.x == 0) *abort_flag = 0;
  if (lane == 0) {
    for (int d = 0; d < depth; ++d) tc::mbar_init(bars_a + 8 * d, (boxes ? 1 : 0) + (MODE == kAny ? 32 : 0));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  __syncwarp();
  dependent_wait();
  launch_dependents();
  // the cluster's tiles [t0, t1), `group` a round, and how many of them are the warp's
  const int t0 = (int)((int64_t)p.tiles * cluster / p.clusters), t1 = (int)((int64_t)p.tiles * (cluster + 1) / p.clusters);
  const int tile0 = t0 + tw;
  const int mine = tw < group && tile0 < t1 ? (t1 - 1 - tile0) / group + 1 : 0;
  int ahead = mine * ns;  // stages still to be requested
  int ld_tile = tile0;
  const bool tiled = MODE == kAny ? p.words == kTiled : MODE == kTiled;
  Loader<BLOCK, MODE, kRows> ld;
  ld.step = s0;
  ld.row0 = (int)ld.first_row(tile0, tiled);
  auto issue = [&](int at) {
    ld.fill(p, ring_a + at * kPayload, words_a + at * kWords, bars_a + 8 * at, lane);
    --ahead;
    if (ld.step == s0 + ns) {
      ld.step = s0;
      ld_tile += group;
      ld.row0 = (int)ld.first_row(ld_tile, tiled);
    }
  };
  for (int d = 0; d < depth && ahead; ++d) issue(d);

  prepare_x<TX>(j, m0, M, c0, n, xs, pitch, sx, kCols, p.warps);
  __syncthreads();

  const uint8_t *xl[NT];
#pragma unroll
  for (int b = 0; b < NT; ++b) xl[b] = xs + min(8 * b + g, M - 1) * pitch + t * 16;  // columns past M repeat

  const int at0 = ((2 * t) ^ g) << 4;  // the lane's pieces of a row: at0, at0 ^ 16, then 1024 on
  // kPieces: whether rows begin inside words, where a lane's codes begin in
  // their first word (a tile's first row begins with one) and the place of the
  // second
  bool cut = false;
  int bit = 0, next_at = 0, next_hop = 0;
  // not kBoxed: where K ends inside a word, the bytes of the lane's word in the
  // last step that are inside (what follows is a next row's or padding: it
  // would meet zeros, but may be NaN, or the largest MXFP4 scale of a row)
  uint32_t inside = ~0u;
  const int blocks = (int)(j.K / BLOCK), own = BLOCK == 16 ? t : t >> 1;
  if (MODE != kBoxed) {
    const int left = blocks - (p.steps - 1) * (kStep / BLOCK) - 4 * own;
    inside = left >= 4 ? ~0u : left > 0 ? (1u << (8 * left)) - 1 : 0u;
  }
  const int edge = blocks & 3 ? p.steps - 1 : -1;
  if (MODE == kAny) {
    const bool last = own == kStep / BLOCK / 4 - 1;
    cut = blocks & 3;
    bit = 8 * (g * blocks & 3);
    next_at = last ? 512 + 4 * g : 4 * lane + (BLOCK == 16 ? 4 : 8);
    next_hop = last ? 32 : 128;
  }
  int slot = 0;
  uint32_t phase = 0;
  bool live = true;  // false once a wait ran out: no more loads, results void
  int flying = 0;    // stages in flight when it did
  for (int r = 0; r < p.rounds; ++r) {
    float acc[NT][kPairs][4] = {};
    int largest[kGroups] = {};  // E8M0 codes of the rows
    const int half = kRows == 16 ? ((tile0 + r * group) >> 2 & 1) * 8 : 0;  // kTiled: words 0, 1 or 2, 3
    int xo = (s0 - c0) * 512;
    const float *sxl = sx + (s0 - c0) * kCols + 2 * t;
    for (int st = s0; st < (r < mine && live ? s0 + ns : s0); ++st) {
      if (!__all_sync(~0u, tc::mbar_wait_inl(bars_a + 8 * slot, phase, abort_flag, p.status))) {
        live = false;
        flying = min(depth, (mine - r - 1) * ns + s0 + ns - st);
        break;
      }
      uint32_t codes[kGroups];
      const uint8_t *wl = word_ring + slot * kWords;
      if (tiled) {
        const uint8_t *at = wl + (BLOCK == 16 ? t : t >> 1) * 128 + g * 16;
        if (kRows == 32) {
          const uint4 v = *reinterpret_cast<const uint4 *>(at);
          codes[0] = v.x, codes[1] = v.y, codes[kGroups - 2] = v.z, codes[kGroups - 1] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2 *>(at + half);
          codes[0] = v.x, codes[1] = v.y;
        }
      } else {
        // with 32-element blocks a box holds two steps' words
        const int o = BLOCK == 32 && MODE == kBoxed ? (4 * g + (t >> 1) + 2 * (st & 1)) * 4 : lane * 4;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) codes[i] = *reinterpret_cast<const uint32_t *>(wl + 128 * i + o);
        if (MODE == kAny && cut) {
#pragma unroll
          for (int i = 0; i < kGroups; ++i)
            codes[i] = __funnelshift_r(codes[i], *reinterpret_cast<const uint32_t *>(wl + next_at + next_hop * i), bit);
        }
      }
      if (MODE != kBoxed && __builtin_expect(st == edge, 0)) {
#pragma unroll
        for (int i = 0; i < kGroups; ++i) codes[i] &= inside;
      }
      float f[kGroups];
      int top[kGroups] = {};
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        if (BLOCK == 32 && (t & 1)) codes[i] >>= 16;  // the lane's half of the word
        if (KIND == kMXFP4) {
          top[i] = max((int)(codes[i] & 255u), (int)((codes[i] >> 8) & 255u));
          top[i] = max(top[i], __shfl_xor_sync(~0u, top[i], 1));
          top[i] = max(top[i], __shfl_xor_sync(~0u, top[i], 2));
          f[i] = pow2(top[i] - 140);  // 2^(top - 127) / 2^13
          largest[i] = max(largest[i], top[i]);
        }
      }
      float d[NT][kPairs][4] = {};
      const uint8_t *ra = ring + slot * kPayload + g * 128 + at0;
      // 32 of the lane's 64 columns at a time, a 16-byte piece of each row.
      // Not unrolled: at twice the size the loop outgrew the instruction cache
      // (a third of all stalls for 16 tokens).
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        uint4 w[kGroups];
        uint32_t sc[kGroups];
#pragma unroll
        for (int i = 0; i < kGroups; ++i) w[i] = *reinterpret_cast<const uint4 *>(ra + 1024 * i);
        ra = ring + slot * kPayload + g * 128 + (at0 ^ 16);
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
          sc[i] = scale_pair<KIND, BLOCK>(codes[i], top[i]);
          codes[i] >>= BLOCK == 16 ? 16 : 8;
        }
        if (h) {
          __syncwarp();  // every lane has read the stage: it is filled again meanwhile
          if (ahead) issue(slot);
          if (++slot == depth) {
            slot = 0;
            phase ^= 1;
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint4 v[NT];
#pragma unroll
          for (int c = 0; c < NT; ++c)
            v[c] = *reinterpret_cast<const uint4 *>(xl[c] + xo + q * 64);
#pragma unroll
          for (int u = 0; u < kPairs; ++u) {
            uint32_t a[4], b[4];
            const uint4 &wa = w[2 * u], &wb = w[2 * u + 1];
            decode8(q == 0 ? wa.x : q == 1 ? wa.y : q == 2 ? wa.z : wa.w, a);
            decode8(q == 0 ? wb.x : q == 1 ? wb.y : q == 2 ? wb.z : wb.w, b);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              a[e] = hmul2_by(a[e], sc[2 * u], BLOCK == 16 && q >= 2);
              b[e] = hmul2_by(b[e], sc[2 * u + 1], BLOCK == 16 && q >= 2);
            }
#pragma unroll
            for (int c = 0; c < NT; ++c) {
              mma(d[c][u], a[0], b[0], a[1], b[1], v[c].x, v[c].y);
              mma(d[c][u], a[2], b[2], a[3], b[3], v[c].z, v[c].w);
            }
          }
        }
        xo += 256;
      }
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        const float2 fx = *reinterpret_cast<const float2 *>(sxl + 8 * c);
#pragma unroll
        for (int u = 0; u < kPairs; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = e & 1 ? fx.y : fx.x;
            acc[c][u][e] = KIND == kMXFP4 ? fmaf(d[c][u][e] * x, f[2 * u + (e >> 1)], acc[c][u][e])
                                          : fmaf(d[c][u][e], x, acc[c][u][e]);
          }
      }
      sxl += kCols;
    }
    if (KIND == kMXFP4) {  // 255 is NaN
#pragma unroll
      for (int i = 0; i < kGroups; ++i)
        if (largest[i] == 255) {
#pragma unroll
          for (int c = 0; c < NT; ++c)
            acc[c][i >> 1][2 * (i & 1)] = acc[c][i >> 1][2 * (i & 1) + 1] = __uint_as_float(0x7FC00000u);
        }
    }
    // join the parts of the tiles of this round, in K order; a warp whose tile
    // is its own joins nothing and waits for nobody
    const bool alone = S == 1 && sk == 1;
    auto sync = [&] {
      if (S > 1)
        cg::this_cluster().sync();
      else if (alone)
        __syncwarp();
      else
        __syncthreads();
    };
    if (r > 0) sync();  // the parts of the round before have been read
    {
      float *o = parts + warp * (kRows * kCols);
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int u = 0; u < kPairs; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o[(8 * c + 2 * t + (e & 1)) * kRows + g + 16 * u + 8 * (e >> 1)] = acc[c][u][e];
    }
    // A warp writes the rows of a tile for one token (16 rows: two) at a time,
    // a row a lane; (tile, tokens) go around the warps of the cluster.  What a
    // row is multiplied by is requested before the wait.
    constexpr int kTokens = 32 / kRows;
    const int row = lane % kRows, turns = (M + kTokens - 1) / kTokens;
    const int size = j.y_type == FP4_F32 ? 4 : 2;
    int shift = 0;
    float sd = 0.0f;
    int64_t n = j.N;
    auto row_of = [&](int to) {
      const int tile = t0 + r * group + to;
      n = j.N;
      if (tile >= t1) return;
      n = ld.first_row(tile, tiled) + (tiled ? 32 * (row >> 3) + (row & 7) : row);
      if (n >= j.N) return;
      shift = (KIND == kUE5M3 ? 3 : 0) + (j.shift ? j.shift[n] : 0);
      sd = j.sd[j.stripes ? n >> 7 : 0];
    };
    const int outs = alone ? turns : group * turns, hops = alone ? 1 : kWarps * S;
    int i = alone ? 0 : warp * S + rank, tg = alone ? tw : i / turns;
    if (i < outs) row_of(tg);
    sync();
#pragma unroll 1
    while (i < outs) {
      const int m = (alone ? i : i - tg * turns) * kTokens + lane / kRows;
      if (n < j.N && m < M) {
        float v = 0.0f;
        for (int q = 0; q < S; ++q) {
          const float *from = S > 1 ? cg::this_cluster().map_shared_rank(parts, q) : parts;
          from += (tg * sk * kCols + m) * kRows + row;
          for (int w = 0; w < sk; ++w) v += from[w * kCols * kRows];
        }
        // the exponent in two steps: no overflow between
        v = v * pow2(shift >> 1) * pow2(shift - (shift >> 1)) * sd;
        uint8_t *to = static_cast<uint8_t *>(j.y) + ((m0 + m) * j.ys + n) * size;
        if (j.y_type == FP4_F32)
          *reinterpret_cast<float *>(to) = v;
        else if (j.y_type == FP4_BF16)
          *reinterpret_cast<__nv_bfloat16 *>(to) = __float2bfloat16_rn(v);
        else
          *reinterpret_cast<__half *>(to) = __float2half_rn(v);
      }
      i += hops;
      if (!alone && i < outs) {
        const int next = i / turns;
        if (next != tg) row_of(next);
        tg = next;
      }
    }
  }
  if (!live) {  // copies still in flight land (bounded) before the ring goes away
    for (; flying > 0; --flying) {
      tc::mbar_wait_drain(bars_a + 8 * slot, phase);
      if (++slot == depth) {
        slot = 0;
        phase ^= 1;
      }
    }
  }
  if (S > 1) cg::this_cluster().sync();  // nobody leaves while its parts may be read
}

// Shared memory for M tokens over ceil(steps / S) steps, NT column tiles.
size_t smem_bytes(int M, int steps, int S, int nt, int words, int warps, int depth) {
  const size_t span = (steps + S - 1) / S;
  return (size_t)warps * depth * (payload_of(nt) + words) + warps * kMaxDepth * 8 + span * 8 * nt * 4 +
         warps * rows_of(nt) * 8 * nt * 4 + M * (span * 512 + 64) + 16;
}

// Bytes [z][y][x] without gaps as a tensor map (2-D for z = 0), boxes of
// box_x x box_y; what lies past an end reads as zero.
bool byte_map(CUtensorMap *m, const void *base, int64_t x, int64_t y, int64_t z, int box_x, int box_y,
              bool swizzle) {
  auto fn = tc::encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)x, (cuuint64_t)y, (cuuint64_t)z};
  cuuint64_t strides[2] = {(cuuint64_t)x, (cuuint64_t)(x * y)};
  cuuint32_t box[3] = {(cuuint32_t)box_x, (cuuint32_t)box_y, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, z ? 3 : 2, const_cast<void *>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What a kernel may use, asked once per kernel and device: raises its shared
// memory limit, then counts the clusters of 1, 2, 4 and 8 CTAs of the
// largest kind that are resident at once (0: not asked yet, -1: failed).
struct Residence {
  std::atomic<int> clusters[4];
};
template <typename Kern>
int resident(Kern kern, Residence *per_device, int S, int kThreads) {
  constexpr int kMaxDev = 64;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return -1;
  const int i = S == 1 ? 0 : S == 2 ? 1 : S == 4 ? 2 : 3;
  Residence &r = per_device[dev];
  int n = r.clusters[i].load(std::memory_order_acquire);
  if (n) return n;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) != cudaSuccess)
    return -1;
  n = sm_count();
  if (S > 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(S);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kMaxSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)S;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) n = -1;
  }
  r.clusters[i].store(n, std::memory_order_release);
  return n;
}

template <int KIND, int BLOCK, int MODE, typename TX, int NT>
fp4_status launch(const MatvecJob &j, cudaStream_t s) {
  static Residence residence[64];
  auto kern = k_matvec<KIND, BLOCK, MODE, TX, NT>;
  MvParams p{};
  p.j = j;
  p.steps = (int)ceil_div(j.K, kStep);
  p.tiles = (int)(128 / rows_of(NT) * ceil_div(j.N, 128));
  p.mc = (int)(j.M < 8 * NT ? j.M : 8 * NT);
  const int64_t row_words = j.K / j.block;
  p.words = j.sf_mma ? kTiled : row_words % 16 == 0 ? kBoxed : kPieces;
  p.status = status_word();
  if (!p.status) return FP4_ERR_CUDA;
  const bool tiled = p.words == kTiled;
  p.tma = j.K % 32 == 0;
  if (p.tma && !byte_map(&p.map, j.q, j.K / 2, j.N, 0, kStep / 2, tiled ? 8 : rows_of(NT), true)) return FP4_ERR_CUDA;
  if (tiled && !byte_map(&p.smap, j.sf, 512, ceil_div(row_words, 4), ceil_div(j.N, 128), 128, kStep / BLOCK / 4, false))
    return FP4_ERR_CUDA;
  if (p.words == kBoxed && !byte_map(&p.smap, j.sf, row_words, j.N, 0, 16, rows_of(NT), false)) return FP4_ERR_CUDA;
  // The split: of those that fit shared memory (x of a CTA's tokens over its
  // part of K beside rings of two stages), the least estimated time, in units
  // of 30 ns: the steps of an SM, those of the longest warp one after the
  // other, the preparation of x, and each round's join (over warps; over a
  // cluster, by barriers that grow with it; rings run dry between rounds).  The weights are a fit to 50
  // sizes (1 .. 24 tokens, 141 .. 32768 rows, 256 .. 15040 columns) with every
  // split that fits: the choice takes 3% longer than the best on average, 12%
  // at worst.  Tokens are halved until something fits.
  int64_t best = INT64_MAX;
  auto fits = [&](int S, int warps, int depth) {
    return smem_bytes(p.mc, p.steps, S, NT, words_of(MODE), warps, depth) <= (size_t)kMaxSmem;
  };
  while (best == INT64_MAX) {
    for (int S = 1; S <= 8 && S <= p.steps; S *= 2) {
      int warps = kMaxWarps;
      while (warps >= 8 && !fits(S, warps, 2)) warps -= 2;
      if (warps < 8) continue;
      const int room = resident(kern, residence, S, 32 * kMaxWarps);
      if (room < 1) return FP4_ERR_CUDA;
      const int64_t span = ceil_div(p.steps, S);
      const int64_t clusters = p.tiles < room ? p.tiles : room, most = ceil_div(p.tiles, clusters);
      const int64_t waves = ceil_div(clusters * ceil_div(j.M, p.mc), room);
      for (int sk = 1; sk <= warps && sk <= span; ++sk) {
        const int group = warps / sk;
        if (sk > 1 && sk < warps && sk < span && warps / (sk + 1) == group) continue;  // a larger one keeps as many tiles
        const int64_t rounds = ceil_div(most, group);
        const int join = (sk > 1 ? 10 + sk : 0) + (S > 1 ? 8 + 20 * S : 0), dry = sk > 1 || S > 1 ? 40 : 0;
        const int64_t cost = waves * (rows_of(NT) / 4 * most * span + 4 * most + p.mc * span / 2 +
                                      rounds * (22 * ceil_div(span, sk) + join) + (rounds - 1) * dry);
        if (cost >= best) continue;
        best = cost;
        p.S = S;
        p.sk = sk;
        p.warps = warps;
        p.rounds = (int)rounds;
        p.clusters = (int)clusters;
        // small calls: half the warps start sooner (148 x 576, 1 token: 4.0 us
        // for 4.3), and with two rounds of tokens two CTAs fit an SM (5957 x 448,
        // 24 tokens: 7.7 us for 11.2); large ones want them all for x and the join
        if (most * sk <= 8 && p.mc * span <= 32) p.warps = 8;
      }
    }
    if (best < INT64_MAX) break;
    if (p.mc == 1) return FP4_ERR_SHAPE;
    p.mc = (p.mc + 1) / 2;
  }
  p.depth = 2;
  while (p.depth < kMaxDepth && fits(p.S, p.warps, p.depth + 1)) ++p.depth;
  const size_t smem = smem_bytes(p.mc, p.steps, p.S, NT, words_of(MODE), p.warps, p.depth);
  const int64_t most = (int64_t)p.mc * 65535;  // tokens a launch takes
  const size_t xe = 2, ye = j.y_type == FP4_F32 ? 4 : 2;
  for (int64_t m = 0; m < j.M; m += most) {
    p.j.M = j.M - m < most ? j.M - m : most;
    p.j.x = static_cast<const uint8_t *>(j.x) + m * j.xs * xe;
    p.j.y = static_cast<uint8_t *>(j.y) + m * j.ys * ye;
    const dim3 grid((unsigned)(p.clusters * p.S), (unsigned)ceil_div(p.j.M, p.mc));
    if (launch_dependent_clusters(kern, p.S, grid, dim3(32 * p.warps), smem, s, p) != cudaSuccess) return FP4_ERR_CUDA;
  }
  return FP4_OK;
}

template <int KIND, int BLOCK, int MODE, typename TX>
fp4_status launch_nt(const MatvecJob &j, cudaStream_t s) {
  return j.M <= 8 ? launch<KIND, BLOCK, MODE, TX, 1>(j, s) : launch<KIND, BLOCK, MODE, TX, 2>(j, s);
}

// Rows of K / 2 payload bytes and of K / BLOCK scales that are TMA strides,
// or the tensor-core layout, have kernels of their own.
template <int KIND, int BLOCK, typename TX>
fp4_status launch_mode(const MatvecJob &j, cudaStream_t s) {
  if (j.K % 32 == 0) {
    if (j.sf_mma) return launch_nt<KIND, BLOCK, kTiled, TX>(j, s);
    if (j.K % (16 * BLOCK) == 0) return launch_nt<KIND, BLOCK, kBoxed, TX>(j, s);
  }
  return launch_nt<KIND, BLOCK, kAny, TX>(j, s);
}

template <typename TX>
fp4_status launch_x(const MatvecJob &j, cudaStream_t s) {
  switch (j.kind) {
    case kMXFP4: return launch_mode<kMXFP4, 32, TX>(j, s);
    case kNVFP4: return launch_mode<kNVFP4, 16, TX>(j, s);
    default: return j.block == 16 ? launch_mode<kUE5M3, 16, TX>(j, s) : launch_mode<kUE5M3, 32, TX>(j, s);
  }
}

template <typename TY>
__global__ void k_zero(MatvecJob j) {
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < j.M * j.N;
       i += (int64_t)gridDim.x * blockDim.x)
    static_cast<TY *>(j.y)[i / j.N * j.ys + i % j.N] = from_f32<TY>(0.0f);
}

}  // namespace

fp4_status launch_matvec(const MatvecJob &j, cudaStream_t s) {
  if (j.K == 0) {
    const int64_t want = ceil_div(j.M * j.N, 256);
    const unsigned grid = (unsigned)(want < 1024 ? want : 1024);
    switch (j.y_type) {
      case FP4_BF16: k_zero<__nv_bfloat16><<<grid, 256, 0, s>>>(j); break;
      case FP4_F16: k_zero<__half><<<grid, 256, 0, s>>>(j); break;
      default: k_zero<float><<<grid, 256, 0, s>>>(j); break;
    }
    return cudaGetLastError() == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
  }
  return j.x_type == FP4_BF16 ? launch_x<__nv_bfloat16>(j, s) : launch_x<__half>(j, s);
}

}  // namespace fp4
