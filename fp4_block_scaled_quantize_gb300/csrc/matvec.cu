// matvec.cu -- y = x W^T for a few tokens, W a 4-bit copy with block scales,
// x in 16 bits (sm_103a):
//   y[m][n] = s_dec 2^shift[n] sum_b dec(sf[n][b]) sum_{k in b} e2m1(q[n][k]) x[m][k]
//
// Bound: HBM, 0.5 + 1/B bytes per weight read once; at 6.8 TB/s an SM has
// about 7 issue slots for each 32 weights, so the arithmetic is the m16n8k16
// f16 MMA with the weight as its 16-row operand and up to 8 NT tokens as
// columns.  (tcgen05 reads its operands from shared or tensor memory: 4-bit
// weights would have to be decoded into it first, for a 128-row tile of which
// all but M columns of work are padding.)
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
// Layout.  A warp takes 16 weight rows and 256 columns a step.  The order of
// k within an MMA is free as long as both operands share it: lane (g, t)
// takes columns 64 t .. 64 t + 63 of rows g and g + 8, four 16-byte pieces of
// payload and the four scale codes over 64 columns of each row -- whole loads
// and no exchange between lanes -- and each MMA four of its weights.  A step's payload is one
// TMA box of 16 rows x 128 bytes in the 128-byte swizzle (rows g, g + 1 of a
// quarter-warp then read different banks); x lies in shared memory as f16,
// the 16-byte pieces of 256 columns in the order (piece of the lane, t), so
// that four lanes read 64 contiguous bytes, tokens 64 mod 128 bytes apart.
//
// Split.  One CTA of 16 warps per SM; each warp runs its own ring of 2 to 4
// stages (payload by TMA, scale words by 4-byte cp.async, one mbarrier), so
// that 64 KB or more of weights are in flight per SM across tiles and before
// x is ready, and no warp waits for another inside a tile.  The CTA holds x
// for its K range; sk of its warps share a row tile along K, and a cluster
// of S CTAs splits K where x for all of it does not fit.  The parts are
// added in shared memory (over the cluster: distributed) in a fixed order.
// A row pitch that is not a multiple of 16 bytes (K / 16 odd) is no TMA
// stride: the ring is then filled by 8-byte cp.async.
#include <cooperative_groups.h>

#include "serve.cuh"
#include "tcgen05.cuh"

namespace fp4 {

namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kStep = 256;             // columns a step
constexpr int kPayload = 16 * kStep / 2;  // bytes of a stage: payload, then scale words
constexpr int kWords = 32 * 8;
constexpr int kMaxDepth = 4;
constexpr int kMaxSmem = 227 * 1024;

struct MvParams {
  CUtensorMap map;   // payload [N][K / 2], boxes of 16 rows x 128 bytes
  MatvecJob j;
  int steps;         // ceil(K / 256)
  int tiles;         // ceil(N / 16)
  int sk, S;         // warps and CTAs that share a tile along K
  int rounds;        // row tiles a warp takes, one after the other
  int clusters;
  int mc;            // tokens a CTA takes (blockIdx.y counts them off)
  int depth;         // stages of a warp's ring
  int words;         // scale words can be copied whole (4-byte aligned rows)
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

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(on ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(on ? 8 : 0)
               : "memory");
}
// The lane's arrival, when its cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Fills a warp's stages one after the other: the payload of 16 rows x 256
// columns and, per lane, the scale words over its 64 columns of rows g and
// g + 8 ({a, b} at 8 * lane; a word holds the codes of 64 columns, or with
// 32-element blocks of 128 columns).  Addresses advance by constants inside
// a tile and are formed anew at the next.
template <int BLOCK, bool TMA>
struct Loader {
  const uint8_t *sa, *sb;  // the lane's next scale words
  int sstep;               // bytes from a step's words to the next's
  int words_left;          // steps whose word (of a row) lies inside K
  bool row_a, row_b;
  int step, row0;          // of the next stage

  __device__ __forceinline__ void set(const MvParams &p, int64_t tile, int s, int lane) {
    const MatvecJob &j = p.j;
    const int g = lane >> 2, t = lane & 3;
    step = s;
    row0 = (int)tile * 16;
    const int64_t blocks = j.K / BLOCK;
    const int per = kStep / BLOCK, first = BLOCK == 16 ? 4 * t : 2 * (t & 2);
    const int64_t at = (int64_t)s * per + first;  // the next word's first block
    const int64_t left = blocks - at;
    words_left = left > 0 ? (int)((left + per - 1) / per) : 0;
    const int64_t ra = tile * 16 + g, rb = ra + 8;
    row_a = ra < j.N;
    row_b = rb < j.N;
    if (j.sf_mma) {
      const int64_t c4 = (blocks + 3) >> 2;
      const int64_t o = (at >> 2) * 512;
      sa = j.sf + (ra >> 7) * c4 * 512 + (ra & 31) * 16 + ((ra >> 5) & 3) * 4 + o;
      sb = j.sf + (rb >> 7) * c4 * 512 + (rb & 31) * 16 + ((rb >> 5) & 3) * 4 + o;
      sstep = per / 4 * 512;
    } else {
      sa = j.sf + ra * blocks + at;
      sb = j.sf + rb * blocks + at;
      sstep = per;
    }
    if (!row_a) sa = j.sf;
    if (!row_b) sb = j.sf;
  }

  __device__ __forceinline__ void fill(const MvParams &p, uint32_t payload, uint32_t words,
                                       uint32_t bar, int lane) {
    const MatvecJob &j = p.j;
    if (TMA) {
      if (lane == 0) {
        tc::mbar_expect_tx(bar, kPayload);  // the full box, whatever part of it lies outside
        tc::tma_load_2d(payload, &p.map, bar, step * (kStep / 2), row0);
      }
    } else {
      // 16 rows x 16 pieces of 8 bytes; lane: piece lane % 16 of every other row
      const int64_t at = (int64_t)step * (kStep / 2) + (lane & 15) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 2 * i + (lane >> 4);
        const int64_t n = (int64_t)row0 + r;
        const bool on = n < j.N && at < j.K / 2;
        const int c16 = (lane & 15) >> 1;  // in the swizzled place the TMA would use
        cp_async8(payload + r * 128 + ((c16 ^ (r & 7)) << 4) + (lane & 1) * 8,
                  j.q + (on ? n * (j.K / 2) + at : 0), on);
      }
    }
    const uint32_t dst = words + lane * 8;
    if (p.words) {
      cp_async4(dst, words_left > 0 ? sa : j.sf, row_a && words_left > 0);
      cp_async4(dst + 4, words_left > 0 ? sb : j.sf, row_b && words_left > 0);
    } else {  // rows of scales that start on no word (plain layout): by bytes
      const int first = step * (kStep / BLOCK) + (BLOCK == 16 ? 4 * (lane & 3) : 2 * (lane & 2));
      const int blocks = (int)(j.K / BLOCK);
      uint32_t wa = 0, wb = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (first + b < blocks) {
          if (row_a) wa |= (uint32_t)__ldg(sa + b) << (8 * b);
          if (row_b) wb |= (uint32_t)__ldg(sb + b) << (8 * b);
        }
      }
      asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(dst), "r"(wa), "r"(wb) : "memory");
    }
    cp_async_arrive(bar);
    ++step;
    --words_left;
    sa += sstep;
    sb += sstep;
  }
};

// The f16 scales over the lane's 64 columns of one row: blocks of 16, pairs
// {0, 1} and {2, 3} (block h in half h % 2 of h[h / 2]); blocks of 32, one pair.
template <int KIND, int BLOCK>
__device__ __forceinline__ void scale_pairs(uint32_t w, int top, uint32_t *h) {
  if (KIND == kMXFP4) {
    // 2^(code - top + 13): f16 exponent field 28 + code - top, subnormal below 1
    const int e0 = 28 + (int)(w & 255u) - top, e1 = 28 + (int)((w >> 8) & 255u) - top;
    const uint32_t v0 = e0 >= 1 ? (uint32_t)e0 << 10 : (e0 >= -9 ? 1u << (e0 + 9) : 0u);
    const uint32_t v1 = e1 >= 1 ? (uint32_t)e1 << 10 : (e1 >= -9 ? 1u << (e1 + 9) : 0u);
    h[0] = v0 | (v1 << 16);
    return;
  }
#pragma unroll
  for (int i = 0; i < 32 / BLOCK; ++i) {
    if (KIND == kNVFP4) {
      asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
          : "=r"(h[i])
          : "r"(i ? w >> 16 : w));
    } else {
      // E5M3 is the head of an f16; times 2^-3 to leave room for a product
      h[i] = hmul2(__byte_perm(w, 0, i ? 0x3424 : 0x1404) >> 1, 0x30003000u);
    }
  }
}

template <typename TX>
struct Is {
  static constexpr bool bf16 = false;
};
template <>
struct Is<__nv_bfloat16> {
  static constexpr bool bf16 = true;
};

// x[0 .. M) over steps [s0, s0 + n) as f16 into shared memory, and the power
// of two taken out of each (token, step); a warp per (token, step), eight
// elements a lane.
template <typename TX>
__device__ void prepare_x(const MatvecJob &j, int64_t m0, int M, int s0, int n, uint8_t *xs, int pitch,
                          float *sx, int cols) {
  const TX *x = static_cast<const TX *>(j.x) + m0 * j.xs;
  const bool vec = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && (M == 1 || j.xs % 8 == 0);
  const int piece = threadIdx.x & 31;
  for (int u = threadIdx.x >> 5; u < M * n; u += kWarps) {
    const int m = u / n, c = u - m * n;
    const int64_t k = (int64_t)(s0 + c) * kStep + piece * 8;
    uint32_t w[4] = {0, 0, 0, 0};
    if (k < j.K) {  // K is a multiple of 16: a piece is inside or outside
      const TX *p = x + m * j.xs + k;
      if (vec) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p));
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
      } else {
        const uint16_t *e = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = e[2 * q] | ((uint32_t)e[2 * q + 1] << 16);
      }
    }
    int ex = 0;
    if (Is<TX>::bf16) {
      uint32_t top = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) top = max(top, max(w[q] & 0x7FFFu, (w[q] >> 16) & 0x7FFFu));
      top = __reduce_max_sync(~0u, top);
      // exponent of the largest finite magnitude (2^133 x subnormals: 1 + mantissa bits)
      const int f = (int)(top >> 7);
      const int e = f >= 255 ? 127 : f > 0 ? f - 127 : top ? (31 - __clz((int)top)) - 133 : 0;
      ex = e - 15;
      const int h1 = -ex / 2;  // 2^-ex in two factors that binary32 holds
      const float f1 = pow2(h1), f2 = pow2(-ex - h1);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const __half2 v = __floats2half2_rn(bf16_lo(w[q]) * f1 * f2, bf16_hi(w[q]) * f1 * f2);
        w[q] = *reinterpret_cast<const uint32_t *>(&v);
      }
    }
    // piece i of lane t (piece = 8 t + i) lies at 64 i + 16 t
    *reinterpret_cast<uint4 *>(xs + m * pitch + c * 512 + (piece & 7) * 64 + (piece >> 3) * 16) =
        make_uint4(w[0], w[1], w[2], w[3]);
    if (piece == 0) sx[c * cols + m] = pow2(ex);
  }
}

template <int KIND, int BLOCK, bool TMA, typename TX, int NT>
__global__ void __launch_bounds__(kThreads, 1) k_matvec(const __grid_constant__ MvParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int kCols = 8 * NT;
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
  float *parts = sx + span * kCols;  // [2][kWarps][16 * kCols]
  uint8_t *xs = reinterpret_cast<uint8_t *>(parts + 2 * kWarps * 16 * kCols);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(xs + p.mc * (span * 512 + 64));
  const uint32_t ring_a = tc::smem_u32(ring), words_a = tc::smem_u32(word_ring), bars_a = tc::smem_u32(bars);

  // the warp's own ring: 32 lanes arrive for their copies, with TMA one more
  // arrival that also expects the box
  if (threadIdx.x == 0) *abort_flag = 0;
  if (lane == 0) {
    for (int d = 0; d < depth; ++d) tc::mbar_init(bars_a + 8 * d, TMA ? 33 : 32);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  __syncwarp();
  const int64_t tile0 = (int64_t)cluster * group + tw, hop = (int64_t)p.clusters * group;
  const int mine = tw < group && tile0 < p.tiles ? (int)((p.tiles - 1 - tile0) / hop) + 1 : 0;  // the warp's tiles
  int64_t ahead = (int64_t)mine * ns, flying = 0;  // stages to request, requested and not read
  int64_t ld_tile = tile0;
  int ld_left = ns, ld_slot = 0;
  Loader<BLOCK, TMA> ld;
  ld.set(p, tile0, s0, lane);
  auto issue = [&] {
    ld.fill(p, ring_a + ld_slot * kPayload, words_a + ld_slot * kWords, bars_a + 8 * ld_slot, lane);
    --ahead;
    ++flying;
    if (++ld_slot == depth) ld_slot = 0;
    if (--ld_left == 0) {
      ld_left = ns;
      ld_tile += hop;
      ld.set(p, ld_tile, s0, lane);
    }
  };
  for (int d = 0; d < depth && ahead; ++d) issue();

  prepare_x<TX>(j, m0, M, c0, n, xs, pitch, sx, kCols);
  __syncthreads();

  const uint8_t *xl[NT];
#pragma unroll
  for (int b = 0; b < NT; ++b) xl[b] = xs + min(8 * b + g, M - 1) * pitch + t * 16;  // columns past M repeat

  const int at0 = ((2 * t) ^ g) << 4;  // the lane's pieces of a row: at0, at0 ^ 16, then 1024 on
  int slot = 0;
  uint32_t phase = 0;
  bool live = true;  // false once a wait ran out: no more loads, results void
  for (int r = 0; r < p.rounds; ++r) {
    float acc[NT][4];
#pragma unroll
    for (int b = 0; b < NT; ++b) acc[b][0] = acc[b][1] = acc[b][2] = acc[b][3] = 0.0f;
    int xo = (s0 - c0) * 512;
    const float *sxl = sx + (s0 - c0) * kCols + 2 * t;
    for (int s = r < mine && live ? ns : 0; s > 0; --s) {
      if (!__all_sync(~0u, tc::mbar_wait_inl(bars_a + 8 * slot, phase, abort_flag, p.status))) {
        live = false;
        break;
      }
      uint2 codes = *reinterpret_cast<const uint2 *>(word_ring + slot * kWords + lane * 8);
      const uint8_t *ra = ring + slot * kPayload + g * 128;
      float d[NT][2][4] = {};
      float fa = 1.0f, fb = 1.0f;
      int topa = 0, topb = 0;
      if (BLOCK == 32 && (t & 1)) codes.x >>= 16, codes.y >>= 16;  // the lane's half of the word
      if (KIND == kMXFP4) {
        topa = max((int)(codes.x & 255u), (int)((codes.x >> 8) & 255u));
        topb = max((int)(codes.y & 255u), (int)((codes.y >> 8) & 255u));
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          topa = max(topa, __shfl_xor_sync(~0u, topa, o));
          topb = max(topb, __shfl_xor_sync(~0u, topb, o));
        }
        fa = pow2(topa - 140);  // 2^(top - 127) / 2^13
        fb = pow2(topb - 140);
      }
      uint32_t ha[2], hb[2];
      scale_pairs<KIND, BLOCK>(codes.x, topa, ha);
      scale_pairs<KIND, BLOCK>(codes.y, topb, hb);
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // 32 of the lane's 64 columns: a 16-byte piece of each row
        const uint4 wa = *reinterpret_cast<const uint4 *>(ra + (at0 ^ (16 * h)));
        const uint4 wb = *reinterpret_cast<const uint4 *>(ra + 1024 + (at0 ^ (16 * h)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t a[4], b[4];
          decode8(i == 0 ? wa.x : i == 1 ? wa.y : i == 2 ? wa.z : wa.w, a);
          decode8(i == 0 ? wb.x : i == 1 ? wb.y : i == 2 ? wb.z : wb.w, b);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            a[q] = BLOCK == 16 ? hmul2_by(a[q], ha[h], i >= 2) : hmul2_by(a[q], ha[0], h);
            b[q] = BLOCK == 16 ? hmul2_by(b[q], hb[h], i >= 2) : hmul2_by(b[q], hb[0], h);
          }
#pragma unroll
          for (int c = 0; c < NT; ++c) {
            const uint4 v = *reinterpret_cast<const uint4 *>(xl[c] + xo + (4 * h + i) * 64);
            mma(d[c][0], a[0], b[0], a[1], b[1], v.x, v.y);
            mma(d[c][1], a[2], b[2], a[3], b[3], v.z, v.w);
          }
        }
      }
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        const float2 f = *reinterpret_cast<const float2 *>(sxl + 8 * c);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = d[c][0][e] + d[c][1][e];
          const float fx = e & 1 ? f.y : f.x;
          acc[c][e] = KIND == kMXFP4 ? fmaf(v * fx, e < 2 ? fa : fb, acc[c][e]) : fmaf(v, fx, acc[c][e]);
        }
      }
      xo += 512;
      sxl += kCols;
      --flying;
      if (++slot == depth) {
        slot = 0;
        phase ^= 1;
      }
      __syncwarp();  // every lane has read the stage: it can be filled again
      if (ahead) issue();
    }
    // join the parts of the tiles of this round, in K order
    float *share = parts + (r & 1) * (kWarps * 16 * kCols);
    {
      float *o = share + warp * (16 * kCols);
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[(8 * c + 2 * t + (e & 1)) * 16 + g + 8 * (e >> 1)] = acc[c][e];
    }
    if (S > 1) {
      cg::this_cluster().sync();
    } else if (sk > 1) {
      __syncthreads();
    } else {
      __syncwarp();
    }
    // outputs of the round: group tiles x M tokens x 16 rows, shared by the cluster's CTAs;
    // a warp whose tile is its own joins nothing and waits for nobody
    const bool alone = S == 1 && sk == 1;
    const int outs = (alone ? 1 : group) * M * 16;
    for (int i = alone ? lane : (int)threadIdx.x * S + rank; i < outs; i += alone ? 32 : kThreads * S) {
      const int row = i & 15, mt = i >> 4, m = mt % M, tg = alone ? tw : mt / M;
      const int64_t nrow = ((int64_t)(r * (int64_t)p.clusters + cluster) * group + tg) * 16 + row;
      if (nrow >= j.N) continue;
      float v = 0.0f;
      for (int q = 0; q < S; ++q) {
        const float *from = S > 1 ? cg::this_cluster().map_shared_rank(share, q) : share;
        for (int w = 0; w < sk; ++w) v += from[(tg * sk + w) * (16 * kCols) + m * 16 + row];
      }
      const int shift = (KIND == kUE5M3 ? 3 : 0) + (j.shift ? j.shift[nrow] : 0);
      v = scalbnf(v, shift) * j.sd[j.stripes ? nrow >> 7 : 0];
      const int64_t at = (m0 + m) * j.ys + nrow;
      if (j.y_type == FP4_F32)
        static_cast<float *>(j.y)[at] = v;
      else if (j.y_type == FP4_BF16)
        static_cast<__nv_bfloat16 *>(j.y)[at] = __float2bfloat16_rn(v);
      else
        static_cast<__half *>(j.y)[at] = __float2half_rn(v);
    }
    if (alone) __syncwarp();
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
size_t smem_bytes(int M, int steps, int S, int nt, int depth) {
  const size_t span = (steps + S - 1) / S;
  return (size_t)kWarps * depth * (kPayload + kWords) + kWarps * kMaxDepth * 8 + span * 8 * nt * 4 +
         2 * kWarps * 16 * 8 * nt * 4 + M * (span * 512 + 64) + 16;
}

// Payload rows as a tensor map: boxes of 16 rows x 128 bytes, swizzled; what
// lies past the last row or column reads as zero.
bool payload_map(CUtensorMap *m, const void *base, int64_t rows, int64_t row_bytes) {
  return tc::make_map(m, base, rows, row_bytes, 16, kStep / 2);
}

// What a kernel may use, asked once per kernel and device: raises its shared
// memory limit, then counts the clusters of 1, 2, 4 and 8 CTAs of the
// largest kind that are resident at once (0: not asked yet, -1: failed).
struct Residence {
  std::atomic<int> clusters[4];
};
template <typename Kern>
int resident(Kern kern, Residence *per_device, int S) {
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

template <int KIND, int BLOCK, bool TMA, typename TX, int NT>
fp4_status launch(const MatvecJob &j, cudaStream_t s) {
  static Residence residence[64];
  auto kern = k_matvec<KIND, BLOCK, TMA, TX, NT>;
  MvParams p{};
  p.j = j;
  p.steps = (int)ceil_div(j.K, kStep);
  p.tiles = (int)ceil_div(j.N, 16);
  p.mc = (int)(j.M < 8 * NT ? j.M : 8 * NT);
  p.words = j.sf_mma || (j.K / j.block) % 4 == 0;
  p.status = status_word();
  if (!p.status) return FP4_ERR_CUDA;
  if (TMA && !payload_map(&p.map, j.q, j.N, j.K / 2)) return FP4_ERR_CUDA;
  // x of a CTA's tokens over its part of K beside rings of 3 stages or more:
  // more CTAs per tile until it fits; then fewer stages, then fewer tokens
  p.S = 1;
  p.depth = 3;
  while (p.S < 8 && smem_bytes(p.mc, p.steps, p.S, NT, p.depth) > (size_t)kMaxSmem) p.S *= 2;
  if (smem_bytes(p.mc, p.steps, p.S, NT, 3) > (size_t)kMaxSmem) p.depth = 2;
  while (p.mc > 1 && smem_bytes(p.mc, p.steps, p.S, NT, p.depth) > (size_t)kMaxSmem) p.mc = (p.mc + 1) / 2;
  if (smem_bytes(p.mc, p.steps, p.S, NT, kMaxDepth) <= (size_t)kMaxSmem) p.depth = kMaxDepth;
  const size_t smem = smem_bytes(p.mc, p.steps, p.S, NT, p.depth);
  if (smem > (size_t)kMaxSmem) return FP4_ERR_SHAPE;
  const int room = resident(kern, residence, p.S);
  if (room < 1) return FP4_ERR_CUDA;
  // warps per tile: the fewest steps on the busiest warp; a round costs about
  // one step more for its join, so ties go to fewer and longer ones
  int64_t cost = INT64_MAX;
  for (int sk = 1; sk <= kWarps && (sk == 1 || p.S * sk <= p.steps); sk *= 2) {
    const int group = kWarps / sk;
    const int64_t rounds = ceil_div(p.tiles, (int64_t)room * group);
    const int64_t c = rounds * (ceil_div(p.steps, (int64_t)p.S * sk) + 1);
    if (c >= cost) continue;
    cost = c;
    p.sk = sk;
    p.rounds = (int)rounds;
    p.clusters = (int)ceil_div(p.tiles, rounds * group);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.S;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.S > 1 ? 1 : 0;
  const int64_t most = (int64_t)p.mc * 65535;  // tokens a launch takes
  const size_t xe = 2, ye = j.y_type == FP4_F32 ? 4 : 2;
  for (int64_t m = 0; m < j.M; m += most) {
    p.j.M = j.M - m < most ? j.M - m : most;
    p.j.x = static_cast<const uint8_t *>(j.x) + m * j.xs * xe;
    p.j.y = static_cast<uint8_t *>(j.y) + m * j.ys * ye;
    cfg.gridDim = dim3((unsigned)(p.clusters * p.S), (unsigned)ceil_div(p.j.M, p.mc));
    if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return FP4_ERR_CUDA;
  }
  return FP4_OK;
}

template <int KIND, int BLOCK, bool TMA, typename TX>
fp4_status launch_nt(const MatvecJob &j, cudaStream_t s) {
  return j.M <= 8 ? launch<KIND, BLOCK, TMA, TX, 1>(j, s) : launch<KIND, BLOCK, TMA, TX, 2>(j, s);
}

// Rows of K / 2 bytes are a TMA stride when K is a multiple of 32, as it is
// with 32-element blocks.
template <int KIND, typename TX>
fp4_status launch_k(const MatvecJob &j, cudaStream_t s) {
  if (j.K % 32 != 0) return launch_nt<KIND, 16, false, TX>(j, s);
  return j.block == 16 ? launch_nt<KIND, 16, true, TX>(j, s) : launch_nt<KIND, 32, true, TX>(j, s);
}

template <typename TX>
fp4_status launch_x(const MatvecJob &j, cudaStream_t s) {
  switch (j.kind) {
    case kMXFP4: return launch_nt<kMXFP4, 32, true, TX>(j, s);
    case kNVFP4: return j.K % 32 != 0 ? launch_nt<kNVFP4, 16, false, TX>(j, s) : launch_nt<kNVFP4, 16, true, TX>(j, s);
    default: return launch_k<kUE5M3, TX>(j, s);
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
