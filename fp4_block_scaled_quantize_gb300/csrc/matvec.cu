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
// e2m1 * dec(sf) 2^c is exact in f16 for the constant c below (E4M3: 2^-8,
// UE5M3: 2^-3, smallest product 2^-18 and 2^-21, largest 10.5 and 46,080).
// E8M0 scales span more than f16: per row and 128 columns they are taken
// relative to the largest of the four (2^13 at most, exact 36 binades down)
// and the largest is applied in binary32.  A BF16 x is multiplied per token
// and 128 columns by the power of two that puts its largest magnitude in
// [2^15, 2^16): 8 significant bits stay exact in f16 for 32 binades below
// it.  Products are exact, the MMA adds 128 columns in binary32, and these
// sums are multiplied by the power(s) of two and added in binary32 with
// nearest rounding.
//
// Layout.  A warp takes 16 weight rows and 128 columns a step.  The order of
// k within an MMA is free as long as both operands share it: lane (g, t)
// loads 16 bytes (32 weights) of rows g and g + 8 from column 32 t on --
// a whole 16-byte load per row and no exchange between lanes -- and MMA j of
// eight takes its weights 4 j .. 4 j + 3.  x lies in shared memory as f16,
// each 128-column chunk with its 16-byte pieces in the order (i, t), so that
// four lanes read 64 contiguous bytes; the token pitch is 64 mod 128 bytes,
// so the two tokens of a quarter-warp use different banks.
//
// Split.  One CTA of 16 warps per SM keeps 64 KB of weight loads in flight
// (4 steps a warp, requested before x is prepared and across tiles).  The
// CTA holds x for its K range; SK of its warps share one row tile along K,
// and a cluster of S CTAs splits K where x for all of it does not fit.  The
// parts are added in shared memory (over the cluster: distributed) in a
// fixed order.
#include <cooperative_groups.h>

#include "serve.cuh"

namespace fp4 {

namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kStep = 128;      // columns a step
constexpr int kDepth = 4;       // steps in flight per warp
constexpr int kMaxSmem = 227 * 1024;
constexpr int kXBytes = 160 * 1024;  // above this K is split over more CTAs first

struct MvParams {
  MatvecJob j;
  int steps;         // ceil(K / 128)
  int tiles;         // ceil(N / 16)
  int sk, S;         // warps and CTAs that share a tile along K
  int rounds;        // row tiles a warp takes, one after the other
  int clusters;
  int mc;            // tokens a CTA takes (blockIdx.y counts them off)
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

__device__ __forceinline__ uint4 ldg16(const uint8_t *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ldg8(const uint8_t *p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// What a lane holds of one step: 32 weights of rows g and g + 8, and the
// codes of the scales over them (first block in the low byte).
struct Stage {
  uint4 wa, wb;
  uint32_t sa, sb;
};

// A row tile's addresses: the lane's payload and scales at step 0.
template <int KIND, bool K32>
struct Rows {
  const uint8_t *qa, *qb, *sa, *sb;
  int64_t sstep;  // bytes from one step's scales to the next's

  __device__ __forceinline__ void set(const MatvecJob &j, int64_t tile, int g, int t) {
    int64_t ra = tile * 16 + g, rb = ra + 8;
    if (ra >= j.N) ra = j.N - 1;  // rows past the end repeat the last; not stored
    if (rb >= j.N) rb = j.N - 1;
    qa = j.q + ra * (j.K / 2) + 16 * t;
    qb = j.q + rb * (j.K / 2) + 16 * t;
    const int64_t blocks = j.K / j.block;
    const int first = 32 * t / j.block;  // the lane's first block of a step
    if (j.sf_mma) {
      const int64_t c4 = (blocks + 3) >> 2;
      const int64_t at = (first >> 2) * 512 + (first & 3);
      sa = j.sf + (ra >> 7) * c4 * 512 + (ra & 31) * 16 + ((ra >> 5) & 3) * 4 + at;
      sb = j.sf + (rb >> 7) * c4 * 512 + (rb & 31) * 16 + ((rb >> 5) & 3) * 4 + at;
      sstep = kStep / j.block / 4 * 512;
    } else {
      sa = j.sf + ra * blocks + first;
      sb = j.sf + rb * blocks + first;
      sstep = kStep / j.block;
    }
  }

  // left: columns from the lane's first one to K (32 or more: all there)
  __device__ __forceinline__ void load(Stage &s, int step, int left, bool two) const {
    s.wa = s.wb = make_uint4(0, 0, 0, 0);
    s.sa = s.sb = 0;
    if (left <= 0) return;
    const int64_t o = (int64_t)step * (kStep / 2), p = step * sstep;
    if (K32) {
      s.wa = ldg16(qa + o);
      s.wb = ldg16(qb + o);
      if (two) {
        s.sa = __ldg(reinterpret_cast<const uint16_t *>(sa + p));
        s.sb = __ldg(reinterpret_cast<const uint16_t *>(sb + p));
      } else {
        s.sa = __ldg(sa + p);
        s.sb = __ldg(sb + p);
      }
    } else {  // K is an odd number of 16-element blocks: rows start on 8 bytes
      const uint2 a0 = ldg8(qa + o), b0 = ldg8(qb + o);
      uint2 a1 = make_uint2(0, 0), b1 = make_uint2(0, 0);
      s.sa = __ldg(sa + p);
      s.sb = __ldg(sb + p);
      if (left > 16) {
        a1 = ldg8(qa + o + 8);
        b1 = ldg8(qb + o + 8);
        s.sa |= (uint32_t)__ldg(sa + p + 1) << 8;
        s.sb |= (uint32_t)__ldg(sb + p + 1) << 8;
      }
      s.wa = make_uint4(a0.x, a0.y, a1.x, a1.y);
      s.wb = make_uint4(b0.x, b0.y, b1.x, b1.y);
    }
  }
};

// f16 pairs (v, v) of the scales of the lane's two 16-element halves.
template <int KIND>
__device__ __forceinline__ void scale_pairs(uint32_t codes, bool two, int top, uint32_t *h) {
  if (KIND == kMXFP4) {
    // 2^(code - top + 13): f16 exponent field 28 + code - top, subnormal below 1
    const int e = 28 + (int)(codes & 255u) - top;
    const uint32_t v = e >= 1 ? (uint32_t)e << 10 : (e >= -9 ? 1u << (e + 9) : 0u);
    h[0] = h[1] = v * 0x10001u;
    return;
  }
  uint32_t c0 = codes & 255u, c1 = two ? codes >> 8 : c0;
  if (KIND == kNVFP4) {
    // E4M3's fields at f16's: value 2^(7 - 15)
    h[0] = (c0 & 127u) * (128u * 0x10001u);
    h[1] = (c1 & 127u) * (128u * 0x10001u);
  } else {
    // E5M3 is the head of an f16; times 2^-3 to leave room for a product
    h[0] = hmul2(c0 * (128u * 0x10001u), 0x30003000u);
    h[1] = hmul2(c1 * (128u * 0x10001u), 0x30003000u);
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
// of two taken out of each (token, step).
template <typename TX>
__device__ void prepare_x(const MatvecJob &j, int64_t m0, int M, int s0, int n, uint8_t *xs, int pitch,
                          float *sx, int cols) {
  const TX *x = static_cast<const TX *>(j.x) + m0 * j.xs;
  const bool vec = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && (M == 1 || j.xs % 8 == 0);
  // 16 lanes a (token, step); eight elements each
  const int total = M * n * 16;
  for (int i = threadIdx.x; i < (total + 31) / 32 * 32; i += kThreads) {
    const bool on = i < total;
    const int unit = i >> 4, piece = i & 15;
    const int m = on ? unit / n : 0, c = on ? unit - m * n : 0;
    const int64_t k = (int64_t)(s0 + c) * kStep + piece * 8;
    uint32_t w[4] = {0, 0, 0, 0};
    if (on && k < j.K) {  // K is a multiple of 16: a piece is inside or outside
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
#pragma unroll
      for (int o = 8; o; o >>= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
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
    if (on) {
      // piece (t, i) = (piece / 4, piece % 4) lies at 16 (4 i + t)
      *reinterpret_cast<uint4 *>(xs + (int64_t)m * pitch + c * 256 + ((piece & 3) * 4 + (piece >> 2)) * 16) =
          make_uint4(w[0], w[1], w[2], w[3]);
      if (piece == 0) sx[c * cols + m] = pow2(ex);
    }
  }
}

template <int KIND, bool K32, typename TX, int NT>
__global__ void __launch_bounds__(kThreads, 1) k_matvec(const __grid_constant__ MvParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  constexpr int kCols = 8 * NT;
  const MatvecJob &j = p.j;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int S = p.S, sk = p.sk;
  const int rank = blockIdx.x % S, cluster = blockIdx.x / S;
  const int64_t m0 = (int64_t)blockIdx.y * p.mc;
  const int M = (int)min((int64_t)p.mc, j.M - m0);
  // the CTA's steps, and the warp's share of them
  const int c0 = (int)((int64_t)p.steps * rank / S), c1 = (int)((int64_t)p.steps * (rank + 1) / S);
  const int kw = warp % sk, tw = warp / sk, group = kWarps / sk;
  const int n = c1 - c0;
  const int s0 = c0 + n * kw / sk, s1 = c0 + n * (kw + 1) / sk;
  const int pitch = n * 256 + 64;
  const int span = (p.steps + S - 1) / S;  // same on every CTA of the cluster
  uint8_t *xs = smem;
  float *sx = reinterpret_cast<float *>(smem + M * (span * 256 + 64));
  float *parts = sx + span * kCols;  // [2][kWarps][16 * kCols]
  const bool two = j.block == 16;

  Rows<KIND, K32> rows;
  Stage st[kDepth];
  int64_t tile = (int64_t)cluster * group + tw;  // rounds step by clusters * group
  const int lane_col = 32 * t;
  const int K = (int)j.K;
  rows.set(j, tile < p.tiles ? tile : p.tiles - 1, g, t);
#pragma unroll
  for (int u = 0; u < kDepth; ++u)
    if (s0 + u < s1) rows.load(st[u], s0 + u, K - (s0 + u) * kStep - lane_col, two);

  prepare_x<TX>(j, m0, M, c0, n, xs, pitch, sx, kCols);
  __syncthreads();

  const uint8_t *xl[NT];
#pragma unroll
  for (int b = 0; b < NT; ++b) xl[b] = xs + min(8 * b + g, M - 1) * pitch + t * 16;  // columns past M repeat

  for (int r = 0; r < p.rounds; ++r) {
    const int64_t next = tile + (int64_t)p.clusters * group;
    float acc[NT][4];
#pragma unroll
    for (int b = 0; b < NT; ++b) acc[b][0] = acc[b][1] = acc[b][2] = acc[b][3] = 0.0f;
    for (int s = s0; s < s1; s += kDepth) {
      const bool last = s + kDepth >= s1;
      if (last) rows.set(j, next < p.tiles ? next : p.tiles - 1, g, t);
#pragma unroll
      for (int u = 0; u < kDepth; ++u) {
        if (s + u < s1) {
          float d[NT][2][4] = {};
          uint32_t ha[2], hb[2];
          float fa = 1.0f, fb = 1.0f;
          int topa = 0, topb = 0;
          if (KIND == kMXFP4) {
            topa = (int)st[u].sa, topb = (int)st[u].sb;
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
              topa = max(topa, __shfl_xor_sync(~0u, topa, o));
              topb = max(topb, __shfl_xor_sync(~0u, topb, o));
            }
            fa = pow2(topa - 140);  // 2^(top - 127) / 2^13
            fb = pow2(topb - 140);
          }
          scale_pairs<KIND>(st[u].sa, two, topa, ha);
          scale_pairs<KIND>(st[u].sb, two, topb, hb);
          const int xo = (s + u - c0) * 256;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t w0 = i == 0 ? st[u].wa.x : i == 1 ? st[u].wa.y : i == 2 ? st[u].wa.z : st[u].wa.w;
            const uint32_t w1 = i == 0 ? st[u].wb.x : i == 1 ? st[u].wb.y : i == 2 ? st[u].wb.z : st[u].wb.w;
            uint32_t a[4], b[4];
            decode8(w0, a);
            decode8(w1, b);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              a[q] = hmul2(a[q], ha[i >> 1]);
              b[q] = hmul2(b[q], hb[i >> 1]);
            }
#pragma unroll
            for (int c = 0; c < NT; ++c) {
              const uint4 v = *reinterpret_cast<const uint4 *>(xl[c] + xo + i * 64);
              mma(d[c][0], a[0], b[0], a[1], b[1], v.x, v.y);
              mma(d[c][1], a[2], b[2], a[3], b[3], v.z, v.w);
            }
          }
#pragma unroll
          for (int c = 0; c < NT; ++c) {
            const float2 f = *reinterpret_cast<const float2 *>(sx + (s + u - c0) * kCols + 8 * c + 2 * t);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float v = d[c][0][e] + d[c][1][e];
              const float fx = e & 1 ? f.y : f.x;
              if (KIND == kMXFP4) {
                acc[c][e] = fmaf(v * fx, e < 2 ? fa : fb, acc[c][e]);
              } else {
                acc[c][e] = fmaf(v, fx, acc[c][e]);
              }
            }
          }
        }
        // request the step this stage holds next: of this tile, or of the next
        const int ahead = last ? s0 + u : s + kDepth + u;
        if (ahead < s1 && (!last || r + 1 < p.rounds))
          rows.load(st[u], ahead, K - ahead * kStep - lane_col, two);
      }
    }
    // join the parts of the tiles of this round, in K order
    float *mine = parts + (r & 1) * (kWarps * 16 * kCols);
    {
      float *o = mine + warp * (16 * kCols);
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
      const int64_t nrow = ((int64_t)(r * p.clusters + cluster) * group + tg) * 16 + row;
      if (nrow >= j.N) continue;
      float v = 0.0f;
      for (int q = 0; q < S; ++q) {
        const float *from = S > 1 ? cg::this_cluster().map_shared_rank(mine, q) : mine;
        for (int w = 0; w < sk; ++w) v += from[(tg * sk + w) * (16 * kCols) + m * 16 + row];
      }
      const int shift = (KIND == kNVFP4 ? 8 : KIND == kMXFP4 ? 0 : 3) + (j.shift ? j.shift[nrow] : 0);
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
    tile = next;
  }
  if (S > 1) cg::this_cluster().sync();  // nobody leaves while its parts may be read
}

// Shared memory for M tokens over ceil(steps / S) steps, NT column tiles.
size_t smem_bytes(int M, int steps, int S, int nt) {
  const size_t span = (steps + S - 1) / S;
  return M * (span * 256 + 64) + span * 8 * nt * 4 + 2 * kWarps * 16 * 8 * nt * 4;
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

template <int KIND, bool K32, typename TX, int NT>
fp4_status launch(const MatvecJob &j, cudaStream_t s) {
  static Residence residence[64];
  auto kern = k_matvec<KIND, K32, TX, NT>;
  MvParams p{};
  p.j = j;
  p.steps = (int)ceil_div(j.K, kStep);
  p.tiles = (int)ceil_div(j.N, 16);
  p.mc = (int)(j.M < 8 * NT ? j.M : 8 * NT);
  // x of a CTA's tokens over its part of K: more CTAs per tile, then fewer
  // tokens, until it fits
  p.S = 1;
  while (p.S < 8 && smem_bytes(p.mc, p.steps, p.S, NT) > (size_t)kXBytes) p.S *= 2;
  while (p.mc > 1 && smem_bytes(p.mc, p.steps, p.S, NT) > (size_t)kMaxSmem) p.mc = (p.mc + 1) / 2;
  const size_t smem = smem_bytes(p.mc, p.steps, p.S, NT);
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

template <int KIND, bool K32, typename TX>
fp4_status launch_nt(const MatvecJob &j, cudaStream_t s) {
  return j.M <= 8 ? launch<KIND, K32, TX, 1>(j, s) : launch<KIND, K32, TX, 2>(j, s);
}

template <int KIND, typename TX>
fp4_status launch_k(const MatvecJob &j, cudaStream_t s) {
  if constexpr (KIND == kMXFP4) return launch_nt<KIND, true, TX>(j, s);  // K is a multiple of 32
  return j.K % 32 == 0 ? launch_nt<KIND, true, TX>(j, s) : launch_nt<KIND, false, TX>(j, s);
}

template <typename TX>
fp4_status launch_x(const MatvecJob &j, cudaStream_t s) {
  switch (j.kind) {
    case kMXFP4: return launch_k<kMXFP4, TX>(j, s);
    case kNVFP4: return launch_k<kNVFP4, TX>(j, s);
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
