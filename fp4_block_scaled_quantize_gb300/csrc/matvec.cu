// matvec.cu -- y = x W^T for a few tokens, W a 4-bit copy with block scales,
// x in 16 bits (sm_103a):
//   y[m][n] = s_dec 2^shift[n] sum_b dec(sf[n][b]) sum_{k in b} e2m1(q[n][k]) x[m][k]
//
// First form: one warp per weight row and token, lanes over the 16-element
// blocks of the row, binary32 products and sums.
#include "serve.cuh"

namespace fp4 {

namespace {

constexpr int kThreads = 256;

// Value of a scale code: the format's exponent and mantissa bits moved into
// a binary32 (subnormal codes land in its subnormals) and rebiased by one
// exact multiplication.
__device__ __forceinline__ float scale_value(int kind, uint32_t code) {
  if (kind == kMXFP4) return __uint_as_float(code ? code << 23 : 0x400000u);
  if (kind == kNVFP4) return __uint_as_float((code & 0x7Fu) << 20) * 0x1p120f;
  return __uint_as_float(code << 20) * 0x1p112f;
}

__device__ __forceinline__ int64_t scale_index(int64_t n, int64_t b, int64_t blocks, bool mma) {
  if (!mma) return n * blocks + b;
  return ((n >> 7) * ((blocks + 3) >> 2) + (b >> 2)) * 512 + (n & 31) * 16 + ((n >> 5) & 3) * 4 + (b & 3);
}

template <typename TX, typename TY>
__global__ void __launch_bounds__(kThreads) k_matvec(MatvecJob j) {
  const int64_t n = blockIdx.x * (int64_t)(kThreads / 32) + threadIdx.x / 32;
  const int64_t m = blockIdx.y;
  const int lane = threadIdx.x & 31;
  if (n >= j.N) return;
  const TX *x = static_cast<const TX *>(j.x) + m * j.xs;
  const int64_t blocks = j.K / j.block;
  float acc = 0.0f;
  for (int64_t b = lane; b < blocks; b += 32) {
    float part = 0.0f;
    for (int i = 0; i < j.block; ++i) {
      const int64_t k = b * j.block + i;
      const uint32_t code = (j.q[n * (j.K / 2) + k / 2] >> (4 * (k & 1))) & 15u;
      const float mag = (code & 7u) < 2 ? 0.5f * (code & 7u)
                                        : (1.0f + 0.5f * (code & 1u)) * (1 << (((code >> 1) & 3u) - 1));
      part = fmaf(code & 8u ? -mag : mag, to_f32(x[k]), part);
    }
    acc = fmaf(scale_value(j.kind, j.sf[scale_index(n, b, blocks, j.sf_mma)]), part, acc);
  }
  for (int o = 16; o; o >>= 1) acc += __shfl_xor_sync(~0u, acc, o);
  if (lane == 0) {
    const float sd = j.sd[j.stripes ? n >> 7 : 0];
    const float v = (j.shift ? scalbnf(acc, j.shift[n]) : acc) * sd;
    static_cast<TY *>(j.y)[m * j.ys + n] = from_f32<TY>(v);
  }
}

template <typename TX>
fp4_status launch_y(const MatvecJob &j, cudaStream_t s) {
  if (j.M > 65535) return FP4_ERR_SHAPE;
  const dim3 grid((unsigned)ceil_div(j.N, kThreads / 32), (unsigned)j.M);
  switch (j.y_type) {
    case FP4_BF16: k_matvec<TX, __nv_bfloat16><<<grid, kThreads, 0, s>>>(j); break;
    case FP4_F16: k_matvec<TX, __half><<<grid, kThreads, 0, s>>>(j); break;
    default: k_matvec<TX, float><<<grid, kThreads, 0, s>>>(j); break;
  }
  return cudaGetLastError() == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

}  // namespace

fp4_status launch_matvec(const MatvecJob &j, cudaStream_t s) {
  return j.x_type == FP4_BF16 ? launch_y<__nv_bfloat16>(j, s) : launch_y<__half>(j, s);
}

}  // namespace fp4
