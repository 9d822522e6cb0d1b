// attention.cu -- attention of one new token per sequence over a paged cache
// (sm_103a):  out = sum_j w_j v_j,  w = softmax_j(scale q . k_j).
//
// First form: one CTA per sequence and query head; each warp walks every
// fourth position with a running maximum and sum in binary32, the four are
// joined in shared memory.
#include <cmath>

#include "serve.cuh"

namespace fp4 {

namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32, kPer = 8;  // 8 elements of a head per lane

template <typename T>
__global__ void __launch_bounds__(kThreads) k_attention(fp4_attention_params p, uint32_t *status) {
  const fp4_kv_cache &c = p.cache;
  const int D = c.head_dim, s = blockIdx.x, h = blockIdx.y;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int64_t hk = h / (p.heads / c.kv_heads);
  const int64_t room = (int64_t)c.seq_pages * c.page_size;
  int64_t len = p.lengths[s];
  if ((len < 0 || len > room) && threadIdx.x == 0) raise_status(status, kStatusIndex);
  len = len < 0 ? 0 : (len > room ? room : len);
  const int64_t from = p.window && len > p.window ? len - p.window : 0;
  float q[kPer], acc[kPer], top = -INFINITY, sum = 0.0f;
  const T *qp = static_cast<const T *>(p.q) + s * p.q_seq + h * p.q_head;
  for (int i = 0; i < kPer; ++i) {
    q[i] = lane + 32 * i < D ? to_f32(qp[lane + 32 * i]) * p.scale : 0.0f;
    acc[i] = 0.0f;
  }
  bool any = false;
  for (int64_t j = from + warp; j < len; j += kWarps) {
    const int64_t page = c.table[s * c.table_stride + j / c.page_size], place = j % c.page_size;
    if (page < 0 || page >= c.pages) {
      if (lane == 0) raise_status(status, kStatusIndex);
      continue;
    }
    any = true;
    const T *k = static_cast<const T *>(c.k) + page * c.k_page + place * c.k_place + hk * c.k_head;
    const T *v = static_cast<const T *>(c.v) + page * c.v_page + place * c.v_place + hk * c.v_head;
    float dot = 0.0f;
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i < D) dot = fmaf(q[i], to_f32(k[lane + 32 * i]), dot);
    for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(~0u, dot, o);
    const float now = fmaxf(top, dot), base = now == -INFINITY ? 0.0f : now;
    const float fade = expf(top - base), w = expf(dot - base);
    top = now;
    sum = sum * fade + w;
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i < D) acc[i] = fmaf(w, to_f32(v[lane + 32 * i]), acc[i] * fade);
  }
  __shared__ float tops[kWarps], sums[kWarps], accs[kWarps][32 * kPer];
  __shared__ int anys[kWarps];
  if (lane == 0) {
    tops[warp] = top;
    sums[warp] = sum;
    anys[warp] = any;
  }
  for (int i = 0; i < kPer; ++i) accs[warp][lane + 32 * i] = acc[i];
  __syncthreads();
  if (warp) return;
  float all = -INFINITY, total = 0.0f;
  int seen = 0;
  for (int w = 0; w < kWarps; ++w) {
    all = fmaxf(all, tops[w]);
    seen |= anys[w];
  }
  const float base = all == -INFINITY ? 0.0f : all;
  for (int w = 0; w < kWarps; ++w) total += sums[w] * expf(tops[w] - base);
  T *out = static_cast<T *>(p.out) + s * p.out_seq + h * p.out_head;
  for (int i = 0; i < kPer; ++i) {
    const int d = lane + 32 * i;
    if (d >= D) break;
    float v = 0.0f;
    for (int w = 0; w < kWarps; ++w) v += accs[w][d] * expf(tops[w] - base);
    out[d] = from_f32<T>(seen ? v / total : 0.0f);
  }
  if (p.lse && lane == 0) p.lse[(int64_t)s * p.heads + h] = seen ? base + logf(total) : -INFINITY;
}

}  // namespace

int64_t decode_attention_workspace(int heads, int kv_heads, int head_dim) { return 0; }

fp4_status launch_decode_attention(const fp4_attention_params &p, cudaStream_t s) {
  uint32_t *status = status_word();
  if (!status) return FP4_ERR_CUDA;
  const dim3 grid((unsigned)p.cache.seqs, (unsigned)p.heads);
  if (p.cache.type == FP4_BF16)
    k_attention<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p, status);
  else
    k_attention<__half><<<grid, kThreads, 0, s>>>(p, status);
  return cudaGetLastError() == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

}  // namespace fp4
