// append.cu -- keys and values of new tokens into a paged cache, keys and
// queries rotated by their positions on the way (sm_103a):
//   (a, b) -> (a cos - b sin, b cos + a sin) per pair, binary32, rounded once.
//
// First form: one CTA per token, one thread per pair or element at a time.
#include "serve.cuh"

namespace fp4 {

namespace {

constexpr int kThreads = 128;

template <typename T>
__global__ void __launch_bounds__(kThreads) k_append(fp4_append_params p, uint32_t *status) {
  const fp4_kv_cache &c = p.cache;
  const int D = c.head_dim, half = p.rot_dim / 2, units = D - half;  // pairs, then single elements
  for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    const int pos = p.pos[t];
    const int64_t seq = p.seq ? p.seq[t] : t;
    bool keep = pos >= 0, bad = false;
    int64_t page = 0;
    if (keep) {
      bad = seq < 0 || seq >= c.seqs || pos >= (int64_t)c.seq_pages * c.page_size ||
            (half && pos >= p.rope_len);
      if (!bad) {
        page = c.table[seq * c.table_stride + pos / c.page_size];
        bad = page < 0 || page >= c.pages;
      }
      if (bad && threadIdx.x == 0) raise_status(status, kStatusIndex);
      keep = !bad;
    }
    const int place = keep ? pos % c.page_size : 0;
    const float *cs = p.rope + (int64_t)(keep ? pos : 0) * p.rot_dim;
    const int heads = p.q ? p.heads : 0, rows = heads + 2 * c.kv_heads;
    for (int i = threadIdx.x; i < rows * units; i += kThreads) {
      const int r = i / units, u = i % units;
      const T *src;
      T *dst;
      if (r < heads) {
        src = static_cast<const T *>(p.q) + t * p.q_token + r * p.q_head;
        dst = static_cast<T *>(p.q_out) + t * p.qo_token + r * p.qo_head;
      } else if (r < heads + c.kv_heads) {
        const int64_t h = r - heads;
        src = static_cast<const T *>(p.k) + t * p.k_token + h * p.k_head;
        dst = static_cast<T *>(c.k) + page * c.k_page + place * c.k_place + h * c.k_head;
      } else {
        const int64_t h = r - heads - c.kv_heads;
        src = static_cast<const T *>(p.v) + t * p.v_token + h * p.v_head;
        dst = static_cast<T *>(c.v) + page * c.v_page + place * c.v_place + h * c.v_head;
      }
      if (!keep && r >= heads) continue;
      const bool value = r >= heads + c.kv_heads;
      if (u < half) {
        const int ia = p.interleaved ? 2 * u : u, ib = p.interleaved ? 2 * u + 1 : u + half;
        const T a = src[ia], b = src[ib];
        if (!keep) {
          dst[ia] = dst[ib] = from_f32<T>(0.0f);
        } else if (value) {
          dst[ia] = a;
          dst[ib] = b;
        } else {
          const float fa = to_f32(a), fb = to_f32(b), co = cs[u], si = cs[half + u];
          dst[ia] = from_f32<T>(fa * co - fb * si);
          dst[ib] = from_f32<T>(fb * co + fa * si);
        }
      } else {
        const int e = half + u;
        dst[e] = keep ? src[e] : from_f32<T>(0.0f);
      }
    }
  }
}

}  // namespace

fp4_status launch_kv_append(const fp4_append_params &p, cudaStream_t s) {
  uint32_t *status = status_word();
  if (!status) return FP4_ERR_CUDA;
  const unsigned grid = (unsigned)(p.tokens < 65535 ? p.tokens : 65535);
  if (p.cache.type == FP4_BF16)
    k_append<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p, status);
  else
    k_append<__half><<<grid, kThreads, 0, s>>>(p, status);
  return cudaGetLastError() == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

}  // namespace fp4
