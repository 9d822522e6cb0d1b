// append.cu -- keys and values of new tokens into a paged cache, keys and
// queries rotated by their positions on the way (sm_103a):
//   (a, b) -> (a cos - b sin, b cos + a sin) per pair, binary32, rounded once.
//
// Bound: HBM for prompts (every row read and written once, 4 bytes per
// element; cos and sin are reused over the heads of a token), launch and three
// dependent loads (position, page, nothing else) for a few tokens.
//
// Layout.  A thread owns one unit of a head -- two pieces of 16 bytes, in the
// rotated part the two whose elements form pairs (i, i + rot_dim / 2) -- for
// one token, and walks over the token's query, key and value heads with cos
// and sin held in registers; neighbours touch neighbouring pieces of a row.
// Three rows are requested together and nothing of a token's place is waited
// for before its stores; the next token's place is looked up meanwhile.  Rows
// whose pointers, strides or sizes are not whole pieces of 16 bytes (half of
// an odd number of eights rotated, say) go by pieces of 8, the rest by single
// elements.
// Measured: 8191 tokens, 32 + 2 x 8 heads of 128, BF16: 34.4 us (5.9 TB/s, 87%
// of a copy's rate; 36.6 as an ordinary launch, then 41 with four CTAs an SM
// and 46 without looking ahead); one token 2.3 us in a graph.  8000 tokens, 48
// heads of 80 with 40 rotated: 42 us by pieces of 8 bytes, 98 by elements.
#include "serve.cuh"

namespace fp4 {

namespace {

constexpr int kThreads = 256, kResident = 3;  // CTAs per SM

struct ApParams {
  fp4_append_params p;
  int units;      // units of a head
  int lanes;      // head lanes: threads of a token / units
  int tokens;     // tokens of a CTA at a time
  int splits;     // CTAs that share a token's heads (few tokens)
  uint32_t *status;
};

// Where a token at position pos goes: false if it is skipped or lies outside
// a table.
__device__ __forceinline__ bool locate(const fp4_append_params &p, int64_t t, int pos, uint32_t *status,
                                       int &page, int &place) {
  const fp4_kv_cache &c = p.cache;
  page = 0;
  place = 0;
  if (pos < 0) return false;
  const int64_t seq = p.seq ? p.seq[t] : t;
  bool ok = seq >= 0 && seq < c.seqs && pos < c.seq_pages * c.page_size &&
            (p.rot_dim == 0 || pos < p.rope_len);
  if (ok) {
    const int e = pos / c.page_size;
    place = pos - e * c.page_size;
    page = c.table[seq * c.table_stride + e];
    ok = page >= 0 && page < c.pages;
  }
  if (!ok && status) raise_status(status, kStatusIndex);
  return ok;
}

// Row r of a token: its query heads, then its key heads, then its value heads.
template <typename T>
__device__ __forceinline__ const T *source(const fp4_append_params &p, int64_t t, int r, int heads) {
  if (r < heads) return static_cast<const T *>(p.q) + t * p.q_token + r * p.q_head;
  r -= heads;
  if (r < p.cache.kv_heads) return static_cast<const T *>(p.k) + t * p.k_token + r * p.k_head;
  return static_cast<const T *>(p.v) + t * p.v_token + (r - p.cache.kv_heads) * p.v_head;
}
template <typename T>
__device__ __forceinline__ T *target(const fp4_append_params &p, int64_t t, int r, int heads,
                                     int page, int place) {
  const fp4_kv_cache &c = p.cache;
  if (r < heads) return static_cast<T *>(p.q_out) + t * p.qo_token + r * p.qo_head;
  r -= heads;
  if (r < c.kv_heads) return static_cast<T *>(c.k) + (int64_t)page * c.k_page + place * c.k_place + r * c.k_head;
  return static_cast<T *>(c.v) + (int64_t)page * c.v_page + place * c.v_place + (r - c.kv_heads) * c.v_head;
}

template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
  static __device__ __forceinline__ float2 get(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }
  static __device__ __forceinline__ uint32_t put(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
};
template <>
struct Pair<__half> {
  static __device__ __forceinline__ float2 get(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
  }
  static __device__ __forceinline__ uint32_t put(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
};


// Pieces of eight elements turned: pairs of one element of each piece, or
// pairs of neighbours within a piece.
template <typename T, typename V>
__device__ __forceinline__ void turn_halves(V &x, V &y, const float *co, const float *si) {
  uint32_t *a = reinterpret_cast<uint32_t *>(&x), *b = reinterpret_cast<uint32_t *>(&y);
#pragma unroll
  for (int i = 0; i < (int)sizeof(V) / 4; ++i) {
    const float2 u = Pair<T>::get(a[i]), v = Pair<T>::get(b[i]);
    const float c0 = co[2 * i], c1 = co[2 * i + 1], s0 = si[2 * i], s1 = si[2 * i + 1];
    a[i] = Pair<T>::put(u.x * c0 - v.x * s0, u.y * c1 - v.y * s1);
    b[i] = Pair<T>::put(v.x * c0 + u.x * s0, v.y * c1 + u.y * s1);
  }
}
template <typename T, typename V>
__device__ __forceinline__ void turn_pairs(V &x, const float *co, const float *si) {
  uint32_t *a = reinterpret_cast<uint32_t *>(&x);
#pragma unroll
  for (int i = 0; i < (int)sizeof(V) / 4; ++i) {
    const float2 u = Pair<T>::get(a[i]);
    a[i] = Pair<T>::put(u.x * co[i] - u.y * si[i], u.y * co[i] + u.x * si[i]);
  }
}

// Whole pieces V of P elements (16 or 8 bytes), two a unit: with halves the
// pieces P u and rot_dim / 2 + P u of the rotated part, else 2 P consecutive
// elements (the last unit may hold one piece).  The rows are requested before anything is known of the
// token's place; only their stores wait for it, and a thread's next token is
// looked up meanwhile.
template <typename T, bool INTER, typename V>
__global__ void __launch_bounds__(kThreads, kResident) k_append_pieces(const __grid_constant__ ApParams a) {
  constexpr int P = sizeof(V) / 2;
  const fp4_append_params &p = a.p;
  const int heads = p.q ? p.heads : 0, rows = heads + 2 * p.cache.kv_heads, D = p.cache.head_dim;
  const int half = p.rot_dim / 2, turned = INTER ? 0 : p.rot_dim / (2 * P);
  const int per = a.units * a.lanes;  // threads of a token
  const int tl = threadIdx.x / per, in = threadIdx.x - tl * per;
  const int lane = in / a.units, unit = in - lane * a.units;
  if (tl >= a.tokens) return;
  const int split = blockIdx.x % a.splits;
  const int hop = (int)(gridDim.x / a.splits) * a.tokens, tokens = (int)p.tokens;
  const bool halves = unit < turned;
  const int o1 = halves ? P * unit : 2 * P * unit + (INTER ? 0 : p.rot_dim - 2 * P * turned);
  const int o2 = halves ? o1 + half : o1 + P;
  const bool two = o2 < D, rot1 = halves || (INTER && o1 < p.rot_dim), rot2 = halves || (INTER && o2 < p.rot_dim);
  constexpr int kBatch = 3;  // rows requested together
  const int stride = a.lanes * a.splits;
  uint32_t *const status = in == 0 && split == 0 ? a.status : nullptr;
  dependent_wait();
  launch_dependents();
  int t = (int)(blockIdx.x / a.splits) * a.tokens + tl;  // below 2^31, and so is t + hop
  int next_pos = t < tokens ? p.pos[t] : -1, next_place = 0, next_page = 0;
  bool next_keep = t < tokens && locate(p, t, next_pos, status, next_page, next_place);
  for (; t < tokens; t += hop) {
    const int pos = next_pos, place = next_place, page = next_page;
    const bool keep = next_keep, more = t + hop < tokens;
    next_pos = more ? p.pos[t + hop] : -1;
    __align__(16) float co[P], si[P];
    for (int r0 = split * a.lanes + lane, first = 1; r0 < rows; r0 += kBatch * stride, first = 0) {
      V x[kBatch], y[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        x[i] = y[i] = V{};
        const int r = r0 + i * stride;
        if (r >= rows) continue;
        const T *src = source<T>(p, t, r, heads);
        x[i] = *reinterpret_cast<const V *>(src + o1);
        if (two) y[i] = *reinterpret_cast<const V *>(src + o2);
      }
      if (first) {
        if (keep && (rot1 || rot2)) {
          const float *cs = p.rope + (int64_t)pos * p.rot_dim + P * unit;
#pragma unroll
          for (int i = 0; i < P; i += 4) {
            if (i == 4 && !rot2) continue;
            *reinterpret_cast<float4 *>(co + i) = *reinterpret_cast<const float4 *>(cs + i);
            *reinterpret_cast<float4 *>(si + i) = *reinterpret_cast<const float4 *>(cs + half + i);
          }
        }
        next_keep = more && locate(p, t + hop, next_pos, status, next_page, next_place);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int r = r0 + i * stride;
        if (r >= rows || (!keep && r >= heads)) continue;
        if (!keep) {
          x[i] = y[i] = V{};
        } else if (r < heads + p.cache.kv_heads) {
          if (halves) {
            turn_halves<T>(x[i], y[i], co, si);
          } else {
            if (rot1) turn_pairs<T>(x[i], co, si);
            if (rot2) turn_pairs<T>(y[i], co + P / 2, si + P / 2);
          }
        }
        T *dst = target<T>(p, t, r, heads, page, place);
        *reinterpret_cast<V *>(dst + o1) = x[i];
        if (two) *reinterpret_cast<V *>(dst + o2) = y[i];
      }
    }
  }
}

// Single elements: any pointers, strides and sizes.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_append1(const __grid_constant__ ApParams a) {
  const fp4_append_params &p = a.p;
  const int D = p.cache.head_dim, half = p.rot_dim / 2, units = D - half;  // pairs, then single elements
  const int heads = p.q ? p.heads : 0, rows = heads + 2 * p.cache.kv_heads;
  dependent_wait();
  launch_dependents();
  for (int64_t t = blockIdx.x; t < p.tokens; t += gridDim.x) {
    const int pos = p.pos[t];
    int place, page;
    const bool keep = locate(p, t, pos, threadIdx.x == 0 ? a.status : nullptr, page, place);
    const float *cs = p.rope + (int64_t)(keep ? pos : 0) * p.rot_dim;
    for (int i = threadIdx.x; i < (keep ? rows : heads) * units; i += kThreads) {
      const int r = i / units, u = i - r * units;
      const T *src = source<T>(p, t, r, heads);
      T *dst = target<T>(p, t, r, heads, page, place);
      if (u < half) {
        const int ia = p.interleaved ? 2 * u : u, ib = p.interleaved ? 2 * u + 1 : u + half;
        const T x = src[ia], y = src[ib];
        if (!keep) {
          dst[ia] = dst[ib] = from_f32<T>(0.0f);
        } else if (r >= heads + p.cache.kv_heads) {
          dst[ia] = x;
          dst[ib] = y;
        } else {
          const float fx = to_f32(x), fy = to_f32(y), co = cs[u], si = cs[half + u];
          dst[ia] = from_f32<T>(fx * co - fy * si);
          dst[ib] = from_f32<T>(fy * co + fx * si);
        }
      } else {
        dst[half + u] = keep ? src[half + u] : from_f32<T>(0.0f);
      }
    }
  }
}

// Whether rows at this address, so many elements apart, are whole pieces of P.
bool whole(int P, const void *ptr, int64_t s0, int64_t s1) {
  return reinterpret_cast<uintptr_t>(ptr) % (2 * P) == 0 && s0 % P == 0 && s1 % P == 0;
}
bool whole(int P, const fp4_append_params &p) {
  const fp4_kv_cache &c = p.cache;
  return c.head_dim % P == 0 && p.rot_dim % (p.interleaved ? 8 : 2 * P) == 0 && whole(P, p.k, p.k_token, p.k_head) &&
         whole(P, p.v, p.v_token, p.v_head) && whole(P, c.k, c.k_page, c.k_place) && whole(P, c.v, c.v_page, c.v_place) &&
         c.k_head % P == 0 && c.v_head % P == 0 && aligned16(p.rope) &&
         (!p.q || (whole(P, p.q, p.q_token, p.q_head) && whole(P, p.q_out, p.qo_token, p.qo_head)));
}

template <typename T, typename V>
fp4_status launch_pieces(ApParams &a, cudaStream_t s) {
  constexpr int P = sizeof(V) / 2;
  const fp4_append_params &p = a.p;
  const fp4_kv_cache &c = p.cache;
  const int rows = (p.q ? p.heads : 0) + 2 * c.kv_heads;
  const int64_t most = kResident * (int64_t)sm_count();  // CTAs resident at once
  const int turned = p.interleaved ? 0 : p.rot_dim / (2 * P);
  a.units = turned + (c.head_dim - 2 * P * turned + 2 * P - 1) / (2 * P);  // <= 32
  // a token's rows over the threads of a CTA, four or fewer each; what is left
  // of the CTA takes further tokens, and where there are few tokens a token's
  // rows go to several CTAs, one or two each
  const int enough = (rows + 3) / 4;
  a.lanes = 1;
  while (a.lanes < enough && 2 * a.lanes * a.units <= kThreads) a.lanes *= 2;
  a.tokens = kThreads / (a.units * a.lanes);
  a.splits = 1;
  const int64_t ctas = ceil_div(p.tokens, a.tokens);
  while (ctas * a.splits * 2 <= most / 2 && a.lanes * a.splits < rows) a.splits *= 2;
  const int64_t want = ctas < most / a.splits ? ctas : most / a.splits;
  const dim3 grid((unsigned)((want < 1 ? 1 : want) * a.splits));
  const auto kern = p.interleaved ? k_append_pieces<T, true, V> : k_append_pieces<T, false, V>;
  return launch_dependent(kern, grid, dim3(kThreads), 0, s, a) == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

template <typename T>
fp4_status launch_append(ApParams &a, cudaStream_t s) {
  const fp4_append_params &p = a.p;
  if (whole(8, p)) return launch_pieces<T, uint4>(a, s);
  if (whole(4, p)) return launch_pieces<T, uint2>(a, s);
  const unsigned grid = (unsigned)(p.tokens < 65535 ? p.tokens : 65535);
  return launch_dependent(k_append1<T>, dim3(grid), dim3(kThreads), 0, s, a) == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

}  // namespace

fp4_status launch_kv_append(const fp4_append_params &p, cudaStream_t s) {
  ApParams a{};
  a.p = p;
  a.status = status_word();
  if (!a.status) return FP4_ERR_CUDA;
  return p.cache.type == FP4_BF16 ? launch_append<__nv_bfloat16>(a, s) : launch_append<__half>(a, s);
}

}  // namespace fp4
