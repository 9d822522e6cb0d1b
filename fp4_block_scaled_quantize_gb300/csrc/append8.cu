// append8.cu -- keys and values of new tokens into a paged cache of E4M3 codes
// with a power-of-two scale for each block of places and head, keys and queries
// rotated by their positions on the way; and stored tokens back in 16 bits
// (sm_103a).
//   scale' = need, or max(scale, need) where the block holds earlier tokens
//   need   = smallest 2^e with max |x| <= 448 2^e,  code = E4M3(x / scale')
// A scale that rises takes the block's other codes along: code' = E4M3(code
// scale / scale'), exact but for what falls among E4M3's subnormals.
//
// Bound: HBM for prompts (2 bytes read and 1 written per element of keys and
// values, 2 and 2 of queries), launch and dependent loads (position, page,
// scale) for a few tokens.
//
// Layout.  A warp takes the tokens of one block and one key or value head: lanes
// hold units of 16 elements (two pieces of 8, in the rotated part those whose
// elements form pairs) of 32 / units rows at a time.  It goes over its rows
// twice, for the largest magnitude and for the codes; the second time they come
// from L1.  Warps look for blocks in windows of up to 32 tokens, of which each
// lane locates one.  The queries' rows are shared out to the CTAs behind those.
#include "serve.cuh"

namespace fp4 {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

struct Ap8Params {
  fp4_append_params p;
  fp4_kv_scales s;
  int units;     // units of 16 elements of a head
  int window;    // tokens that a warp looks at together
  int kv_ctas;   // CTAs for keys and values; further ones for queries
  uint32_t *status;
};

// Where a token at position pos of a sequence lies: false if it is skipped or
// outside a table.
__device__ __forceinline__ bool locate8(const fp4_kv_cache &c, int64_t seq, int pos, int64_t limit, uint32_t *status,
                                        int &page, int &place) {
  page = place = 0;
  if (pos < 0) return false;
  bool ok = seq >= 0 && seq < c.seqs && pos < c.seq_pages * c.page_size && pos < limit;
  if (ok) {
    const int e = pos / c.page_size;
    place = pos - e * c.page_size;
    page = c.table[seq * c.table_stride + e];
    ok = page >= 0 && page < c.pages;
  }
  if (!ok && status) raise_status(status, kStatusIndex);
  return ok;
}

template <typename T>
struct Two;
template <>
struct Two<__nv_bfloat16> {
  static __device__ __forceinline__ float2 get(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }
  static __device__ __forceinline__ uint32_t put(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
};
template <>
struct Two<__half> {
  static __device__ __forceinline__ float2 get(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
  }
  static __device__ __forceinline__ uint32_t put(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
};

// Two values as E4M3 codes (nearest-even; not finite: NaN), the first low.
__device__ __forceinline__ uint32_t codes2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
// (the conversion saturates infinities: NaN in their place)
__device__ __forceinline__ float or_nan(float v) { return fabsf(v) <= 3.4028235e38f ? v : NAN; }

__device__ __forceinline__ float e8m0_value(int code) {  // 0 .. 254
  return __uint_as_float(code ? (uint32_t)code << 23 : 0x00400000u);
}
__device__ __forceinline__ float e8m0_inverse(int code) {
  return __uint_as_float(code == 254 ? 0x00400000u : (uint32_t)(254 - code) << 23);
}
// Code of the smallest power of two, 2^-127 at least, that brings `top` to 448 or less.
__device__ __forceinline__ int code_for(float top) {
  // 448 = 1.75 * 2^8
  const uint32_t bits = __float_as_uint(top);
  const int e = (int)(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u);
  return e > 0 ? e : 0;  // (a subnormal top has e <= 0 too)
}

// Where the two pieces of a unit lie, and what turns them.
struct Unit {
  int o1, o2;
  bool halves, turn1, turn2;
};
__device__ __forceinline__ Unit unit_at(const fp4_append_params &p, int u) {
  Unit r;
  const int turned = p.interleaved ? 0 : p.rot_dim / 16;
  r.halves = u < turned;
  r.o1 = r.halves ? 8 * u : 16 * u;  // 16 u = rot_dim + 16 (u - turned)
  r.o2 = r.halves ? r.o1 + p.rot_dim / 2 : r.o1 + 8;
  r.turn1 = r.halves || (p.interleaved && r.o1 < p.rot_dim);
  r.turn2 = r.halves || (p.interleaved && r.o2 < p.rot_dim);
  return r;
}
struct Turn {
  float co[8], si[8];
};
// cos and sin of a unit at a position.
__device__ __forceinline__ void load_turn(const fp4_append_params &p, const Unit &u, int pos, Turn &r) {
  if (!u.turn1 && !u.turn2) return;
  const float *cs = p.rope + (int64_t)pos * p.rot_dim + (u.halves ? u.o1 : u.o1 / 2);
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    if (i == 4 && !u.turn2) continue;
    *reinterpret_cast<float4 *>(r.co + i) = *reinterpret_cast<const float4 *>(cs + i);
    *reinterpret_cast<float4 *>(r.si + i) = *reinterpret_cast<const float4 *>(cs + p.rot_dim / 2 + i);
  }
}
// A unit's 16 values, turned.
template <typename T>
__device__ __forceinline__ void turn_unit(const Unit &u, uint4 a, uint4 b, const Turn &r, float (&x)[16]) {
  const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 va = Two<T>::get(wa[i]), vb = Two<T>::get(wb[i]);
    x[2 * i] = va.x, x[2 * i + 1] = va.y, x[8 + 2 * i] = vb.x, x[8 + 2 * i + 1] = vb.y;
  }
  if (u.halves) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = x[i], w = x[8 + i];
      x[i] = v * r.co[i] - w * r.si[i];
      x[8 + i] = w * r.co[i] + v * r.si[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < 4 ? u.turn1 : u.turn2) {
        const float v = x[2 * i], w = x[2 * i + 1];
        x[2 * i] = v * r.co[i] - w * r.si[i];
        x[2 * i + 1] = w * r.co[i] + v * r.si[i];
      }
  }
}
// The same without whole pieces: 16 consecutive elements, any pointers and
// strides, any rot_dim.
template <typename T>
__device__ __forceinline__ void turn_any(const fp4_append_params &p, const T *src, int u, int pos, bool key, float (&x)[16]) {
  const int half = p.rot_dim / 2;
  const float *cs = p.rope + (int64_t)pos * p.rot_dim;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int d = 16 * u + i;
    const float v = to_f32(src[d]);
    x[i] = v;
    if (!key || d >= p.rot_dim) continue;
    const int j = p.interleaved ? d / 2 : d < half ? d : d - half;
    const bool first = p.interleaved ? d % 2 == 0 : d < half;
    const float w = to_f32(src[p.interleaved ? d ^ 1 : first ? d + half : d - half]);
    x[i] = first ? v * cs[j] - w * cs[half + j] : v * cs[j] + w * cs[half + j];
  }
}

// Keys and values.  Item i of a warp: window i / (2 kv_heads), head i % (2
// kv_heads) of the keys, then of the values.
template <typename T, bool WHOLE>
__device__ __forceinline__ void store_blocks(const Ap8Params &a) {
  const fp4_append_params &p = a.p;
  const fp4_kv_cache &c = p.cache;
  const int lane = threadIdx.x & 31, block = a.s.block, Hk = c.kv_heads;
  const int rows = 32 / a.units, my_row = lane / a.units, my_unit = lane - my_row * a.units;
  const bool busy = my_row < rows;
  const int64_t limit = p.rot_dim ? p.rope_len : INT64_MAX;
  const int64_t windows = (p.tokens + a.window - 1) / a.window, items = windows * 2 * Hk;
  const Unit unit = unit_at(p, my_unit);
  for (int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); item < items; item += (int64_t)a.kv_ctas * kWarps) {
    const int64_t t0 = item / (2 * Hk) * a.window;
    const int hv = (int)(item % (2 * Hk)), head = hv < Hk ? hv : hv - Hk;
    const bool key = hv < Hk;
    // token t0 + lane: its place, and whether it goes on with the block of the one before
    auto joins = [&](int64_t t) {
      if (t < 1 || t >= p.tokens) return false;
      const int pos = p.pos[t], last = p.pos[t - 1];
      return pos > 0 && pos % block != 0 && pos == last + 1 && (p.seq ? p.seq[t] == p.seq[t - 1] : false);
    };
    const int64_t mine = t0 + lane;
    const bool in = lane < a.window && mine < p.tokens;
    const int my_pos = in ? p.pos[mine] : -1;
    const int my_seq = in ? (p.seq ? p.seq[mine] : (int)mine) : 0;
    int my_page, my_place;
    const bool keep = locate8(c, my_seq, my_pos, limit, hv == 0 ? a.status : nullptr, my_page, my_place);
    uint32_t leaders = __ballot_sync(~0u, keep && !joins(mine));
    uint8_t *const sf0 = key ? a.s.k_sf : a.s.v_sf;
    const int64_t sf_page = key ? a.s.k_page : a.s.v_page, sf_block = key ? a.s.k_block : a.s.v_block;
    const int64_t sf_head = key ? a.s.k_head : a.s.v_head;
    const int64_t my_sf = (int64_t)my_page * sf_page + (my_place / block) * sf_block + head * sf_head;
    const int my_old = keep ? sf0[my_sf] : 0;
    while (leaders) {
      const int L = __ffs(leaders) - 1;
      leaders &= leaders - 1;
      const int64_t t = t0 + L;
      const int pos0 = __shfl_sync(~0u, my_pos, L), page = __shfl_sync(~0u, my_page, L);
      const int place0 = __shfl_sync(~0u, my_place, L), old = __shfl_sync(~0u, my_old, L);
      uint8_t *const sf = sf0 + __shfl_sync(~0u, my_sf, L);
      const int begin = place0 % block, room = block - begin;
      int n = 1;  // tokens of the block from here on (positions behind a table's end are not in them)
      for (int base = 1; base < room; base += 32) {
        const int i = base + lane;
        const uint32_t on = __ballot_sync(~0u, i < room && joins(t + i) && pos0 + i < limit);
        const int more = on == ~0u ? 32 : __ffs(~on) - 1;
        n += more;
        if (more < 32) break;
      }
      const T *const src = (key ? static_cast<const T *>(p.k) + t * p.k_token + head * p.k_head
                                : static_cast<const T *>(p.v) + t * p.v_token + head * p.v_head);
      const int64_t step = key ? p.k_token : p.v_token;
      uint8_t *const dst = static_cast<uint8_t *>(key ? c.k : c.v) + (int64_t)page * (key ? c.k_page : c.v_page) +
                           head * (key ? c.k_head : c.v_head);
      const int64_t place = key ? c.k_place : c.v_place;
      Unit u = unit;
      if (!key) u.turn1 = u.turn2 = u.halves = false;
      auto values = [&](int r, float (&x)[16]) {
        const T *row = src + r * step;
        if (WHOLE) {
          Turn turn;
          load_turn(p, u, pos0 + r, turn);
          const uint4 v = *reinterpret_cast<const uint4 *>(row + unit.o1), w = *reinterpret_cast<const uint4 *>(row + unit.o2);
          turn_unit<T>(u, v, w, turn, x);
        } else {
          turn_any(p, row, my_unit, pos0 + r, key, x);
        }
      };
      float top = 0.0f;
      for (int r = my_row; r < n && busy; r += rows) {
        float x[16];
        values(r, x);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float v = fabsf(x[i]);
          if (v <= 3.4028235e38f) top = fmaxf(top, v);
        }
      }
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, x));
      const bool fresh = begin == 0;
      const int need = code_for(top), code = fresh || need > old ? need : old;
      const float f = e8m0_inverse(code < 255 ? code : 254);
      for (int r = my_row; r < n && busy; r += rows) {
        float x[16];
        values(r, x);
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = codes2(or_nan(x[2 * i]) * f, or_nan(x[2 * i + 1]) * f);
        uint8_t *to = dst + (place0 + r) * place;
        const int o1 = WHOLE ? unit.o1 : 16 * my_unit, o2 = WHOLE ? unit.o2 : o1 + 8;
        *reinterpret_cast<uint2 *>(to + o1) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
        *reinterpret_cast<uint2 *>(to + o2) = make_uint2(w[4] | w[5] << 16, w[6] | w[7] << 16);
      }
      if (!fresh && code > old) {  // the block's other places, in the new unit
        const float down = e8m0_inverse(127 + min(code - old, 100));
        for (int r = my_row; r < block - n && busy; r += rows) {
          const int q = place0 - begin + (r < begin ? r : r + n);
          uint4 *at = reinterpret_cast<uint4 *>(dst + q * place + 16 * my_unit);
          uint4 v = *at;
          uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t lo, hi;
            asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
                : "=r"(lo), "=r"(hi)
                : "r"(w[i]));
            const float2 x = Two<__half>::get(lo), y = Two<__half>::get(hi);
            w[i] = codes2(x.x * down, x.y * down) | codes2(y.x * down, y.y * down) << 16;
          }
          *at = v;
        }
      }
      if (lane == 0 && code != old) *sf = (uint8_t)code;
    }
  }
}

// Queries: a warp takes up to 4 * (32 / units) heads of a token at a time.
constexpr int kBatch = 4;
template <typename T, bool WHOLE>
__device__ __forceinline__ void turn_queries(const Ap8Params &a) {
  const fp4_append_params &p = a.p;
  const fp4_kv_cache &c = p.cache;
  const int lane = threadIdx.x & 31;
  const int rows = 32 / a.units, my_row = lane / a.units, my_unit = lane - my_row * a.units;
  const int64_t limit = p.rot_dim ? p.rope_len : INT64_MAX;
  const int parts = (p.heads + kBatch * rows - 1) / (kBatch * rows);
  const Unit u = unit_at(p, my_unit);
  const int64_t ctas = gridDim.x - a.kv_ctas;
  for (int64_t item = ((int64_t)blockIdx.x - a.kv_ctas) * kWarps + (threadIdx.x >> 5); item < p.tokens * parts;
       item += ctas * kWarps) {
    const int64_t t = item / parts;
    const int h0 = (int)(item - t * parts) * kBatch * rows;
    const T *const src = static_cast<const T *>(p.q) + t * p.q_token;
    T *const dst = static_cast<T *>(p.q_out) + t * p.qo_token;
    const int pos = p.pos[t];
    int page, place;
    if (WHOLE) {
      uint4 v[kBatch], w[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = h0 + i * rows + my_row;
        v[i] = w[i] = make_uint4(0, 0, 0, 0);
        if (my_row >= rows || h >= p.heads) continue;
        v[i] = *reinterpret_cast<const uint4 *>(src + h * p.q_head + u.o1);
        w[i] = *reinterpret_cast<const uint4 *>(src + h * p.q_head + u.o2);
      }
      const bool keep = locate8(c, p.seq ? p.seq[t] : t, pos, limit, nullptr, page, place);
      Turn turn;
      if (keep) load_turn(p, u, pos, turn);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = h0 + i * rows + my_row;
        if (my_row >= rows || h >= p.heads) continue;
        uint4 *at1 = reinterpret_cast<uint4 *>(dst + h * p.qo_head + u.o1);
        uint4 *at2 = reinterpret_cast<uint4 *>(dst + h * p.qo_head + u.o2);
        if (!keep) {
          *at1 = *at2 = make_uint4(0, 0, 0, 0);
          continue;
        }
        float x[16];
        turn_unit<T>(u, v[i], w[i], turn, x);
        *at1 = make_uint4(Two<T>::put(x[0], x[1]), Two<T>::put(x[2], x[3]), Two<T>::put(x[4], x[5]), Two<T>::put(x[6], x[7]));
        *at2 = make_uint4(Two<T>::put(x[8], x[9]), Two<T>::put(x[10], x[11]), Two<T>::put(x[12], x[13]),
                          Two<T>::put(x[14], x[15]));
      }
    } else {  // by pairs, then single elements
      const bool keep = locate8(c, p.seq ? p.seq[t] : t, pos, limit, nullptr, page, place);
      const int half = p.rot_dim / 2, per = c.head_dim - half, heads = min(kBatch * rows, p.heads - h0);
      const float *cs = p.rope + (int64_t)(keep ? pos : 0) * p.rot_dim;
      for (int i = lane; i < heads * per; i += 32) {
        const int h = h0 + i / per, d = i % per;
        const T *from = src + h * p.q_head;
        T *to = dst + h * p.qo_head;
        if (d >= half) {
          to[half + d] = keep ? from[half + d] : from_f32<T>(0.0f);
          continue;
        }
        const int i1 = p.interleaved ? 2 * d : d, i2 = p.interleaved ? 2 * d + 1 : d + half;
        const float x = to_f32(from[i1]), y = to_f32(from[i2]);
        to[i1] = from_f32<T>(keep ? x * cs[d] - y * cs[half + d] : 0.0f);
        to[i2] = from_f32<T>(keep ? y * cs[d] + x * cs[half + d] : 0.0f);
      }
    }
  }
}

template <typename T, bool WHOLE>
__global__ void __launch_bounds__(kThreads) k_append8(const __grid_constant__ Ap8Params a) {
  dependent_wait();
  launch_dependents();
  if (blockIdx.x < a.kv_ctas)
    store_blocks<T, WHOLE>(a);
  else
    turn_queries<T, WHOLE>(a);
}

bool whole8(const void *ptr, int64_t s0, int64_t s1) { return aligned16(ptr) && s0 % 8 == 0 && s1 % 8 == 0; }

template <typename T>
fp4_status launch_append(Ap8Params &a, cudaStream_t s) {
  const fp4_append_params &p = a.p;
  const bool whole = p.rot_dim % (p.interleaved ? 8 : 16) == 0 && whole8(p.k, p.k_token, p.k_head) &&
                     whole8(p.v, p.v_token, p.v_head) && aligned16(p.rope) &&
                     (!p.q || (whole8(p.q, p.q_token, p.q_head) && whole8(p.q_out, p.qo_token, p.qo_head)));
  a.units = p.cache.head_dim / 16;
  const int heads = 2 * p.cache.kv_heads, rows = 32 / a.units;
  const int64_t most = 8 * (int64_t)sm_count();  // CTAs resident at once, about
  a.window = 1;
  while (a.window < 32 && ceil_div(p.tokens, a.window) * heads > most * kWarps) a.window *= 2;
  const int64_t kv = ceil_div(ceil_div(p.tokens, a.window) * heads, kWarps);
  a.kv_ctas = (int)(kv < most ? kv : most);
  const int64_t qn = p.q ? ceil_div(p.tokens * ceil_div(p.heads, kBatch * rows), kWarps) : 0;
  const unsigned grid = (unsigned)(a.kv_ctas + (qn < most ? qn : most));
  const auto kern = whole ? k_append8<T, true> : k_append8<T, false>;
  return launch_dependent(kern, dim3(grid), dim3(kThreads), 0, s, a) == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

// ------------------------------------------------------------- reading back

struct RdParams {
  fp4_read_params p;
  int pieces;    // 16-byte pieces of a stored head
  int tokens;    // tokens of a CTA at a time
  uint32_t *status;
};

// A thread takes a piece of 16 stored bytes: codes become 16 elements, 16-bit
// elements are copied.  Neighbours take neighbouring pieces of a token's heads.
template <typename T, bool CODES>
__global__ void __launch_bounds__(kThreads) k_read(const __grid_constant__ RdParams a) {
  const fp4_read_params &p = a.p;
  const fp4_kv_cache &c = p.cache;
  constexpr int kEach = CODES ? 16 : 8;
  dependent_wait();
  launch_dependents();
  const int per = 2 * c.kv_heads * a.pieces;  // of a token: its keys, its values
  const int width = kThreads / a.tokens, tl = threadIdx.x / width, in = threadIdx.x - tl * width;
  if (tl >= a.tokens) return;
  for (int64_t t = (int64_t)blockIdx.x * a.tokens + tl; t < p.tokens; t += (int64_t)gridDim.x * a.tokens) {
    int page, place;
    const bool keep = locate8(c, p.seq ? p.seq[t] : t, p.pos[t], INT64_MAX, in == 0 ? a.status : nullptr, page, place);
    for (int i = in; i < per; i += width) {
      const int row = i / a.pieces, d = (i - row * a.pieces) * kEach;
      const bool key = row < c.kv_heads;
      const int head = key ? row : row - c.kv_heads;
      T *out = key ? static_cast<T *>(p.k_out) + t * p.k_token + head * p.k_out_head + d
                   : static_cast<T *>(p.v_out) + t * p.v_token + head * p.v_out_head + d;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (keep) {
        const int64_t at = key ? (int64_t)page * c.k_page + place * c.k_place + head * c.k_head + d
                               : (int64_t)page * c.v_page + place * c.v_place + head * c.v_head + d;
        v = *reinterpret_cast<const uint4 *>(static_cast<const char *>(key ? c.k : c.v) + at * (CODES ? 1 : 2));
      }
      if (!CODES) {
        *reinterpret_cast<uint4 *>(out) = v;
        continue;
      }
      float f = 0.0f;
      if (keep) {
        const int b = place / p.scales.block;
        const int code = key ? p.scales.k_sf[(int64_t)page * p.scales.k_page + b * p.scales.k_block + head * p.scales.k_head]
                             : p.scales.v_sf[(int64_t)page * p.scales.v_page + b * p.scales.v_block + head * p.scales.v_head];
        f = code == 255 ? NAN : e8m0_value(code);
      }
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t r[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t lo, hi;
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w[j]));
        const float2 x = Two<__half>::get(lo), y = Two<__half>::get(hi);
        r[2 * j] = Two<T>::put(x.x * f, x.y * f);
        r[2 * j + 1] = Two<T>::put(y.x * f, y.y * f);
      }
      reinterpret_cast<uint4 *>(out)[0] = make_uint4(r[0], r[1], r[2], r[3]);
      reinterpret_cast<uint4 *>(out)[1] = make_uint4(r[4], r[5], r[6], r[7]);
    }
  }
}

template <typename T>
fp4_status launch_read(RdParams &a, cudaStream_t s) {
  const fp4_read_params &p = a.p;
  const bool codes = p.scales.k_sf != nullptr;
  a.pieces = p.cache.head_dim / (codes ? 16 : 8);
  const int per = 2 * p.cache.kv_heads * a.pieces;
  a.tokens = 1;
  while (a.tokens < 32 && kThreads / (2 * a.tokens) >= per) a.tokens *= 2;
  const int64_t most = 8 * (int64_t)sm_count(), want = ceil_div(p.tokens, a.tokens);
  const auto kern = codes ? k_read<T, true> : k_read<T, false>;
  return launch_dependent(kern, dim3((unsigned)(want < most ? want : most)), dim3(kThreads), 0, s, a) == cudaSuccess
             ? FP4_OK
             : FP4_ERR_CUDA;
}

}  // namespace

fp4_status launch_kv_append8(const fp4_append8_params &p, cudaStream_t s) {
  Ap8Params a{};
  a.p = p.base;
  a.s = p.scales;
  a.status = status_word();
  if (!a.status) return FP4_ERR_CUDA;
  return a.p.cache.type == FP4_BF16 ? launch_append<__nv_bfloat16>(a, s) : launch_append<__half>(a, s);
}

fp4_status launch_kv_read(const fp4_read_params &p, cudaStream_t s) {
  RdParams a{};
  a.p = p;
  a.status = status_word();
  if (!a.status) return FP4_ERR_CUDA;
  return p.cache.type == FP4_BF16 ? launch_read<__nv_bfloat16>(a, s) : launch_read<__half>(a, s);
}

}  // namespace fp4
