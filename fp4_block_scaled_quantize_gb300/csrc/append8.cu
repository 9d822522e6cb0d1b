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
// Measured in a graph: 192 tokens of 192 sequences, 16 + 2 x 16 heads of 64 in
// blocks of 8 4.1 us, one token 3.6; 8191 prompt tokens of 32 + 2 x 8 heads of 128
// in blocks of 64 51.1 us (3.6 TB/s, 54% of a copy's rate; without queries 27: some
// 700 instructions of a warp a head and 64 tokens, 16 warps an SM by 128 registers, of
// which the forms that hold two rows spill 120 - 128 bytes); rows whose rotated part
// is not whole pieces go element by element (8000 tokens, heads of 80 with 40 rotated
// 283 us, with 32 or 80 49); reading 100003 tokens back 97.5 us (6.3 TB/s, 93%), 300
// 2.1 us.
//
// A rotated key is rounded to binary32 before it is rounded to its code: about one
// code in a million is the other neighbour of a number that lies within 2^-20 of
// the middle of two.  Rotations whose binary32 result is rounded to odd wherever a
// middle is near have none of these, and took 59.8 us for 50.8.
//
// Order.  A block whose tokens stand apart in the call would be written by teams
// that know nothing of each other.  CTAs of their own look for that and report it:
// of each 256 tokens those that go on with a block without the token before them
// (none in whole prompts) into a table in shared memory, which every token of the
// call is then looked up in, beside the work of the others.  They come first in the
// grid: 8191 prompt tokens 51.1 us (50.5 without, 51.6 last), 8000 single tokens
// 57.5 (56.5, 67.6), 192 of them 4.4 (4.35).
//
// Layout.  Lanes hold units of 16 elements (two pieces of 8, in the rotated part
// those whose elements form pairs) of 32 / units rows; a team of warps takes the
// tokens of one block and one key or value head.  Teams look for blocks in windows
// of up to 32 tokens, of which each lane locates one.  The queries' rows are taken
// by CTAs of their own, every so many.
#include "serve.cuh"

namespace fp4 {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kResident = 2;  // CTAs an SM holds at least

struct Ap8Params {
  fp4_append_params p;
  fp4_kv_scales s;
  int units;     // units of 16 elements of a head
  int team;      // warps that take a run together
  int window;    // tokens that a team looks at together
  int chunks;    // parts of the heads, each a team's
  Divisor page, block;
  int kv_ctas;   // CTAs for keys and values; further ones for queries: `ctas` of both
  int ctas;
  int checks;    // CTAs before those, for the order of the tokens
  uint32_t *status;
};

// Where a token at position pos of a sequence lies: false if it is skipped or
// outside a table.
__device__ __forceinline__ bool locate8(const fp4_kv_cache &c, const Divisor &by, int64_t seq, int pos, int64_t limit,
                                        uint32_t *status, int &page, int &place) {
  page = place = 0;
  if (pos < 0) return false;
  bool ok = seq >= 0 && seq < c.seqs && pos < c.seq_pages * c.page_size && pos < limit;
  if (ok) {
    const int e = over(pos, by);
    place = pos - e * c.page_size;
    page = c.table[seq * c.table_stride + e];
    ok = page >= 0 && page < c.pages;
  }
  if (!ok && status) raise_status(status, kStatusIndex);
  return ok;
}

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

// How rows are read: whole pieces, pairs (i, i + rot_dim / 2) or neighbours, with
// strides of rows and heads in 32 bits; or any pointers, strides and rot_dim.
enum Kind { kHalves, kPairs, kAny };

// Where the two pieces of a unit lie, and which of them are turned.
struct Unit {
  int o1, o2;
  bool turn1, turn2;
};
template <int KIND>
__device__ __forceinline__ Unit unit_at(const fp4_append_params &p, int u) {
  Unit r;
  const bool halves = KIND == kHalves && u < p.rot_dim / 16;
  r.o1 = halves ? 8 * u : 16 * u;  // behind the rotated part 16 u = rot_dim + 16 (u - rot_dim / 16)
  r.o2 = halves ? r.o1 + p.rot_dim / 2 : r.o1 + 8;
  r.turn1 = halves || (KIND == kPairs && r.o1 < p.rot_dim);
  r.turn2 = halves || (KIND == kPairs && r.o2 < p.rot_dim);
  return r;
}
struct Turn {
  float co[8], si[8];
};
// cos and sin of a unit at a position.
template <int KIND>
__device__ __forceinline__ void load_turn(const fp4_append_params &p, const Unit &u, bool key, int pos, Turn &r) {
  if (!key || !u.turn1) return;
  const float *cs = p.rope + (int64_t)pos * p.rot_dim + (KIND == kHalves ? u.o1 : u.o1 / 2);
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    if (i == 4 && KIND == kPairs && !u.turn2) continue;
    const float4 co = *reinterpret_cast<const float4 *>(cs + i);
    const float4 si = *reinterpret_cast<const float4 *>(cs + p.rot_dim / 2 + i);
    r.co[i] = co.x, r.co[i + 1] = co.y, r.co[i + 2] = co.z, r.co[i + 3] = co.w;
    r.si[i] = si.x, r.si[i + 1] = si.y, r.si[i + 2] = si.z, r.si[i + 3] = si.w;
  }
}
// A unit's 16 values, turned.
template <typename T, int KIND>
__device__ __forceinline__ void turn_unit(bool key, const Unit &u, uint4 a, uint4 b, const Turn &r, float (&x)[16]) {
  const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 va = unpack<T>(wa[i]), vb = unpack<T>(wb[i]);
    x[2 * i] = va.x, x[2 * i + 1] = va.y, x[8 + 2 * i] = vb.x, x[8 + 2 * i + 1] = vb.y;
  }
  if (!key || !u.turn1) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int j = KIND == kHalves ? i : 2 * i, k = KIND == kHalves ? 8 + i : 2 * i + 1;
    if (KIND == kPairs && i >= 4 && !u.turn2) continue;
    const float v = x[j], w = x[k];
    x[j] = v * r.co[i] - w * r.si[i];
    x[k] = w * r.co[i] + v * r.si[i];
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

// Keys and values.  Item i of a team of warps: window i / chunks, of its 2 kv_heads
// heads (keys', then values') the chunk i % chunks.  The tokens of a window fall
// into runs, each of one block, at consecutive places; a run may go on behind the
// window.  Either the team takes one run after the other, its groups of lanes a
// token each, or each group takes a run of its own.  A group holds kHold rows at a
// time (more than one costs registers: 192 tokens of 192 sequences take 5.4 us with
// two, 4.0 with one); of longer runs all but the last are loaded again for their
// codes.
template <typename T, int KIND, int kHold>
__device__ __forceinline__ void store_blocks(const Ap8Params &a, int cta) {
  const fp4_append_params &p = a.p;
  const fp4_kv_cache &c = p.cache;
  using Step = typename std::conditional<KIND == kAny, int64_t, int>::type;
  __shared__ unsigned top_sh[2][kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, block = a.s.block, Hk = c.kv_heads;
  const int groups = 32 / a.units, my_group = lane / a.units, my_unit = lane - my_group * a.units;
  const int teams = kWarps / a.team, team = warp / a.team, mate = warp % a.team;
  const int all = groups * a.team, my_all = mate * groups + my_group;  // the team's groups
  int parity = 0;
  const int64_t limit = p.rot_dim ? p.rope_len : INT64_MAX;
  const int64_t windows = (p.tokens + a.window - 1) / a.window, items = windows * a.chunks;
  const Unit unit = unit_at<KIND>(p, my_unit);
  for (int64_t item = (int64_t)cta * teams + team; item < items; item += (int64_t)a.kv_ctas * teams) {
    const int64_t t0 = item / a.chunks * a.window;
    const int chunk = (int)(item % a.chunks), hv0 = 2 * Hk * chunk / a.chunks, hv1 = 2 * Hk * (chunk + 1) / a.chunks;
    // whether token t goes on with the block of the one before
    auto joins = [&](int64_t t) {
      if (!p.seq || t < 1 || t >= p.tokens) return false;
      const int pos = p.pos[t], last = p.pos[t - 1];
      const bool same = p.seq[t] == p.seq[t - 1];
      return pos > 0 && pos == last + 1 && same && pos != over(pos, a.block) * block;
    };
    const int64_t mine = t0 + lane;
    const bool in = lane < a.window && mine < p.tokens;
    const int my_pos = in ? p.pos[mine] : -1;
    const int my_seq = in ? (p.seq ? p.seq[mine] : (int)mine) : 0;
    const bool my_join = in && joins(mine);
    const bool ranged = my_pos >= 0 && my_seq >= 0 && my_seq < c.seqs && my_pos < c.seq_pages * c.page_size && my_pos < limit;
    if (my_pos >= 0 && !ranged && chunk == 0 && mate == 0) raise_status(a.status, kStatusIndex);
    const int my_entry = over(max(my_pos, 0), a.page), my_place = my_pos - my_entry * c.page_size;
    int my_page = -1;
    if (ranged) my_page = c.table[my_seq * c.table_stride + my_entry];
    const uint32_t joined = __ballot_sync(~0u, ranged && my_join), leaders = __ballot_sync(~0u, ranged && !my_join);
    const int count = __popc(leaders);
    // steps of a run after the other, and of runs side by side, with a run's own
    // latencies as three steps
    const int length = count ? (__popc(joined) + count - 1) / count + 1 : 1;
    const bool apart = !p.seq || (count > 1 && (count + all - 1) / all * (length + 3) < count * ((length + all - 1) / all + 3));
    for (int base = 0; base < count; base += apart ? all : 1) {
      const int which = base + (apart ? my_all : 0);
      const bool active = my_group < groups && which < count;
      uint32_t rest = leaders;
      for (int i = 0; i < (active ? which : base); ++i) rest &= rest - 1;
      const int L = __ffs(rest) - 1;
      const int64_t t = t0 + L;
      const int pos0 = __shfl_sync(~0u, my_pos, L), place0 = __shfl_sync(~0u, my_place, L);
      const int blk = over(place0, a.block), begin = place0 - blk * block;
      const uint32_t on = L < 31 ? joined >> (L + 1) : 0;
      int n = __ffs(~on);  // tokens of the run in the window
      const int most = (int)min((int64_t)(block - begin), limit - pos0);
      if (!apart) {
        if (L + n == a.window)  // it may go on behind
          for (;; n += 32) {
            const uint32_t more = __ballot_sync(~0u, n + lane < most && joins(t + n + lane));
            if (more != ~0u) {
              n += __ffs(~more) - 1;
              break;
            }
          }
      } else {
        while (active && L + n >= a.window && n < most && joins(t + n)) ++n;
      }
      const int page = __shfl_sync(~0u, my_page, L);
      const bool there = page >= 0 && page < c.pages;
      if (active && !there && my_unit == 0) raise_status(a.status, kStatusIndex);
      const int r0 = apart ? 0 : my_all, hop = apart ? 1 : all, rows = active && there ? n : 0;
      int steps = (n + kHold * hop - 1) / (kHold * hop);
      if (apart) steps = __reduce_max_sync(~0u, active ? steps : 1);
      // kHold rows from r on; behind the last row, and for lanes without one, a row
      // that is there again, which changes no largest.  Runs of one step: the next
      // head's are requested before this one's are done with (two or four heads
      // ahead measured the same), and the heads share their cosines and sines.
      uint4 v[kHold], w[kHold];
      Turn turn[kHold];
      // the head whose rows are asked for next, and the one that is stored: where
      // token t's row, its scale and the steps to other rows and heads are
      const T *src = nullptr;
      Step src_row = 0, src_head = 0;
      int ahead[kHold];
#pragma unroll
      for (int h = 0; h < kHold; ++h) ahead[h] = max(min(r0 + h * hop, rows - 1), 0);
      uint8_t *dst = nullptr, *sf = nullptr;
      Step dst_row = 0, dst_head = 0, sf_head = 0;
      auto read_from = [&](int hv) {
        const bool key = hv < Hk;
        const int head = key ? hv : hv - Hk;
        src_row = (Step)(key ? p.k_token : p.v_token);
        src_head = (Step)(key ? p.k_head : p.v_head);
        src = static_cast<const T *>(key ? p.k : p.v) + t * src_row + (int64_t)head * src_head;
      };
      auto store_to = [&](int hv) {
        const bool key = hv < Hk;
        const int head = key ? hv : hv - Hk;
        dst_row = (Step)(key ? c.k_place : c.v_place);
        dst_head = (Step)(key ? c.k_head : c.v_head);
        sf_head = (Step)(key ? a.s.k_head : a.s.v_head);
        dst = static_cast<uint8_t *>(key ? c.k : c.v) + (int64_t)page * (key ? c.k_page : c.v_page) +
              (int64_t)head * dst_head + (int64_t)place0 * dst_row;
        sf = (key ? a.s.k_sf : a.s.v_sf) + (int64_t)head * sf_head + (int64_t)page * (key ? a.s.k_page : a.s.v_page) +
             blk * (key ? a.s.k_block : a.s.v_block);
      };
      auto next_read = [&](int hv) {
        if (hv == Hk) read_from(hv);
        else src += src_head;
      };
      auto ask = [&](int r) {
#pragma unroll
        for (int h = 0; h < kHold; ++h) {
          if (KIND == kAny) continue;
          const T *const row = src + (int64_t)(r == r0 ? ahead[h] : max(min(r + h * hop, rows - 1), 0)) * src_row;
          v[h] = *reinterpret_cast<const uint4 *>(row + unit.o1);
          w[h] = *reinterpret_cast<const uint4 *>(row + unit.o2);
        }
      };
      auto ask_turns = [&](bool key, int r) {
#pragma unroll
        for (int h = 0; h < kHold; ++h)
          if (KIND != kAny) load_turn<KIND>(p, unit, key, pos0 + max(min(r + h * hop, rows - 1), 0), turn[h]);
      };
      const bool single = steps == 1;
      read_from(hv0);
      store_to(hv0);
      if (single) {
        ask(r0);
        ask_turns(hv0 < Hk, r0);
      }
      for (int hv = hv0; hv < hv1; ++hv) {
        const bool key = hv < Hk;
        if (hv == Hk && hv != hv0) store_to(hv);
        const int old = rows ? *sf : 0;
        float x[kHold][16];
        auto over_team = [&](float top) {
          if (apart) {
            const float own = top;
            for (int o = 1; o < a.units; ++o) {
              const int from = my_unit + o < a.units ? lane + o : lane + o - a.units;
              top = fmaxf(top, __shfl_sync(~0u, own, from & 31));
            }
            return top;
          }
          // (numbers that are not negative are ordered as their bits are)
          unsigned bits = __reduce_max_sync(~0u, __float_as_uint(top));
          if (a.team > 1) {
            if (lane == 0) top_sh[parity][warp] = bits;
            asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * a.team) : "memory");
            bits = __reduce_max_sync(~0u, top_sh[parity][team * a.team + (lane & (a.team - 1))]);
            parity ^= 1;
          }
          return __uint_as_float(bits);
        };
        auto take = [&](int r) {
#pragma unroll
          for (int h = 0; h < kHold; ++h) {
            const int q = max(min(r + h * hop, rows - 1), 0);
            if (KIND == kAny)
              turn_any(p, src + (int64_t)q * src_row, my_unit, pos0 + q, key, x[h]);
            else
              turn_unit<T, KIND>(key, unit, v[h], w[h], turn[h], x[h]);
          }
        };
        auto leave_out = [&] {
#pragma unroll
          for (int h = 0; h < kHold; ++h)
#pragma unroll
            for (int e = 0; e < 16; ++e) x[h][e] = or_nan(x[h][e]);
        };
        auto largest = [&](float &top, float &more) {  // (of a number and a NaN: the number)
#pragma unroll
          for (int h = 0; h < kHold; ++h)
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              top = fmaxf(top, fabsf(x[h][e]));
              more = fmaxf(more, fabsf(x[h][e + 1]));
            }
        };
        // the largest; where that is an infinity, once more without infinities
        float top;
        bool infinite = false;
        if (single) {
          float more = top = 0.0f;
          take(r0);
          largest(top, more);
          top = over_team(fmaxf(top, more));
          infinite = apart ? __any_sync(~0u, isinf(top)) : isinf(top);
          if (infinite) {
            more = top = 0.0f;
            leave_out();
            largest(top, more);
            top = over_team(fmaxf(top, more));
          }
        } else {
          for (;; infinite = true) {
            float more = top = 0.0f;
            for (int i = 0; i < steps; ++i) {
              ask(r0 + i * kHold * hop);
              ask_turns(key, r0 + i * kHold * hop);
              take(r0 + i * kHold * hop);
              if (infinite) leave_out();
              largest(top, more);
            }
            top = over_team(fmaxf(top, more));
            if (infinite || !(apart ? __any_sync(~0u, isinf(top)) : isinf(top))) break;
          }
        }
        if (single && hv + 1 < hv1) {
          next_read(hv + 1);
          ask(r0);
        }
        const int need = code_for(top), code = begin == 0 || need > old ? need : old;
        const float f = e8m0_inverse(code < 255 ? code : 254);
        for (int i = steps - 1;;) {
#pragma unroll
          for (int h = 0; h < kHold; ++h) {
            const int r = r0 + (i * kHold + h) * hop;
            if (r >= rows) continue;
            uint32_t z[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = codes2(x[h][2 * e] * f, x[h][2 * e + 1] * f);
            uint8_t *to = dst + (int64_t)r * dst_row;
            const int o1 = KIND != kAny ? unit.o1 : 16 * my_unit, o2 = KIND != kAny ? unit.o2 : o1 + 8;
            *reinterpret_cast<uint2 *>(to + o1) = make_uint2(z[0] | z[1] << 16, z[2] | z[3] << 16);
            *reinterpret_cast<uint2 *>(to + o2) = make_uint2(z[4] | z[5] << 16, z[6] | z[7] << 16);
          }
          if (i-- == 0) break;
          ask(r0 + i * kHold * hop);
          ask_turns(key, r0 + i * kHold * hop);
          take(r0 + i * kHold * hop);
          if (infinite) leave_out();
        }
        if (rows && begin != 0 && code > old) {  // the block's other places, in the new unit
          const float down = e8m0_inverse(127 + min(code - old, 100));
#pragma unroll 4
          for (int r = r0; r < block - n; r += hop) {
            const int q = (r < begin ? r : r + n) - begin;
            uint4 *at = reinterpret_cast<uint4 *>(dst + (int64_t)q * dst_row + 16 * my_unit);
            const uint4 o = *at;
            uint32_t z[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t lo, hi;
              e4m3_halves(z[e], lo, hi);
              const float2 x = unpack<__half>(lo), y = unpack<__half>(hi);
              z[e] = codes2(x.x * down, x.y * down) | codes2(y.x * down, y.y * down) << 16;
            }
            *at = make_uint4(z[0], z[1], z[2], z[3]);
          }
        }
        if (rows && my_unit == 0 && (apart || my_all == 0) && code != old) *sf = (uint8_t)code;
        dst += dst_head;
        sf += sf_head;
        if (!single) next_read(hv + 1);
      }
    }
  }
}

// Whether tokens of one block stand apart.  Any two runs of a block have one that
// begins inside it: for each of those, is there a token of its block that is not
// part of the run?  (a token of the same distance in position and index behind it
// is, or is behind a run of its own)
constexpr int kSlots = 4 * kThreads;
__device__ __forceinline__ void check_order(const Ap8Params &a, int cta) {
  const fp4_append_params &p = a.p;
  const fp4_kv_cache &c = p.cache;
  __shared__ int4 begun[kThreads];  // sequence, first position of the block, position - index, index
  __shared__ int slot[kSlots];      // which of those, by a hash of the first two; -1: none
  const int block = a.s.block, tokens = (int)p.tokens;
  auto hash = [](int seq, int first) {
    return (int)(((uint32_t)seq * 0x9E3779B1u + (uint32_t)first * 0x85EBCA77u) >> 22) & (kSlots - 1);
  };
  bool apart = false;
  for (int base = cta * kThreads; base < tokens; base += a.checks * kThreads) {
    const int t = base + threadIdx.x;
    int4 mine = make_int4(0, 0, 0, t);
    bool inside = false;
    if (t < tokens) {
      const int pos = p.pos[t], seq = p.seq[t];
      const int first = over(max(pos, 0), a.block) * block;
      inside = pos > first && seq >= 0 && seq < c.seqs && pos < c.seq_pages * c.page_size &&
               !(t > 0 && p.seq[t - 1] == seq && p.pos[t - 1] == pos - 1);
      mine = make_int4(seq, first, pos - t, t);
    }
    if (!__syncthreads_or(inside)) continue;
    for (int i = threadIdx.x; i < kSlots; i += kThreads) slot[i] = -1;
    begun[threadIdx.x] = mine;
    __syncthreads();
    if (inside)  // (a slot in four is taken at most, so there is a free one)
      for (int h = hash(mine.x, mine.y);; h = (h + 1) & (kSlots - 1)) {
        const int other = atomicCAS(&slot[h], -1, threadIdx.x);
        if (other < 0) break;
        if (begun[other].x == mine.x && begun[other].y == mine.y) {
          apart = true;
          break;
        }
      }
    __syncthreads();
#pragma unroll 4
    for (int j = threadIdx.x; j < tokens; j += kThreads) {
      const int pos = p.pos[j], seq = p.seq[j];
      if (pos < 0) continue;
      const int first = over(pos, a.block) * block;
      for (int h = hash(seq, first), i; (i = slot[h]) >= 0; h = (h + 1) & (kSlots - 1)) {
        const int4 e = begun[i];
        if (e.x != seq || e.y != first) continue;
        apart |= j < e.w || pos - j != e.z;
        break;
      }
    }
    __syncthreads();
  }
  if (__syncthreads_or(apart) && threadIdx.x == 0) raise_status(a.status, kStatusIndex);
}

// Queries: a warp takes up to 4 * (32 / units) heads of a token at a time.
constexpr int kBatch = 4;
template <typename T, int KIND>
__device__ __forceinline__ void turn_queries(const Ap8Params &a, int cta) {
  const fp4_append_params &p = a.p;
  const fp4_kv_cache &c = p.cache;
  const int lane = threadIdx.x & 31;
  const int rows = 32 / a.units, my_row = lane / a.units, my_unit = lane - my_row * a.units;
  const int64_t limit = p.rot_dim ? p.rope_len : INT64_MAX;
  const int parts = (p.heads + kBatch * rows - 1) / (kBatch * rows);
  const Unit u = unit_at<KIND>(p, my_unit);
  const int64_t ctas = a.ctas - a.kv_ctas;
  for (int64_t item = (int64_t)cta * kWarps + (threadIdx.x >> 5); item < p.tokens * parts;
       item += ctas * kWarps) {
    const int64_t t = item / parts;
    const int h0 = (int)(item - t * parts) * kBatch * rows;
    const T *const src = static_cast<const T *>(p.q) + t * p.q_token;
    T *const dst = static_cast<T *>(p.q_out) + t * p.qo_token;
    const int pos = p.pos[t];
    int page, place;
    if (KIND != kAny) {
      uint4 v[kBatch], w[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = h0 + i * rows + my_row;
        v[i] = w[i] = make_uint4(0, 0, 0, 0);
        if (my_row >= rows || h >= p.heads) continue;
        v[i] = *reinterpret_cast<const uint4 *>(src + h * p.q_head + u.o1);
        w[i] = *reinterpret_cast<const uint4 *>(src + h * p.q_head + u.o2);
      }
      const bool keep = locate8(c, a.page, p.seq ? p.seq[t] : t, pos, limit, nullptr, page, place);
      Turn turn;
      load_turn<KIND>(p, u, keep, pos, turn);
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
        turn_unit<T, KIND>(true, u, v[i], w[i], turn, x);
        *at1 = make_uint4(pack<T>(x[0], x[1]), pack<T>(x[2], x[3]), pack<T>(x[4], x[5]), pack<T>(x[6], x[7]));
        *at2 = make_uint4(pack<T>(x[8], x[9]), pack<T>(x[10], x[11]), pack<T>(x[12], x[13]),
                          pack<T>(x[14], x[15]));
      }
    } else {  // by pairs, then single elements
      const bool keep = locate8(c, a.page, p.seq ? p.seq[t] : t, pos, limit, nullptr, page, place);
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

template <typename T, int KIND, int HOLD>
__global__ void __launch_bounds__(kThreads, kResident) k_append8(const __grid_constant__ Ap8Params a) {
  dependent_wait();
  launch_dependents();
  const int cta = (int)blockIdx.x - a.checks;
  if (cta < 0) {
    check_order(a, blockIdx.x);
    return;
  }
  // CTAs for keys and values, and for queries, in turn
  const int before = (int)((int64_t)cta * a.kv_ctas / a.ctas);
  if (before != (int)(((int64_t)cta + 1) * a.kv_ctas / a.ctas))
    store_blocks<T, KIND, HOLD>(a, before);
  else
    turn_queries<T, KIND>(a, cta - before);
}

bool whole8(const void *ptr, int64_t s0, int64_t s1) { return aligned16(ptr) && s0 % 8 == 0 && s1 % 8 == 0; }

template <typename T>
fp4_status launch_append(Ap8Params &a, cudaStream_t s) {
  const fp4_append_params &p = a.p;
  const int64_t steps[] = {p.k_token, p.k_head, p.v_token, p.v_head, p.cache.k_place, p.cache.k_head, p.cache.v_place,
                           p.cache.v_head, a.s.k_head, a.s.v_head};
  bool whole = true;
  for (int64_t step : steps) whole = whole && step <= INT32_MAX;
  whole = whole && p.rot_dim % (p.interleaved ? 8 : 16) == 0 && whole8(p.k, p.k_token, p.k_head) &&
          whole8(p.v, p.v_token, p.v_head) && aligned16(p.rope) &&
          (!p.q || (whole8(p.q, p.q_token, p.q_head) && whole8(p.q_out, p.qo_token, p.qo_head)));
  a.units = p.cache.head_dim / 16;
  const int heads = 2 * p.cache.kv_heads, rows = 32 / a.units;
  const int64_t most = kResident * (int64_t)sm_count(), grid_most = 1 << 20;
  // as many warps as hold a block's rows, if runs may be as long; as many tokens
  // as these have groups of lanes, or more; the heads in as few parts as leave one
  // for every warp, of windows in which a run begins
  const int64_t run = !p.seq ? 1 : p.tokens < a.s.block ? p.tokens : a.s.block, warps = most * kWarps;
  const bool two = run > kWarps * rows;
  a.team = 1;
  while (a.team < kWarps && a.team * rows * (two ? 2 : 1) < run) a.team *= 2;
  a.window = 1;
  while (a.window < 32 && ((2 * a.window <= rows * a.team && 2 * a.window <= p.tokens) ||
                           ceil_div(p.tokens, a.window) * heads * a.team > warps))
    a.window *= 2;
  const int64_t full = ceil_div(p.tokens, a.window > run ? a.window : run);
  a.chunks = heads;
  while (a.chunks > 1 && full * (a.chunks / 2) * a.team >= warps) a.chunks = (a.chunks + 1) / 2;
  a.page = divisor(p.cache.page_size);
  a.block = divisor(a.s.block);
  const int64_t kv = ceil_div(ceil_div(p.tokens, a.window) * a.chunks * a.team, kWarps);
  a.kv_ctas = (int)(kv < grid_most ? kv : grid_most);
  const int64_t qn = p.q ? ceil_div(p.tokens * ceil_div(p.heads, kBatch * rows), kWarps) : 0;
  a.ctas = a.kv_ctas + (int)(qn < grid_most ? qn : grid_most);
  // (without seq every token has a sequence, and so a block, of its own)
  const int64_t looks = p.seq && a.s.block > 1 && p.tokens > 1 ? ceil_div(p.tokens, kThreads) : 0;
  a.checks = (int)(looks < most ? looks : most);
  const unsigned grid = (unsigned)(a.checks + a.ctas);
  const auto kern = !whole          ? k_append8<T, kAny, 1>
                    : p.interleaved ? (two ? k_append8<T, kPairs, 2> : k_append8<T, kPairs, 1>)
                    : two           ? k_append8<T, kHalves, 2>
                                    : k_append8<T, kHalves, 1>;
  return launch_dependent(kern, dim3(grid), dim3(kThreads), 0, s, a) == cudaSuccess ? FP4_OK : FP4_ERR_CUDA;
}

// ------------------------------------------------------------- reading back

struct RdParams {
  fp4_read_params p;
  Divisor page, block, piece;  // piece: by the pieces of a head
  int pieces;                  // of 16 stored bytes, of a head
  int parts;                   // CTAs of the same tokens: keys', then values'
  int tokens;                  // of a CTA at a time
  bool wide;                   // rows of results begin at multiples of 32 bytes
  uint32_t *status;
};
constexpr int kReadThreads = 256, kReaders = 8;  // CTAs an SM holds

__device__ __forceinline__ void store32(void *to, const uint4 &a, const uint4 &b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(a.x), "r"(a.y), "r"(a.z),
               "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// A thread has a piece of 16 stored bytes, always the same of keys or of values, of
// one token after the other: codes become 16 elements, 16-bit elements are copied.
// Neighbours have neighbouring pieces; the next token is looked up before this
// one's piece is waited for.  Warps cover the latency, not pieces ahead: 100003
// tokens take 98 us with 8 CTAs an SM, 101 with 6; two pieces at a time and 6 CTAs
// 114, four and 4 148.  Stores of 32 bytes: with two of 16 123 became 136.
template <typename T, bool CODES>
__global__ void __launch_bounds__(kReadThreads, kReaders) k_read(const __grid_constant__ RdParams a) {
  const fp4_read_params &p = a.p;
  const fp4_kv_cache &c = p.cache;
  constexpr int kEach = CODES ? 16 : 8;
  dependent_wait();
  launch_dependents();
  const int group = blockIdx.x / a.parts, part = blockIdx.x - group * a.parts;
  const bool key = part < a.parts / 2;
  const int width = kReadThreads / a.tokens, tl = threadIdx.x / width;
  const int i = (key ? part : part - a.parts / 2) * width + threadIdx.x - tl * width;
  const int head = over(i, a.piece), d = (i - head * a.pieces) * kEach;
  if (tl >= a.tokens || head >= c.kv_heads) return;
  const int hop = gridDim.x / a.parts * a.tokens, tokens = (int)p.tokens;  // (below 2^30)
  const int64_t in_page = key ? c.k_page : c.v_page, in_place = key ? c.k_place : c.v_place;
  const int64_t sf_page = key ? p.scales.k_page : p.scales.v_page, sf_block = key ? p.scales.k_block : p.scales.v_block;
  const int64_t out_token = key ? p.k_token : p.v_token;
  const char *const from = static_cast<const char *>(key ? c.k : c.v) + (head * (key ? c.k_head : c.v_head) + d) * (CODES ? 1 : 2);
  const uint8_t *const sf = CODES ? (key ? p.scales.k_sf : p.scales.v_sf) + head * (key ? p.scales.k_head : p.scales.v_head) : nullptr;
  T *const to = static_cast<T *>(key ? p.k_out : p.v_out) + head * (key ? p.k_out_head : p.v_out_head) + d;
  int page = 0, place = 0;
  auto look = [&](int t) {
    return t < tokens && locate8(c, a.page, p.seq ? p.seq[t] : t, p.pos[t], INT64_MAX, i == 0 && key ? a.status : nullptr,
                                 page, place);
  };
  int t = group * a.tokens + tl;
  bool there = look(t);
  for (; t < tokens; t += hop) {
    uint4 v = make_uint4(0, 0, 0, 0);
    int code = 127;
    if (there) {
      v = *reinterpret_cast<const uint4 *>(from + (page * in_page + place * in_place) * (CODES ? 1 : 2));
      if (CODES) code = sf[page * sf_page + over(place, a.block) * sf_block];
    }
    there = look(t + hop);
    T *const out = to + t * out_token;
    if (!CODES) {
      *reinterpret_cast<uint4 *>(out) = v;
      continue;
    }
    const float f = code == 255 ? NAN : e8m0_value(code);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t r[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t lo, hi;
      e4m3_halves(w[e], lo, hi);
      const float2 x = unpack<__half>(lo), y = unpack<__half>(hi);
      r[2 * e] = pack<T>(x.x * f, x.y * f);
      r[2 * e + 1] = pack<T>(y.x * f, y.y * f);
    }
    const uint4 r0 = make_uint4(r[0], r[1], r[2], r[3]), r1 = make_uint4(r[4], r[5], r[6], r[7]);
    if (a.wide) {
      store32(out, r0, r1);
    } else {
      reinterpret_cast<uint4 *>(out)[0] = r0;
      reinterpret_cast<uint4 *>(out)[1] = r1;
    }
  }
}

template <typename T>
fp4_status launch_read(RdParams &a, cudaStream_t s) {
  const fp4_read_params &p = a.p;
  const bool codes = p.scales.k_sf != nullptr;
  a.pieces = p.cache.head_dim / (codes ? 16 : 8);
  if (2 * (int64_t)p.cache.kv_heads * a.pieces > INT32_MAX / 2) return FP4_ERR_SHAPE;
  const int per = p.cache.kv_heads * a.pieces;  // pieces of a token's keys
  a.tokens = 1;
  while (a.tokens < 32 && kReadThreads / (2 * a.tokens) >= per) a.tokens *= 2;
  a.parts = 2 * (int)ceil_div(per, kReadThreads / a.tokens);
  a.page = divisor(p.cache.page_size);
  a.block = divisor(codes ? p.scales.block : 1);
  a.piece = divisor(a.pieces);
  auto whole32 = [](const void *to, int64_t token, int64_t head) {
    return reinterpret_cast<uintptr_t>(to) % 32 == 0 && token % 16 == 0 && head % 16 == 0;
  };
  a.wide = whole32(p.k_out, p.k_token, p.k_out_head) && whole32(p.v_out, p.v_token, p.v_out_head);
  // as many groups of CTAs as fit, or fewer that have equally many tokens
  const int64_t most = ceil_div(kReaders * (int64_t)sm_count(), a.parts), want = ceil_div(p.tokens, a.tokens);
  const int64_t groups = want ? ceil_div(want, ceil_div(want, most)) : 0;
  const auto kern = codes ? k_read<T, true> : k_read<T, false>;
  return launch_dependent(kern, dim3((unsigned)(groups * a.parts)), dim3(kReadThreads), 0, s, a) == cudaSuccess
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
