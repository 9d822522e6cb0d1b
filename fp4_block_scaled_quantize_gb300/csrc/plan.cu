// plan.cu -- pages and places for new tokens, from what sequences hold and are
// to get (sm_103a): block tables, slot maps, and the pool of free pages.
//
// Bound: latency (a launch, two dependent loads, scans over the sequences, a
// look-up), and for prompts the 16 bytes written a token.
//
// Layout.  Where no sequence gets or loses more than kFew tokens (decoding), one
// CTA scans the sequences and a thread does all of a sequence's work.  Else every
// CTA scans all sequences, a run of them a thread: the new tokens' offsets, the
// pages that each gets, those that each gives back.  It then writes its share of
// the table entries, the token maps and the pages that go back, finding sequences
// by bisection in the threads' sums and a walk within a thread's run (up to 512
// sequences: none, and what is known of them is in shared memory).  Page numbers of
// new entries come from the stack, not from the table, so no CTA waits for another;
// the last one (counted in the pool's second word) writes the state that the others
// read: lengths, rooms, how many are free, and, where the call also gives out pages
// from those places of the stack, what goes back.
// Measured in a graph, two calls, pages given back and taken again: 256 sequences
// by a token 6.8 us (by bisection, with the state written by the last CTA to
// finish, 12.6); 96 prompts of 250000 tokens in all 15.0.  Two empty launches take
// 1.2, with the loads 1.9, with the scans 3.6.
#include "serve.cuh"

namespace fp4 {

namespace {

constexpr int kThreads = 512, kW = kThreads / 32;
constexpr int kTokens = 4;  // consecutive tokens of a thread
// Where no sequence gets or loses more than kFew tokens (and each has a thread),
// its thread does all of its work: no look-ups, and one CTA writes everything but
// the maps' ends.
constexpr int kFew = 4;

struct PlanParams {
  fp4_plan_params p;
  Divisor page;
  int limit;  // positions that a row of the table can name
  int most;   // that a sequence may grow to
  bool wide;  // maps allow stores of whole groups of tokens
  uint32_t *status;
};

// What becomes of a sequence whose new tokens begin at `first` in the maps.
struct Change {
  int n, length, held, want;
  int64_t after;
  bool fits;
  __device__ __forceinline__ int grows() const { return fits && n >= 0 && want > held ? want - held : 0; }
  __device__ __forceinline__ int gives() const { return n < 0 && held > want ? held - want : 0; }
  __device__ __forceinline__ int adds() const { return max(n, 0); }
  // with `upto` pages granted up to and with it, of `free`
  __device__ __forceinline__ bool granted(int64_t upto, int64_t free) const {
    return n < 0 || (fits && (grows() == 0 || upto <= free));
  }
};
__device__ __forceinline__ Change change_of(const PlanParams &a, int n, int length, int held, int64_t first) {
  Change c;
  c.n = n, c.length = length, c.held = held;
  c.after = max((int64_t)length + n, (int64_t)0);
  c.fits = c.after <= (n > 0 ? a.most : a.limit) && (a.p.tokens < 0 || first + max(n, 0) <= a.p.tokens);
  c.want = c.after > a.limit ? a.p.seq_pages : c.after > 0 ? over((int)c.after - 1, a.page) + 1 : 0;
  return c;
}

// Exclusive prefix of v over the threads; the total goes to sums[kThreads],
// each thread's prefix to sums[thread].
__device__ __forceinline__ int64_t scan(int64_t v, int64_t *sums, int64_t *warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(~0u, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) warps[warp] = inc;
  __syncthreads();
  int64_t w = lane < kW ? warps[lane] : 0;
#pragma unroll
  for (int o = 1; o < kW; o <<= 1) {
    const int64_t x = __shfl_up_sync(~0u, w, o);
    if (lane >= o) w += x;
  }
  const int64_t before = inc - v + (warp ? __shfl_sync(~0u, w, warp - 1) : 0);
  sums[threadIdx.x] = before;
  if (threadIdx.x == kThreads - 1) sums[kThreads] = before + v;
  __syncthreads();
  return before;
}
// The thread whose run holds element x < sums[kThreads].
__device__ __forceinline__ int thread_of(const int64_t *sums, int64_t x) {
  int lo = 0, hi = kThreads;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The whole call by one CTA, a thread a sequence.
__device__ __forceinline__ void plan_few(const PlanParams &a, const Change &c, int64_t add0, int64_t total, int64_t free,
                                         int64_t *sums, int64_t *warps, int *taken_sh) {
  const fp4_plan_params &p = a.p;
  const int s = threadIdx.x;
  const bool mine = s < p.seqs;
  const int grows = mine ? c.grows() : 0, gives = mine ? c.gives() : 0;
  const bool back_too = __syncthreads_or(gives > 0);
  const int64_t grow0 = scan(grows, sums, warps);
  const bool ok = mine && c.granted(grow0 + grows, free);
  if (ok && grows) atomicMax(taken_sh, (int)(grow0 + grows));
  const int32_t *const stack = p.pool + 2 + free - 1 - grow0;  // downwards, the pages that the sequence gets
  int32_t *const row = p.table + s * p.table_stride;
  for (int i = 0; ok && i < grows; ++i) row[c.held + i] = stack[-i];
  if (mine && p.tokens >= 0)
#pragma unroll
    for (int i = 0; i < kFew; ++i) {
      const int64_t t = add0 + i;
      if (i >= c.n || t >= p.tokens) break;
      const int pos = c.length + i, e = ok ? over(pos, a.page) : 0;
      if (p.seq) p.seq[t] = s;
      if (p.pos) p.pos[t] = ok ? pos : -1;
      if (p.slot)
        p.slot[t] = ok ? (int64_t)(e < c.held ? row[e] : stack[c.held - e]) * p.page_size + (pos - e * p.page_size) : -1;
    }
  __syncthreads();  // what goes back may lie on places that were read above
  const int64_t taken = *taken_sh, left = free - taken;
  int64_t fit = 0, back = 0;
  if (back_too) {
    const int64_t give0 = scan(gives, sums, warps);
    back = sums[kThreads];
    fit = min(back, p.pool_pages - left);  // (more than the pool's pages: what is left over is lost)
    for (int i = 0; i < gives; ++i) {
      const int64_t at = back - 1 - (give0 + i);
      if (at < fit) p.pool[2 + left + at] = row[c.want + i];
      row[c.want + i] = -1;
    }
  }
  if (mine && p.offsets) p.offsets[s] = (int32_t)min(add0, (int64_t)INT32_MAX);
  if (mine && !ok) raise_status(a.status, kStatusIndex);
  if (ok) {
    p.lengths[s] = (int32_t)c.after;
    p.room[s] = (c.n < 0 ? min(c.held, c.want) : c.held + grows) * p.page_size;
  }
  if (threadIdx.x == 0) {
    if (p.offsets) p.offsets[p.seqs] = (int32_t)min(total, (int64_t)INT32_MAX);
    if (back > fit) raise_status(a.status, kStatusIndex);
    p.pool[0] = (int32_t)(left + fit);
  }
}

__global__ void __launch_bounds__(kThreads) k_plan(const __grid_constant__ PlanParams a) {
  __shared__ int64_t add_sh[kThreads + 1], grow_sh[kThreads + 1], give_sh[kThreads + 1], warps[kW];
  __shared__ int n_sh[kThreads], length_sh[kThreads], held_sh[kThreads], last_sh, taken_sh, free_sh;
  const fp4_plan_params &p = a.p;
  const int per = (p.seqs + kThreads - 1) / kThreads;
  const int s0 = min((int)threadIdx.x * per, p.seqs), s1 = min(s0 + per, p.seqs);
  dependent_wait();
  launch_dependents();
  auto load = [&](int s, int64_t first) {
    return change_of(a, p.new_tokens[s], max(p.lengths[s], 0), min(over(max(p.room[s], 0), a.page), p.seq_pages), first);
  };
  int64_t add = 0;
  bool back_too = false, few = per == 1;
  for (int s = s0; s < s1; ++s) {
    const Change c = load(s, 0);
    if (s == s0) n_sh[threadIdx.x] = c.n, length_sh[threadIdx.x] = c.length, held_sh[threadIdx.x] = c.held;
    add += c.adds();
    back_too |= c.n < 0;
    few &= c.n <= kFew && c.n >= -kFew;
  }
  if (threadIdx.x == 0) {
    taken_sh = 0;
    free_sh = (int)min((int64_t)max(p.pool[0], 0), p.pool_pages);
  }
  // sequence s, the first of thread th's run if there is one a thread
  auto change = [&](int s, int64_t first) {
    return per == 1 ? change_of(a, n_sh[s], length_sh[s], held_sh[s], first) : load(s, first);
  };
  few = __syncthreads_and(few);
  const int64_t add0 = scan(add, add_sh, warps), free = free_sh;
  const int64_t step = (int64_t)gridDim.x * kThreads, me = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (few) {
    const int64_t total = add_sh[kThreads];
    for (int64_t t = total + me; t < p.tokens; t += step) {
      if (p.seq) p.seq[t] = -1;
      if (p.pos) p.pos[t] = -1;
      if (p.slot) p.slot[t] = -1;
    }
    // (the others have read what they go by: nothing but new_tokens)
    if (blockIdx.x == 0) {
      Change c{};
      if (threadIdx.x < p.seqs) c = change(threadIdx.x, add0);
      plan_few(a, c, add0, total, free, grow_sh, warps, &taken_sh);
    }
    return;
  }
  // One thread a sequence: everything that is read of the state has been read, so
  // the CTA that comes last may write it while others still work.
  const bool early = per == 1 && gridDim.x > 1;
  unsigned *const tickets = reinterpret_cast<unsigned *>(p.pool + 1);
  if (early && threadIdx.x == 0) {
    __threadfence();
    last_sh = (atomicAdd(tickets, 1u) & 0xFFFFu) == gridDim.x - 1;
    __threadfence();
  }
  int64_t grow = 0, give = 0, at = add0;
  for (int s = s0; s < s1; ++s) {
    const Change c = change(s, at);
    grow += c.grows();
    give += c.gives();
    at += c.adds();
  }
  const int64_t grow0 = scan(grow, grow_sh, warps);
  back_too = __syncthreads_or(back_too);
  const int64_t give0 = back_too ? scan(give, give_sh, warps) : 0;

  // table entries: page j of those to be granted
  const int64_t pages = min(grow_sh[kThreads], free);
  for (int64_t j = me; j < pages; j += step) {
    const int th = thread_of(grow_sh, j);
    int64_t g = grow_sh[th], t = add_sh[th];
    for (int s = th * per;; ++s) {
      const Change c = change(s, t);
      if (j < g + c.grows()) {
        if (g + c.grows() <= free) p.table[s * p.table_stride + c.held + (j - g)] = p.pool[2 + free - 1 - j];
        break;
      }
      g += c.grows();
      t += c.adds();
    }
  }

  // token maps
  const int64_t total = add_sh[kThreads];
  for (int64_t t0 = me * kTokens; t0 < p.tokens; t0 += step * kTokens) {
    int s = -1, known = -1, page = 0;
    int64_t begin = 0, end = 0, g = 0;  // the tokens of sequence s; pages granted before it
    Change c{};
    bool ok = false;
    int seq[kTokens], pos[kTokens];
    int64_t slot[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      const int64_t t = t0 + i;
      seq[i] = pos[i] = -1;
      slot[i] = -1;
      if (t >= total) continue;
      if (s < 0 || t >= end) {
        if (s < 0) {
          const int th = thread_of(add_sh, t);
          s = th * per;
          begin = add_sh[th];
          g = grow_sh[th];
        } else {
          g += c.grows();
          begin = end;
          ++s;
        }
        c = change(s, begin);
        while (t >= (end = begin + c.adds())) {
          g += c.grows();
          begin = end;
          c = change(++s, begin);
        }
        ok = c.granted(g + c.grows(), free);
        known = -1;
      }
      seq[i] = s;
      if (!ok) continue;
      pos[i] = c.length + (int)(t - begin);
      const int e = over(pos[i], a.page);
      if (e != known) page = e < c.held ? p.table[s * p.table_stride + e] : p.pool[2 + free - 1 - (g + e - c.held)];
      known = e;
      slot[i] = (int64_t)page * p.page_size + (pos[i] - e * p.page_size);
    }
    if (a.wide && t0 + kTokens <= p.tokens) {
      *reinterpret_cast<int4 *>(p.seq + t0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
      *reinterpret_cast<int4 *>(p.pos + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      *reinterpret_cast<longlong2 *>(p.slot + t0) = make_longlong2(slot[0], slot[1]);
      *reinterpret_cast<longlong2 *>(p.slot + t0 + 2) = make_longlong2(slot[2], slot[3]);
      continue;
    }
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      if (t0 + i >= p.tokens) break;
      if (p.seq) p.seq[t0 + i] = seq[i];
      if (p.pos) p.pos[t0 + i] = pos[i];
      if (p.slot) p.slot[t0 + i] = slot[i];
    }
  }

  // how many pages are given out: those up to the last sequence that gets any
  at = add0;
  int64_t g = grow0, taken = 0;
  for (int s = s0; s < s1; ++s) {
    const Change c = change(s, at);
    g += c.grows();
    if (c.grows() && c.granted(g, free)) taken = g;
    at += c.adds();
  }
  if (taken) atomicMax(&taken_sh, (int)taken);
  __syncthreads();
  taken = taken_sh;
  const int64_t left = free - taken, back = back_too ? give_sh[kThreads] : 0;
  const int64_t fit = min(back, p.pool_pages - left);  // (more than the pool's pages: what is left over is lost)
  // pages that go back, as if the last had gone first
  auto give_back = [&](int64_t from, int64_t stride) {
    for (int64_t j = from; j < back; j += stride) {
      const int th = thread_of(give_sh, j);
      int64_t f = give_sh[th];
      for (int s = th * per;; ++s) {
        const Change c = change(s, 0);
        if (j < f + c.gives()) {
          int32_t *entry = p.table + s * p.table_stride + c.want + (j - f);
          if (back - 1 - j < fit) p.pool[2 + left + (back - 1 - j)] = *entry;
          *entry = -1;
          break;
        }
        f += c.gives();
      }
    }
  };
  if (taken == 0) give_back(me, step);  // onto places of the stack that nobody reads

  // the last CTA writes the state: the last to have read it, or, where pages go back
  // onto places of the stack that others read, or the state is read all along, the
  // last to come here
  if (gridDim.x > 1 && (!early || (taken != 0 && back != 0))) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last_sh = atomicAdd(tickets, 1u << 16) >> 16 == gridDim.x - 1;
    __syncthreads();
    if (!last_sh) return;
    __threadfence();
  } else {
    __syncthreads();
    if (early && !last_sh) return;
  }
  if (taken != 0) {
    give_back(threadIdx.x, kThreads);
    if (per > 1) __syncthreads();  // lengths and rooms are read there
  }
  at = add0;
  g = grow0;
  for (int s = s0; s < s1; ++s) {
    const Change c = change(s, at);
    g += c.grows();
    if (p.offsets) p.offsets[s] = (int32_t)min(at, (int64_t)INT32_MAX);
    at += c.adds();
    if (!c.granted(g, free)) {
      raise_status(a.status, kStatusIndex);
      continue;
    }
    p.lengths[s] = (int32_t)c.after;
    p.room[s] = (c.n < 0 ? min(c.held, c.want) : c.held + c.grows()) * p.page_size;
  }
  if (threadIdx.x == 0) {
    if (p.offsets) p.offsets[p.seqs] = (int32_t)min(add_sh[kThreads], (int64_t)INT32_MAX);
    if (back > fit) raise_status(a.status, kStatusIndex);
    p.pool[0] = (int32_t)(left + fit);
    p.pool[1] = 0;
  }
}

}  // namespace

fp4_status launch_page_plan(const fp4_plan_params &p, int64_t max_len, cudaStream_t s) {
  PlanParams a{};
  a.p = p;
  a.page = divisor(p.page_size);
  a.limit = p.seq_pages * p.page_size;
  a.most = max_len < a.limit ? (int)max_len : a.limit;
  a.wide = p.seq && p.pos && p.slot && aligned16(p.seq) && aligned16(p.pos) && aligned16(p.slot);
  a.status = status_word();
  if (!a.status) return FP4_ERR_CUDA;
  // CTAs for the tokens, or for pages that may go back
  const int64_t tokens = ceil_div(p.tokens > 0 ? p.tokens : 1, kThreads * kTokens);
  const int64_t pages = ceil_div(p.pool_pages, 4 * kThreads);
  const int64_t want = p.tokens >= 0 ? tokens : pages < 16 ? (pages > 1 ? pages : 1) : 16, most = sm_count();
  return launch_dependent(k_plan, dim3((unsigned)(want < most ? want : most)), dim3(kThreads), 0, s, a) == cudaSuccess
             ? FP4_OK
             : FP4_ERR_CUDA;
}

}  // namespace fp4
