// plan.cu -- pages and places for new tokens, from what sequences hold and are
// to get (sm_103a): block tables, slot maps, and the pool of free pages.
//
// Bound: latency (a launch, two dependent loads, two scans over the sequences,
// a look-up), and for prompts the 16 bytes written a token.
//
// Layout.  Every CTA scans all sequences, a run of them a thread: the new
// tokens' offsets, then the pages that each gets.  It then writes its share of
// the granted table entries and of the token maps, finding sequences by
// bisection in the threads' sums and a walk within a thread's run.  Page numbers
// of new entries come from the stack, not from the table, so no CTA waits for
// another; the last one to finish (counted in the pool's second word) writes the
// state that the others read: lengths, rooms, the stack and what goes back.
#include "serve.cuh"

namespace fp4 {

namespace {

constexpr int kThreads = 512, kW = kThreads / 32;
constexpr int kTokens = 4;  // consecutive tokens of a thread

struct PlanParams {
  fp4_plan_params p;
  uint32_t *status;
};

// What becomes of sequence s whose new tokens begin at `first` in the maps.
struct Change {
  int64_t length, after;
  int n, held, want;
  bool fits;
  __device__ __forceinline__ int64_t grows() const { return fits && n >= 0 && want > held ? want - held : 0; }
  __device__ __forceinline__ int64_t gives() const { return n < 0 && held > want ? held - want : 0; }
};
__device__ __forceinline__ Change change_of(const fp4_plan_params &p, int s, int64_t first) {
  Change c;
  c.n = p.new_tokens[s];
  c.length = max(p.lengths[s], 0);
  c.held = min(max(p.room[s], 0) / p.page_size, p.seq_pages);
  c.after = max(c.length + c.n, (int64_t)0);
  const int64_t want = (c.after + p.page_size - 1) / p.page_size;
  c.fits = want <= p.seq_pages && (p.tokens < 0 || first + max(c.n, 0) <= p.tokens);
  c.want = (int)min(want, (int64_t)p.seq_pages);
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
  int64_t before = inc - v;
  for (int w = 0; w < warp; ++w) before += warps[w];
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

__global__ void __launch_bounds__(kThreads) k_plan(const __grid_constant__ PlanParams a) {
  __shared__ int64_t add_sh[kThreads + 1], grow_sh[kThreads + 1], give_sh[kThreads + 1], warps[kW];
  __shared__ int last_sh;
  const fp4_plan_params &p = a.p;
  const int per = (p.seqs + kThreads - 1) / kThreads;
  const int s0 = min((int)threadIdx.x * per, p.seqs), s1 = min(s0 + per, p.seqs);
  dependent_wait();
  launch_dependents();
  const int64_t free = min((int64_t)max(p.pool[0], 0), p.pool_pages);
  int64_t add = 0;
  for (int s = s0; s < s1; ++s) add += max(p.new_tokens[s], 0);
  const int64_t add0 = scan(add, add_sh, warps);
  int64_t grow = 0, at = add0;
  for (int s = s0; s < s1; ++s) {
    const Change c = change_of(p, s, at);
    grow += c.grows();
    at += max(c.n, 0);
  }
  const int64_t grow0 = scan(grow, grow_sh, warps);
  // sequence s with `upto` pages granted up to and with it: whether it gets them
  auto granted = [&](const Change &c, int64_t upto) { return c.n < 0 || (c.fits && (c.grows() == 0 || upto <= free)); };

  // table entries: page j of those to be granted
  const int64_t pages = min(grow_sh[kThreads], free);
  const int64_t step = (int64_t)gridDim.x * kThreads, me = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  for (int64_t j = me; j < pages; j += step) {
    const int th = thread_of(grow_sh, j);
    int64_t g = grow_sh[th], t = add_sh[th];
    for (int s = th * per;; ++s) {
      const Change c = change_of(p, s, t);
      if (j < g + c.grows()) {
        if (g + c.grows() <= free) p.table[s * p.table_stride + c.held + (j - g)] = p.pool[2 + free - 1 - j];
        break;
      }
      g += c.grows();
      t += max(c.n, 0);
    }
  }

  // token maps
  const int64_t total = add_sh[kThreads];
  for (int64_t t0 = me * kTokens; t0 < p.tokens; t0 += step * kTokens) {
    int s = -1;
    int64_t begin = 0, end = 0, g = 0;  // the tokens of sequence s; pages granted before it
    Change c{};
    bool ok = false;
    for (int64_t t = t0; t < min(t0 + kTokens, p.tokens); ++t) {
      int seq = -1, pos = -1;
      int64_t slot = -1;
      if (t < total) {
        if (s < 0) {
          const int th = thread_of(add_sh, t);
          s = th * per;
          begin = add_sh[th];
          g = grow_sh[th];
          c = change_of(p, s, begin);
          end = begin + max(c.n, 0);
          ok = granted(c, g + c.grows());
        }
        while (t >= end) {
          g += c.grows();
          begin = end;
          c = change_of(p, ++s, begin);
          end = begin + max(c.n, 0);
          ok = granted(c, g + c.grows());
        }
        seq = s;
        if (ok) {
          pos = (int)(c.length + (t - begin));
          const int e = pos / p.page_size;
          const int page = e < c.held ? p.table[s * p.table_stride + e] : p.pool[2 + free - 1 - (g + e - c.held)];
          slot = (int64_t)page * p.page_size + (pos - e * p.page_size);
        }
      }
      if (p.seq) p.seq[t] = seq;
      if (p.pos) p.pos[t] = pos;
      if (p.slot) p.slot[t] = slot;
    }
  }

  // the last CTA writes the state
  if (gridDim.x > 1) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last_sh = atomicAdd(reinterpret_cast<unsigned *>(p.pool + 1), 1u) == gridDim.x - 1;
    __syncthreads();
    if (!last_sh) return;
    __threadfence();
  } else {
    __syncthreads();
  }
  int64_t give = 0, taken = 0;
  at = add0;
  int64_t g = grow0;
  for (int s = s0; s < s1; ++s) {
    const Change c = change_of(p, s, at);
    g += c.grows();
    if (granted(c, g)) taken = c.grows() ? g : taken;  // the last one granted: pages up to it
    else raise_status(a.status, kStatusIndex);
    give += c.gives();
    at += max(c.n, 0);
  }
  const int64_t give0 = scan(give, give_sh, warps);
  // pages granted: those of the last sequence that got any
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) taken = max(taken, __shfl_xor_sync(~0u, taken, o));
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = taken;
  __syncthreads();
  for (int w = 0; w < kW; ++w) taken = max(taken, warps[w]);
  const int64_t left = free - taken, back = give_sh[kThreads];
  const int64_t fit = min(back, p.pool_pages - left);  // (more than the pool's pages: what is left over is lost)
  for (int64_t j = threadIdx.x; j < back; j += kThreads) {
    const int th = thread_of(give_sh, j);
    int64_t f = give_sh[th];
    for (int s = th * per;; ++s) {
      const Change c = change_of(p, s, 0);
      if (j < f + c.gives()) {
        int32_t *entry = p.table + s * p.table_stride + c.want + (j - f);
        if (back - 1 - j < fit) p.pool[2 + left + (back - 1 - j)] = *entry;
        *entry = -1;
        break;
      }
      f += c.gives();
    }
  }
  __syncthreads();  // lengths and rooms are read above
  at = add0;
  g = grow0;
  for (int s = s0; s < s1; ++s) {
    const Change c = change_of(p, s, at);
    g += c.grows();
    const bool ok = granted(c, g);
    if (p.offsets) p.offsets[s] = (int32_t)min(at, (int64_t)INT32_MAX);
    at += max(c.n, 0);
    if (!ok) continue;
    p.lengths[s] = (int32_t)c.after;
    p.room[s] = (int32_t)((c.n < 0 ? min(c.held, c.want) : c.held + c.grows()) * p.page_size);
  }
  if (threadIdx.x == 0) {
    if (p.offsets) p.offsets[p.seqs] = (int32_t)min(add_sh[kThreads], (int64_t)INT32_MAX);
    if (back > fit) raise_status(a.status, kStatusIndex);
    p.pool[0] = (int32_t)(left + fit);
    p.pool[1] = 0;
  }
}

}  // namespace

fp4_status launch_page_plan(const fp4_plan_params &p, cudaStream_t s) {
  PlanParams a{};
  a.p = p;
  a.status = status_word();
  if (!a.status) return FP4_ERR_CUDA;
  const int64_t want = ceil_div(p.tokens > 0 ? p.tokens : 1, kThreads * kTokens), most = sm_count();
  return launch_dependent(k_plan, dim3((unsigned)(want < most ? want : most)), dim3(kThreads), 0, s, a) == cudaSuccess
             ? FP4_OK
             : FP4_ERR_CUDA;
}

}  // namespace fp4
