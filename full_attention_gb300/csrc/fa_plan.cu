// One step's block tables and slot maps, from the numbers of new tokens
// (fa_plan_step): what a serving loop otherwise builds on the host and copies
// before every step ("FreeToken PR #898", description: tables and slots per
// group of layers; "pegainfer issue #807", Description: the sliding group gives
// pages up that the full group still reads).
//
// Sequence b holds len_b tokens in pages first_b .. ceil(len_b / ps) - 1 of its
// table row; n_b tokens join it.  With
//   have = ceil(len / ps), want = ceil((len + n) / ps), keep = max(first, (len - W + 1)+ / ps)
// its row takes want - have pages off the head of the ring of free pages and its
// pages [first, keep) go behind the ring's end, in order of sequence and page:
// prefix sums over b give every sequence its place in the tokens, the ring's
// head and the ring's end.
//
// One launch.  Every CTA sums over all sequences (12 bytes each, from L2) and
// keeps the sums in shared memory; a warp's run of tokens then finds its
// sequence by bisection, once where it lies in one.  The ring's pops and pushes never meet (they lie count
// apart in a ring that holds every page), so only the state waits until every CTA has
// read it: the last to arrive writes it, and the state read and the one written may be the same.
// 64 sequences of one token 3.2 us, 128 in a window's pool 4.2, 512 prompts (2.1 million
// tokens) 13 us, 1.3 TB/s: of those 6 are the launch, the sums and 17 MB written (2 million rows
// of padding alone take 6.0), the rest the lookups: 126 instructions a token, as each lane looks
// its tokens up alone, at 2.1 instructions a cycle (of 4) between their loads.  More CTAs repeat the
// sums and take longer: 17 us for twice as many.
#include <algorithm>

#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {

constexpr int kPlanThreads = 256;

struct PlanK {
  const int32_t* new_lens;
  const int32_t* state_in;
  int32_t* state_out;   // may be state_in
  int32_t* ring;
  int32_t* table;
  int32_t* qo_indptr;
  int32_t* prefix_lens;
  int32_t* positions;
  int32_t* slots;
  unsigned int* err;
  int B, N, page_size, num_pages, max_pages, window;   // window 0: every page is kept
  int chunk;   // tokens a warp takes, a multiple of 128
  int top;     // the largest power of two below B (0: one sequence)
  FastDiv by_page;
};

// Of sequences before one: new tokens, pages taken, pages given up.  Sums stop at 2^31 - 1,
// more than any step has of each (a step with a sum there is refused).
struct Sums {
  uint32_t tok, need, gone;
};
__device__ __forceinline__ uint32_t add_most(uint32_t a, uint32_t b) { return min(a + b, 0x7fffffffu); }
__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return {add_most(a.tok, b.tok), add_most(a.need, b.need), add_most(a.gone, b.gone)};
}

struct PlanSeq {
  int len, first, n, have, want, keep;
  bool ended;
  unsigned bad;   // FA_DEV_ERR_* bits
};

__device__ __forceinline__ PlanSeq plan_seq(const PlanK& p, int b) {
  PlanSeq s;
  s.len = p.state_in[4 + b];
  s.first = p.state_in[4 + p.B + b];
  const int n = __ldg(p.new_lens + b);
  s.ended = n < 0;
  s.n = max(n, 0);
  s.bad = 0;
  const long long room = static_cast<long long>(p.max_pages) * p.page_size;   // below 2^31
  if (s.len < 0 || s.len > room || s.first < 0) s.bad |= FA_DEV_ERR_WORKSPACE;
  if (static_cast<long long>(s.len) + s.n > room || s.n > p.N) s.bad |= FA_DEV_ERR_BOUND;
  if (s.bad) {
    s.n = s.have = s.want = s.keep = 0;
    return s;
  }
  s.have = static_cast<int>(p.by_page.div(s.len + p.page_size - 1));
  if (s.first > s.have) s.bad |= FA_DEV_ERR_WORKSPACE;
  s.want = s.ended ? s.have : static_cast<int>(p.by_page.div(s.len + s.n + p.page_size - 1));
  s.keep = s.first;
  if (s.ended) s.keep = s.have;
  else if (p.window > 0 && s.len >= p.window) s.keep = max(s.first, static_cast<int>(p.by_page.div(s.len - p.window + 1)));
  return s;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanK p) {
  extern __shared__ int32_t sh[];   // [B + 1] tokens before, [B] pages taken before, [B] given up before, [B] lengths
  int32_t* tok = sh;
  int32_t* need = tok + p.B + 1;
  int32_t* gone = need + p.B;
  int32_t* len = gone + p.B;
  __shared__ Sums warp_sums[kPlanThreads / 32];
  __shared__ unsigned warp_bad[kPlanThreads / 32];
  __shared__ int last;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int head = p.state_in[0], count = p.state_in[1];
  // (the third word counts arrivals where several CTAs change a state in place)
  auto counted = [&] { return p.state_in == p.state_out && gridDim.x > 1; };
  unsigned bad = (p.state_in[3] | (counted() ? 0 : p.state_in[2])) != 0 ? FA_DEV_ERR_WORKSPACE : 0;

  Sums run{0, 0, 0};
  for (int base = 0; base < p.B; base += kPlanThreads) {
    const int b = base + tid;
    Sums mine{0, 0, 0};
    unsigned mybad = 0;
    if (b < p.B) {
      const PlanSeq s = plan_seq(p, b);
      mine = {static_cast<uint32_t>(s.n), static_cast<uint32_t>(s.want - s.have), static_cast<uint32_t>(max(s.keep - s.first, 0))};
      mybad = s.bad;
      len[b] = s.len;
    }
    Sums incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Sums up{__shfl_up_sync(0xffffffffu, incl.tok, o), __shfl_up_sync(0xffffffffu, incl.need, o),
                    __shfl_up_sync(0xffffffffu, incl.gone, o)};
      if (lane >= o) incl = incl + up;
    }
    mybad = __reduce_or_sync(0xffffffffu, mybad);
    if (lane == 31) warp_sums[warp] = incl;
    if (lane == 0) warp_bad[warp] = mybad;
    __syncthreads();
    Sums before = run;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w < warp) before = before + warp_sums[w];
      run = run + warp_sums[w];
      bad |= warp_bad[w];
    }
    if (b < p.B) {   // (a sum that reached 2^31 - 1 is refused below, and these are not used)
      tok[b] = static_cast<int32_t>(before.tok + incl.tok - mine.tok);
      need[b] = static_cast<int32_t>(before.need + incl.need - mine.need);
      gone[b] = static_cast<int32_t>(before.gone + incl.gone - mine.gone);
    }
    __syncthreads();
  }
  if (head < 0 || head >= p.num_pages || count < 0 || count > p.num_pages ||
      static_cast<long long>(count) + run.gone > p.num_pages)
    bad |= FA_DEV_ERR_WORKSPACE;
  if (run.tok > static_cast<uint32_t>(p.N)) bad |= FA_DEV_ERR_BOUND;
  if (count >= 0 && run.need > static_cast<uint32_t>(count)) bad |= FA_DEV_ERR_POOL;
  if (tid == 0) {
    tok[p.B] = static_cast<int32_t>(run.tok);
    if (bad && blockIdx.x == 0) atomicOr(p.err, bad);
  }
  __syncthreads();
  const int total = bad ? 0 : static_cast<int>(run.tok);   // a refused step has no tokens and changes nothing
  auto in_ring = [&](int i) { return i - (i >= 2 * p.num_pages ? 2 * p.num_pages : i >= p.num_pages ? p.num_pages : 0); };

  if (blockIdx.x == 0)
    for (int b = tid; b <= p.B; b += kPlanThreads) {
      p.qo_indptr[b] = bad ? 0 : tok[b];
      if (b < p.B) p.prefix_lens[b] = !bad && __ldg(p.new_lens + b) < 0 ? 0 : len[b];
    }

  // ---- pages given up, behind the ring's end: a warp a sequence
  if (!bad && run.gone > 0) {
    const int warps = gridDim.x * (kPlanThreads / 32);
    for (int b = blockIdx.x * (kPlanThreads / 32) + warp; b < p.B; b += warps) {
      int n = (b + 1 < p.B ? gone[b + 1] : static_cast<int>(run.gone)) - gone[b];
      if (n == 0) continue;
      const int first = p.state_in[4 + p.B + b];
      n = min(n, p.max_pages - first);   // (a state whose third word was not 0 may have been written meanwhile)
      const int32_t* row = p.table + static_cast<size_t>(b) * p.max_pages + first;
      for (int i = lane; i < n; i += 32) p.ring[in_ring(head + count + gone[b] + i)] = row[i];
    }
  }

  // ---- a state changed in place is written, below, by the last CTA to have read it
  __syncthreads();
  if (tid == 0) {
    last = blockIdx.x == 0;
    if (counted()) {
      const int before = atom_add_acq_rel_gpu(p.state_out + 2, 1);
      last = before == static_cast<int>(gridDim.x) - 1;
      if (before < 0 || before >= static_cast<int>(gridDim.x)) atomicOr(p.err, FA_DEV_ERR_WORKSPACE);   // it did not start at 0
    }
  }

  // ---- the tokens: position, slot, and at a new page's first token its table entry.  Where
  // a warp's next 128 tokens lie in one sequence they share its numbers; otherwise
  // each finds its own, a lane's four side by side.
  constexpr int R = 4;   // tokens a lane looks up at once
  const int run_beg = static_cast<int>(min(static_cast<long long>(p.N), (static_cast<long long>(blockIdx.x) * (kPlanThreads / 32) + warp) * p.chunk));
  const int run_end = static_cast<int>(min(static_cast<long long>(p.N), static_cast<long long>(run_beg) + p.chunk));
  int seq = 0;   // a sequence that holds run tokens up to its end
#pragma unroll 1
  for (int t0 = run_beg; t0 < run_end; t0 += 32 * R) {
    const int used = min(run_end, total) - t0;   // of the tokens from t0 on, some sequence's (the others: padding)
    int b[R];
#pragma unroll
    for (int r = 0; r < R; ++r) b[r] = seq;
    if (used > 0 && min(t0 + 32 * R, t0 + used) > tok[seq + 1]) {
      // the last sequence that begins at the token or before (those with no new token end where they begin)
#pragma unroll
      for (int r = 0; r < R; ++r) b[r] = 0;
#pragma unroll 1
      for (int step = p.top; step > 0; step >>= 1)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int next = b[r] + step;
          if (next < p.B && tok[next] <= t0 + lane + 32 * r) b[r] = next;
        }
      seq = __shfl_sync(0xffffffffu, b[R - 1], 31);
    }
    int page[R], pos[R], off[R];
    int32_t* entry[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      entry[r] = nullptr;
      page[r] = -1;
      pos[r] = off[r] = 0;
      if (lane + 32 * r >= used) continue;
      const int l = len[b[r]];
      pos[r] = l + t0 + lane + 32 * r - tok[b[r]];
      const int pi = static_cast<int>(p.by_page.div(pos[r])), have = static_cast<int>(p.by_page.div(l + p.page_size - 1));
      off[r] = pos[r] - pi * p.page_size;
      int32_t* at = p.table + static_cast<size_t>(b[r]) * p.max_pages + pi;
      if (off[r] == 0 && pi >= have) entry[r] = at;
      page[r] = __ldcg(pi < have ? at : p.ring + in_ring(head + need[b[r]] + pi - have));
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int t = t0 + lane + 32 * r;
      if (t >= run_end) break;
      const bool good = page[r] >= 0 && page[r] < p.num_pages;
      if (entry[r]) *entry[r] = page[r];
      p.positions[t] = pos[r];
      p.slots[t] = good ? page[r] * p.page_size + off[r] : -1;   // below 2^31 (fa_cache_create)
      if (!good && lane + 32 * r < used) atomicOr(p.err, FA_DEV_ERR_PAGE);
    }
  }

  // ---- the state
  __syncthreads();
  if (!last) return;
  for (int b = tid; b < p.B; b += kPlanThreads) {
    const int first = p.state_in[4 + p.B + b];
    int l = len[b], f = first;
    if (!bad) {
      const int n = __ldg(p.new_lens + b);
      l = n < 0 ? 0 : l + n;
      f = n < 0 ? 0 : first + (b + 1 < p.B ? gone[b + 1] : static_cast<int>(run.gone)) - gone[b];
    }
    p.state_out[4 + b] = l;
    p.state_out[4 + p.B + b] = f;
  }
  if (tid == 0) {
    p.state_out[0] = bad ? head : in_ring(head + static_cast<int>(run.need));
    p.state_out[1] = bad ? count : count - static_cast<int>(run.need) + static_cast<int>(run.gone);
    p.state_out[2] = 0;   // arrivals
  }
}

cudaError_t launch_plan(const PlanArgs& a, cudaStream_t s) {
  // two CTAs an SM at most, and no less than 128 tokens a warp
  const long long warps = 2LL * sm_count() * (kPlanThreads / 32);
  const long long chunk = std::max(1LL, (a.num_tokens + 128 * warps - 1) / (128 * warps)) * 128;
  const long long per = chunk * (kPlanThreads / 32);
  PlanK k{a.new_lens, a.state_in, a.state_out, a.free_pages, a.block_table, a.qo_indptr, a.prefix_lens, a.positions, a.slots,
          a.err, a.B, a.num_tokens, a.page_size, a.num_pages, a.max_pages_per_seq, a.window, static_cast<int>(chunk), 0, FastDiv(a.page_size)};
  for (int step = 1; step < a.B; step *= 2) k.top = step;
  const int smem = (4 * a.B + 1) * static_cast<int>(sizeof(int32_t));
  static unsigned int done = 0;
  const cudaError_t e = set_smem_once(reinterpret_cast<const void*>(plan_kernel), (4 * FA_MAX_STEP_BATCH + 1) * 4, &done);
  if (e != cudaSuccess) return e;
  return launch_pdl(plan_kernel, dim3(static_cast<unsigned>(std::max(1LL, (a.num_tokens + per - 1) / per))), dim3(kPlanThreads),
                    static_cast<size_t>(smem), s, k);
}

}  // namespace fa
