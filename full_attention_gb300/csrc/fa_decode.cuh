// What the decode kernels share: their parameters, the work list of units and
// its cut into CTA shares, the current token's store, and empty sequences.
#pragma once
#include <climits>

#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_row.cuh"

namespace fa {

struct DecK {
  const __nv_bfloat16* q;
  const int32_t* block_table;
  const int32_t* seq_lens;
  uint8_t* kb;    // slab bases and int8 scales (L2 prefetch, the current token's store)
  uint8_t* vb;
  float* ksb;
  float* vsb;
  const __nv_bfloat16* k_new;   // current token's rows [B][Hkv][D] and their slots, stored by
  const __nv_bfloat16* v_new;   // the CTA that reads the unit's last tile (null: no store)
  const int32_t* slots;
  __nv_bfloat16* out;
  float* lse;
  int* counters;    // arrivals, indexed by share: a unit's by the second of its shares, the first that
                    // begins inside it (fp4: see merge_tree); zero between calls; null: one CTA
  float* ml_part;   // [(ncta + U) * 8][2] (fp4: [4])
  float* o_part;    // [(ncta + U) * 8][D]
  unsigned int* err;
  int B, Hq, Hkv, g, chunks, kind, window, page_size, tiles_per_page, num_pages, max_pages_per_seq;
  int max_seq_len, units, min_tiles, early_metadata;
  int shares;         // fp4: shares the work may be cut into
  float scale_log2;   // sm_scale * log2(e)
};

struct Unit {
  int b, h, c, L, lo, t_first, n;
};

__device__ __forceinline__ Unit unit_of(const DecK& p, int u) {
  Unit x;
  x.b = u / (p.Hkv * p.chunks);
  const int r = u % (p.Hkv * p.chunks);
  x.h = r / p.chunks;
  x.c = r % p.chunks;
  const int L = __ldg(p.seq_lens + x.b);
  x.L = min(L, p.max_seq_len);
  if (x.L <= 0) {
    x.lo = x.t_first = x.n = 0;
    return x;
  }
  x.lo = (p.kind == FA_SLIDING) ? max(0, x.L - p.window) : 0;
  x.t_first = x.lo / kTile;
  x.n = (x.L - 1) / kTile + 1 - x.t_first;
  return x;
}

// CTA that owns global tile g when T tiles are split evenly over n CTAs.
__device__ __forceinline__ int cta_of(long long g, int n, long long T) {
  return static_cast<int>(((g + 1) * n - 1) / T);
}

// Exclusive block scan over all threads of the block; *total gets the sum.
__device__ __forceinline__ int block_excl_scan(int v, int* sm, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) sm[warp] = incl;
  __syncthreads();
  int base = 0, tot = 0;
  for (int w = 0; w < nw; ++w) {
    if (w < warp) base += sm[w];
    tot += sm[w];
  }
  __syncthreads();
  *total = tot;
  return base + incl - v;
}

// Block-wide (min, max) of one value per thread; sm holds 2 ints per warp.
__device__ __forceinline__ int2 block_min_max(int mn, int mx, int* sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    mn = min(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  if (lane == 0) {
    sm[2 * warp] = mn;
    sm[2 * warp + 1] = mx;
  }
  __syncthreads();
  int a = sm[0], b = sm[1];
  for (int w = 1; w < nw; ++w) {
    a = min(a, sm[2 * w]);
    b = max(b, sm[2 * w + 1]);
  }
  __syncthreads();
  return make_int2(a, b);
}

// One CTA's share of the concatenated tile lists: tiles [s_beg, s_end) of the T,
// starting in unit u0, whose first tile is p0.
struct Share {
  long long s_beg, s_end;
  int T, ncta, kper;   // kper: CTAs per unit of the unit-aligned cut (0: concatenated cut)
  int u0, p0;
};
struct ShareWork {   // shared memory of the cut
  int scan[8], mm[16];
  int u0, p0, n0;
};
__device__ __forceinline__ ShareWork& share_work() {
  __shared__ ShareWork w;
  return w;
}

// Cut the work into CTA shares.  Run by the whole block; false: no share for
// this CTA (s.ncta says how many CTAs have one).  After it returns true the
// block synchronises, then calls finish_share.
__device__ __forceinline__ bool cut_share(const DecK& p, int cta, int grid, Share& s) {
  ShareWork& w = share_work();
  int* sm_scan = w.scan;
  int* sm_mm = w.mm;
  // One block scan gives every unit's first global tile P_u and the total T.
  // Two ways to cut the tile lists into CTA shares:
  //  * unit-aligned: when every unit has about the same number of tiles (the
  //    sliding layers once L >= W), each unit is cut into kper equal parts,
  //    one CTA each, so no CTA crosses a unit boundary and every merge has
  //    exactly kper partials;
  //  * concatenated: otherwise the lists are laid end to end and cut into
  //    ncta equal shares, so every CTA moves the same bytes whatever the
  //    length mix.
  int T = 0, my_n = 0, my_P = 0;
  {
    int running = 0;
    for (int base = 0; base < p.units; base += blockDim.x) {
      const int u = base + threadIdx.x;
      Unit x{};
      if (u < p.units) {
        x = unit_of(p, u);
        if (cta == 0 && __ldg(p.seq_lens + x.b) > p.max_seq_len) atomicOr(p.err, FA_DEV_ERR_BOUND);
      }
      int tot;
      const int P = running + block_excl_scan(x.n, sm_scan, &tot);
      if (base == 0) {
        my_n = x.n;
        my_P = P;
      }
      running += tot;
    }
    T = running;
  }
  int ncta = (T == 0) ? 0 : min(grid, max(1, (T + p.min_tiles - 1) / p.min_tiles));
  int kper = 0;   // CTAs per unit of the unit-aligned cut (0: concatenated cut)
  if (ncta > 0 && p.units <= static_cast<int>(blockDim.x)) {
    const bool mine = static_cast<int>(threadIdx.x) < p.units;
    const int2 r = block_min_max(mine ? my_n : INT_MAX, mine ? my_n : 0, sm_mm);
    if (r.x >= 1 && r.y - r.x <= max(1, r.x >> 3)) {
      const int k = min(ncta / p.units, r.x);
      // take it only if it keeps at least 85% of the concatenated cut's CTAs
      if (k >= 1 && 20 * k * p.units >= 17 * ncta) {
        kper = k;
        ncta = k * p.units;
      }
    }
  }
  s.T = T;
  s.ncta = ncta;
  s.kper = kper;
  if (cta >= ncta) return false;
  const long long s_beg = static_cast<long long>(cta) * T / ncta;
  s.s_beg = s_beg;
  s.s_end = static_cast<long long>(cta + 1) * T / ncta;
  if (kper) {
    if (static_cast<int>(threadIdx.x) == cta / kper) {
      w.u0 = threadIdx.x;
      w.p0 = my_P;
      w.n0 = my_n;
    }
  } else if (p.units <= static_cast<int>(blockDim.x)) {
    if (my_n > 0 && my_P <= s_beg && s_beg < my_P + my_n) {
      w.u0 = threadIdx.x;
      w.p0 = my_P;
    }
  } else {
    int running = 0;
    for (int base = 0; base < p.units; base += blockDim.x) {
      const int u = base + threadIdx.x;
      const int n = (u < p.units) ? unit_of(p, u).n : 0;
      int tot;
      const int P = running + block_excl_scan(n, sm_scan, &tot);
      if (n > 0 && P <= s_beg && s_beg < P + n) {
        w.u0 = u;
        w.p0 = P;
      }
      running += tot;
    }
  }
  return true;
}

__device__ __forceinline__ void finish_share(int cta, Share& s) {
  const ShareWork& w = share_work();
  s.u0 = w.u0;
  s.p0 = w.p0;
  if (s.kper) {   // part r of unit u0
    const int r = cta % s.kper;
    s.s_beg = s.p0 + static_cast<long long>(r) * w.n0 / s.kper;
    s.s_end = s.p0 + static_cast<long long>(r + 1) * w.n0 / s.kper;
  }
}

// The current token's K and V rows of (sequence b, KV head h) into slot `slot`
// (one warp; slot < 0 skips, a slot past the pool is reported).
template <int D, int KV>
__device__ __forceinline__ void store_current(const DecK& p, const RowRegs<D>& rk, const RowRegs<D>& rv, int h,
                                              int slot, int lane) {
  if (slot < 0) return;
  const int page = slot / p.page_size, off = slot % p.page_size;
  if (page >= p.num_pages) {
    if (lane == 0) atomicOr(p.err, FA_DEV_ERR_SLOT);
    return;
  }
  const size_t row = (static_cast<size_t>(page) * p.Hkv + h) * p.page_size + off;
  constexpr size_t rb = kRowBytes<D, KV>;
  row_store<D, KV>(rk, p.kb + row * rb, KV == FA_KV_BF16 ? nullptr : p.ksb + row, lane);
  row_store<D, KV>(rv, p.vb + row * rb, KV == FA_KV_BF16 ? nullptr : p.vsb + row, lane);
}

// Sequences of length <= 0 get out = 0 and lse = -inf; CTA `cta` of `ncta`
// writes the units u with u % ncta == cta.
template <int D, int KV>
__device__ void zero_empty_units(const DecK& p, int cta, int ncta, int tid, int nthr) {
  for (int u = cta; u < p.units; u += ncta) {
    const Unit x = unit_of(p, u);
    if (x.L > 0) continue;
    if (p.slots && x.c == 0 && tid < 32) {   // nothing to attend, but the row is still stored
      RowRegs<D> rk, rv;
      const size_t src = (static_cast<size_t>(x.b) * p.Hkv + x.h) * D;
      row_load<D>(rk, p.k_new + src, tid);
      row_load<D>(rv, p.v_new + src, tid);
      store_current<D, KV>(p, rk, rv, x.h, __ldg(p.slots + x.b), tid);
    }
    const int nh = min(8, p.g - x.c * 8), head0 = x.h * p.g + x.c * 8;
    for (int i = tid; i < nh * D; i += nthr)
      p.out[(static_cast<size_t>(x.b) * p.Hq + head0 + i / D) * D + i % D] = __float2bfloat16(0.0f);
    if (p.lse && tid < nh) p.lse[static_cast<size_t>(x.b) * p.Hq + head0 + tid] = -INFINITY;
  }
}

// The kernel parameters of one layer's decode.
inline DecK make_deck(const DecodeArgs& a) {
  DecK k{};
  k.q = static_cast<const __nv_bfloat16*>(a.q);
  k.block_table = a.block_table;
  k.seq_lens = a.seq_lens;
  k.kb = static_cast<uint8_t*>(const_cast<void*>(a.k));
  k.vb = static_cast<uint8_t*>(const_cast<void*>(a.v));
  k.ksb = const_cast<float*>(a.k_scale);
  k.vsb = const_cast<float*>(a.v_scale);
  k.k_new = static_cast<const __nv_bfloat16*>(a.k_new);
  k.v_new = static_cast<const __nv_bfloat16*>(a.v_new);
  k.slots = a.slots;
  k.out = static_cast<__nv_bfloat16*>(a.out);
  k.lse = a.lse;
  if (a.partials) {
    k.counters = a.counters;
    k.ml_part = static_cast<float*>(a.partials);
    k.o_part = reinterpret_cast<float*>(static_cast<char*>(a.partials) + a.plan.off_o);
  }
  k.err = a.err;
  k.B = a.B;
  k.Hq = a.Hq;
  k.Hkv = a.Hkv;
  k.g = a.Hq / a.Hkv;
  k.chunks = a.plan.head_chunks;
  k.kind = a.kind;
  k.window = a.window;
  k.page_size = a.page_size;
  k.tiles_per_page = a.page_size / kTile;
  k.num_pages = a.num_pages;
  k.max_pages_per_seq = a.max_pages_per_seq;
  k.max_seq_len = a.max_seq_len;
  k.units = a.plan.units;
  k.min_tiles = a.plan.min_tiles;
  k.early_metadata = a.early_metadata;
  k.shares = a.plan.ncta;
  k.scale_log2 = a.sm_scale * 1.4426950408889634f;
  return k;
}

}  // namespace fa
