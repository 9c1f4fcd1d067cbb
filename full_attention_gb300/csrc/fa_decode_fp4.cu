// Paged decode attention over microscaled 4-bit slabs (FA_KV_FP4).
//
// Per unit (sequence, KV head, chunk of up to 8 query heads) with visible rows
// j, in the log2 domain:
//   s_j = sm_scale log2(e) * ks_j * (q . kc_j),      kc_j = code * block scale
//   o   = sum_j 2^(s_j + e_j - M) vc_j * 2^M / L,    L = sum_j 2^(s_j - m) * 2^m
// where ks_j and 2^e_j are the rows' fp32 scales (powers of two) and kc, vc are
// exact f16 numbers.  The base M tracks the largest s_j + e_j, not the largest
// score, so a row whose values are tiny against its neighbours' cannot push
// their weights out of f16's range, nor an all-zero V row (e = -116) under a
// sink token's weight; L keeps a base of its own.
//
// What bounds it: a row is 148 bytes at head_dim 256 and 292 at 512, but every
// pair of codes passes through one e2m1 -> f16 conversion and one f16 product
// with its block's scale before a matrix instruction can take it: 2 cycles of a
// scheduler each for a warp's 64 codes, side by side on two pipes, and the matrix
// instructions (8.5 cycles) do not run beside them.  Measured with the loads left
// out, long sequences took 98% of their time: 8 sequences of 32k to 131k keys at
// 512 take 85 us, 5.0 TB/s of 6.8; 64 of 512 to 4096 keys 28 us, 128 windows of
// 1024 at 256 18 us, where the start (3 us to the first copy, 2 more until it
// lands) and the joining of the parts (1 to 5 us) weigh as much.
//
// Work decomposition: one CTA per SM of three groups, each with a share of the
// tile lists and shared memory, barriers and five warps of its own.  (Three CTAs
// of one group on an SM read as fast, but joined their partials through memory:
// 95.5, 31.4 and 22.6 us for the above.)  A step is 128 keys at 256, 64 at 512
// (64 at 256 as well: 18.6 us for the windows):
//   warp 4      producer: finds the share; per step one bulk copy per 16-row tile
//               of K and of V (a tile's rows are contiguous) and of their row
//               scales, into a ring of three slots, K and V alternating;
//   warps 0-3   S^T = K Q^T, each warp two tiles or one over the full head_dim
//               (keys on the MMA's M side, the 8 heads on N), the softmax weights
//               of its tiles against O's base, or a base of their own where they
//               exceed that by more than the slack, into shared memory as f16;
//               barrier; then O^T += V^T P^T, each warp a quarter of the columns.
// The weights' rounding to f16 is the only one below 32 bits: 2^-11 relative
// each, and below 2^-14 steps of 2^-24, while the largest lies between 2^3 and
// 2^12 (P_OFF, SLACK): a key whose weight times value scale is 2^-17 of the
// largest or less loses bits, together at most 2^-28 of the largest a key.  The
// sum of the weights, in fp32, takes them unrounded.
//
// Rows are 144 or 288 bytes apart in shared memory, so the fragment loads (one
// 4-byte word of 8 codes a lane at 256, 8 bytes at 512) hit 32 different banks
// without any swizzle; at 512 the MMA's key index r stands for tile row
// key_row(r) to that end.  The MMA contraction over head_dim may run in any
// order, so a lane's codes are taken in the order they are stored, and Q
// likewise (as f16, whose 11 bits hold bf16's 8; past f16's range it is reported).
#include "fa_decode.cuh"

namespace fa {

template <int D>
struct F4Cfg {
  static constexpr int NW = D / 256;                   // words of 8 codes a lane loads at a time
  static constexpr int ROWB = kRowBytes<D, FA_KV_FP4>; // 144, 288
  static constexpr int TILE_BYTES = kTile * ROWB;
  static constexpr int NCW = 4;                        // consumer warps
  static constexpr int TPW = D == 256 ? 2 : 1;         // tiles of a step whose scores a warp works out
  static constexpr int NT = TPW * NCW;                 // tiles per step
  static constexpr int SC_BYTES = NT * kTile * 4;      // one step's K (or V) row scales
  static constexpr int SLOT = NT * TILE_BYTES + 2 * SC_BYTES;   // rows; in K slots also both row scales
  static constexpr int NSLOT = 3;
  static constexpr int GROUPS = 3;                     // shares a CTA works on side by side
  static constexpr int GTHR = (NCW + 1) * 32;          // threads of a group
  static constexpr int NTHR = GROUPS * GTHR;
  static constexpr int JOIN = D == 256 ? 48 : 24;      // tiles a share reads in the time that joining parts takes it
  static constexpr int NJ = 8;                         // loads of NW words a lane makes per row
  static constexpr int MT = D / 4 / 16;                // m16 tiles of O^T per warp
  static constexpr int P_HEAD = 48;                    // bytes per head of a tile's weights (16 f16 + padding)
  static constexpr int P_TILE = 8 * P_HEAD;
  static constexpr int OFF_Q = NSLOT * SLOT;           // Q^T fragments [NJ][NW][32 lanes] of 16 bytes
  static constexpr int OFF_P = OFF_Q + 8 * D * 2;      // [2][NT] tiles of weights
  static constexpr int OFF_MW = OFF_P + 2 * NT * P_TILE;   // [2][8 heads][NCW] bases of a warp's tiles
  static constexpr int OFF_FLAG = OFF_MW + 2 * 8 * NCW * 4; // [2][NCW] they are the warp's own
  static constexpr int OFF_ML = OFF_FLAG + 2 * NCW * 4;    // [NCW][8] (m, l)
  static constexpr int OFF_BAR = OFF_ML + NCW * 8 * 8;
  static constexpr int GSMEM = (OFF_BAR + (2 * NSLOT + 1) * 8 + 127) / 128 * 128;   // a group's
  static constexpr int SMEM = GROUPS * GSMEM;
  static_assert(SLOT % 128 == 0, "slot alignment");
  static constexpr int R = D == 256 ? 6 : 5;           // partials merged at a time
  static_assert(OFF_MW >= (R - 1) * 8 * D * 4, "the ring, Q and weights hold the others");
  static_assert(SMEM + 256 <= 227 * 1024, "shared memory");
};

// "No score yet": finite, so that differences against it are never NaN.
constexpr float kNoScore = -3.402823466e38f;
// O's base is an integer, so that sums with it and the values' exponents are
// exact: up to this magnitude (a larger one is reported).
constexpr float kMaxBase = 8388608.0f;   // 2^23

// What runs once or rarely in a launch stays out of line: all of the code has to
// come through the instruction cache, which short launches wait for.
static __device__ __noinline__ int3 unit_place(int Hkv, int chunks, int u) {   // (sequence, KV head, chunk)
  const uint32_t b = static_cast<uint32_t>(u) / (Hkv * chunks), r = u - b * (Hkv * chunks), h = r / chunks;
  return make_int3(b, h, r - h * chunks);
}
static __device__ __noinline__ uint32_t div_u32(uint32_t n, uint32_t d) { return n / d; }

__device__ __forceinline__ Unit unit_at(const DecK& p, int u) {
  Unit x;
  x.b = u;
  x.h = x.c = 0;
  if (p.Hkv * p.chunks != 1) {
    const int3 at = unit_place(p.Hkv, p.chunks, u);
    x.b = at.x;
    x.h = at.y;
    x.c = at.z;
  }
  x.L = min(__ldg(p.seq_lens + x.b), p.max_seq_len);
  x.lo = (p.kind == FA_SLIDING) ? max(0, x.L - p.window) : 0;
  x.t_first = x.lo / kTile;
  x.n = x.L > 0 ? (x.L - 1) / kTile + 1 - x.t_first : 0;
  return x;
}

// Tile row that MMA key index r stands for.  Rows 288 bytes apart start 8 banks
// apart, so a half-warp's 8-byte loads are free of conflicts when its four rows
// differ modulo 4: for S those of r = 0..3 (and 4..7), for PV those of r = 0, 2,
// 4, 6 (and 1, 3, 5, 7).
template <int D>
__device__ __forceinline__ int key_row(int r) {
  if constexpr (D == 256) return r;
  else return (r & 8) | ((r & 1) ? 4 | (((r >> 1) & 3) ^ 2) : (r >> 1) & 3);
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, __half2 b) {
  const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&a), b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The f16 block scales of the lane's words j = 2 i (low half) and 2 i + 1 (high
// half) of a row whose block scales start at sc.
template <int D>
__device__ __forceinline__ __half2 block_scales(const uint8_t* sc, int i, int tig) {
  uint32_t two;
  if constexpr (D == 256) {   // words 4 j + tig: block 2 j + tig / 2
    const uint32_t h = tig >> 1;
    two = __byte_perm(*reinterpret_cast<const uint32_t*>(sc + 4 * i), 0, h | ((2 + h) << 4));
  } else {                    // words 8 j + 2 tig, + 1: block 4 j + tig
    const uint2 w = *reinterpret_cast<const uint2*>(sc + 8 * i);
    two = __byte_perm(w.x, w.y, tig | ((4 + tig) << 4));
  }
  const uint32_t h = e4m3x2_to_f16x2(two & 0xffffu);
  return *reinterpret_cast<const __half2*>(&h);
}

template <int N>
__device__ __forceinline__ void lds_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    w[0] = x.x;
    w[1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(p + 4 * i);
      w[i] = x.x;
      w[i + 1] = x.y;
      w[i + 2] = x.z;
      w[i + 3] = x.w;
    }
  }
}

// floor(c * T / n) for c <= n, in 32 bits: with T = q n + r it is c q + floor(c r / n).
__device__ __forceinline__ uint32_t share_begin(uint32_t c, uint32_t n, uint32_t q, uint32_t r) {
  return c * q + (r ? c * r / n : 0u);
}

// One group's share of the concatenated tile lists: tiles [s_beg, s_end) of the
// T, starting in unit u0, whose first tile is p0.
struct F4Share {
  int s_beg, s_end, T, u0, p0;
  int n, i, nb;        // shares in use, this one, CTAs in use
  int sb, se;          // the CTA's shares
  int cf, nct;         // the whole-unit cut: the unit's first share and its shares (nct 0: laid end to end)
  int u_end;           // where units are not split: the end of the share's units; else of all
  bool unsplit;
};

// The cut, found by one warp from shuffles: one round of loads up to 32
// sequences, and 32-bit divisions only (a 64-bit one costs some 0.3 us on the
// way to the first copy).  Where it can, it gives every
// share a part of one unit only: unit u is cut into ceil(n_u / Q) equal parts, Q
// the smallest quota found for which the launch's shares suffice.  A share that
// crosses from one unit to the next pays a second query load, epilogue and merge
// in the middle of its stream, which costs more than the uneven parts as long as
// Q stays below 3/2 of the even share; past that (many units, few shares for
// each) all lists are laid end to end and cut evenly; but where there are more
// units than shares and a share's units together are not much longer than the even
// share, units are dealt out unsplit: parts of units that lie across two shares
// cost both about what JOIN tiles do.  (Cut evenly against unsplit, us: 255
// sequences of 4 to 34 keys, 10 heads at 512 19.4 : 11.7; 8 KV heads, 128 sequences
// of 200 to 256 keys at 512 49.0 : 41.7; at 256 of 1 to 64 keys 27.8 : 15.5, 256
// sequences of 128 to 256 keys 59.4 : 45.8.)  The shares go to the CTAs evenly, in
// order.  False: nothing to do for this group; s.n is set all the same.
//
// A sequence's units (KV head x chunk) are all alike, so a lane looks at
// sequences only.  Past 128 of them the loops stay rolled and read the lengths
// again (from L1): the whole kernel has to come through the instruction cache
// once per launch, and unrolled copies cost short launches more than the loads.
template <int JOIN>
__device__ __forceinline__ bool cut_share_warp(const DecK& p, int cta, int nblk, int group, F4Share& s) {
  const int lane = threadIdx.x & 31;
  const int per = (p.B + 31) / 32;       // sequences of a lane: [lane * per, ...)
  const int hc = p.Hkv * p.chunks;       // units of a sequence
  bool past = false;
  auto tiles = [&](int i) {              // of each unit of the lane's sequence i
    const int b = lane * per + i;
    int len = b < p.B ? __ldg(p.seq_lens + b) : 0;
    past |= len > p.max_seq_len;
    len = min(len, p.max_seq_len);
    if (len <= 0) return 0;
    const uint32_t lo = p.kind == FA_SLIDING ? max(0, len - p.window) : 0;
    return static_cast<int>(static_cast<uint32_t>(len - 1) / kTile + 1 - lo / kTile);
  };
  auto scan = [&](int v) {               // inclusive, over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += t;
    }
    return v;
  };
  int n4[4];                             // the first four stay in registers
#pragma unroll
  for (int i = 0; i < 4; ++i) n4[i] = i < per ? tiles(i) : 0;
  int sum = n4[0] + n4[1] + n4[2] + n4[3], most_n = max(max(n4[0], n4[1]), max(n4[2], n4[3])), some = (n4[0] > 0) + (n4[1] > 0) + (n4[2] > 0) + (n4[3] > 0);
#pragma unroll 1
  for (int i = 4; i < per; ++i) {
    const int n = tiles(i);
    sum += n;
    most_n = max(most_n, n);
    some += n > 0;
  }
  if (past && cta == 0 && group == 0) atomicOr(p.err, FA_DEV_ERR_BOUND);
  sum *= hc;
  const int incl = scan(sum);
  const int T = __shfl_sync(0xffffffffu, incl, 31);
  s.T = T;
  s.nct = s.cf = s.n = 0;
  s.u_end = p.units;
  if (T == 0) return false;
  const int grid = p.shares;
  const uint32_t even = max((static_cast<uint32_t>(T) + grid - 1) / grid, static_cast<uint32_t>(p.min_tiles));
  int ks = 0, total = __reduce_add_sync(0xffffffffu, some * hc);
  const bool few = total <= grid;        // else no whole-unit cut: there are more units than shares
  most_n = __reduce_max_sync(0xffffffffu, most_n);
  s.unsplit = !few && (p.units + grid - 1) / grid * most_n <= T / grid + JOIN;
  uint32_t Q = even;
  float rq;
  auto parts = [&](int n) {              // ceil(n / Q): the fp32 estimate is put right by one either way
    const int m = n + static_cast<int>(Q) - 1;
    int c = static_cast<int>(static_cast<float>(m) * rq);
    c -= c * static_cast<int>(Q) > m;
    c += (c + 1) * static_cast<int>(Q) <= m;
    return c;
  };
  while (few) {
    rq = __frcp_rn(static_cast<float>(Q));
    ks = parts(n4[0]) + parts(n4[1]) + parts(n4[2]) + parts(n4[3]);
#pragma unroll 1
    for (int i = 4; i < per; ++i) ks += parts(tiles(i));
    ks *= hc;
    total = __reduce_add_sync(0xffffffffu, ks);
    if (total <= grid || 2 * Q >= 3 * even) break;
    // in proportion, as far as the fractions of a part allow
    Q = max(Q + 1, static_cast<uint32_t>(static_cast<float>(Q) * total / grid));
  }
  const bool whole = total <= grid;
  const int ncta = whole ? total : min(grid, T);
  s.n = ncta;
  // as few CTAs as the fullest one allows: fewer units lie across two of them
  const uint32_t most = (static_cast<uint32_t>(ncta) + nblk - 1) / nblk;
  const uint32_t nb = s.nb = (ncta + most - 1) / most, bq = static_cast<uint32_t>(ncta) / nb, br = ncta - bq * nb;
  if (cta >= s.nb) return false;
  s.sb = share_begin(cta, nb, bq, br);
  s.se = share_begin(cta + 1, nb, bq, br);
  const int me = s.i = s.sb + group;
  if (me >= s.se) return false;
  if (s.unsplit) {
    const uint32_t q = static_cast<uint32_t>(p.units) / ncta, r = p.units - q * ncta;
    s.u0 = share_begin(me, ncta, q, r);
    s.u_end = share_begin(me + 1, ncta, q, r);
    s.p0 = s.s_beg = 0;
    s.s_end = INT_MAX;
    return true;
  }
  const uint32_t q = static_cast<uint32_t>(T) / ncta, r = T - q * ncta;
  const int s_beg = share_begin(me, ncta, q, r);
  int b0 = -1, p0 = 0, un = 0, k0 = 0, c0 = 0, P = incl - sum, K = scan(ks) - ks;
  auto look = [&](int i, int n) {
    const int k = whole ? parts(n) : 0;
    if (whole ? K <= me && me < K + k * hc : P <= s_beg && s_beg < P + n * hc) {
      b0 = lane * per + i;
      p0 = P;
      un = n;
      k0 = k;
      c0 = K;
    }
    P += n * hc;
    K += k * hc;
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) look(i, n4[i]);
#pragma unroll 1
  for (int i = 4; i < per; ++i) look(i, tiles(i));
  const int src = __ffs(__ballot_sync(0xffffffffu, b0 >= 0)) - 1;
  b0 = __shfl_sync(0xffffffffu, b0, src);
  p0 = __shfl_sync(0xffffffffu, p0, src);
  un = __shfl_sync(0xffffffffu, un, src);
  if (whole) {
    c0 = __shfl_sync(0xffffffffu, c0, src);
    k0 = __shfl_sync(0xffffffffu, k0, src);
    const int j = static_cast<uint32_t>(me - c0) / static_cast<uint32_t>(k0);   // unit in the sequence
    s.u0 = b0 * hc + j;
    s.p0 = p0 + j * un;
    s.cf = c0 + j * k0;
    s.nct = k0;
    const uint32_t i = me - s.cf, uq = static_cast<uint32_t>(un) / k0, ur = un - uq * k0;
    s.s_beg = s.p0 + share_begin(i, k0, uq, ur);
    s.s_end = s.p0 + share_begin(i + 1, k0, uq, ur);
  } else {
    const int j = static_cast<uint32_t>(s_beg - p0) / static_cast<uint32_t>(un);
    s.u0 = b0 * hc + j;
    s.p0 = p0 + j * un;
    s.s_beg = s_beg;
    s.s_end = share_begin(me + 1, ncta, q, r);
  }
  return true;
}

// The part that owns item g of T cut over n: cta_of without its 64-bit division.
// The quotient is estimated in fp32 and put right against share_begin.
static __device__ __noinline__ int part_of(uint32_t g, uint32_t n, uint32_t T) {
  const uint32_t q = T / n, r = T - q * n;
  int c = static_cast<int>(__fdividef(static_cast<float>(g) * static_cast<float>(n), static_cast<float>(T)));
  c = max(0, min(c, static_cast<int>(n) - 1));
  while (c > 0 && share_begin(c, n, q, r) > g) --c;
  while (c + 1 < static_cast<int>(n) && share_begin(c + 1, n, q, r) <= g) ++c;
  return c;
}

// ((0 + 1) + (2 + 3)) + (4 + 5) by index of R terms given by the part played in
// merge_tree (mp: this one's pair); the sums of two are the same either way round.
__device__ __forceinline__ float add_rn(float a, float b) { return __fadd_rn(a, b); }
__device__ __forceinline__ uint64_t add_rn(uint64_t a, uint64_t b) { return add_f32x2(a, b); }
template <int R, typename T>
__device__ __forceinline__ T sum_parts(const T* x, int mp) {
  const T a = add_rn(x[2], x[3]);
  if constexpr (R == 6) {
    const T own = add_rn(x[0], x[1]), b = add_rn(x[4], x[5]);
    return add_rn(add_rn(a, mp == 2 ? b : own), mp == 2 ? own : b);
  } else {
    return add_rn(add_rn(a, add_rn(mp == 2 ? x[4] : x[0], x[1])), mp == 2 ? x[0] : x[4]);
  }
}

// Combine the partials that n CTAs (or shares) have of one unit, as a tree of
// groups of R in order: the last of a group to arrive merges the group's
// partials and goes on to the next level; false: someone else does.  (One CTA
// merging all of a long sequence's partials alone, 57 of 16 KB with 8 sequences
// on 152 SMs, took 32 us after the last byte had been read.)  A partial lies in
// memory lane by lane as the registers do, so the last to arrive keeps its own
// and adds the others to it: ((0 + 1) + (2 + 3)) + (4 + 5), each sum rounded
// alike either way round, so results do not depend on who arrives last.  R (six
// at head_dim 256, five at 512) is what one round of copies can bring in.  Run by the 128 consumer threads of a group; cf: the CTA (or share)
// of the unit's first partial, slot0: its slot, i: this one's place; o, and Mo,
// m, l (of head gid).
template <int D>
__device__ __forceinline__ bool merge_tree(const DecK& p, int cf, size_t slot0, int n, int i, float (&o)[F4Cfg<D>::MT][4], float& Mo,
                                           float& m, float& l, volatile int* last, uint8_t* ring, uint64_t* bar,
                                           uint32_t& phase, int tid, int bid) {
  using C = F4Cfg<D>;
  constexpr int PART = 8 * D * 4, R = C::R;
  const int gid = (tid & 31) >> 2, tig = tid & 3;
  int st = 1;
#pragma unroll 1
  for (int level = 0; n > 1; ++level, i /= R, st *= R) {
    const int mine = i % R, first = i - mine, cnt = min(R, n - first);
    const size_t base = slot0 + static_cast<size_t>(first) * st;   // slot of the group's first partial
    n = (n + R - 1) / R;
    if (cnt == 1) continue;   // alone in its group (others exist: n > 1)
    {
      const size_t slot = base + static_cast<size_t>(mine) * st;
      float4* dst = reinterpret_cast<float4*>(p.o_part + slot * 8 * D) + tid;
#pragma unroll
      for (int j = 0; j < C::MT; ++j) dst[j * 128] = make_float4(o[j][0], o[j][1], o[j][2], o[j][3]);
      if (tid < 32 && tig == 0) reinterpret_cast<float4*>(p.ml_part)[slot * 8 + gid] = make_float4(Mo, m, l, 0.f);
    }
    // arrive: the barrier orders the CTA's partial writes before thread 0's
    // release/acquire add, which publishes them and, for the last arrival,
    // makes the other CTAs' rows visible.  A group's counter is that of one of
    // its CTAs past the first, all of which begin inside this unit: at level l <
    // R its partials are R^l apart, and the offset l + 1 keeps the levels' apart.
    named_bar_sync(bid, 128);
    // the parts played: 0 this one, 1 its neighbour, 2 and 3 the first other
    // pair, 4 and 5 the second.  (Of five, only the last has two other pairs and
    // no neighbour: 1 is then the second pair's second.)
    const int mp = mine >> 1, ka = mp == 0 ? 2 : 0, kb = mp == 2 ? 2 : 4;
    auto index = [&](int part) {
      if (part == 0) return mine;
      if (part == 1) return R == 5 && mp == 2 ? kb + 1 : mine ^ 1;
      return part < 4 ? ka + part - 2 : kb + part - 4;
    };
    if (tid == 0) {
      int* c = p.counters + cf + first * st + 1 + level;
      const int old = atom_add_acq_rel_gpu(c, 1);
      if (old == cnt - 1) atomicExch(c, 0);   // zero for the next call
      else if (old < 0 || old >= cnt) atomicOr(p.err, FA_DEV_ERR_WORKSPACE);
      *last = old == cnt - 1;
      if (old == cnt - 1 && ring) {
        // the others by bulk copies into the ring, Q and weights, idle by now
        fence_proxy_async_global();   // the other CTAs' rows, seen through the acquire, for the bulk copies
        fence_proxy_async_smem();     // the ring's generic reads and zeroed scales before them
        mbar_arrive_expect_tx(bar, (cnt - 1) * PART);
#pragma unroll 1
        for (int k = 0; k < R - 1; ++k) {
          const int of = index(k + 1);
          if (of < cnt) bulk_load(ring + k * PART, p.o_part + (base + static_cast<size_t>(of) * st) * 8 * D, PART, bar);
        }
      }
    }
    named_bar_sync(bid, 128);
    if (!*last) return false;
    // bases, denominator and weights
    uint64_t w[R];   // of this lane's two heads
    {
      float4 v[R];
      Mo = m = kNoScore;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int k = index(r);
        v[r] = k < cnt ? __ldcg(reinterpret_cast<const float4*>(p.ml_part) + (base + static_cast<size_t>(k) * st) * 8 + gid)
                       : make_float4(kNoScore, kNoScore, 0.f, 0.f);
        Mo = fmaxf(Mo, v[r].x);
        m = fmaxf(m, v[r].y);
      }
      float lp[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float x = ex2(v[r].x - Mo);
        w[r] = pack_f32x2(__shfl_sync(0xffffffffu, x, 8 * tig), __shfl_sync(0xffffffffu, x, 8 * tig + 4));
        lp[r] = __fmul_rn(v[r].z, ex2(v[r].y - m));
      }
      l = sum_parts<R>(lp, mp);
    }
    if (ring) {
      if (!mbar_wait(bar, phase)) *last = 2;
      phase ^= 1;
      named_bar_sync(bid, 128);
      if (*last == 2) {   // a copy that did not land in time: everyone leaves
        if (tid == 0) atomicOr(p.err, FA_DEV_ERR_TIMEOUT);
        return false;
      }
    } else {
      // warp 0 writes the next level's bases over this one's first: not before
      // every warp has read them (with the ring the barrier above sees to it)
      named_bar_sync(bid, 128);
    }
    // a partial that is not there has weight 0 and stands for one that is
    const int some = index(1) < cnt ? 1 : 2;
    auto add_up = [&](auto at, auto load) {
      decltype(at(1)) src[R];
#pragma unroll
      for (int r = 1; r < R; ++r) src[r] = at(index(r) < cnt ? r : some);
#pragma unroll
      for (int j = 0; j < C::MT; ++j) {
        float4 v[R];
        v[0] = make_float4(o[j][0], o[j][1], o[j][2], o[j][3]);
#pragma unroll
        for (int r = 1; r < R; ++r) v[r] = load(src[r], j);
#pragma unroll
        for (int h = 0; h < 4; h += 2) {
          uint64_t x[R];
#pragma unroll
          for (int r = 0; r < R; ++r) x[r] = mul_f32x2(h ? pack_f32x2(v[r].z, v[r].w) : pack_f32x2(v[r].x, v[r].y), w[r]);
          unpack_f32x2(sum_parts<R>(x, mp), o[j][h], o[j][h + 1]);
        }
      }
    };
    if (ring)
      add_up([&](int r) { return smem_u32(ring) + (r - 1) * PART + tid * 16; },
             [](uint32_t at, int j) {
               float4 v;
               asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at + j * 2048) : "memory");
               return v;
             });
    else
      add_up([&](int r) { return reinterpret_cast<const float4*>(p.o_part + (base + static_cast<size_t>(index(r)) * st) * 8 * D) + tid; },
             [](const float4* at, int j) { return __ldcg(at + j * 128); });
  }
  return true;
}

// The current token's rows of (sequence b, KV head h) into their slot (one warp).
template <int D>
__device__ __noinline__ void store_now(const DecK& p, int b, int h, int lane) {
  RowRegs<D> rk, rv;
  const size_t src = (static_cast<size_t>(b) * p.Hkv + h) * D;
  row_load<D>(rk, p.k_new + src, lane);
  row_load<D>(rv, p.v_new + src, lane);
  store_current<D, FA_KV_FP4>(p, rk, rv, h, __ldg(p.slots + b), lane);
}

// Sequences of length <= 0 get out = 0 and lse = -inf, and their row is still
// stored; CTA `cta` of `ncta` writes the units u with u % ncta == cta.
template <int D>
__device__ __noinline__ void empty_units(const DecK& p, int cta, int ncta, int tid, int nthr) {
#pragma unroll 1
  for (int u = cta; u < p.units; u += ncta) {
    const Unit x = unit_at(p, u);
    if (x.L > 0) continue;
    if (p.slots && x.c == 0 && tid < 32) store_now<D>(p, x.b, x.h, tid);
    const int nh = min(8, p.g - x.c * 8);
    const size_t head = static_cast<size_t>(x.b) * p.Hq + x.h * p.g + x.c * 8;
#pragma unroll 1
    for (int i = tid; i < nh * D / 8; i += nthr) *(reinterpret_cast<uint4*>(p.out + head * D) + i) = make_uint4(0u, 0u, 0u, 0u);
    if (p.lse && tid < nh) p.lse[head + tid] = -INFINITY;
  }
}

template <int D>
__device__ __forceinline__ void decode_fp4_body(const DecK& p, const int cta, const int nblk) {
  using C = F4Cfg<D>;
  extern __shared__ __align__(128) uint8_t smem_all[];
  __shared__ int abort_flags[C::GROUPS], lasts[C::GROUPS], local_cnt[C::GROUPS];
  __shared__ F4Share shares[C::GROUPS];   // what the epilogue needs of the cut, out of the registers meanwhile

  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int group = wid / (C::NCW + 1), warp = wid - group * (C::NCW + 1);   // a group: 4 consumer warps, a producer
  const int tid = warp * 32 + lane;
  const int gid = lane >> 2, tig = lane & 3;
  uint8_t* smem = smem_all + group * C::GSMEM;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* empty = full + C::NSLOT;
  uint64_t* mbar_merge = empty + C::NSLOT;
  int& abort_flag = abort_flags[group];
  F4Share& share = shares[group];
  const int bid = 1 + group;   // the barrier of the group's consumers

  if (tid == 0) {
    for (int s = 0; s < C::NSLOT; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], C::NCW);
    }
    mbar_init(mbar_merge, 1);
    abort_flag = 0;
    local_cnt[group] = 0;
    fence_mbar_init();
  }
  __syncthreads();
  if (!p.early_metadata) griddep_wait();
  griddep_launch_dependents();

  // one warp of a group finds its share: all fifteen warps of the CTA at it
  // would share the issue slots, 1 us or more on the way to the first copy
  if (warp == C::NCW) {
    F4Share sh;
    const bool any = cut_share_warp<C::JOIN>(p, cta, nblk, group, sh);
    if (!any) sh.i = -1;
    if (lane == 0) share = sh;
  }
  named_bar_sync(1 + C::GROUPS + group, C::GTHR);
  if (share.i < 0) {
    if (share.n == 0 && cta == 0 && group == 0) {   // nothing visible anywhere: only empty outputs to write
      griddep_wait();
      empty_units<D>(p, 0, 1, tid, C::GTHR);
    }
    return;
  }
  if (warp == C::NCW) {
    // ------------------------------------------------------------ producer
    int e = 0;   // slots filled
    bool ok = true, first = true;
    const bool one = p.tiles_per_page == 1;   // the usual page of 16: no division
    const int s_beg = share.s_beg, s_end = share.s_end;
    int P = share.p0;
    for (int u = share.u0; ok && P < s_end && u < share.u_end; ++u) {
      const Unit x = unit_at(p, u);
      if (x.n > 0) {
        const int ta = x.t_first + max(s_beg, P) - P;
        const int tz = x.t_first + min(s_end, P + x.n) - P;
        const int32_t* bt = p.block_table + static_cast<size_t>(x.b) * p.max_pages_per_seq;
        // the CTA that reads the unit's last tile (it holds position L - 1)
        // stores the current token's rows first, so its own copy sees them
        const bool store_here = p.slots != nullptr && tz == x.t_first + x.n;
        for (int k0 = ta; ok && k0 < tz; k0 += 32) {
          int pid = -1;
          if (k0 + lane < tz) {
            pid = __ldg(bt + (one ? k0 + lane : div_u32(k0 + lane, p.tiles_per_page)));
            if (pid < 0 || pid >= p.num_pages) {
              atomicOr(p.err, FA_DEV_ERR_PAGE);
              pid = -1;
            }
          }
          if (first) griddep_wait();   // from here on the slab is read
          first = false;
          for (int k = k0; k < min(k0 + 32, tz); k += C::NT) {
            const int ntl = min(C::NT, tz - k);
            if (store_here && k + ntl >= tz) {
              store_now<D>(p, x.b, x.h, lane);
              // each lane orders its generic writes before the async-proxy
              // read of the tile that holds them
              fence_proxy_async_global();
              __syncwarp();
            }
            const int pg = __shfl_sync(0xffffffffu, pid, (k - k0 + lane) & 31);
            const bool mine = lane < ntl;
            const unsigned bad = __ballot_sync(0xffffffffu, mine && pg < 0);
            const int nbad = __popc(bad);
            const int tile = k + lane;
            const size_t row0 = mine && pg >= 0
                                    ? (static_cast<size_t>(pg) * p.Hkv + x.h) * p.page_size +
                                          (one ? 0 : tile - div_u32(tile, p.tiles_per_page) * p.tiles_per_page) * kTile
                                    : 0;
#pragma unroll 1
            for (int side = 0; side < 2; ++side, ++e) {
              const int st = e % C::NSLOT;
              uint8_t* dst = smem + st * C::SLOT;
              bool w = true;
              if (lane == 0) w = mbar_wait(&empty[st], ((e / C::NSLOT) & 1) ^ 1);
              ok = __shfl_sync(0xffffffffu, w, 0) && ok;
              if (!ok) break;
              if (bad) {   // tiles without a page (reported) read as zeros
                for (int t = 0; t < ntl; ++t)
                  if (bad >> t & 1) {
                    for (int i = lane; i < C::TILE_BYTES / 16; i += 32)
                      reinterpret_cast<uint4*>(dst + t * C::TILE_BYTES)[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (side == 0 && lane < kTile) {
                      float* sc = reinterpret_cast<float*>(dst + C::NT * C::TILE_BYTES);
                      sc[t * kTile + lane] = 1.0f;
                      sc[(C::NT + t) * kTile + lane] = 1.0f;
                    }
                  }
                fence_proxy_async_smem();   // before later copies into the slot
                __syncwarp();
              }
              if (lane == 0)
                mbar_arrive_expect_tx(&full[st], (ntl - nbad) * (C::TILE_BYTES + (side == 0 ? 2 * kTile * 4 : 0)));
              __syncwarp();
              if (mine && pg >= 0) {
                bulk_load(dst + lane * C::TILE_BYTES, (side ? p.vb : p.kb) + row0 * C::ROWB, C::TILE_BYTES, &full[st]);
                if (side == 0) {
                  uint8_t* sc = dst + C::NT * C::TILE_BYTES;
                  bulk_load(sc + lane * kTile * 4, p.ksb + row0, kTile * 4, &full[st]);
                  bulk_load(sc + C::SC_BYTES + lane * kTile * 4, p.vsb + row0, kTile * 4, &full[st]);
                }
              }
              __syncwarp();
            }
            if (!ok) break;
          }
        }
      }
      P += x.n;
    }
    if (lane == 0) {
      if (!ok) atomicOr(p.err, FA_DEV_ERR_TIMEOUT);
      // drain: no bulk copy may still be landing when the CTA exits
      for (int i = max(0, e - C::NSLOT); i < e; ++i)
        if (!mbar_wait(&full[i % C::NSLOT], (i / C::NSLOT) & 1)) atomicOr(p.err, FA_DEV_ERR_TIMEOUT);
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  griddep_wait();
  empty_units<D>(p, share.i, share.n, tid, C::NCW * 32);
  constexpr float P_OFF = 4.0f;    // weights reach 2^P_OFF against a base of their own tile's,
  constexpr float SLACK = 8.0f;    // and 2^(P_OFF + SLACK) against O's base before it is raised
  int slot = 0, step = 0;      // the ring's next slot, and its round's parity
  uint32_t round = 0;
  auto advance = [&]() {
    if (++slot == C::NSLOT) {
      slot = 0;
      round ^= 1;
    }
  };
  uint32_t merge_phase = 0;
  int P = share.p0;
  for (int u = share.u0; P < share.s_end && u < share.u_end; ++u) {
    const Unit x = unit_at(p, u);
    if (x.n == 0) continue;   // an empty unit advances nothing
    const int ta = x.t_first + max(share.s_beg, P) - P;
    const int tz = x.t_first + min(share.s_end, P + x.n) - P;
    const int nh = min(8, p.g - x.c * 8), head0 = x.h * p.g + x.c * 8;
    const int qpos = x.L - 1, lo = x.lo;
    const bool hv = gid < nh;

    // queries: Q^T fragments (B operand) as f16, in the order the codes are
    // stored, zero for padded heads; the warps share the conversion.  (Every
    // warp has left the previous segment's QK phase: the epilogue's barrier.)
    {
      uint32_t qbig = 0;
      const __nv_bfloat16* qrow = p.q + (static_cast<size_t>(x.b) * p.Hq + head0 + (hv ? gid : 0)) * D;
#pragma unroll
      for (int jj = 0; jj < C::NJ * C::NW / 4; ++jj) {
        const int jw = warp * (C::NJ * C::NW / 4) + jj, j = jw / C::NW, w = jw % C::NW;
        const uint4 v = hv ? __ldcg(reinterpret_cast<const uint4*>(qrow) + (4 * j + tig) * C::NW + w)
                           : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t vv[4] = {v.x, v.y, v.z, v.w};
        uint32_t f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          qbig |= bf16x2_past_f16(vv[i]);
          f[i] = pack_f16x2_sat(__uint_as_float(vv[i] << 16), __uint_as_float(vv[i] & 0xffff0000u));
        }
        *reinterpret_cast<uint4*>(smem + C::OFF_Q + (jw * 32 + lane) * 16) = make_uint4(f[0], f[1], f[2], f[3]);
      }
      if (__any_sync(0xffffffffu, qbig != 0) && lane == 0) atomicOr(p.err, FA_DEV_ERR_RANGE);
      named_bar_sync(bid, C::NCW * 32);
    }

    float o[C::MT][4];
#pragma unroll
    for (int i = 0; i < C::MT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    float M = kNoScore;                            // O's base, head gid
    float Mh[2] = {kNoScore, kNoScore};            // the same, heads 2 tig, 2 tig + 1
    float ml[2] = {kNoScore, kNoScore}, ll[2] = {0.f, 0.f};   // this lane's keys: base and sum of the denominator

    for (int tile0 = ta; tile0 < tz; tile0 += C::NT, ++step) {
      const int ntl = min(C::NT, tz - tile0);
      const int buf = step & 1;
      uint8_t* pbuf = smem + C::OFF_P + buf * C::NT * C::P_TILE;
      float* mw = reinterpret_cast<float*>(smem + C::OFF_MW) + buf * 8 * C::NCW;
      int* flag = reinterpret_cast<int*>(smem + C::OFF_FLAG) + buf * C::NCW;
      const bool edge = tile0 * kTile < lo || (tile0 + ntl) * kTile - 1 > qpos;   // some keys are masked
      const int kst = slot;
      if (!__all_sync(0xffffffffu, mbar_wait(&full[kst], round)) && lane == 0) {
        abort_flag = 1;   // everyone leaves at the barrier below
        atomicOr(p.err, FA_DEV_ERR_TIMEOUT);
      }
      advance();
      const uint8_t* kslot = smem + kst * C::SLOT;
      const float* scl = reinterpret_cast<const float*>(kslot + C::NT * C::TILE_BYTES);
      if (warp < ntl) {
        // ---- S^T of this warp's tiles, warp and (TPW = 2) warp + 4: keys gid, gid
        // + 8 (as MMA rows), heads 2 tig, 2 tig + 1.  A tile past the step's last
        // runs over whatever the slot holds; its keys count as masked.
        const uint8_t* ra = kslot + warp * C::TILE_BYTES + key_row<D>(gid) * C::ROWB;   // key_row(gid + 8) = key_row(gid) + 8
        float acc[C::TPW][2][4] = {};
#pragma unroll
        for (int i = 0; i < C::NJ / 2; ++i) {
          __half2 sca[C::TPW], scb[C::TPW];
#pragma unroll
          for (int t = 0; t < C::TPW; ++t) {
            sca[t] = block_scales<D>(ra + t * C::NCW * C::TILE_BYTES + D / 2, i, tig);
            scb[t] = block_scales<D>(ra + t * C::NCW * C::TILE_BYTES + 8 * C::ROWB + D / 2, i, tig);
          }
#pragma unroll
          for (int jj = 0; jj < 2; ++jj) {
            const int j = 2 * i + jj;
            uint32_t wa[C::TPW][C::NW], wb[C::TPW][C::NW];
#pragma unroll
            for (int t = 0; t < C::TPW; ++t) {
              lds_words(ra + t * C::NCW * C::TILE_BYTES + (4 * j + tig) * 4 * C::NW, wa[t]);
              lds_words(ra + t * C::NCW * C::TILE_BYTES + 8 * C::ROWB + (4 * j + tig) * 4 * C::NW, wb[t]);
            }
#pragma unroll
            for (int w = 0; w < C::NW; ++w) {
              const uint4 qf = *reinterpret_cast<const uint4*>(smem + C::OFF_Q + ((j * C::NW + w) * 32 + lane) * 16);
#pragma unroll
              for (int t = 0; t < C::TPW; ++t) {
                const __half2 fa_ = jj ? __high2half2(sca[t]) : __low2half2(sca[t]);
                const __half2 fb_ = jj ? __high2half2(scb[t]) : __low2half2(scb[t]);
                uint32_t ha[4], hb[4];
                e2m1x8_to_f16(wa[t][w], ha);
                e2m1x8_to_f16(wb[t][w], hb);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  ha[c] = hmul2(ha[c], fa_);
                  hb[c] = hmul2(hb[c], fb_);
                }
                mma_f16(acc[t][0], ha[0], hb[0], ha[1], hb[1], qf.x, qf.y);
                mma_f16(acc[t][1], ha[2], hb[2], ha[3], hb[3], qf.z, qf.w);
              }
            }
          }
        }
        // ---- scores and weights
        const bool part = C::TPW > 1 && warp + (C::TPW - 1) * C::NCW >= ntl;   // the last tile is not there
        float s[C::TPW][2][2], ve[C::TPW][2];
        bool grow = false;
#pragma unroll
        for (int t = 0; t < C::TPW; ++t)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int key = (warp + t * C::NCW) * kTile + key_row<D>(gid) + 8 * r;
            const int pos = tile0 * kTile + key;
            const bool vis = !(part && t == C::TPW - 1) && (!edge || (pos >= lo && pos <= qpos));
            const float ks = scl[key] * p.scale_log2;
            // the exponent of the row's V scale, as a float: behind 2^23, without its bias
            ve[t][r] = __uint_as_float(0x4b000000u | (__float_as_uint(scl[C::NT * kTile + key]) >> 23)) - 8388735.0f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              s[t][r][h] = vis ? (acc[t][0][2 * r + h] + acc[t][1][2 * r + h]) * ks : -INFINITY;
              grow |= s[t][r][h] + ve[t][r] > Mh[h] + SLACK || s[t][r][h] > ml[h] + 30.0f;
            }
          }
        float base[2] = {Mh[0], Mh[1]};
        grow = __any_sync(0xffffffffu, grow);
        if (grow) {
          // rare once O's base has settled: these tiles' own base where it
          // exceeds O's by more than the slack, and the denominators' bases
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float mn = ml[h], v = -INFINITY;
#pragma unroll
            for (int t = 0; t < C::TPW; ++t) {
              mn = fmaxf(mn, fmaxf(s[t][0][h], s[t][1][h]));
              v = fmaxf(v, fmaxf(s[t][0][h] + ve[t][0], s[t][1][h] + ve[t][1]));
            }
            ll[h] *= ex2(ml[h] - mn);
            ml[h] = mn;
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            if (v > Mh[h] + SLACK) base[h] = ceilf(v);
            if (gid == 0) mw[(2 * tig + h) * C::NCW + warp] = base[h];
          }
        }
        // s - (base - P_OFF - e): the bracket holds integers alone and is exact, and
        // so is a difference of neighbours; s + e would round at s's own scale
#pragma unroll
        for (int t = 0; t < C::TPW; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float bp = base[h] - P_OFF;
            ll[h] += ex2(s[t][0][h] - ml[h]) + ex2(s[t][1][h] - ml[h]);
            uint8_t* ph = pbuf + (warp + t * C::NCW) * C::P_TILE + (2 * tig + h) * C::P_HEAD + gid * 2;
            *reinterpret_cast<__half*>(ph) = __float2half_rn(ex2(s[t][0][h] - (bp - ve[t][0])));
            *reinterpret_cast<__half*>(ph + 16) = __float2half_rn(ex2(s[t][1][h] - (bp - ve[t][1])));
          }
        if (lane == 0) flag[warp] = grow;
      } else if (lane == 0) {
        flag[warp] = 0;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[kst]);
      named_bar_sync(bid, C::NCW * 32);   // every tile's weights and base are there
      if (*reinterpret_cast<volatile int*>(&abort_flag)) return;

      // ---- tiles with a base of their own: raise O's base to the largest, and
      // bring every tile's weights to it (exact powers of two)
      float f[C::NCW] = {1.f, 1.f, 1.f, 1.f};
      const int4 fl = *reinterpret_cast<const int4*>(flag);
      const bool scaled = (fl.x | fl.y | fl.z | fl.w) != 0;
      if (scaled) {
        const float4 v = *reinterpret_cast<const float4*>(mw + gid * C::NCW);
        f[0] = fl.x ? v.x : M;
        f[1] = fl.y ? v.y : M;
        f[2] = fl.z ? v.z : M;
        f[3] = fl.w ? v.w : M;
        const float Mn = fmaxf(M, fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3])));
        const float r = ex2(M - Mn);   // 0 where O is still empty
        M = Mn;
#pragma unroll
        for (int i = 0; i < C::NCW; ++i) f[i] = ex2(f[i] - M);
        const float rA = __shfl_sync(0xffffffffu, r, 8 * tig), rB = __shfl_sync(0xffffffffu, r, 8 * tig + 4);
        Mh[0] = __shfl_sync(0xffffffffu, M, 8 * tig);
        Mh[1] = __shfl_sync(0xffffffffu, M, 8 * tig + 4);
#pragma unroll
        for (int i = 0; i < C::MT; ++i) {
          o[i][0] *= rA;
          o[i][1] *= rB;
          o[i][2] *= rA;
          o[i][3] *= rB;
        }
      }

      const int vst = slot;
      if (!__all_sync(0xffffffffu, mbar_wait(&full[vst], round)) && lane == 0) {
        abort_flag = 1;   // everyone leaves at the next barrier
        atomicOr(p.err, FA_DEV_ERR_TIMEOUT);
      }
      advance();
      uint8_t* vslot = smem + vst * C::SLOT;
      constexpr int SB = D / 64;   // this warp's block scales per row (bytes)
      if (edge) {
        // masked keys have weight 0, but their rows may hold anything (block
        // scales of NaN included): zero this warp's block scales of those rows
#pragma unroll 1
        for (int r = lane; r < ntl * kTile; r += 32) {
          const int pos = tile0 * kTile + r;
          if (pos < lo || pos > qpos) {
            uint32_t* z = reinterpret_cast<uint32_t*>(vslot + r * C::ROWB + D / 2 + warp * SB);
            z[0] = 0u;
            if constexpr (SB == 8) z[1] = 0u;
          }
        }
        fence_proxy_async_smem();   // before the copy that refills the slot
        __syncwarp();
      }
      // ---- O^T += V^T P^T over this warp's columns
      auto pv_tile = [&](int t) {
        const uint8_t* vt = vslot + t * C::TILE_BYTES;
        const uint32_t* pw = reinterpret_cast<const uint32_t*>(pbuf + t * C::P_TILE + gid * C::P_HEAD);
        uint32_t b0 = pw[tig], b1 = pw[tig + 4];
        if (scaled) {
          const __half2 fh = __float2half2_rn((t & 3) == 0 ? f[0] : (t & 3) == 1 ? f[1] : (t & 3) == 2 ? f[2] : f[3]);
          b0 = hmul2(b0, fh);
          b1 = hmul2(b1, fh);
        }
        uint32_t w[4][C::NW], sc[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {   // keys 2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9
          const uint8_t* row = vt + key_row<D>(2 * tig + (r & 1) + (r >> 1) * 8) * C::ROWB;
          lds_words(row + (8 * warp + gid) * 4 * C::NW, w[r]);
          sc[r] = row[D / 2 + warp * SB + (D == 256 ? gid >> 1 : gid)];
        }
        const uint32_t s01 = e4m3x2_to_f16x2(sc[0] | (sc[1] << 8)), s23 = e4m3x2_to_f16x2(sc[2] | (sc[3] << 8));
#pragma unroll
        for (int q = 0; q < C::NW; ++q) {
          // code pairs of two keys at one column: even columns, odd columns
          constexpr uint32_t LOW = 0x0f0f0f0fu;
          uint32_t e01[4], d01[4], e23[4], d23[4];
          e2m1x8_to_f16((w[0][q] & LOW) | ((w[1][q] << 4) & ~LOW), e01);
          e2m1x8_to_f16(((w[0][q] >> 4) & LOW) | (w[1][q] & ~LOW), d01);
          e2m1x8_to_f16((w[2][q] & LOW) | ((w[3][q] << 4) & ~LOW), e23);
          e2m1x8_to_f16(((w[2][q] >> 4) & LOW) | (w[3][q] & ~LOW), d23);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mma_f16(o[4 * q + i], hmul2(e01[i], s01), hmul2(d01[i], s01), hmul2(e23[i], s23), hmul2(d23[i], s23), b0, b1);
        }
      };
#pragma unroll 4
      for (int t = 0; t < ntl; ++t) pv_tile(t);
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[vst]);
    }

    // -------------------------------------------------------- segment epilogue
    // the denominator: lanes of a head, then the warps, in a fixed order
    float2* mls = reinterpret_cast<float2*>(smem + C::OFF_ML);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int of = 4; of < 32; of <<= 1) {
        const float mo = __shfl_xor_sync(0xffffffffu, ml[h], of), lo_ = __shfl_xor_sync(0xffffffffu, ll[h], of);
        const float mn = fmaxf(ml[h], mo);
        ll[h] = ll[h] * ex2(ml[h] - mn) + lo_ * ex2(mo - mn);
        ml[h] = mn;
      }
      if (gid == 0) mls[warp * 8 + 2 * tig + h] = make_float2(ml[h], ll[h]);
    }
    named_bar_sync(bid, C::NCW * 32);
    if (*reinterpret_cast<volatile int*>(&abort_flag)) return;
    float m = kNoScore, l = 0.f;   // of head gid
#pragma unroll
    for (int w = 0; w < C::NCW; ++w) m = fmaxf(m, mls[w * 8 + gid].x);
#pragma unroll
    for (int w = 0; w < C::NCW; ++w) {
      const float2 v = mls[w * 8 + gid];
      l += v.y * ex2(v.x - m);
    }
    if (fabsf(M) >= kMaxBase && M > kNoScore) atomicOr(p.err, FA_DEV_ERR_RANGE);
    float Mo = M - P_OFF;
    // The partials of the unit's shares in this CTA (the whole-unit cut) meet in
    // shared memory: each group leaves its own in the idle ring, lane by lane as
    // the registers lie; the last to arrive adds them up in order and goes on.
    bool here = share.unsplit;   // and they are all there are
    if (share.nct > 0) {
      const int sb = max(share.sb, share.cf), cnt = min(share.se, share.cf + share.nct) - sb, mine = share.i - sb;
      here = cnt == share.nct;
      if (cnt > 1) {
        constexpr int PART = 8 * D * 4;
        float4* dst = reinterpret_cast<float4*>(smem) + tid;
#pragma unroll
        for (int i = 0; i < C::MT; ++i) dst[i * 128] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
        if (warp == 0 && tig == 0) reinterpret_cast<float4*>(smem + PART)[gid] = make_float4(Mo, m, l, 0.f);
        volatile int* last = &lasts[group];
        named_bar_sync(bid, C::NCW * 32);
        if (tid == 0) {
          __threadfence_block();
          *last = atomicAdd(&local_cnt[sb - share.sb], 1) == cnt - 1;
          __threadfence_block();
        }
        named_bar_sync(bid, C::NCW * 32);
        if (!*last) return;   // its only segment
        const uint8_t* src = smem - mine * C::GSMEM;
        float4 v[C::GROUPS];
        Mo = m = kNoScore;
#pragma unroll
        for (int k = 0; k < C::GROUPS; ++k) {
          v[k] = k < cnt ? reinterpret_cast<const float4*>(src + k * C::GSMEM + PART)[gid]
                         : make_float4(kNoScore, kNoScore, 0.f, 0.f);
          Mo = fmaxf(Mo, v[k].x);
          m = fmaxf(m, v[k].y);
        }
        l = 0.f;
        uint64_t acc[C::MT][2] = {};
#pragma unroll
        for (int k = 0; k < C::GROUPS; ++k) {
          if (k >= cnt) continue;
          l += v[k].z * ex2(v[k].y - m);
          const float w = ex2(v[k].x - Mo);
          const uint64_t w2 = pack_f32x2(__shfl_sync(0xffffffffu, w, 8 * tig), __shfl_sync(0xffffffffu, w, 8 * tig + 4));
#pragma unroll
          for (int i = 0; i < C::MT; ++i) {
            const float4 t = reinterpret_cast<const float4*>(src + k * C::GSMEM)[i * 128 + tid];
            acc[i][0] = fma_f32x2(pack_f32x2(t.x, t.y), w2, acc[i][0]);
            acc[i][1] = fma_f32x2(pack_f32x2(t.z, t.w), w2, acc[i][1]);
          }
        }
#pragma unroll
        for (int i = 0; i < C::MT; ++i) {
          unpack_f32x2(acc[i][0], o[i][0], o[i][1]);
          unpack_f32x2(acc[i][1], o[i][2], o[i][3]);
        }
      }
    }
    // The unit's partials in memory: slot (less u) of the first, their number,
    // this one's place
    int cf = 0, nct = 1, me = 0;
    if (!here) {
      const bool whole = share.nct > 0;   // one partial a CTA, else one a share
      const int a = whole ? share.cf : P, z = whole ? a + share.nct - 1 : P + x.n - 1;
      const int parts = whole ? share.nb : share.n, of = whole ? share.n : share.T;
      cf = part_of(a, parts, of);
      nct = part_of(z, parts, of) - cf + 1;
      me = (whole ? cta : share.i) - cf;
    }
    const bool mine = merge_tree<D>(p, cf, static_cast<size_t>(cf) + u, nct, me, o, Mo, m, l, &lasts[group],
                                    P + x.n >= share.s_end ? smem : nullptr, mbar_merge, merge_phase, tid, bid);
    if (mine) {
      const int d0 = (8 * warp + gid) * 8 * C::NW;   // this lane's columns: 8 NW from d0 on
      const float r = ex2(Mo - m) / l;
      const float r2[2] = {__shfl_sync(0xffffffffu, r, 8 * tig), __shfl_sync(0xffffffffu, r, 8 * tig + 4)};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (2 * tig + h >= nh) continue;
        uint4* dst = reinterpret_cast<uint4*>(p.out + (static_cast<size_t>(x.b) * p.Hq + head0 + 2 * tig + h) * D + d0);
#pragma unroll
        for (int q = 0; q < C::NW; ++q) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(o[4 * q + i][h] * r2[h], o[4 * q + i][2 + h] * r2[h]);
          dst[q] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if (p.lse && warp == 0 && tig == 0 && hv)
        p.lse[static_cast<size_t>(x.b) * p.Hq + head0 + gid] = (m + __log2f(l)) * 0.69314718055994531f;
    }
    P += x.n;
  }
}

template <int D>
__global__ void __launch_bounds__(F4Cfg<D>::NTHR, 1) decode_fp4_kernel(const __grid_constant__ DecK p) {
  decode_fp4_body<D>(p, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
}

// Several layers in one launch: the CTAs of layer i are [cta0[i], cta0[i + 1]).
struct F4Layers {
  DecK k[kMaxLayersPerLaunch];
  int cta0[kMaxLayersPerLaunch + 1];
  int n;
};

template <int D>
__global__ void __launch_bounds__(F4Cfg<D>::NTHR, 1) decode_fp4_layers_kernel(const __grid_constant__ F4Layers m) {
  const int b = static_cast<int>(blockIdx.x);
  int li = 0;
  while (li + 1 < m.n && b >= m.cta0[li + 1]) ++li;
  decode_fp4_body<D>(m.k[li], b - m.cta0[li], m.cta0[li + 1] - m.cta0[li]);
}

// Groups of a CTA: no more than the plan's shares need.
static int groups_of(const DecodePlan& p) { return (p.ncta + p.blocks - 1) / p.blocks; }

template <int D>
static cudaError_t launch_fp4(const DecodeArgs* a, int n, cudaStream_t s) {
  using C = F4Cfg<D>;
  cudaError_t e;
  if (n == 1) {
    static unsigned int done = 0;
    e = set_smem_once(reinterpret_cast<const void*>(decode_fp4_kernel<D>), C::SMEM, &done);
    if (e != cudaSuccess) return e;
    return launch_pdl(decode_fp4_kernel<D>, dim3(a->plan.blocks), dim3(groups_of(a->plan) * C::GTHR),
                      groups_of(a->plan) * C::GSMEM, s, make_deck(*a));
  }
  static unsigned int done = 0;
  e = set_smem_once(reinterpret_cast<const void*>(decode_fp4_layers_kernel<D>), C::SMEM, &done);
  if (e != cudaSuccess) return e;
  F4Layers m{};
  m.n = n;
  int groups = 1;
  for (int i = 0; i < n; ++i) {
    m.k[i] = make_deck(a[i]);
    m.cta0[i + 1] = m.cta0[i] + a[i].plan.blocks;
    groups = max(groups, groups_of(a[i].plan));
  }
  return launch_pdl(decode_fp4_layers_kernel<D>, dim3(m.cta0[n]), dim3(groups * C::GTHR), groups * C::GSMEM, s, m);
}

cudaError_t launch_decode_fp4(const DecodeArgs* a, int n, cudaStream_t s) {
  return a[0].D == 256 ? launch_fp4<256>(a, n, s) : launch_fp4<512>(a, n, s);
}

}  // namespace fa
