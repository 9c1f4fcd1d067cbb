// Norms of queries, keys and values for each head, the rotation by position, and
// the K and V rows' store into the paged slab, in one pass: what a layer does
// between its projection and fa_kv_store, whose rows are "post-RoPE" ("unsloth
// commit dee9371": the store layer writes its post-rotary k, v).
//
//   y = x / sqrt(mean(x^2) + eps) * (offset + w)
//   z_i = y_i cos(p f_i) - y_{i+h} sin(p f_i),  z_{i+h} = y_{i+h} cos(p f_i) + y_i sin(p f_i),  i < h = R / 2
//
// in fp32, rounded once to bf16 (a model's activations are bf16, and the slab's
// quantisation starts from bf16 rows in every other call).
//
// Angles.  The caller gives each frequency as a step in turns, a 64-bit fraction
// of 2^64: position * step modulo 2^64 is the phase, exact for every position (no
// table of cosines to read, which at head_dim 512 would be 2 KB a token).  Its
// upper 32 bits leave an angle in [-pi, pi), where the hardware's sine and cosine
// are off by 2^-21 at most: an 8192nd of a bf16 rounding of the pair's length.
//
// With A_i = w_i cos, B_i = -w_{i+h} sin (i < h; A_{i+h} = w_{i+h} cos, B_{i+h} = w_i sin), made once
// an item (below), a value costs z = f (x A + x' B), x' its partner, f the row's 1 / root.
//
// A memory pass: each row read once, written once (rows out, slab).  Warps are
// persistent and independent: each walks items (up to 16 heads of one kind of one
// token: its sines serve them all), with the next rows' loads in flight
// while it works on the ones before.  30011 tokens of 16 + 2 + 2 heads at head_dim 512, bf16:
// 197 us, 6.25 TB/s of 6.8 (copied without arithmetic 186); 2048 tokens of 16 + 8 + 8 at 256
// with the rows out: 17.8 us, 4.7 TB/s (there the schedulers issue half of the time, on shuffles and
// short rows).  Blocks of their own for each token's heads took 224 and 20 us (their
// loads waited for their sines, and blocks start at one a nanosecond), rows through
// a ring of shared memory with a copying warp 263 and 18.6.
#include <algorithm>

#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_row.cuh"

namespace fa {

// A block's warps are independent: 64 threads so that it starts and ends easily.  16 warps an
// SM at 128 registers: a warp's rows and the ones on their way (4 KB at
// head_dim 512, 2 x 2 rows; 256, 2 x 4) without spills.  20 and 24 warps, which spill, took 1.2 to 1.8 times as long.
constexpr int kRowsThreads = 64, kRowsWarps = 16;
// Heads of an item, at most: 16 against 8, 30011 tokens of 16 + 2 + 2 heads at 512 197 us against 201.
constexpr int kRowsHeads = 16;

struct RowsK {
  const __nv_bfloat16* src[3];   // q, k, v
  long long stride[3];           // elements from token to token
  __nv_bfloat16* dst[3];         // dense rows out (k, v: may be null)
  const __nv_bfloat16* weight[2];   // q, k (null: ones)
  uint8_t* slab[2];              // k, v (null slots: no store)
  float* scale[2];
  const int32_t* positions;
  const int32_t* slots;
  const uint64_t* steps;
  unsigned int* err;
  int T, Hq, Hkv, nq, rows;      // nq: query rows of a token taken (Hq or 0); rows: with keys and values
  int half8;                     // R / 16: 8-element vectors in half of the rotated columns
  int norm, page_size, num_pages;
  float eps, offset;
  int per_q, per_kv, groups_q, groups_kv;   // heads a warp, groups of a token (groups_kv of keys and of values each)
  uint32_t items;                // groups x tokens, group by group
  FastDiv by_T, by_page;
};

// Cosine and sine of a phase, in turns of 2^64.
__device__ __forceinline__ void turn1(uint64_t phase, float& c, float& s) {
  const float a = static_cast<float>(static_cast<int32_t>(static_cast<uint32_t>(phase >> 32))) * 1.4629180792671596e-9f;   // pi / 2^31
  c = __cosf(a);
  s = __sinf(a);
}

template <int NV>
__device__ __forceinline__ float square_sum(const float (&x)[NV][8]) {
  uint64_t acc = pack_f32x2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const uint64_t p = pack_f32x2(x[j][e], x[j][e + 1]);
      acc = fma_f32x2(p, p, acc);
    }
  float lo, hi;
  unpack_f32x2(acc, lo, hi);
  return lo + hi;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// 1 / sqrt(mean(x^2) + eps) of a row.  Where the squares leave fp32 (magnitudes near 2^64,
// infinities, NaN) the row is multiplied by `small`, 2^-70, first.
template <int D, int NV>
__device__ __forceinline__ float row_factor(float (&x)[NV][8], float eps, float& small) {
  const float ss = warp_sum(square_sum(x));
  if (ss <= 1e38f) return rsqrtf(fmaf(ss, 1.0f / D, eps));
  small = 8.470329472543003e-22f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) x[j][e] *= small;
  return rsqrtf(warp_sum(square_sum(x)) * (1.0f / D));
}

// Where a rotated vector's partner is: in its own lane (D = 512, R = D), in a lane's
// first vector (2 R / 16 <= 32 vectors rotated: exchanged by shuffles), or in any (read
// again: the row was just loaded, so from L1).
enum { kOwnLane, kFirst, kAnywhere };

// Cosines and sines of pairs 8 c .. 8 c + 7 at position pos.
__device__ __forceinline__ void turns8(const uint64_t* steps, int c, int pos, float (&cs)[8], float (&sn)[8]) {
  const ulonglong2* s = reinterpret_cast<const ulonglong2*>(steps) + 4 * c;
  const uint64_t p = static_cast<uint64_t>(static_cast<int64_t>(pos));
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const ulonglong2 w = __ldg(s + e);
    turn1(p * w.x, cs[2 * e], sn[2 * e]);
    turn1(p * w.y, cs[2 * e + 1], sn[2 * e + 1]);
  }
}

// Some heads of one kind of one token, from head h on.
struct RowItem {
  uint32_t i;   // >= items: none
  int kind, t, h, h1, pos, slot;
  const uint4* src;
};

template <int D, int KV, int RH, int ROT>
__global__ void __launch_bounds__(kRowsThreads, kRowsWarps * 32 / kRowsThreads)
    rows_kernel(const __grid_constant__ RowsK a) {
  constexpr int NV = RowRegs<D>::NV;
  static_assert(ROT == kFirst || NV == 2, "head_dim 256 has one vector a lane");
  constexpr int NR = ROT == kFirst ? 1 : NV;   // vectors that rotation reaches
  // Index arrays are read after the wait even under FA_FLAG_EARLY_METADATA: they
  // usually come from the kernel before (fa_plan_step).
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const uint32_t nwarps = gridDim.x * (kRowsThreads / 32);
  auto item = [&](uint32_t i) {
    RowItem x;
    x.i = i;
    if (i >= a.items) {
      x.kind = x.t = x.h = x.h1 = x.pos = 0;
      x.slot = -1;
      x.src = nullptr;
      return x;
    }
    int g = static_cast<int>(a.by_T.div(i));
    x.t = static_cast<int>(i - g * a.by_T.d);
    x.kind = 0;
    if (g >= a.groups_q) {
      g -= a.groups_q;
      x.kind = g >= a.groups_kv ? 2 : 1;
      g -= x.kind == 2 ? a.groups_kv : 0;
    }
    const int per = x.kind == 0 ? a.per_q : a.per_kv;
    x.h = g * per;
    x.h1 = min(x.h + per, x.kind == 0 ? a.nq : a.Hkv);
    const __nv_bfloat16* base = x.kind == 0 ? a.src[0] : x.kind == 1 ? a.src[1] : a.src[2];
    const long long stride = x.kind == 0 ? a.stride[0] : x.kind == 1 ? a.stride[1] : a.stride[2];
    x.src = reinterpret_cast<const uint4*>(base + static_cast<size_t>(x.t) * stride) + lane;
    x.pos = a.half8 > 0 && x.kind < 2 ? __ldg(a.positions + x.t) : 0;
    x.slot = x.kind > 0 && a.slots ? __ldg(a.slots + x.t) : -1;
    return x;
  };
  auto load = [&](const RowItem& x, RowRegs<D> (&r)[RH]) {   // (plain loads: a row may be its own output)
#pragma unroll
    for (int i = 0; i < RH; ++i)
      if (x.h + i < x.h1)
#pragma unroll
        for (int j = 0; j < NV; ++j) r[i].v[j] = x.src[(x.h + i) * (D / 8) + j * 32];
  };

  RowItem x = item((blockIdx.x * kRowsThreads + threadIdx.x) >> 5);
  if (x.i >= a.items) return;
  RowRegs<D> r[RH], next[RH];
  load(x, r);
  bool fresh = true, norm = false, turn = false;
  long long to = -1;   // slab row of head 0
  __nv_bfloat16* dst = nullptr;
  uint8_t* slab = nullptr;
  float* scale = nullptr;
  // the coefficients of own values and partners, and where the partners are
  float ca[NV][8], cb[NR][8];
  int from[NR];
  auto make = [&]() {
    norm = (a.norm >> x.kind) & 1;
    turn = a.half8 > 0 && x.kind < 2;
    to = -1;
    if (x.slot >= 0) {   // a negative slot is a padding token
      const uint32_t page = a.by_page.div(x.slot), off = x.slot - page * a.page_size;
      if (page < static_cast<uint32_t>(a.num_pages)) to = static_cast<long long>(page) * a.Hkv * a.page_size + off;
      else if (lane == 0 && x.h == 0) atomicOr(a.err, FA_DEV_ERR_SLOT);
    }
    dst = x.kind == 0 ? a.dst[0] : x.kind == 1 ? a.dst[1] : a.dst[2];
    if (dst) dst += static_cast<size_t>(x.t) * (x.kind == 0 ? a.Hq : a.Hkv) * D;
    slab = x.kind == 2 ? a.slab[1] : a.slab[0];
    scale = x.kind == 2 ? a.scale[1] : a.scale[0];
    const uint4* w = norm && x.kind < 2 ? reinterpret_cast<const uint4*>(x.kind == 0 ? a.weight[0] : a.weight[1]) : nullptr;
    float wt[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (w) bf16x8_to_f32(__ldg(w + j * 32 + lane), wt[j]);
#pragma unroll
      for (int e = 0; e < 8; ++e) ca[j][e] = wt[j][e] = w ? wt[j][e] + a.offset : 1.0f;
    }
    if (turn) {
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        const int v = j * 32 + lane;
        const bool first = v < a.half8, none = v >= 2 * a.half8;
        const int o = none ? v : first ? v + a.half8 : v - a.half8;
        from[j] = o;
        float cs[8], sn[8], ow[8];
        turns8(a.steps, none ? 0 : min(v, o), x.pos, cs, sn);
        if (ROT != kOwnLane && w) bf16x8_to_f32(__ldg(w + o), ow);   // the partner's weights
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float wo = ROT == kOwnLane ? wt[NV - 1 - j][e] : w ? ow[e] + a.offset : 1.0f;
          cb[j][e] = none ? 0.f : first ? -sn[e] * wo : sn[e] * wo;
          ca[j][e] = none ? ca[j][e] : ca[j][e] * cs[e];
        }
      }
    }
  };

  while (true) {
    RowItem y = x;   // what comes next: its loads go out before this one's arithmetic
    y.h += RH;
    const bool another = y.h >= x.h1;
    if (another) y = item(x.i + nwarps);
    const bool more = y.i < a.items;
    if (more) load(y, next);
    if (fresh) make();
    fresh = another;
#pragma unroll
    for (int i = 0; i < RH; ++i) {
      if (x.h + i >= x.h1) break;
      if (norm || turn) {   // (else the row goes on bit for bit)
        float v[NV][8], small = 1.0f;
        uint4 o[NR];
        if (ROT == kAnywhere && turn) {
#pragma unroll
          for (int j = 0; j < NR; ++j) o[j] = x.src[(x.h + i) * (D / 8) + from[j] - lane];
          __syncwarp();   // every lane has read the row (which may be its own output)
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) bf16x8_to_f32(r[i].v[j], v[j]);
        const float f = norm ? row_factor<D>(v, a.eps, small) : 1.0f;
        const uint64_t f2 = pack_f32x2(f, f);
        uint64_t z[NV][4];
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            z[j][k] = mul_f32x2(pack_f32x2(v[j][2 * k], v[j][2 * k + 1]), pack_f32x2(ca[j][2 * k], ca[j][2 * k + 1]));
        if (turn) {
#pragma unroll
          for (int j = 0; j < NR; ++j) {
            float p[8];
            if constexpr (ROT == kAnywhere) bf16x8_to_f32(o[j], p);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if constexpr (ROT == kOwnLane) p[e] = v[NV - 1 - j][e];
              if constexpr (ROT == kFirst) p[e] = __shfl_sync(0xffffffffu, v[0][e], from[j] & 31);
              if constexpr (ROT == kAnywhere) p[e] *= small;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
              z[j][k] = fma_f32x2(pack_f32x2(p[2 * k], p[2 * k + 1]), pack_f32x2(cb[j][2 * k], cb[j][2 * k + 1]), z[j][k]);
          }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          uint32_t out[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float lo, up;
            unpack_f32x2(mul_f32x2(z[j][k], f2), lo, up);
            out[k] = pack_bf16x2(lo, up);
          }
          // a vector neither normed nor turned stays as it is, infinities and all
          if (norm || ROT == kOwnLane || j * 32 + lane < 2 * a.half8) r[i].v[j] = make_uint4(out[0], out[1], out[2], out[3]);
        }
      }
      if (dst) row_store_bf16<D>(r[i], dst + static_cast<size_t>(x.h + i) * D, lane);
      if (to < 0) continue;
      const size_t row = static_cast<size_t>(to) + static_cast<size_t>(x.h + i) * a.page_size;
      row_store<D, KV>(r[i], slab + row * kRowBytes<D, KV>, KV == FA_KV_BF16 ? nullptr : scale + row, lane);
    }
    if (!more) break;
    x = y;
#pragma unroll
    for (int i = 0; i < RH; ++i) r[i] = next[i];
  }
}

template <int D, int KV>
static cudaError_t launch_rows_t(RowsK k, cudaStream_t s) {
  constexpr int RH = D == 256 ? 4 : 2;   // rows in flight behind those in work
  // as many heads an item as leave every resident warp one
  const long long resident = static_cast<long long>(kRowsWarps) * sm_count();
  const long long share = (static_cast<long long>(k.T) * k.rows + resident - 1) / resident;
  k.per_q = k.per_kv = static_cast<int>(std::min<long long>(share, kRowsHeads));
  k.groups_q = (k.nq + k.per_q - 1) / k.per_q;
  k.groups_kv = k.rows > k.nq ? (k.Hkv + k.per_kv - 1) / k.per_kv : 0;
  const long long items = static_cast<long long>(k.T) * (k.groups_q + 2 * k.groups_kv);
  if (items >= (1LL << 31) - (1 << 20)) return cudaErrorInvalidConfiguration;
  k.items = static_cast<uint32_t>(items);
  k.by_T = FastDiv(k.T);
  constexpr int wpb = kRowsThreads / 32;
  const dim3 g(static_cast<unsigned>((std::min(items, resident) + wpb - 1) / wpb)), b(kRowsThreads);
  if (k.half8 <= 16) return launch_pdl(rows_kernel<D, KV, RH, kFirst>, g, b, 0, s, k);
  if constexpr (D == 512) {
    if (k.half8 == 32) return launch_pdl(rows_kernel<D, KV, RH, kOwnLane>, g, b, 0, s, k);
    return launch_pdl(rows_kernel<D, KV, 1, kAnywhere>, g, b, 0, s, k);   // (its partners take the room: 83 us, 2 rows with spills 96)
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_rows(const RowsArgs& a, cudaStream_t s) {
  RowsK k{};
  const void* src[3] = {a.q, a.k, a.v};
  void* dst[3] = {a.q_out, a.k_out, a.v_out};
  const long long stride[3] = {a.q_stride, a.k_stride, a.v_stride};
  for (int i = 0; i < 3; ++i) {
    k.src[i] = static_cast<const __nv_bfloat16*>(src[i]);
    k.dst[i] = static_cast<__nv_bfloat16*>(dst[i]);
    k.stride[i] = stride[i];
  }
  k.weight[0] = static_cast<const __nv_bfloat16*>(a.q_weight);
  k.weight[1] = static_cast<const __nv_bfloat16*>(a.k_weight);
  k.slab[0] = static_cast<uint8_t*>(a.k_slab);
  k.slab[1] = static_cast<uint8_t*>(a.v_slab);
  k.scale[0] = a.k_scale;
  k.scale[1] = a.v_scale;
  k.positions = a.positions;
  k.slots = a.slots;
  k.steps = a.steps;
  k.err = a.err;
  k.T = a.T;
  k.Hq = a.Hq;
  k.Hkv = a.Hkv;
  k.nq = a.q ? a.Hq : 0;
  k.rows = k.nq + (a.k ? 2 * a.Hkv : 0);
  k.half8 = a.rotary_dim / 16;
  k.norm = a.norm;
  k.page_size = a.page_size;
  k.num_pages = a.num_pages;
  k.eps = a.eps;
  k.offset = a.weight_offset;
  k.by_page = FastDiv(a.page_size);
  switch (a.kv_dtype) {
    case FA_KV_INT8: return a.D == 256 ? launch_rows_t<256, FA_KV_INT8>(k, s) : launch_rows_t<512, FA_KV_INT8>(k, s);
    case FA_KV_FP8: return a.D == 256 ? launch_rows_t<256, FA_KV_FP8>(k, s) : launch_rows_t<512, FA_KV_FP8>(k, s);
    case FA_KV_FP4: return a.D == 256 ? launch_rows_t<256, FA_KV_FP4>(k, s) : launch_rows_t<512, FA_KV_FP4>(k, s);
    default: return a.D == 256 ? launch_rows_t<256, FA_KV_BF16>(k, s) : launch_rows_t<512, FA_KV_BF16>(k, s);
  }
}

}  // namespace fa
