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
// A memory pass: each row read once, written once (rows out, slab).  A warp takes
// RH rows of one token, so that a token's sines serve several heads and RH * D / 256
// 16-byte loads are in flight per lane.
#include <algorithm>

#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_row.cuh"

namespace fa {

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
  FastDiv by_groups, by_page;
};

// Cosines and sines of pairs 8 c .. 8 c + 7 at position pos.
__device__ __forceinline__ void turns8(const uint64_t* steps, int c, int pos, float (&cs)[8], float (&sn)[8]) {
  const ulonglong2* s = reinterpret_cast<const ulonglong2*>(steps) + 4 * c;
  const uint64_t p = static_cast<uint64_t>(static_cast<int64_t>(pos));
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const ulonglong2 w = __ldg(s + e);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int32_t phase = static_cast<int32_t>(static_cast<uint32_t>((p * (k ? w.y : w.x)) >> 32));
      const float a = static_cast<float>(phase) * 1.4629180792671596e-9f;   // pi / 2^31
      cs[2 * e + k] = __cosf(a);
      sn[2 * e + k] = __sinf(a);
    }
  }
}

template <int D>
__device__ __forceinline__ float row_square_sum(const RowRegs<D>& r, float pre) {
  float s0 = 0.f, s1 = 0.f;
#pragma unroll
  for (int i = 0; i < RowRegs<D>::NV; ++i) {
    float x[8];
    bf16x8_to_f32(r.v[i], x);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      s0 = fmaf(x[e] * pre, x[e] * pre, s0);
      s1 = fmaf(x[e + 1] * pre, x[e + 1] * pre, s1);
    }
  }
  return s0 + s1;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// FULL: the whole head is rotated (R = D), and pairs sit in one lane (D = 512:
// vectors l and l + 32) or 16 lanes apart (D = 256).  Otherwise partners meet
// through a row of shared memory.
template <int D, int KV, int RH, bool FULL>
__global__ void __launch_bounds__(256) rows_kernel(const __grid_constant__ RowsK a) {
  constexpr int NV = RowRegs<D>::NV;
  constexpr int NC = FULL ? 1 : NV;   // sets of 8 cosines a lane needs
  __shared__ float4 meet[FULL ? 1 : 8 * D / 4];
  // Index arrays are read after the wait even under FA_FLAG_EARLY_METADATA: they
  // usually come from the kernel before (fa_plan_step).
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const uint32_t warp = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const uint32_t t = a.by_groups.div(warp);
  if (t >= static_cast<uint32_t>(a.T)) return;
  const int r0 = static_cast<int>(warp - t * a.by_groups.d) * RH;
  auto kind_of = [&](int row) { return row < a.nq ? 0 : row < a.nq + a.Hkv ? 1 : 2; };
  auto head_of = [&](int row, int kind) { return row - (kind == 0 ? 0 : kind == 1 ? a.nq : a.nq + a.Hkv); };

  RowRegs<D> r[RH];
#pragma unroll
  for (int i = 0; i < RH; ++i) {
    const int row = r0 + i;
    if (row < a.rows) {
      const int kind = kind_of(row);
      const uint4* s = reinterpret_cast<const uint4*>(a.src[kind] + static_cast<size_t>(t) * a.stride[kind] +
                                                      static_cast<size_t>(head_of(row, kind)) * D);
#pragma unroll
      for (int j = 0; j < NV; ++j) r[i].v[j] = s[j * 32 + lane];
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) r[i].v[j] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  const bool turned = a.half8 > 0 && kind_of(r0) < 2;
  float cs[NC][8], sn[NC][8];
  int part[NV];   // 0: first of its pair, 1: second, 2: not rotated
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int v = j * 32 + lane;
    part[j] = v < a.half8 ? 0 : v < 2 * a.half8 ? 1 : 2;
  }
  if (turned) {
    const int pos = __ldg(a.positions + t);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int v = j * 32 + lane;
      const int c = FULL ? (D == 256 ? lane & 15 : lane) : part[j] == 0 ? v : part[j] == 1 ? v - a.half8 : 0;
      turns8(a.steps, c, pos, cs[j], sn[j]);
    }
  }
  float ss[RH];
#pragma unroll
  for (int i = 0; i < RH; ++i) ss[i] = row_square_sum<D>(r[i], 1.0f);
#pragma unroll
  for (int i = 0; i < RH; ++i) ss[i] = warp_sum(ss[i]);
  const int slot = a.slots && r0 + RH > a.nq ? __ldg(a.slots + t) : -1;

#pragma unroll
  for (int i = 0; i < RH; ++i) {
    const int row = r0 + i;
    if (row >= a.rows) break;
    const int kind = kind_of(row), head = head_of(row, kind);
    const bool norm = (a.norm >> kind) & 1, turn = turned && kind < 2;
    if (norm || turn) {   // (else the row goes on bit for bit)
      float f = 1.0f;
      if (norm) {
        if (ss[i] <= 1e38f) {
          f = rsqrtf(fmaf(ss[i], 1.0f / D, a.eps));
        } else {   // squares past fp32 (magnitudes near 2^64), infinities, NaN: the row over 2^70
          constexpr float pre = 8.470329472543003e-22f;
          f = pre * rsqrtf(warp_sum(row_square_sum<D>(r[i], pre)) * (1.0f / D));
        }
      }
      float y[NV][8];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        bf16x8_to_f32(r[i].v[j], y[j]);
        if (norm) {
#pragma unroll
          for (int e = 0; e < 8; ++e) y[j][e] *= f;
          if (kind < 2 && a.weight[kind]) {
            float w[8];
            bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(a.weight[kind]) + j * 32 + lane), w);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[j][e] *= w[e] + a.offset;
          }
        }
      }
      if (turn) {
        float z[NV][8];   // the partners
        if constexpr (FULL && D == 512) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            z[0][e] = y[NV - 1][e];
            z[NV - 1][e] = y[0][e];
          }
        } else if constexpr (FULL) {
#pragma unroll
          for (int e = 0; e < 8; ++e) z[0][e] = __shfl_xor_sync(0xffffffffu, y[0][e], 16);
        } else {
          float4* m = meet + (threadIdx.x >> 5) * (D / 4);
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            m[2 * (j * 32 + lane)] = make_float4(y[j][0], y[j][1], y[j][2], y[j][3]);
            m[2 * (j * 32 + lane) + 1] = make_float4(y[j][4], y[j][5], y[j][6], y[j][7]);
          }
          __syncwarp();
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            const int v = j * 32 + lane, o = part[j] == 0 ? v + a.half8 : part[j] == 1 ? v - a.half8 : v;
            const float4 lo = m[2 * o], hi = m[2 * o + 1];
            z[j][0] = lo.x, z[j][1] = lo.y, z[j][2] = lo.z, z[j][3] = lo.w;
            z[j][4] = hi.x, z[j][5] = hi.y, z[j][6] = hi.z, z[j][7] = hi.w;
          }
          __syncwarp();
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          if (part[j] == 2) continue;
          const float sign = part[j] == 0 ? -1.0f : 1.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) y[j][e] = fmaf(y[j][e], cs[j % NC][e], sign * z[j][e] * sn[j % NC][e]);
        }
      }
#pragma unroll
      for (int j = 0; j < NV; ++j)
        r[i].v[j] = make_uint4(pack_bf16x2(y[j][0], y[j][1]), pack_bf16x2(y[j][2], y[j][3]), pack_bf16x2(y[j][4], y[j][5]),
                               pack_bf16x2(y[j][6], y[j][7]));
    }
    if (a.dst[kind])
      row_store_bf16<D>(r[i], a.dst[kind] + (static_cast<size_t>(t) * (kind == 0 ? a.Hq : a.Hkv) + head) * D, lane);
    if (kind == 0 || slot < 0) continue;   // a negative slot is a padding token
    const uint32_t page = a.by_page.div(slot), off = slot - page * a.page_size;
    if (page >= static_cast<uint32_t>(a.num_pages)) {
      if (lane == 0) atomicOr(a.err, FA_DEV_ERR_SLOT);
      continue;
    }
    const size_t to = (static_cast<size_t>(page) * a.Hkv + head) * a.page_size + off;
    row_store<D, KV>(r[i], a.slab[kind - 1] + to * kRowBytes<D, KV>, KV == FA_KV_BF16 ? nullptr : a.scale[kind - 1] + to, lane);
  }
}

template <int D, int KV>
static cudaError_t launch_rows_t(RowsK k, cudaStream_t s) {
  constexpr int RH = D == 256 ? 8 : 4;
  const long long all = static_cast<long long>(k.T) * k.rows;
  // few rows: a warp each, for the shortest path; many: RH a warp
  const int rh = all <= 64LL * sm_count() ? 1 : RH;
  const int groups = (k.rows + rh - 1) / rh;
  const long long warps = static_cast<long long>(k.T) * groups;
  if (warps >= (1LL << 31) - 8) return cudaErrorInvalidConfiguration;
  k.by_groups = FastDiv(groups);
  const int block = rh == 1 && warps < 8LL * sm_count() ? 64 : 256;
  const dim3 g(static_cast<unsigned>((warps * 32 + block - 1) / block)), b(block);
  const bool full = k.half8 * 16 == D;
  if (rh == 1) return full ? launch_pdl(rows_kernel<D, KV, 1, true>, g, b, 0, s, k) : launch_pdl(rows_kernel<D, KV, 1, false>, g, b, 0, s, k);
  return full ? launch_pdl(rows_kernel<D, KV, RH, true>, g, b, 0, s, k) : launch_pdl(rows_kernel<D, KV, RH, false>, g, b, 0, s, k);
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
