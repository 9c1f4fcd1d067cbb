// One (token, KV head) row of k or v moved into its slab row by one warp:
// bf16 copied verbatim, or quantised to an 8-bit per-token-head format
// ("FreeToken PR #898", description: one fp32 scale per token and head;
// int8 codes in [-127, 127], or fp8 e4m3 codes) or to microscaled 4-bit codes.
// Used by the store kernel and by the decode kernels that store the current
// token themselves, so both write identical bytes.  The reverse, a slab row
// read back as bf16, is raw_load and raw_to_bf16 below.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cstdint>

#include "fa.h"

namespace fa {

template <int D>
struct RowRegs {
  static constexpr int NV = D / 256;   // 16-byte vectors (8 bf16) per lane
  uint4 v[NV];
};

template <int D>
__device__ __forceinline__ void row_load(RowRegs<D>& r, const __nv_bfloat16* src, int lane) {
  const uint4* s = reinterpret_cast<const uint4*>(src);
#pragma unroll
  for (int i = 0; i < RowRegs<D>::NV; ++i) r.v[i] = __ldg(s + i * 32 + lane);
}

template <int D>
__device__ __forceinline__ void row_store_bf16(const RowRegs<D>& r, __nv_bfloat16* dst, int lane) {
  uint4* d = reinterpret_cast<uint4*>(dst);
#pragma unroll
  for (int i = 0; i < RowRegs<D>::NV; ++i) d[i * 32 + lane] = r.v[i];
}

__device__ __forceinline__ void bf16x8_to_f32(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// a = max |x| (fp32), s = a / 127, c = rint(x / s) clamped to [-127, 127],
// both divisions IEEE round-to-nearest; a = 0 gives s = 0 and all-zero codes.
// Lane l holds values [i * 256 + 8 l, i * 256 + 8 l + 8) of the row.
template <int D>
__device__ __forceinline__ void row_store_int8(const RowRegs<D>& r, int8_t* dst, float* scale, int lane) {
  constexpr int NV = RowRegs<D>::NV;
  float x[NV][8];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    bf16x8_to_f32(r.v[i], x[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[i][e]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float s = __fdiv_rn(amax, 127.0f);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    uint32_t packed[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      int c = 0;
      if (amax != 0.0f) {
        float qv = rintf(__fdiv_rn(x[i][e], s));
        qv = fminf(fmaxf(qv, -127.0f), 127.0f);
        c = static_cast<int>(qv);
      }
      packed[e >> 2] |= (static_cast<uint32_t>(c) & 0xffu) << (8 * (e & 3));
    }
    *reinterpret_cast<uint2*>(dst + i * 256 + lane * 8) = make_uint2(packed[0], packed[1]);
  }
  if (lane == 0) *scale = s;
}

// a = max |x| (fp32), s = a / 448 (IEEE), c = the e4m3 value nearest to the
// IEEE quotient x / s, ties to the even mantissa, saturating at the largest
// finite magnitude 448; a = 0 gives s = 0 and all-zero codes.  Same lane
// layout as row_store_int8.
template <int D>
__device__ __forceinline__ void row_store_fp8(const RowRegs<D>& r, uint8_t* dst, float* scale, int lane) {
  constexpr int NV = RowRegs<D>::NV;
  float x[NV][8];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    bf16x8_to_f32(r.v[i], x[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[i][e]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float s = __fdiv_rn(amax, 448.0f);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    uint32_t packed[2] = {0u, 0u};
    if (amax != 0.0f) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float2 qv = make_float2(__fdiv_rn(x[i][e], s), __fdiv_rn(x[i][e + 1], s));
        // element e in the lower byte of the pair
        const uint32_t pair = __nv_cvt_float2_to_fp8x2(qv, __NV_SATFINITE, __NV_E4M3);
        packed[e >> 2] |= (pair & 0xffffu) << (8 * (e & 3));
      }
    }
    *reinterpret_cast<uint2*>(dst + i * 256 + lane * 8) = make_uint2(packed[0], packed[1]);
  }
  if (lane == 0) *scale = s;
}

// Bytes of one slab row of D values (without its fp32 scale).
template <int D, int KV>
constexpr int kRowBytes = KV == FA_KV_BF16 ? 2 * D : KV == FA_KV_FP4 ? D / 2 + D / 16 : D;

// Four pairs of fp32 values -> eight e2m1 codes, the first value in the lowest
// nibble; round to nearest, ties to the even code, saturating at 6.
__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// Eight e2m1 codes -> four f16 pairs (exact), in order of the nibbles.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t c, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(c));
}

// Two e4m3 codes (bits 0-7 and 8-15 of w) -> an f16 pair (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3);
  return static_cast<uint32_t>(h.x) | (static_cast<uint32_t>(h.y) << 16);
}

// bf16 magnitudes as integers: 2^127 is the largest a 4-bit row keeps (the
// largest code times the block scale, rounded up, still fits bf16).
constexpr uint32_t kFp4MaxBits = 0x7f00u;

// Two fp32 values in a register pair, for the packed fp32 arithmetic.
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The fp4 format (fa.h, fa_kv_dtype): the row scale 2^e, per block of 16 values
// the e4m3 scale b nearest to amax_b / (6 * 2^e), per value the e2m1 code
// nearest to x / (2^e b).  Every rounding is decided exactly without a division
// per value:
//  * amax_b * 2^-e is exact (a power of two); its product with fp32(1/6) equals
//    the midpoint of two e4m3 values exactly when the quotient does (fp32(1/6)
//    is off by 2^-25 relative, less than half a step of any midpoint, which has
//    5 significant bits), and otherwise stays on its side (the quotient of an
//    8-bit number by 6 is 2^-9 or more away from every midpoint, relatively);
//  * x * (2^-e / b), with the hardware's reciprocal (2^-23 relative), is within
//    2^-20 of the quotient where that is below 8, and rounding it to a multiple of 2^-12 (a
//    fused product and sum with 2560, whose last place is 2^-12, and the sum
//    undone) puts an exact tie between two e2m1 values, a multiple of 1/4, back
//    on the midpoint and moves nothing across one: a quotient of 8 significant
//    bits by 4 that is not on a midpoint is 2^-10 or more away from it.
//    Quotients past 8 saturate either way.
// The 8-bit formats divide each value instead and take twice as long.
// Lane l holds values [i * 256 + 8 l, i * 256 + 8 l + 8) of the row; blocks are
// lane pairs.
template <int D>
__device__ __forceinline__ void row_store_fp4(const RowRegs<D>& r, uint8_t* dst, float* scale, int lane) {
  constexpr int NV = RowRegs<D>::NV;
  uint32_t w[NV][4], blk[NV], amax;
  auto maxima = [&]() {   // blk: the block's largest magnitude (bf16 bits); amax: the row's
    uint32_t row = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      auto h = [&](int e) { return *reinterpret_cast<const __nv_bfloat162*>(&w[i][e]); };
      const __nv_bfloat162 m2 = __hmax2_nan(__hmax2_nan(__habs2(h(0)), __habs2(h(1))), __hmax2_nan(__habs2(h(2)), __habs2(h(3))));
      const uint32_t b2 = *reinterpret_cast<const uint32_t*>(&m2);
      const uint32_t m = max(b2 & 0xffffu, b2 >> 16);
      blk[i] = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      row = max(row, blk[i]);
    }
    amax = __reduce_max_sync(0xffffffffu, row);
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    w[i][0] = r.v[i].x;
    w[i][1] = r.v[i].y;
    w[i][2] = r.v[i].z;
    w[i][3] = r.v[i].w;
  }
  maxima();
  if (amax > kFp4MaxBits) {   // the whole warp: NaN becomes 0, larger magnitudes (infinities) 2^127
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t out = 0;
#pragma unroll
        for (int half = 0; half < 32; half += 16) {
          const uint32_t x = (w[i][e] >> half) & 0xffffu, mag = x & 0x7fffu;
          const uint32_t y = mag > 0x7f80u ? 0u : mag > kFp4MaxBits ? (x & 0x8000u) | kFp4MaxBits : x;
          out |= y << half;
        }
        w[i][e] = out;
      }
    maxima();
  }
  // amax = (1 + m / 128) 2^(p - 127); 2688 = 1.3125 * 2^11 and 0.3125 * 128 = 40
  const int p = static_cast<int>(amax >> 7), m = static_cast<int>(amax & 127u);
  const int e = max(p - 127 - 11 + (m > 40 ? 1 : 0), -116);
  const float inv_s = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const float ab = __uint_as_float(blk[i] << 16) * inv_s;
    const uint32_t sb = __nv_cvt_float_to_fp8(__fmul_rn(ab, 1.0f / 6.0f), __NV_SATFINITE, __NV_E4M3);
    const float b = __half2float(__ushort_as_half(static_cast<unsigned short>(e4m3x2_to_f16x2(sb) & 0xffffu)));
    const float t = sb ? inv_s * rcp_approx(b) : 0.0f;
    const uint64_t t2 = pack_f32x2(t, t), c2 = pack_f32x2(2560.0f, 2560.0f), n2 = pack_f32x2(-2560.0f, -2560.0f);
    float q[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint64_t x2 = pack_f32x2(__uint_as_float(w[i][k] << 16), __uint_as_float(w[i][k] & 0xffff0000u));
      unpack_f32x2(add_f32x2(fma_f32x2(x2, t2, c2), n2), q[2 * k], q[2 * k + 1]);
    }
    uint32_t c = e2m1x8(q);
    c = (c & 0x77777777u) | (c & ((c | (c >> 1) | (c >> 2)) << 3) & 0x88888888u);   // no negative zeros
    *reinterpret_cast<uint32_t*>(dst + i * 128 + lane * 4) = c;
    if (!(lane & 1)) dst[D / 2 + i * 16 + (lane >> 1)] = static_cast<uint8_t>(sb);
  }
  if (lane == 0) *scale = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// A slab row as it lies in memory, this lane's values [i * 256 + 8 l, ... + 8).
// (Read through L2: the row may have been written by the kernel this one was
// launched behind.)
template <int D, int KV>
struct RawRow {
  static constexpr int NV = RowRegs<D>::NV;
  uint32_t c[NV][KV == FA_KV_BF16 ? 4 : KV == FA_KV_FP4 ? 1 : 2];   // codes
  uint32_t b[KV == FA_KV_FP4 ? NV : 1];                              // fp4: the block's scale
  float s;
};

template <int D, int KV>
__device__ __forceinline__ void raw_load(RawRow<D, KV>& r, const uint8_t* row, const float* scale, int lane) {
#pragma unroll
  for (int i = 0; i < RawRow<D, KV>::NV; ++i) {
    if constexpr (KV == FA_KV_BF16) {
      const uint4 x = __ldcg(reinterpret_cast<const uint4*>(row) + i * 32 + lane);
      r.c[i][0] = x.x;
      r.c[i][1] = x.y;
      r.c[i][2] = x.z;
      r.c[i][3] = x.w;
    } else if constexpr (KV == FA_KV_FP4) {
      r.c[i][0] = __ldcg(reinterpret_cast<const uint32_t*>(row) + i * 32 + lane);
      r.b[i] = __ldcg(row + D / 2 + i * 16 + (lane >> 1));
    } else {
      const uint2 x = __ldcg(reinterpret_cast<const uint2*>(row) + i * 32 + lane);
      r.c[i][0] = x.x;
      r.c[i][1] = x.y;
    }
  }
  if constexpr (KV != FA_KV_BF16) r.s = __ldcg(scale);
}

// The row's values as bf16.  fp4: code * (block scale * row scale) is exact in
// fp32 and in bf16; the 8-bit formats round code * scale to fp32, then to bf16.
template <int D, int KV>
__device__ __forceinline__ void raw_to_bf16(const RawRow<D, KV>& r, __nv_bfloat16* dst, int lane) {
#pragma unroll
  for (int i = 0; i < RawRow<D, KV>::NV; ++i) {
    uint32_t o[4];
    if constexpr (KV == FA_KV_BF16) {
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = r.c[i][k];
    } else {
      float x[8];
      float s = r.s;
      if constexpr (KV == FA_KV_FP4) {
        uint32_t h[4];
        e2m1x8_to_f16(r.c[i][0], h);
        s *= __half2float(__ushort_as_half(static_cast<unsigned short>(e4m3x2_to_f16x2(r.b[i]) & 0xffffu)));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
          x[2 * k] = f.x;
          x[2 * k + 1] = f.y;
        }
      } else if constexpr (KV == FA_KV_FP8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t h = e4m3x2_to_f16x2((r.c[i][k >> 1] >> (16 * (k & 1))) & 0xffffu);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
          x[2 * k] = f.x;
          x[2 * k + 1] = f.y;
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = static_cast<float>(static_cast<int8_t>(r.c[i][k >> 2] >> (8 * (k & 3))));
      }
      const uint64_t s2 = pack_f32x2(s, s);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float lo, hi;
        unpack_f32x2(mul_f32x2(pack_f32x2(x[2 * k], x[2 * k + 1]), s2), lo, hi);
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        o[k] = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
    *(reinterpret_cast<uint4*>(dst) + i * 32 + lane) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// The slab format's per-row store: KV is the fa_kv_dtype of the slab.
template <int D, int KV>
__device__ __forceinline__ void row_store(const RowRegs<D>& r, void* dst, float* scale, int lane) {
  if constexpr (KV == FA_KV_BF16) row_store_bf16<D>(r, static_cast<__nv_bfloat16*>(dst), lane);
  else if constexpr (KV == FA_KV_INT8) row_store_int8<D>(r, static_cast<int8_t*>(dst), scale, lane);
  else if constexpr (KV == FA_KV_FP8) row_store_fp8<D>(r, static_cast<uint8_t*>(dst), scale, lane);
  else row_store_fp4<D>(r, static_cast<uint8_t*>(dst), scale, lane);
}

}  // namespace fa
