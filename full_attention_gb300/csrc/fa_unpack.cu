// The fp4 rows an extend or multi-token decode call can see, unpacked to bf16.
//
// An extend over a 4-bit slab multiplies every prefix key with every 128-row
// block of queries.  Converting codes inside the kernel repeats the conversion
// for each block and paces it: 8 sequences of 4096 keys at head_dim 512, 2 KV
// heads, 256 queries each, take 1218 us converting and 556 us unpacked.  A value of the format has 6 significant bits, so a bf16 row holds it exactly,
// and the bf16 kernel over unpacked rows does the same arithmetic without it.
// This kernel writes them: a memory pass over the rows some query can see, 0.58
// bytes in and 2 out per value, most of which the extend kernel then finds in
// L2: 11 us for 4 sequences, a window of 1024 before chunks of 512, at 256 with 8
// KV heads.
//
// The rows of sequence b and KV head h form a ring of `ring` rows (a multiple
// of 16): position pos lies in row (b * Hkv + h) * ring + pos % ring.  To the
// extend kernel that is a slab of pages of `ring` rows whose block table says b
// for every page of sequence b; the table is written here too.
//
// Differential extend over an 8-bit slab is paced by the same conversion (2753
// tokens of 5 prompts over up to 3814 keys at 512, 16 and 2 heads, fp8: 1670 us converting, 1050 over f16 rows, 17 of them here).  A
// code is exact in f16, the operands' type there, and its row's scale goes to the
// scores and weights; so this kernel writes codes as f16, their scales beside them,
// and the chunk's rows as f16 with the range's checks: operands equal in every bit to
// those of the converting path, 3 bytes a value of the prefix and 4 of the chunk.
#include <algorithm>
#include <type_traits>

#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_row.cuh"

namespace fa {

constexpr long long kMaxBlocks = 16384;

// 8-bit: the row's codes as f16, and its scale.
template <int D, int KV>
__device__ __forceinline__ void raw_to_f16(const RawRow<D, KV>& r, __half* dst, float* scale, int lane) {
#pragma unroll
  for (int i = 0; i < RawRow<D, KV>::NV; ++i) {
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t two = r.c[i][k >> 1] >> (16 * (k & 1));
      if constexpr (KV == FA_KV_FP8) o[k] = e4m3x2_to_f16x2(two & 0xffffu);
      else o[k] = pack_f16x2(static_cast<float>(static_cast<int8_t>(two)), static_cast<float>(static_cast<int8_t>(two >> 8)));
    }
    reinterpret_cast<uint4*>(dst)[i * 32 + lane] = make_uint4(o[0], o[1], o[2], o[3]);
  }
  if (lane == 0) *scale = r.s;
}

template <int D, int KV>
__global__ void __launch_bounds__(256, 6) unpack_kernel(UnpackArgs a) {
  constexpr bool F4 = KV == FA_KV_FP4;
  constexpr int R = D == 256 ? 8 : 4;   // rows a warp moves at a time, K and V alternating
  if (!a.early_metadata) griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.y / a.Hkv, h = blockIdx.y % a.Hkv;
  const int lane = threadIdx.x & 31;
  // rows [first, P): extend, the prefix; multi-token decode, the whole sequence,
  // whose last n tokens are the queries.  Nothing sees the rows of a sequence
  // without new tokens: its pages may be anyone's.
  const int fresh = min(max(__ldg(a.qo_indptr + b + 1) - __ldg(a.qo_indptr + b), 0), a.max_q_len);
  const int P = fresh > 0 ? min(__ldg(a.lens + b), a.max_len) : 0;
  const int n = a.stored ? min(fresh, P) : 0;   // (a length below the new tokens is reported by the extend kernel)
  if (blockIdx.x == 0 && h == 0) {
    griddep_wait();   // the table may still be read by the previous call's kernel
    for (int i = threadIdx.x; i < a.table_pages; i += blockDim.x) a.table[static_cast<size_t>(b) * a.table_pages + i] = b;
  }
  // the first query sees from P - W + 1 on; the extend kernel's tiles start on 16 rows
  const int first = a.window > 0 ? max(0, P - n - a.window + 1) : 0;
  const uint32_t last = first < P ? P : 0, step = gridDim.x * 8 * (R / 2);
  for (uint32_t pos0 = (first & ~15) + (blockIdx.x * 8 + (threadIdx.x >> 5)) * (R / 2); pos0 < last; pos0 += step) {
    // R / 2 divides 16, so a warp's positions share a page and lie together in the ring
    const uint32_t pg = a.by_page.div(pos0);
    const int pid = __ldg(a.block_table + static_cast<size_t>(b) * a.max_pages_per_seq + pg);
    const bool there = pid >= 0 && pid < a.num_pages;
    if (!there && lane == 0) atomicOr(a.err, FA_DEV_ERR_PAGE);   // reads as zeros
    const size_t src = there ? (static_cast<size_t>(pid) * a.Hkv + h) * a.page_size + (pos0 - pg * a.page_size) : 0;
    const size_t dst = (static_cast<size_t>(b) * a.Hkv + h) * a.ring + (pos0 - a.by_ring.div(pos0) * a.ring);
    griddep_wait();
    RawRow<D, KV> raw[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (there && pos0 + i / 2 < last) {
        const size_t r = src + i / 2;
        raw_load<D, KV>(raw[i], static_cast<const uint8_t*>((i & 1) ? a.v_slab : a.k_slab) + r * kRowBytes<D, KV>,
                        ((i & 1) ? a.v_scale : a.k_scale) + r, lane);
      } else {
        raw[i] = RawRow<D, KV>{};
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (pos0 + i / 2 >= last) continue;
      const size_t d = dst + i / 2;
      if constexpr (F4) raw_to_bf16<D, KV>(raw[i], static_cast<__nv_bfloat16*>((i & 1) ? a.v : a.k) + d * D, lane);
      else raw_to_f16<D, KV>(raw[i], static_cast<__half*>((i & 1) ? a.v : a.k) + d * D, ((i & 1) ? a.vs : a.ks) + d, lane);
    }
  }
  if constexpr (!F4) {
    // the sequence's chunk rows; values that f16 cannot hold saturate and are reported
    griddep_wait();
    const int qo0 = __ldg(a.qo_indptr + b);
    uint32_t big = 0;
    for (int t0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * (R / 2); t0 < fresh; t0 += static_cast<int>(step)) {
      RowRegs<D> row[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int t = qo0 + t0 + i / 2;
        if (t0 + i / 2 < fresh && t >= 0 && t < a.num_tokens)
          row_load(row[i], static_cast<const __nv_bfloat16*>((i & 1) ? a.v_ext : a.k_ext) + (static_cast<size_t>(t) * a.Hkv + h) * D, lane);
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int t = qo0 + t0 + i / 2;
        if (t0 + i / 2 >= fresh || t < 0 || t >= a.num_tokens) continue;
        uint4* out = reinterpret_cast<uint4*>(static_cast<__half*>((i & 1) ? a.vx : a.kx) + (static_cast<size_t>(t) * a.Hkv + h) * D);
#pragma unroll
        for (int c = 0; c < RowRegs<D>::NV; ++c) {
          uint32_t w[4] = {row[i].v[c].x, row[i].v[c].y, row[i].v[c].z, row[i].v[c].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            big |= bf16x2_past_f16(w[k]);
            w[k] = pack_f16x2_sat(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
          }
          out[c * 32 + lane] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
    if (__any_sync(0xffffffffu, big != 0) && lane == 0) atomicOr(a.err, FA_DEV_ERR_RANGE);
  }
  griddep_wait();   // the grid ends only after the kernel before it
}

cudaError_t launch_unpack(const UnpackArgs& args, cudaStream_t s) {
  UnpackArgs a = args;
  a.by_page = FastDiv(a.page_size);
  a.by_ring = FastDiv(a.ring);
  const int per_block = 8 * (a.D == 256 ? 4 : 2);   // positions
  const int span = std::max(std::min(a.ring, a.max_len), a.kv_dtype == FA_KV_FP4 ? 1 : a.max_q_len);
  const long long gy = static_cast<long long>(a.B) * a.Hkv;
  if (gy > 65535) return cudaErrorInvalidConfiguration;   // the caller takes the direct path
  // the bound may be far above the lengths, and blocks that find nothing cost their
  // launch: 8 prefixes of 1000 rows, 2 KV heads at 512, under a bound of 131072 took
  // 176 us with a block for every 16 rows of it, 62 with these, 54 with 4096 (which
  // cost 64 prefixes of 4096 rows 538 us for 529); converting in the kernel 93
  const long long most = std::max(1LL, (kMaxBlocks + gy - 1) / gy);
  const dim3 g(static_cast<unsigned>(std::min<long long>((span + per_block - 1) / per_block, most)), static_cast<unsigned>(gy)), b(256);
  auto run = [&](auto kv) {
    constexpr int KV = decltype(kv)::value;
    return a.D == 256 ? launch_pdl(unpack_kernel<256, KV>, g, b, 0, s, a) : launch_pdl(unpack_kernel<512, KV>, g, b, 0, s, a);
  };
  if (a.kv_dtype == FA_KV_INT8) return run(std::integral_constant<int, FA_KV_INT8>{});
  if (a.kv_dtype == FA_KV_FP8) return run(std::integral_constant<int, FA_KV_FP8>{});
  return run(std::integral_constant<int, FA_KV_FP4>{});
}

}  // namespace fa
