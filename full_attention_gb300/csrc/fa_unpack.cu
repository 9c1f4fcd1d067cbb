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
#include <algorithm>

#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_row.cuh"

namespace fa {

constexpr long long kMaxBlocks = 16384;

template <int D>
__global__ void __launch_bounds__(256, 6) unpack_kernel(UnpackArgs a) {
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
    RawRow<D, FA_KV_FP4> raw[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (there && pos0 + i / 2 < last) {
        const size_t r = src + i / 2;
        raw_load<D, FA_KV_FP4>(raw[i], static_cast<const uint8_t*>((i & 1) ? a.v_slab : a.k_slab) + r * kRowBytes<D, FA_KV_FP4>,
                               ((i & 1) ? a.v_scale : a.k_scale) + r, lane);
      } else {
        raw[i] = RawRow<D, FA_KV_FP4>{};
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (pos0 + i / 2 >= last) continue;
      raw_to_bf16<D, FA_KV_FP4>(raw[i], static_cast<__nv_bfloat16*>((i & 1) ? a.v : a.k) + (dst + i / 2) * D, lane);
    }
  }
  griddep_wait();   // the grid ends only after the kernel before it
}

cudaError_t launch_unpack(const UnpackArgs& args, cudaStream_t s) {
  UnpackArgs a = args;
  a.by_page = FastDiv(a.page_size);
  a.by_ring = FastDiv(a.ring);
  const int per_block = 8 * (a.D == 256 ? 4 : 2);   // positions
  const int span = a.ring < a.max_len ? a.ring : a.max_len;
  const long long gy = static_cast<long long>(a.B) * a.Hkv;
  if (gy > 65535) return cudaErrorInvalidConfiguration;   // the caller takes the direct path
  // the bound may be far above the lengths, and blocks that find nothing cost their
  // launch: 8 prefixes of 1000 rows, 2 KV heads at 512, under a bound of 131072 took
  // 176 us with a block for every 16 rows of it, 62 with these, 54 with 4096 (which
  // cost 64 prefixes of 4096 rows 538 us for 529); converting in the kernel 93
  const long long most = std::max(1LL, (kMaxBlocks + gy - 1) / gy);
  const dim3 g(static_cast<unsigned>(std::min<long long>((span + per_block - 1) / per_block, most)), static_cast<unsigned>(gy)), b(256);
  return a.D == 256 ? launch_pdl(unpack_kernel<256>, g, b, 0, s, a) : launch_pdl(unpack_kernel<512>, g, b, 0, s, a);
}

}  // namespace fa
