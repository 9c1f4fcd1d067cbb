// Paged KV store: scatter post-RoPE k, v rows of new tokens into their slots
// ("FreeToken PR #898", description bullet on store_kv; "unsloth commit
// dee9371": the store layer writes its post-rotary k, v into its paged cache).
//
// One warp moves one (token, KV head, K-or-V) row with 16-byte vector loads
// and stores.  The 8-bit per-token-head formats quantise the row on the way:
// a = max|x| (fp32, warp-shuffle reduction); int8: s = a / 127, c = rint(x / s)
// clamped to [-127, 127]; fp8: s = a / 448, c = the e4m3 value nearest x / s,
// saturating at 448; every division IEEE round-to-nearest.  The microscaled
// 4-bit format is in fa_row.cuh (row_store_fp4).
//
// The reverse, fa_kv_load, reads rows back as bf16.
#include <algorithm>
#include <cstdio>
#include <mutex>

#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_row.cuh"

// Device error words: one per live cache descriptor (the cache's slot), where
// every kernel a call on that cache launches ORs its FA_DEV_ERR_* bits.
// File-scope device storage: nothing is allocated for them.
__device__ unsigned int g_fa_device_error[FA_MAX_CACHES];

namespace fa {

// Base of the error words on the current device.  In host code the array's
// name is a host-side stand-in, so its device address is looked up once per
// device, with that device current.
static unsigned int* device_error_words(cudaError_t* err) {
  static std::mutex mu;
  static unsigned int* ptrs[128] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 128) {
    *err = e != cudaSuccess ? e : cudaErrorInvalidDevice;
    return nullptr;
  }
  std::lock_guard<std::mutex> lock(mu);
  if (!ptrs[dev]) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_fa_device_error);
    if (e != cudaSuccess) {
      *err = e;
      return nullptr;
    }
    ptrs[dev] = static_cast<unsigned int*>(p);
  }
  *err = cudaSuccess;
  return ptrs[dev];
}

unsigned int* device_error_word(const fa_cache* c, cudaError_t* err) {
  unsigned int* base = device_error_words(err);
  return base ? base + c->err_slot : nullptr;
}

cudaError_t clear_device_error_word(const fa_cache* c) {
  cudaError_t e;
  unsigned int* w = device_error_word(c, &e);
  if (!w) return e;
  const unsigned int zero = 0;
  return cudaMemcpy(w, &zero, sizeof(zero), cudaMemcpyHostToDevice);
}

// R consecutive (token, KV head, K or V) rows per warp, `warp` counting the
// launch's warps for this layer.  The warp loads the R slots, then (once the
// previous kernel's rows may be read) all R rows, whose addresses do not
// depend on the slots, then stores them: R * D / 256 16-byte vectors per lane
// in flight behind one load latency.  Row t * Hkv * 2 + 2 h (+1) is token t's
// K (V) row of KV head h.
template <int D>
struct StoreShape {
  static constexpr int R = D == 256 ? 8 : 4;   // rows per warp: 128 bytes per lane in flight
};

template <int D, int KV>
__device__ __forceinline__ void store_rows(const StoreArgs& a, int warp, int lane) {
  constexpr int R = StoreShape<D>::R;
  const int rows = a.T * a.Hkv * 2;
  const int r0 = warp * R;
  if (r0 >= rows) return;
  int slot[R];
#pragma unroll
  for (int i = 0; i < R; ++i) slot[i] = (r0 + i < rows) ? __ldg(a.slots + ((r0 + i) >> 1) / a.Hkv) : -1;
  griddep_wait();   // the rows (and the slab) may belong to the previous kernel
  RowRegs<D> r[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (r0 + i < rows)
      row_load<D>(r[i], static_cast<const __nv_bfloat16*>(((r0 + i) & 1) ? a.v : a.k) +
                            static_cast<size_t>((r0 + i) >> 1) * D, lane);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int row = r0 + i;
    if (row >= rows || slot[i] < 0) continue;   // a negative slot is a padding token
    const int page = slot[i] / a.page_size, off = slot[i] % a.page_size;
    if (page >= a.num_pages) {
      if (lane == 0) atomicOr(a.err, FA_DEV_ERR_SLOT);
      continue;
    }
    const int h = (row >> 1) % a.Hkv;
    const size_t dst = (static_cast<size_t>(page) * a.Hkv + h) * a.page_size + off;
    const int which = row & 1;
    row_store<D, KV>(r[i], static_cast<uint8_t*>(which ? a.v_slab : a.k_slab) + dst * kRowBytes<D, KV>,
                     KV == FA_KV_BF16 ? nullptr : (which ? a.v_scale : a.k_scale) + dst, lane);
  }
}

// fp4: the same with the warp's R rows those of R consecutive tokens for one
// (KV head, K or V).  Tokens stored together mostly lie in consecutive slots, so
// the warp's 144- or 288-byte rows and their scales are neighbours in the slab
// and share their sectors.  A memory pass whose arithmetic just fits beside it at
// head_dim 512: 30011 tokens of 2 KV heads, 158 MB, take 27 us, 5.8 TB/s of 6.8;
// at 256 it does not quite: 8192 tokens of 8 KV heads, 86 MB, 18 us (with a
// reciprocal rounded to the last place 30 and 21 us).
template <int D>
__device__ __forceinline__ void store_rows_fp4(const StoreArgs& a, int warp, int lane) {
  constexpr int R = StoreShape<D>::R;
  const uint32_t per = 2 * a.Hkv;
  const uint32_t tg = a.by_rows.div(warp), q = warp - tg * per;   // token group, 2 h + side
  const int t0 = static_cast<int>(tg) * R;
  if (t0 >= a.T) return;
  const uint32_t h = q >> 1, which = q & 1;
  int slot[R];
#pragma unroll
  for (int i = 0; i < R; ++i) slot[i] = (t0 + i < a.T) ? __ldg(a.slots + t0 + i) : -1;
  griddep_wait();   // the rows (and the slab) may belong to the previous kernel
  RowRegs<D> r[R];
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(which ? a.v : a.k) + (static_cast<size_t>(t0) * a.Hkv + h) * D;
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (t0 + i < a.T) row_load<D>(r[i], src + static_cast<size_t>(i) * a.Hkv * D, lane);
  uint8_t* slab = static_cast<uint8_t*>(which ? a.v_slab : a.k_slab);
  float* scale = which ? a.v_scale : a.k_scale;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (slot[i] < 0) continue;   // a padding token
    const uint32_t page = a.by_page.div(slot[i]), off = slot[i] - page * a.page_size;
    if (page >= static_cast<uint32_t>(a.num_pages)) {
      if (lane == 0) atomicOr(a.err, FA_DEV_ERR_SLOT);
      continue;
    }
    const size_t dst = (page * a.Hkv + h) * a.page_size + off;   // below 2^31 (fa_cache_create)
    row_store_fp4<D>(r[i], slab + dst * kRowBytes<D, FA_KV_FP4>, scale + dst, lane);
  }
}

template <int D, int KV>
__device__ __forceinline__ void store_warp(const StoreArgs& a, int warp, int lane) {
  if constexpr (KV == FA_KV_FP4) store_rows_fp4<D>(a, warp, lane);
  else store_rows<D, KV>(a, warp, lane);
}

template <int D, int KV>
__global__ void __launch_bounds__(256) store_kernel(StoreArgs a) {
  if (!a.early_metadata) griddep_wait();
  griddep_launch_dependents();
  store_warp<D, KV>(a, (blockIdx.x * blockDim.x + threadIdx.x) >> 5, threadIdx.x & 31);
}

// Several layers' stores in one launch: blockIdx.y picks the layer.
struct StoreLayers {
  StoreArgs a[kMaxLayersPerLaunch];
};

template <int KV>
__global__ void __launch_bounds__(256) store_layers_kernel(const __grid_constant__ StoreLayers m) {
  const StoreArgs& a = m.a[blockIdx.y];
  if (!a.early_metadata) griddep_wait();
  griddep_launch_dependents();
  const int warp = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
  if (a.D == 256) store_warp<256, KV>(a, warp, lane);
  else store_warp<512, KV>(a, warp, lane);
}

// Warps a store of T tokens needs.
static long store_warps(const StoreArgs& a) {
  const long rows = static_cast<long>(a.T) * a.Hkv * 2;
  const int R = a.D == 256 ? StoreShape<256>::R : StoreShape<512>::R;
  if (a.kv_dtype == FA_KV_FP4) return static_cast<long>((a.T + R - 1) / R) * a.Hkv * 2;
  return (rows + R - 1) / R;
}

static StoreArgs with_divs(StoreArgs a) {
  a.by_page = FastDiv(a.page_size);
  a.by_rows = FastDiv(2 * a.Hkv);
  return a;
}

cudaError_t launch_store_layers(const StoreArgs* a, int n, cudaStream_t s) {
  if (n < 1 || n > kMaxLayersPerLaunch) return cudaErrorInvalidValue;
  StoreLayers m{};
  long warps = 0;
  for (int i = 0; i < n; ++i) {
    m.a[i] = with_divs(a[i]);
    warps = std::max(warps, store_warps(a[i]));
  }
  const int block = 256;
  const long grid = (warps * 32 + block - 1) / block;
  if (grid > 0x7fffffffL) return cudaErrorInvalidValue;
  const dim3 g(static_cast<unsigned>(grid), static_cast<unsigned>(n)), b(block);
  if (a[0].kv_dtype == FA_KV_INT8) return launch_pdl(store_layers_kernel<FA_KV_INT8>, g, b, 0, s, m);
  if (a[0].kv_dtype == FA_KV_FP8) return launch_pdl(store_layers_kernel<FA_KV_FP8>, g, b, 0, s, m);
  if (a[0].kv_dtype == FA_KV_FP4) return launch_pdl(store_layers_kernel<FA_KV_FP4>, g, b, 0, s, m);
  return launch_pdl(store_layers_kernel<FA_KV_BF16>, g, b, 0, s, m);
}

cudaError_t launch_store(const StoreArgs& args, cudaStream_t s) {
  const StoreArgs a = with_divs(args);
  const long warps = store_warps(a);
  const int block = 256;
  const long grid = (warps * 32 + block - 1) / block;
  if (grid > 0x7fffffffL) return cudaErrorInvalidValue;
  const dim3 g(static_cast<unsigned>(grid)), b(block);
  if (a.kv_dtype == FA_KV_INT8)
    return a.D == 256 ? launch_pdl(store_kernel<256, FA_KV_INT8>, g, b, 0, s, a)
                      : launch_pdl(store_kernel<512, FA_KV_INT8>, g, b, 0, s, a);
  if (a.kv_dtype == FA_KV_FP8)
    return a.D == 256 ? launch_pdl(store_kernel<256, FA_KV_FP8>, g, b, 0, s, a)
                      : launch_pdl(store_kernel<512, FA_KV_FP8>, g, b, 0, s, a);
  if (a.kv_dtype == FA_KV_FP4)
    return a.D == 256 ? launch_pdl(store_kernel<256, FA_KV_FP4>, g, b, 0, s, a)
                      : launch_pdl(store_kernel<512, FA_KV_FP4>, g, b, 0, s, a);
  return a.D == 256 ? launch_pdl(store_kernel<256, FA_KV_BF16>, g, b, 0, s, a)
                    : launch_pdl(store_kernel<512, FA_KV_BF16>, g, b, 0, s, a);
}

// The reverse, any format: a warp's R rows are those of R consecutive tokens for
// one (KV head, K or V).  Slots, then every row's raw bytes, then the rows out:
// loads in flight are what it needs.  fp4, the shapes above: 26 and 15 us.
template <int D, int KV>
__global__ void __launch_bounds__(256) load_kernel(LoadArgs a) {
  constexpr int R = StoreShape<D>::R;
  if (!a.early_metadata) griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const uint32_t sides = a.k && a.v ? 2 : 1;
  const uint32_t warp = (blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const uint32_t tg = a.by_rows.div(warp), q = warp - tg * a.by_rows.d;
  const long long t0 = static_cast<long long>(tg) * R;
  if (t0 >= a.T) {
    griddep_wait();   // the grid ends only after the kernel before it
    return;
  }
  const uint32_t h = sides == 2 ? q >> 1 : q;
  const bool which = sides == 2 ? (q & 1) : a.v != nullptr;
  int slot[R];
#pragma unroll
  for (int i = 0; i < R; ++i) slot[i] = (t0 + i < a.T) ? __ldg(a.slots + t0 + i) : -1;
  griddep_wait();   // the slab's rows may belong to the previous kernel
  const uint8_t* slab = static_cast<const uint8_t*>(which ? a.v_slab : a.k_slab);
  const float* scale = which ? a.v_scale : a.k_scale;
  RawRow<D, KV> raw[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (slot[i] < 0) continue;   // a padding token: its rows stay as they are
    const uint32_t page = a.by_page.div(slot[i]), off = slot[i] - page * a.page_size;
    if (page >= static_cast<uint32_t>(a.num_pages)) {
      if (lane == 0) atomicOr(a.err, FA_DEV_ERR_SLOT);
      slot[i] = -1;
      continue;
    }
    const size_t src = (page * a.Hkv + h) * a.page_size + off;   // below 2^31 (fa_cache_create)
    raw_load<D, KV>(raw[i], slab + src * kRowBytes<D, KV>, scale + src, lane);
  }
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(which ? a.v : a.k) + (static_cast<size_t>(t0) * a.Hkv + h) * D;
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (slot[i] >= 0) raw_to_bf16<D, KV>(raw[i], dst + static_cast<size_t>(i) * a.Hkv * D, lane);
}

cudaError_t launch_load(const LoadArgs& args, cudaStream_t s) {
  LoadArgs a = args;
  const int R = a.D == 256 ? StoreShape<256>::R : StoreShape<512>::R;
  const int per = a.Hkv * (a.k && a.v ? 2 : 1);
  a.by_page = FastDiv(a.page_size);
  a.by_rows = FastDiv(per);
  const long long warps = (static_cast<long long>(a.T) + R - 1) / R * per;
  const int block = 256;
  const long long grid = (warps * 32 + block - 1) / block;
  if (warps >= (1LL << 31) - 8) return cudaErrorInvalidValue;
  const dim3 g(static_cast<unsigned>(grid)), b(block);
  auto run = [&](auto k256, auto k512) {
    return a.D == 256 ? launch_pdl(k256, g, b, 0, s, a) : launch_pdl(k512, g, b, 0, s, a);
  };
  if (a.kv_dtype == FA_KV_INT8) return run(load_kernel<256, FA_KV_INT8>, load_kernel<512, FA_KV_INT8>);
  if (a.kv_dtype == FA_KV_FP8) return run(load_kernel<256, FA_KV_FP8>, load_kernel<512, FA_KV_FP8>);
  if (a.kv_dtype == FA_KV_FP4) return run(load_kernel<256, FA_KV_FP4>, load_kernel<512, FA_KV_FP4>);
  return run(load_kernel<256, FA_KV_BF16>, load_kernel<512, FA_KV_BF16>);
}

}  // namespace fa

extern "C" fa_status fa_get_device_error(fa_cache* cache, int32_t* code, void* stream) {
  if (!cache) return fa::fail(FA_ERR_INVALID_ARG, "cache is NULL");
  if (!code) return fa::fail(FA_ERR_INVALID_ARG, "code is NULL");
  cudaError_t ce;
  unsigned int* p = fa::device_error_word(cache, &ce);
  if (!p) return fa::fail(FA_ERR_CUDA, "device error word: %s", cudaGetErrorString(ce));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned int v = 0;
  if ((ce = cudaStreamSynchronize(s)) != cudaSuccess ||
      (ce = cudaMemcpyAsync(&v, p, sizeof(v), cudaMemcpyDeviceToHost, s)) != cudaSuccess ||
      (ce = cudaMemsetAsync(p, 0, sizeof(v), s)) != cudaSuccess || (ce = cudaStreamSynchronize(s)) != cudaSuccess)
    return fa::fail(FA_ERR_CUDA, "reading the device error word: %s", cudaGetErrorString(ce));
  *code = static_cast<int32_t>(v);
  return FA_OK;
}
