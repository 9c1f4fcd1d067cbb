// Internal declarations shared by the host API and the kernel launchers.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <vector>

#include "fa.h"

namespace fa {

// Token rows are processed in 16-row tiles: one m16 tile of the warp MMAs and
// one TMA box height.  Page sizes are multiples of it.
constexpr int kTile = 16;
// Layers one multi-layer launch can hold.
constexpr int kMaxLayersPerLaunch = FA_MAX_LAYERS_PER_LAUNCH;

struct Slab {
  void* k = nullptr;
  void* v = nullptr;
  float* k_scale = nullptr;
  float* v_scale = nullptr;
  bool bound = false;
  // TMA descriptors over K and V, 3-D: (64-element column block, block index,
  // row) with rows = num_pages * Hkv * page_size; see fa_cache_bind_slab.
  CUtensorMap tm_k;
  CUtensorMap tm_v;
  // The same slabs as (column-block element, row, column block): one box is
  // a whole 16-row tile, all column blocks, landing block-major like 16-row
  // boxes of tm_k / tm_v side by side (one copy per tile).
  CUtensorMap tm_kt;
  CUtensorMap tm_vt;
  // fp4 format: tm_k and tm_v (and tm_kt, tm_vt, unused) are 2-D maps over
  // the row bytes (codes, then block scales), boxes of 32 bytes x 16 rows.
  // Quantised formats: 2-D maps over the fp32 scales, one 16-float box per tile.
  CUtensorMap tm_ks;
  CUtensorMap tm_vs;
};

struct Layer {
  fa_layer_desc d;
  int owner = -1;   // slab owner (itself if it owns a slab)
};

}  // namespace fa

struct fa_cache {
  std::vector<fa::Layer> layers;
  std::vector<fa::Slab> slabs;   // indexed by layer; only owners are bound
  int32_t num_pages = 0;      // pages of each full layer's slab
  int32_t window_pages = 0;   // pages of each sliding layer's slab (0: num_pages)
  int32_t page_size = 0;
  int32_t kv_dtype = FA_KV_BF16;
  uint32_t flags = 0;   // FA_FLAG_*
  int32_t err_slot = -1;   // this cache's device error word (index into the per-device array)
  void* split_ws = nullptr;   // extend split workspace (caller's memory), split_cap jobs
  int32_t split_cap = 0;
  void* unpack_ws = nullptr;  // fp4: what the extend workspace holds past its split part
  size_t unpack_bytes = 0;
};

namespace fa {

// Pages in the slab a layer reads: sliding layers may have a pool of their own.
inline int32_t layer_pages(const fa_cache* c, int32_t layer) {
  return (c->layers[layer].d.kind == FA_SLIDING && c->window_pages > 0) ? c->window_pages : c->num_pages;
}

// thread-local error message
fa_status fail(fa_status st, const char* fmt, ...);

// The cache's device error word on the current device (file-scope
// __device__ storage, one word per live cache), and its synchronous clear.
unsigned int* device_error_word(const fa_cache* c, cudaError_t* err);
cudaError_t clear_device_error_word(const fa_cache* c);

int sm_count();

// Set a kernel's dynamic shared-memory limit once per device.
cudaError_t set_smem_once(const void* fn, int bytes, unsigned int* done_mask);

// ---------------------------------------------------------------- decode plan
// The decode kernel splits the concatenated tile lists of all (sequence, KV
// head, head chunk) units evenly over at most `ncta` CTAs; a unit whose tiles
// land on one CTA is finished there, the others are merged by the last CTA of
// the unit to finish, through arrival counters at the head of the workspace.
//
// Counters have to be zero when a call starts, partial rows may be anything, and
// one workspace serves calls of every size: so the counters' place is the same
// for every call whatever its layers, batch, bound, format or device.  It can be,
// because a counter belongs to a share of the cut, not to a unit: parts of a unit
// are joined only where shares begin inside it, a share begins inside one unit
// at most, and a launch has at most kLayerCounters shares a layer.  (Counters by
// unit, in front of partials that began where they ended, took an earlier call's
// partials for counters as soon as a call's batch or bound was larger.)
constexpr int kLayerCounters = 512;   // three shares on each of up to 170 SMs
constexpr size_t kCounterBytes = kMaxLayersPerLaunch * kLayerCounters * sizeof(int32_t);   // layer i's at i * kLayerCounters
static_assert(kCounterBytes == FA_DECODE_COUNTER_BYTES, "fa.h");
struct DecodePlan {
  int head_chunks = 1;      // ceil(g / 8): query heads are packed 8 per MMA column block
  int units = 0;            // B * Hkv * head_chunks
  int max_tiles = 0;        // 16-row tiles a unit can touch under the length bound
  int min_tiles = 0;        // fewest tiles a CTA is given
  int ncta = 0;             // shares the work may be cut into: CTAs launched (fp4: three a CTA)
  int blocks = 0;           // fp4: CTAs launched
  size_t off_o = 0;         // partials: (m, l) rows, then from off_o on the rows of O (bytes)
  size_t off_joins = 0;     // differential attention: behind the rows of O, a pair of ints a CTA
  size_t part_bytes = 0;    // 0: nothing to join, no workspace needed
  // the workspace of a call of this layer alone: counters, partials
  size_t ws_bytes() const { return part_bytes ? kCounterBytes + part_bytes : 0; }
};
// max_cta > 0 caps the launch's CTAs for this layer (default: two per SM).
// maps: softmax maps a query head (2 in differential attention), each with partial rows.
DecodePlan plan_decode(const fa_cache* c, int layer, int B, int max_seq_len, long long max_cta = 0, int maps = 1);

// Launch with programmatic stream serialisation (overlaps launch latency with
// the previous kernel's tail); every kernel waits on griddepcontrol first.
bool pdl_enabled();

template <typename Kern, typename... Args>
static cudaError_t launch_pdl(Kern kern, dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Division by an invariant: n / d for 0 <= n < 2^31 as one high product and a
// shift (Granlund and Montgomery's method, the multiplier rounded up).
struct FastDiv {
  uint32_t mul, shift, d;
  FastDiv() = default;
  explicit FastDiv(uint32_t div) : d(div) {
    shift = 0;
    while ((1ull << shift) < div) ++shift;   // ceil(log2 d)
    mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << shift) - div)) / div + 1);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
#endif
};

struct StoreArgs {
  const void* k;
  const void* v;
  const int32_t* slots;
  void* k_slab;
  void* v_slab;
  float* k_scale;
  float* v_scale;
  int T, Hkv, D, page_size, num_pages, kv_dtype, early_metadata;
  unsigned int* err;
  FastDiv by_page, by_rows;   // page_size; 2 Hkv (set by the launch, fp4)
};
cudaError_t launch_store(const StoreArgs& a, cudaStream_t s);
// The stores of several layers in one launch (n <= kMaxLayersPerLaunch; any head_dim mix).
cudaError_t launch_store_layers(const StoreArgs* a, int n, cudaStream_t s);

struct LoadArgs {
  const int32_t* slots;
  const void* k_slab;
  const void* v_slab;
  const float* k_scale;
  const float* v_scale;
  void* k;   // either may be null
  void* v;
  int T, Hkv, D, page_size, num_pages, kv_dtype, early_metadata;
  unsigned int* err;
  FastDiv by_page, by_rows;   // page_size; Hkv x sides (set by the launch)
};
cudaError_t launch_load(const LoadArgs& a, cudaStream_t s);

// Norms, rotation and store of one layer's rows (fa_rows.cu).
struct RowsArgs {
  const void* q;
  const void* k;
  const void* v;
  long long q_stride, k_stride, v_stride;   // elements from token to token
  const void* q_weight;
  const void* k_weight;
  const uint64_t* steps;
  const int32_t* positions;
  const int32_t* slots;   // null: nothing is stored
  void* q_out;
  void* k_out;
  void* v_out;
  void* k_slab;
  void* v_slab;
  float* k_scale;
  float* v_scale;
  int T, Hq, Hkv, D, rotary_dim, norm, page_size, num_pages, kv_dtype;   // norm: bit 0 q, 1 k, 2 v
  float eps, weight_offset;
  unsigned int* err;
};
cudaError_t launch_rows(const RowsArgs& a, cudaStream_t s);

// One step's tables and slots (fa_plan.cu).
struct PlanArgs {
  const int32_t* new_lens;
  const int32_t* state_in;
  int32_t* state_out;
  int32_t* free_pages;
  int32_t* block_table;
  int32_t* qo_indptr;
  int32_t* prefix_lens;
  int32_t* positions;
  int32_t* slots;
  int B, num_tokens, page_size, num_pages, max_pages_per_seq, window;   // window 0: every page is kept
  unsigned int* err;
};
cudaError_t launch_plan(const PlanArgs& a, cudaStream_t s);

struct DecodeArgs {
  const void* q;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const void* k;   // slab bases (L2 prefetch, the current token's store)
  const void* v;
  const void* k_new;        // fused store of the current token (null: none)
  const void* v_new;
  const int32_t* slots;
  const float* k_scale;
  const float* v_scale;
  void* out;
  float* lse;
  int32_t* counters;        // [kLayerCounters] (null: nothing to join)
  void* partials;
  const CUtensorMap* tm_k;
  const CUtensorMap* tm_v;
  const CUtensorMap* tm_ks;
  const CUtensorMap* tm_vs;
  int B, Hq, Hkv, D, kind, window, page_size, num_pages, max_pages_per_seq, max_seq_len, kv_dtype;
  int early_metadata;
  float sm_scale;
  const float* lambda;      // differential attention (null: plain): [Hq]
  DecodePlan plan;
  unsigned int* err;
};
cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t s);
// Differential attention (bf16 and 8-bit slabs).
cudaError_t launch_decode_diff(const DecodeArgs& a, cudaStream_t s);
// Several layers of one head_dim and KV format in one launch (n <= kMaxLayersPerLaunch).
cudaError_t launch_decode_layers(const DecodeArgs* a, int n, cudaStream_t s);

// The same over fp4 slabs (fa_decode_fp4.cu); n = 1 for a single layer.
cudaError_t launch_decode_fp4(const DecodeArgs* a, int n, cudaStream_t s);

struct ExtendArgs {
  const void* q;
  const void* k_ext;
  const void* v_ext;
  const int32_t* qo_indptr;
  const int32_t* prefix_lens;
  const int32_t* seq_lens;   // keys_in_pages: lengths including the new tokens
  const int32_t* block_table;
  const void* k_slab;
  const void* v_slab;
  const float* k_scale;
  const float* v_scale;
  const CUtensorMap* tm_k;
  const CUtensorMap* tm_v;
  const CUtensorMap* tm_ks;
  const CUtensorMap* tm_vs;
  void* out;
  float* lse;
  int B, Hq, Hkv, D, kind, window, page_size, num_pages, max_pages_per_seq, max_q_len,
      max_prefix_len, kv_dtype, num_tokens, early_metadata;
  int keys_in_pages;   // 1: every key from the slab (new tokens already stored), no k_ext / v_ext
  float sm_scale;
  unsigned int* err;
  const float* lambda;   // differential attention (null: plain): [Hq]
  // per-call maps: q as (64-column block, head, token, block index) boxes of
  // (64, g, 128/g, 1); k_ext / v_ext as (64, block, KV head, token) boxes of (64, 1, 1, 64)
  CUtensorMap tm_q, tm_kx, tm_vx;
  // the cache's split workspace (null: none), the jobs it holds, and the
  // mode: 0 no split, 1 the last wave's jobs when that wave is at most half
  // full and the jobs are long, 2 the last split_cap jobs whatever their size
  void* split_ws;
  int split_cap, split_mode;
};
cudaError_t launch_extend(const ExtendArgs& a, cudaStream_t s);

// ExtendArgs::kv_dtype of rows that launch_unpack wrote from 8-bit codes: f16 codes
// and the keys' scales, the chunk in f16 too.
constexpr int32_t kRowsF16 = 16;

// The fp4 rows of an extend or multi-token decode call as bf16, or the 8-bit
// codes and the chunk of a differential extend call as f16 (fa_unpack.cu).
struct UnpackArgs {
  const int32_t* lens;        // prefix lengths, or (stored) sequence lengths
  const int32_t* qo_indptr;
  const int32_t* block_table;
  const void* k_slab;
  const void* v_slab;
  const float* k_scale;
  const float* v_scale;
  void* k;          // [B][Hkv][ring][D] bf16, or f16
  void* v;
  int32_t* table;   // [B][table_pages]
  // 8-bit: the rows' scales [B][Hkv][ring], and the chunk, [num_tokens][Hkv][D] bf16
  // in, f16 out
  float* ks;
  float* vs;
  const void* k_ext;
  const void* v_ext;
  void* kx;
  void* vx;
  int kv_dtype, num_tokens;
  int B, Hkv, D, window, page_size, num_pages, max_pages_per_seq, max_len, max_q_len, early_metadata;
  int stored;   // multi-token decode: the queries are the sequences' last tokens
  int ring, table_pages;
  unsigned int* err;
  FastDiv by_page, by_ring;   // page_size, ring (set by the launch)
};
cudaError_t launch_unpack(const UnpackArgs& a, cudaStream_t s);

// Split workspace of extend for `cap` jobs: arrival counters, then per job
// and CTA 128 rows of (base, rounded sum, unrounded sum, 0), then per job
// and CTA a 128 x 256 fp32 partial O; each part 256-byte aligned.
struct ExtSplitLayout {
  size_t off_ml, off_o, bytes;
};
inline ExtSplitLayout ext_split_layout(int cap) {
  auto up = [](size_t b) { return (b + 255) / 256 * 256; };
  ExtSplitLayout l;
  l.off_ml = up(static_cast<size_t>(cap) * sizeof(int));
  l.off_o = l.off_ml + up(static_cast<size_t>(cap) * 2 * 128 * 16);
  l.bytes = l.off_o + static_cast<size_t>(cap) * 2 * 128 * 256 * sizeof(float);
  return l;
}
// Jobs the split workspace of this device holds: half the SMs (the largest
// last wave worth splitting in two).
inline int ext_split_cap() {
  const int n = sm_count() / 2;
  return n > 0 ? n : 1;
}

}  // namespace fa
