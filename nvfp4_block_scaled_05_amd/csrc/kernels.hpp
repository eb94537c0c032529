// Internal launch interface between the C-ABI layer and the HIP kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nvfp4.h"

namespace nvfp4 {

// Compute units of the current device (256 if the query fails).
int compute_units();

// Upper bound on the partial maxima the amax pass writes (workspace words).
static constexpr int kMaxAmaxPartials = 1024;

// Quantizer workspace, in 32-bit words: the single-pass kernel's arrival
// counters, release words and tagged partial slots in [0, kQuantSyncWords)
// (they must start zeroed and every call leaves them consistent), the
// two-pass kernels' partial maxima after them (written before they are read
// by every call).
static constexpr int kQuantSyncWords = 1024;
static constexpr int kQuantTwoPassWords = kMaxAmaxPartials;
static constexpr int kQuantWorkspaceWords = kQuantSyncWords + kQuantTwoPassWords;

int amax_partial_count(int64_t numel);

// The library-owned quantizer workspace of the current device (a static
// device array of static_scratch_bytes(), zero when loaded): its device
// address, looked up once per device.
hipError_t static_scratch(uint32_t** out);
size_t static_scratch_bytes();

hipError_t launch_quantize(const void* x, int64_t rows, int64_t cols, uint8_t* codes,
                           uint8_t* scales, float* tensor_scale, const float* amax_in,
                           uint32_t* workspace, size_t workspace_bytes, int32_t* dev_status,
                           hipStream_t stream);

hipError_t launch_dequantize(const uint8_t* codes, const uint8_t* scales,
                             const float* tensor_scale, int64_t rows, int64_t cols, void* y,
                             hipStream_t stream);

hipError_t launch_gemm_nvfp4(const uint8_t* a_codes, const uint8_t* a_scales,
                             const float* a_tensor_scale, const uint8_t* w_codes,
                             const uint8_t* w_scales, const float* w_tensor_scale,
                             const void* bias, int64_t M, int64_t N, int64_t K, int epilogue,
                             void* y, float* y_amax, void* workspace, size_t workspace_bytes,
                             hipStream_t stream);

// The same GEMM writing Y as NVFP4 (codes, scales, tensor scale) quantized
// with the static amax *y_amax_static; N % 16 == 0.
hipError_t launch_gemm_nvfp4_quantized(const uint8_t* a_codes, const uint8_t* a_scales,
                                       const float* a_tensor_scale, const uint8_t* w_codes,
                                       const uint8_t* w_scales, const float* w_tensor_scale,
                                       const void* bias, int64_t M, int64_t N, int64_t K,
                                       int epilogue, const float* y_amax_static, uint8_t* y_codes,
                                       uint8_t* y_scales, float* y_tensor_scale,
                                       hipStream_t stream);

// Workspace bytes launch_gemm_nvfp4 can use to split the tail tiles over K
// (0: no split for this shape).
size_t gemm_nvfp4_workspace_bytes(int64_t M, int64_t N, int64_t K);

// The FP8 row-wise variant.
hipError_t launch_fp8_quantize_rowwise(const void* x, int64_t rows, int64_t cols, uint8_t* codes,
                                       float* row_scales, int32_t* dev_status, hipStream_t stream);
hipError_t launch_gemm_fp8(const uint8_t* a_codes, const float* a_scales, const uint8_t* w_codes,
                           const float* w_scales, const void* bias, int64_t M, int64_t N,
                           int64_t K, int epilogue, void* y, void* workspace,
                           size_t workspace_bytes, hipStream_t stream);
// Workspace bytes launch_gemm_fp8 can use to split the tail tiles over K.
size_t gemm_fp8_workspace_bytes(int64_t M, int64_t N, int64_t K);

hipError_t launch_gemm_bf16(const void* x, const void* w, const void* bias, int64_t M, int64_t N,
                            int64_t K, int epilogue, void* y, hipStream_t stream);

// The operators between the linears of a block.  Sizes and strides in elements.
struct GatedNorm {
  const void* x;                 // [rows, channels] bf16 or fp32
  const uint16_t* y;             // [rows, channels] or null
  const void *gate, *scale, *shift;   // [batch, channels] rows, or null
  int64_t gate_stride, scale_stride, shift_stride;
  const float *weight, *bias, *post_weight;
  int64_t rows, tokens;          // rows = batch * tokens
  int channels, norm, post_norm;
  bool mod_fp32;
  float residual_scale, eps, inv_c;
  void* residual;                // as x, or null
  uint16_t* h;                   // or null
  uint32_t* amax;                // or null
};
hipError_t launch_gated_norm(const GatedNorm& a, bool x_fp32, hipStream_t stream);

struct RotaryHeads {
  const uint16_t* in;
  int64_t in_batch, in_token, in_head;
  uint16_t* out;
  int64_t out_batch, out_token, out_head;
  const float* weight;           // the norm's, or null: no norm
  int heads;                     // 0: absent
};
struct Rotary {
  RotaryHeads q, k;
  const int32_t* positions;      // [rows, axes]
  const double* turns;           // [rotary_dim / 2]
  const int32_t* axis;           // [rotary_dim / 2], or null: all 0
  int64_t rows, tokens;          // rows = batch * tokens
  int axes, dim, rotary_dim, layout, tokens_per_group;
  float magnitude, eps, inv_dim;
};
hipError_t launch_rotary(Rotary a, hipStream_t stream);

struct Attention {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  int64_t q_batch, q_token, q_head, k_batch, k_token, k_head;
  int64_t v_batch, v_token, v_head, o_batch, o_token, o_head;
  const int32_t* lengths;        // [batch] keys each batch entry sees, or null
  const uint8_t* mask;           // [batch][keys], nonzero: seen; or null
  int64_t mask_stride;
  int batch, queries, keys, kv_heads, group, dim;   // group: query heads per kv head
  float scale;
  // filled in by the launch: row tiles per kv head (0: few rows), work units (a row
  // tile of a head, or a head), the splits of each over its keys, and of the few-row
  // kernel the groups of four 32-key tiles a split has
  int64_t row_tiles, units;
  int splits, share;
  float* part;                   // [unit][split][row][padded dim]
  float2* stats;                 // [unit][split][row]: maximum, sum
};
// Workspace bytes launch_attention can use to split the keys (0: no split).
size_t attention_workspace_bytes(int64_t batch, int64_t queries, int64_t keys, int64_t heads,
                                 int64_t kv_heads, int64_t dim);
hipError_t launch_attention(Attention a, void* workspace, size_t workspace_bytes,
                            hipStream_t stream);

struct Lora {
  const uint16_t *y, *x;         // [rows, outer], [rows, inner]
  const uint16_t *down, *up;     // [adapters, rank, inner], [adapters, outer, rank]
  const int32_t* ids;            // [rows]; outside [0, adapters): no adapter
  const float* scales;           // [adapters], or null: 1
  int64_t rows;
  int inner, outer, rank, adapters, epilogue;
  uint16_t* out;                 // may be y
  uint32_t* amax;                // or null
  // filled in by the launch
  float* t;                      // [slices][rows][padded rank]
  int slices, slice;
  bool skip_idle;
};
size_t lora_workspace_bytes(int64_t rows, int64_t inner, int64_t rank);
hipError_t launch_lora(Lora a, void* workspace, hipStream_t stream);

// An NVFP4 key/value cache (kv_cache), checked.
struct Cache {
  uint8_t *k_codes, *k_scales, *v_codes, *v_scales;   // [pages][kv_heads][page_size][dim / 2 or / 16]
  const float* amax;             // [2]: of keys, of values
  const int32_t* table;          // [batch][table_pages], or null: entry b is page b
  int64_t pages, table_pages;
  int64_t capacity;              // positions of an entry
  int page_size, page_shift;     // page_size = 1 << page_shift with a table
  int kv_heads, dim;
};
// Division by a number that the launch knows (cache.hpp).
struct Divisor {
  uint32_t magic, shift;
};
struct CacheCopy {
  Cache c;
  const uint16_t *k, *v;         // what is written, or
  uint16_t *k_out, *v_out;       // where what is read goes
  int64_t k_batch, k_token, k_head, v_batch, v_token, v_head;
  const int32_t *starts, *counts;     // [batch], or null: 0, all tokens
  int32_t* status;
  int64_t batch, tokens;
  // filled in by the launch
  uint32_t blocks, total;        // of a row, of the call (fewer than 2^31)
  Divisor by_blocks, by_tokens, by_heads;
};
hipError_t launch_cache_copy(CacheCopy a, bool write, hipStream_t stream);

struct CacheAttention {
  Cache c;
  const uint16_t* q;
  uint16_t* out;
  int64_t q_batch, q_token, q_head, o_batch, o_token, o_head;
  const int32_t* lengths;        // [batch]: keys that an entry holds
  const int32_t* starts;         // [batch]: position of its first query; null: no causal order
  int batch, queries, group;     // group: query heads per kv head
  float scale;
  // filled in by the launch
  int rows, row_tiles;           // query rows of a kv head, and their tiles
  int slot_rows;                 // rows of a slot of partial sums
  int workers, least;            // workgroups over the keys of all units, tiles each takes at least; 0: one a unit
  float* part;                   // [slot][row][padded dim]
  float2* stats;                 // [slot][row]: maximum, sum
};
// Workspace bytes with which launch_cache_attention spreads the keys over the compute
// units (0: it does not).
size_t cache_attention_workspace_bytes(int64_t batch, int64_t queries, int64_t heads, int64_t kv_heads,
                                       int64_t dim, int64_t capacity);
hipError_t launch_cache_attention(CacheAttention a, void* workspace, size_t workspace_bytes,
                                  hipStream_t stream);

// Y = epi(s_w * X W_hat^T + bias), X bf16 as it is.
struct WeightOnly {
  const uint16_t* x;             // [M, K]
  const uint8_t *codes, *scales; // [N, K / 2], [N, K / 16]
  const float* tensor_scale;
  const uint16_t* bias;          // [N] or null
  int64_t M;
  int N, K, epilogue;
  uint16_t* y;
  uint32_t* amax;                // or null
};
hipError_t launch_weight_only(WeightOnly a, hipStream_t stream);

}  // namespace nvfp4
