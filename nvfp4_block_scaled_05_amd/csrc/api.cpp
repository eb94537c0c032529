// extern "C" entry points declared in include/nvfp4.h: argument validation,
// the gfx950 device check, and launches on the caller's stream.
//
// Validation never touches the GPU: sizes, NULL pointers of non-empty buffers,
// shape multiples, alignment and workspace are checked first, in that order,
// then the current device is checked (once per device, cached), then the
// kernels are enqueued.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cfloat>
#include <cstring>
#include <regex>
#include <string>
#include <string_view>

#include "kernels.hpp"
#include "nvfp4.h"

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 31;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

std::atomic<int> g_arch_ok[64];   // 0 unknown, 1 gfx950, -1 other / error

int check_device() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return NVFP4_ERR_DEVICE;
  int c = g_arch_ok[dev].load(std::memory_order_relaxed);
  if (c == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess)
      c = -1;
    else
      c = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : -1;
    g_arch_ok[dev].store(c, std::memory_order_relaxed);
  }
  return c == 1 ? NVFP4_OK : NVFP4_ERR_DEVICE;
}

int hip_status(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP; }

bool bad_dim(int64_t v) { return v < 0 || v >= kMaxDim; }

// The page's exclude pattern, ^(?!.*(embedder|norm_out|proj_out|to_add_out|
// to_added_qkv|stream)).*, matched from the start of the name: the lookahead
// fails exactly when one of these words occurs before the name's first line
// terminator (the pattern's `.` stops at \n and \r).  Evaluated as that
// substring search, so a name of any length costs one linear scan.
constexpr const char* kExcludedWords[] = {"embedder", "norm_out",     "proj_out",
                                          "to_add_out", "to_added_qkv", "stream"};

int page_pattern_matches(const char* name) {
  std::string_view s(name);
  s = s.substr(0, s.find_first_of("\n\r"));
  for (const char* w : kExcludedWords)
    if (s.find(w) != std::string_view::npos) return 0;
  return 1;
}

// The regex engine recurses once per character of the subject, so a caller's
// pattern is only applied to names up to this length.
constexpr size_t kMaxPatternName = 1024;

// Operators between the linears: what their views and vectors must keep.

bool bad_heads(const dit_heads& v) {
  for (const int64_t s : {v.batch_stride, v.token_stride, v.head_stride})
    if (s < 0 || s % 8 != 0 || s >= ((int64_t)1 << 40)) return true;
  return false;
}

// Sizes dit_cross_attention does not take.  Rows and their tiles are counted in
// 32 bits, as are the keys of one tile past the last.
bool bad_attention(int64_t batch, int64_t queries, int64_t keys, int64_t heads, int64_t kv_heads,
                   int64_t dim) {
  if (bad_dim(batch) || bad_dim(queries) || bad_dim(keys) || keys > kMaxDim - 256) return true;
  if (heads <= 0 || heads > (1 << 16) || kv_heads <= 0 || kv_heads > heads || heads % kv_heads != 0)
    return true;
  if (dim <= 0 || dim % 8 != 0 || dim > 128) return true;
  if (batch * heads >= kMaxDim || (queries > 0 && batch * heads >= kMaxDim / queries)) return true;
  // at most 2^23 workgroups before the keys are split (only small calls are)
  return batch * kv_heads * ((queries * (heads / kv_heads) + 127) / 128) > (1 << 23);
}

// Sizes dit_lora_add does not take (element offsets within a row are 32-bit).
bool bad_lora(int64_t rows, int64_t inner, int64_t outer, int64_t rank, int64_t adapters) {
  // a workgroup of up to 768 threads for 16 rows, counted in 32 bits
  if (bad_dim(rows) || rows >= (1 << 26)) return true;
  if (inner <= 0 || inner % 8 != 0 || inner >= (1 << 28)) return true;
  if (outer < 0 || outer % 8 != 0 || outer >= (1 << 28)) return true;
  return rank <= 0 || rank % 8 != 0 || rank > 128 || adapters <= 0 || adapters >= kMaxDim;
}

// Positive, finite and not subnormal (the kernels' reciprocal square root takes a
// subnormal for zero).
bool finite_positive(float v) { return v >= FLT_MIN && v <= FLT_MAX; }

nvfp4::RotaryHeads rotary_heads(const dit_heads& in, const dit_heads& out, const float* weight,
                                int64_t heads) {
  return {static_cast<const uint16_t*>(in.data), in.batch_stride, in.token_stride, in.head_stride,
          static_cast<uint16_t*>(out.data), out.batch_stride, out.token_stride, out.head_stride,
          weight, (int)heads};
}

}  // namespace

extern "C" {

int nvfp4_abi_version(void) { return NVFP4_ABI_VERSION; }

const char* nvfp4_status_string(int status) {
  switch (status) {
    case NVFP4_OK: return "ok";
    case NVFP4_ERR_NULL: return "null pointer";
    case NVFP4_ERR_SHAPE: return "invalid shape";
    case NVFP4_ERR_ALIGN: return "misaligned pointer";
    case NVFP4_ERR_WORKSPACE: return "workspace too small";
    case NVFP4_ERR_DEVICE: return "no gfx950 device";
    case NVFP4_ERR_ARG: return "invalid argument";
    case NVFP4_ERR_HIP: return "HIP error";
    case NVFP4_ERR_NONFINITE: return "non-finite input";
    default: return "unknown status";
  }
}

size_t nvfp4_quantize_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0 || bad_dim(rows) || bad_dim(cols)) return 0;
  // the single-pass kernel's arrival words and partial slots, then the
  // two-pass kernels' partial maxima
  return 4u * (size_t)nvfp4::kQuantWorkspaceWords;
}

int nvfp4_quantize(const void* x_bf16, int64_t rows, int64_t cols, uint8_t* codes,
                   uint8_t* scales, float* tensor_scale, const float* amax_in, void* workspace,
                   size_t workspace_bytes, int32_t* dev_status, void* stream) {
  if (bad_dim(rows) || bad_dim(cols) || rows * cols >= ((int64_t)1 << 40)) return NVFP4_ERR_SHAPE;
  const bool empty = rows == 0;
  if (!tensor_scale) return NVFP4_ERR_NULL;
  if (!empty && (!x_bf16 || !codes || !scales)) return NVFP4_ERR_NULL;
  if (!empty && !amax_in && !workspace) return NVFP4_ERR_NULL;
  if (cols == 0 || cols % 16 != 0) return NVFP4_ERR_SHAPE;
  if (!aligned(x_bf16, 16) || !aligned(codes, 8) || !aligned(tensor_scale, 4) ||
      !aligned(amax_in, 4) || !aligned(workspace, 8) || !aligned(dev_status, 4))
    return NVFP4_ERR_ALIGN;
  if (!empty && !amax_in && workspace_bytes < nvfp4_quantize_workspace_bytes(rows, cols))
    return NVFP4_ERR_WORKSPACE;
  int st = check_device();
  if (st != NVFP4_OK) return st;
  if (empty) return NVFP4_OK;
  return hip_status(nvfp4::launch_quantize(x_bf16, rows, cols, codes, scales, tensor_scale,
                                           amax_in, static_cast<uint32_t*>(workspace),
                                           workspace_bytes, dev_status,
                                           static_cast<hipStream_t>(stream)));
}

int nvfp4_quantize_no_alloc(const void* x_bf16, int64_t rows, int64_t cols, uint8_t* codes,
                            uint8_t* scales, float* tensor_scale, int32_t* dev_status,
                            void* stream) {
  if (bad_dim(rows) || bad_dim(cols) || rows * cols >= ((int64_t)1 << 40)) return NVFP4_ERR_SHAPE;
  const bool empty = rows == 0;
  if (!tensor_scale) return NVFP4_ERR_NULL;
  if (!empty && (!x_bf16 || !codes || !scales)) return NVFP4_ERR_NULL;
  if (cols == 0 || cols % 16 != 0) return NVFP4_ERR_SHAPE;
  if (!aligned(x_bf16, 16) || !aligned(codes, 8) || !aligned(tensor_scale, 4) ||
      !aligned(dev_status, 4))
    return NVFP4_ERR_ALIGN;
  if (nvfp4_quantize_workspace_bytes(rows, cols) > nvfp4::static_scratch_bytes())
    return NVFP4_ERR_WORKSPACE;
  int st = check_device();
  if (st != NVFP4_OK) return st;
  if (empty) return NVFP4_OK;
  uint32_t* ws = nullptr;
  if (nvfp4::static_scratch(&ws) != hipSuccess) return NVFP4_ERR_HIP;
  return hip_status(nvfp4::launch_quantize(x_bf16, rows, cols, codes, scales, tensor_scale,
                                           nullptr, ws, nvfp4::static_scratch_bytes(), dev_status,
                                           static_cast<hipStream_t>(stream)));
}

int nvfp4_dequantize(const uint8_t* codes, const uint8_t* scales, const float* tensor_scale,
                     int64_t rows, int64_t cols, void* y_bf16, void* stream) {
  if (bad_dim(rows) || bad_dim(cols) || rows * cols >= ((int64_t)1 << 40)) return NVFP4_ERR_SHAPE;
  const bool empty = rows == 0;
  if (!empty && (!codes || !scales || !tensor_scale || !y_bf16)) return NVFP4_ERR_NULL;
  if (cols == 0 || cols % 16 != 0) return NVFP4_ERR_SHAPE;
  if (!aligned(codes, 8) || !aligned(tensor_scale, 4) || !aligned(y_bf16, 16))
    return NVFP4_ERR_ALIGN;
  int st = check_device();
  if (st != NVFP4_OK) return st;
  if (empty) return NVFP4_OK;
  return hip_status(nvfp4::launch_dequantize(codes, scales, tensor_scale, rows, cols, y_bf16,
                                             static_cast<hipStream_t>(stream)));
}

size_t nvfp4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (bad_dim(M) || bad_dim(N) || bad_dim(K) || K % 16 != 0) return 0;
  return nvfp4::gemm_nvfp4_workspace_bytes(M, N, K);
}

int nvfp4_gemm(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_tensor_scale,
               const uint8_t* w_codes, const uint8_t* w_scales, const float* w_tensor_scale,
               const void* bias_bf16, int64_t M, int64_t N, int64_t K, int epilogue, void* y_bf16,
               float* y_amax, void* workspace, size_t workspace_bytes, void* stream) {
  if (bad_dim(M) || bad_dim(N) || bad_dim(K)) return NVFP4_ERR_SHAPE;
  const bool empty = M == 0 || N == 0;
  if (!empty && (!a_codes || !a_scales || !a_tensor_scale || !w_codes || !w_scales ||
                 !w_tensor_scale || !y_bf16))
    return NVFP4_ERR_NULL;
  if (K == 0 || K % 16 != 0) return NVFP4_ERR_SHAPE;
  if (((M + 127) / 128) * ((N + 127) / 128) >= ((int64_t)1 << 24)) return NVFP4_ERR_SHAPE;
  if (!aligned(a_codes, 8) || !aligned(w_codes, 8) || !aligned(a_tensor_scale, 4) ||
      !aligned(w_tensor_scale, 4) || !aligned(bias_bf16, 2) || !aligned(y_bf16, 2) ||
      !aligned(y_amax, 4) || !aligned(workspace, 256))
    return NVFP4_ERR_ALIGN;
  if (epilogue != NVFP4_EPI_NONE && epilogue != NVFP4_EPI_GELU) return NVFP4_ERR_ARG;
  int st = check_device();
  if (st != NVFP4_OK) return st;
  return hip_status(nvfp4::launch_gemm_nvfp4(a_codes, a_scales, a_tensor_scale, w_codes, w_scales,
                                             w_tensor_scale, bias_bf16, M, N, K, epilogue, y_bf16,
                                             y_amax, workspace, workspace ? workspace_bytes : 0,
                                             static_cast<hipStream_t>(stream)));
}

int nvfp4_gemm_quantized(const uint8_t* a_codes, const uint8_t* a_scales,
                         const float* a_tensor_scale, const uint8_t* w_codes,
                         const uint8_t* w_scales, const float* w_tensor_scale,
                         const void* bias_bf16, int64_t M, int64_t N, int64_t K, int epilogue,
                         const float* y_amax, uint8_t* y_codes, uint8_t* y_scales,
                         float* y_tensor_scale, void* stream) {
  if (bad_dim(M) || bad_dim(N) || bad_dim(K)) return NVFP4_ERR_SHAPE;
  const bool empty = M == 0 || N == 0;
  if (!empty && (!a_codes || !a_scales || !a_tensor_scale || !w_codes || !w_scales ||
                 !w_tensor_scale || !y_amax || !y_codes || !y_scales || !y_tensor_scale))
    return NVFP4_ERR_NULL;
  if (K == 0 || K % 16 != 0 || N % 16 != 0) return NVFP4_ERR_SHAPE;
  if (((M + 127) / 128) * ((N + 127) / 128) >= ((int64_t)1 << 24)) return NVFP4_ERR_SHAPE;
  if (!aligned(a_codes, 8) || !aligned(w_codes, 8) || !aligned(a_tensor_scale, 4) ||
      !aligned(w_tensor_scale, 4) || !aligned(bias_bf16, 2) || !aligned(y_amax, 4) ||
      !aligned(y_codes, 8) || !aligned(y_tensor_scale, 4))
    return NVFP4_ERR_ALIGN;
  if (epilogue != NVFP4_EPI_NONE && epilogue != NVFP4_EPI_GELU) return NVFP4_ERR_ARG;
  int st = check_device();
  if (st != NVFP4_OK) return st;
  if (empty) return NVFP4_OK;
  return hip_status(nvfp4::launch_gemm_nvfp4_quantized(
      a_codes, a_scales, a_tensor_scale, w_codes, w_scales, w_tensor_scale, bias_bf16, M, N, K,
      epilogue, y_amax, y_codes, y_scales, y_tensor_scale, static_cast<hipStream_t>(stream)));
}

int nvfp4_fp8_quantize_rowwise(const void* x_bf16, int64_t rows, int64_t cols, uint8_t* codes,
                               float* row_scales, int32_t* dev_status, void* stream) {
  if (bad_dim(rows) || bad_dim(cols) || rows * cols >= ((int64_t)1 << 40)) return NVFP4_ERR_SHAPE;
  const bool empty = rows == 0;
  if (!empty && (!x_bf16 || !codes || !row_scales)) return NVFP4_ERR_NULL;
  if (cols == 0 || cols % 16 != 0) return NVFP4_ERR_SHAPE;
  if (!aligned(x_bf16, 16) || !aligned(codes, 8) || !aligned(row_scales, 4) ||
      !aligned(dev_status, 4))
    return NVFP4_ERR_ALIGN;
  int st = check_device();
  if (st != NVFP4_OK) return st;
  return hip_status(nvfp4::launch_fp8_quantize_rowwise(x_bf16, rows, cols, codes, row_scales,
                                                       dev_status,
                                                       static_cast<hipStream_t>(stream)));
}

size_t nvfp4_fp8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (bad_dim(M) || bad_dim(N) || bad_dim(K) || K % 16 != 0) return 0;
  return nvfp4::gemm_fp8_workspace_bytes(M, N, K);
}

int nvfp4_fp8_gemm(const uint8_t* a_codes, const float* a_scales, const uint8_t* w_codes,
                   const float* w_scales, const void* bias_bf16, int64_t M, int64_t N, int64_t K,
                   int epilogue, void* y_bf16, void* workspace, size_t workspace_bytes,
                   void* stream) {
  if (bad_dim(M) || bad_dim(N) || bad_dim(K)) return NVFP4_ERR_SHAPE;
  const bool empty = M == 0 || N == 0;
  if (!empty && (!a_codes || !a_scales || !w_codes || !w_scales || !y_bf16)) return NVFP4_ERR_NULL;
  if (K == 0 || K % 16 != 0) return NVFP4_ERR_SHAPE;
  if (((M + 255) / 256) * ((N + 255) / 256) >= ((int64_t)1 << 24)) return NVFP4_ERR_SHAPE;
  if (!aligned(a_codes, 16) || !aligned(w_codes, 16) || !aligned(a_scales, 4) ||
      !aligned(w_scales, 4) || !aligned(bias_bf16, 2) || !aligned(y_bf16, 2) ||
      !aligned(workspace, 256))
    return NVFP4_ERR_ALIGN;
  if (epilogue != NVFP4_EPI_NONE && epilogue != NVFP4_EPI_GELU) return NVFP4_ERR_ARG;
  int st = check_device();
  if (st != NVFP4_OK) return st;
  if (empty) return NVFP4_OK;
  return hip_status(nvfp4::launch_gemm_fp8(a_codes, a_scales, w_codes, w_scales, bias_bf16, M, N,
                                           K, epilogue, y_bf16, workspace,
                                           workspace ? workspace_bytes : 0,
                                           static_cast<hipStream_t>(stream)));
}

int nvfp4_gemm_bf16(const void* x_bf16, const void* w_bf16, const void* bias_bf16, int64_t M,
                    int64_t N, int64_t K, int epilogue, void* y_bf16, void* stream) {
  if (bad_dim(M) || bad_dim(N) || bad_dim(K)) return NVFP4_ERR_SHAPE;
  const bool empty = M == 0 || N == 0;
  if (!empty && (!x_bf16 || !w_bf16 || !y_bf16)) return NVFP4_ERR_NULL;
  if (K == 0 || K % 8 != 0) return NVFP4_ERR_SHAPE;
  if (((M + 127) / 128) * ((N + 127) / 128) >= ((int64_t)1 << 24)) return NVFP4_ERR_SHAPE;
  if (!aligned(x_bf16, 16) || !aligned(w_bf16, 16) || !aligned(bias_bf16, 2) ||
      !aligned(y_bf16, 2))
    return NVFP4_ERR_ALIGN;
  if (epilogue != NVFP4_EPI_NONE && epilogue != NVFP4_EPI_GELU) return NVFP4_ERR_ARG;
  int st = check_device();
  if (st != NVFP4_OK) return st;
  if (empty) return NVFP4_OK;
  return hip_status(nvfp4::launch_gemm_bf16(x_bf16, w_bf16, bias_bf16, M, N, K, epilogue, y_bf16,
                                            static_cast<hipStream_t>(stream)));
}

int nvfp4_graph_begin(void* stream) {
  if (!stream) return NVFP4_ERR_NULL;
  int st = check_device();
  if (st != NVFP4_OK) return st;
  return hip_status(
      hipStreamBeginCapture(static_cast<hipStream_t>(stream), hipStreamCaptureModeThreadLocal));
}

int nvfp4_graph_end(void* stream, void** graph) {
  if (!stream || !graph) return NVFP4_ERR_NULL;
  hipGraph_t g = nullptr;
  if (hipStreamEndCapture(static_cast<hipStream_t>(stream), &g) != hipSuccess || !g)
    return NVFP4_ERR_HIP;
  hipGraphExec_t exec = nullptr;
  const hipError_t e = hipGraphInstantiate(&exec, g, nullptr, nullptr, 0);
  // the instantiated graph does not need the captured one
  static_cast<void>(hipGraphDestroy(g));
  if (e != hipSuccess) return NVFP4_ERR_HIP;
  *graph = exec;
  return NVFP4_OK;
}

int nvfp4_graph_launch(void* graph, void* stream) {
  if (!graph) return NVFP4_ERR_NULL;
  return hip_status(
      hipGraphLaunch(static_cast<hipGraphExec_t>(graph), static_cast<hipStream_t>(stream)));
}

int nvfp4_graph_destroy(void* graph) {
  if (!graph) return NVFP4_ERR_NULL;
  return hip_status(hipGraphExecDestroy(static_cast<hipGraphExec_t>(graph)));
}

int nvfp4_layer_is_quantized(const char* layer_name, const char* pattern) {
  if (!layer_name) return NVFP4_ERR_NULL;
  if (!pattern) return page_pattern_matches(layer_name);
  try {
    const std::regex re(pattern, std::regex::ECMAScript);
    const std::string name(layer_name);
    if (name.size() > kMaxPatternName) return NVFP4_ERR_ARG;
    return std::regex_search(name, re, std::regex_constants::match_continuous) ? 1 : 0;
  } catch (const std::exception&) {
    return NVFP4_ERR_ARG;
  }
}

int dit_gated_norm(const void* x, int x_fp32, const void* y_bf16, const void* gate,
                   int64_t gate_stride, const void* scale, int64_t scale_stride,
                   const void* shift, int64_t shift_stride, int mod_fp32, const float* weight,
                   const float* bias, const float* post_weight, int64_t batch, int64_t tokens,
                   int64_t channels, int norm, int post_norm, float residual_scale, float eps,
                   void* residual, void* h_bf16, float* amax, void* stream) {
  if (bad_dim(batch) || bad_dim(tokens) || bad_dim(channels)) return NVFP4_ERR_SHAPE;
  const bool empty = batch == 0 || tokens == 0;
  if (!empty && (!x || (!residual && !h_bf16))) return NVFP4_ERR_NULL;
  if (amax && !empty && !h_bf16) return NVFP4_ERR_NULL;
  if (channels == 0 || channels % 8 != 0 || channels > 16384) return NVFP4_ERR_SHAPE;
  if (batch * tokens >= kMaxDim) return NVFP4_ERR_SHAPE;
  for (const int64_t s : {gate ? gate_stride : 0, scale ? scale_stride : 0, shift ? shift_stride : 0})
    if (s < 0 || s % 8 != 0 || s >= ((int64_t)1 << 31)) return NVFP4_ERR_SHAPE;
  for (const void* p : {x, y_bf16, gate, scale, shift, static_cast<const void*>(weight),
                        static_cast<const void*>(bias), static_cast<const void*>(post_weight),
                        static_cast<const void*>(residual), static_cast<const void*>(h_bf16)})
    if (!aligned(p, 16)) return NVFP4_ERR_ALIGN;
  if (!aligned(amax, 4)) return NVFP4_ERR_ALIGN;
  for (const int n : {norm, post_norm})
    if (n != DIT_NORM_NONE && n != DIT_NORM_LAYER && n != DIT_NORM_RMS) return NVFP4_ERR_ARG;
  if (!finite_positive(eps) || !(residual_scale >= -FLT_MAX && residual_scale <= FLT_MAX))
    return NVFP4_ERR_ARG;
  if (!y_bf16 && !empty &&
      (gate || post_norm != DIT_NORM_NONE || post_weight || residual || residual_scale != 1.0f))
    return NVFP4_ERR_ARG;
  int st = check_device();
  if (st != NVFP4_OK) return st;
  const nvfp4::GatedNorm a{x, static_cast<const uint16_t*>(y_bf16), gate, scale, shift,
                           gate_stride, scale_stride, shift_stride, weight, bias, post_weight,
                           batch * tokens, tokens, (int)channels, norm, post_norm, mod_fp32 != 0,
                           residual_scale, eps, (float)(1.0 / (double)channels), residual,
                           static_cast<uint16_t*>(h_bf16), reinterpret_cast<uint32_t*>(amax)};
  return hip_status(nvfp4::launch_gated_norm(a, x_fp32 != 0, static_cast<hipStream_t>(stream)));
}

int dit_rotary(const dit_heads* q, const dit_heads* q_out, int64_t heads, const dit_heads* k,
               const dit_heads* k_out, int64_t kv_heads, const int32_t* positions, int64_t axes,
               const double* turns, const int32_t* axis, float magnitude, const float* q_weight,
               const float* k_weight, float eps, int64_t batch, int64_t tokens, int64_t dim,
               int64_t rotary_dim, int layout, void* stream) {
  if (bad_dim(batch) || bad_dim(tokens) || bad_dim(heads) || bad_dim(kv_heads))
    return NVFP4_ERR_SHAPE;
  const bool empty = batch == 0 || tokens == 0;
  if (!q || !q_out || (kv_heads > 0 && (!k || !k_out))) return NVFP4_ERR_NULL;
  if (!empty && (!q->data || !q_out->data || !positions || !turns || (axes > 1 && !axis)))
    return NVFP4_ERR_NULL;
  if (!empty && kv_heads > 0 && (!k->data || !k_out->data)) return NVFP4_ERR_NULL;
  if (heads == 0 || heads + kv_heads > (1 << 16) || batch * tokens >= kMaxDim)
    return NVFP4_ERR_SHAPE;
  if (dim <= 0 || dim % 8 != 0 || dim > 256 || rotary_dim <= 0 || rotary_dim % 16 != 0 ||
      rotary_dim > dim || axes < 1 || axes > 16)
    return NVFP4_ERR_SHAPE;
  if (bad_heads(*q) || bad_heads(*q_out)) return NVFP4_ERR_SHAPE;
  if (kv_heads > 0 && (bad_heads(*k) || bad_heads(*k_out))) return NVFP4_ERR_SHAPE;
  if (!aligned(q->data, 16) || !aligned(q_out->data, 16) || !aligned(positions, 4) ||
      !aligned(turns, 8) || !aligned(axis, 4) || !aligned(q_weight, 4) || !aligned(k_weight, 4))
    return NVFP4_ERR_ALIGN;
  if (kv_heads > 0 && (!aligned(k->data, 16) || !aligned(k_out->data, 16))) return NVFP4_ERR_ALIGN;
  if ((layout != DIT_ROTARY_INTERLEAVED && layout != DIT_ROTARY_HALF) || !finite_positive(eps) ||
      !finite_positive(magnitude))
    return NVFP4_ERR_ARG;
  int st = check_device();
  if (st != NVFP4_OK) return st;
  nvfp4::Rotary a{};
  a.q = rotary_heads(*q, *q_out, q_weight, heads);
  if (kv_heads > 0) a.k = rotary_heads(*k, *k_out, k_weight, kv_heads);
  a.positions = positions;
  a.turns = turns;
  a.axis = axis;
  a.rows = batch * tokens;
  a.tokens = tokens;
  a.axes = (int)axes;
  a.dim = (int)dim;
  a.rotary_dim = (int)rotary_dim;
  a.layout = layout;
  a.magnitude = magnitude;
  a.eps = eps;
  a.inv_dim = (float)(1.0 / (double)dim);
  return hip_status(nvfp4::launch_rotary(a, static_cast<hipStream_t>(stream)));
}

size_t dit_cross_attention_workspace_bytes(int64_t batch, int64_t queries, int64_t keys,
                                           int64_t heads, int64_t kv_heads, int64_t dim) {
  if (bad_attention(batch, queries, keys, heads, kv_heads, dim)) return 0;
  return nvfp4::attention_workspace_bytes(batch, queries, keys, heads, kv_heads, dim);
}

int dit_cross_attention(const dit_heads* q, const dit_heads* k, const dit_heads* v,
                        const int32_t* kv_lengths, const uint8_t* key_mask, int64_t mask_stride,
                        int64_t batch, int64_t queries, int64_t keys, int64_t heads,
                        int64_t kv_heads, int64_t dim, float scale, const dit_heads* out,
                        void* workspace, size_t workspace_bytes, void* stream) {
  if (bad_dim(batch) || bad_dim(queries) || bad_dim(keys)) return NVFP4_ERR_SHAPE;
  const bool empty = batch == 0 || queries == 0;
  if (!q || !k || !v || !out) return NVFP4_ERR_NULL;
  if (!empty && (!q->data || !out->data || (keys > 0 && (!k->data || !v->data))))
    return NVFP4_ERR_NULL;
  if (bad_attention(batch, queries, keys, heads, kv_heads, dim)) return NVFP4_ERR_SHAPE;
  for (const dit_heads* h : {q, k, v, out})
    if (bad_heads(*h)) return NVFP4_ERR_SHAPE;
  // a tile's 64 rows are addressed with 32-bit offsets
  if (k->token_stride >= (1 << 23) || v->token_stride >= (1 << 23)) return NVFP4_ERR_SHAPE;
  if (key_mask && (mask_stride < 0 || mask_stride >= ((int64_t)1 << 40))) return NVFP4_ERR_SHAPE;
  for (const dit_heads* h : {q, k, v, out})
    if (!aligned(h->data, 16)) return NVFP4_ERR_ALIGN;
  if (!aligned(kv_lengths, 4) || !aligned(workspace, 256)) return NVFP4_ERR_ALIGN;
  if (!finite_positive(scale)) return NVFP4_ERR_ARG;
  int st = check_device();
  if (st != NVFP4_OK) return st;
  if (empty) return NVFP4_OK;
  nvfp4::Attention a{};
  a.q = static_cast<const uint16_t*>(q->data);
  a.k = static_cast<const uint16_t*>(k->data);
  a.v = static_cast<const uint16_t*>(v->data);
  a.out = static_cast<uint16_t*>(out->data);
  a.q_batch = q->batch_stride, a.q_token = q->token_stride, a.q_head = q->head_stride;
  a.k_batch = k->batch_stride, a.k_token = k->token_stride, a.k_head = k->head_stride;
  a.v_batch = v->batch_stride, a.v_token = v->token_stride, a.v_head = v->head_stride;
  a.o_batch = out->batch_stride, a.o_token = out->token_stride, a.o_head = out->head_stride;
  a.lengths = kv_lengths;
  a.mask = key_mask;
  a.mask_stride = mask_stride;
  a.batch = (int)batch;
  a.queries = (int)queries;
  a.keys = (int)keys;
  a.kv_heads = (int)kv_heads;
  a.group = (int)(heads / kv_heads);
  a.dim = (int)dim;
  a.scale = scale;
  return hip_status(nvfp4::launch_attention(a, workspace, workspace ? workspace_bytes : 0,
                                            static_cast<hipStream_t>(stream)));
}

size_t dit_lora_workspace_bytes(int64_t rows, int64_t inner, int64_t rank) {
  if (rows <= 0 || bad_lora(rows, inner, 8, rank, 1)) return 0;
  return nvfp4::lora_workspace_bytes(rows, inner, rank);
}

int dit_lora_add(const void* y_bf16, const void* x_bf16, const void* down, const void* up,
                 const int32_t* ids, const float* scales, int64_t rows, int64_t inner,
                 int64_t outer, int64_t rank, int64_t adapters, int epilogue, void* out_bf16,
                 float* out_amax, void* workspace, size_t workspace_bytes, void* stream) {
  if (bad_dim(rows) || bad_dim(outer)) return NVFP4_ERR_SHAPE;
  const bool empty = rows == 0 || outer == 0;
  if (!empty && (!y_bf16 || !x_bf16 || !down || !up || !ids || !out_bf16 || !workspace))
    return NVFP4_ERR_NULL;
  if (bad_lora(rows, inner, outer, rank, adapters)) return NVFP4_ERR_SHAPE;
  for (const void* p : {y_bf16, x_bf16, down, up, static_cast<const void*>(out_bf16)})
    if (!aligned(p, 16)) return NVFP4_ERR_ALIGN;
  if (!aligned(ids, 4) || !aligned(scales, 4) || !aligned(out_amax, 4) || !aligned(workspace, 256))
    return NVFP4_ERR_ALIGN;
  if (epilogue != NVFP4_EPI_NONE && epilogue != NVFP4_EPI_GELU) return NVFP4_ERR_ARG;
  if (!empty && workspace_bytes < nvfp4::lora_workspace_bytes(rows, inner, rank))
    return NVFP4_ERR_WORKSPACE;
  int st = check_device();
  if (st != NVFP4_OK) return st;
  nvfp4::Lora a{};
  a.y = static_cast<const uint16_t*>(y_bf16);
  a.x = static_cast<const uint16_t*>(x_bf16);
  a.down = static_cast<const uint16_t*>(down);
  a.up = static_cast<const uint16_t*>(up);
  a.ids = ids;
  a.scales = scales;
  a.rows = rows;
  a.inner = (int)inner;
  a.outer = (int)outer;
  a.rank = (int)rank;
  a.adapters = (int)adapters;
  a.epilogue = epilogue;
  a.out = static_cast<uint16_t*>(out_bf16);
  a.amax = reinterpret_cast<uint32_t*>(out_amax);
  return hip_status(nvfp4::launch_lora(a, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
