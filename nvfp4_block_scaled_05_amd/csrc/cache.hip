// kv_cache_write and kv_cache_read: keys and values into an NVFP4 cache as they
// are produced, and out of it again.
//
// A thread has one block of 16 neighbours: their largest magnitude, the E4M3 scale
// from it and the static amax, 16 codes: the bytes that nvfp4_quantize gives with this
// amax.  A block with an infinity or NaN gets the scale 0x7F (NaN), so that it reads
// as NaN instead of as some number.  Blocks are taken along a head's tokens, a token's
// after one another: 8 tokens of a head of 128 a wave, which reads 256-byte pieces of
// the projection and writes 512 neighbouring bytes of the page (and the reverse).
// Both directions are bound by memory: 7097 tokens of 24 heads of 128, keys and values,
// are written in 24 us (112 MB, 4.7 TB/s) and read, with what is behind them, in 25 (125
// MB, 5.0 TB/s), a copy's rate being 5.2; one token of 32 sequences takes 3.2 us each way.
#include "cache.hpp"

namespace nvfp4 {

namespace {

// The block of this thread: entry, kv head, token, block of the head.
struct BlockAt {
  uint32_t b, h, t, n;
};
__device__ __forceinline__ BlockAt block_at(const CacheCopy& a, uint32_t i) {
  BlockAt p;
  uint32_t q = divide(i, a.by_blocks);
  p.n = i - q * a.blocks;
  i = divide(q, a.by_tokens);
  p.t = q - i * (uint32_t)a.tokens;
  p.b = divide(i, a.by_heads);
  p.h = i - p.b * (uint32_t)a.c.kv_heads;
  return p;
}

// The row of token t of entry b in the cache, -1 if it has none.
__device__ __forceinline__ int64_t row_of(const CacheCopy& a, const BlockAt& p) {
  if (a.counts && (int)p.t >= a.counts[p.b]) return -1;
  const int64_t at = (int64_t)(a.starts ? a.starts[p.b] : 0) + p.t;
  if (at < 0 || at >= a.c.capacity) return -1;
  const int64_t page = cache_page(a.c, p.b, (int)at);
  return page < 0 ? -1 : cache_rows(a.c, page, (int)p.h) + cache_place(a.c, (int)at);
}

__global__ void clear_status_kernel(int32_t* p) { *p = 0; }

__global__ __launch_bounds__(256) void cache_write_kernel(CacheCopy a) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= a.total) return;
  const BlockAt p = block_at(a, i);
  const int64_t row = row_of(a, p);
  if (row < 0) return;
  const bool second = blockIdx.y != 0;
  const uint16_t* x = second ? a.v + p.b * a.v_batch + p.t * a.v_token + p.h * a.v_head
                             : a.k + p.b * a.k_batch + p.t * a.k_token + p.h * a.k_head;
  const u32x4* from = reinterpret_cast<const u32x4*>(x + 16 * p.n);
  const u32x4 lo = from[0], hi = from[1];
  bool degenerate;
  float s_enc, s_dec;
  tensor_scales(a.c.amax[second], degenerate, s_enc, s_dec);
  const uint32_t top = block_max_bits(lo, hi);
  uint32_t S = degenerate ? 0u : block_scale_e4m3(bf16_bits_to_f32(top), s_enc);
  const float e = encode_factor(S, s_dec);
  u32x2 codes = {encode8(lo, e), encode8(hi, e)};
  if (top >= 0x7F80u) {
    S = 0x7Fu;
    codes = u32x2{0u, 0u};
    if (a.status) *a.status = NVFP4_ERR_NONFINITE;
  }
  const int64_t at = row * a.blocks + p.n;
  *reinterpret_cast<u32x2*>((second ? a.c.v_codes : a.c.k_codes) + 8 * at) = codes;
  (second ? a.c.v_scales : a.c.k_scales)[at] = (uint8_t)S;
}

__global__ __launch_bounds__(256) void cache_read_kernel(CacheCopy a) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= a.total) return;
  const BlockAt p = block_at(a, i);
  const int64_t row = row_of(a, p);
  const bool second = blockIdx.y != 0;
  uint16_t* y = second ? a.v_out + p.b * a.v_batch + p.t * a.v_token + p.h * a.v_head
                       : a.k_out + p.b * a.k_batch + p.t * a.k_token + p.h * a.k_head;
  u32x4 out[2] = {};
  if (row >= 0) {
    bool degenerate;
    float s_enc, s_dec;
    tensor_scales(a.c.amax[second], degenerate, s_enc, s_dec);
    const int64_t at = row * a.blocks + p.n;
    const u32x2 codes = *reinterpret_cast<const u32x2*>((second ? a.c.v_codes : a.c.k_codes) + 8 * at);
    const float S = __builtin_amdgcn_cvt_f32_fp8((second ? a.c.v_scales : a.c.k_scales)[at], 0);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const f32x2 v[4] = {e2m1_unpack2_f32<0>(codes[j]), e2m1_unpack2_f32<1>(codes[j]),
                          e2m1_unpack2_f32<2>(codes[j]), e2m1_unpack2_f32<3>(codes[j])};
#pragma unroll
      for (int u = 0; u < 4; ++u) out[j][u] = bf16x2_rne(v[u].x * S * s_dec, v[u].y * S * s_dec);
    }
  }
  u32x4* to = reinterpret_cast<u32x4*>(y + 16 * p.n);
  to[0] = out[0];
  to[1] = out[1];
}

Divisor divisor(uint32_t d) {
  uint32_t s = 0;
  while ((1ull << s) < d) ++s;
  return {(uint32_t)((((1ull << s) - d) << 32) / d + 1), s};
}

}  // namespace

hipError_t launch_cache_copy(CacheCopy a, bool write, hipStream_t stream) {
  if (a.status) clear_status_kernel<<<1, 1, 0, stream>>>(a.status);
  if (a.batch == 0 || a.tokens == 0) return hipGetLastError();
  a.blocks = (uint32_t)(a.c.dim / 16);
  a.by_blocks = divisor(a.blocks);
  a.by_tokens = divisor((uint32_t)a.tokens);
  a.by_heads = divisor((uint32_t)a.c.kv_heads);
  a.total = (uint32_t)(a.batch * a.tokens * a.c.kv_heads * a.blocks);
  const dim3 grid((a.total + 255) / 256, 2), block(256);
  if (write)
    cache_write_kernel<<<grid, block, 0, stream>>>(a);
  else
    cache_read_kernel<<<grid, block, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace nvfp4
