// w4_gemm_weight_only: a few rows of bf16 activations, not quantized, times an NVFP4
// weight.
//
// A wave has 16 weight rows and up to 64 rows of x and every WAVES-th step of 128 k; the
// waves of a workgroup are joined in LDS, in wave order.  A code times its block scale
// has at most six significant bits, so bf16 holds it and the products are those of the
// formula.  Bound by the stream of codes.
#include "device_common.hpp"
#include "kernels.hpp"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kStepK = 128;

__global__ void zero_product_amax_kernel(uint32_t* p) { *p = 0u; }

// 8 codes times their scale, as bf16.
__device__ __forceinline__ bf16x8 decode8_bf16(uint32_t w, float s) {
  const f32x2 a = e2m1_unpack2_f32<0>(w), b = e2m1_unpack2_f32<1>(w), c = e2m1_unpack2_f32<2>(w), d = e2m1_unpack2_f32<3>(w);
  return __builtin_bit_cast(bf16x8, u32x4{bf16x2_rne(a.x * s, a.y * s), bf16x2_rne(b.x * s, b.y * s),
                                          bf16x2_rne(c.x * s, c.y * s), bf16x2_rne(d.x * s, d.y * s)});
}

// Loads of any alignment.
__device__ __forceinline__ u32x4 load16(const uint8_t* p) {
  u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
__device__ __forceinline__ uint32_t load2(const uint8_t* p) {
  uint16_t v;
  __builtin_memcpy(&v, p, 2);
  return v;
}

// One output: tensor scale, bias, GELU, bf16.
__device__ __forceinline__ uint32_t finish(const WeightOnly& a, float y, float sw, int n) {
  float z = y * sw;
  if (a.bias) z += bf16_bits_to_f32(a.bias[n]);
  if (a.epilogue == NVFP4_EPI_GELU) z = gelu_erf(z);
  return bf16x2_rne(z, 0.0f);
}

template <int RT, int MT, int U, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void weight_only_kernel(WeightOnly a) {
  __shared__ f32x4 park[WAVES][RT * MT][64];
  const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4, wave = wave_id();
  const int n0 = (int)blockIdx.x * (16 * RT);
  const int64_t m0 = (int64_t)blockIdx.y * (16 * MT);
  const uint8_t *codes[RT], *scales[RT];
  const uint16_t* x[MT];
  bool live[MT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int64_t n = min(n0 + 16 * rt + m, a.N - 1);
    codes[rt] = a.codes + n * (a.K / 2);
    scales[rt] = a.scales + n * (a.K / 16);
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    live[mt] = m0 + 16 * mt + m < a.M;
    x[mt] = a.x + (live[mt] ? m0 + 16 * mt + m : 0) * a.K;
  }
  f32x4 acc[RT][MT] = {};
  for (int step = wave; step * (U * kStepK) < a.K; step += WAVES) {
    u32x4 c[U][RT];
    uint32_t sc[U][RT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (step * U + u) * kStepK + 32 * g, blocks = min(max((a.K - k) / 16, 0), 2);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        c[u][rt] = u32x4{};
        sc[u][rt] = 0;
        if (blocks == 2) {
          c[u][rt] = load16(codes[rt] + (uint32_t)(k / 2));
          sc[u][rt] = load2(scales[rt] + (uint32_t)(k / 16));
        } else if (blocks == 1) {
          const u32x2 v = *reinterpret_cast<const u32x2*>(codes[rt] + (uint32_t)(k / 2));
          c[u][rt] = u32x4{v.x, v.y, 0u, 0u};
          sc[u][rt] = scales[rt][(uint32_t)(k / 16)];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (step * U + u) * kStepK + 32 * g;
      u32x4 xv[MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          xv[mt][i] = u32x4{};
          if (live[mt] && k + 8 * i < a.K) xv[mt][i] = *reinterpret_cast<const u32x4*>(x[mt] + k + 8 * i);
        }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const float s0 = __builtin_amdgcn_cvt_f32_fp8(sc[u][rt], 0), s1 = __builtin_amdgcn_cvt_f32_fp8(sc[u][rt], 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bf16x8 w = decode8_bf16(c[u][rt][i], i < 2 ? s0 : s1);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            acc[rt][mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8, xv[mt][i]), acc[rt][mt], 0, 0, 0);
        }
      }
    }
  }
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) park[wave][rt * MT + mt][lane] = acc[rt][mt];
  __syncthreads();
  const float sw = *a.tensor_scale;
  uint32_t top = 0;
  for (int tile = wave; tile < RT * MT; tile += WAVES) {
    f32x4 y = park[0][tile][lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) y += park[w][tile][lane];
    const int n = n0 + 16 * (tile / MT) + 4 * g;
    const int64_t row = m0 + 16 * (tile % MT) + m;
    if (row >= a.M || n >= a.N) continue;
    uint16_t out[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      out[r] = (uint16_t)finish(a, y[r], sw, min(n + r, a.N - 1));
      if (n + r < a.N) top = max(top, (uint32_t)out[r] & 0x7FFFu);
    }
    uint16_t* to = a.y + row * a.N + n;
    if (a.N % 4 == 0) {
      *reinterpret_cast<u32x2*>(to) = u32x2{(uint32_t)out[0] | (uint32_t)out[1] << 16, (uint32_t)out[2] | (uint32_t)out[3] << 16};
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < a.N) to[r] = out[r];
    }
  }
  if (a.amax) {
    top = wave_max_u32(top);
    if (lane == 0 && top) raise_amax(a.amax, top << 16);
  }
}

// One or two rows of x: the lanes lie along k, 32 each, so a wave reads 1 KiB of a
// weight row at a time and keeps its part of x in registers over kRows weight rows.
// Sums over the lanes come last.  The dot instruction takes pairs of codes as bf16
// without their scale; a block's sum is multiplied by it in binary32.
constexpr int kRows = 8;                       // weight rows of a wave
constexpr int kChunk = 2048;                   // k of a wave

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

template <int BYTE>
__device__ __forceinline__ float dot_byte(uint32_t codes, uint32_t x, float sum) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, 1.0f, BYTE),
                                         __builtin_bit_cast(bf16x2, x), sum, false);
}
__device__ __forceinline__ float dot8(uint32_t codes, u32x4 x, float sum) {
  return dot_byte<3>(codes, x.w, dot_byte<2>(codes, x.z, dot_byte<1>(codes, x.y, dot_byte<0>(codes, x.x, sum))));
}

template <int M>
__global__ __launch_bounds__(256) void weight_only_vector_kernel(WeightOnly a, int ways) {
  __shared__ float park[4][kRows][M];
  const int lane = threadIdx.x & 63, wave = wave_id(), slot = wave % ways;
  const int64_t m0 = (int64_t)blockIdx.y * M;
  const int n0 = ((int)blockIdx.x * (4 / ways) + wave / ways) * kRows;       // the wave's first weight row
  float acc[kRows][M] = {};
  for (int c = slot; c * kChunk < a.K; c += ways) {
    const int k = c * kChunk + 32 * lane, blocks = min(max((a.K - k) / 16, 0), 2);
    u32x4 codes[kRows];
    uint32_t scales[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t n = min(n0 + r, a.N - 1);
      const uint8_t *cr = a.codes + n * (a.K / 2), *sr = a.scales + n * (a.K / 16);
      codes[r] = u32x4{};
      scales[r] = 0;
      if (blocks == 2) {
        codes[r] = load16(cr + (uint32_t)(k / 2));
        scales[r] = load2(sr + (uint32_t)(k / 16));
      } else if (blocks == 1) {
        const u32x2 v = *reinterpret_cast<const u32x2*>(cr + (uint32_t)(k / 2));
        codes[r] = u32x4{v.x, v.y, 0u, 0u};
        scales[r] = sr[(uint32_t)(k / 16)];
      }
    }
    u32x4 x[M][4];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[m][i] = u32x4{};
        if (i / 2 < blocks) x[m][i] = *reinterpret_cast<const u32x4*>(a.x + min(m0 + m, a.M - 1) * a.K + k + 8 * i);
      }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const float s0 = __builtin_amdgcn_cvt_f32_fp8(scales[r], 0), s1 = __builtin_amdgcn_cvt_f32_fp8(scales[r], 1);
#pragma unroll
      for (int m = 0; m < M; ++m) {
        acc[r][m] = __builtin_fmaf(dot8(codes[r].y, x[m][1], dot8(codes[r].x, x[m][0], 0.0f)), s0, acc[r][m]);
        acc[r][m] = __builtin_fmaf(dot8(codes[r].w, x[m][3], dot8(codes[r].z, x[m][2], 0.0f)), s1, acc[r][m]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const float sum = wave_sum(acc[r][m]);
      if (lane == 0) park[wave][r][m] = sum;
    }
  __syncthreads();
  uint32_t top = 0;
  const int of = (int)threadIdx.x / (kRows * M), r = (int)threadIdx.x / M % kRows, m = (int)threadIdx.x % M;
  if (of < 4 / ways) {
    float y = park[of * ways][r][m];
    for (int w = 1; w < ways; ++w) y += park[of * ways + w][r][m];
    const int n = ((int)blockIdx.x * (4 / ways) + of) * kRows + r;
    if (n < a.N && m0 + m < a.M) {
      const uint32_t out = finish(a, y, *a.tensor_scale, n);
      a.y[(m0 + m) * a.N + n] = (uint16_t)out;
      top = out & 0x7FFFu;
    }
  }
  if (a.amax) {                                // outputs are the first wave's
    top = wave_max_u32(top);
    if (threadIdx.x == 0 && top) raise_amax(a.amax, top << 16);
  }
}

template <int RT, int MT, int U, int WAVES>
void launch_rows(const WeightOnly& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.N + 16 * RT - 1) / (16 * RT)), (unsigned)((a.M + 16 * MT - 1) / (16 * MT)));
  weight_only_kernel<RT, MT, U, WAVES><<<grid, 64 * WAVES, 0, stream>>>(a);
}

}  // namespace

hipError_t launch_weight_only(WeightOnly a, hipStream_t stream) {
  if (a.amax) zero_product_amax_kernel<<<1, 1, 0, stream>>>(a.amax);
  if (a.M == 0 || a.N == 0) return hipGetLastError();
  if (a.M <= 2) {
    const int ways = a.K <= kChunk ? 1 : a.K <= 2 * kChunk ? 2 : 4, rows = kRows * 4 / ways;
    const dim3 grid((unsigned)((a.N + rows - 1) / rows));
    if (a.M == 1)
      weight_only_vector_kernel<1><<<grid, 256, 0, stream>>>(a, ways);
    else
      weight_only_vector_kernel<2><<<grid, 256, 0, stream>>>(a, ways);
    return hipGetLastError();
  }
  const int64_t tiles = (a.N + 15) / 16;
  if (a.M <= 32 && tiles >= 4 * 192)
    a.M <= 16 ? launch_rows<4, 1, 1, 8>(a, stream) : launch_rows<4, 2, 1, 8>(a, stream);
  else if (tiles >= 2 * 192)
    a.M <= 16   ? launch_rows<2, 1, 2, 8>(a, stream)
    : a.M <= 32 ? launch_rows<2, 2, 1, 8>(a, stream)
                : launch_rows<2, 4, 1, 8>(a, stream);
  else
    a.M <= 16   ? launch_rows<1, 1, 4, 8>(a, stream)
    : a.M <= 32 ? launch_rows<1, 2, 2, 8>(a, stream)
                : launch_rows<1, 4, 1, 8>(a, stream);
  return hipGetLastError();
}

}  // namespace nvfp4
