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

// The 32 k from k0 on that a lane has of a step: codes and scales of RT weight rows, MT
// rows of x.
template <int RT, int MT>
struct Step {
  u32x4 codes[RT];
  uint32_t scales[RT];
  u32x4 x[MT][4];
};

template <int RT, int MT, int WAVES>
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
  using S = Step<RT, MT>;
  auto load = [&](int step, S& s) {
    const int k = step * kStepK + 32 * g, blocks = min(max((a.K - k) / 16, 0), 2);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      s.codes[rt] = u32x4{};
      s.scales[rt] = 0;
      if (blocks == 2) {
        __builtin_memcpy(&s.codes[rt], codes[rt] + k / 2, 16);
        s.scales[rt] = scales[rt][k / 16] | scales[rt][k / 16 + 1] << 8;
      } else if (blocks == 1) {
        const u32x2 c = *reinterpret_cast<const u32x2*>(codes[rt] + k / 2);
        s.codes[rt] = u32x4{c.x, c.y, 0u, 0u};
        s.scales[rt] = scales[rt][k / 16];
      }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s.x[mt][i] = u32x4{};
        if (live[mt] && i / 2 < blocks) s.x[mt][i] = *reinterpret_cast<const u32x4*>(x[mt] + k + 8 * i);
      }
  };
  f32x4 acc[RT][MT] = {};
  auto multiply = [&](const S& s) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const float s0 = __builtin_amdgcn_cvt_f32_fp8(s.scales[rt], 0), s1 = __builtin_amdgcn_cvt_f32_fp8(s.scales[rt], 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bf16x8 w = decode8_bf16(s.codes[rt][i], i < 2 ? s0 : s1);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          acc[rt][mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8, s.x[mt][i]), acc[rt][mt], 0, 0, 0);
      }
    }
  };
  const int steps = (a.K + kStepK - 1) / kStepK;
  S s0, s1;
  int t = wave;
  if (t < steps) load(t, s0);
  while (t < steps) {
    if (t + WAVES < steps) load(t + WAVES, s1);
    multiply(s0);
    t += WAVES;
    if (t >= steps) break;
    if (t + WAVES < steps) load(t + WAVES, s0);
    multiply(s1);
    t += WAVES;
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
      float z = y[r] * sw;
      if (a.bias) z += bf16_bits_to_f32(a.bias[min(n + r, a.N - 1)]);
      if (a.epilogue == NVFP4_EPI_GELU) z = gelu_erf(z);
      out[r] = (uint16_t)bf16x2_rne(z, 0.0f);
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

template <int RT, int WAVES>
void launch_rows(const WeightOnly& a, int mt, hipStream_t stream) {
  const dim3 grid((unsigned)((a.N + 16 * RT - 1) / (16 * RT)), (unsigned)((a.M + 16 * mt - 1) / (16 * mt))), block(64 * WAVES);
  if (mt == 1)
    weight_only_kernel<RT, 1, WAVES><<<grid, block, 0, stream>>>(a);
  else if (mt == 2)
    weight_only_kernel<RT, 2, WAVES><<<grid, block, 0, stream>>>(a);
  else
    weight_only_kernel<RT, 4, WAVES><<<grid, block, 0, stream>>>(a);
}

}  // namespace

hipError_t launch_weight_only(WeightOnly a, hipStream_t stream) {
  if (a.amax) zero_product_amax_kernel<<<1, 1, 0, stream>>>(a.amax);
  if (a.M > 0 && a.N > 0) launch_rows<1, 8>(a, a.M <= 16 ? 1 : a.M <= 32 ? 2 : 4, stream);
  return hipGetLastError();
}

}  // namespace nvfp4
