// w4_gemm_weight_only: a few rows of bf16 activations, not quantized, times an NVFP4
// weight.
//
// Bound by the stream of codes, 0.5625 bytes an element: at a copy's 5.16 TB/s a weight
// of 28672 x 8192 takes 25.6 us, one of 4096 x 4096 1.8.  A code times its block scale
// has at most six significant bits, so bf16 holds it and the products are those of the
// formula; sums are binary32.
//
// weight_only_vector_kernel: one or two rows, by dot products along k.
// weight_only_ring_kernel: up to 16, by matrix instructions; codes and x reach LDS in whole
// lines.
// weight_only_lds_kernel: more rows of a large weight; x to registers.
// weight_only_kernel: codes straight to registers too, for any K and any place of the
// codes, and for more than 16 rows of a small weight.
// All of them split K over the waves of a workgroup, which meet in LDS in a fixed order.
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
__device__ __forceinline__ uint32_t finish(const WeightOnly& a, float y, float sw, float bias) {
  float z = __builtin_fmaf(y, sw, bias);
  if (a.epilogue == NVFP4_EPI_GELU) z = gelu_erf(z);
  return bf16x2_rne(z, 0.0f);
}

// Raises the amax word to the largest magnitude of a workgroup, each wave's in its lanes'
// `top`.  One atomic a workgroup, without a look at the word before: few end at a time,
// and a look would be waited for.
template <int WAVES>
__device__ __forceinline__ void raise_by(const WeightOnly& a, uint32_t top) {
  __shared__ uint32_t tops[WAVES];
  if (!a.amax) return;
  top = wave_max_u32(top);
  if ((threadIdx.x & 63) == 0) tops[wave_id()] = top;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < WAVES; ++w) top = max(top, tops[w]);
    if (top) atomicMax(a.amax, top << 16);
  }
}

// The end of a workgroup: the waves' sums of its tiles, in wave order, to outputs, a tile
// a wave.  Bias and tensor scale are on their way from the start.
template <int RT, int MT, int WAVES>
struct Ending {
  static_assert(RT * MT <= WAVES, "a tile a wave");
  int n;
  int64_t row;
  bool live;
  float sw;
  uint32_t bias[4];                            // bf16

  __device__ __forceinline__ void start(const WeightOnly& a, int n0, int64_t m0) {
    const int lane = threadIdx.x & 63, wave = wave_id();
    n = n0 + 16 * (wave / MT) + 4 * (lane >> 4);
    row = m0 + 16 * (wave % MT) + (lane & 15);
    live = wave < RT * MT && row < a.M && n < a.N;
    sw = *a.tensor_scale;
    // (without a bias the loads are of the tensor scale: a branch would be waited for here)
    const uint16_t* from = a.bias ? a.bias : reinterpret_cast<const uint16_t*>(a.tensor_scale);
#pragma unroll
    for (int r = 0; r < 4; ++r) bias[r] = from[a.bias ? min(n + r, a.N - 1) : 0];
  }
  __device__ __forceinline__ void write(const WeightOnly& a, const f32x4 (&acc)[RT][MT], f32x4 (*park)[RT * MT][64]) const {
    const int lane = threadIdx.x & 63, wave = wave_id();
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) park[wave][rt * MT + mt][lane] = acc[rt][mt];
    __syncthreads();
    uint32_t top = 0;
    if (live) {
      f32x4 y = park[0][wave][lane];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) y += park[w][wave][lane];
      uint32_t out[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        out[r] = finish(a, y[r], sw, a.bias ? bf16_bits_to_f32(bias[r]) : 0.0f);
        if (n + r < a.N) top = max(top, out[r] & 0x7FFFu);
      }
      uint16_t* to = a.y + row * a.N + n;
      if (a.N % 4 == 0) {
        *reinterpret_cast<u32x2*>(to) = u32x2{(out[0] & 0xFFFFu) | out[1] << 16, (out[2] & 0xFFFFu) | out[3] << 16};
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (n + r < a.N) to[r] = (uint16_t)out[r];
      }
    }
    raise_by<WAVES>(a, top);
  }
};

// A wave has RT tiles of 16 weight rows and MT of 16 rows of x, and steps of U times 128
// k, whose codes are on their way together; x is read from the caches step by step.  The
// matrix instruction wants 16 bytes of 16 weight rows from neighbouring lanes, so every
// load touches 64 places, one a cycle: 28672 x 8192 takes 45 to 58 us for 4 rows, whatever
// RT (1, 2, 4), U (1 to 8) and WAVES (2 to 16), and no longer for more bytes in flight.
template <int RT, int MT, int U, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void weight_only_kernel(WeightOnly a) {
  __shared__ f32x4 park[WAVES][RT * MT][64];
  const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4, wave = wave_id();
  const int n0 = (int)blockIdx.x * (16 * RT);
  const int64_t m0 = (int64_t)blockIdx.y * (16 * MT);
  Ending<RT, MT, WAVES> ending;
  ending.start(a, n0, m0);
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
  ending.write(a, acc, park);
}

// One or two rows of x: the lanes lie along k, 32 each, so a wave reads 1 KiB of a
// weight row at a time and keeps its part of x in registers over kRows weight rows.
// Sums over the lanes come last.  The dot instruction takes pairs of codes as bf16
// without their scale; a block's sum is multiplied by it in binary32, so an element costs
// about one instruction (with matrix instructions, two to decode it).  28672 x 8192: 24 to
// 25 us for one row (43 with matrix instructions), 5.2 TB/s, 31 for two; 8192 x 28672 28;
// 4096 x 4096 4.7, of which the codes' stream is 1.8 and the rest is a launch's latencies.
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
      const uint32_t out = finish(a, y, *a.tensor_scale, a.bias ? bf16_bits_to_f32(a.bias[n]) : 0.0f);
      a.y[(m0 + m) * a.N + n] = (uint16_t)out;
      top = out & 0x7FFFu;
    }
  }
  if (a.amax) {                                // outputs are the first wave's
    top = wave_max_u32(top);
    if (threadIdx.x == 0 && top) raise_amax(a.amax, top << 16);
  }
}

// Steps of 256 k, 128 bytes of each of 16 RT weight rows, on their way to LDS of a wave's
// own, 8 rows to a load, so that a load touches 16 places instead of 64; the 16-byte
// pieces of a row are permuted by XOR, so that the reads of 16 rows spread over the banks.
constexpr int kRingK = 256, kCodes = 16 * 128;

template <int RT>
struct WeightRing {
  static constexpr int kBytes = RT * (kCodes + 256), kLoads = 3 * RT;     // of a step
  const uint8_t *codes[RT][2], *scales[RT];
  uint32_t at[2], at_s;

  // own_at: the LDS address of the wave's first stage.
  __device__ __forceinline__ void start(const WeightOnly& a, int n0, uint32_t own_at) {
    const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = 8 * i + lane / 8, piece = (lane & 7) ^ (row >> 1);
        codes[rt][i] = a.codes + (int64_t)min(n0 + 16 * rt + row, a.N - 1) * (a.K / 2) + 16 * piece;
      }
      scales[rt] = a.scales + (int64_t)min(n0 + 16 * rt + lane / 4, a.N - 1) * (a.K / 16) + 4 * (lane & 3);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) at[u] = own_at + (uint32_t)(m * 128 + (((4 * u + g) ^ (m >> 1)) << 4));
    at_s = own_at + (uint32_t)(RT * kCodes + m * 16 + 2 * g);
  }
  __device__ __forceinline__ void fetch(int step, uint8_t* stage) const {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) to_lds<16>(codes[rt][i] + (uint32_t)step * 128u, stage + rt * kCodes + i * 1024);
      to_lds<4>(scales[rt] + (uint32_t)step * 16u, stage + RT * kCodes + rt * 256);
    }
  }
  // Adds the products of a step that has arrived, `stage` bytes behind the first stage;
  // v: x at k 128 u + 32 g + 8 i.
  template <int MT>
  __device__ __forceinline__ void multiply(uint32_t stage, const u32x4 (&v)[2][MT][4], f32x4 (&acc)[RT][MT]) const {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      u32x4 c[2];
      uint32_t sc[2];
      const uint32_t to = stage + (uint32_t)(rt * kCodes), to_s = stage + (uint32_t)(rt * 256);
      asm volatile(
          "ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\tds_read_u16 %2, %6\n\tds_read_u16 %3, %6 offset:8\n\t"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(c[0]), "=&v"(c[1]), "=&v"(sc[0]), "=&v"(sc[1])
          : "v"(at[0] + to), "v"(at[1] + to), "v"(at_s + to_s)
          : "memory");
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float s0 = __builtin_amdgcn_cvt_f32_fp8(sc[u], 0), s1 = __builtin_amdgcn_cvt_f32_fp8(sc[u], 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bf16x8 w = decode8_bf16(c[u][i], i < 2 ? s0 : s1);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            acc[rt][mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8, v[u][mt][i]), acc[rt][mt], 0, 0, 0);
        }
      }
    }
  }
};

// Waits until all but the last N loads have arrived.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "the count is 6 bits");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
  asm volatile("" ::: "memory");
}

// 3 to 16 rows of x, which goes to LDS as well, two rows of 512 bytes to a load, its pieces
// permuted the same way (loaded as the matrix instruction wants it, each load touches 64
// places: 14336 x 4096 13.5 us instead of 12.1, 28672 x 8192 45 instead of 39 to 41, 8192 x
// 28672 48 instead of 38 to 42, for 16 rows; 14336 x 4096 with bias, GELU and amax 16.9
// instead of 14.9).  A ring of two stages a wave.  What is left is decoding, about two
// instructions an element, with one wave a SIMD to hide the rest.
template <int RT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void weight_only_ring_kernel(WeightOnly a) {
  constexpr int kAtX = WeightRing<RT>::kBytes, kStage = kAtX + 16 * 2 * kRingK, kXLoads = 8;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[WAVES * 2 * kStage];
  static_assert(sizeof(ring) >= WAVES * RT * 1024, "the waves' sums meet in the ring");
  const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4, wave = wave_id();
  const int n0 = (int)blockIdx.x * (16 * RT);
  Ending<RT, 1, WAVES> ending;
  ending.start(a, n0, 0);
  uint8_t* own = ring + wave * (2 * kStage);
  const uint32_t own_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)own;
  WeightRing<RT> weight;
  weight.start(a, n0, own_at);
  const uint16_t* x[kXLoads];                  // (rows past the last are the last's)
#pragma unroll
  for (int j = 0; j < kXLoads; ++j) {
    const int row = 2 * j + lane / 32, piece = (lane & 31) ^ row;
    x[j] = a.x + min((int64_t)row, a.M - 1) * a.K + 8 * piece;
  }
  uint32_t at_x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) at_x[i] = own_at + (uint32_t)(kAtX + m * 512 + (((4 * g + i) ^ m) << 4));
  auto fetch = [&](int step, int stage) {
    uint8_t* to = own + stage * kStage;
#pragma unroll
    for (int j = 0; j < kXLoads; ++j)
      to_lds<16, 0>(reinterpret_cast<const uint8_t*>(x[j] + (uint32_t)(step * kRingK)), to + kAtX + j * 1024);
    weight.fetch(step, to);
  };
  const int steps = a.K / kRingK;
  f32x4 acc[RT][1] = {};
  if (wave < steps) fetch(wave, 0);
  int stage = 0;
  for (int t = wave; t < steps; t += WAVES, stage ^= 1) {
    if (t + WAVES < steps) {
      fetch(t + WAVES, stage ^ 1);
      wait_loads<WeightRing<RT>::kLoads + kXLoads>();      // this step's are in
    } else {
      wait_loads<0>();
    }
    u32x4 v[2][1][4];
    const uint32_t to = (uint32_t)(stage * kStage);
    asm volatile(
        "ds_read_b128 %0, %8\n\tds_read_b128 %1, %9\n\tds_read_b128 %2, %10\n\tds_read_b128 %3, %11\n\t"
        "ds_read_b128 %4, %8 offset:256\n\tds_read_b128 %5, %9 offset:256\n\t"
        "ds_read_b128 %6, %10 offset:256\n\tds_read_b128 %7, %11 offset:256\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(v[0][0][0]), "=&v"(v[0][0][1]), "=&v"(v[0][0][2]), "=&v"(v[0][0][3]), "=&v"(v[1][0][0]),
          "=&v"(v[1][0][1]), "=&v"(v[1][0][2]), "=&v"(v[1][0][3])
        : "v"(at_x[0] + to), "v"(at_x[1] + to), "v"(at_x[2] + to), "v"(at_x[3] + to)
        : "memory");
    weight.multiply(to, v, acc);
  }
  __syncthreads();                             // the rings are free
  ending.write(a, acc, reinterpret_cast<f32x4(*)[RT][64]>(ring));
}

// 17 rows and more: two tiles of x, in registers a step ahead, before the codes (loads
// return in order); in LDS they would leave room for three waves.  The next step is on its
// way in every second turn alone: in the others the compiler waits for all loads before
// the products (x's registers come from two paths, with and without a next step; turns
// with one path spill).  28672 x 8192: 55 us for 17 rows, 65 for 32, 71 by
// weight_only_kernel; 8192 x 28672 77 and 90.
template <int RT, int MT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void weight_only_lds_kernel(WeightOnly a) {
  constexpr int kStage = WeightRing<RT>::kBytes;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[WAVES * 2 * kStage];
  static_assert(sizeof(ring) >= WAVES * RT * MT * 1024, "the waves' sums meet in the ring");
  const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4, wave = wave_id();
  const int n0 = (int)blockIdx.x * (16 * RT);
  const int64_t m0 = (int64_t)blockIdx.y * (16 * MT);
  Ending<RT, MT, WAVES> ending;
  ending.start(a, n0, m0);
  const uint16_t* x[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) x[mt] = a.x + min(m0 + 16 * mt + m, a.M - 1) * a.K + 32 * g;
  uint8_t* own = ring + wave * (2 * kStage);
  WeightRing<RT> weight;
  weight.start(a, n0, (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)own);
  u32x4 xv[2][2][MT][4];
  auto load_x = [&](int step, u32x4 (&v)[2][MT][4]) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[u][mt][i] = *reinterpret_cast<const u32x4*>(x[mt] + step * kRingK + 128 * u + 8 * i);
  };
  const int steps = a.K / kRingK;
  f32x4 acc[RT][MT] = {};
  auto turn = [&](int t, int stage, u32x4 (&now)[2][MT][4], u32x4 (&next)[2][MT][4]) {
    if (t + WAVES < steps) {
      load_x(t + WAVES, next);
      weight.fetch(t + WAVES, own + (stage ^ 1) * kStage);
      wait_loads<WeightRing<RT>::kLoads + 8 * MT>();       // this step's are in
    } else {
      wait_loads<0>();
    }
    weight.multiply((uint32_t)(stage * kStage), now, acc);
  };
  int t = wave;
  if (t < steps) {
    load_x(t, xv[0]);
    weight.fetch(t, own);
  }
  while (t < steps) {
    turn(t, 0, xv[0], xv[1]);
    t += WAVES;
    if (t >= steps) break;
    turn(t, 1, xv[1], xv[0]);
    t += WAVES;
  }
  __syncthreads();                             // the rings are free
  ending.write(a, acc, reinterpret_cast<f32x4(*)[RT * MT][64]>(ring));
}

template <int RT, int MT, int U, int WAVES>
void launch_rows(const WeightOnly& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.N + 16 * RT - 1) / (16 * RT)), (unsigned)((a.M + 16 * MT - 1) / (16 * MT)));
  weight_only_kernel<RT, MT, U, WAVES><<<grid, 64 * WAVES, 0, stream>>>(a);
}
template <int RT>
void launch_ring(const WeightOnly& a, hipStream_t stream) {
  weight_only_ring_kernel<RT, 4><<<(unsigned)((a.N + 16 * RT - 1) / (16 * RT)), 256, 0, stream>>>(a);
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
  const int64_t tiles = (a.N + 15) / 16, cus = compute_units();
  const bool one = a.M <= 16;
  // (the rings take 16 and 4 bytes at a time from rows that begin so)
  const bool placed = a.K % kRingK == 0 && ((uintptr_t)a.codes & 15) == 0 && ((uintptr_t)a.scales & 3) == 0;
  if (placed && one) {
    // The fewest tiles a workgroup that leave a compute unit one, whose LDS its rings fill;
    // four are the most.  16 rows with one, two and four tiles: 4096 x 4096 6.0, 7.2 and
    // 11.1 us; 8192 x 28672 50, 38 and 54; 14336 x 4096 18.9, 13.9 and 12.2.  In workgroups
    // of 6 or 7 waves the first two take as long or longer.
    if (tiles <= cus)
      launch_ring<1>(a, stream);
    else if (tiles <= 2 * cus)
      launch_ring<2>(a, stream);
    else
      launch_ring<4>(a, stream);
  } else if (placed && tiles >= 3 * cus) {
    // 17 to 32 rows of a large weight 18.6 us against 20.0 by weight_only_kernel, of a small
    // one 40 against 12.  More than 32 rows in passes of 32: 64 rows of 28672 x 8192 124 us,
    // in one pass of four tiles of x 159.
    const dim3 grid((unsigned)((a.N + 63) / 64), (unsigned)((a.M + 31) / 32));
    weight_only_lds_kernel<4, 2, 8><<<grid, 512, 0, stream>>>(a);
  } else if (2 * tiles >= 3 * cus) {
    one ? launch_rows<2, 1, 2, 8>(a, stream) : launch_rows<2, 2, 1, 8>(a, stream);
  } else {
    one ? launch_rows<1, 1, 4, 8>(a, stream) : launch_rows<1, 2, 2, 8>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace nvfp4
