// dit_gated_norm: what lies between two linears of a transformer block, in one
// pass over the tokens.  Per token row of C channels:
//
//   z = y                       or  P(y) * post_weight   (P: layer or RMS norm)
//   r = residual_scale * x + gate * z                    (written; stays unrounded below)
//   h = (N(r) * weight + bias) * (1 + scale) + shift     (N: layer or RMS norm)
//
// layer: (v - mean) / sqrt(mean((v - mean)^2) + eps);  RMS: v / sqrt(mean(v^2) + eps).
//
// Bound: HBM.  x and y are read once, r and h written once (8 bytes a channel
// with a bf16 stream); the vectors over channels (gate, scale, shift, weights)
// are re-read per row from the caches or held.  One workgroup owns a row at a time and
// keeps it in registers between the statistics and the outputs, so each
// statistic is over values already on chip; mean and variance are two sums, the
// second of squared distances from the mean, so channels with a large common
// offset lose nothing.  All of it is binary32; r and h are each rounded once.
//
// Measured at 16896 x 3072 (bf16, gate, norm, scale and shift): 77 us, 415 MB at
// 5.4 TB/s; a copy of 1 GiB reaches 4.6.
#include "device_common.hpp"
#include "kernels.hpp"

namespace nvfp4 {

namespace {

// Sum over a row.  LANES > 0: the row is LANES neighbouring lanes.  LANES 0: it is
// the whole workgroup of `waves` waves; `red` alternates between two halves from
// one sum to the next, so one barrier a sum is enough.
template <int LANES>
__device__ __forceinline__ float row_sum(float v, int waves, float (*red)[16], int& half) {
  if constexpr (LANES == 64) return wave_sum(v);
  if constexpr (LANES > 0) return group_sum<LANES>(v);
  v = wave_sum(v);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (lane == 0) red[half][wave] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < waves; ++w) s += red[half][w];
  half ^= 1;
  return s;
}

template <class T> struct Raw;
template <> struct Raw<uint16_t> { u32x4 v; };            // 8 bf16
template <> struct Raw<float> { f32x4 lo, hi; };

__device__ __forceinline__ Raw<uint16_t> load8(const uint16_t* p) {
  return {*reinterpret_cast<const u32x4*>(p)};
}
// x, y, r and h pass through once: they are streamed past the caches, which stay
// with the vectors over channels (76 us against 81 at 16896 x 3072, 135 against 147
// at 6144 channels; with an fp32 stream it does not matter at 3072, 124 against 122,
// and costs up to 8 % at 4608 and 5120).
__device__ __forceinline__ Raw<uint16_t> take8(const uint16_t* p) {
  return {__builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p))};
}
__device__ __forceinline__ Raw<float> take8(const float* p) {
  return {__builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p)),
          __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p) + 1)};
}
__device__ __forceinline__ Raw<float> load8(const float* p) {
  return {reinterpret_cast<const f32x4*>(p)[0], reinterpret_cast<const f32x4*>(p)[1]};
}
__device__ __forceinline__ void widen(const Raw<uint16_t>& a, float (&f)[8]) {
  const uint32_t w[4] = {a.v.x, a.v.y, a.v.z, a.v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = __uint_as_float(w[j] << 16);
    f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void widen(const Raw<float>& a, float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[j] = a.lo[j];
    f[4 + j] = a.hi[j];
  }
}
__device__ __forceinline__ u32x4 pack8(const float (&f)[8]) {
  return u32x4{bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]), bf16x2_rne(f[4], f[5]),
               bf16x2_rne(f[6], f[7])};
}
__device__ __forceinline__ void put8(uint16_t* p, const float (&f)[8]) {
  __builtin_nontemporal_store(pack8(f), reinterpret_cast<u32x4*>(p));
}
__device__ __forceinline__ void put8(float* p, const float (&f)[8]) {
  __builtin_nontemporal_store(f32x4{f[0], f[1], f[2], f[3]}, reinterpret_cast<f32x4*>(p));
  __builtin_nontemporal_store(f32x4{f[4], f[5], f[6], f[7]}, reinterpret_cast<f32x4*>(p) + 1);
}

// v := (v - mean) * rstd of the row, in place; `mine[i]`: chunk i of this
// thread exists.
template <int LANES, int CH>
__device__ __forceinline__ void normalise(float (&v)[CH][8], const bool (&mine)[CH], int kind,
                                          float inv_c, float eps, int waves, float (*red)[16],
                                          int& half) {
  float mean = 0.0f;
  if (kind == DIT_NORM_LAYER) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[i][j];      // absent chunks hold zeros
    mean = row_sum<LANES>(s, waves, red, half) * inv_c;
  }
  float q = 0.0f;
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[i][j] -= mean;
      q = mine[i] ? __builtin_fmaf(v[i][j], v[i][j], q) : q;
    }
  const float rstd = __builtin_amdgcn_rsqf(row_sum<LANES>(q, waves, red, half) * inv_c + eps);
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] *= rstd;
}

// Rows of up to 64 chunks of 8 channels are held by LANES neighbouring lanes, one
// chunk each, and a workgroup of 256 threads takes 256 / LANES of them at a time;
// longer ones (LANES 0) by the whole workgroup, CH chunks a thread.
//
// HOLD: gate, scale and shift (of type MT) stay in registers for as long as the batch
// entry lasts.  Loaded within the row they come after the next row's loads, and
// waiting for them is waiting for those: at 16896 x 3072 83 us against 76, with an
// fp32 stream 156 against 124, with weights and a post-norm besides 188 against 145.
// Two chunks a lane would take too many registers.
template <class XT, class MT, bool HOLD, int CH, int LANES>
__global__ __launch_bounds__(LANES > 0 ? 256 : 1024) void gated_norm_kernel(GatedNorm a) {
  __shared__ float red[2][16];
  int half = 0;
  const int waves = blockDim.x >> 6, chunks = a.channels >> 3;
  bool mine[CH];
  int at[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = LANES > 0 ? threadIdx.x % (LANES > 0 ? LANES : 1) : threadIdx.x + i * blockDim.x;
    mine[i] = c < chunks;
    at[i] = mine[i] ? 8 * c : 0;
  }
  const XT* x = static_cast<const XT*>(a.x);
  XT* r_out = static_cast<XT*>(a.residual);
  u16x2 top = {0, 0};
  constexpr int kRows = LANES > 0 ? 256 / (LANES > 0 ? LANES : 1) : 1;    // at a time
  int64_t row = (int64_t)blockIdx.x * kRows + (LANES > 0 ? threadIdx.x / (LANES > 0 ? LANES : 1) : 0);
  const int64_t step = (int64_t)gridDim.x * kRows;
  Raw<XT> xr[CH];
  Raw<uint16_t> yr[CH];
  auto fetch = [&](int64_t of) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (!mine[i]) continue;
      xr[i] = take8(x + of * a.channels + at[i]);
      if (a.y) yr[i] = take8(a.y + of * a.channels + at[i]);
    }
  };
  Raw<MT> gate[CH], scale[CH], shift[CH];
  auto modulation = [&](const void* base, int64_t stride, int64_t batch, int i) {
    return load8(static_cast<const MT*>(base) + batch * stride + at[i]);
  };
  int64_t entry = -1;                            // whose modulation is held
  if (row < a.rows) fetch(row);
  while (row < a.rows) {
    const int64_t batch = row / a.tokens;
    if (HOLD && batch != entry) {
      entry = batch;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        if (a.gate) gate[i] = modulation(a.gate, a.gate_stride, batch, i);
        if (a.scale) scale[i] = modulation(a.scale, a.scale_stride, batch, i);
        if (a.shift) shift[i] = modulation(a.shift, a.shift_stride, batch, i);
      }
    }
    float v[CH][8], z[CH][8];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = z[i][j] = 0.0f;
      if (!mine[i]) continue;
      widen(xr[i], v[i]);
      if (a.y) widen(yr[i], z[i]);
    }
    const int64_t next = row + step;
    if (next < a.rows) fetch(next);          // the next row's loads run under this row's sums
    if (a.y) {
      if (a.post_norm != DIT_NORM_NONE)
        normalise<LANES, CH>(z, mine, a.post_norm, a.inv_c, a.eps, waves, red, half);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        if (!mine[i]) continue;
        float f[8];
        if (a.post_weight) {
          widen(load8(a.post_weight + at[i]), f);
#pragma unroll
          for (int j = 0; j < 8; ++j) z[i][j] *= f[j];
        }
        if (a.gate) {
          widen(HOLD ? gate[i] : modulation(a.gate, a.gate_stride, batch, i), f);
#pragma unroll
          for (int j = 0; j < 8; ++j) z[i][j] *= f[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = __builtin_fmaf(a.residual_scale, v[i][j], z[i][j]);
      }
    }
    if (r_out) {
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if (mine[i]) put8(r_out + row * a.channels + at[i], v[i]);
    }
    if (a.h) {
      if (a.norm != DIT_NORM_NONE)
        normalise<LANES, CH>(v, mine, a.norm, a.inv_c, a.eps, waves, red, half);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        if (!mine[i]) continue;
        float f[8];
        if (a.weight) {
          widen(load8(a.weight + at[i]), f);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] *= f[j];
        }
        if (a.bias) {
          widen(load8(a.bias + at[i]), f);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] += f[j];
        }
        if (a.scale) {
          widen(HOLD ? scale[i] : modulation(a.scale, a.scale_stride, batch, i), f);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] = __builtin_fmaf(v[i][j], f[j], v[i][j]);
        }
        if (a.shift) {
          widen(HOLD ? shift[i] : modulation(a.shift, a.shift_stride, batch, i), f);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] += f[j];
        }
        const u32x4 p = pack8(v[i]);
        __builtin_nontemporal_store(p, reinterpret_cast<u32x4*>(a.h + row * a.channels + at[i]));
        top = max_u16x2(top, max8(p));
      }
    }
    row = next;
  }
  if (a.amax) {
    __shared__ uint32_t wave_top[16];
    const uint32_t m = wave_max_u32((uint32_t)(top.x > top.y ? top.x : top.y) << 16);
    if ((threadIdx.x & 63) == 0) wave_top[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
      uint32_t t = 0;
      for (int w = 0; w < (int)(blockDim.x >> 6); ++w) t = max(t, wave_top[w]);
      raise_amax(a.amax, t);
    }
  }
}

__global__ void zero_amax_kernel(uint32_t* p) { *p = 0u; }

template <class XT, class MT, int CH, int LANES>
hipError_t launch_hold(const GatedNorm& a, bool hold, int threads, int64_t grid, hipStream_t stream) {
  if (CH == 1 && hold)
    gated_norm_kernel<XT, MT, CH == 1, CH, LANES><<<dim3((unsigned)grid), dim3(threads), 0, stream>>>(a);
  else
    gated_norm_kernel<XT, MT, false, CH, LANES><<<dim3((unsigned)grid), dim3(threads), 0, stream>>>(a);
  return hipGetLastError();
}

template <int CH, int LANES>
hipError_t launch(const GatedNorm& a, bool x_fp32, bool hold, int threads, int64_t grid,
                  hipStream_t stream) {
  if (x_fp32)
    return a.mod_fp32 ? launch_hold<float, float, CH, LANES>(a, hold, threads, grid, stream)
                      : launch_hold<float, uint16_t, CH, LANES>(a, hold, threads, grid, stream);
  return a.mod_fp32 ? launch_hold<uint16_t, float, CH, LANES>(a, hold, threads, grid, stream)
                    : launch_hold<uint16_t, uint16_t, CH, LANES>(a, hold, threads, grid, stream);
}

}  // namespace

hipError_t launch_gated_norm(const GatedNorm& a, bool x_fp32, hipStream_t stream) {
  if (a.amax) {
    zero_amax_kernel<<<1, 1, 0, stream>>>(a.amax);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.rows == 0) return hipSuccess;
  const int chunks = a.channels / 8;
  // One chunk a lane up to 8192 channels: more waves with less to hold each load
  // more at once (at 16896 x 3072, nothing held, two chunks a lane take 106 us, one
  // 83).  Rows are spread evenly over the rounds.  Up to two rounds of 24 waves a
  // compute unit nothing is held: the first loads count (3063 x 1536, fp32 stream, all
  // vectors: 14.2 us, 15.3 held; at 16896 x 3072, nothing held, 18 waves take 89 us, 24
  // 83, 30, more than the registers hold, 107).  Past that modulations are held, and a
  // compute unit has the whole workgroups that 20 waves make, of an fp32 stream 16: at
  // 3072 channels, 6 waves a workgroup, 3 and 2 (76 and 124 us; 2 and 4 of bf16 80 and
  // 85, 3 of fp32 143).  From 5128 channels on (fp32: 4104) it is one workgroup, no
  // slower than two held (16896 x 6144: 135 us against 149, fp32 241 both) and, but
  // for 2 % of an fp32 stream, than nothing held (150, 237).  Above 8192 channels two
  // chunks a lane and one workgroup of 16 waves: 4224 x 16384 110 us, 5.0 TB/s, 8448 x
  // 8200, where one lane alone has a second chunk, 144 us, 3.8.
  const int lanes = chunks <= 8 ? 8 : chunks <= 16 ? 16 : chunks <= 32 ? 32 : chunks <= 64 ? 64 : 0;
  const int waves = lanes ? 4 : chunks <= 1024 ? (chunks + 63) / 64 : 16;
  const int64_t turns = lanes ? (a.rows + 256 / lanes - 1) / (256 / lanes) : a.rows;
  const int64_t units = compute_units();
  const bool hold = turns > 2 * units * (24 / waves) && chunks <= 1024;
  const int64_t cap = units * ((!hold ? 24 : x_fp32 ? 16 : 20) / waves);
  const int64_t rounds = (turns + cap - 1) / cap;
  const int64_t grid = (turns + rounds - 1) / rounds;
  switch (lanes) {
    case 8: return launch<1, 8>(a, x_fp32, hold, 256, grid, stream);
    case 16: return launch<1, 16>(a, x_fp32, hold, 256, grid, stream);
    case 32: return launch<1, 32>(a, x_fp32, hold, 256, grid, stream);
    case 64: return launch<1, 64>(a, x_fp32, hold, 256, grid, stream);
  }
  return chunks <= 1024 ? launch<1, 0>(a, x_fp32, hold, 64 * waves, grid, stream)
                        : launch<2, 0>(a, x_fp32, hold, 1024, grid, stream);
}

}  // namespace nvfp4
