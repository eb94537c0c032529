// dit_rotary: rotary positions on query and key heads, with the per-head RMS
// norm in front of them, in one launch over both tensors.
//
//   z = v, or v * rsqrt(mean(v^2) + eps) * weight        (over the head's `dim` elements)
//   pair j of the first rotary_dim elements, t = turns[j] * position[axis[j]]:
//     a' = m (a cos 2 pi t - b sin 2 pi t),  b' = m (b cos 2 pi t + a sin 2 pi t)
//
// (a, b) are elements (2j, 2j + 1) of the interleaved layout, (j, j + rotary_dim
// / 2) of the half layout; elements from rotary_dim on are z.
//
// Bound: HBM, 4 bytes an element.  Angles: turns are binary64 and so is their
// product with the position, of which only the fraction of a turn is kept
// before it becomes binary32 -- an angle in binary32 would be off by 1e-2 rad
// at position 10^5.  A workgroup takes a few tokens, computes their cosines and
// sines once into LDS, and every head of the token reads them there; a table in
// memory would add a pass for its making and its bytes to every call.
#include "device_common.hpp"
#include "kernels.hpp"

namespace nvfp4 {

namespace {

constexpr int kRotThreads = 256;
constexpr int kRotEntries = 512;   // (cos, sin) pairs a workgroup keeps: 4 KB of LDS

__device__ __forceinline__ void unpack8(u32x4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = __uint_as_float(w[j] << 16);
    f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}

// One head is held by LANES neighbouring lanes of 8 elements each (the ones
// past dim / 8 idle), so a head's norm is a sum over LANES lanes and the half
// layout's partner elements are one lane exchange away.
template <int LANES>
__global__ __launch_bounds__(kRotThreads) void rotary_kernel(Rotary a) {
  __shared__ float2 turn[kRotEntries];
  const int pairs = a.rotary_dim / 2;
  const int64_t first = (int64_t)blockIdx.x * a.tokens_per_group;
  const int here = (int)(a.rows - first < a.tokens_per_group ? a.rows - first : a.tokens_per_group);
  for (int e = threadIdx.x; e < here * pairs; e += kRotThreads) {
    const int t = e / pairs, j = e - t * pairs;
    // an axis index outside the positions' axes reads the nearest one
    const int ax = a.axis ? min(max(a.axis[j], 0), a.axes - 1) : 0;
    const double rev = a.turns[j] * (double)a.positions[(first + t) * a.axes + ax];
    const float part = (float)(rev - __builtin_rint(rev));    // [-1/2, 1/2]
    float s, c;
    sincospif(2.0f * part, &s, &c);
    turn[e] = float2{c * a.magnitude, s * a.magnitude};
  }
  __syncthreads();
  const int chunk = threadIdx.x % LANES, slot = threadIdx.x / LANES;
  const int chunks = a.dim / 8, rot_chunks = a.rotary_dim / 8;
  const bool mine = chunk < chunks;
  const bool turned = chunk < rot_chunks;
  const int heads = a.q.heads + a.k.heads;
  const int half_chunks = rot_chunks / 2;
  // the half layout's partner chunk: that many lanes up or down
  const bool upper = chunk >= half_chunks;
  const int partner = (threadIdx.x & 63) + (upper ? -half_chunks : half_chunks);
  for (int base = 0; base < here * heads; base += kRotThreads / LANES) {
    const int item = base + slot;
    const bool live = item < here * heads && mine;
    const int t = item / heads, head = item - t * heads;
    const bool is_q = head < a.q.heads;
    const RotaryHeads& v = is_q ? a.q : a.k;
    const int hd = is_q ? head : head - a.q.heads;
    const int64_t row = first + t, batch = row / a.tokens, token = row - batch * a.tokens;
    u32x4 raw = u32x4{0u, 0u, 0u, 0u};
    if (live)
      raw = *reinterpret_cast<const u32x4*>(v.in + batch * v.in_batch + token * v.in_token +
                                            hd * v.in_head + 8 * chunk);
    float f[8];
    unpack8(raw, f);
    float rstd = 1.0f;
    if (v.weight) {
      float q = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) q = __builtin_fmaf(f[j], f[j], q);
#pragma unroll
      for (int o = LANES / 2; o >= 1; o >>= 1) q += __shfl_xor(q, o, 64);
      rstd = 1.0f / __builtin_sqrtf(q * a.inv_dim + a.eps);
      if (live) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = f[j] * rstd * v.weight[8 * chunk + j];
      }
    }
    u32x4 out;
    if (a.layout == DIT_ROTARY_INTERLEAVED) {
      if (live && turned) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 cs = turn[t * pairs + 4 * chunk + j];
          const float x = f[2 * j], y = f[2 * j + 1];
          f[2 * j] = x * cs.x - y * cs.y;
          f[2 * j + 1] = y * cs.x + x * cs.y;
        }
      }
    } else {
      float g[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = __shfl(f[j], partner, 64);
      if (live && turned) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 cs = turn[t * pairs + 8 * (upper ? chunk - half_chunks : chunk) + j];
          f[j] = upper ? f[j] * cs.x + g[j] * cs.y : f[j] * cs.x - g[j] * cs.y;
        }
      }
    }
    out = u32x4{bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]), bf16x2_rne(f[4], f[5]),
                bf16x2_rne(f[6], f[7])};
    if (!v.weight && !turned) out = raw;      // untouched elements keep their bits
    if (live)
      *reinterpret_cast<u32x4*>(v.out + batch * v.out_batch + token * v.out_token +
                                hd * v.out_head + 8 * chunk) = out;
  }
}

template <int LANES>
hipError_t launch(const Rotary& a, int64_t grid, hipStream_t stream) {
  rotary_kernel<LANES><<<dim3((unsigned)grid), dim3(kRotThreads), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rotary(Rotary a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  // tokens a workgroup takes: as many as its table holds, fewer while that
  // would leave compute units without a workgroup
  const int64_t fill = (a.rows + 4 * compute_units() - 1) / (4 * compute_units());
  int per = kRotEntries / (a.rotary_dim / 2);
  if (per > 8) per = 8;
  if (per > fill) per = (int)fill;
  a.tokens_per_group = per;
  const int64_t grid = (a.rows + per - 1) / per;
  const int chunks = a.dim / 8;
  if (chunks <= 4) return launch<4>(a, grid, stream);
  if (chunks <= 8) return launch<8>(a, grid, stream);
  if (chunks <= 16) return launch<16>(a, grid, stream);
  return launch<32>(a, grid, stream);
}

}  // namespace nvfp4
