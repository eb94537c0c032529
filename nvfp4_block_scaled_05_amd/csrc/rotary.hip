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
//
// Measured in place on 24 + 24 heads of 128 in 16896 rows of a fused projection,
// with both norms, three axes: 77 us, 415 MB at 5.4 TB/s.
#include "device_common.hpp"
#include "kernels.hpp"

namespace nvfp4 {

namespace {

constexpr int kRotThreads = 256;
constexpr int kRotEntries = 512;   // (cos, sin) pairs a workgroup keeps: 4 KB of LDS
constexpr int kRotTokens = 32;     // and tokens, at most

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
template <int LANES, bool HALF, bool NORM, bool STREAM>
__global__ __launch_bounds__(kRotThreads) void rotary_kernel(Rotary a) {
  __shared__ float2 turn[kRotEntries];
  __shared__ __attribute__((aligned(16))) float weight[NORM ? 2 : 1][NORM ? 8 * LANES : 1];
  __shared__ int64_t place[kRotTokens][4];       // where each token's heads start: q, k, q out, k out
  const int pairs = a.rotary_dim / 2;
  const int chunk = threadIdx.x % LANES, slot = threadIdx.x / LANES;
  const int rot_chunks = a.rotary_dim / 8, half_chunks = rot_chunks / 2;
  const bool mine = chunk < a.dim / 8, turned = chunk < rot_chunks;
  const int heads = a.q.heads + a.k.heads;
  // the half layout's partner chunk: that many lanes up or down
  const bool upper = chunk >= half_chunks;
  const int partner = chunk + (upper ? -half_chunks : half_chunks);
  const int partner_lane = (threadIdx.x & 63) - chunk + partner;
  float wq[8], wk[8], pq[8], pk[8];              // the norms' weights of this lane's and its partner's elements
  if (NORM) {                                    // through LDS: loaded from memory by every lane, 106 us for 79
    for (int d = threadIdx.x; d < a.dim; d += kRotThreads) {
      weight[0][d] = a.q.weight ? a.q.weight[d] : 1.0f;
      weight[1][d] = a.k.weight ? a.k.weight[d] : 1.0f;
    }
    __syncthreads();
    const int own = mine ? 8 * chunk : 0, other = turned ? 8 * partner : 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      wq[j] = weight[0][own + j];
      wk[j] = weight[1][own + j];
      if (HALF) {
        pq[j] = weight[0][other + j];
        pk[j] = weight[1][other + j];
      }
    }
  }
  for (int64_t first = (int64_t)blockIdx.x * a.tokens_per_group; first < a.rows;
       first += (int64_t)gridDim.x * a.tokens_per_group) {
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
    if (threadIdx.x < here) {
      const uint32_t row = (uint32_t)(first + threadIdx.x), batch = row / (uint32_t)a.tokens;
      const int64_t token = row - batch * (uint32_t)a.tokens;
      place[threadIdx.x][0] = batch * a.q.in_batch + token * a.q.in_token;
      place[threadIdx.x][1] = batch * a.k.in_batch + token * a.k.in_token;
      place[threadIdx.x][2] = batch * a.q.out_batch + token * a.q.out_token;
      place[threadIdx.x][3] = batch * a.k.out_batch + token * a.k.out_token;
    }
    __syncthreads();
    const int items = here * heads;
    int t = 0, head = slot;                      // item = t * heads + head
    while (head >= heads) head -= heads, ++t;
    u32x4 raw = u32x4{0u, 0u, 0u, 0u};
    auto fetch = [&](int tt, int hh) {
      const bool is_q = hh < a.q.heads;
      const RotaryHeads& v = is_q ? a.q : a.k;
      const int64_t at = place[tt][is_q ? 0 : 1] + (is_q ? hh : hh - a.q.heads) * v.in_head + 8 * chunk;
      const u32x4* from = reinterpret_cast<const u32x4*>(v.in + at);
      return STREAM ? __builtin_nontemporal_load(from) : *from;
    };
    if (slot < items && mine) raw = fetch(t, head);
    for (int base = 0; base < items; base += kRotThreads / LANES) {
      const bool live = base + slot < items && mine;
      const u32x4 now = raw;
      const int t_now = t, head_now = head;
      head += kRotThreads / LANES;
      while (head >= heads) head -= heads, ++t;
      // the next item's load runs under this one's arithmetic
      if (base + slot + kRotThreads / LANES < items && mine) raw = fetch(t, head);
      const bool is_q = head_now < a.q.heads;
      const bool normed = NORM && (is_q ? a.q.weight : a.k.weight) != nullptr;
      float f[8], g[8];
      unpack8(now, f);
      if (HALF)
        unpack8(u32x4{(uint32_t)__shfl((int)now.x, partner_lane, 64), (uint32_t)__shfl((int)now.y, partner_lane, 64),
                      (uint32_t)__shfl((int)now.z, partner_lane, 64), (uint32_t)__shfl((int)now.w, partner_lane, 64)},
                g);
      if (NORM) {
        float q = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) q = __builtin_fmaf(f[j], f[j], q);
        q = group_sum<LANES>(q);
        const float rstd = normed ? __builtin_amdgcn_rsqf(q * a.inv_dim + a.eps) : 1.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          f[j] = f[j] * rstd * (is_q ? wq[j] : wk[j]);
          if (HALF) g[j] = g[j] * rstd * (is_q ? pq[j] : pk[j]);
        }
      }
      if (live && turned) {
        if (HALF) {
          const float2* cs = turn + t_now * pairs + 8 * (upper ? partner : chunk);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 v = cs[j];
            f[j] = __builtin_fmaf(f[j], v.x, g[j] * (upper ? v.y : -v.y));
          }
        } else {
          const float2* cs = turn + t_now * pairs + 4 * chunk;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 v = cs[j];
            const float x = f[2 * j], y = f[2 * j + 1];
            f[2 * j] = __builtin_fmaf(x, v.x, -(y * v.y));
            f[2 * j + 1] = __builtin_fmaf(y, v.x, x * v.y);
          }
        }
      }
      u32x4 out = u32x4{bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]), bf16x2_rne(f[4], f[5]),
                        bf16x2_rne(f[6], f[7])};
      if (!normed && !turned) out = now;         // untouched elements keep their bits
      if (live) {
        const RotaryHeads& v = is_q ? a.q : a.k;
        const int64_t at = place[t_now][is_q ? 2 : 3] + (is_q ? head_now : head_now - a.q.heads) * v.out_head;
        u32x4* to = reinterpret_cast<u32x4*>(v.out + at + 8 * chunk);
        if constexpr (STREAM)
          __builtin_nontemporal_store(out, to);
        else
          *to = out;
      }
    }
    __syncthreads();                             // before the next tokens' table
  }
}

template <int LANES, bool HALF, bool STREAM>
hipError_t launch_norm(const Rotary& a, int64_t grid, hipStream_t stream) {
  if (a.q.weight || a.k.weight)
    rotary_kernel<LANES, HALF, true, STREAM><<<dim3((unsigned)grid), dim3(kRotThreads), 0, stream>>>(a);
  else
    rotary_kernel<LANES, HALF, false, STREAM><<<dim3((unsigned)grid), dim3(kRotThreads), 0, stream>>>(a);
  return hipGetLastError();
}

template <int LANES, bool STREAM>
hipError_t launch_layout(const Rotary& a, int64_t grid, hipStream_t stream) {
  return a.layout == DIT_ROTARY_HALF ? launch_norm<LANES, true, STREAM>(a, grid, stream)
                                     : launch_norm<LANES, false, STREAM>(a, grid, stream);
}

template <int LANES>
hipError_t launch(const Rotary& a, int64_t grid, hipStream_t stream) {
  // what the last-level cache cannot hold is streamed past the others (16896 tokens
  // of 48 heads of 128: 79 us against 86; 4608, which it holds: 27 against 22)
  const bool streaming = a.rows * (a.q.heads + a.k.heads) * a.dim * 4 > ((int64_t)256 << 20);
  return streaming ? launch_layout<LANES, true>(a, grid, stream) : launch_layout<LANES, false>(a, grid, stream);
}

}  // namespace

hipError_t launch_rotary(Rotary a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  // tokens a workgroup takes: two (at 16896 tokens of 48 heads of 128, 1 takes 80 us,
  // 2 79, 4 83, 8 95), more where a token's heads do not fill the workgroup four
  // times over (53396 tokens of 6 heads of 96: 41 to 45 us, filled twice 49 to 51;
  // without the norm 31, so what is above the 27 of their bytes is mostly its weights, fetched
  // again by each workgroup), as many as its table holds, and fewer while that would
  // leave compute units without a workgroup
  const int chunks = a.dim / 8, lanes = chunks <= 4 ? 4 : chunks <= 8 ? 8 : chunks <= 16 ? 16 : 32;
  const int heads = a.q.heads + a.k.heads;
  int per = 4 * (kRotThreads / lanes) / heads;
  if (per < 2) per = 2;
  if (per > kRotTokens) per = kRotTokens;
  if (per > kRotEntries / (a.rotary_dim / 2)) per = kRotEntries / (a.rotary_dim / 2);
  const int64_t fill = (a.rows + 4 * compute_units() - 1) / (4 * compute_units());
  if (per > fill) per = (int)fill;
  a.tokens_per_group = per;
  const int64_t groups = (a.rows + per - 1) / per;
  const int64_t grid = groups < (1 << 20) ? groups : (1 << 20);    // the kernel strides over the rest
  switch (lanes) {
    case 4: return launch<4>(a, grid, stream);
    case 8: return launch<8>(a, grid, stream);
    case 16: return launch<16>(a, grid, stream);
    default: return launch<32>(a, grid, stream);
  }
}

}  // namespace nvfp4
