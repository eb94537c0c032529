// dit_lora_add: low-rank adapters of many requests beside a shared projection.
//
//   out[m] = epi( y[m] + s_a * up_a (down_a x[m]) ),  a = ids[m]
//
// Two kernels.  The first computes t = s_a * down_a x per row (a product of
// depth `inner` with 8..128 columns), the second up_a t and the sum, the
// epilogue and the amax.  Between them t, rank fp32 values a row, is in the
// workspace.  Bound: HBM -- x is read once by the first, y read and out written
// once by the second; the adapters come from the caches.
//
// Rows of one request lie together, but any order is right: a tile of 16 rows
// takes its distinct adapters one after another through the whole tile, and
// each row keeps the result of its own (a select, so what another adapter holds
// cannot reach it).
#include "device_common.hpp"
#include "kernels.hpp"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kLoraThreads = 256;
constexpr int kRowTile = 16;
constexpr int kColBlock = 32;                // output columns per pair of MFMA tiles
constexpr int kColBlocks = 4;                // pairs a wave takes: 128 columns

__device__ __forceinline__ bf16x8 frag(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }
__device__ __forceinline__ u32x4 load16(const uint16_t* p, bool live) {
  return live ? *reinterpret_cast<const u32x4*>(p) : u32x4{0u, 0u, 0u, 0u};
}

// The adapter of this lane's row (lane % 16 of the tile): -1 for none.
__device__ __forceinline__ int row_adapter(const Lora& a, int64_t row) {
  if (row >= a.rows) return -1;
  const int id = a.ids[row];
  return id >= 0 && id < a.adapters ? id : -1;
}

// t[slice][row][16 * RT]: this slice's part of s_a * down_a x.  RT: 16-wide
// tiles over the rank; the four waves take every fourth group of U 32-deep
// steps of the slice and add their sums in wave order.
template <int RT>
__global__ __launch_bounds__(kLoraThreads) void lora_down_kernel(Lora a) {
  constexpr int U = RT <= 2 ? 8 : (RT <= 4 ? 4 : 2);
  __shared__ float red[4][RT * 4][64];
  if (a.amax && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.amax = 0u;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int r = lane & 15, q = lane >> 4;
  const int64_t row0 = (int64_t)blockIdx.x * kRowTile;
  const int64_t row = row0 + r < a.rows ? row0 + r : a.rows - 1;
  const int id = row_adapter(a, row0 + r);
  const int k_end = min(a.inner, (int)(blockIdx.y + 1) * a.slice);
  const uint16_t* x = a.x + row * a.inner + 8 * q;
  float t[RT][4] = {};
  uint64_t todo = __ballot(lane < 16 && id >= 0);
  while (todo) {
    const int cur = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    const uint32_t same = (uint32_t)__ballot(lane < 16 && id == cur);
    todo &= ~(uint64_t)same;
    f32x4 acc[RT];
#pragma unroll
    for (int c = 0; c < RT; ++c) acc[c] = f32x4{};
    const uint16_t* down = a.down + (int64_t)cur * a.rank * a.inner + 8 * q;
    for (int k = blockIdx.y * a.slice + wave * 32 * U; k < k_end; k += 4 * 32 * U) {
      u32x4 xa[U], wb[U][RT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = k + 32 * u;
        const bool in = at + 8 * q < k_end;
        xa[u] = load16(x + at, in);
#pragma unroll
        for (int c = 0; c < RT; ++c)
          wb[u][c] = load16(down + (int64_t)(16 * c + r) * a.inner + at, in && 16 * c + r < a.rank);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int c = 0; c < RT; ++c)
          acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(xa[u]), frag(wb[u][c]), acc[c], 0, 0, 0);
    }
    const float s = a.scales ? a.scales[cur] : 1.0f;
#pragma unroll
    for (int c = 0; c < RT; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if ((same >> (4 * q + i)) & 1) t[c][i] = acc[c][i] * s;
  }
#pragma unroll
  for (int c = 0; c < RT; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][c * 4 + i][lane] = t[c][i];
  __syncthreads();
  // element e of a lane: column 16 (e / 4) + lane % 16, row 4 (lane / 16) + e % 4
  for (int e = wave; e < RT * 4; e += 4) {
    const float v = ((red[0][e][lane] + red[1][e][lane]) + red[2][e][lane]) + red[3][e][lane];
    const int64_t to = row0 + 4 * q + e % 4;
    if (to < a.rows) a.t[((int64_t)blockIdx.y * a.rows + to) * (16 * RT) + 16 * (e / 4) + r] = v;
  }
}

// out = epi(y + up_a t).  A wave takes 16 rows and 128 columns at a time.  The
// weight is the MFMA's first operand, so a lane holds columns of one row; the
// weight rows of a pair of tiles are dealt so that the 4 + 4 columns a lane
// gets are 8 neighbours (16 bytes of y and out).
template <int RT>
__global__ __launch_bounds__(kLoraThreads) void lora_up_kernel(Lora a) {
  constexpr int KS = (RT + 1) / 2;             // 32-deep steps over the rank
  const int lane = threadIdx.x & 63;
  const int r = lane & 15, q = lane >> 4;
  const int64_t row_tiles = (a.rows + kRowTile - 1) / kRowTile;
  const int64_t items = row_tiles * ((a.outer + kColBlock * kColBlocks - 1) / (kColBlock * kColBlocks));
  u16x2 top = {0, 0};
  for (int64_t item = (int64_t)blockIdx.x * 4 + wave_id(); item < items; item += (int64_t)gridDim.x * 4) {
    const int64_t col_item = item / row_tiles;
    const int64_t row = (item - col_item * row_tiles) * kRowTile + r;
    const int col0 = (int)col_item * kColBlock * kColBlocks;
    const bool live = row < a.rows;
    const int id = row_adapter(a, row);
    uint64_t todo = __ballot(lane < 16 && id >= 0);
    if (!todo && a.skip_idle) continue;        // in place, nothing to add
    u32x4 yv[kColBlocks];
#pragma unroll
    for (int b = 0; b < kColBlocks; ++b) {
      const int col = col0 + kColBlock * b + 8 * q;
      yv[b] = load16(a.y + row * a.outer + col, live && col < a.outer);
    }
    bf16x8 tf[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      f32x4 lo = f32x4{}, hi = f32x4{};
      if (live && id >= 0 && 32 * s + 8 * q < a.rank)
        for (int sl = 0; sl < a.slices; ++sl) {
          const float* p = a.t + (sl * a.rows + row) * (16 * RT) + 32 * s + 8 * q;
          lo += reinterpret_cast<const f32x4*>(p)[0];
          hi += reinterpret_cast<const f32x4*>(p)[1];
        }
      // rounded to bf16 for the product with up: a relative 2^-8 of each of
      // the adapter's `rank` terms
      tf[s] = frag(u32x4{bf16x2_rne(lo[0], lo[1]), bf16x2_rne(lo[2], lo[3]), bf16x2_rne(hi[0], hi[1]),
                         bf16x2_rne(hi[2], hi[3])});
    }
    f32x4 d[kColBlocks][2];
#pragma unroll
    for (int b = 0; b < kColBlocks; ++b) d[b][0] = d[b][1] = f32x4{};
    while (todo) {
      const int cur = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
      todo &= ~__ballot(lane < 16 && id == cur);
      const uint16_t* up = a.up + (int64_t)cur * a.outer * a.rank;
#pragma unroll
      for (int b = 0; b < kColBlocks; ++b)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int n = col0 + kColBlock * b + 8 * (r >> 2) + 4 * p + (r & 3);
          f32x4 acc = f32x4{};
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            const u32x4 f = load16(up + (int64_t)n * a.rank + 32 * s + 8 * q,
                                   n < a.outer && 32 * s + 8 * q < a.rank);
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(f), tf[s], acc, 0, 0, 0);
          }
          if (id == cur) d[b][p] = acc;
        }
    }
#pragma unroll
    for (int b = 0; b < kColBlocks; ++b) {
      const int col = col0 + kColBlock * b + 8 * q;
      const uint32_t w[4] = {yv[b].x, yv[b].y, yv[b].z, yv[b].w};
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16) + d[b][j / 2][2 * (j & 1)];
        f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u) + d[b][j / 2][2 * (j & 1) + 1];
      }
      if (a.epilogue == NVFP4_EPI_GELU) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = gelu_erf(f[j]);
      }
      const u32x4 v = u32x4{bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]), bf16x2_rne(f[4], f[5]),
                            bf16x2_rne(f[6], f[7])};
      if (live && col < a.outer) {
        *reinterpret_cast<u32x4*>(a.out + row * a.outer + col) = v;
        top = max_u16x2(top, max8(v));
      }
    }
  }
  if (a.amax) {
    __shared__ uint32_t wave_top[kLoraThreads / 64];
    const uint32_t m = wave_max_u32((uint32_t)(top.x > top.y ? top.x : top.y) << 16);
    if (lane == 0) wave_top[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x == 0)
      atomicMax(a.amax, max(max(wave_top[0], wave_top[1]), max(wave_top[2], wave_top[3])));
  }
}

__global__ void zero_lora_amax_kernel(uint32_t* p) { *p = 0u; }

// Slices of `inner` in the first kernel: enough that the row tiles fill the
// compute units twice, each at least 512 deep (one group of steps per wave).
int slices_for(int64_t rows, int64_t inner) {
  const int64_t tiles = (rows + kRowTile - 1) / kRowTile;
  int64_t s = 2 * compute_units() / (tiles > 0 ? tiles : 1);
  if (s > inner / 512) s = inner / 512;
  return (int)(s < 1 ? 1 : s > 16 ? 16 : s);
}

int rank_tiles(int64_t rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8; }

template <int RT>
hipError_t launch(const Lora& a, hipStream_t stream) {
  const int64_t tiles = (a.rows + kRowTile - 1) / kRowTile;
  lora_down_kernel<RT><<<dim3((unsigned)tiles, a.slices), dim3(kLoraThreads), 0, stream>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t waves = tiles * ((a.outer + kColBlock * kColBlocks - 1) / (kColBlock * kColBlocks));
  const int64_t cap = (int64_t)compute_units() * 8;
  const int64_t grid = (waves + 3) / 4 < cap ? (waves + 3) / 4 : cap;
  lora_up_kernel<RT><<<dim3((unsigned)grid), dim3(kLoraThreads), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t lora_workspace_bytes(int64_t rows, int64_t inner, int64_t rank) {
  return (size_t)slices_for(rows, inner) * rows * 16 * rank_tiles(rank) * sizeof(float);
}

hipError_t launch_lora(Lora a, void* workspace, hipStream_t stream) {
  if (a.rows == 0 || a.outer == 0) {
    if (!a.amax) return hipSuccess;
    zero_lora_amax_kernel<<<1, 1, 0, stream>>>(a.amax);
    return hipGetLastError();
  }
  a.t = static_cast<float*>(workspace);
  a.slices = slices_for(a.rows, a.inner);
  a.slice = (((a.inner + a.slices - 1) / a.slices) + 31) / 32 * 32;
  a.skip_idle = a.out == a.y && a.epilogue == NVFP4_EPI_NONE && !a.amax;
  switch (rank_tiles(a.rank)) {
    case 1: return launch<1>(a, stream);
    case 2: return launch<2>(a, stream);
    case 4: return launch<4>(a, stream);
    default: return launch<8>(a, stream);
  }
}

}  // namespace nvfp4
