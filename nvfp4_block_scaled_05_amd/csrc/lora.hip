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
// Rows of one request lie together, but any order is right: each distinct adapter
// of a tile of 16 rows goes through the whole tile, and each row keeps the result
// of its own (a select, so what another adapter holds cannot reach it).
//
// Measured at 4608 rows, 3072 to 9216, rank 32, five requests: 16 us and 42 to 46 us,
// the second at 3.7 to 4.0 TB/s of y and out; at 48 rows of 12 requests, 3072 to 12288, rank
// 16, with GELU and amax: 4.2 us and 8.6 us, bound by the latency of their chains
// of loads (ids, adapter, product).
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

// Depth of one group of steps of a wave of the first kernel, all loaded at once
// (9 to 24 16-byte loads a lane), and the most waves of its workgroup.
constexpr int group_steps(int rt, int mt) { return rt * mt <= 2 ? 8 : rt * mt <= 4 ? 4 : 1; }
constexpr int kDownWaves = 12;

// t[slice][row][16 * RT]: this slice's part of s_a * down_a x.  RT: 16-wide
// tiles over the rank, MT: row tiles of the workgroup.  It has as many waves (up
// to 12) as the slice has groups of steps, so that few rounds of loads take it
// through the slice; their sums are added in wave order.  With gridDim.z > 1
// workgroup z has the z-th distinct adapter of its tile, and that one's rows, alone.
template <int RT, int MT>
__global__ __launch_bounds__(64 * kDownWaves) void lora_down_kernel(Lora a) {
  constexpr int U = group_steps(RT, MT);
  __shared__ float red[kDownWaves][MT * RT * 4][64];
  const int waves = blockDim.x >> 6;
  if (a.amax && blockIdx.x + blockIdx.y + blockIdx.z == 0 && threadIdx.x == 0) *a.amax = 0u;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int r = lane & 15, q = lane >> 4;
  const int64_t row0 = (int64_t)blockIdx.x * (kRowTile * MT);
  const int id = row_adapter(a, row0 + lane % (kRowTile * MT));      // rows past the last: none
  const int k_end = min(a.inner, (int)(blockIdx.y + 1) * a.slice);
  const uint16_t* x[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) x[m] = a.x + min(row0 + 16 * m + r, a.rows - 1) * a.inner + 8 * q;
  // element e of a lane: row tile e / (4 RT), column 16 (e / 4 % RT) + lane % 16,
  // row 4 (lane / 16) + e % 4; rows without an adapter stay zero
#pragma unroll
  for (int e = 0; e < MT * RT * 4; ++e) red[wave][e][lane] = 0.0f;
  const bool one = gridDim.z > 1;
  uint32_t skip = blockIdx.z;
  uint64_t todo = __ballot(lane < kRowTile * MT && id >= 0), mine = ~0ull;
  while (todo) {
    const int cur = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
    const uint64_t same = __ballot(lane < kRowTile * MT && id == cur);
    todo &= ~same;
    if (one) {
      if (skip > 0) {
        --skip;
        continue;
      }
      todo = 0;
      mine = same;
    }
    f32x4 acc[MT][RT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int c = 0; c < RT; ++c) acc[m][c] = f32x4{};
    const uint16_t* down = a.down + (int64_t)cur * a.rank * a.inner + 8 * q;
    // columns past the rank read its last row; no one reads what they compute
    const uint16_t* col[RT];
#pragma unroll
    for (int c = 0; c < RT; ++c) col[c] = down + (int64_t)min(16 * c + r, a.rank - 1) * a.inner;
    int k = blockIdx.y * a.slice + wave * 32 * U;
    for (; k + 32 * U <= k_end; k += waves * 32 * U) {
      u32x4 xa[U][MT], wb[U][RT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int m = 0; m < MT; ++m) xa[u][m] = *reinterpret_cast<const u32x4*>(x[m] + k + 32 * u);
#pragma unroll
        for (int c = 0; c < RT; ++c) wb[u][c] = *reinterpret_cast<const u32x4*>(col[c] + k + 32 * u);
      }
      __builtin_amdgcn_sched_barrier(0);       // every load of the group before its first product
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int c = 0; c < RT; ++c)
            acc[m][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(xa[u][m]), frag(wb[u][c]), acc[m][c], 0, 0, 0);
    }
    for (int end = min(k + 32 * U, k_end); k < end; k += 32) {     // the last, shorter group
      const bool in = k + 8 * q < k_end;
#pragma unroll
      for (int c = 0; c < RT; ++c) {
        const u32x4 wb = load16(col[c] + k, in);
#pragma unroll
        for (int m = 0; m < MT; ++m)
          acc[m][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(load16(x[m] + k, in)), frag(wb), acc[m][c], 0, 0, 0);
      }
    }
    const float s = a.scales ? a.scales[cur] : 1.0f;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int c = 0; c < RT; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((same >> (16 * m + 4 * q + i)) & 1) red[wave][(m * RT + c) * 4 + i][lane] = acc[m][c][i] * s;
  }
  if (one && mine == ~0ull) return;              // the tile has fewer adapters
  __syncthreads();
  for (int e = wave; e < MT * RT * 4; e += waves) {
    float v = red[0][e][lane];
    for (int w = 1; w < waves; ++w) v += red[w][e][lane];
    const int in = 16 * (e / (4 * RT)) + 4 * q + e % 4;
    const int64_t to = row0 + in;
    if (to < a.rows && ((mine >> in) & 1))
      a.t[((int64_t)blockIdx.y * a.rows + to) * (16 * RT) + 16 * (e / 4 % RT) + r] = v;
  }
}

// out = epi(y + up_a t).  A wave takes MT row tiles and 128 columns at a time, the
// column blocks of the rows side by side, so y and out are read and written in
// long pieces (with a workgroup's waves on four row tiles of one column block
// instead, sharing the adapter's weights in the cache: 5 % slower).  An access is
// of 16 rows' 64 bytes, halves of cache lines that meet in the cache: streamed past
// it, 4608 x 9216 take 50 us, not 46, and 16896 x 9216 166, not 139.  The
// weight is the MFMA's first operand, so a lane holds columns of one row; the
// weight rows of a pair of MFMA tiles are dealt so that the 4 + 4 columns a lane
// gets are 8 neighbours (16 bytes of y and out).
template <int RT, int MT>
__global__ __launch_bounds__(kLoraThreads) void lora_up_kernel(Lora a) {
  constexpr int KS = (RT + 1) / 2;             // 32-deep steps over the rank
  // column blocks that a tile of several adapters loads weights for at once: all of
  // them where rows are few (8.5 us against 10.3 at 48 rows), one where the registers
  // cost waves (46 us against 49 at 4608 rows, 139 against 152 at 16896).  Many rows of
  // rank 33 to 64, which run one row tile, pay for it: 82 us against 75 at 4608.
  constexpr int NB = MT > 1 ? 1 : KS <= 2 ? kColBlocks : kColBlocks / KS;
  const int lane = threadIdx.x & 63;
  const int r = lane & 15, q = lane >> 4;
  const int col_items = (a.outer + kColBlock * kColBlocks - 1) / (kColBlock * kColBlocks);
  const int64_t items = (a.rows + kRowTile * MT - 1) / (kRowTile * MT) * col_items;
  u16x2 top = {0, 0};
  for (int64_t item = (int64_t)blockIdx.x * 4 + wave_id(); item < items; item += (int64_t)gridDim.x * 4) {
    const int64_t row_item = items < (1ll << 31) ? (int64_t)((uint32_t)item / (uint32_t)col_items) : item / col_items;
    const int64_t row0 = row_item * (kRowTile * MT) + r;
    const int col0 = (int)(item - row_item * col_items) * kColBlock * kColBlocks;
    int id[MT], first = -1;
    uint64_t any = 0;
    bool uniform = true;                       // one adapter at most
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      id[m] = row_adapter(a, row0 + 16 * m);
      const uint64_t has = __ballot(lane < 16 && id[m] >= 0);
      if (has && first < 0) first = __builtin_amdgcn_readlane(id[m], __builtin_ctzll(has));
      uniform &= has == __ballot(lane < 16 && id[m] >= 0 && id[m] == first);
      any |= has;
    }
    if (!any && a.skip_idle) continue;         // in place, nothing to add
    // rows and columns past the last read the last row's, the first column's;
    // what they compute is not stored
    u32x4 yv[MT][kColBlocks];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int b = 0; b < kColBlocks; ++b) {
        const int col = col0 + kColBlock * b + 8 * q;
        yv[m][b] = *reinterpret_cast<const u32x4*>(a.y + min(row0 + 16 * m, a.rows - 1) * a.outer +
                                                   (col < a.outer ? col : 0));
      }
    bf16x8 tf[MT][KS];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        f32x4 lo = f32x4{}, hi = f32x4{};
        if (id[m] >= 0 && 32 * s + 8 * q < a.rank)
          for (int sl = 0; sl < a.slices; ++sl) {
            const float* p = a.t + (sl * a.rows + row0 + 16 * m) * (16 * RT) + 32 * s + 8 * q;
            lo += reinterpret_cast<const f32x4*>(p)[0];
            hi += reinterpret_cast<const f32x4*>(p)[1];
          }
        // rounded to bf16 for the product with up: a relative 2^-8 of each of
        // the adapter's `rank` terms
        tf[m][s] = frag(u32x4{bf16x2_rne(lo[0], lo[1]), bf16x2_rne(lo[2], lo[3]), bf16x2_rne(hi[0], hi[1]),
                              bf16x2_rne(hi[2], hi[3])});
      }
    // columns past the last read it; depth past the rank is zeros
    auto weights = [&](int of, int b, int p, int s) {
      const int n = min(col0 + kColBlock * b + 8 * (r >> 2) + 4 * p + (r & 3), a.outer - 1);
      const int j = 32 * s + 8 * q;
      const u32x4 f = *reinterpret_cast<const u32x4*>(a.up + ((int64_t)of * a.outer + n) * a.rank +
                                                      (j < a.rank ? j : 0));
      return j < a.rank ? f : u32x4{0u, 0u, 0u, 0u};
    };
    auto finish = [&](int m, int b, const f32x4 (&d)[2]) {
      const int64_t row = row0 + 16 * m;
      const int col = col0 + kColBlock * b + 8 * q;
      const uint32_t w[4] = {yv[m][b].x, yv[m][b].y, yv[m][b].z, yv[m][b].w};
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16) + d[j / 2][2 * (j & 1)];
        f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u) + d[j / 2][2 * (j & 1) + 1];
      }
      if (a.epilogue == NVFP4_EPI_GELU) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = gelu_erf(f[j]);
      }
      const u32x4 v = u32x4{bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]), bf16x2_rne(f[4], f[5]),
                            bf16x2_rne(f[6], f[7])};
      if (row < a.rows && col < a.outer) {
        *reinterpret_cast<u32x4*>(a.out + row * a.outer + col) = v;
        top = max_u16x2(top, max8(v));
      }
    };
    if (uniform) {                             // its weights all at once
      u32x4 uf[KS][kColBlocks][2];
      if (first >= 0) {
#pragma unroll
        for (int b = 0; b < kColBlocks; ++b)
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int s = 0; s < KS; ++s) uf[s][b][p] = weights(first, b, p, s);
      }
#pragma unroll
      for (int b = 0; b < kColBlocks; ++b)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          f32x4 d[2] = {f32x4{}, f32x4{}};
          if (first >= 0) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
#pragma unroll
              for (int s = 0; s < KS; ++s)
                d[p] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(uf[s][b][p]), tf[m][s], d[p], 0, 0, 0);
              if (id[m] < 0) d[p] = f32x4{};   // a row of none beside it
            }
          }
          finish(m, b, d);
        }
    } else {                                   // one adapter after another through the tile
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int b0 = 0; b0 < kColBlocks; b0 += NB) {
          f32x4 d[NB][2];
#pragma unroll
          for (int b = 0; b < NB; ++b) d[b][0] = d[b][1] = f32x4{};
          for (uint64_t left = __ballot(lane < 16 && id[m] >= 0); left;) {
            const int cur = __builtin_amdgcn_readlane(id[m], __builtin_ctzll(left));
            left &= ~__ballot(lane < 16 && id[m] == cur);
            u32x4 uf[KS][NB][2];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
              for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int s = 0; s < KS; ++s) uf[s][b][p] = weights(cur, b0 + b, p, s);
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
              for (int p = 0; p < 2; ++p) {
                f32x4 acc = f32x4{};
#pragma unroll
                for (int s = 0; s < KS; ++s)
                  acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(uf[s][b][p]), tf[m][s], acc, 0, 0, 0);
                if (id[m] == cur) d[b][p] = acc;
              }
          }
#pragma unroll
          for (int b = 0; b < NB; ++b) finish(m, b0 + b, d[b]);
        }
    }
  }
  if (a.amax) {
    __shared__ uint32_t wave_top[kLoraThreads / 64];
    const uint32_t m = wave_max_u32((uint32_t)(top.x > top.y ? top.x : top.y) << 16);
    if (lane == 0) wave_top[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x == 0)
      raise_amax(a.amax, max(max(wave_top[0], wave_top[1]), max(wave_top[2], wave_top[3])));
  }
}

__global__ void zero_lora_amax_kernel(uint32_t* p) { *p = 0u; }

// Ranks are padded to one of these many 16-wide tiles; above two, both kernels run one
// row tile at a time, so the adapters' weights come from the caches twice as often (4608
// x 9216: rank 32 62 us, 40 88, 64 116, 128 180).
int rank_tiles(int64_t rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8; }

// Slices of `inner` in the first kernel, while the row tiles alone leave compute
// units without work: at most 8, each at least 512 deep (the second kernel adds
// them up, for every column block again).
int slices_for(int64_t rows, int64_t inner) {
  const int64_t tiles = (rows + kRowTile - 1) / kRowTile;
  int64_t s = compute_units() / (tiles > 0 ? tiles : 1);
  if (s > inner / 512) s = inner / 512;
  return (int)(s < 1 ? 1 : s > 8 ? 8 : s);
}

template <int RT>
hipError_t launch(const Lora& a, hipStream_t stream) {
  const int64_t tiles = (a.rows + kRowTile - 1) / kRowTile;
  // a workgroup of 12 waves fills a compute unit: two row tiles each (every weight
  // fragment then serves both) where that saves rounds over the compute units: at
  // 4608 rows of 3072, rank 32, 144 workgroups take 16 us, 288 take 22
  const int64_t units = compute_units();
  const int64_t one = (tiles + units - 1) / units, two = ((tiles + 1) / 2 + units - 1) / units;
  const int mt = RT <= 2 && 4 * two < 3 * one ? 2 : 1;
  const int groups = (a.slice + 32 * group_steps(RT, mt) - 1) / (32 * group_steps(RT, mt));
  const dim3 block(64 * (groups < kDownWaves ? groups : kDownWaves));
  // Few tiles: a workgroup for each adapter that a tile can have, those past its
  // number leaving at once, so that no tile takes two one after another (16 us
  // against 26 where 4 of 144 tiles have two adapters, 4.0 against 8.5 where 3
  // tiles of 48 rows have four each).  Many: the tail of one such tile is small
  // beside the rounds.
  int64_t each = a.adapters < kRowTile * mt ? a.adapters : kRowTile * mt;
  if ((tiles + mt - 1) / mt * a.slices * each > 4 * units) each = 1;
  const dim3 down((unsigned)((tiles + mt - 1) / mt), a.slices, (unsigned)each);
  if (mt == 2)
    lora_down_kernel<RT, RT <= 2 ? 2 : 1><<<down, block, 0, stream>>>(a);
  else
    lora_down_kernel<RT, 1><<<down, block, 0, stream>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // two row tiles a wave (the adapter's weights then serve both: 46 us against 48
  // at 4608 x 9216, rank 32, 139 against 161 at 16896 rows) where that still leaves every compute unit 16 waves
  const int64_t cols = (a.outer + kColBlock * kColBlocks - 1) / (kColBlock * kColBlocks);
  const int64_t cap = units * 64;
  const int up = RT <= 2 && tiles * cols >= 32 * units ? 2 : 1;
  const int64_t waves = (tiles + up - 1) / up * cols;
  const int64_t grid = (waves + 3) / 4 < cap ? (waves + 3) / 4 : cap;
  if (up == 2)
    lora_up_kernel<RT, RT <= 2 ? 2 : 1><<<dim3((unsigned)grid), dim3(kLoraThreads), 0, stream>>>(a);
  else
    lora_up_kernel<RT, 1><<<dim3((unsigned)grid), dim3(kLoraThreads), 0, stream>>>(a);
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
