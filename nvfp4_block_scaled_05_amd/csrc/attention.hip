// dit_cross_attention: softmax(scale q k^T) v of query heads over the keys and
// values of an encoder (or of any other length), with key heads shared by
// groups of query heads, key lengths and a key mask.
#include "device_common.hpp"
#include "kernels.hpp"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kKeys = 64;                       // keys per tile
constexpr uint32_t kNoData = 0x80000000u;       // a lane offset past every tile: loads zeros

// Where a 16-byte piece of a K / V row lies in its LDS row: pieces are permuted
// by XOR so that the fragment reads spread over all banks.  K fragments read
// one piece of 32 consecutive rows; V fragments (transposing) read 4 pieces of
// 4 consecutive rows.
template <int DP>
__device__ __forceinline__ int k_swizzle(int key) {
  return DP == 128 ? (key & 15) : ((key >> 1) & 7);
}
template <int DP>
__device__ __forceinline__ int v_swizzle(int key) {
  return DP == 128 ? ((key & 3) << 2) : (((key >> 1) & 1) << 2);
}

// 16 bytes per lane from base + offset straight into LDS; offsets from kNoData
// up are out of the resource's range and load zeros.
__device__ __forceinline__ void tile_load(const void* base, uint32_t offset, void* lds) {
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<void*>(base), (short)0, (int)kNoData, kBufferWord3);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16,
                                           offset, 0, 0, 0);
}

__device__ __forceinline__ s16x4 transposed4(const uint8_t* lds) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) s16x4*)const_cast<uint8_t*>(lds));
}

__device__ __forceinline__ bf16x8 as_bf16x8(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

// The other half-wave's value of `v` (lane ^ 32).
__device__ __forceinline__ float other_half(float v) { return __shfl_xor(v, 32, 64); }

template <int DP, int RB>
struct Attend {
  static constexpr int kSteps = DP / 16;        // MFMA steps over the head size
  static constexpr int kBlocks = DP / 32;       // 32-row blocks of the transposed output
  static constexpr int kPieces = DP / 8;        // 16-byte pieces of a row
  static constexpr int kLoads = kKeys * kPieces / 256;   // per thread and operand
  static constexpr int kRows = 4 * 32 * RB;     // query rows a workgroup takes
  static constexpr int kTileBytes = kKeys * DP * 2;

  bf16x8 q[RB][kSteps];
  f32x16 o[RB][kBlocks];
  float top[RB], sum[RB];                       // running maximum (times c) and sum, per query
  float c;                                      // scale * log2(e)
  int lane, half, col;
  uint32_t k_off[kLoads], v_off[kLoads];

  __device__ __forceinline__ void issue(const uint16_t* k, const uint16_t* v, uint64_t seen,
                                        uint8_t* lds_k, uint8_t* lds_v) const {
    const int wave = wave_id();
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = (wave * kLoads + i) * 1024;
      uint32_t ko = k_off[i], vo = v_off[i];
      if (seen != ~0ull) {                      // keys out of sight load as zeros
        const int key = (at >> 4) / kPieces + lane / kPieces;
        if (!((seen >> key) & 1)) ko = vo = kNoData;
      }
      tile_load(k, ko, lds_k + at);
      tile_load(v, vo, lds_v + at);
    }
  }

  // One tile of 64 keys, the bits of `seen` the visible ones.
  __device__ __forceinline__ void tile(const uint8_t* lds_k, const uint8_t* lds_v, uint64_t seen) {
    f32x16 s[RB][2];
#pragma unroll
    for (int r = 0; r < RB; ++r) s[r][0] = s[r][1] = f32x16{};
    // S^T = K Q^T: column = query, row = key
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      const int key = kb * 32 + col;
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        const u32x4 f = *reinterpret_cast<const u32x4*>(
            lds_k + key * (DP * 2) + (((2 * st + half) ^ k_swizzle<DP>(key)) << 4));
#pragma unroll
        for (int r = 0; r < RB; ++r)
          s[r][kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(f), q[r][st], s[r][kb], 0, 0, 0);
      }
    }
    if (seen != ~0ull) {
      const uint64_t mine = seen >> (4 * half);
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const bool on = (mine >> (32 * kb + 8 * (i / 4) + i % 4)) & 1;
#pragma unroll
          for (int r = 0; r < RB; ++r) s[r][kb][i] = on ? s[r][kb][i] : -__builtin_inff();
        }
    }
    bf16x8 p[RB][4];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      float m = s[r][0][0];
#pragma unroll
      for (int i = 1; i < 32; ++i) m = __builtin_fmaxf(m, s[r][i / 16][i % 16]);
      m = __builtin_fmaxf(m, other_half(m)) * c;
      if (__any(m > top[r] + 8.0f)) {           // sums may reach 2^8 times the true ones
        const float now = __builtin_fmaxf(top[r], m);
        const float f = __builtin_amdgcn_exp2f(top[r] - now);
        top[r] = now;
        sum[r] *= f;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[r][b][i] *= f;
      }
      float e[32];
#pragma unroll
      for (int i = 0; i < 32; ++i)
        e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r][i / 16][i % 16], c, -top[r]));
      float t = 0.0f;
#pragma unroll
      for (int i = 0; i < 32; ++i) t += e[i];
      sum[r] += t;
#pragma unroll
      for (int g = 0; g < 4; ++g)
        p[r][g] = as_bf16x8(u32x4{bf16x2_rne(e[8 * g], e[8 * g + 1]), bf16x2_rne(e[8 * g + 2], e[8 * g + 3]),
                                  bf16x2_rne(e[8 * g + 4], e[8 * g + 5]), bf16x2_rne(e[8 * g + 6], e[8 * g + 7])});
    }
    // O^T += V^T P^T.  A lane's 8 probabilities of 16-key group g are those of
    // keys 16 g + 4 half + {0..3, 8..11}; the transposing reads take V's rows
    // in the same order, so P needs no exchange between lanes.
    const int row4 = (lane & 15) >> 2, quad = lane & 3, side = (lane >> 4) & 1;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        s16x4 v[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int key = 16 * g + 8 * u + 4 * half + row4;
          const int piece = 4 * b + 2 * side + (quad >> 1);
          v[u] = transposed4(lds_v + key * (DP * 2) + ((piece ^ v_swizzle<DP>(key)) << 4) + (quad & 1) * 8);
        }
        const u32x2 lo = __builtin_bit_cast(u32x2, v[0]), hi = __builtin_bit_cast(u32x2, v[1]);
        const bf16x8 f = as_bf16x8(u32x4{lo.x, lo.y, hi.x, hi.y});
#pragma unroll
        for (int r = 0; r < RB; ++r)
          o[r][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, p[r][g], o[r][b], 0, 0, 0);
      }
    }
  }
};

template <int DP, int RB>
__global__ __launch_bounds__(256, RB == 1 ? 2 : 1) void attention_kernel(Attention a) {
  using A = Attend<DP, RB>;
  __shared__ __attribute__((aligned(1024))) uint8_t k0[A::kTileBytes], v0[A::kTileBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t k1[A::kTileBytes], v1[A::kTileBytes];
  A w;
  w.lane = threadIdx.x & 63;
  w.half = w.lane >> 5;
  w.col = w.lane & 31;
  const int wave = wave_id();
  const int64_t pos = xcd_order(blockIdx.x, gridDim.x);
  const int64_t pair = pos / a.row_tiles;                       // (batch, kv head, split)
  const int row_tile = (int)(pos - pair * a.row_tiles);
  const int64_t bh = pair / a.splits;
  const int split = (int)(pair - bh * a.splits);
  const int64_t batch = bh / a.kv_heads;
  const int kvh = (int)(bh - batch * a.kv_heads);

  int keys = a.keys;
  if (a.lengths) keys = min(max(__builtin_amdgcn_readfirstlane(a.lengths[batch]), 0), keys);
  const uint8_t* mask = a.mask ? a.mask + batch * a.mask_stride : nullptr;
  const int tiles = (keys + kKeys - 1) / kKeys, share = (tiles + a.splits - 1) / a.splits;
  const int last = min((split + 1) * share, tiles);

  // this wave's query rows: row = token * group + head within the group
  const int64_t row0 = (int64_t)row_tile * A::kRows + wave * 32 * RB + w.col;
  const int64_t rows = (int64_t)a.queries * a.group;
#pragma unroll
  for (int r = 0; r < RB; ++r) {
    int64_t row = row0 + 32 * r;
    row = row < rows ? row : rows - 1;
    const int64_t token = row / a.group, head = kvh * a.group + (row - token * a.group);
    const uint16_t* p = a.q + batch * a.q_batch + token * a.q_token + head * a.q_head;
#pragma unroll
    for (int st = 0; st < A::kSteps; ++st) {
      const int at = 16 * st + 8 * w.half;
      u32x4 f = u32x4{0u, 0u, 0u, 0u};
      if (at < a.dim) f = *reinterpret_cast<const u32x4*>(p + at);
      w.q[r][st] = as_bf16x8(f);
    }
    w.top[r] = -__builtin_inff();
    w.sum[r] = 0.0f;
#pragma unroll
    for (int b = 0; b < A::kBlocks; ++b) w.o[r][b] = f32x16{};
  }
  w.c = a.scale * 1.44269504f;
#pragma unroll
  for (int i = 0; i < A::kLoads; ++i) {
    const int at = (wave * A::kLoads + i) * 64 + w.lane;
    const int key = at / A::kPieces, piece = at % A::kPieces;
    const int kp = piece ^ k_swizzle<DP>(key), vp = piece ^ v_swizzle<DP>(key);
    w.k_off[i] = 8 * kp < a.dim ? (uint32_t)(key * a.k_token * 2 + kp * 16) : kNoData;
    w.v_off[i] = 8 * vp < a.dim ? (uint32_t)(key * a.v_token * 2 + vp * 16) : kNoData;
  }
  const uint16_t* kp = a.k + batch * a.k_batch + kvh * a.k_head;
  const uint16_t* vp = a.v + batch * a.v_batch + kvh * a.v_head;

  // the visible keys of tile t, and the next tile that has any
  auto seen_in = [&](int t) -> uint64_t {
    const int n = keys - t * kKeys;
    uint64_t s = n >= kKeys ? ~0ull : (1ull << n) - 1;
    if (mask) s &= __ballot(w.lane < n && mask[(int64_t)t * kKeys + w.lane] != 0);
    return s;
  };
  auto next = [&](int t, uint64_t& seen) {
    for (++t; t < last; ++t)
      if ((seen = seen_in(t)) != 0) break;
    return t;
  };
  uint64_t seen = 0, seen_next = 0;
  int t = next(split * share - 1, seen);
  if (t < last)
    w.issue(kp + (int64_t)t * kKeys * a.k_token, vp + (int64_t)t * kKeys * a.v_token, seen, k0, v0);
  // every wave of the workgroup sees the same lengths and mask, so all take
  // the same turns and meet at every barrier
#define ATTEND_TURN(kc, vc, kn, vn)                                                              \
  {                                                                                              \
    const int tn = next(t, seen_next);                                                           \
    __builtin_amdgcn_s_waitcnt(0x0070); /* vmcnt(0) lgkmcnt(0): own loads in LDS, reads done */   \
    asm volatile("s_barrier" ::: "memory"); /* everyone's is, and the other buffers are free */ \
    if (tn < last)                                                                               \
      w.issue(kp + (int64_t)tn * kKeys * a.k_token, vp + (int64_t)tn * kKeys * a.v_token,        \
              seen_next, kn, vn);                                                                \
    w.tile(kc, vc, seen);                                                                        \
    t = tn;                                                                                      \
    seen = seen_next;                                                                            \
  }
  while (t < last) {
    ATTEND_TURN(k0, v0, k1, v1)
    if (t >= last) break;
    ATTEND_TURN(k1, v1, k0, v0)
  }
#undef ATTEND_TURN

#pragma unroll
  for (int r = 0; r < RB; ++r) {
    const int64_t row = row0 + 32 * r;
    const float l = w.sum[r] + other_half(w.sum[r]);
    if (a.splits > 1) {      // unnormalised partial sums, the maximum and the sum
      if (row >= rows) continue;
      const int64_t slot = pair * rows + row;
      float* out = a.part + slot * DP;
#pragma unroll
      for (int b = 0; b < A::kBlocks; ++b)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<f32x4*>(out + 32 * b + 8 * g + 4 * w.half) =
              f32x4{w.o[r][b][4 * g], w.o[r][b][4 * g + 1], w.o[r][b][4 * g + 2], w.o[r][b][4 * g + 3]};
      if (w.half == 0) a.stats[slot] = float2{w.top[r], l};
      continue;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;   // no key seen: zeros
    const int64_t token = (row < rows ? row : 0) / a.group;
    const int64_t head = kvh * a.group + (row < rows ? row - token * a.group : 0);
    uint16_t* out = a.out + batch * a.o_batch + token * a.o_token + head * a.o_head;
#pragma unroll
    for (int b = 0; b < A::kBlocks; ++b)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int at = 32 * b + 8 * g + 4 * w.half;
        const u32x2 v = u32x2{bf16x2_rne(w.o[r][b][4 * g] * inv, w.o[r][b][4 * g + 1] * inv),
                              bf16x2_rne(w.o[r][b][4 * g + 2] * inv, w.o[r][b][4 * g + 3] * inv)};
        if (row < rows && at < a.dim) *reinterpret_cast<u32x2*>(out + at) = v;
      }
  }
}

// Joins the splits of a row, one wave per row: partial sums weighted by
// 2^(their maximum - the largest), in split order.
template <int DP>
__global__ __launch_bounds__(256) void attention_join_kernel(Attention a) {
  const int lane = threadIdx.x & 63;
  const int64_t rows = (int64_t)a.queries * a.group;
  const int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);      // (batch, kv head, row)
  if (at >= (int64_t)a.batch * a.kv_heads * rows) return;
  const int64_t bh = at / rows, row = at - bh * rows;
  float top = -__builtin_inff();
  for (int s = 0; s < a.splits; ++s) {
    const float2 st = a.stats[(bh * a.splits + s) * rows + row];
    if (st.y != 0.0f) top = __builtin_fmaxf(top, st.x);
  }
  float l = 0.0f, o[DP / 64] = {};
  for (int s = 0; s < a.splits; ++s) {
    const int64_t slot = (bh * a.splits + s) * rows + row;
    const float2 st = a.stats[slot];
    if (st.y == 0.0f) continue;                  // this split saw no key
    const float f = __builtin_amdgcn_exp2f(st.x - top);
    l = __builtin_fmaf(st.y, f, l);
#pragma unroll
    for (int j = 0; j < DP / 64; ++j)
      o[j] = __builtin_fmaf(a.part[slot * DP + lane * (DP / 64) + j], f, o[j]);
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int64_t batch = bh / a.kv_heads, token = row / a.group;
  const int64_t head = (bh - batch * a.kv_heads) * a.group + (row - token * a.group);
  uint16_t* out = a.out + batch * a.o_batch + token * a.o_token + head * a.o_head;
  if (DP == 128) {
    if (2 * lane < a.dim)
      *reinterpret_cast<uint32_t*>(out + 2 * lane) = bf16x2_rne(o[0] * inv, o[DP / 64 - 1] * inv);
  } else if (lane < a.dim) {
    out[lane] = (uint16_t)bf16x2_rne(o[0] * inv, 0.0f);
  }
}

template <int DP, int RB>
hipError_t launch(Attention a, hipStream_t stream) {
  const int64_t rows = (int64_t)a.queries * a.group;
  a.row_tiles = (rows + Attend<DP, RB>::kRows - 1) / Attend<DP, RB>::kRows;
  const int64_t grid = (int64_t)a.batch * a.kv_heads * a.splits * a.row_tiles;
  attention_kernel<DP, RB><<<dim3((unsigned)grid), dim3(256), 0, stream>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t all = (int64_t)a.batch * a.kv_heads * rows;
  attention_join_kernel<DP><<<dim3((unsigned)((all + 3) / 4)), dim3(256), 0, stream>>>(a);
  return hipGetLastError();
}

// Ways the keys are split: as many as give every compute unit two workgroups,
// each split keeping at least four tiles.
int splits_for(int64_t batch, int64_t kv_heads, int64_t rows, int64_t keys) {
  const int64_t groups = batch * kv_heads * ((rows + 127) / 128);
  const int64_t tiles = (keys + kKeys - 1) / kKeys;
  int64_t s = 2 * compute_units() / (groups > 0 ? groups : 1);
  if (s > tiles / 4) s = tiles / 4;
  return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}

int padded_dim(int64_t dim) { return dim <= 64 ? 64 : 128; }

}  // namespace

size_t attention_workspace_bytes(int64_t batch, int64_t queries, int64_t keys, int64_t heads,
                                 int64_t kv_heads, int64_t dim) {
  if (batch == 0 || queries == 0) return 0;
  const int64_t rows = queries * (heads / kv_heads);
  const int splits = splits_for(batch, kv_heads, rows, keys);
  if (splits == 1) return 0;
  return (size_t)(batch * kv_heads * splits * rows) * (padded_dim(dim) * 4 + 8);
}

hipError_t launch_attention(Attention a, void* workspace, size_t workspace_bytes,
                            hipStream_t stream) {
  const int64_t rows = (int64_t)a.queries * a.group;
  a.splits = splits_for(a.batch, a.kv_heads, rows, a.keys);
  const size_t need = attention_workspace_bytes(a.batch, a.queries, a.keys,
                                                (int64_t)a.kv_heads * a.group, a.kv_heads, a.dim);
  if (!workspace || workspace_bytes < need) a.splits = 1;
  if (a.splits > 1) {
    a.part = static_cast<float*>(workspace);
    a.stats = reinterpret_cast<float2*>(a.part + (int64_t)a.batch * a.kv_heads * a.splits * rows *
                                                    padded_dim(a.dim));
  }
  return padded_dim(a.dim) == 64 ? launch<64, 1>(a, stream) : launch<128, 1>(a, stream);
}

}  // namespace nvfp4
