// The state of a wave in attention over tiles of keys in LDS, shared by the kernels
// over bf16 keys and over a cache in 4 bits: scores, running softmax and the product
// with the values for 32 query rows.  HALF: the operands are fp16 (what a 4-bit
// value times its block scale is exactly), else bf16.
#pragma once

#include <type_traits>

#include "device_common.hpp"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float kLowest = 3.40282347e38f;       // the largest finite binary32 value

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

__device__ __forceinline__ s16x4 transposed4(const uint8_t* lds, int at) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) s16x4*)const_cast<uint8_t*>(lds + at));
}

__device__ __forceinline__ bf16x8 as_bf16x8(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

// The product of two 16-bit fragments, and two binary32 values as a pair of its type.
template <bool HALF>
__device__ __forceinline__ f32x16 product32(u32x4 a, bf16x8 b, f32x16 c) {
  if constexpr (HALF)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(a), b, c, 0, 0, 0);
}
template <bool HALF>
__device__ __forceinline__ uint32_t pair_rne(float lo, float hi) {
  if constexpr (HALF) {
    typedef float pair_f32 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(pair_f32{lo, hi}, f16x2));
  } else {
    return bf16x2_rne(lo, hi);
  }
}

// This lane's value with the one of lane ^ 32 (permlane32_swap of v with itself
// leaves the lower half's values in the first result, the upper's in the second).
__device__ __forceinline__ float halves_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __builtin_fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float halves_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// The running state of a wave's 32 query rows over tiles of 32 * KB keys.
template <int DP, int KB, bool HALF = false>
struct Attend {
  static constexpr int kSteps = DP / 16;        // MFMA steps over the head size
  static constexpr int kBlocks = DP / 32;       // 32-row blocks of the transposed output
  static constexpr int kPieces = DP / 8;        // 16-byte pieces of a row
  static constexpr int kKeys = 32 * KB;
  static constexpr int kRowBytes = DP * 2;
  static constexpr int kTileBytes = kKeys * kRowBytes;
  static constexpr uint64_t kAll = KB == 2 ? ~0ull : 0xFFFFFFFFull;   // every key of a tile seen

  // fp16 has the range for probabilities up to 2^15: the maximum is held 2^7 low, so
  // that together with the growth that is let pass (below) they use it, and those
  // down to 2^-21 of the largest keep all their bits
  static constexpr float kLift = HALF ? 7.0f : 0.0f;

  bf16x8 q[kSteps];                             // fragments, of either type
  f32x16 o[kBlocks];
  float top, sum;                               // running maximum (times c) and sum, per query
  float c;                                      // scale * log2(e)
  int lane, half, col;

  __device__ __forceinline__ void start(float scale) {
    lane = threadIdx.x & 63;
    half = lane >> 5;
    col = lane & 31;
    c = scale * 1.44269504f;
    top = -kLowest;                             // finite: a score of -inf then weighs 0
    sum = 0.0f;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) o[b] = f32x16{};
  }

  // K fragment st of 32-key block kb: 8 elements of key `col` of the block.
  static __device__ __forceinline__ u32x4 k_frag(const uint8_t* lds_k, int kb, int st, int col, int half) {
    const int key = kb * 32 + col;
    return *reinterpret_cast<const u32x4*>(
        lds_k + (key * kRowBytes + (((2 * st + half) ^ k_swizzle<DP>(key)) << 4)));
  }
  // V fragment of 16-key group g and 32-column block b, transposed.  A lane's 8
  // probabilities of group g are those of keys 16 g + 4 half + {0..3, 8..11};
  // the rows of V are taken in the same order, so P needs no exchange of lanes.
  static __device__ __forceinline__ u32x4 v_frag(const uint8_t* lds_v, int g, int b, int lane) {
    const int row4 = (lane & 15) >> 2, quad = lane & 3, side = (lane >> 4) & 1, half = lane >> 5;
    u32x2 v[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int key = 16 * g + 8 * u + 4 * half + row4;
      const int piece = 4 * b + 2 * side + (quad >> 1);
      v[u] = __builtin_bit_cast(
          u32x2, transposed4(lds_v, key * kRowBytes + ((piece ^ v_swizzle<DP>(key)) << 4) + (quad & 1) * 8));
    }
    return u32x4{v[0].x, v[0].y, v[1].x, v[1].y};
  }

  // The scores of a tile (S^T: column = query, row = key) become probabilities;
  // the bits of `seen` are its visible keys (at least one).
  __device__ __forceinline__ void weigh(f32x16 (&s)[KB], uint64_t seen) {
    if (seen != kAll) {
      const uint64_t mine = seen >> (4 * half);
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          s[kb][i] = (mine >> (32 * kb + 8 * (i / 4) + i % 4)) & 1 ? s[kb][i] : -__builtin_inff();
    }
    float m = s[0][0];
#pragma unroll
    for (int i = 1; i < 16 * KB; ++i) m = __builtin_fmaxf(m, s[i / 16][i % 16]);
    m = halves_max(m) * c;
    // the sums are rescaled only when the maximum has grown by more than 2^8:
    // until then they are at most that much larger than with the true maximum
    if (__any(m > top + (8.0f + kLift))) {
      const float now = __builtin_fmaxf(top, m - kLift);
      const float f = __builtin_amdgcn_exp2f(top - now);
      top = now;
      sum *= f;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[b][i] *= f;
    }
  }
  // Probabilities of 16-key group g, rounded for the product with V; their sum
  // takes them unrounded.
  __device__ __forceinline__ bf16x8 probabilities(const f32x16 (&s)[KB], int g, float (&t)[4]) const {
    float e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[g / 2][8 * (g % 2) + i], c, -top));
      t[i % 4] += e[i];
    }
    return as_bf16x8(u32x4{pair_rne<HALF>(e[0], e[1]), pair_rne<HALF>(e[2], e[3]), pair_rne<HALF>(e[4], e[5]),
                           pair_rne<HALF>(e[6], e[7])});
  }
  // O^T += V^T P^T over the tile, each group's fragments read while the group
  // before it is multiplied.
  __device__ __forceinline__ void gather(const f32x16 (&s)[KB], const uint8_t* lds_v, u32x4 (&first)[kBlocks]) {
    float t[4] = {};
    u32x4 vf[2][kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) vf[0][b] = first[b];
    bf16x8 p = probabilities(s, 0, t);
#pragma unroll
    for (int g = 0; g < 2 * KB; ++g) {
      bf16x8 pn = p;
      if (g + 1 < 2 * KB) {
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) vf[(g + 1) & 1][b] = v_frag(lds_v, g + 1, b, lane);
      }
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
        o[b] = product32<HALF>(vf[g & 1][b], p, o[b]);
      if (g + 1 < 2 * KB) pn = probabilities(s, g + 1, t);
      if (g + 1 < 2 * KB) __builtin_amdgcn_sched_group_barrier(0x100, 2 * kBlocks, 0);    // DS reads
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                               // MFMA
        if (g + 1 < 2 * KB) __builtin_amdgcn_sched_group_barrier(0x002, 32 / kBlocks, 0); // VALU
      }
      p = pn;
    }
    sum += (t[0] + t[1]) + (t[2] + t[3]);
  }

  // The same with every group's fragments read and waited for in one asm block:
  // the compiler does not see LDS reads there, so it puts no wait of its own (for
  // every load in flight) before them.  `at`: where block b's rows of V start in
  // LDS for this lane; the caller has waited for the tile.
  __device__ __forceinline__ void gather_in_flight(const f32x16 (&s)[KB], const uint32_t (&at)[kBlocks]) {
    float t[4] = {};
    const auto group = [&](auto gc) {
      constexpr int g = decltype(gc)::value, lo = 16 * g * kRowBytes, hi = lo + 8 * kRowBytes;
      u32x2 v[kBlocks][2];
      if constexpr (kBlocks == 4)
        asm volatile(
            "ds_read_b64_tr_b16 %0, %8 offset:%12\n\tds_read_b64_tr_b16 %1, %8 offset:%13\n\t"
            "ds_read_b64_tr_b16 %2, %9 offset:%12\n\tds_read_b64_tr_b16 %3, %9 offset:%13\n\t"
            "ds_read_b64_tr_b16 %4, %10 offset:%12\n\tds_read_b64_tr_b16 %5, %10 offset:%13\n\t"
            "ds_read_b64_tr_b16 %6, %11 offset:%12\n\tds_read_b64_tr_b16 %7, %11 offset:%13\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(v[0][0]), "=&v"(v[0][1]), "=&v"(v[1][0]), "=&v"(v[1][1]), "=&v"(v[2][0]), "=&v"(v[2][1]),
              "=&v"(v[3][0]), "=&v"(v[3][1])
            : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(lo), "n"(hi)
            : "memory");
      else
        asm volatile(
            "ds_read_b64_tr_b16 %0, %4 offset:%6\n\tds_read_b64_tr_b16 %1, %4 offset:%7\n\t"
            "ds_read_b64_tr_b16 %2, %5 offset:%6\n\tds_read_b64_tr_b16 %3, %5 offset:%7\n\t"
            "s_waitcnt lgkmcnt(0)"
            : "=&v"(v[0][0]), "=&v"(v[0][1]), "=&v"(v[1][0]), "=&v"(v[1][1])
            : "v"(at[0]), "v"(at[1]), "n"(lo), "n"(hi)
            : "memory");
      const bf16x8 p = probabilities(s, g, t);
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
        o[b] = product32<HALF>(u32x4{v[b][0].x, v[b][0].y, v[b][1].x, v[b][1].y}, p, o[b]);
    };
    group(std::integral_constant<int, 0>{});
    group(std::integral_constant<int, 1>{});
    if constexpr (KB == 2) {
      group(std::integral_constant<int, 2>{});
      group(std::integral_constant<int, 3>{});
    }
    sum += (t[0] + t[1]) + (t[2] + t[3]);
  }
  // The K fragments of a tile's first 32 keys, read and waited for in one asm block
  // for the same reason.
  static __device__ __forceinline__ void k_read(const uint32_t (&at)[kSteps], u32x4 (&f)[kSteps]) {
    if constexpr (kSteps == 8)
      asm volatile(
          "ds_read_b128 %0, %8\n\tds_read_b128 %1, %9\n\tds_read_b128 %2, %10\n\tds_read_b128 %3, %11\n\t"
          "ds_read_b128 %4, %12\n\tds_read_b128 %5, %13\n\tds_read_b128 %6, %14\n\tds_read_b128 %7, %15\n\t"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(f[0]), "=&v"(f[1]), "=&v"(f[2]), "=&v"(f[3]), "=&v"(f[4]), "=&v"(f[5]), "=&v"(f[6]), "=&v"(f[7])
          : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "v"(at[4]), "v"(at[5]), "v"(at[6]), "v"(at[7])
          : "memory");
    else
      asm volatile(
          "ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\tds_read_b128 %2, %6\n\tds_read_b128 %3, %7\n\t"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(f[0]), "=&v"(f[1]), "=&v"(f[2]), "=&v"(f[3])
          : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3])
          : "memory");
  }
  // Where fragment st of K starts for this lane, in a tile at `lds`.
  __device__ __forceinline__ void k_rows(uint8_t* lds, uint32_t (&at)[kSteps]) const {
#pragma unroll
    for (int st = 0; st < kSteps; ++st)
      at[st] = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds + col * kRowBytes +
               (((2 * st + half) ^ k_swizzle<DP>(col)) << 4);
  }
  // Where block b's rows of V start for this lane, in a tile at `lds`.
  __device__ __forceinline__ void v_rows(uint8_t* lds, uint32_t (&at)[kBlocks]) const {
    const int row4 = (lane & 15) >> 2, quad = lane & 3, side = (lane >> 4) & 1, key = 4 * half + row4;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
      at[b] = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds + key * kRowBytes +
              (((4 * b + 2 * side + (quad >> 1)) ^ v_swizzle<DP>(key)) << 4) + (quad & 1) * 8;
  }

  // One tile in LDS.
  __device__ __forceinline__ void tile(const uint8_t* lds_k, const uint8_t* lds_v, uint64_t seen) {
    f32x16 s[KB];
    u32x4 kf[KB][kSteps];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) s[kb] = f32x16{};
#pragma unroll
    for (int st = 0; st < kSteps; ++st)
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) kf[kb][st] = k_frag(lds_k, kb, st, col, half);
#pragma unroll
    for (int st = 0; st < kSteps; ++st)
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
        s[kb] = product32<HALF>(kf[kb][st], q[st], s[kb]);
    u32x4 vf[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) vf[b] = v_frag(lds_v, 0, b, lane);
    __builtin_amdgcn_sched_group_barrier(0x100, kSteps, 0);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
#pragma unroll
    for (int i = 0; i < 2 * kBlocks; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    weigh(s, seen);
    gather(s, lds_v, vf);
  }
};

}  // namespace

}  // namespace nvfp4
