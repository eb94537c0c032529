// kv_cache_attention: softmax(scale q k^T) v over keys and values held in NVFP4, by
// pages, with key heads shared by groups of query heads, a length for each entry and,
// where the queries' positions are given, the causal order.
//
// A code times its block scale has at most six significant bits: both products run on
// fp16 matrix instructions whose key and value operands are exact.  Query rows are
// multiplied by a power of two of their own that brings their largest element into
// [2^13, 2^14), so that fp16 holds bf16 queries of any size; it goes back into the
// row's softmax scale with the keys' tensor scale.  Probabilities are 2^(c s - m),
// rounded to fp16 (2^-11 relative; their sum is not rounded); all else is binary32, and
// the values' tensor scale is applied with the division by the sum.
//
// cache_few_kernel: up to 32 query rows a kv head, bound by the stream of codes, which
// reach the waves through rings of LDS of their own and are decoded in registers.
// cache_many_kernel: tiles of keys decoded into LDS for all of a workgroup's rows.
// cache_join_kernel: joins the workgroups that share a unit's keys.
#include <algorithm>

#include "attend.hpp"
#include "cache.hpp"

namespace nvfp4 {

namespace {

// -------------------------------------------------------------- the work and its parts

// A unit is a tile of a kv head's query rows of an entry; its keys are counted in tiles
// of KEYS, at least one (an entry that sees nothing still has zeros to write).  All
// units' tiles, entry after entry, are dealt to the workgroups in equal ranges, whatever
// the lengths.  A unit's beginning costs about as much as kStart tiles, and counts as so
// many before its first: 16 entries of 0 to 8192 keys take 23 us instead of 36.

// The keys that some query of entry b sees.
__device__ __forceinline__ int seen_by(const CacheAttention& a, int64_t b) {
  int64_t n = min((int64_t)max(a.lengths[b], 0), a.c.capacity);
  if (a.starts) n = min(n, max((int64_t)a.starts[b] + a.queries, (int64_t)0));
  return (int)n;
}

__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {               // inclusive
#define CACHE_SHIFTED(ctrl, rows) (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xF, false)
  v += CACHE_SHIFTED(0x111, 0xF);    // from 1, 2, 4, 8 lanes below, within 16
  v += CACHE_SHIFTED(0x112, 0xF);
  v += CACHE_SHIFTED(0x114, 0xF);
  v += CACHE_SHIFTED(0x118, 0xF);
  v += CACHE_SHIFTED(0x142, 0xA);    // rows 1 and 3 take the row before, then 2 and 3 lane 31
  v += CACHE_SHIFTED(0x143, 0xC);
#undef CACHE_SHIFTED
  return v;
}

// The lengths of the first 64 entries are kept, a lane each: one wait for most calls.
template <int KEYS>
struct Work {
  static constexpr uint32_t kStart = KEYS == 128 ? 3 : 5;       // (1 and 2: 27 and 26 us there, 3: 25)
  uint32_t total, share;         // what all units count, and a workgroup's part
  uint32_t units;                // of an entry
  int seen0;                     // keys that this lane's entry sees, and what a unit of it and
  uint32_t upto0;                // one of each entry before it count

  static __device__ __forceinline__ uint32_t tiles(int seen) { return (uint32_t)max((seen + KEYS - 1) / KEYS, 1); }
  // What a unit counts.
  static __device__ __forceinline__ uint32_t parts(int seen) { return tiles(seen) + kStart; }
  __device__ __forceinline__ uint32_t scan_from(const CacheAttention& a, int b0) const {
    const int b = b0 + (int)(threadIdx.x & 63);
    return wave_scan(b < a.batch ? parts(seen_by(a, b)) : 0u);
  }
  static __device__ __forceinline__ uint32_t lane_of(uint32_t v, int lane) {
    return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
  }

  __device__ __forceinline__ void start(const CacheAttention& a) {
    const int lane = threadIdx.x & 63;
    units = (uint32_t)(a.c.kv_heads * a.row_tiles);
    seen0 = lane < a.batch ? seen_by(a, lane) : 0;
    upto0 = wave_scan(lane < a.batch ? parts(seen0) : 0u);
    uint32_t sum = lane_of(upto0, 63);
    for (int b0 = 64; b0 < a.batch; b0 += 64) sum += lane_of(scan_from(a, b0), 63);
    total = sum * units;
    share = max((total + (uint32_t)a.workers - 1) / (uint32_t)a.workers, (uint32_t)a.least);
  }
  // The entry with part `at` (below the total), and its first part.
  __device__ __forceinline__ void entry_at(const CacheAttention& a, uint32_t at, int& entry, uint32_t& first) const {
    uint32_t before = 0;
    for (int b0 = 0;; b0 += 64) {
      const uint32_t upto = (before + (b0 == 0 ? upto0 : scan_from(a, b0))), all = lane_of(upto, 63);
      if (at < all * units) {
        const int i = __popcll(__ballot(upto * units <= at));
        entry = b0 + i;
        first = (i == 0 ? before : lane_of(upto, i - 1)) * units;
        return;
      }
      before = all;
    }
  }
  // The first part of entry b.
  __device__ __forceinline__ uint32_t first_of(const CacheAttention& a, int b) const {
    uint32_t sum = 0;
    int b0 = 0;
    for (; b0 + 64 <= b; b0 += 64) sum += lane_of(b0 == 0 ? upto0 : scan_from(a, b0), 63);
    if (b > b0) sum += lane_of(b0 == 0 ? upto0 : scan_from(a, b0), b - b0 - 1);
    return sum * units;
  }
  __device__ __forceinline__ int seen(const CacheAttention& a, int b) const {
    return b < 64 ? (int)lane_of((uint32_t)seen0, b) : __builtin_amdgcn_readfirstlane(seen_by(a, b));
  }
};

// The query rows of a kv head: row = token * group + head within the group.
__device__ __forceinline__ int64_t row_at(const CacheAttention& a, int64_t b, int kvh, int row,
                                          int64_t batch, int64_t token_stride, int64_t head_stride) {
  const uint32_t r = (uint32_t)row, g = (uint32_t)a.group, token = g == 1 ? r : r / g;
  return b * batch + token * token_stride + (int64_t)(kvh * g + (r - token * g)) * head_stride;
}
// The keys that row `row` of entry b sees, of the `seen` that any does.
__device__ __forceinline__ int row_limit(const CacheAttention& a, int64_t b, int row, int seen) {
  if (!a.starts) return seen;
  const int64_t n = (int64_t)a.starts[b] + row / a.group + 1;
  return (int)min(max(n, (int64_t)0), (int64_t)seen);
}

__device__ __forceinline__ float stored_scale(float amax) {
  bool degenerate;
  float s_enc, s_dec;
  tensor_scales(amax, degenerate, s_enc, s_dec);
  return s_dec;
}

// A row's power of two, from its largest magnitude (infinity and NaN stay what they
// are): `up` brings it into [2^13, 2^14), `down` is 1 / up.  Rows below 2^-100 are taken
// as if they reached it.
__device__ __forceinline__ void row_power(float top, float& up, float& down) {
  const int e = max((int)(__float_as_uint(top) >> 23), 27);
  up = __uint_as_float((uint32_t)(267 - e) << 23);
  down = __uint_as_float((uint32_t)(e - 13) << 23);
}

// What a row's score is multiplied with, log2(e) in it.  The scale meets the row's power
// first: it may be large because the queries are small, and neither part is past binary32
// then.  Never zero or infinite: a score out of sight is -infinity and has to stay that,
// one of zero is zero.
__device__ __forceinline__ float score_factor(float scale, float k_scale, float down) {
  return __builtin_fminf(__builtin_fmaxf(scale * down * (1.44269504f * k_scale), 0x1p-126f), kLowest);
}

__device__ __forceinline__ uint32_t f16x2_rne(float lo, float hi) { return pair_rne<true>(lo, hi); }

// 8 bf16 times `up`, as fp16.
__device__ __forceinline__ u32x4 scaled_f16(u32x4 v, float up) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = f16x2_rne(bf16_bits_to_f32(v[i] & 0xFFFFu) * up, __uint_as_float(v[i] & 0xFFFF0000u) * up);
  return r;
}
__device__ __forceinline__ float top_magnitude(u32x4 v) {
  const u16x2 m = max8(v);
  return bf16_bits_to_f32(m.x > m.y ? m.x : m.y);
}

// Largest over aligned groups of N = 8 or 16 lanes.
template <int N>
__device__ __forceinline__ float group_max(float v) {
#define CACHE_LANES(ctrl) \
  __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), ctrl, 0xF, 0xF, false))
  v = __builtin_fmaxf(v, CACHE_LANES(0xB1));                  // lane ^ 1
  v = __builtin_fmaxf(v, CACHE_LANES(0x4E));                  // lane ^ 2
  v = __builtin_fmaxf(v, CACHE_LANES(0x141));                 // mirrored within 8
  if (N == 16) v = __builtin_fmaxf(v, CACHE_LANES(0x140));    // mirrored within 16
#undef CACHE_LANES
  return v;
}

// Largest over the four 16-lane rows of a wave, lane by lane.
__device__ __forceinline__ float rows_max(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return halves_max(__builtin_fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float rows_sum(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return halves_sum(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// ------------------------------------------------------------------- few query rows
//
// A wave has RT tiles of 16 query rows and steps of 32 keys, two 16-key blocks T, in a
// ring of LDS of its own: up to kStages - 1 steps are on their way while one is used,
// straight from memory to LDS, so the bytes in flight take no registers.  (With a table
// fewer are: the compiler puts a wait for all loads before a look-up, also where it reads
// no new entries.  131071 keys in pages of 64 take 43 us with the join, without a table
// 42; 16 entries of 4096 keys 27.3 and 26.6.)  With 16x16x32 products
// S^T = K Q^T, O^T += V^T P^T, and lane = 16 g + m:
//   K operand   key 16 T + 4 (m % 4) + m / 4, elements g D / 4 ...
//   scores      row m, keys 16 T + 4 r + g, r = 0..3
//   P operand   the same, as it comes
//   V operand   columns m D / 16 ..., of those keys; pairs of keys are zipped nibble by
//               nibble before the conversion, which then gives pairs along the keys
// so nothing is exchanged between lanes.
//
// An element of K costs one instruction to decode and one of V one and a quarter, a
// quarter of the vector units' time at the rate of memory; what counts is bytes in flight:
// 131071 keys of 8 heads (151 MB, 29 us at a copy's rate) take 34 us and 4.7 for the join,
// 50 with a step ahead in registers; 16 entries of 0 to 8192 keys (61 MB) 20 and 4.  Of
// both, about 8 us are the chain of a workgroup's first loads (lengths, queries and table,
// codes) and its end.
constexpr int kStages = 4;

template <int D>
struct Codes;
template <>
struct Codes<128> {
  u32x4 k[2];
  uint32_t ks[2], v[2][4], vs[2][4];
};
template <>
struct Codes<64> {
  u32x2 k[2];
  uint32_t ks[2], v[2][4], vs[2][4];
};

template <int D, bool EXACT, int RT>
struct FewRows {
  static constexpr int kSteps = D / 32;        // products over the head size
  static constexpr int kCols = D / 16;         // columns of the output a lane has, a block scale each 16
  static constexpr float kLift = 7.0f;         // as in Attend

  u32x4 q[RT][kSteps];
  f32x4 o[RT][kCols];
  float top[RT], sum[RT], c[RT];
  int limit[RT];
  int lane, g, m;
  int code_bytes, scale_bytes;                 // of a token's row
  bool live_k[2], live_v;                      // this lane's blocks are within the head size
  // of a stage: K's rows of D / 2 bytes, V's, K's scales (128 bytes a 16-key block), V's
  static constexpr int kV = 16 * D, kKs = 32 * D, kVs = kKs + 256, kStage = kKs + 512;
  static constexpr int kLoads = (EXACT ? 2 * (D / 64) : 2 * (D / 16)) + 2;       // of a stage
  uint32_t at_k, at_v, at_ks, at_vs[EXACT ? 1 : 4];                              // this lane's reads in a stage

  __device__ __forceinline__ void start(const CacheAttention& a) {
    lane = threadIdx.x & 63;
    g = lane >> 4;
    m = lane & 15;
    code_bytes = EXACT ? D / 2 : a.c.dim / 2;
    scale_bytes = EXACT ? D / 16 : a.c.dim / 16;
#pragma unroll
    for (int i = 0; i < 2; ++i) live_k[i] = EXACT || (D / 64) * g + i < scale_bytes;
    live_v = EXACT || (D / 32) * m < code_bytes;
    const int key = 4 * (m & 3) + (m >> 2);
    // (16-byte pieces of K's rows are permuted by XOR, so that the reads of 8 lanes spread
    // over the banks)
    at_k = (uint32_t)(key * (D / 2) + (D == 128 && EXACT ? (g ^ (m & 3)) << 4 : (D / 8) * g));
    at_v = (uint32_t)(kV + g * (D / 2) + (D / 32) * m);
    at_ks = (uint32_t)(kKs + key * scale_bytes + min((D / 64) * g, scale_bytes - 1));
    const int block = min(m >> (D == 128 ? 1 : 2), scale_bytes - 1);
#pragma unroll
    for (int r = 0; r < (EXACT ? 1 : 4); ++r) at_vs[r] = (uint32_t)(kVs + (4 * r + g) * scale_bytes + block);
  }

  // The rows of a unit; rows past the last are the last.
  __device__ __forceinline__ void load_rows(const CacheAttention& a, int64_t b, int kvh) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int row = min(16 * rt + m, a.rows - 1);
      const uint16_t* at = a.q + row_at(a, b, kvh, row, a.q_batch, a.q_token, a.q_head) + (D / 4) * g;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        q[rt][s] = u32x4{};
        if (live_k[s / 2]) q[rt][s] = *reinterpret_cast<const u32x4*>(at + 8 * s);
      }
    }
  }
  __device__ __forceinline__ void start_rows(const CacheAttention& a, int64_t b, int seen, float k_scale) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int row = min(16 * rt + m, a.rows - 1);
      float most = 0.0f;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        most = __builtin_fmaxf(most, top_magnitude(q[rt][s]));
      }
      float up, down;
      row_power(rows_max(most), up, down);
#pragma unroll
      for (int s = 0; s < kSteps; ++s) q[rt][s] = scaled_f16(q[rt][s], up);
      c[rt] = score_factor(a.scale, k_scale, down);
      limit[rt] = row_limit(a, b, row, seen);
      top[rt] = -kLowest;
      sum[rt] = 0.0f;
#pragma unroll
      for (int j = 0; j < kCols; ++j) o[rt][j] = f32x4{};
    }
  }

  // The 16-key blocks whose rows begin at row[0] and row[1] (of a head's tokens in pages),
  // on their way to a stage.  Whole blocks: they lie in the page, whatever the length.
  __device__ __forceinline__ void load(const Cache& c, const int64_t (&row)[2], uint8_t* stage) const {
    const auto codes = [&](const uint8_t* base, uint8_t* to, bool swizzle) {
      const uint8_t* first[2] = {base + row[0] * code_bytes, base + row[1] * code_bytes};
      if constexpr (EXACT && D == 128) {
        const int r = lane >> 2, piece = (lane & 3) ^ (swizzle ? (r >> 2) & 3 : 0);
#pragma unroll
        for (int T = 0; T < 2; ++T) to_lds<16>(first[T] + (uint32_t)(r * 64 + piece * 16), to + T * 1024);
      } else if constexpr (EXACT) {
        to_lds<16>((lane < 32 ? first[0] : first[1]) + (uint32_t)((lane & 31) * 16), to);
      } else {
        constexpr int kWords = D / 8;          // of a row of D
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const int n = i * 64 + lane, token = n / kWords, word = n % kWords;
          to_lds<4>(first[i >= D / 32] + (uint32_t)((token & 15) * code_bytes + (4 * word < code_bytes ? 4 * word : 0)),
                    to + i * 256);
        }
      }
    };
    const auto scales = [&](const uint8_t* base, uint8_t* to) {
      const uint8_t* first = base + (lane < 32 ? row[0] : row[1]) * scale_bytes;
      const int word = lane & 31;
      to_lds<4>(first + (uint32_t)(word < 4 * scale_bytes ? 4 * word : 0), to);
    };
    codes(c.k_codes, stage, true);
    scales(c.k_scales, stage + kKs);
    codes(c.v_codes, stage + kV, false);
    scales(c.v_scales, stage + kVs);
  }

  // This lane's K, or V, of a stage, waited for (the compiler sees no LDS read here, and
  // puts no wait of its own for all that is on its way before it).
  __device__ __forceinline__ void read_k(uint32_t stage, Codes<D>& x) const {
    const uint32_t k = stage + at_k, s = stage + at_ks;
    if constexpr (EXACT && D == 128) {
      asm volatile(
          "ds_read_b128 %0, %4\n\tds_read_b128 %1, %4 offset:1024\n\t"
          "ds_read_u16 %2, %5\n\tds_read_u16 %3, %5 offset:128\n\ts_waitcnt lgkmcnt(0)"
          : "=&v"(x.k[0]), "=&v"(x.k[1]), "=&v"(x.ks[0]), "=&v"(x.ks[1])
          : "v"(k), "v"(s)
          : "memory");
    } else if constexpr (D == 128) {
      uint32_t s0, s1;
      asm volatile(
          "ds_read_b128 %0, %6\n\tds_read_b128 %1, %6 offset:1024\n\t"
          "ds_read_u8 %2, %7\n\tds_read_u8 %3, %7 offset:128\n\t"
          "ds_read_u8 %4, %7 offset:1\n\tds_read_u8 %5, %7 offset:129\n\ts_waitcnt lgkmcnt(0)"
          : "=&v"(x.k[0]), "=&v"(x.k[1]), "=&v"(x.ks[0]), "=&v"(x.ks[1]), "=&v"(s0), "=&v"(s1)
          : "v"(k), "v"(s)
          : "memory");
      x.ks[0] = (live_k[0] ? x.ks[0] : 0u) | (live_k[1] ? s0 << 8 : 0u);
      x.ks[1] = (live_k[0] ? x.ks[1] : 0u) | (live_k[1] ? s1 << 8 : 0u);
    } else {
      asm volatile(
          "ds_read_b64 %0, %4\n\tds_read_b64 %1, %4 offset:512\n\t"
          "ds_read_u8 %2, %5\n\tds_read_u8 %3, %5 offset:128\n\ts_waitcnt lgkmcnt(0)"
          : "=&v"(x.k[0]), "=&v"(x.k[1]), "=&v"(x.ks[0]), "=&v"(x.ks[1])
          : "v"(k), "v"(s)
          : "memory");
      if (!EXACT && !live_k[0]) x.ks[0] = x.ks[1] = 0;
    }
  }
  __device__ __forceinline__ void read_v(uint32_t stage, Codes<D>& x) const {
    const uint32_t v = stage + at_v;
    uint32_t s[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) s[r] = stage + (EXACT ? at_vs[0] + 4 * r * (D / 16) : at_vs[EXACT ? 0 : r]);
    if constexpr (D == 128)
      asm volatile(
          "ds_read_b32 %0, %16\n\tds_read_b32 %1, %16 offset:256\n\t"
          "ds_read_b32 %2, %16 offset:512\n\tds_read_b32 %3, %16 offset:768\n\t"
          "ds_read_b32 %4, %16 offset:1024\n\tds_read_b32 %5, %16 offset:1280\n\t"
          "ds_read_b32 %6, %16 offset:1536\n\tds_read_b32 %7, %16 offset:1792\n\t"
          "ds_read_u8 %8, %17\n\tds_read_u8 %9, %18\n\tds_read_u8 %10, %19\n\tds_read_u8 %11, %20\n\t"
          "ds_read_u8 %12, %17 offset:128\n\tds_read_u8 %13, %18 offset:128\n\t"
          "ds_read_u8 %14, %19 offset:128\n\tds_read_u8 %15, %20 offset:128\n\ts_waitcnt lgkmcnt(0)"
          : "=&v"(x.v[0][0]), "=&v"(x.v[0][1]), "=&v"(x.v[0][2]), "=&v"(x.v[0][3]), "=&v"(x.v[1][0]),
            "=&v"(x.v[1][1]), "=&v"(x.v[1][2]), "=&v"(x.v[1][3]), "=&v"(x.vs[0][0]), "=&v"(x.vs[0][1]),
            "=&v"(x.vs[0][2]), "=&v"(x.vs[0][3]), "=&v"(x.vs[1][0]), "=&v"(x.vs[1][1]), "=&v"(x.vs[1][2]),
            "=&v"(x.vs[1][3])
          : "v"(v), "v"(s[0]), "v"(s[1]), "v"(s[2]), "v"(s[3])
          : "memory");
    else
      asm volatile(
          "ds_read_u16 %0, %16\n\tds_read_u16 %1, %16 offset:128\n\t"
          "ds_read_u16 %2, %16 offset:256\n\tds_read_u16 %3, %16 offset:384\n\t"
          "ds_read_u16 %4, %16 offset:512\n\tds_read_u16 %5, %16 offset:640\n\t"
          "ds_read_u16 %6, %16 offset:768\n\tds_read_u16 %7, %16 offset:896\n\t"
          "ds_read_u8 %8, %17\n\tds_read_u8 %9, %18\n\tds_read_u8 %10, %19\n\tds_read_u8 %11, %20\n\t"
          "ds_read_u8 %12, %17 offset:128\n\tds_read_u8 %13, %18 offset:128\n\t"
          "ds_read_u8 %14, %19 offset:128\n\tds_read_u8 %15, %20 offset:128\n\ts_waitcnt lgkmcnt(0)"
          : "=&v"(x.v[0][0]), "=&v"(x.v[0][1]), "=&v"(x.v[0][2]), "=&v"(x.v[0][3]), "=&v"(x.v[1][0]),
            "=&v"(x.v[1][1]), "=&v"(x.v[1][2]), "=&v"(x.v[1][3]), "=&v"(x.vs[0][0]), "=&v"(x.vs[0][1]),
            "=&v"(x.vs[0][2]), "=&v"(x.vs[0][3]), "=&v"(x.vs[1][0]), "=&v"(x.vs[1][1]), "=&v"(x.vs[1][2]),
            "=&v"(x.vs[1][3])
          : "v"(v), "v"(s[0]), "v"(s[1]), "v"(s[2]), "v"(s[3])
          : "memory");
    if (!EXACT && !live_v) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x.vs[i / 4][i % 4] = 0;
    }
  }

  // One step of 32 keys from `first` on.  `blocks`: bit T, the 16-key block lies on a
  // page (if not, its codes are those of some other and count nowhere).  `all`: every
  // row sees every key.
  __device__ __forceinline__ void step(uint32_t stage, int first, int blocks, bool all) {
    f32x4 s[RT][2];
    Codes<D> x;
    read_k(stage, x);
#pragma unroll
    for (int T = 0; T < 2; ++T) {
      const f16x2 sc = e4m3_pair_to_f16x2<false>(x.ks[T]);
      f16x8 k[kSteps];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) k[i] = decode8(x.k[T][i], D == 128 && i >= 2 ? sc.y : sc.x);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        s[rt][T] = f32x4{};
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
          s[rt][T] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k[i], __builtin_bit_cast(f16x8, q[rt][i]), s[rt][T], 0, 0, 0);
      }
    }
    read_v(stage, x);
    if (!all) hide(x, s, first, blocks);
    u32x4 p[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float most = s[rt][0][0];
#pragma unroll
      for (int i = 1; i < 8; ++i) most = __builtin_fmaxf(most, s[rt][i / 4][i % 4]);
      most *= c[rt];
      // rescaled only when the maximum has grown by more than 2^8, as in Attend
      if (__any(most > top[rt] + (8.0f + kLift))) {
        const float now = __builtin_fmaxf(top[rt], rows_max(most) - kLift);
        const float f = __builtin_amdgcn_exp2f(top[rt] - now);
        top[rt] = now;
        sum[rt] *= f;
#pragma unroll
        for (int j = 0; j < kCols; ++j) o[rt][j] *= f;
      }
      float e[8], t = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[rt][i / 4][i % 4], c[rt], -top[rt]));
        t += e[i];
      }
      sum[rt] += t;
      p[rt] = u32x4{f16x2_rne(e[0], e[1]), f16x2_rne(e[2], e[3]), f16x2_rne(e[4], e[5]), f16x2_rne(e[6], e[7])};
    }
    // pairs of keys: (T, r) and (T, r + 1), r = 0, 2
    f16x2 sc[4];
    uint32_t even[4], odd[4];                  // columns 2 i and 2 i + 1 of the pair in byte i
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int T = i / 2, r = 2 * (i % 2);
      sc[i] = e4m3_pair_to_f16x2<false>(x.vs[T][r] | x.vs[T][r + 1] << 8);
      const uint32_t u = x.v[T][r], w = x.v[T][r + 1];
      even[i] = (u & 0x0F0F0F0Fu) | ((w << 4) & 0xF0F0F0F0u);
      odd[i] = ((u >> 4) & 0x0F0F0F0Fu) | (w & 0xF0F0F0F0u);
    }
    columns<0>(even, odd, sc, p);
    columns<1>(even, odd, sc, p);
    if constexpr (D == 128) {
      columns<2>(even, odd, sc, p);
      columns<3>(even, odd, sc, p);
    }
  }

  template <int BYTE>
  __device__ __forceinline__ void columns(const uint32_t (&even)[4], const uint32_t (&odd)[4], const f16x2 (&sc)[4],
                                          const u32x4 (&p)[RT]) {
    u32x4 v[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[0][i] = __builtin_bit_cast(uint32_t, e2m1_unpack2_f16<BYTE>(even[i]) * sc[i]);
      v[1][i] = __builtin_bit_cast(uint32_t, e2m1_unpack2_f16<BYTE>(odd[i]) * sc[i]);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
        o[rt][2 * BYTE + u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
            __builtin_bit_cast(f16x8, v[u]), __builtin_bit_cast(f16x8, p[rt]), o[rt][2 * BYTE + u], 0, 0, 0);
  }

  // Scores that a row does not see become -infinity.  Values that are NaN are taken out
  // of the product, where 0 times them would reach rows that do not see them, and go to
  // the rows that do.
  __device__ __forceinline__ void hide(Codes<D>& x, f32x4 (&s)[RT][2], int first, int blocks) {
    u32x4 nan = {};
    bool any = false;
#pragma unroll
    for (int T = 0; T < 2; ++T)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool is = (blocks >> T & 1) && (x.vs[T][r] & 0x7Fu) == 0x7Fu;
        any |= is;
        if (is || !(blocks >> T & 1)) x.vs[T][r] = 0;
        nan[2 * T + r / 2] |= (is ? 0x3C00u : 0u) << (16 * (r % 2));       // 1 in fp16
      }
    const bool mend = __any(any);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      u32x4 sees = {};
#pragma unroll
      for (int T = 0; T < 2; ++T)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const bool in = (blocks >> T & 1) && first + 16 * T + 4 * r + g < limit[rt];
          s[rt][T][r] = in ? s[rt][T][r] : -__builtin_inff();
          sees[2 * T + r / 2] |= (in ? 0x3C00u : 0u) << (16 * (r % 2));
        }
      if (mend) {
        // how many NaN of block m's (of lane m's columns) row n sees
        const f32x4 n = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, nan),
                                                               __builtin_bit_cast(f16x8, sees), f32x4{}, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (n[r] > 0.0f) {
#pragma unroll
            for (int j = 0; j < kCols; ++j) o[rt][j][r] = __builtin_nanf("");
          }
      }
    }
  }
};

template <int D, bool EXACT, int RT>
__global__ __launch_bounds__(256, 2) void cache_few_kernel(CacheAttention a) {
  constexpr int kKeys = 128;                   // of a tile: a step of 32 for each wave
  constexpr int kRow = D + 4;                  // of LDS, in floats
  using F = FewRows<D, EXACT, RT>;
  // the waves' rings, and where their states meet after it
  __shared__ __attribute__((aligned(1024))) uint8_t ring[4 * kStages * F::kStage];
  __shared__ float park_top[4][16], park_sum[4][16];
  static_assert(4 * kStages * F::kStage >= 4 * 16 * kRow * 4, "");
  float(*park)[16][kRow] = reinterpret_cast<float(*)[16][kRow]>(ring);
  F w;
  w.start(a);
  const int wave = wave_id();
  const float k_scale = stored_scale(a.c.amax[0]), v_scale = stored_scale(a.c.amax[1]);

  Work<kKeys> work;
  uint32_t at, end, first;
  int b;
  if (a.workers) {
    work.start(a);
    at = blockIdx.x * work.share;
    if (at >= work.total) return;
    end = min(at + work.share, work.total);
    work.entry_at(a, at, b, first);
  } else {
    b = (int)(blockIdx.x / (uint32_t)a.c.kv_heads);
    first = 0;
    at = (blockIdx.x - (uint32_t)(b * a.c.kv_heads)) * Work<kKeys>::parts(seen_by(a, b));
    end = at + 1;                              // of any size: the unit is taken whole
  }
  const uint32_t begin = at;

  while (at < end) {
    const int seen = a.workers ? work.seen(a, b) : __builtin_amdgcn_readfirstlane(seen_by(a, b));
    const uint32_t tiles = Work<kKeys>::tiles(seen), parts = tiles + Work<kKeys>::kStart;
    const uint32_t kvh = (at - first) / parts, in = at - first - kvh * parts;
    const uint32_t upto_part = a.workers ? min(in + (end - at), parts) : parts;
    const uint32_t from = in - min(in, Work<kKeys>::kStart), upto = upto_part - min(upto_part, Work<kKeys>::kStart);
    const bool whole = upto - from == tiles;
    if (upto == 0) return;                     // the range ends in the unit's beginning
    const uint32_t done = at;
    at += upto_part - in;
    w.load_rows(a, b, (int)kvh);               // on their way while the pages are looked up
    // the least that a row sees; rows are in the order of their tokens
    const int least = row_limit(a, b, 0, seen);

    const int last = min((int)upto * 4, (seen + 31) / 32);
    uint8_t* own = ring + wave * (kStages * F::kStage);
    const uint32_t own_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)own;
    // where the two 16-key blocks of step t lie; bit T: block T is on a page (its codes are
    // loaded from another if not)
    int64_t row[2];
    int held = 0, held_from = -64;             // 64 entries of the table, a lane each
    auto look_up = [&](int t) {
      uint32_t blocks = 0;
#pragma unroll
      for (int T = 0; T < 2; ++T) {
        const int key = min(32 * t + 16 * T, (seen - 1) & ~15);
        int page = b;
        if (a.c.table) {
          const int n = key >> a.c.page_shift;
          if (n >= held_from + 64) {
            held_from = n;
            held = a.c.table[b * a.c.table_pages + min((int64_t)n + w.lane, a.c.table_pages - 1)];
          }
          page = __builtin_amdgcn_readlane(held, n - held_from);
          if (page >= a.c.pages) page = -1;
        }
        blocks |= (page >= 0 ? 1u : 0u) << T;
        row[T] = cache_rows(a.c, page < 0 ? 0 : page, (int)kvh) + cache_place(a.c, key);
      }
      return blocks;
    };
    auto load = [&](int t, int stage) {
      const uint32_t blocks = look_up(t);
      w.load(a.c, row, own + stage * F::kStage);
      return blocks << (2 * stage);
    };
    int t = (int)from * 4 + wave;
    uint32_t blocks = 0;                       // two bits a stage
    if (t < last) blocks = look_up(t);
    w.start_rows(a, b, seen, k_scale);
    if (t < last) w.load(a.c, row, own);
    static_assert(F::kLoads * (kStages - 1) < 64, "the wait's count is 6 bits");
    constexpr int kWait = F::kLoads * (kStages - 1);
#pragma unroll
    for (int i = 1; i < kStages - 1; ++i)
      if (t + 4 * i < last) blocks |= load(t + 4 * i, i);
    for (int stage = 0; t < last; t += 4, stage = stage + 1 == kStages ? 0 : stage + 1) {
      const int free = stage == 0 ? kStages - 1 : stage - 1;
      if (t + 4 * (kStages - 1) < last) {
        blocks = (blocks & ~(3u << (2 * free))) | load(t + 4 * (kStages - 1), free);
        __builtin_amdgcn_s_waitcnt(0x0F70 | (kWait & 15) | (kWait >> 4) << 14);     // vmcnt: this step's are in
      } else {
        __builtin_amdgcn_s_waitcnt(0x0F70);
      }
      asm volatile("" ::: "memory");
      const int on = (int)(blocks >> (2 * stage)) & 3;
      w.step(own_at + (uint32_t)(stage * F::kStage), 32 * t, on, on == 3 && 32 * t + 32 <= least);
    }
    __syncthreads();                           // the rings are free

    // the four waves' states meet in LDS, in wave order
    const uint32_t slot = (2 * blockIdx.x + (done != begin)) * (uint32_t)a.rows;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const float l = rows_sum(w.sum[rt]);
      if (w.g == 0) {
        park_top[wave][w.m] = w.top[rt];
        park_sum[wave][w.m] = l;
      }
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int j = 0; j < F::kCols; j += 4)
          *reinterpret_cast<f32x4*>(&park[wave][w.m][F::kCols * (4 * w.g + r) + j]) =
              f32x4{w.o[rt][j][r], w.o[rt][j + 1][r], w.o[rt][j + 2][r], w.o[rt][j + 3][r]};
      __syncthreads();
      const int here = min(a.rows - 16 * rt, 16);
      for (int e = threadIdx.x; e < here * (D / 4); e += 256) {
        const int r = e / (D / 4), col = 4 * (e % (D / 4)), row = 16 * rt + r;
        float most = -__builtin_inff(), total = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (park_sum[i][r] != 0.0f) most = __builtin_fmaxf(most, park_top[i][r]);
        f32x4 s = {};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (park_sum[i][r] != 0.0f) {        // a wave that saw no key left nothing
            const float f = __builtin_amdgcn_exp2f(park_top[i][r] - most);
            total = __builtin_fmaf(park_sum[i][r], f, total);
            s += *reinterpret_cast<const f32x4*>(&park[i][r][col]) * f;
          }
        if (whole) {
          if (EXACT || col < a.c.dim) {
            const float inv = total == 0.0f ? 0.0f : v_scale / total;
            *reinterpret_cast<u32x2*>(a.out + row_at(a, b, (int)kvh, row, a.o_batch, a.o_token, a.o_head) + col) =
                u32x2{bf16x2_rne(s[0] * inv, s[1] * inv), bf16x2_rne(s[2] * inv, s[3] * inv)};
          }
        } else {
          *reinterpret_cast<f32x4*>(a.part + (int64_t)(slot + row) * D + col) = s;
          if (col == 0) a.stats[slot + row] = float2{most, total};
        }
      }
      __syncthreads();
    }
    if (!a.workers) return;
    // the next unit is the entry's next head, or the next entry's first
    if (at - first == parts * (uint32_t)a.c.kv_heads) {
      first = at;
      ++b;
    }
  }
}

// Joins what the workgroups left of a unit whose tiles several of them had: partial
// sums weighted by 2^(their maximum - the largest).  A row has N groups of D / 4 lanes,
// each of which takes every N-th of its parts in order; they meet in LDS.  4 to 5 us where
// rows are few (the lengths' and the parts' latencies), 8.4 for 64 units of 128 rows, whose
// parts (up to 67 MB) are still in the last-level cache.
template <int D, int KEYS, int TILE_ROWS, int N>
__global__ __launch_bounds__(256) void cache_join_kernel(CacheAttention a) {
  constexpr int G = D / 4, R = 256 / G / N;    // rows of a workgroup
  __shared__ f32x4 park[R][N][G];
  __shared__ float2 park_stats[R][N];
  const uint32_t units = (uint32_t)(a.c.kv_heads * a.row_tiles);
  const uint32_t rows = (uint32_t)min(a.rows, TILE_ROWS), groups = (rows + R - 1) / R;     // of a unit, at most
  const uint32_t u = blockIdx.x / groups;
  const int sub = threadIdx.x % G, n = threadIdx.x / G % N, r = threadIdx.x / G / N;
  const uint32_t in = (blockIdx.x - u * groups) * R + (uint32_t)r;
  const int b = (int)(u / units);
  const uint32_t of = u - (uint32_t)b * units, kvh = of / (uint32_t)a.row_tiles;
  const int row = (int)(of - kvh * (uint32_t)a.row_tiles) * TILE_ROWS + (int)in;
  Work<KEYS> work;
  work.start(a);
  const uint32_t parts = Work<KEYS>::parts(work.seen(a, b));
  const uint32_t from = work.first_of(a, b) + of * parts, last = from + parts - 1;
  // the workgroups that have its first and its last tile
  const uint32_t w0 = (from + Work<KEYS>::kStart) / work.share, w1 = last / work.share;
  if (w0 == w1) return;                        // one workgroup had it all
  const bool live = in < rows && row < a.rows;
  float most = -__builtin_inff(), total = 0.0f;
  f32x4 s = {};
  if (live)
    for (uint32_t w = w0 + n; w <= w1; w += 4 * N) {
      float2 st[4];                            // four parts are on their way at once
      f32x4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t u = min(w + i * N, w1);
        const int64_t slot = (int64_t)(2 * u + (u * work.share < from ? 1 : 0)) * a.slot_rows + in;
        st[i] = w + i * N <= w1 ? a.stats[slot] : float2{0.0f, 0.0f};
        v[i] = *reinterpret_cast<const f32x4*>(a.part + slot * D + 4 * sub);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (st[i].y != 0.0f) {
          const float now = __builtin_fmaxf(most, st[i].x);
          const float f0 = total == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(most - now);
          const float f1 = __builtin_amdgcn_exp2f(st[i].x - now);
          total = total == 0.0f ? st[i].y * f1 : __builtin_fmaf(total, f0, st[i].y * f1);
          s = s * f0 + v[i] * f1;
          most = now;
        }
    }
  if (N > 1) {
    park[r][n][sub] = s;
    if (sub == 0) park_stats[r][n] = float2{most, total};
    __syncthreads();
    if (n != 0) return;
    most = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (park_stats[r][i].y != 0.0f) most = __builtin_fmaxf(most, park_stats[r][i].x);
    total = 0.0f;
    s = f32x4{};
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (park_stats[r][i].y != 0.0f) {
        const float f = __builtin_amdgcn_exp2f(park_stats[r][i].x - most);
        total = __builtin_fmaf(park_stats[r][i].y, f, total);
        s += park[r][i][sub] * f;
      }
  }
  if (live && 4 * sub < a.c.dim) {
    const float inv = total == 0.0f ? 0.0f : stored_scale(a.c.amax[1]) / total;
    *reinterpret_cast<u32x2*>(a.out + row_at(a, b, (int)kvh, row, a.o_batch, a.o_token, a.o_head) + 4 * sub) =
        u32x2{bf16x2_rne(s[0] * inv, s[1] * inv), bf16x2_rne(s[2] * inv, s[3] * inv)};
  }
}

// ------------------------------------------------------------------ many query rows
//
// The waves of a workgroup have 32 rows each and share tiles of 64 keys, decoded into
// LDS in fp16: while a tile is used, the next one's blocks are decoded into the other
// buffers, between the matrix instructions of the scores, and the one after that is on
// its way.
//
// 4096 queries of 4608 keys of 24 heads: 253 to 272 us (the kernel over bf16 keys: 237 to
// 250), 0.85 to 0.92 PFLOP/s; decoding costs 54 of them (timed without), since each of 32 row
// tiles does it again.  A SIMD's time is nearly the sum of its matrix products (41%) and
// its vector instructions (52%, a third of them the decode).  2 x 16384 queries of 512 and
// 77 keys: 206 to 230; 2 x 128 queries of four heads over 16384 and 9001 keys in pages of
// 64: 76 to 85 and 8 for the join.  Not faster: one block of 32 keys after the other (309 us
// for 291, the same otherwise), V's pieces in an order without bank conflicts, wave
// priorities around the products, pages looked up tile by tile (108 us for 97).
template <int DP, int WAVES, bool PAGED>
struct ManyRows {
  using A = Attend<DP, 2, true>;
  static constexpr int kBlocksRow = DP / 16;
  static constexpr int kGroupKeys = 64 / kBlocksRow;        // keys whose blocks a wave has at once
  static constexpr int kGroups = 64 / kGroupKeys / WAVES;   // of a tile, for each wave
  static constexpr int kAll = kGroups * WAVES;
  static_assert(kGroups > 0 && 16 % kGroupKeys == 0, "a group's keys lie on one page");

  struct Tile {
    u32x2 k[kGroups], v[kGroups];
    uint32_t ks[kGroups], vs[kGroups];
    bool none[kGroups];        // the group lies on no page
  };
  // What is out of the ordinary in a tile, a byte for each block of each key: 1, its
  // values are NaN (they are zeros in LDS); 2, the key lies on no page.
  struct Odd {
    uint8_t of[64][kBlocksRow];
  };

  int wave, key, blk;          // this lane's key of a group, its block of the head
  bool live;                   // the block is within the head size
  int row_blocks;
  // of the unit: its head's first page, the blocks of a page, the entry's table
  const uint8_t *kc, *ks, *vc, *vs;
  const int32_t* table;
  int64_t page_blocks;
  int pages, shift, seen, last_group;
  int entries, held, held_from;        // of the table; 64 of them from held_from on, a lane each

  __device__ __forceinline__ void start(const CacheAttention& a) {
    const int lane = threadIdx.x & 63;
    wave = wave_id();
    key = lane / kBlocksRow;
    blk = lane % kBlocksRow;
    row_blocks = a.c.dim >> 4;
    live = blk < row_blocks;
  }
  __device__ __forceinline__ void unit(const CacheAttention& a, int64_t b, int kvh, int seen_) {
    page_blocks = (int64_t)a.c.kv_heads * a.c.page_size * row_blocks;
    const int64_t at = (int64_t)kvh * a.c.page_size * row_blocks + (PAGED ? 0 : b * page_blocks);
    kc = a.c.k_codes + 8 * at;
    ks = a.c.k_scales + at;
    vc = a.c.v_codes + 8 * at;
    vs = a.c.v_scales + at;
    table = PAGED ? a.c.table + b * a.c.table_pages : nullptr;
    pages = (int)a.c.pages;
    shift = a.c.page_shift;
    entries = (int)a.c.table_pages;
    held_from = -64;
    seen = seen_;
    last_group = (seen - 1) & ~(kGroupKeys - 1);
  }

  // Where group i of tile t begins; past the last key, the last one's group.
  __device__ __forceinline__ int first(int t, int i) const {
    return min(64 * t + (i * WAVES + wave) * kGroupKeys, last_group);
  }
  // (Tiles come in order, so the table is read 64 entries at a time.  As with few rows, a
  // look-up waits for all loads on their way, the next tile's among them.)
  __device__ __forceinline__ void look_up(int t, int (&page)[kGroups]) {
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      page[i] = 0;
      if constexpr (PAGED) {
        const int n = first(t, i) >> shift;
        if (n >= held_from + 64) {
          held_from = n;
          held = table[min(n + (int)(threadIdx.x & 63), entries - 1)];
        }
        page[i] = __builtin_amdgcn_readlane(held, n - held_from);
      }
    }
  }
  __device__ __forceinline__ void load(int t, const int (&page)[kGroups], Tile& x) const {
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const int f = first(t, i);
      x.none[i] = PAGED && (uint32_t)page[i] >= (uint32_t)pages;
      const int64_t block = PAGED ? (x.none[i] ? 0 : page[i]) * page_blocks + (f & ((1 << shift) - 1)) * row_blocks
                                  : (int64_t)f * row_blocks;
      // keys past the last are taken as the last
      const uint32_t at = (uint32_t)(min(key, seen - 1 - f) * row_blocks + blk);
      x.k[i] = x.v[i] = u32x2{0u, 0u};
      x.ks[i] = x.vs[i] = 0u;
      if (live) {
        x.k[i] = *reinterpret_cast<const u32x2*>(kc + 8 * block + 8 * at);
        x.v[i] = *reinterpret_cast<const u32x2*>(vc + 8 * block + 8 * at);
        x.ks[i] = (ks + block)[at];
        x.vs[i] = (vs + block)[at];
      }
    }
  }
  __device__ __forceinline__ void store(const Tile& x, uint8_t* lds_k, uint8_t* lds_v, Odd& odd) const {
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const int in = (i * WAVES + wave) * kGroupKeys + key;
      const bool is = !x.none[i] && (x.vs[i] & 0x7Fu) == 0x7Fu;
      odd.of[in][blk] = (uint8_t)((is ? 1 : 0) | (x.none[i] ? 2 : 0));
      const _Float16 k = e4m3_pair_to_f16x2<false>(x.ks[i]).x, v = e4m3_pair_to_f16x2<false>(is || x.none[i] ? 0u : x.vs[i]).x;
      uint8_t *to_k = lds_k + in * A::kRowBytes, *to_v = lds_v + in * A::kRowBytes;
      *reinterpret_cast<f16x8*>(to_k + (((2 * blk) ^ k_swizzle<DP>(in)) << 4)) = decode8(x.k[i].x, k);
      *reinterpret_cast<f16x8*>(to_k + (((2 * blk + 1) ^ k_swizzle<DP>(in)) << 4)) = decode8(x.k[i].y, k);
      *reinterpret_cast<f16x8*>(to_v + (((2 * blk) ^ v_swizzle<DP>(in)) << 4)) = decode8(x.v[i].x, v);
      *reinterpret_cast<f16x8*>(to_v + (((2 * blk + 1) ^ v_swizzle<DP>(in)) << 4)) = decode8(x.v[i].y, v);
    }
  }
  static __device__ __forceinline__ bool any_odd(const Odd& odd) {
    const int lane = threadIdx.x & 63;
    if constexpr (DP == 128)
      return __any(*reinterpret_cast<const uint64_t*>(odd.of[lane]) != 0);
    else
      return __any(*reinterpret_cast<const uint32_t*>(odd.of[lane]) != 0);
  }
  // Of the keys that this lane's row sees (`mine`): those on no page are taken out, the
  // blocks whose values are NaN are returned.
  static __device__ __forceinline__ uint32_t odd_seen(const Odd& odd, uint64_t& mine) {
    uint32_t hit = 0;
    for (int i = 0; i < 64; ++i) {
      uint32_t blocks = 0;
      for (int j = 0; j < kBlocksRow; ++j) {
        if (odd.of[i][j] & 2) mine &= ~(1ull << i);
        blocks |= (odd.of[i][j] & 1u) << j;
      }
      hit |= mine >> i & 1 ? blocks : 0u;
    }
    return hit;
  }
  // The scores of a tile in LDS, with the next tile decoded between the matrix
  // instructions, whose time covers it; the first fragments of V are read.
  __device__ __forceinline__ void scores(const A& w, const uint8_t* lds_k, const uint8_t* lds_v, f32x16 (&s)[2],
                                         u32x4 (&vf)[A::kBlocks], const Tile& x, uint8_t* next_k, uint8_t* next_v,
                                         Odd& next_odd) const {
    u32x4 kf[2][A::kSteps];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) s[kb] = f32x16{};
#pragma unroll
    for (int st = 0; st < A::kSteps; ++st)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) kf[kb][st] = A::k_frag(lds_k, kb, st, w.col, w.half);
#pragma unroll
    for (int st = 0; st < A::kSteps; ++st)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) s[kb] = product32<true>(kf[kb][st], w.q[st], s[kb]);
    store(x, next_k, next_v, next_odd);
#pragma unroll
    for (int b = 0; b < A::kBlocks; ++b) vf[b] = A::v_frag(lds_v, 0, b, w.lane);
    __builtin_amdgcn_sched_group_barrier(0x100, A::kSteps, 0);                     // DS reads
#pragma unroll
    for (int i = 0; i < 2 * A::kSteps; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                           // MFMA
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, 6, 0);                           // VALU
      if (i % 2) __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);                // DS write
    }
    __builtin_amdgcn_sched_barrier(0);
  }
};

template <int DP, int WAVES, bool PAGED>
__global__ __launch_bounds__(64 * WAVES, 2) void cache_many_kernel(CacheAttention a) {
  using M = ManyRows<DP, WAVES, PAGED>;
  using A = typename M::A;
  constexpr int kKeys = 64, kTileRows = 32 * WAVES;
  constexpr int kRowPieces = A::kPieces, kRowsPerLoad = 64 / kRowPieces;
  __shared__ __attribute__((aligned(1024))) uint8_t k0[A::kTileBytes], v0[A::kTileBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t k1[A::kTileBytes], v1[A::kTileBytes];
  __shared__ typename M::Odd odd0, odd1;
  __shared__ float row_down[kTileRows];
  static_assert(WAVES == 4, "a wave's 32 rows of LDS are half a buffer of the second pair");
  M part;
  part.start(a);
  const int wave = part.wave;
  const float k_scale = stored_scale(a.c.amax[0]), v_scale = stored_scale(a.c.amax[1]);
  uint8_t* own = (wave < 2 ? k1 : v1) + (wave & 1) * (32 * A::kRowBytes);

  Work<kKeys> work;
  uint32_t at, end, first;
  int b;
  const uint32_t units = (uint32_t)(a.c.kv_heads * a.row_tiles);
  if (a.workers) {
    work.start(a);
    at = blockIdx.x * work.share;
    if (at >= work.total) return;
    end = min(at + work.share, work.total);
    work.entry_at(a, at, b, first);
  } else {
    b = (int)(blockIdx.x / units);
    first = 0;
    at = (blockIdx.x - (uint32_t)b * units) * Work<kKeys>::parts(seen_by(a, b));
    end = at + 1;
  }
  const uint32_t begin = at;

  while (at < end) {
    const int seen = a.workers ? work.seen(a, b) : __builtin_amdgcn_readfirstlane(seen_by(a, b));
    const uint32_t tiles = Work<kKeys>::tiles(seen), parts = tiles + Work<kKeys>::kStart;
    const uint32_t of = (at - first) / parts, in = at - first - of * parts;
    const uint32_t upto_part = a.workers ? min(in + (end - at), parts) : parts;
    const uint32_t from = in - min(in, Work<kKeys>::kStart), upto = upto_part - min(upto_part, Work<kKeys>::kStart);
    const bool whole = upto - from == tiles;
    if (upto == 0) return;                     // the range ends in the unit's beginning
    const uint32_t done = at;
    at += upto_part - in;
    const int kvh = (int)(of / (uint32_t)a.row_tiles), row0 = (int)(of - (uint32_t)(kvh * a.row_tiles)) * kTileRows + wave * 32;

    // the queries and the first tile are on their way before anything is waited for
    u32x4 qrow[32 / kRowsPerLoad];
    {
      const int lane = opaque_lane(), piece = lane % kRowPieces;
#pragma unroll
      for (int i = 0; i < 32 / kRowsPerLoad; ++i) {
        const int row = min(row0 + i * kRowsPerLoad + lane / kRowPieces, a.rows - 1);
        qrow[i] = u32x4{};
        if (8 * piece < a.c.dim)
          qrow[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(
              a.q + row_at(a, b, kvh, row, a.q_batch, a.q_token, a.q_head) + 8 * piece));
      }
    }
    // tiles that no row of the workgroup sees are left out
    const int most = row_limit(a, b, min(row0 - wave * 32 + kTileRows, a.rows) - 1, seen);
    const int last = min((int)upto, (most + kKeys - 1) / kKeys);
    typename M::Tile x;
    int page[M::kGroups];
    uint32_t hit = 0;
    int t = (int)from;
    if (t < last) {
      part.unit(a, b, kvh, seen);
      part.look_up(t, page);
      part.load(t, page, x);
      part.look_up(t + 1, page);
    }
    A w;
    w.start(a.scale);
    {
      const int lane = opaque_lane(), piece = lane % kRowPieces;
#pragma unroll
      for (int i = 0; i < 32 / kRowsPerLoad; ++i) {
        const int r = i * kRowsPerLoad + lane / kRowPieces;
        float up, down;
        row_power(group_max<kRowPieces>(top_magnitude(qrow[i])), up, down);
        *reinterpret_cast<u32x4*>(own + r * A::kRowBytes + ((piece ^ k_swizzle<DP>(r)) << 4)) = scaled_f16(qrow[i], up);
        if (piece == 0) row_down[wave * 32 + r] = down;
      }
#pragma unroll
      for (int st = 0; st < A::kSteps; ++st)
        w.q[st] = as_bf16x8(*reinterpret_cast<const u32x4*>(
            own + w.col * A::kRowBytes + (((2 * st + w.half) ^ k_swizzle<DP>(w.col)) << 4)));
      w.c = score_factor(a.scale, k_scale, row_down[wave * 32 + w.col]);
    }
    const int limit = row_limit(a, b, min(row0 + w.col, a.rows - 1), seen);
    // of the wave's rows, which are in the order of their tokens
    const int least = row_limit(a, b, min(row0, a.rows - 1), seen);
    if (t < last) {
      part.store(x, k0, v0, odd0);
      if (t + 1 < last) part.load(t + 1, page, x);
      part.look_up(t + 2, page);
    }
    // one tile: the next is decoded into the other buffers, the one after is loaded, the
    // pages of the one after that are looked up
#define CACHE_TURN(kc, vc, oc, kn, vn, on)                                                       \
  {                                                                                              \
    __builtin_amdgcn_s_waitcnt(0xC07F); /* lgkmcnt(0): own writes are in LDS, own reads done */  \
    asm volatile("s_barrier" ::: "memory");                                                      \
    f32x16 s[2];                                                                                 \
    u32x4 vf[A::kBlocks];                                                                        \
    const bool odd = M::any_odd(oc);                                                             \
    part.scores(w, kc, vc, s, vf, x, kn, vn, on); /* (after the last, what x held before) */     \
    if (t + 2 < last) {                                                                          \
      part.load(t + 2, page, x);                                                                 \
      part.look_up(t + 3, page);                                                                 \
    }                                                                                            \
    uint64_t mine = ~0ull;                                                                       \
    if (64 * t + 64 > least) {                                                                   \
      const int n = limit - 64 * t;                                                              \
      mine = n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1;                                  \
    }                                                                                            \
    if (odd) hit |= M::odd_seen(oc, mine);                                                       \
    w.weigh(s, mine);                                                                            \
    w.gather(s, vc, vf);                                                                         \
    ++t;                                                                                         \
  }
    while (t < last) {
      CACHE_TURN(k0, v0, odd0, k1, v1, odd1)
      if (t >= last) break;
      CACHE_TURN(k1, v1, odd1, k0, v0, odd0)
    }
#undef CACHE_TURN
    // NaN values, which are zeros in LDS, go to the rows that see them
    if (__any(hit != 0)) {
#pragma unroll
      for (int o = 0; o < A::kBlocks; ++o)
#pragma unroll
        for (int e = 0; e < 16; ++e) w.o[o][e] += hit >> (2 * o + e / 8) & 1 ? __builtin_nanf("") : 0.0f;
    }

    const float l = halves_sum(w.sum);
    __syncthreads();
    const int lane = opaque_lane(), piece = lane % kRowPieces, col = lane & 31, half = lane >> 5;
    // through the wave's rows of LDS again, so that whole rows are stored
    if (!whole) {
      const int64_t slot = (int64_t)(2 * blockIdx.x + (done != begin)) * kTileRows + wave * 32;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int o = 0; o < A::kBlocks / 2; ++o)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const f32x16& v = w.o[h * (A::kBlocks / 2) + o];
            *reinterpret_cast<f32x4*>(own + col * A::kRowBytes + (((8 * o + 2 * g + half) ^ k_swizzle<DP>(col)) << 4)) =
                f32x4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
          }
#pragma unroll
        for (int i = 0; i < 32 / kRowsPerLoad; ++i) {
          const int r = i * kRowsPerLoad + lane / kRowPieces;
          *reinterpret_cast<f32x4*>(a.part + (slot + r) * DP + h * (DP / 2) + 4 * piece) =
              *reinterpret_cast<const f32x4*>(own + r * A::kRowBytes + ((piece ^ k_swizzle<DP>(r)) << 4));
        }
      }
      if (half == 0) a.stats[slot + col] = float2{w.top, l};
    } else {
      const uint32_t any = l == 0.0f ? 0u : ~0u;
      const float inv = v_scale / l;
#pragma unroll
      for (int o = 0; o < A::kBlocks; ++o)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<u32x2*>(own + col * A::kRowBytes + (((4 * o + g) ^ k_swizzle<DP>(col)) << 4) + 8 * half) =
              u32x2{bf16x2_rne(w.o[o][4 * g] * inv, w.o[o][4 * g + 1] * inv) & any,
                    bf16x2_rne(w.o[o][4 * g + 2] * inv, w.o[o][4 * g + 3] * inv) & any};
#pragma unroll
      for (int i = 0; i < 32 / kRowsPerLoad; ++i) {
        const int r = i * kRowsPerLoad + lane / kRowPieces, row = row0 + r;
        const u32x4 f = *reinterpret_cast<const u32x4*>(own + r * A::kRowBytes + ((piece ^ k_swizzle<DP>(r)) << 4));
        if (row < a.rows && 8 * piece < a.c.dim)
          __builtin_nontemporal_store(f, reinterpret_cast<u32x4*>(a.out + row_at(a, b, kvh, row, a.o_batch, a.o_token, a.o_head) + 8 * piece));
      }
    }
    __syncthreads();
    if (!a.workers) return;
    if (at - first == parts * units) {
      first = at;
      ++b;
    }
  }
}

// How a call is run.
//   Up to 32 rows a kv head: cache_few_kernel (32 rows of 16 entries of 4096 keys 44 us,
// 66 by tiles in LDS; 48 rows 92 in three tiles of 16 against 70).
//   Otherwise tiles of 128 rows.
//   Keys are dealt to two workgroups a compute unit, all that fit, where units alone leave
// some idle: 8 units of 131071 keys; from 256 units on only long ones (512 units of 512 keys
// 17.9 us dealt, 14.6 whole; lengths may be very unequal), from 1024 on none (2048 units of
// 1 to 512 keys 173 and 42, 1024 of 1 to 2048 55 and 53).  The host knows the capacity, not
// the lengths: where units alone fill the card, one long entry among many is its few
// workgroups' alone (128 entries of 8 kv heads: 27 us for 512 keys each, 487 with 65536 in
// one of them, whose bytes take 29 at a copy's rate).
struct Plan {
  int few;                       // 16-row tiles of cache_few_kernel, 1 or 2; 0: cache_many_kernel
  int64_t rows, row_tiles, units, slot_rows;
  int workers, least;
};

// A cache holds head sizes as they are; the kernels pad them to one of two in registers and
// LDS.
int padded_dim(int64_t dim) { return dim <= 64 ? 64 : 128; }

Plan plan_for(int64_t batch, int64_t queries, int64_t heads, int64_t kv_heads, int64_t capacity) {
  Plan p{};
  const int64_t cus = compute_units();
  p.rows = queries * (heads / kv_heads);
  if (p.rows <= 32) {
    p.few = p.rows <= 16 ? 1 : 2;
    p.row_tiles = 1;
    p.units = batch * kv_heads;
    p.slot_rows = p.rows;
    const int64_t tiles = (capacity + 127) / 128;
    p.least = 2;
    if (p.units <= cus ? tiles > 2 : p.units < 4 * cus && tiles > 8) p.workers = (int)(2 * cus);
  } else {
    p.row_tiles = (p.rows + 127) / 128;
    p.units = batch * kv_heads * p.row_tiles;
    p.slot_rows = 128;
    const int64_t tiles = (capacity + 63) / 64;
    p.least = 4;
    // (768 units of 72 tiles: 283 us dealt, 261 whole; 64 units of 397 tiles on average 84 + 8)
    if (tiles > 4 && p.units <= cus) p.workers = (int)(2 * cus);
  }
  return p;
}

size_t plan_bytes(const Plan& p, int dp) {
  return p.workers ? (size_t)(2 * p.workers) * (size_t)p.slot_rows * (size_t)(dp * 4 + 8) : 0;
}

template <int D, bool EXACT>
void launch_few(const CacheAttention& a, int few, dim3 grid, hipStream_t stream) {
  if (few == 1)
    cache_few_kernel<D, EXACT, 1><<<grid, 256, 0, stream>>>(a);
  else
    cache_few_kernel<D, EXACT, 2><<<grid, 256, 0, stream>>>(a);
}

}  // namespace

size_t cache_attention_workspace_bytes(int64_t batch, int64_t queries, int64_t heads, int64_t kv_heads,
                                       int64_t dim, int64_t capacity) {
  if (batch == 0 || queries == 0) return 0;
  return plan_bytes(plan_for(batch, queries, heads, kv_heads, capacity), padded_dim(dim));
}

hipError_t launch_cache_attention(CacheAttention a, void* workspace, size_t workspace_bytes,
                                  hipStream_t stream) {
  const int dp = padded_dim(a.c.dim);
  Plan p = plan_for(a.batch, a.queries, (int64_t)a.group * a.c.kv_heads, a.c.kv_heads, a.c.capacity);
  if (!workspace || workspace_bytes < plan_bytes(p, dp)) p.workers = 0;
  a.rows = (int)p.rows;
  a.row_tiles = (int)p.row_tiles;
  a.slot_rows = (int)p.slot_rows;
  a.workers = p.workers;
  a.least = p.least;
  if (p.workers) {
    a.part = static_cast<float*>(workspace);
    a.stats = reinterpret_cast<float2*>(a.part + (size_t)(2 * p.workers) * p.slot_rows * dp);
  }
  const dim3 grid((unsigned)(p.workers ? p.workers : p.units));
  if (p.few) {
    if (dp == 64)
      a.c.dim == 64 ? launch_few<64, true>(a, p.few, grid, stream) : launch_few<64, false>(a, p.few, grid, stream);
    else
      a.c.dim == 128 ? launch_few<128, true>(a, p.few, grid, stream) : launch_few<128, false>(a, p.few, grid, stream);
  } else if (dp == 64) {
    a.c.table ? cache_many_kernel<64, 4, true><<<grid, 256, 0, stream>>>(a)
              : cache_many_kernel<64, 4, false><<<grid, 256, 0, stream>>>(a);
  } else {
    a.c.table ? cache_many_kernel<128, 4, true><<<grid, 256, 0, stream>>>(a)
              : cache_many_kernel<128, 4, false><<<grid, 256, 0, stream>>>(a);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !p.workers) return e;
  const int n = p.few ? (dp == 64 ? 16 : 8) : 1, per = 256 / (dp / 4) / n;        // rows a workgroup of the join has
  const int64_t rows = std::min<int64_t>(p.rows, p.few ? 32 : 128);
  const dim3 join((unsigned)(p.units * ((rows + per - 1) / per)));
  if (p.few)
    dp == 64 ? cache_join_kernel<64, 128, 32, 16><<<join, 256, 0, stream>>>(a)
             : cache_join_kernel<128, 128, 32, 8><<<join, 256, 0, stream>>>(a);
  else
    dp == 64 ? cache_join_kernel<64, 64, 128, 1><<<join, 256, 0, stream>>>(a)
             : cache_join_kernel<128, 64, 128, 1><<<join, 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace nvfp4
