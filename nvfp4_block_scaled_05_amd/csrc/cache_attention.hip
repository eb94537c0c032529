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
// cache_few_kernel: up to 64 query rows a kv head, bound by the stream of codes, which
// go from memory to registers in the order in which the matrix instructions take them.
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
// the lengths.

// The keys that some query of entry b sees.
__device__ __forceinline__ int seen_by(const CacheAttention& a, int64_t b) {
  int64_t n = min((int64_t)max(a.lengths[b], 0), a.c.capacity);
  if (a.starts) n = min(n, max((int64_t)a.starts[b] + a.queries, (int64_t)0));
  return (int)n;
}

template <int KEYS>
__device__ __forceinline__ uint32_t tiles_of(const CacheAttention& a, int64_t b) {
  return (uint32_t)max((seen_by(a, b) + KEYS - 1) / KEYS, 1);
}

__device__ __forceinline__ uint32_t wave_scan(uint32_t v, int lane) {     // inclusive
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t o = __shfl_up(v, off, 64);
    v += lane >= off ? o : 0u;
  }
  return v;
}

struct Work {
  uint32_t total, share;         // tiles in all, of a workgroup

  // Every wave reads all lengths.
  template <int KEYS>
  __device__ __forceinline__ void start(const CacheAttention& a) {
    const int lane = threadIdx.x & 63;
    uint32_t sum = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 64) {
      const uint32_t n = b0 + lane < a.batch ? tiles_of<KEYS>(a, b0 + lane) : 0u;
      sum += __builtin_amdgcn_readlane(wave_scan(n, lane), 63);
    }
    total = sum * (uint32_t)(a.c.kv_heads * a.row_tiles);
    share = max((total + (uint32_t)a.workers - 1) / (uint32_t)a.workers, (uint32_t)a.least);
  }
  // The entry with tile `at` (below the total), and its first tile.
  template <int KEYS>
  __device__ __forceinline__ void entry_at(const CacheAttention& a, uint32_t at, int& entry, uint32_t& first) {
    const int lane = threadIdx.x & 63;
    const uint32_t units = (uint32_t)(a.c.kv_heads * a.row_tiles);
    uint32_t before = 0;
    for (int b0 = 0;; b0 += 64) {
      const uint32_t n = b0 + lane < a.batch ? tiles_of<KEYS>(a, b0 + lane) * units : 0u;
      const uint32_t upto = before + wave_scan(n, lane);
      const uint32_t all = __builtin_amdgcn_readlane(upto, 63);
      if (at < all) {
        const int i = __popcll(__ballot(upto <= at));
        entry = b0 + i;
        first = i == 0 ? before : __builtin_amdgcn_readlane(upto, i - 1);
        return;
      }
      before = all;
    }
  }
  // The first tile of entry b.
  template <int KEYS>
  __device__ __forceinline__ uint32_t first_of(const CacheAttention& a, int b) {
    const int lane = threadIdx.x & 63;
    uint32_t sum = 0;
    for (int b0 = 0; b0 < b; b0 += 64) {
      const uint32_t n = b0 + lane < b ? tiles_of<KEYS>(a, b0 + lane) : 0u;
      sum += __builtin_amdgcn_readlane(wave_scan(n, lane), 63);
    }
    return sum * (uint32_t)(a.c.kv_heads * a.row_tiles);
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

// A row's power of two, from its largest magnitude: `up` brings it into [2^13, 2^14),
// `down` is 1 / up.  Rows below 2^-100 are taken as if they reached it.
__device__ __forceinline__ void row_power(float top, float& up, float& down) {
  const int e = max((int)(__float_as_uint(top) >> 23), 27);
  up = __uint_as_float((uint32_t)(267 - e) << 23);
  down = __uint_as_float((uint32_t)(e - 13) << 23);
}

// What a row's score is multiplied with, log2(e) in it.  Never zero: a score out of
// sight is -infinity and has to stay that.
__device__ __forceinline__ float score_factor(float scale, float k_scale, float down) {
  return __builtin_fmaxf(scale * 1.44269504f * k_scale * down, 0x1p-126f);
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
// A wave has RT tiles of 16 query rows and steps of 32 keys, two 16-key blocks T.  With
// 16x16x32 products S^T = K Q^T, O^T += V^T P^T, and lane = 16 g + m:
//   K operand   key 16 T + 4 (m % 4) + m / 4, elements g D / 4 ...: one load a block
//   scores      row m, keys 16 T + 4 r + g, r = 0..3
//   P operand   the same, as it comes
//   V operand   columns m D / 16 ..., of those keys: a load for each T, r, of four
//               neighbouring rows; pairs of keys are zipped nibble by nibble before
//               the conversion, which then gives pairs along the keys
// so nothing is exchanged between lanes.
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

  __device__ __forceinline__ void start(const CacheAttention& a) {
    lane = threadIdx.x & 63;
    g = lane >> 4;
    m = lane & 15;
    code_bytes = EXACT ? D / 2 : a.c.dim / 2;
    scale_bytes = EXACT ? D / 16 : a.c.dim / 16;
#pragma unroll
    for (int i = 0; i < 2; ++i) live_k[i] = EXACT || (D / 64) * g + i < scale_bytes;
    live_v = EXACT || (D / 32) * m < code_bytes;
  }

  // The rows of a unit from `row0` on; rows past the last are the last.
  __device__ __forceinline__ void rows(const CacheAttention& a, int64_t b, int kvh, int row0, int seen, float k_scale) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int row = min(row0 + 16 * rt + m, a.rows - 1);
      const uint16_t* at = a.q + row_at(a, b, kvh, row, a.q_batch, a.q_token, a.q_head) + (D / 4) * g;
      float most = 0.0f;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        q[rt][s] = u32x4{};
        if (live_k[s / 2]) q[rt][s] = *reinterpret_cast<const u32x4*>(at + 8 * s);
        // an integer maximum: NaN is the largest
        const float v = top_magnitude(q[rt][s]);
        most = __uint_as_float(max(__float_as_uint(most), __float_as_uint(v)));
      }
      uint32_t w = __float_as_uint(most);
      w = max(w, (uint32_t)__shfl_xor((int)w, 16, 64));
      w = max(w, (uint32_t)__shfl_xor((int)w, 32, 64));
      float up, down;
      row_power(__uint_as_float(w), up, down);
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

  // The codes of one 16-key block T: keys past `room` are taken as that one.
  __device__ __forceinline__ void load(const Cache& c, int64_t row, int room, int T, Codes<D>& x) const {
    const uint8_t* kc = c.k_codes + row * code_bytes;
    const uint8_t* ks = c.k_scales + row * scale_bytes;
    const uint8_t* vc = c.v_codes + row * code_bytes;
    const uint8_t* vs = c.v_scales + row * scale_bytes;
    const int key = min(4 * (m & 3) + (m >> 2), room);
    {
      const uint8_t* at = kc + (uint32_t)(key * code_bytes + (D / 8) * g);
      const uint8_t* sc = ks + (uint32_t)(key * scale_bytes + (D / 64) * g);
      if constexpr (D == 128) {
        if constexpr (EXACT) {
          x.k[T] = *reinterpret_cast<const u32x4*>(at);
          x.ks[T] = *reinterpret_cast<const uint16_t*>(sc);
        } else {
          u32x2 lo = {}, hi = {};
          uint32_t s0 = 0, s1 = 0;
          if (live_k[0]) {
            lo = *reinterpret_cast<const u32x2*>(at);
            s0 = sc[0];
          }
          if (live_k[1]) {
            hi = *reinterpret_cast<const u32x2*>(at + 8);
            s1 = sc[1];
          }
          x.k[T] = u32x4{lo.x, lo.y, hi.x, hi.y};
          x.ks[T] = s0 | s1 << 8;
        }
      } else {
        x.k[T] = u32x2{};
        x.ks[T] = 0;
        if (live_k[0]) {
          x.k[T] = *reinterpret_cast<const u32x2*>(at);
          x.ks[T] = sc[0];
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = min(4 * r + g, room);
      x.v[T][r] = x.vs[T][r] = 0;
      if (live_v) {
        const uint8_t* at = vc + (uint32_t)(t * code_bytes + (D / 32) * m);
        if constexpr (D == 128)
          x.v[T][r] = *reinterpret_cast<const uint32_t*>(at);
        else
          x.v[T][r] = *reinterpret_cast<const uint16_t*>(at);
        x.vs[T][r] = vs[(uint32_t)(t * scale_bytes + (m >> (D == 128 ? 1 : 2)))];
      }
    }
  }

  // One step of 32 keys from `first` on.  `blocks`: bit T, the 16-key block lies on a
  // page (if not, its codes are those of some other and count nowhere).  `all`: every
  // row sees every key.
  __device__ __forceinline__ void step(Codes<D>& x, int first, int blocks, bool all) {
    f32x4 s[RT][2];
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
__global__ __launch_bounds__(256) void cache_few_kernel(CacheAttention a) {
  constexpr int kKeys = 128;                   // of a tile: a step of 32 for each wave
  constexpr int kRow = D + 4;                  // of LDS, in floats
  __shared__ float park[4][16][kRow];
  __shared__ float park_top[4][16], park_sum[4][16];
  using F = FewRows<D, EXACT, RT>;
  F w;
  w.start(a);
  const int wave = wave_id();
  const float k_scale = stored_scale(a.c.amax[0]), v_scale = stored_scale(a.c.amax[1]);

  Work work;
  uint32_t at, end, first;
  int b;
  if (a.workers) {
    work.start<kKeys>(a);
    at = blockIdx.x * work.share;
    if (at >= work.total) return;
    end = min(at + work.share, work.total);
    work.entry_at<kKeys>(a, at, b, first);
  } else {
    b = (int)(blockIdx.x / (uint32_t)a.c.kv_heads);
    first = 0;
    at = (blockIdx.x - (uint32_t)(b * a.c.kv_heads)) * tiles_of<kKeys>(a, b);
    end = at + 1;                              // of any size: the unit is taken whole
  }
  const uint32_t begin = at;

  while (at < end) {
    const int seen = __builtin_amdgcn_readfirstlane(seen_by(a, b));
    const uint32_t tiles = (uint32_t)max((seen + kKeys - 1) / kKeys, 1);
    const uint32_t kvh = (at - first) / tiles, from = at - first - kvh * tiles;
    const uint32_t upto = a.workers ? min(from + (end - at), tiles) : tiles;
    const bool whole = upto - from == tiles;
    w.rows(a, b, (int)kvh, 0, seen, k_scale);
    // the least that a row sees; rows are in the order of their tokens
    const int least = row_limit(a, b, 0, seen);

    const int last = min((int)upto * 4, (seen + 31) / 32);
    auto load = [&](int t, Codes<D>& x) {
      int blocks = 0;
#pragma unroll
      for (int T = 0; T < 2; ++T) {
        const int key = min(32 * t + 16 * T, (seen - 1) & ~15);
        const int64_t page = cache_page(a.c, b, key);
        blocks |= (page >= 0 ? 1 : 0) << T;
        w.load(a.c, cache_rows(a.c, page < 0 ? 0 : page, (int)kvh) + cache_place(a.c, key), min(seen - 1 - key, 15), T, x);
      }
      return blocks;
    };
    Codes<D> x0, x1;
    int t = (int)from * 4 + wave, b0 = 0, b1 = 0;
    if (t < last) b0 = load(t, x0);
    while (t < last) {
      if (t + 4 < last) b1 = load(t + 4, x1);
      w.step(x0, 32 * t, b0, b0 == 3 && 32 * t + 32 <= least);
      t += 4;
      if (t >= last) break;
      if (t + 4 < last) b0 = load(t + 4, x0);
      w.step(x1, 32 * t, b1, b1 == 3 && 32 * t + 32 <= least);
      t += 4;
    }

    // the four waves' states meet in LDS, in wave order
    const uint32_t slot = (2 * blockIdx.x + (at != begin)) * (uint32_t)a.rows;
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
    at += upto - from;
    if (!a.workers) return;
    // the next unit is the entry's next head, or the next entry's first
    if (at - first == tiles * (uint32_t)a.c.kv_heads) {
      first = at;
      ++b;
    }
  }
}

// Joins what the workgroups left of a unit whose tiles several of them had: partial
// sums weighted by 2^(their maximum - the largest), a workgroup a row: groups of D / 4
// lanes take every (256 / (D / 4))-th of them in order and meet in LDS.
template <int D, int KEYS, int TILE_ROWS>
__global__ __launch_bounds__(256) void cache_join_kernel(CacheAttention a) {
  constexpr int G = D / 4, N = 256 / G;
  __shared__ f32x4 park[N][G];
  __shared__ float2 park_stats[N];
  const uint32_t units = (uint32_t)(a.c.kv_heads * a.row_tiles);
  const uint32_t rows = (uint32_t)min(a.rows, TILE_ROWS);             // of a unit, at most
  const uint32_t u = blockIdx.x / rows, in = blockIdx.x - u * rows;
  const int b = (int)(u / units);
  const uint32_t of = u - (uint32_t)b * units, kvh = of / (uint32_t)a.row_tiles;
  const int row = (int)(of - kvh * (uint32_t)a.row_tiles) * TILE_ROWS + (int)in;
  if (row >= a.rows) return;
  Work work;
  work.start<KEYS>(a);
  const uint32_t tiles = tiles_of<KEYS>(a, b);
  const uint32_t from = work.first_of<KEYS>(a, b) + of * tiles, last = from + tiles - 1;
  const uint32_t w0 = from / work.share, w1 = last / work.share;
  if (w0 == w1) return;                        // one workgroup had it all
  const int sub = threadIdx.x % G, n = threadIdx.x / G;
  // each group's own maximum first, then the whole row's
  float most = -__builtin_inff(), total = 0.0f;
  f32x4 s = {};
  for (uint32_t w = w0 + n; w <= w1; w += N) {
    const int64_t slot = (int64_t)(2 * w + (w * work.share < from ? 1 : 0)) * a.slot_rows + in;
    const float2 st = a.stats[slot];
    const f32x4 v = *reinterpret_cast<const f32x4*>(a.part + slot * D + 4 * sub);
    if (st.y != 0.0f) {
      const float now = __builtin_fmaxf(most, st.x);
      const float f0 = total == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(most - now), f1 = __builtin_amdgcn_exp2f(st.x - now);
      // (what a NaN sum has left stays NaN)
      total = total == 0.0f ? st.y * f1 : __builtin_fmaf(total, f0, st.y * f1);
      s = s * f0 + v * f1;
      most = now;
    }
  }
  park[n][sub] = s;
  if (sub == 0) park_stats[n] = float2{most, total};
  __syncthreads();
  if (n != 0) return;
  most = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (park_stats[i].y != 0.0f) most = __builtin_fmaxf(most, park_stats[i].x);
  total = 0.0f;
  s = f32x4{};
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (park_stats[i].y != 0.0f) {
      const float f = __builtin_amdgcn_exp2f(park_stats[i].x - most);
      total = __builtin_fmaf(park_stats[i].y, f, total);
      s += park[i][sub] * f;
    }
  if (4 * sub < a.c.dim) {
    const float inv = total == 0.0f ? 0.0f : stored_scale(a.c.amax[1]) / total;
    *reinterpret_cast<u32x2*>(a.out + row_at(a, b, (int)kvh, row, a.o_batch, a.o_token, a.o_head) + 4 * sub) =
        u32x2{bf16x2_rne(s[0] * inv, s[1] * inv), bf16x2_rne(s[2] * inv, s[3] * inv)};
  }
}

// ------------------------------------------------------------------ many query rows
//
// The waves of a workgroup have 32 rows each and share tiles of 64 keys, decoded into
// LDS in fp16: while a tile is used, the next one's blocks (a thread has kItems of
// them) are decoded into the other buffers and the one after that is on its way.
template <int DP, int WAVES>
struct ManyRows {
  using A = Attend<DP, 2, true>;
  static constexpr int kBlocksRow = DP / 16;
  static constexpr int kHalf = 64 * kBlocksRow;             // blocks of K, and of V, of a tile
  static constexpr int kItems = 2 * kHalf / (64 * WAVES);
  static_assert(kItems > 0 && kHalf % 64 == 0, "an item is K's or V's for a whole wave");

  struct Tile {
    u32x2 codes[kItems];
    uint32_t scale[kItems];
    uint64_t seen;             // keys below the entry's length and on a page
  };

  int wave, lane;

  __device__ __forceinline__ int item(int i) const { return (i * WAVES + wave) * 64 + lane; }

  // The pages of the keys of tile t, a lane each (-1: none).
  __device__ __forceinline__ int pages(const CacheAttention& a, int64_t b, int seen, int t) const {
    const int key = 64 * t + lane;
    return (int)cache_page(a.c, b, min(key, seen - 1));
  }
  __device__ __forceinline__ void load(const CacheAttention& a, int kvh, int seen, int t, int page, Tile& x) const {
    x.seen = __ballot(64 * t + lane < seen && page >= 0);
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int n = item(i), of = n % kHalf, key = of / kBlocksRow, blk = of % kBlocksRow;
      const bool value = n >= kHalf;
      const int from = __shfl(page, key, 64), at = min(64 * t + key, seen - 1);
      x.codes[i] = u32x2{0u, 0u};
      x.scale[i] = 0u;
      if (16 * blk < a.c.dim && from >= 0) {
        const int64_t row = cache_rows(a.c, from, kvh) + cache_place(a.c, at);
        const int64_t block = row * (a.c.dim >> 4) + blk;
        x.codes[i] = *reinterpret_cast<const u32x2*>((value ? a.c.v_codes : a.c.k_codes) + 8 * block);
        x.scale[i] = (value ? a.c.v_scales : a.c.k_scales)[block];
      }
    }
  }
  // `nan`: for each wave, the value blocks of its items that are NaN.  They are written
  // as zeros.
  __device__ __forceinline__ void store(Tile& x, uint8_t* lds_k, uint8_t* lds_v, uint64_t (*nan)[WAVES]) const {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int n = item(i), of = n % kHalf, key = of / kBlocksRow, blk = of % kBlocksRow;
      const bool value = n >= kHalf;
      bool is = false;
      if (value) is = (x.scale[i] & 0x7Fu) == 0x7Fu;
      const uint64_t bits = __ballot(is);
      if (lane == 0) nan[i][wave] = bits;
      const f16x2 s = e4m3_pair_to_f16x2<false>(is ? 0u : x.scale[i]);
      uint8_t* to = (value ? lds_v : lds_k) + key * A::kRowBytes;
      const int swizzle = value ? v_swizzle<DP>(key) : k_swizzle<DP>(key);
      *reinterpret_cast<f16x8*>(to + (((2 * blk) ^ swizzle) << 4)) = decode8(x.codes[i].x, s.x);
      *reinterpret_cast<f16x8*>(to + (((2 * blk + 1) ^ swizzle) << 4)) = decode8(x.codes[i].y, s.x);
    }
  }
};

template <int DP, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 2) void cache_many_kernel(CacheAttention a) {
  using M = ManyRows<DP, WAVES>;
  using A = typename M::A;
  constexpr int kKeys = 64, kTileRows = 32 * WAVES;
  constexpr int kRowPieces = A::kPieces, kRowsPerLoad = 64 / kRowPieces;
  __shared__ __attribute__((aligned(1024))) uint8_t k0[A::kTileBytes], v0[A::kTileBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t k1[A::kTileBytes], v1[A::kTileBytes];
  __shared__ uint64_t nan0[M::kItems][WAVES], nan1[M::kItems][WAVES];
  __shared__ float row_down[kTileRows];
  static_assert(WAVES == 4, "a wave's 32 rows of LDS are half a buffer of the second pair");
  M part;
  part.wave = wave_id();
  part.lane = threadIdx.x & 63;
  const int wave = part.wave, lane = part.lane;
  const float k_scale = stored_scale(a.c.amax[0]), v_scale = stored_scale(a.c.amax[1]);
  uint8_t* own = (wave < 2 ? k1 : v1) + (wave & 1) * (32 * A::kRowBytes);
  const int piece = lane % kRowPieces;

  Work work;
  uint32_t at, end, first;
  int b;
  const uint32_t units = (uint32_t)(a.c.kv_heads * a.row_tiles);
  if (a.workers) {
    work.start<kKeys>(a);
    at = blockIdx.x * work.share;
    if (at >= work.total) return;
    end = min(at + work.share, work.total);
    work.entry_at<kKeys>(a, at, b, first);
  } else {
    b = (int)(blockIdx.x / units);
    first = 0;
    at = (blockIdx.x - (uint32_t)b * units) * tiles_of<kKeys>(a, b);
    end = at + 1;
  }
  const uint32_t begin = at;

  while (at < end) {
    const int seen = __builtin_amdgcn_readfirstlane(seen_by(a, b));
    const uint32_t tiles = (uint32_t)max((seen + kKeys - 1) / kKeys, 1);
    const uint32_t of = (at - first) / tiles, from = at - first - of * tiles;
    const uint32_t upto = a.workers ? min(from + (end - at), tiles) : tiles;
    const bool whole = upto - from == tiles;
    const int kvh = (int)(of / (uint32_t)a.row_tiles), row0 = (int)(of - (uint32_t)(kvh * a.row_tiles)) * kTileRows + wave * 32;

    A w;
    w.start(a.scale);
    {
      u32x4 qrow[32 / kRowsPerLoad];
#pragma unroll
      for (int i = 0; i < 32 / kRowsPerLoad; ++i) {
        const int row = min(row0 + i * kRowsPerLoad + lane / kRowPieces, a.rows - 1);
        qrow[i] = u32x4{};
        if (8 * piece < a.c.dim)
          qrow[i] = *reinterpret_cast<const u32x4*>(a.q + row_at(a, b, kvh, row, a.q_batch, a.q_token, a.q_head) + 8 * piece);
      }
#pragma unroll
      for (int i = 0; i < 32 / kRowsPerLoad; ++i) {
        const int r = i * kRowsPerLoad + lane / kRowPieces;
        uint32_t top = __float_as_uint(top_magnitude(qrow[i]));
#pragma unroll
        for (int off = 1; off < kRowPieces; off <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, 64));
        float up, down;
        row_power(__uint_as_float(top), up, down);
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
    const int most = row_limit(a, b, min(row0 + 31, a.rows - 1), seen);

    const int last = seen > 0 ? (int)upto : (int)from;
    typename M::Tile x;
    uint64_t sight = 0;
    int page = -1;
    int t = (int)from;
    if (t < last) {
      part.load(a, kvh, seen, t, part.pages(a, b, seen, t), x);
      if (t + 1 < last) page = part.pages(a, b, seen, t + 1);
      part.store(x, k0, v0, nan0);
      sight = x.seen;
      if (t + 1 < last) {
        part.load(a, kvh, seen, t + 1, page, x);
        if (t + 2 < last) page = part.pages(a, b, seen, t + 2);
      }
    }
    // one tile: the next is decoded into the other buffers, the one after is loaded
#define CACHE_TURN(kc, vc, nc, kn, vn, nn)                                                             {                                                                                                      __builtin_amdgcn_s_waitcnt(0xC07F); /* lgkmcnt(0): own writes are in LDS, own reads done */          asm volatile("s_barrier" ::: "memory");                                                              uint64_t sight_next = 0;                                                                             if (t + 1 < last) {                                                                                    part.store(x, kn, vn, nn);                                                                           sight_next = x.seen;                                                                                 if (t + 2 < last) {                                                                                    part.load(a, kvh, seen, t + 2, page, x);                                                             if (t + 3 < last) page = part.pages(a, b, seen, t + 3);                                            }                                                                                                  }                                                                                                    if (64 * t < most) {                                                                                   uint64_t mine = sight;                                                                               if (64 * t + 64 > least) {                                                                             const int n = limit - 64 * t;                                                                        mine &= n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1;                                         }                                                                                                    w.tile(kc, vc, mine);                                                                                spread_nan(w, nc, mine);                                                                           }                                                                                                    sight = sight_next;                                                                                  ++t;                                                                                               }
    // NaN values go to the rows that see them
    auto spread_nan = [&](A& w, uint64_t (&nan)[M::kItems][WAVES], uint64_t mine) {
      const uint64_t* flat = &nan[0][0];
      if (__any(lane < M::kItems * WAVES && flat[lane < M::kItems * WAVES ? lane : 0] != 0)) {
        for (int i = 0; i < M::kItems; ++i)
          for (int v = 0; v < WAVES; ++v) {
            const int n = (i * WAVES + v) * 64 - M::kHalf;             // of the values
            const uint64_t bits = nan[i][v];
            if (n < 0 || bits == 0) continue;
            for (int j = 0; j < 64 / M::kBlocksRow; ++j) {
              const uint32_t blocks = (uint32_t)(bits >> (j * M::kBlocksRow)) & ((1u << M::kBlocksRow) - 1);
              if (blocks == 0 || !(mine >> (n / M::kBlocksRow + j) & 1)) continue;
#pragma unroll
              for (int o = 0; o < A::kBlocks; ++o)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  if (blocks >> (2 * o + e / 8) & 1) w.o[o][e] = __builtin_nanf("");
            }
          }
      }
    };
    while (t < last) {
      CACHE_TURN(k0, v0, nan0, k1, v1, nan1)
      if (t >= last) break;
      CACHE_TURN(k1, v1, nan1, k0, v0, nan0)
    }
#undef CACHE_TURN

    const float l = halves_sum(w.sum);
    __syncthreads();
    // through the wave's rows of LDS again, so that whole rows are stored
    if (!whole) {
      const int64_t slot = (int64_t)(2 * blockIdx.x + (at != begin)) * kTileRows + wave * 32;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int o = 0; o < A::kBlocks / 2; ++o)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const f32x16& v = w.o[h * (A::kBlocks / 2) + o];
            *reinterpret_cast<f32x4*>(own + w.col * A::kRowBytes + (((8 * o + 2 * g + w.half) ^ k_swizzle<DP>(w.col)) << 4)) =
                f32x4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
          }
#pragma unroll
        for (int i = 0; i < 32 / kRowsPerLoad; ++i) {
          const int r = i * kRowsPerLoad + lane / kRowPieces;
          *reinterpret_cast<f32x4*>(a.part + (slot + r) * DP + h * (DP / 2) + 4 * piece) =
              *reinterpret_cast<const f32x4*>(own + r * A::kRowBytes + ((piece ^ k_swizzle<DP>(r)) << 4));
        }
      }
      if (w.half == 0) a.stats[slot + w.col] = float2{w.top, l};
    } else {
      const uint32_t any = l == 0.0f ? 0u : ~0u;
      const float inv = v_scale / l;
#pragma unroll
      for (int o = 0; o < A::kBlocks; ++o)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<u32x2*>(own + w.col * A::kRowBytes + (((4 * o + g) ^ k_swizzle<DP>(w.col)) << 4) + 8 * w.half) =
              u32x2{bf16x2_rne(w.o[o][4 * g] * inv, w.o[o][4 * g + 1] * inv) & any,
                    bf16x2_rne(w.o[o][4 * g + 2] * inv, w.o[o][4 * g + 3] * inv) & any};
#pragma unroll
      for (int i = 0; i < 32 / kRowsPerLoad; ++i) {
        const int r = i * kRowsPerLoad + lane / kRowPieces, row = row0 + r;
        const u32x4 f = *reinterpret_cast<const u32x4*>(own + r * A::kRowBytes + ((piece ^ k_swizzle<DP>(r)) << 4));
        if (row < a.rows && 8 * piece < a.c.dim)
          *reinterpret_cast<u32x4*>(a.out + row_at(a, b, kvh, row, a.o_batch, a.o_token, a.o_head) + 8 * piece) = f;
      }
    }
    __syncthreads();
    at += upto - from;
    if (!a.workers) return;
    if (at - first == tiles * units) {
      first = at;
      ++b;
    }
  }
}

// How a call is run.
struct Plan {
  int few;                       // 16-row tiles of cache_few_kernel: 1, 2, 4; 0: cache_many_kernel
  int64_t rows, row_tiles, units, slot_rows;
  int workers, least;
};

int padded_dim(int64_t dim) { return dim <= 64 ? 64 : 128; }

Plan plan_for(int64_t batch, int64_t queries, int64_t heads, int64_t kv_heads, int64_t capacity) {
  Plan p{};
  const int64_t cus = compute_units();
  p.rows = queries * (heads / kv_heads);
  if (p.rows <= 64) {
    p.few = p.rows <= 16 ? 1 : p.rows <= 32 ? 2 : 4;
    p.row_tiles = 1;
    p.units = batch * kv_heads;
    p.slot_rows = p.rows;
    const int64_t tiles = (capacity + 127) / 128;
    p.least = 2;
    if (tiles > 2) p.workers = (int)(2 * cus);
  } else {
    p.row_tiles = (p.rows + 127) / 128;
    p.units = batch * kv_heads * p.row_tiles;
    p.slot_rows = 128;
    const int64_t tiles = (capacity + 63) / 64;
    p.least = 4;
    if (tiles > 4 && p.units < 4 * cus) p.workers = (int)(2 * cus);
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
  else if (few == 2)
    cache_few_kernel<D, EXACT, 2><<<grid, 256, 0, stream>>>(a);
  else
    cache_few_kernel<D, EXACT, 4><<<grid, 256, 0, stream>>>(a);
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
    cache_many_kernel<64, 4><<<grid, 256, 0, stream>>>(a);
  } else {
    cache_many_kernel<128, 4><<<grid, 256, 0, stream>>>(a);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !p.workers) return e;
  const dim3 join((unsigned)(p.units * std::min<int64_t>(p.rows, p.slot_rows)));
  if (p.few)
    dp == 64 ? cache_join_kernel<64, 128, 64><<<join, 256, 0, stream>>>(a)
             : cache_join_kernel<128, 128, 64><<<join, 256, 0, stream>>>(a);
  else
    dp == 64 ? cache_join_kernel<64, 64, 128><<<join, 256, 0, stream>>>(a)
             : cache_join_kernel<128, 64, 128><<<join, 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace nvfp4
