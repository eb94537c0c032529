// dit_cross_attention: softmax(scale q k^T) v of query heads over the keys and
// values of an encoder (or of any other length), with key heads shared by
// groups of query heads, key lengths and a key mask.
//
// One pass over the keys: a wave computes the transposed scores S^T = K Q^T of 32
// query rows and a tile of keys, so a lane holds scores of one query, keeps that
// query's running maximum m and sum l of 2^(c s - m) (c = scale log2 e) and
// accumulates O^T += V^T P^T, P = 2^(c s - m) in bf16: in this form P is already
// where the second product takes it.  All else is binary32.  Query rows are
// (token, head of the group) pairs, so the heads that share keys share their tiles.
//
// Two kernels: attention_kernel, bound by the matrix cores and the exponentials
// beside them, and attention_few_kernel for up to 32 query rows a kv head, bound by
// the stream of keys and values.  A third one joins key splits.
#include "attend.hpp"
#include "kernels.hpp"

namespace nvfp4 {

namespace {

constexpr uint32_t kNoData = 0x80000000u;       // a lane offset past every tile: loads zeros

// 16 bytes per lane from base + offset straight into LDS, `to` bytes into the
// array `lds`; offsets from kNoData up are out of the resource's range and load
// zeros.  (LDS positions are an array and one offset throughout: the compiler
// then still knows which array an access is to, and does not make reads of one
// wait for loads in flight into the other.)  STREAM: past the caches.
template <bool STREAM>
__device__ __forceinline__ void tile_load(const void* base, uint32_t offset, uint8_t* lds, int to) {
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<void*>(base), (short)0, (int)kNoData, kBufferWord3);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      r, (__attribute__((address_space(3))) void*)(lds + to), 16, offset, 0, 0, STREAM ? 2 : 0);   // 2: nt
}

// Global -> LDS loads of one tile by WAVES waves (this one the `wave`-th).  Keys
// out of sight and pieces past the head size load as zeros.
template <int DP, int KB, int WAVES>
struct TileLoader {
  using A = Attend<DP, KB>;
  static constexpr int kLoads = A::kKeys * A::kPieces / (64 * WAVES);   // per operand
  uint32_t k_off[kLoads], v_off[kLoads];
  int key[kLoads], at[kLoads];

  __device__ __forceinline__ void start(const Attention& a, int wave) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      at[i] = (wave * kLoads + i) * 1024;
      const int n = (wave * kLoads + i) * 64 + lane, piece = n % A::kPieces;
      key[i] = n / A::kPieces;
      const int kp = piece ^ k_swizzle<DP>(key[i]), vp = piece ^ v_swizzle<DP>(key[i]);
      k_off[i] = 8 * kp < a.dim ? (uint32_t)(key[i] * a.k_token * 2 + kp * 16) : kNoData;
      v_off[i] = 8 * vp < a.dim ? (uint32_t)(key[i] * a.v_token * 2 + vp * 16) : kNoData;
    }
  }
  __device__ __forceinline__ void issue(const uint16_t* k, const uint16_t* v, uint64_t seen,
                                        uint8_t* lds_k, uint8_t* lds_v) const {
    if (seen == A::kAll) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) tile_load<false>(k, k_off[i], lds_k, at[i]);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) tile_load<false>(v, v_off[i], lds_v, at[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        tile_load<false>(k, k_off[i] | (((uint32_t)(~seen >> key[i]) & 1u) * kNoData), lds_k, at[i]);
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        tile_load<false>(v, v_off[i] | (((uint32_t)(~seen >> key[i]) & 1u) * kNoData), lds_v, at[i]);
    }
  }
};

// Which part of the problem a workgroup has.
struct Place {
  int64_t batch;
  int kvh, row_tile, keys;
  const uint16_t *k, *v;
  const uint8_t* mask;
};

// A (batch, kv head) and the keys its entry sees.
__device__ __forceinline__ void place_head(const Attention& a, Place& p, uint32_t bh) {
  const uint32_t batch = bh / (uint32_t)a.kv_heads;
  p.batch = batch;
  p.kvh = (int)(bh - batch * (uint32_t)a.kv_heads);
  p.k = a.k + p.batch * a.k_batch + p.kvh * a.k_head;
  p.v = a.v + p.batch * a.v_batch + p.kvh * a.v_head;
  p.mask = a.mask ? a.mask + p.batch * a.mask_stride : nullptr;
}
__device__ __forceinline__ int seen_keys(const Attention& a, const Place& p) {
  return a.lengths ? min(max(__builtin_amdgcn_readfirstlane(a.lengths[p.batch]), 0), a.keys) : a.keys;
}

// Work unit u: a row tile of a (batch, kv head).  Workgroups are dealt to the 8
// XCDs in turn; eight heads run side by side, each on one XCD, whose L2 keeps its
// keys, so entries of unequal lengths are spread over all of them.  (One
// contiguous range of heads per XCD gives an XCD one batch entry: 245 us against
// 175 for a CFG pair of 512 and 77 text states.)
__device__ __forceinline__ void place_unit(const Attention& a, Place& p, uint32_t u) {
  const uint32_t tiles = (uint32_t)a.row_tiles, heads = (uint32_t)a.batch * (uint32_t)a.kv_heads;
  const uint32_t full = heads / kXcds * kXcds;
  uint32_t bh;
  if (u < full * tiles) {
    const uint32_t slot = u / kXcds;
    bh = slot / tiles * kXcds + u % kXcds;
    p.row_tile = (int)(slot % tiles);
  } else {
    const uint32_t rest = u - full * tiles;
    bh = full + rest / tiles;
    p.row_tile = (int)(rest % tiles);
  }
  place_head(a, p, bh);
}

// The visible keys among the KEYS from `first` on (wave-uniform).
template <int KEYS>
__device__ __forceinline__ uint64_t seen_from(const Place& p, int first, int lane) {
  const int n = p.keys - first;
  uint64_t s = n >= KEYS ? (KEYS == 64 ? ~0ull : (1ull << (KEYS & 63)) - 1) : n <= 0 ? 0 : (1ull << n) - 1;
  if (p.mask) s &= __ballot(lane < n && lane < KEYS && p.mask[first + lane] != 0);
  return s;
}

// Row = token * group + head within the group (fewer than 2^31 rows a call).
__device__ __forceinline__ int64_t row_offset(const Attention& a, const Place& p, int64_t row, int64_t batch,
                                              int64_t token_stride, int64_t head_stride) {
  const uint32_t r = (uint32_t)row, g = (uint32_t)a.group;
  const uint32_t token = g == 1 ? r : r / g;
  return p.batch * batch + token * token_stride + (int64_t)(p.kvh * g + (r - token * g)) * head_stride;
}
__device__ __forceinline__ const uint16_t* query_row(const Attention& a, const Place& p, int64_t row) {
  return a.q + row_offset(a, p, row, a.q_batch, a.q_token, a.q_head);
}
__device__ __forceinline__ uint16_t* output_row(const Attention& a, const Place& p, int64_t row) {
  return a.out + row_offset(a, p, row, a.o_batch, a.o_token, a.o_head);
}

// A lane's walk over rows: first, first + by, ... as an offset from the batch
// entry's start, stepped without a product or a division.
struct RowStep {
  int64_t at, step, wrap;
  int row, by, head, by_head, group;
  __device__ __forceinline__ RowStep(const Attention& a, const Place& p, int64_t first, int by_, int64_t token_stride,
                                     int64_t head_stride) {
    const uint32_t r = (uint32_t)first, g = (uint32_t)a.group, token = g == 1 ? r : r / g;
    row = (int)r;
    by = by_;
    group = a.group;
    head = (int)(r - token * g);
    const int by_token = by / group;
    by_head = by - by_token * group;
    at = token * token_stride + (p.kvh * group + head) * head_stride;
    step = by_token * token_stride + by_head * head_stride;
    wrap = token_stride - group * head_stride;
  }
  __device__ __forceinline__ void next() {
    row += by;
    head += by_head;
    at += step;
    const bool over = head >= group;
    head -= over ? group : 0;
    at += over ? wrap : 0;
  }
};

// Many query rows: the four waves of a workgroup have 32 rows each and share the
// tiles of 64 keys, which the next turn's loads replace while this turn's are
// used.  At 4096 queries and 4608 keys of 24 heads: 218 to 260 us by card, at best 1.06
// PFLOP/s (the matrix cores alone reach 1.68 on such data); a tile of 32 rows by 64
// keys costs a SIMD 1024 cycles of matrix products and about 950 of exponentials, sums
// and maxima, and two waves a SIMD hide about half of the latter.  The rest is power:
// on zeros the same instructions take a fifth less.  At 2 x 16384 queries of 77 and 512
// keys: 164 to 180 us, at best 0.72 PFLOP/s and 2.5 TB/s.  Not faster, in turn with the
// same kernel: the exponentials of one block of 32 keys under the scores of the next in
// one wave (235 us for 226), 64 rows a wave and the loads spread between the products
// (registers spill), query rows fetched a unit ahead by workgroups that stay (they
// spill: 247 us for 178).
template <int DP>
__global__ __launch_bounds__(256, 2) void attention_kernel(Attention a) {
  using A = Attend<DP, 2>;
  constexpr int kRowPieces = A::kPieces, kRowsPerLoad = 64 / kRowPieces;
  __shared__ __attribute__((aligned(1024))) uint8_t k0[A::kTileBytes], v0[A::kTileBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t k1[A::kTileBytes], v1[A::kTileBytes];
  // every unit's first split, then the second ones, ...
  Place p;
  const uint32_t split = blockIdx.x / (uint32_t)a.units, unit = blockIdx.x - split * (uint32_t)a.units;
  place_unit(a, p, unit);
  const int wave = wave_id();
  A w;
  w.start(a.scale);

  // this wave's query rows (row = token * group + head within the group), read
  // a whole row at a time, before anything that waits
  const int64_t rows = (int64_t)a.queries * a.group;
  const int64_t row0 = (int64_t)p.row_tile * 128 + wave * 32;
  const int piece = w.lane % kRowPieces;
  u32x4 qrow[32 / kRowsPerLoad];
  {
    // Rows past the last read the first token's.  Queries and outputs pass through
    // once and are streamed past the caches, which stay with the keys (173 us against
    // 180 at 2 x 16384 queries of 77 and 512 keys; no difference at 4096).
    const uint16_t* q = a.q + p.batch * a.q_batch + (8 * piece < a.dim ? 8 * piece : 0);
    const int64_t none = (int64_t)p.kvh * a.group * a.q_head;
    RowStep step(a, p, row0 + w.lane / kRowPieces, kRowsPerLoad, a.q_token, a.q_head);
#pragma unroll
    for (int i = 0; i < 32 / kRowsPerLoad; ++i, step.next())
      qrow[i] = __builtin_nontemporal_load(
          reinterpret_cast<const u32x4*>(q + (step.row < rows ? step.at : none)));
  }
  p.keys = seen_keys(a, p);
  TileLoader<DP, 2, 4> load;
  load.start(a, wave);
  const int tiles = (p.keys + A::kKeys - 1) / A::kKeys;
  const int share = (tiles + a.splits - 1) / a.splits;
  const int last = min(((int)split + 1) * share, tiles);
  // the next tile after t that has a visible key
  auto next = [&](int t, uint64_t& seen) {
    for (++t; t < last; ++t)
      if ((seen = seen_from<64>(p, t * A::kKeys, w.lane)) != 0) break;
    return t;
  };
  uint64_t seen = 0, seen_next = 0;
  int t = next((int)split * share - 1, seen);
  if (t < last)
    load.issue(p.k + (int64_t)t * A::kKeys * a.k_token, p.v + (int64_t)t * A::kKeys * a.v_token, seen, k0, v0);

  // the query rows become fragments through 32 rows of the second buffers, which
  // no tile uses yet
  uint8_t* own = (wave < 2 ? k1 : v1) + (wave & 1) * (32 * A::kRowBytes);
  {
#pragma unroll
    for (int i = 0; i < 32 / kRowsPerLoad; ++i) {
      const int r = i * kRowsPerLoad + w.lane / kRowPieces;
      *reinterpret_cast<u32x4*>(own + r * A::kRowBytes + ((piece ^ k_swizzle<DP>(r)) << 4)) =
          8 * piece < a.dim ? qrow[i] : u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int st = 0; st < A::kSteps; ++st)
      w.q[st] = as_bf16x8(*reinterpret_cast<const u32x4*>(
          own + w.col * A::kRowBytes + (((2 * st + w.half) ^ k_swizzle<DP>(w.col)) << 4)));
  }

  // every wave sees the same lengths and mask, so all take the same turns and
  // meet at every barrier
#define ATTEND_TURN(kc, vc, kn, vn)                                                              \
  {                                                                                              \
    const int tn = next(t, seen_next);                                                           \
    __builtin_amdgcn_s_waitcnt(0x0070); /* vmcnt(0) lgkmcnt(0): own loads in LDS, reads done */   \
    asm volatile("s_barrier" ::: "memory"); /* everyone's are, and the other buffers are free */ \
    if (tn < last)                                                                               \
      load.issue(p.k + (int64_t)tn * A::kKeys * a.k_token,                                       \
                 p.v + (int64_t)tn * A::kKeys * a.v_token, seen_next, kn, vn);                   \
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

  const float l = halves_sum(w.sum);
  // through the wave's rows of LDS again, so that whole rows are stored
  __syncthreads();
  if (a.splits > 1) {      // unnormalised partial sums, half a row at a time, the maximum and the sum
    const int64_t slot = ((int64_t)unit * a.splits + split) * 128 + wave * 32;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int b = 0; b < A::kBlocks / 2; ++b)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x16& o = w.o[h * (A::kBlocks / 2) + b];
          *reinterpret_cast<f32x4*>(own + w.col * A::kRowBytes +
                                    (((8 * b + 2 * g + w.half) ^ k_swizzle<DP>(w.col)) << 4)) =
              f32x4{o[4 * g], o[4 * g + 1], o[4 * g + 2], o[4 * g + 3]};
        }
#pragma unroll
      for (int i = 0; i < 32 / kRowsPerLoad; ++i) {
        const int r = i * kRowsPerLoad + w.lane / kRowPieces;
        *reinterpret_cast<f32x4*>(a.part + (slot + r) * DP + h * (DP / 2) + 4 * piece) =
            *reinterpret_cast<const f32x4*>(own + r * A::kRowBytes + ((piece ^ k_swizzle<DP>(r)) << 4));
      }
    }
    if (w.half == 0) a.stats[slot + w.col] = float2{w.top, l};
    return;
  }
  // no key seen, or scores of -infinity alone: zeros, whatever 0 times their values left
  const uint32_t any = l == 0.0f ? 0u : ~0u;
  const float inv = 1.0f / l;
#pragma unroll
  for (int b = 0; b < A::kBlocks; ++b)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      *reinterpret_cast<u32x2*>(own + w.col * A::kRowBytes + (((4 * b + g) ^ k_swizzle<DP>(w.col)) << 4) +
                                8 * w.half) =
          u32x2{bf16x2_rne(w.o[b][4 * g] * inv, w.o[b][4 * g + 1] * inv) & any,
                bf16x2_rne(w.o[b][4 * g + 2] * inv, w.o[b][4 * g + 3] * inv) & any};
  uint16_t* out = a.out + p.batch * a.o_batch + 8 * piece;
  RowStep step(a, p, row0 + w.lane / kRowPieces, kRowsPerLoad, a.o_token, a.o_head);
#pragma unroll
  for (int i = 0; i < 32 / kRowsPerLoad; ++i, step.next()) {
    const int r = i * kRowsPerLoad + w.lane / kRowPieces;
    const u32x4 f =
        *reinterpret_cast<const u32x4*>(own + r * A::kRowBytes + ((piece ^ k_swizzle<DP>(r)) << 4));
    if (step.row < rows && 8 * piece < a.dim)
      __builtin_nontemporal_store(f, reinterpret_cast<u32x4*>(out + step.at));
  }
}

// Few query rows (at most 32 per kv head: single tokens): a workgroup's four
// waves have the same rows and every fourth tile of 32 keys each, so no wave
// waits for another; they are joined at the end.  What is left is the stream of
// keys and values, whole rows at a time into LDS of the wave's own: the next tile's
// K is on its way as soon as this one's fragments are read, its V as soon as this
// one's products are.  They are read once and streamed past the caches (134 MB of
// keys and values: 26 us against 29, 268 MB 45 against 51, 537 MB 87 against 98; only
// what the call before left in the last-level cache is slower to read, 31 against
// 27).  A key mask's bytes are loaded in the turn that looks for the next tile, behind
// the tiles in flight, so their wait is for those too; the other waves run meanwhile:
// a mask that keeps every key takes 46 us of 268 MB, 45 without, of 134 MB 27.7 and 26.
// One token of 8 entries of 1 to 8192 keys, 24 heads over 8: 31 to 33 us and 5 for the
// join, 129 MB at 4.0 TB/s (with K fragments straight to registers, 32 bytes of 32
// rows an access: 41 and 5; in tiles that the waves share, as above, 48 in all).
// What is left is the first loads' latency, with nothing to hide it, and the end, when
// workgroups run out one by one.
template <int DP>
__global__ __launch_bounds__(256, 2) void attention_few_kernel(Attention a) {
  using A = Attend<DP, 1>;
  __shared__ __attribute__((aligned(1024))) uint8_t tile_k[4 * A::kTileBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t tile_v[4 * A::kTileBytes];
  // every head's first split, then the second ones, ...
  Place p;
  const uint32_t heads = (uint32_t)a.units, split = blockIdx.x / heads, head = blockIdx.x - split * heads;
  place_head(a, p, head);
  p.keys = seen_keys(a, p);
  const int64_t rows = (int64_t)a.queries * a.group;
  const int64_t slot0 = ((int64_t)head * a.splits + split) * rows;
  const int first = (int)split * a.share * 4;    // a split is `share` groups of four tiles
  if (a.splits > 1 && first * A::kKeys >= p.keys) {        // past this entry's length
    if (threadIdx.x < rows) a.stats[slot0 + threadIdx.x] = float2{-__builtin_inff(), 0.0f};
    return;
  }
  const int wave = wave_id();
  A w;
  w.start(a.scale);
  const uint16_t* q = query_row(a, p, w.col < rows ? w.col : rows - 1);
#pragma unroll
  for (int st = 0; st < A::kSteps; ++st) {
    const int at = 16 * st + 8 * w.half;
    u32x4 f = u32x4{0u, 0u, 0u, 0u};
    if (at < a.dim) f = *reinterpret_cast<const u32x4*>(q + at);
    w.q[st] = as_bf16x8(f);
  }
  constexpr int kLoads = A::kKeys * A::kPieces / 64;
  uint32_t k_off[kLoads], v_off[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int n = i * 64 + w.lane, key = n / A::kPieces, piece = n % A::kPieces;
    const int kp = piece ^ k_swizzle<DP>(key), vp = piece ^ v_swizzle<DP>(key);
    k_off[i] = 8 * kp < a.dim ? (uint32_t)(key * a.k_token * 2 + kp * 16) : kNoData;
    v_off[i] = 8 * vp < a.dim ? (uint32_t)(key * a.v_token * 2 + vp * 16) : kNoData;
  }
  const int last = min(first + a.share * 4, (p.keys + A::kKeys - 1) / A::kKeys);
  auto next = [&](int t, uint64_t& seen) {
    for (t += 4; t < last; t += 4)
      if ((seen = seen_from<32>(p, t * A::kKeys, w.lane)) != 0) break;
    return t;
  };
  // the rows of a tile from `from` on, `by` offsets of the lane's pieces; keys out of
  // sight load as zeros
  const int own = wave * A::kTileBytes;          // this wave's part of `tile_k` and `tile_v`
  auto load = [&](const uint16_t* from, const uint32_t (&by)[kLoads], uint64_t seen, uint8_t* lds) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int key = (i * 64 + w.lane) / A::kPieces;
      tile_load<true>(from, by[i] | (((uint32_t)(~seen >> key) & 1u) * kNoData), lds, own + i * 1024);
    }
  };
  auto load_k = [&](int t, uint64_t seen) { load(p.k + (int64_t)t * A::kKeys * a.k_token, k_off, seen, tile_k); };
  auto load_v = [&](int t, uint64_t seen) { load(p.v + (int64_t)t * A::kKeys * a.v_token, v_off, seen, tile_v); };
  uint32_t v_at[A::kBlocks];
  w.v_rows(tile_v + own, v_at);
  uint32_t k_at[A::kSteps];
  w.k_rows(tile_k + own, k_at);
  uint64_t seen = 0, seen_next = 0;
  int t = next(first + wave - 4, seen);
  if (t < last) {
    load_k(t, seen);
    load_v(t, seen);
    // the query fragments are waited for here (they came first), not in the
    // loop, where the wait would cover the loads in flight
#pragma unroll
    for (int st = 0; st < A::kSteps; ++st) asm volatile("" : "+v"(w.q[st]));
    static_assert(kLoads < 16, "the wait's count is 4 bits");
    do {
      const int tn = next(t, seen_next);
      __builtin_amdgcn_s_waitcnt(0x0F70 | kLoads);         // vmcnt: K is in, V may be on its way
      asm volatile("" ::: "memory");
      u32x4 kf[A::kSteps];
      w.k_read(k_at, kf);
      if (tn < last) load_k(tn, seen_next);
      f32x16 s[1] = {f32x16{}};
#pragma unroll
      for (int st = 0; st < A::kSteps; ++st)
        s[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(kf[st]), w.q[st], s[0], 0, 0, 0);
      w.weigh(s, seen);
      if (tn < last)
        __builtin_amdgcn_s_waitcnt(0x0F70 | kLoads);       // V is in, the next K may be on its way
      else
        __builtin_amdgcn_s_waitcnt(0x0F70);
      asm volatile("" ::: "memory");
      w.gather_in_flight(s, v_at);                         // its reads are done when it ends
      if (tn < last) load_v(tn, seen_next);
      t = tn;
      seen = seen_next;
    } while (t < last);
  }

  // the four waves' states meet in LDS, in wave order: first the maxima and sums,
  // then the outputs, half the columns at a time (32 rows x DP / 2 of each wave
  // in binary32 are what `tile_k` holds)
  float* park = reinterpret_cast<float*>(tile_k);
  float(*park_top)[32] = reinterpret_cast<float(*)[32]>(tile_v);
  float(*park_sum)[32] = park_top + 4;
  float *all_top = park_top[8], *all_sum = park_top[9];
  const float l = halves_sum(w.sum);
  __syncthreads();
  if (w.half == 0) {
    park_top[wave][w.col] = w.top;
    park_sum[wave][w.col] = l;
  }
  __syncthreads();
  float top = -__builtin_inff(), sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (park_sum[i][w.col] != 0.0f) top = __builtin_fmaxf(top, park_top[i][w.col]);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (park_sum[i][w.col] != 0.0f)
      sum = __builtin_fmaf(park_sum[i][w.col], __builtin_amdgcn_exp2f(park_top[i][w.col] - top), sum);
  const float mine = l == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(w.top - top);
  if (wave == 0 && w.half == 0) {
    all_top[w.col] = top;
    all_sum[w.col] = sum;
  }
  const int here = (int)rows;                    // at most 32
  constexpr int kPart = DP / 2;
  for (int part = 0; part < 2; ++part) {
    if (w.col < here) {
#pragma unroll
      for (int b = 0; b < A::kBlocks; ++b) {
        if (b / (A::kBlocks / 2) != part) continue;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          f32x4 v = f32x4{};
          if (l != 0.0f)
            v = f32x4{w.o[b][4 * g], w.o[b][4 * g + 1], w.o[b][4 * g + 2], w.o[b][4 * g + 3]} * mine;
          *reinterpret_cast<f32x4*>(park + (wave * 32 + w.col) * kPart + 32 * (b % (A::kBlocks / 2)) +
                                    8 * g + 4 * w.half) = v;
        }
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < here * (kPart / 4); e += 256) {
      const int r = e / (kPart / 4), d = (e % (kPart / 4)) * 4, col = part * kPart + d;
      f32x4 s = f32x4{};
#pragma unroll
      for (int i = 0; i < 4; ++i) s += *reinterpret_cast<const f32x4*>(park + (i * 32 + r) * kPart + d);
      const float total = all_sum[r];
      if (a.splits > 1) {
        const int64_t slot = slot0 + r;
        *reinterpret_cast<f32x4*>(a.part + slot * DP + col) = s;
        if (col == 0) a.stats[slot] = float2{all_top[r], total};
      } else if (col < a.dim) {
        const float inv = total == 0.0f ? 0.0f : 1.0f / total;
        *reinterpret_cast<u32x2*>(output_row(a, p, r) + col) =
            u32x2{bf16x2_rne(s[0] * inv, s[1] * inv), bf16x2_rne(s[2] * inv, s[3] * inv)};
      }
    }
    __syncthreads();
  }
}

// Joins the splits of a row, DP / 4 lanes a row: partial sums weighted by
// 2^(their maximum - the largest), in split order.  Lane n of a row's holds the
// maxima and sums of splits n, n + DP / 4, ... (64 in all).  A unit has
// `unit_rows` rows' slots a split.
template <int DP>
__global__ __launch_bounds__(256) void attention_join_kernel(Attention a, int unit_rows) {
  constexpr int G = DP / 4, kRows = 64 / G, kHeld = 64 / G;
  const int lane = threadIdx.x & 63, sub = lane % G, base = lane - sub;
  const int64_t rows = unit_rows, all = a.units * rows;
  const int64_t n = ((int64_t)blockIdx.x * 4 + wave_id()) * kRows + lane / G, at = min(n, all - 1);
  const uint32_t unit = (uint32_t)(at / rows), in = (uint32_t)(at - unit * rows);
  Place p;
  int64_t row = in;
  if (a.row_tiles == 0) {                        // few rows: a unit is a head
    place_head(a, p, unit);
  } else {
    place_unit(a, p, unit);
    row += (int64_t)p.row_tile * 128;
  }
  const bool live = n < all && row < (int64_t)a.queries * a.group;
  const int64_t first = (int64_t)unit * a.splits * rows + in;
  float2 st[kHeld];
  float top = -__builtin_inff();
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    const int s = j * G + sub;
    st[j] = s < a.splits ? a.stats[first + s * rows] : float2{0.0f, 0.0f};
    if (st[j].y != 0.0f) top = __builtin_fmaxf(top, st[j].x);
  }
#pragma unroll
  for (int off = G / 2; off >= 1; off >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, off, 64));
  // -1: saw no key, what it left is not used.  A weight of 0 is used: a split of
  // NaN scores has no maximum to count with, and one far below the others' may hold
  // NaN or infinite values.
  float weight[kHeld], l = 0.0f;
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    weight[j] = st[j].y != 0.0f ? __builtin_amdgcn_exp2f(st[j].x - top) : -1.0f;
    if (!(weight[j] < 0.0f)) l = __builtin_fmaf(st[j].y, weight[j], l);
  }
#pragma unroll
  for (int off = G / 2; off >= 1; off >>= 1) l += __shfl_xor(l, off, 64);
  f32x4 o = f32x4{};
  constexpr int U = 8;                           // loads in flight
#pragma unroll
  for (int j = 0; j < kHeld; ++j)
    for (int s0 = j * G; s0 < min(a.splits, (j + 1) * G); s0 += U) {
      f32x4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        v[u] = *reinterpret_cast<const f32x4*>(a.part + (first + min(s0 + u, a.splits - 1) * rows) * DP + 4 * sub);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float f = __shfl(weight[j], base + (s0 + u) % G, 64);
        if (s0 + u < a.splits && !(f < 0.0f)) o += v[u] * f;
      }
    }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  if (live && 4 * sub < a.dim)
    *reinterpret_cast<u32x2*>(output_row(a, p, row) + 4 * sub) =
        u32x2{bf16x2_rne(o[0] * inv, o[1] * inv), bf16x2_rne(o[2] * inv, o[3] * inv)};
}

constexpr int64_t kMaxSplits = 64;               // what the join's lanes hold

// How a call is run.
//   few: at most 32 rows per kv head, the kernel whose waves share the rows.  Its
// splits are of a fixed number of keys, so entries of unequal lengths cost their
// own keys only: enough for four workgroups a compute unit, each at least 256
// keys.
//   Otherwise units of 128 rows, whose keys are split where the units leave compute
// units without work and splitting costs less than it saves, by `split_cost`.
struct Plan {
  bool few;
  int64_t row_tiles, units, slots;               // slots: rows of partial sums in the workspace
  int splits, share;
};

// Microseconds of `units` units of `tiles` 64-key tiles in s splits: a tile takes a
// workgroup t1 alone on its compute unit, t2 beside another (1.17 and 1.65 at a
// padded head size of 128, 0.85 and 1.15 at 64); splits add a launch, about 5, and
// their partial sums' way to memory and back at 4.6 TB/s.  Measured, whole against
// split, 24 heads of 128: 512 queries of 512 keys 14 against 21 (2 ways), of 2304 45
// against 32 (4 ways), of 4608 84 against 47; 1024 queries of 2304 47 against 49 (2
// ways), of 4608 89 against 80; 128 queries of 16384 keys 296 against 55 (16 ways).
double split_cost(int64_t units, int64_t tiles, int dp, int64_t s, int64_t cus) {
  const double t1 = dp == 64 ? 0.85 : 1.17, t2 = dp == 64 ? 1.15 : 1.65;
  const int64_t full = units * s / (2 * cus), rest = units * s % (2 * cus);
  const double rounds = full * t2 + (rest > cus ? t2 : rest > 0 ? t1 : 0.0);
  const double cost = rounds * (double)((tiles + s - 1) / s);
  return s == 1 ? cost : cost + 5.0 + (double)(units * s) * 128 * dp * 4 * 2 / 4.6e6;
}

Plan plan_for(int64_t batch, int64_t kv_heads, int64_t rows, int64_t keys, int dp) {
  const int64_t heads = batch * kv_heads;
  if (rows <= 32) {
    const int64_t groups = (keys + 127) / 128;           // of four tiles of 32
    int64_t share = groups * heads / (4 * compute_units());
    if (share < 2) share = 2;
    if (share < (groups + kMaxSplits - 1) / kMaxSplits) share = (groups + kMaxSplits - 1) / kMaxSplits;
    const int64_t splits = groups > 0 ? (groups + share - 1) / share : 1;
    return {true, 0, heads, heads * splits * rows, (int)splits, (int)share};
  }
  const int64_t row_tiles = (rows + 127) / 128, units = heads * row_tiles, tiles = (keys + 63) / 64;
  const int64_t cus = compute_units();
  int64_t splits = 1;
  if (units <= 2 * cus) {
    double least = split_cost(units, tiles, dp, 1, cus);
    for (int64_t s : {2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64}) {
      if (s > tiles || s > kMaxSplits) break;
      const double cost = split_cost(units, tiles, dp, s, cus);
      if (cost < least) {
        least = cost;
        splits = s;
      }
    }
  }
  return {false, row_tiles, units, units * splits * 128, (int)splits, 0};
}

// Head sizes are padded to one of two: at 4096 queries and 4608 keys of 16 heads 64
// takes 97 us, 128 150, and what lies between the time of 128 (72 to 96: 138 to 144,
// 112 and 120: 155 to 159), though 80 has 0.63 of its products.
int padded_dim(int64_t dim) { return dim <= 64 ? 64 : 128; }

}  // namespace

size_t attention_workspace_bytes(int64_t batch, int64_t queries, int64_t keys, int64_t heads,
                                 int64_t kv_heads, int64_t dim) {
  if (batch == 0 || queries == 0) return 0;
  const int dp = padded_dim(dim);
  const Plan plan = plan_for(batch, kv_heads, queries * (heads / kv_heads), keys, dp);
  return plan.splits == 1 ? 0 : (size_t)plan.slots * (dp * 4 + 8);
}

hipError_t launch_attention(Attention a, void* workspace, size_t workspace_bytes,
                            hipStream_t stream) {
  const int64_t rows = (int64_t)a.queries * a.group;
  const int dp = padded_dim(a.dim);
  Plan plan = plan_for(a.batch, a.kv_heads, rows, a.keys, dp);
  if (plan.splits > 1 && (!workspace || workspace_bytes < (size_t)plan.slots * (dp * 4 + 8))) {
    plan.share *= plan.splits;
    plan.splits = 1;
  }
  a.row_tiles = plan.row_tiles;
  a.units = plan.units;
  a.splits = plan.splits;
  a.share = plan.share;
  if (plan.splits > 1) {
    a.part = static_cast<float*>(workspace);
    a.stats = reinterpret_cast<float2*>(a.part + plan.slots * dp);
  }
  const dim3 grid((unsigned)(plan.units * plan.splits)), block(256);
  if (plan.few)
    dp == 64 ? attention_few_kernel<64><<<grid, block, 0, stream>>>(a)
             : attention_few_kernel<128><<<grid, block, 0, stream>>>(a);
  else
    dp == 64 ? attention_kernel<64><<<grid, block, 0, stream>>>(a)
             : attention_kernel<128><<<grid, block, 0, stream>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || plan.splits == 1) return e;
  const int unit_rows = plan.few ? (int)rows : 128;
  const int per = 4 * 64 / (dp / 4);             // rows a workgroup of the join has
  const dim3 join((unsigned)((plan.units * unit_rows + per - 1) / per));
  dp == 64 ? attention_join_kernel<64><<<join, block, 0, stream>>>(a, unit_rows)
           : attention_join_kernel<128><<<join, block, 0, stream>>>(a, unit_rows);
  return hipGetLastError();
}

}  // namespace nvfp4
