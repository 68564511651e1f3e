// Attention over the 4-bit paged K/V cache (fp4_kv.cuh), for sm_100a.
//
//   o[i,h] = sum_j softmax_j( scale q[i,h] . k[j] ) v[j],   lse[i,h] = log sum_j exp(scale q . k[j])
//
// over the tokens j < kv_len of the row's request, with the causal mask
// j <= kv_len - q_len + i for row i of the request's q_len rows.  G query heads
// share a K/V head; a request's rows of one K/V head are its q_len x G pairs.
//
// fp4_kv_rows_kernel: few rows per K/V head (single tokens).  Bound by the
// cache's bytes, so every byte is read once and all of the arithmetic has to
// fit beside the stream: codes go from shared memory to registers, to FP16 by
// one conversion a pair, times their scale (exact), and into mma.m16n8k16
// with the TOKENS as the 16 rows and the query rows as the 8 columns, so that
// 1 to 8 query rows waste no more than the unused columns:
//   S^T [16 tokens, 8] = K [16, D] Q^T,   O^T [D, 8] += V^T [D, 16] P^T
// The order of a product's inner index is free: a thread takes for its K
// elements whatever 16 bytes lie together in its row, and Q is loaded to match.
// For V the two nibbles that share a byte are two d of one token; two tokens'
// words are interleaved to bytes that hold one d of both, which the conversion
// turns into the pair that the second product wants.  P^T is S^T's fragment
// transposed (movmatrix).
// The work is cut evenly: the (request, row tile, head, 64-token chunk) units
// of the whole batch form one sequence, and block c takes the c-th of equal
// ranges, whatever the lengths.  A (request, row tile, head) that ends up in
// several ranges leaves partial sums, which fp4_kv_merge_kernel adds in range
// order (no atomics: the result does not depend on timing).  Measured: 6 requests
// of 30 to 131 thousand tokens, 32 query heads on 4 K/V heads of 128: 67 us (299
// MB, 4.5 TB/s; 74 before the masks went to the edges, 92 with one warp filling a
// ring for the other four); 48 requests of 17 to 6000 tokens, 24 heads on 8: 44 us
// (3.9 TB/s); one of 1001 tokens: 9.5 us.  Some 10 us are the search for the
// range, the first copies and the merge; beside the stream it is the conversions
// (two cycles of the ALU pipe each) that fill the issue slots.
#pragma once

#include "common.cuh"
#include "elementwise.cuh"
#include "fp4_kv.cuh"

#include <type_traits>

namespace fp8ws {

constexpr int kKvRowWarps = 4;
constexpr int kKvRowThreads = kKvRowWarps * 32;
constexpr int kKvChunk = 64;     // tokens of a unit
constexpr int kKvSlots = 3;      // ring slots of a warp, up to 2 strips each
constexpr int kKvMaxBlocks = 444;  // ranges at most: 148 SMs x 3 blocks
// Blocks of an SM: 16 query rows take the registers of two (168 spill).
__host__ __device__ constexpr int kv_blocks_per_sm(int NT) { return NT == 1 ? 3 : 2; }
// A weight is 2^(s - m + kKvLift), m the running maximum in log2 units, and m is
// moved when a weight would pass 2^kKvTop, FP16's last whole power (the sums are
// fp32).  The lift is room below for the small weights of a long tail: FP16 rounds
// to half of 2^-10 down to 2^-14 and to half of 2^-24 below, so a weight is off by
// 2^-11 of itself down to 2^-23 of the largest one, and by 2^-34 of the largest one
// below.  The rest is room above, for maxima that move seldom: lifts of 0, 5 and 9
// take the same time (2048 rows behind 8192 tokens and 1266 behind 4226: 273 us),
// 11 takes 277 and 13 takes 297.
constexpr float kKvTop = 15.0f;
constexpr float kKvLift = 9.0f;

__device__ __forceinline__ uint32_t scaled(uint32_t h, __half2 s) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&h), s);
  return *reinterpret_cast<const uint32_t *>(&r);
}

struct KvAttnArgs {
  const uint16_t *q;
  int total_q;
  int batch;
  int group;  // query heads per K/V head
  const int32_t *cu_q;
  const int32_t *kv_lens;
  const int32_t *table;
  int64_t width;
  KvCache cache;
  const float *s_k;
  const float *s_v;
  float scale;
  int causal;
  int splits;    // of fp4_kv_tiles_kernel's tokens
  int few_rows;  // requests of more rows (tokens x group) are fp4_kv_tiles_kernel's
  const float *s_out;  // null: BF16 output
  void *out;
  float *lse;  // may be null
  float *part;  // [2 * blocks][rows][D] partial sums, then [2 * blocks][rows][2] maxima and sums
  int4 *meta;   // [blocks] see fp4_kv_rows_kernel
};

// A request's rows and tokens, bounded by what the buffers hold.
struct KvRequest {
  int q0, q_len, kv;
};
__device__ __forceinline__ KvRequest kv_request(const KvAttnArgs &a, int b) {
  const int lo = min(max(a.cu_q[b], 0), a.total_q);
  const int hi = min(max(a.cu_q[b + 1], lo), a.total_q);
  const int64_t cap = a.width << a.cache.page_shift;
  const int kv = static_cast<int>(min(static_cast<int64_t>(max(a.kv_lens[b], 0)), cap));
  return KvRequest{lo, hi - lo, kv};
}

// Tokens that row i of a request sees: the first `limit` ones.
__device__ __forceinline__ int kv_limit(const KvRequest &r, int i, int causal) {
  if (i >= r.q_len) return 0;
  return causal ? min(max(r.kv - r.q_len + i + 1, 0), r.kv) : r.kv;
}

// What a segment costs beside its chunks (its queries' loads, the warps' sums),
// in chunks: with ranges cut by chunks alone, the blocks that got many short
// requests ended last (48 requests of 17 to 6000 tokens: 57 us with 2, 45 with 6,
// 48 with 12).
constexpr int kKvSegmentCost = 6;

// Units of a block at least: a range costs its piece in the merge, too (one
// request of 8000 tokens, 4 heads: 19.6 us with 1, 16.0 with 4).
constexpr int kKvLeastUnits = 4;
__device__ __forceinline__ int64_t kv_range(int64_t all) {
  return max((all + gridDim.x - 1) / gridDim.x, static_cast<int64_t>(kKvLeastUnits));
}

// Units of a request's row tiles over all heads: 64-token chunks (one at
// least, so that rows without tokens are written too) and the fixed cost,
// whose units come first.
template <int ROWS>
__device__ __forceinline__ int64_t kv_units(const KvAttnArgs &a, int b, int &tiles, int &chunks) {
  const KvRequest r = kv_request(a, b);
  const int rows = r.q_len * a.group;
  tiles = rows <= a.few_rows ? (rows + ROWS - 1) / ROWS : 0;
  chunks = max(1, (r.kv + kKvChunk - 1) / kKvChunk);
  return static_cast<int64_t>(tiles) * a.cache.heads * (chunks + kKvSegmentCost);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// (a & 0x0F0F0F0F) | (b & 0xF0F0F0F0)
__device__ __forceinline__ uint32_t low_high_nibbles(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xCA;" : "=r"(r) : "r"(0x0F0F0F0Fu), "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Four neighbouring values of a row's output.
__device__ __forceinline__ void kv_store4(const KvAttnArgs &a, int64_t at, float4 v) {
  if (a.s_out) {
    *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(a.out) + at) =
        pack4(cvt_e4m3x2(v.x, v.y), cvt_e4m3x2(v.z, v.w));
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) = make_uint2(
        *reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
  }
}

template <int D, int NT>
struct KvRowsCfg {
  static constexpr int ROWS = 8 * NT;
  static constexpr int SLOT = 2 * strip_bytes(D);
  static constexpr int RING = kKvRowWarps * kKvSlots * SLOT;
  static constexpr int MERGE = kKvRowWarps * ROWS * (D + 2) * 4;
  static constexpr int SMEM = RING + MERGE;
};

// One part of a block's range: units [k0, k1) of a (request, head, row tile).
struct KvSegment {
  KvRequest req;
  int64_t begin;  // its first unit in the whole sequence
  int64_t first;  // the first one of the part
  int b, head, tile, tiles, chunks, k0, k1;
  int strip0, strip1;  // the strips of [k0, k1) that hold tokens
  int per_slot;        // strips of a ring slot: few of them are spread over the warps
};

// Walks a block's range segment by segment; its warps walk it alike.
template <int ROWS>
struct KvWalk {
  const KvAttnArgs &a;
  int64_t u, end, before;
  int b;

  // The next part with a chunk in it (a range may end in a segment's fixed cost).
  __device__ bool next(KvSegment &s) {
    do {
      if (!step(s)) return false;
    } while (s.k1 <= s.k0);
    return true;
  }

  __device__ bool step(KvSegment &s) {
    if (u >= end || b >= a.batch) return false;
    int64_t units = kv_units<ROWS>(a, b, s.tiles, s.chunks);
    while (u >= before + units && b + 1 < a.batch) {
      before += units;
      units = kv_units<ROWS>(a, ++b, s.tiles, s.chunks);
    }
    if (u >= before + units) return false;  // the lengths changed under the kernel
    const int cost = s.chunks + kKvSegmentCost;
    // head-major over (head, row tile); 32 bits but for absurd sizes
    const int64_t seg = units <= INT32_MAX ? static_cast<int>(u - before) / cost
                                           : (u - before) / cost;
    s.req = kv_request(a, b);
    s.b = b;
    s.begin = before + seg * cost;
    s.first = u;
    s.k0 = max(static_cast<int>(u - s.begin) - kKvSegmentCost, 0);
    s.k1 = static_cast<int>(min(end - s.begin, static_cast<int64_t>(cost))) - kKvSegmentCost;
    s.head = static_cast<int>(units <= INT32_MAX ? static_cast<int>(seg) / s.tiles : seg / s.tiles);
    s.tile = static_cast<int>(seg - static_cast<int64_t>(s.head) * s.tiles);
    constexpr int per_chunk = kKvChunk / kStripTokens;
    s.strip0 = s.k0 * per_chunk;
    s.strip1 = max(s.strip0, min(s.k1 * per_chunk, (s.req.kv + kStripTokens - 1) / kStripTokens));
    s.per_slot = s.strip1 - s.strip0 >= 2 * kKvRowWarps ? 2 : 1;
    u = s.begin + s.k1 + kKvSegmentCost;
    return true;
  }
};

template <int D, int NT>
__global__ void __launch_bounds__(kKvRowThreads, kv_blocks_per_sm(NT))
    fp4_kv_rows_kernel(const KvAttnArgs a, uint64_t timeout_ns) {
  using C = KvRowsCfg<D, NT>;
  constexpr int ROWS = C::ROWS;
  constexpr int KB = D / 8;    // code bytes of a row that a thread holds (K), D/8 elements of V
  constexpr int TILES = D / 16;  // K steps of the first product, 16-row tiles of the second
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full[kKvRowWarps][kKvSlots];
  __shared__ int abort_flag;
  __shared__ int64_t s_first[3];  // units before request b0; in all; b0
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t = lane % 4;  // fragment coordinates

  if (lane == 0) {
    for (int s = 0; s < kKvSlots; ++s) mbar_init(&full[warp][s], 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) abort_flag = 0;
  pdl_launch_dependents();
  pdl_wait();

  // this block's range of units, and the request that it starts in
  if (warp == 0) {
    int tiles, chunks;
    int64_t all = 0;
    for (int b = lane; b < a.batch; b += 32) all += kv_units<ROWS>(a, b, tiles, chunks);
#pragma unroll
    for (int d = 16; d; d >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, d);
    const int64_t per = kv_range(all);
    const int64_t begin = per * blockIdx.x;
    int64_t before = 0;
    int b0 = 0;
    if (begin < all) {
      for (; b0 < a.batch; b0 += 32) {
        const int b = b0 + lane;
        int64_t n = b < a.batch ? kv_units<ROWS>(a, b, tiles, chunks) : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int64_t m = __shfl_up_sync(0xFFFFFFFFu, n, d);
          if (lane >= d) n += m;
        }
        const uint32_t past = __ballot_sync(0xFFFFFFFFu, before + n > begin);
        if (past) {
          const int src = __ffs(past) - 1;
          const int64_t upto = __shfl_sync(0xFFFFFFFFu, n, src > 0 ? src - 1 : 0);
          if (src > 0) before += upto;
          b0 += src;
          break;
        }
        before += __shfl_sync(0xFFFFFFFFu, n, 31);
      }
    }
    if (lane == 0) {
      s_first[0] = before;
      s_first[1] = all;
      s_first[2] = b0;
    }
  }
  __syncthreads();
  const int64_t all = s_first[1];
  const int64_t per = kv_range(all);
  const int64_t begin = per * blockIdx.x;
  KvWalk<ROWS> walk{a, begin, min(begin + per, all), s_first[0], static_cast<int>(s_first[2])};
  if (threadIdx.x == 0) a.meta[blockIdx.x] = make_int4(-1, 0, 0, 0);

  // The warp's ring.  Step n of a part is its strips strip0 + (n x 4 + warp) x S,
  // S = per_slot; lanes 2k and 2k + 1 look up, for 16 steps at a time, the pages
  // of step k's strips and start their copies.
  uint8_t *ring = smem + warp * kKvSlots * C::SLOT;
  const uint64_t policy = l2_policy_evict_first();
  const uint8_t *src = nullptr;  // this lane's strip
  bool there = false;
  uint32_t exist = 0;     // lanes whose strip is there
  uint32_t present = 0;   // two bits a slot: the strips that were copied
  int put = 0, take = 0;  // next slot to fill and to read
  uint32_t phase = 0;     // of the slots to be read, a bit each
  int in_flight = 0;
  auto fetch = [&](const KvSegment &s, int step) {
    const int k = step % 16;
    if (k == 0) {
      const int strip = s.strip0 + ((step + lane / 2) * kKvRowWarps + warp) * s.per_slot + (lane & 1);
      int page = -1;
      if ((lane & 1) < s.per_slot && strip < s.strip1)
        page = a.table[static_cast<int64_t>(s.b) * a.width +
                       ((strip * kStripTokens) >> a.cache.page_shift)];
      there = page >= 0 && page < a.cache.pages;
      exist = __ballot_sync(0xFFFFFFFFu, there);
      src = a.cache.data + (((static_cast<int64_t>(there ? page : 0) * a.cache.heads + s.head)
                             << (a.cache.page_shift - 4)) +
                            (strip & ((1 << (a.cache.page_shift - 4)) - 1))) *
                               strip_bytes(D);
    }
    const uint32_t mask = exist >> (2 * k) & 3u;
    if (lane == 0) mbar_arrive_expect_tx(&full[warp][put], __popc(mask) * strip_bytes(D));
    __syncwarp();
    if (lane / 2 == k && there)
      bulk_load_1d(ring + put * C::SLOT + (lane & 1) * strip_bytes(D), src, strip_bytes(D),
                   &full[warp][put], policy);
    present = (present & ~(3u << (2 * put))) | mask << (2 * put);
    put = put == kKvSlots - 1 ? 0 : put + 1;
    ++in_flight;
  };
  auto steps_of = [&](const KvSegment &s) {
    const int mine = s.strip1 - s.strip0 - warp * s.per_slot;  // strips from the first one on
    return mine <= 0 ? 0 : (mine - 1) / (kKvRowWarps * s.per_slot) + 1;
  };
  auto prime = [&](const KvSegment &s) {
    const int steps = steps_of(s);
    for (int n = 0; n < kKvSlots && n < steps; ++n) fetch(s, n);
  };

  float *mo = reinterpret_cast<float *>(smem + C::RING);  // [warp][row][D]
  float *ml = mo + kKvRowWarps * ROWS * D;                // [warp][row][2]
  const float c2 = a.scale * 1.4426950408889634f * __ldg(a.s_k);
  const float out_by = a.s_out ? __ldg(a.s_v) / __ldg(a.s_out) : __ldg(a.s_v);
  bool ok = true;
  KvSegment seg, after;
  bool more = walk.next(seg);
  if (more) prime(seg);
  for (; more; seg = after) {
    const KvRequest req = seg.req;
    const int head = seg.head;
    const int row0 = seg.tile * ROWS;
    const int rows = min(ROWS, req.q_len * a.group - row0);

    // Q of row 8n + g, this thread's elements, as FP16 of q 2^-e with 2^e the
    // row's magnitude: BF16 has 8 significant bits and FP16's smallest step is 2^-24,
    // so it is exact down to 2^-17 of the largest and off by 2^-25 of it below
    uint32_t qf[NT][TILES][2];
    float cq[NT][2];  // 2^e c2 of this thread's two columns (rows 8n + 2t, + 1)
    int lim[NT][2];   // tokens that they see
    int all_see = req.kv;  // tokens that every row of the tile sees
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = 8 * n + g;
      uint32_t raw[D / 8];
      if (r < rows) {
        const int i = (row0 + r) / a.group;
        const int64_t at =
            (static_cast<int64_t>(req.q0 + i) * a.cache.heads + head) * a.group + (row0 + r) % a.group;
        const uint4 *src = reinterpret_cast<const uint4 *>(a.q + at * D + t * (D / 4));
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
          const uint4 w = __ldg(src + x);
          raw[4 * x] = w.x;
          raw[4 * x + 1] = w.y;
          raw[4 * x + 2] = w.z;
          raw[4 * x + 3] = w.w;
        }
      } else {
#pragma unroll
        for (int x = 0; x < D / 8; ++x) raw[x] = 0;
      }
      uint32_t top = 0;  // the largest magnitude's bits
#pragma unroll
      for (int x = 0; x < D / 8; ++x)
        top = max(top, max(raw[x] & 0x7FFFu, (raw[x] >> 16) & 0x7FFFu));
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      const int e = top == 0 ? 0 : min(max(static_cast<int>(top >> 7) - 127, -126), 126);
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
      for (int x = 0; x < TILES; ++x) {
#pragma unroll
        for (int y = 0; y < 2; ++y)
          qf[n][x][y] = pack_f16(bf16_lo(raw[2 * x + y]) * down, bf16_hi(raw[2 * x + y]) * down);
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int col = 2 * t + y;  // held by the four lanes of fragment row `col`
        const int ec = __shfl_sync(0xFFFFFFFFu, e, col * 4);
        cq[n][y] = c2 * __uint_as_float(static_cast<uint32_t>(127 + ec) << 23);
        const int rr = 8 * n + col;
        // columns without a row (their q is 0) see what there is
        lim[n][y] = rr < rows ? kv_limit(req, (row0 + rr) / a.group, a.causal) : req.kv;
        all_see = min(all_see, lim[n][y]);
      }
    }
    all_see = min(all_see, __shfl_xor_sync(0xFFFFFFFFu, all_see, 1));
    all_see = min(all_see, __shfl_xor_sync(0xFFFFFFFFu, all_see, 2));

    float o[NT][TILES][4];
    float neg_m[NT][2], l[NT][2];  // kKvLift - m, the sums of the weights
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int x = 0; x < TILES; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) o[n][x][y] = 0.0f;
      neg_m[n][0] = neg_m[n][1] = INFINITY;
      l[n][0] = l[n][1] = 0.0f;
    }

    // NS neighbouring strips of shared memory at once (the second one's
    // arithmetic fills the first one's waits)
    // EDGE: some row does not see all of the tokens.
    auto multiply = [&](auto ns, auto at_edge, const uint8_t *strips, int tok0) {
      constexpr int NS = decltype(ns)::value;
      constexpr bool EDGE = decltype(at_edge)::value;
      // ---------------------------------------------- S^T = K Q^T
      float s[NS][NT][4];
#pragma unroll
      for (int z = 0; z < NS; ++z) {
        const uint8_t *strip = strips + z * strip_bytes(D);
#pragma unroll
        for (int n = 0; n < NT; ++n) s[z][n][0] = s[z][n][1] = s[z][n][2] = s[z][n][3] = 0.0f;
        uint32_t kw[2][KB / 4];  // codes of rows g and g + 8
        __half2 ks[2];           // their scales (two where a thread spans two groups)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = g + 8 * h;
          uint32_t sc;
          if constexpr (D == 128) {
            const uint4 w = *reinterpret_cast<const uint4 *>(strip + row * 64 + 16 * t);
            kw[h][0] = w.x;
            kw[h][1] = w.y;
            kw[h][2] = w.z;
            kw[h][3] = w.w;
            sc = cvt_f16_e4m3x2(
                *reinterpret_cast<const uint16_t *>(strip + strip_ks(D) + row * 8 + 2 * t));
          } else {
            const uint2 w = *reinterpret_cast<const uint2 *>(strip + row * 32 + 8 * t);
            kw[h][0] = w.x;
            kw[h][1] = w.y;
            sc = cvt_f16_e4m3x2(strip[strip_ks(D) + row * 4 + t]);
          }
          ks[h] = *reinterpret_cast<const __half2 *>(&sc);
        }
#pragma unroll
        for (int x = 0; x < KB / 4; ++x) {
          // scale of this word's 8 elements, in both halves
          const bool second = D == 128 && x >= 2;
          const __half2 s0 = second ? __high2half2(ks[0]) : __low2half2(ks[0]);
          const __half2 s1 = second ? __high2half2(ks[1]) : __low2half2(ks[1]);
          uint32_t h0[4], h1[4];
          cvt_f16_e2m1x8(kw[0][x], h0);
          cvt_f16_e2m1x8(kw[1][x], h1);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            h0[y] = scaled(h0[y], s0);
            h1[y] = scaled(h1[y], s1);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_f16(s[z][n], h0[0], h1[0], h0[1], h1[1], qf[n][2 * x][0], qf[n][2 * x][1]);
            mma_f16(s[z][n], h0[2], h1[2], h0[3], h1[3], qf[n][2 * x + 1][0], qf[n][2 * x + 1][1]);
          }
        }
      }
      // ---------------------------------------------- softmax
      uint32_t p[NS][NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float e[NS][4];  // log2 of the weights
        auto exponents = [&] {
#pragma unroll
          for (int z = 0; z < NS; ++z)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              e[z][y] = fmaf(s[z][n][y], cq[n][y & 1], neg_m[n][y & 1]);
              if (EDGE && tok0 + z * kStripTokens + g + 8 * (y >> 1) >= lim[n][y & 1])
                e[z][y] = -INFINITY;
            }
        };
        exponents();
        float top[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          top[y] = fmaxf(e[0][y], e[0][y + 2]);
#pragma unroll
          for (int z = 1; z < NS; ++z) top[y] = fmaxf(top[y], fmaxf(e[z][y], e[z][y + 2]));
        }
        if (__any_sync(0xFFFFFFFFu, fmaxf(top[0], top[1]) > kKvTop)) {
          // move the maxima (at first from -inf) to the largest scores
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            top[y] = neg_m[n][y];
            neg_m[n][y] = 0.0f;  // the scores themselves
          }
          exponents();
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float old = top[y];
            float now = kKvLift - old;
#pragma unroll
            for (int z = 0; z < NS; ++z) now = fmaxf(now, fmaxf(e[z][y], e[z][y + 2]));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1)
              now = fmaxf(now, __shfl_xor_sync(0xFFFFFFFFu, now, d));
            // nothing seen yet: sums and maximum stay as they are
            neg_m[n][y] = now == -INFINITY ? INFINITY : kKvLift - now;
            const float by = now == -INFINITY ? 1.0f : ex2_approx(neg_m[n][y] - old);
            l[n][y] *= by;
#pragma unroll
            for (int x = 0; x < TILES; ++x) {
              o[n][x][y] *= by;
              o[n][x][y + 2] *= by;
            }
          }
          exponents();
        }
#pragma unroll
        for (int z = 0; z < NS; ++z) {
#pragma unroll
          for (int y = 0; y < 4; ++y) e[z][y] = ex2_approx(e[z][y]);
          l[n][0] += e[z][0] + e[z][2];
          l[n][1] += e[z][1] + e[z][3];
          // P is rounded to FP16 (see kKvLift) for the second product
          p[z][n][0] = transpose_8x8(pack_f16(e[z][0], e[z][1]));
          p[z][n][1] = transpose_8x8(pack_f16(e[z][2], e[z][3]));
        }
      }
      // ---------------------------------------------- O^T += V^T P^T
#pragma unroll
      for (int z = 0; z < NS; ++z) {
        const uint8_t *strip = strips + z * strip_bytes(D);
        const uint8_t *vc = strip + strip_v(D), *vs = strip + strip_vs(D);
        uint32_t vw[4][KB / 8];  // tokens 2t, 2t + 1, 2t + 8, 2t + 9: D/8 elements
        uint32_t sc[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int row = 2 * t + (h & 1) + 8 * (h >> 1);
          if constexpr (D == 128) {
            const uint2 w = *reinterpret_cast<const uint2 *>(vc + row * 64 + 8 * g);
            vw[h][0] = w.x;
            vw[h][1] = w.y;
            sc[h] = vs[row * 8 + g];
          } else {
            vw[h][0] = *reinterpret_cast<const uint32_t *>(vc + row * 32 + 4 * g);
            sc[h] = vs[row * 4 + g / 2];
          }
        }
        if (EDGE) {
          // places past the last token hold anything, a NaN scale too
#pragma unroll
          for (int h = 0; h < 4; ++h)
            if (tok0 + z * kStripTokens + 2 * t + (h & 1) + 8 * (h >> 1) >= req.kv) sc[h] = 0;
        }
        const uint32_t s0 = cvt_f16_e4m3x2(__byte_perm(sc[0], sc[1], 0x0040));
        const uint32_t s1 = cvt_f16_e4m3x2(__byte_perm(sc[2], sc[3], 0x0040));
#pragma unroll
        for (int x = 0; x < KB / 8; ++x) {
          // bytes of (token, token + 1) for even and for odd elements
          uint32_t he0[4], hd0[4], he1[4], hd1[4];
          cvt_f16_e2m1x8(low_high_nibbles(vw[0][x], vw[1][x] << 4), he0);
          cvt_f16_e2m1x8(low_high_nibbles(vw[0][x] >> 4, vw[1][x]), hd0);
          cvt_f16_e2m1x8(low_high_nibbles(vw[2][x], vw[3][x] << 4), he1);
          cvt_f16_e2m1x8(low_high_nibbles(vw[2][x] >> 4, vw[3][x]), hd1);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const uint32_t a0 = mul_f16x2(he0[y], s0), a1 = mul_f16x2(hd0[y], s0);
            const uint32_t a2 = mul_f16x2(he1[y], s1), a3 = mul_f16x2(hd1[y], s1);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma_f16(o[n][4 * x + y], a0, a1, a2, a3, p[z][n][0], p[z][n][1]);
          }
        }
      }
    };

    const int S = seg.per_slot, steps = steps_of(seg);
    for (int step = 0; step < steps && ok; ++step) {
      if (!mbar_wait_polled_warp(&full[warp][take], phase >> take & 1u, &abort_flag, timeout_ns)) {
        if (lane == 0) {
          record_timeout(kSiteKvRows);
          *const_cast<volatile int *>(&abort_flag) = 1;
        }
        ok = false;
        break;
      }
      const uint32_t mask = present >> (2 * take) & 3u;
      const uint8_t *at = ring + take * C::SLOT;
      const int tok0 = (seg.strip0 + (step * kKvRowWarps + warp) * S) * kStripTokens;
      // two strips at once, but for 16 rows of 128, whose sums take the registers
      constexpr int NS = NT * D <= 128 ? 2 : 1;
      if (mask == (NS == 2 ? 3u : mask) && tok0 + 2 * kStripTokens <= all_see) {
#pragma unroll 1
        for (int x = 0; x < 2; x += NS)
          if (mask >> x & 1u)
            multiply(std::integral_constant<int, NS>{}, std::false_type{},
                     at + x * strip_bytes(D), tok0 + x * kStripTokens);
      } else {
#pragma unroll 1
        for (int x = 0; x < 2; ++x)
          if (mask >> x & 1u)
            multiply(std::integral_constant<int, 1>{}, std::true_type{}, at + x * strip_bytes(D),
                     tok0 + x * kStripTokens);
      }
      phase ^= 1u << take;
      take = take == kKvSlots - 1 ? 0 : take + 1;
      --in_flight;
      __syncwarp();  // the slot is read: it may be filled again
      if (step + kKvSlots < steps) fetch(seg, step + kKvSlots);
    }

    // ---------------------------------------------- the four warps' sums
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[n][y] += __shfl_xor_sync(0xFFFFFFFFu, l[n][y], d);
        const int row = warp * ROWS + 8 * n + 2 * t + y;
        if (g == 0) {
          ml[2 * row] = -neg_m[n][y];
          ml[2 * row + 1] = l[n][y];
        }
#pragma unroll
        for (int x = 0; x < TILES; ++x)
          *reinterpret_cast<float2 *>(mo + row * D + g * (D / 8) + 2 * x) =
              make_float2(o[n][x][y], o[n][x][y + 2]);
      }
    }
    // the next part's first copies run during the rest of this one
    more = walk.next(after);
    if (more && ok) prime(after);
    __syncthreads();
    const bool whole = seg.k0 == 0 && seg.k1 == seg.chunks;
    // partial sums: slot 2c for the segment that block c's range starts in,
    // 2c + 1 for one that starts inside the range
    const int64_t piece = 2 * static_cast<int64_t>(blockIdx.x) + (seg.first == begin ? 0 : 1);
    float *pml = a.part + 2 * static_cast<int64_t>(gridDim.x) * ROWS * D;
    for (int x = threadIdx.x; x < rows * (D / 4); x += kKvRowThreads) {
      const int row = x / (D / 4), d = 4 * (x % (D / 4));
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kKvRowWarps; ++w) top = fmaxf(top, ml[2 * (w * ROWS + row)]);
      const float base = top == -INFINITY ? 0.0f : top;
      float sum = 0.0f;
      float4 val = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kKvRowWarps; ++w) {
        const float by = ex2_approx(ml[2 * (w * ROWS + row)] - base);
        const float4 v = *reinterpret_cast<const float4 *>(mo + (w * ROWS + row) * D + d);
        sum += by * ml[2 * (w * ROWS + row) + 1];
        val.x += by * v.x;
        val.y += by * v.y;
        val.z += by * v.z;
        val.w += by * v.w;
      }
      if (whole) {
        const int i = (row0 + row) / a.group;
        const int64_t at = (static_cast<int64_t>(req.q0 + i) * a.cache.heads + head) * a.group +
                           (row0 + row) % a.group;
        const float by = sum != 0.0f ? out_by / sum : 0.0f;
        kv_store4(a, at * D + d, make_float4(val.x * by, val.y * by, val.z * by, val.w * by));
        if (a.lse && d == 0) a.lse[at] = (top + log2f(sum)) * 0.6931471805599453f;
      } else {
        *reinterpret_cast<float4 *>(a.part + (piece * ROWS + row) * D + d) = val;
        if (d == 0) {
          pml[2 * (piece * ROWS + row)] = top;
          pml[2 * (piece * ROWS + row) + 1] = sum;
        }
      }
    }
    __syncthreads();  // the sums are read: they may be overwritten
    // The first boundary inside a segment is where it is merged: block c,
    // whose range starts inside the segment, if block c - 1's did not.
    if (!whole && seg.first == begin && seg.k0 > 0 && threadIdx.x == 0) {
      const int64_t first_block = (seg.begin + kKvSegmentCost) / per;
      if (first_block == static_cast<int64_t>(blockIdx.x) - 1) {
        const int64_t last_block = (seg.begin + kKvSegmentCost + seg.chunks - 1) / per;
        const int head_piece = seg.begin <= first_block * per ? 0 : 1;
        a.meta[blockIdx.x] =
            make_int4(seg.b, head, seg.tile * 2 + head_piece, static_cast<int>(last_block));
      }
    }
  }
  // after a wait that ran out: copies in flight land before the block ends
  for (int zero = 0; in_flight > 0; --in_flight) {
    mbar_wait_polled_warp(&full[warp][take], phase >> take & 1u, &zero, timeout_ns);
    phase ^= 1u << take;
    take = take == kKvSlots - 1 ? 0 : take + 1;
  }
}

// Adds the partial sums of a segment that several blocks worked on, in block
// order.  Block c merges the segment whose first block is c - 1.  All latency:
// a thread owns 4 of a row's D values and every SPLIT-th piece, whose loads do
// not depend on one another, and the shares meet in shared memory.
constexpr int kKvMergeThreads = 512;

template <int D, int NT>
__global__ void __launch_bounds__(kKvMergeThreads)
    fp4_kv_merge_kernel(const KvAttnArgs a, int blocks) {
  constexpr int ROWS = 8 * NT;
  constexpr int LANES = D / 4;
  constexpr int SPLIT = kKvMergeThreads / (ROWS * LANES);
  constexpr int RUN = 2;  // pieces of a thread in flight (more cost blocks an SM)
  __shared__ float4 s_val[SPLIT][ROWS][LANES];
  __shared__ float2 s_sum[SPLIT][ROWS];  // maximum, sum
  pdl_launch_dependents();
  pdl_wait();
  const int4 w = a.meta[blockIdx.x + 1];
  if (w.x < 0) return;
  const int first = static_cast<int>(blockIdx.x), last = w.w;
  const int head = w.y, row0 = (w.z >> 1) * ROWS;
  const KvRequest req = kv_request(a, w.x);
  const int rows = min(ROWS, req.q_len * a.group - row0);
  const int lane = threadIdx.x % LANES, row = threadIdx.x / LANES % ROWS;
  const int share = threadIdx.x / (LANES * ROWS);
  const float2 *pml = reinterpret_cast<const float2 *>(
      a.part + 2 * static_cast<int64_t>(blocks) * ROWS * D);
  float top = -INFINITY, sum = 0.0f;
  float4 val = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add = [&](float m, float l, float4 v) {
    const float now = fmaxf(top, m);
    const float base = now == -INFINITY ? 0.0f : now;
    const float x = ex2_approx(top - base), y = ex2_approx(m - base);
    sum = sum * x + l * y;
    val.x = val.x * x + v.x * y;
    val.y = val.y * x + v.y * y;
    val.z = val.z * x + v.z * y;
    val.w = val.w * x + v.w * y;
    top = now;
  };
  for (int c0 = first + share; c0 <= last; c0 += RUN * SPLIT) {
    float2 ml[RUN];
    float4 v[RUN];
#pragma unroll
    for (int x = 0; x < RUN; ++x) {
      const int c = min(c0 + x * SPLIT, last);
      // piece of block c: the first block's may be its second one
      const int64_t at =
          (2 * static_cast<int64_t>(c) + (c == first ? (w.z & 1) : 0)) * ROWS + row;
      ml[x] = pml[at];
      v[x] = *reinterpret_cast<const float4 *>(a.part + at * D + 4 * lane);
    }
#pragma unroll
    for (int x = 0; x < RUN; ++x)
      if (c0 + x * SPLIT <= last) add(ml[x].x, ml[x].y, v[x]);
  }
  s_val[share][row][lane] = val;
  if (lane == 0) s_sum[share][row] = make_float2(top, sum);
  __syncthreads();
  if (share != 0 || row >= rows) return;
#pragma unroll
  for (int x = 1; x < SPLIT; ++x)
    add(s_sum[x][row].x, s_sum[x][row].y, s_val[x][row][lane]);
  const float out_by = a.s_out ? __ldg(a.s_v) / __ldg(a.s_out) : __ldg(a.s_v);
  const float by = sum != 0.0f ? out_by / sum : 0.0f;
  const int i = (row0 + row) / a.group;
  const int64_t at = (static_cast<int64_t>(req.q0 + i) * a.cache.heads + head) * a.group +
                     (row0 + row) % a.group;
  kv_store4(a, at * D + 4 * lane,
            make_float4(val.x * by, val.y * by, val.z * by, val.w * by));
  if (a.lse && lane == 0) a.lse[at] = (top + log2f(sum)) * 0.6931471805599453f;
}

}  // namespace fp8ws
