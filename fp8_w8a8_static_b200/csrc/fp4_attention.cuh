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
// order (no atomics: the result does not depend on timing).
#pragma once

#include "common.cuh"
#include "elementwise.cuh"
#include "fp4_kv.cuh"

namespace fp8ws {

constexpr int kKvRowWarps = 4;
constexpr int kKvRowThreads = kKvRowWarps * 32;
constexpr int kKvChunk = 64;     // tokens of a unit
constexpr int kKvStages = 2;     // ring slots of a warp, up to 4 strips each
constexpr int kKvMaxBlocks = 444;  // ranges at most: 148 SMs x 3 blocks
// p = 2^(s - m) may exceed 1 by this many powers of two before the running
// maximum m is moved: FP16 holds 2^15, the sums are fp32
constexpr float kKvSlack = 10.0f;

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

// Units (64-token chunks, one at least so that rows without tokens are
// written too) of a request's row tiles over all heads.
template <int ROWS>
__device__ __forceinline__ int64_t kv_units(const KvAttnArgs &a, int b, int &tiles, int &chunks) {
  const KvRequest r = kv_request(a, b);
  tiles = static_cast<int>((static_cast<int64_t>(r.q_len) * a.group + ROWS - 1) / ROWS);
  chunks = max(1, (r.kv + kKvChunk - 1) / kKvChunk);
  return static_cast<int64_t>(tiles) * a.cache.heads * chunks;
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

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// One row's output, D values spread over the threads: y[d] = o[d] * by.
__device__ __forceinline__ void kv_store(const KvAttnArgs &a, int64_t at, float v) {
  if (a.s_out)
    static_cast<uint8_t *>(a.out)[at] = static_cast<uint8_t>(cvt_e4m3x2(v, 0.0f));
  else
    static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(v);
}

template <int D, int NT>
struct KvRowsCfg {
  static constexpr int ROWS = 8 * NT;
  static constexpr int STAGE = 4 * strip_bytes(D);
  static constexpr int RING = kKvRowWarps * kKvStages * STAGE;
  static constexpr int MERGE = kKvRowWarps * ROWS * (D + 2) * 4;  // laid over the ring
  static constexpr int SMEM = (RING > MERGE ? RING : MERGE) + 128;
};

template <int D, int NT>
__global__ void __launch_bounds__(kKvRowThreads, 3)
    fp4_kv_rows_kernel(const KvAttnArgs a, uint64_t timeout_ns) {
  using C = KvRowsCfg<D, NT>;
  constexpr int ROWS = C::ROWS;
  constexpr int KB = D / 8;    // code bytes of a row that a thread holds (K), D/8 elements of V
  constexpr int TILES = D / 16;  // K steps of the first product, 16-row tiles of the second
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full[kKvRowWarps][kKvStages];
  __shared__ int abort_flag;
  __shared__ int64_t s_first[3];  // units before request b0; in all; b0
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t = lane % 4;  // fragment coordinates

  if (lane == 0) {
    for (int s = 0; s < kKvStages; ++s) mbar_init(&full[warp][s], 1);
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
    const int64_t per = (all + gridDim.x - 1) / gridDim.x;
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
  const int64_t per = (all + gridDim.x - 1) / gridDim.x;
  const int64_t begin = per * blockIdx.x;
  const int64_t end = min(begin + per, all);
  if (threadIdx.x == 0) a.meta[blockIdx.x] = make_int4(-1, 0, 0, 0);

  uint8_t *ring = smem + warp * kKvStages * C::STAGE;
  uint32_t phase = 0;  // bit per slot
  const float c2 = a.scale * 1.4426950408889634f * __ldg(a.s_k);
  const float out_by = a.s_out ? __ldg(a.s_v) / __ldg(a.s_out) : __ldg(a.s_v);
  bool ok = true;

  int b = static_cast<int>(s_first[2]);
  int64_t before = s_first[0];
  for (int64_t u = begin; u < end && b < a.batch;) {
    // ---------------------------------------------- the segment that u lies in
    int tiles, chunks;
    int64_t units = kv_units<ROWS>(a, b, tiles, chunks);
    while (u >= before + units && b + 1 < a.batch) {
      before += units;
      units = kv_units<ROWS>(a, ++b, tiles, chunks);
    }
    if (u >= before + units) break;  // the lengths changed under the kernel
    const KvRequest req = kv_request(a, b);
    const int64_t seg = (u - before) / chunks;  // head-major over (head, row tile)
    const int64_t seg_begin = before + seg * chunks;
    const int k0 = static_cast<int>(u - seg_begin);
    const int k1 = static_cast<int>(min(end - seg_begin, static_cast<int64_t>(chunks)));
    const int head = static_cast<int>(seg / tiles), tile = static_cast<int>(seg % tiles);
    const int row0 = tile * ROWS;
    const int rows = min(ROWS, req.q_len * a.group - row0);
    const int32_t *table = a.table + static_cast<int64_t>(b) * a.width;

    // Q of row 8n + g, this thread's elements, as FP16 of q 2^-e with 2^e the
    // row's magnitude (exact but for elements below 2^-24 of the largest)
    uint32_t qf[NT][TILES][2];
    float cq[NT][2];  // 2^e c2 of this thread's two columns (rows 8n + 2t, + 1)
    int lim[NT][2];
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
        lim[n][y] = rr < rows ? kv_limit(req, (row0 + rr) / a.group, a.causal) : 0;
      }
    }

    float o[NT][TILES][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int x = 0; x < TILES; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) o[n][x][y] = 0.0f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.0f;
    }

    // -------------------------------------------------- this warp's strips
    const int strip0 = k0 * (kKvChunk / kStripTokens);
    const int strip1 = min(k1 * (kKvChunk / kStripTokens), (req.kv + kStripTokens - 1) / kStripTokens);
    const int n_strips = max(strip1 - strip0, 0);
    // strips of a step: few of them are spread over the warps
    const int S = n_strips >= 4 * kKvRowWarps ? 4 : (n_strips >= 2 * kKvRowWarps ? 2 : 1);
    const int steps = (n_strips + S * kKvRowWarps - 1) / (S * kKvRowWarps);
    // lane l < S looks up the page of strip l of a step
    auto page_of = [&](int step) -> int {
      const int strip = strip0 + (step * kKvRowWarps + warp) * S + lane;
      if (step >= steps || lane >= S || strip >= strip1) return -1;
      return table[(strip * kStripTokens) >> a.cache.page_shift];
    };
    // starts the copies of a step's strips; returns which of them exist
    auto fetch = [&](int step, int page) -> uint32_t {
      const bool there = page >= 0 && page < a.cache.pages;
      const uint32_t mask = __ballot_sync(0xFFFFFFFFu, there);
      const int slot = step % kKvStages;
      if (lane == 0 && mask)
        mbar_arrive_expect_tx(&full[warp][slot], __popc(mask) * strip_bytes(D));
      __syncwarp();
      if (there) {
        const int strip = strip0 + (step * kKvRowWarps + warp) * S + lane;
        const int in_page = strip & ((1 << (a.cache.page_shift - 4)) - 1);
        const uint8_t *src =
            a.cache.data +
            (((static_cast<int64_t>(page) * a.cache.heads + head) << (a.cache.page_shift - 4)) +
             in_page) *
                strip_bytes(D);
        bulk_load_1d(ring + slot * C::STAGE + lane * strip_bytes(D), src, strip_bytes(D),
                     &full[warp][slot], l2_policy_evict_first());
      }
      return mask;
    };
    uint32_t masks[kKvStages];
    int next_page = page_of(0);
#pragma unroll
    for (int s = 0; s < kKvStages; ++s) {
      masks[s] = s < steps ? fetch(s, next_page) : 0;
      next_page = page_of(s + 1);
    }
    for (int step = 0; step < steps && ok; ++step) {
      const int slot = step % kKvStages;
      uint32_t mask = masks[0];
#pragma unroll
      for (int s = 1; s < kKvStages; ++s)
        if (slot == s) mask = masks[s];
      if (mask) {
        if (!mbar_wait_bounded_warp(&full[warp][slot], (phase >> slot) & 1u, &abort_flag,
                                    timeout_ns)) {
          if (lane == 0) {
            record_timeout(kSiteKvRows);
            *const_cast<volatile int *>(&abort_flag) = 1;
          }
          ok = false;
          break;
        }
        phase ^= 1u << slot;
      }
      const int first = strip0 + (step * kKvRowWarps + warp) * S;
#pragma unroll 1
      for (int i = 0; i < S; ++i) {
        if (!(mask >> i & 1u)) continue;
        const uint8_t *strip = ring + slot * C::STAGE + i * strip_bytes(D);
        const int tok0 = (first + i) * kStripTokens;
        // ---------------------------------------------- S^T = K Q^T
        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
        {
          uint32_t kw[2][KB / 4];  // codes of rows g and g + 8
          uint32_t ks[2];          // their scales, FP16 (two where a thread spans two groups)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = g + 8 * h;
            if constexpr (D == 128) {
              const uint4 w = *reinterpret_cast<const uint4 *>(strip + row * 64 + 16 * t);
              kw[h][0] = w.x;
              kw[h][1] = w.y;
              kw[h][2] = w.z;
              kw[h][3] = w.w;
              ks[h] = cvt_f16_e4m3x2(
                  *reinterpret_cast<const uint16_t *>(strip + strip_ks(D) + row * 8 + 2 * t));
            } else {
              const uint2 w = *reinterpret_cast<const uint2 *>(strip + row * 32 + 8 * t);
              kw[h][0] = w.x;
              kw[h][1] = w.y;
              ks[h] = cvt_f16_e4m3x2(strip[strip_ks(D) + row * 4 + t]);
            }
          }
#pragma unroll
          for (int x = 0; x < KB / 4; ++x) {
            // scale of this word's 8 elements, in both halves
            const uint32_t sel = (D == 128 && x >= 2) ? 0x3232u : 0x1010u;
            const uint32_t s0 = __byte_perm(ks[0], 0, sel), s1 = __byte_perm(ks[1], 0, sel);
            uint32_t h0[4], h1[4];
            cvt_f16_e2m1x8(kw[0][x], h0);
            cvt_f16_e2m1x8(kw[1][x], h1);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              h0[y] = mul_f16x2(h0[y], s0);
              h1[y] = mul_f16x2(h1[y], s1);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma_f16(s[n], h0[0], h1[0], h0[1], h1[1], qf[n][2 * x][0], qf[n][2 * x][1]);
              mma_f16(s[n], h0[2], h1[2], h0[3], h1[3], qf[n][2 * x + 1][0], qf[n][2 * x + 1][1]);
            }
          }
        }
        // ---------------------------------------------- softmax of the 16 tokens
        uint32_t p[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int tok = tok0 + g + 8 * (y >> 1);
            s[n][y] = tok < lim[n][y & 1] ? s[n][y] * cq[n][y & 1] : -INFINITY;
          }
          const bool over = s[n][0] > m[n][0] + kKvSlack || s[n][2] > m[n][0] + kKvSlack ||
                            s[n][1] > m[n][1] + kKvSlack || s[n][3] > m[n][1] + kKvSlack;
          if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              float top = fmaxf(s[n][y], s[n][y + 2]);
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
              const float now = fmaxf(m[n][y], top);
              const float by = now == -INFINITY ? 1.0f : ex2_approx(m[n][y] - now);
              m[n][y] = now;
              l[n][y] *= by;
#pragma unroll
              for (int x = 0; x < TILES; ++x) {
                o[n][x][y] *= by;
                o[n][x][y + 2] *= by;
              }
            }
          }
          const float m0 = m[n][0] == -INFINITY ? 0.0f : m[n][0];
          const float m1 = m[n][1] == -INFINITY ? 0.0f : m[n][1];
          const float p0 = ex2_approx(s[n][0] - m0), p1 = ex2_approx(s[n][1] - m1);
          const float p2 = ex2_approx(s[n][2] - m0), p3 = ex2_approx(s[n][3] - m1);
          l[n][0] += p0 + p2;
          l[n][1] += p1 + p3;
          // P is rounded to FP16 (2^-11 of each weight) for the second product
          p[n][0] = transpose_8x8(pack_f16(p0, p1));
          p[n][1] = transpose_8x8(pack_f16(p2, p3));
        }
        // ---------------------------------------------- O^T += V^T P^T
        {
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
            // places past the last token hold anything, a NaN scale too
            if (tok0 + row >= req.kv) sc[h] = 0;
          }
          const uint32_t s0 = cvt_f16_e4m3x2(sc[0] | sc[1] << 8);
          const uint32_t s1 = cvt_f16_e4m3x2(sc[2] | sc[3] << 8);
#pragma unroll
          for (int x = 0; x < KB / 8; ++x) {
            // bytes of (token, token + 1) for even and for odd elements
            const uint32_t e0 = (vw[0][x] & 0x0F0F0F0Fu) | (vw[1][x] << 4 & 0xF0F0F0F0u);
            const uint32_t d0 = (vw[0][x] >> 4 & 0x0F0F0F0Fu) | (vw[1][x] & 0xF0F0F0F0u);
            const uint32_t e1 = (vw[2][x] & 0x0F0F0F0Fu) | (vw[3][x] << 4 & 0xF0F0F0F0u);
            const uint32_t d1 = (vw[2][x] >> 4 & 0x0F0F0F0Fu) | (vw[3][x] & 0xF0F0F0F0u);
            uint32_t he0[4], hd0[4], he1[4], hd1[4];
            cvt_f16_e2m1x8(e0, he0);
            cvt_f16_e2m1x8(d0, hd0);
            cvt_f16_e2m1x8(e1, he1);
            cvt_f16_e2m1x8(d1, hd1);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const uint32_t a0 = mul_f16x2(he0[y], s0), a1 = mul_f16x2(hd0[y], s0);
              const uint32_t a2 = mul_f16x2(he1[y], s1), a3 = mul_f16x2(hd1[y], s1);
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma_f16(o[n][4 * x + y], a0, a1, a2, a3, p[n][0], p[n][1]);
            }
          }
        }
      }
      __syncwarp();  // the slot is read: it may be filled again
      const uint32_t fresh = step + kKvStages < steps ? fetch(step + kKvStages, next_page) : 0;
#pragma unroll
      for (int s = 0; s < kKvStages; ++s)
        if (slot == s) masks[s] = fresh;
      next_page = page_of(step + kKvStages + 1);
    }
    if (!ok) {  // copies in flight land before the block goes on to leave
      int zero = 0;
      for (int s = 0; s < kKvStages; ++s) {
        bool pending = false;
#pragma unroll
        for (int z = 0; z < kKvStages; ++z)
          if (z == s) pending = masks[z] != 0;
        if (pending) mbar_wait_bounded_warp(&full[warp][s], (phase >> s) & 1u, &zero, timeout_ns);
      }
    }

    // ---------------------------------------------- the four warps' sums
    float *mo = reinterpret_cast<float *>(smem);  // [warp][row][D]
    float *ml = mo + kKvRowWarps * ROWS * D;      // [warp][row][2]
    __syncthreads();  // every warp is done with its ring
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[n][y] += __shfl_xor_sync(0xFFFFFFFFu, l[n][y], d);
        const int row = warp * ROWS + 8 * n + 2 * t + y;
        if (g == 0) {
          ml[2 * row] = m[n][y];
          ml[2 * row + 1] = l[n][y];
        }
#pragma unroll
        for (int x = 0; x < TILES; ++x)
          *reinterpret_cast<float2 *>(mo + row * D + g * (D / 8) + 2 * x) =
              make_float2(o[n][x][y], o[n][x][y + 2]);
      }
    }
    __syncthreads();
    const bool whole = k0 == 0 && k1 == chunks;
    // partial sums: slot 2c for the segment that block c's range starts in,
    // 2c + 1 for one that starts inside the range
    const int64_t piece = 2 * static_cast<int64_t>(blockIdx.x) + (u == begin ? 0 : 1);
    float *pml = a.part + 2 * static_cast<int64_t>(gridDim.x) * ROWS * D;
    for (int x = threadIdx.x; x < rows * D; x += kKvRowThreads) {
      const int row = x / D, d = x % D;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kKvRowWarps; ++w) top = fmaxf(top, ml[2 * (w * ROWS + row)]);
      const float base = top == -INFINITY ? 0.0f : top;
      float sum = 0.0f, val = 0.0f;
#pragma unroll
      for (int w = 0; w < kKvRowWarps; ++w) {
        const float by = ex2_approx(ml[2 * (w * ROWS + row)] - base);
        sum += by * ml[2 * (w * ROWS + row) + 1];
        val += by * mo[(w * ROWS + row) * D + d];
      }
      if (whole) {
        const int i = (row0 + row) / a.group;
        const int64_t at = (static_cast<int64_t>(req.q0 + i) * a.cache.heads + head) * a.group +
                           (row0 + row) % a.group;
        kv_store(a, at * D + d, sum != 0.0f ? val / sum * out_by : 0.0f);
        if (a.lse && d == 0) a.lse[at] = (top + log2f(sum)) * 0.6931471805599453f;
      } else {
        a.part[(piece * ROWS + row) * D + d] = val;
        if (d == 0) {
          pml[2 * (piece * ROWS + row)] = top;
          pml[2 * (piece * ROWS + row) + 1] = sum;
        }
      }
    }
    fence_async_shared();  // the sums above lie where copies will land next
    __syncthreads();
    // The first boundary inside a segment is where it is merged: block c,
    // whose range starts inside the segment, if block c - 1's did not.
    if (!whole && u == begin && k0 > 0 && threadIdx.x == 0) {
      const int64_t first_block = seg_begin / per;
      if (first_block == static_cast<int64_t>(blockIdx.x) - 1) {
        const int64_t last_block = (seg_begin + chunks - 1) / per;
        const int head_piece = seg_begin == first_block * per ? 0 : 1;
        a.meta[blockIdx.x] =
            make_int4(b, head, tile * 2 + head_piece, static_cast<int>(last_block));
      }
    }
    u = seg_begin + k1;
  }
}

// Adds the partial sums of a segment that several blocks worked on, in block
// order.  Block c merges the segment whose first block is c - 1.
template <int D, int NT>
__global__ void __launch_bounds__(D) fp4_kv_merge_kernel(const KvAttnArgs a, int blocks) {
  constexpr int ROWS = 8 * NT;
  pdl_launch_dependents();
  pdl_wait();
  const int4 w = a.meta[blockIdx.x + 1];
  if (w.x < 0) return;
  const int first = static_cast<int>(blockIdx.x), last = w.w;
  const int head = w.y, row0 = (w.z >> 1) * ROWS;
  const KvRequest req = kv_request(a, w.x);
  const int rows = min(ROWS, req.q_len * a.group - row0);
  const float *pml = a.part + 2 * static_cast<int64_t>(blocks) * ROWS * D;
  const float out_by = a.s_out ? __ldg(a.s_v) / __ldg(a.s_out) : __ldg(a.s_v);
  for (int row = 0; row < rows; ++row) {
    float top = -INFINITY, sum = 0.0f, val = 0.0f;
    for (int c = first; c <= last; ++c) {
      const int64_t at = (2 * static_cast<int64_t>(c) + (c == first ? (w.z & 1) : 0)) * ROWS + row;
      const float m = pml[2 * at], l = pml[2 * at + 1], v = a.part[at * D + threadIdx.x];
      const float now = fmaxf(top, m);
      const float base = now == -INFINITY ? 0.0f : now;
      const float x = ex2_approx(top - base), y = ex2_approx(m - base);
      sum = sum * x + l * y;
      val = val * x + v * y;
      top = now;
    }
    const int i = (row0 + row) / a.group;
    const int64_t at = (static_cast<int64_t>(req.q0 + i) * a.cache.heads + head) * a.group +
                       (row0 + row) % a.group;
    kv_store(a, at * D + threadIdx.x, sum != 0.0f ? val / sum * out_by : 0.0f);
    if (a.lse && threadIdx.x == 0) a.lse[at] = (top + log2f(sum)) * 0.6931471805599453f;
  }
}

}  // namespace fp8ws
