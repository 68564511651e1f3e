// Attention over the 4-bit paged K/V cache for many query rows (prompts,
// cross-attention), on the tensor cores of sm_100a (tcgen05).
//
// The operation, the cache and the row packing are those of fp4_attention.cuh.
// A block takes 256 rows (two 128-row tiles) of one request and K/V head and
// walks the tokens that any of them sees, 64 (a chunk) at a time:
//   warp 0        copies the chunk's strips into a ring
//   warps 12..15  turn codes into FP16 once for both row tiles: K and V as
//                 [token][64 elements] 128-byte-swizzled atoms, four chunks
//                 deep.  K is read K-major, V MN-major (its inner index, the
//                 token, is the row), so both are written the same way and
//                 nothing is transposed.
//   warp 1        issues the first product, S = Q_t K^T (M = 128, N = 64) into TMEM
//   warp 2        issues the second, O_t += P_t V, P_t read from TMEM, in S's place
//   warps 4..11   softmax: four warps a row tile, a thread a row, so the maximum
//                 and the sum need no exchange; a chunk's scores stay in
//                 registers from the search for the maximum to the weights.
// Each row tile has two score buffers: while the softmax is on one chunk, the
// next one's scores are computed.  A row's maximum is moved, and its sums in TMEM
// scaled, only when a weight would pass 2^kKvTop, what FP16 holds (kKvLift).
// Where the row blocks do not fill the GPU, `splits` blocks share one's tokens
// and leave partial sums, which fp4_kv_tiles_merge_kernel adds in order.
// Bound, for 256 rows and 64 tokens: 2 x (390 + 260) cycles of the tensor pipe
// (D = 128; the first product, N = 64, is held by the reads of Q) beside 1024 of
// the special function unit (one exponential a score, 16 a cycle).  Measured
// (24 query heads on 8 K/V heads of 128, two requests, 2048 rows behind 8192 tokens
// and 1266 behind 4226): 274 us, about 2200 cycles a chunk, the rest being what the warps wait for one
// another; 45 us for 4096 rows over 1024 tokens, 64-wide heads.
// On the way, for the first of them: 350 us with chunks of 128 tokens and one score
// buffer, 315 with half of a chunk's weights handed over at a time, 320 as now but
// with each MMA issued from one thread's own registers, 283 with the issue
// warp-uniform, 278 with packed fp32 pairs in the softmax, 274 with 16-byte stores
// of FP8 output.  Ranges of tokens cut evenly over persistent blocks were slower
// (300 us): nearly every range then leaves partial sums.
#pragma once

#include "common.cuh"
#include "fp4_attention.cuh"

namespace fp8ws {

constexpr int kKvTileRows = 256;
constexpr int kKvTileSlots = 148;  // partial sums of 256 rows at most
constexpr int kKvTileThreads = 512;
constexpr int kKvChunkStrips = kKvChunk / kStripTokens;
constexpr int kKvRawSlots = 3;  // chunks of raw strips
constexpr int kKvBuffers = 4;   // chunks of K and of V in FP16
constexpr int kKvMasks = 16;    // chunks whose missing strips are remembered

template <int D>
struct KvTilesCfg {
  static constexpr int ATOMS = D / 64;  // 64-element atoms of a row
  static constexpr int Q_ATOM = 128 * 128;
  static constexpr int Q_TILE = ATOMS * Q_ATOM;  // 128 rows
  static constexpr int KV_ATOM = kKvChunk * 128;
  static constexpr int KV_TILE = ATOMS * KV_ATOM;  // 64 tokens of K or V
  static constexpr int RAW = kKvChunkStrips * strip_bytes(D);
  static constexpr int SMEM = 2 * Q_TILE + 2 * kKvBuffers * KV_TILE + kKvRawSlots * RAW + 1024;
  static constexpr int O_COL = 256;  // TMEM columns: S (two buffers of 64) of both tiles, then O
  static_assert(SMEM <= 232448, "shared memory");
};

// kind::f16 descriptor: FP16 A and B, fp32 D; B K-major or MN-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | (b_mn_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// Operand descriptors in two words.  The issuing thread shares its scheduler
// with softmax and conversion warps, so an MMA has to cost it few instructions:
// the high word is a constant, and of the low one only the start address
// (>> 4, the low 14 bits) moves, by a constant from one MMA to the next.  (With
// 64-bit descriptors put together for each MMA its issue took 160 cycles, the
// MMA itself 65.)
//   high word: 8-row groups 1024 bytes apart, version 1, 128-byte swizzle
constexpr uint32_t kDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;
// K-major: rows of 128 bytes (64 elements of the inner index).
__device__ __forceinline__ uint32_t desc_k_major(uint32_t saddr) { return saddr >> 4 | 1u << 16; }
// MN-major: rows are the inner index, 64 elements each; the next 64 elements
// lie `block` bytes on.
__device__ __forceinline__ uint32_t desc_mn_major(uint32_t saddr, uint32_t block) {
  return saddr >> 4 | block >> 4 << 16;
}

// Executed by the whole warp, issued by the lane with leader != 0: the operands
// stay warp-uniform.
template <bool ACC>
__device__ __forceinline__ void umma_f16_ss(uint32_t leader, uint32_t tmem_d, uint32_t a_low,
                                            uint32_t b_low, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %4};\n\tmov.b64 b, {%2, %4};\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 e, %6, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(a_low), "r"(b_low), "r"(idesc), "n"(kDescHigh), "n"(ACC ? 1 : 0), "r"(leader));
}

// A from TMEM: lane = row, a column holds two neighbouring elements.
__device__ __forceinline__ void umma_f16_ts(uint32_t leader, uint32_t tmem_d, uint32_t tmem_a,
                                            uint32_t b_low, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %4};\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 e, %6, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "r"(b_low), "r"(idesc), "n"(kDescHigh), "r"(accumulate), "r"(leader));
}

__device__ __forceinline__ void umma_commit_by(uint32_t leader, uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar)),
      "r"(leader)
      : "memory");
}

__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e;
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Two fp32 at a time: half the issue slots of the softmax's multiply-adds and sums.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  return pair(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  uint32_t lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
  return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, uint32_t b, uint32_t c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;"
      : "=f"(r)
      : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
  return r;
}

// 256-row blocks of request b over all heads, 0 for a request whose rows the
// other kernel takes.
__device__ __forceinline__ int64_t kv_tile_items(const KvAttnArgs &a, int b) {
  const KvRequest r = kv_request(a, b);
  const int64_t rows = static_cast<int64_t>(r.q_len) * a.group;
  if (rows <= a.few_rows) return 0;
  return (rows + kKvTileRows - 1) / kKvTileRows * a.cache.heads;
}

template <int D>
__global__ void __launch_bounds__(kKvTileThreads, 1)
    fp4_kv_tiles_kernel(const KvAttnArgs a, uint64_t timeout_ns) {
  using C = KvTilesCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *sQ = smem;                                // [2]
  uint8_t *sK = sQ + 2 * C::Q_TILE;                  // [kKvBuffers]
  uint8_t *sV = sK + kKvBuffers * C::KV_TILE;        // [kKvBuffers]
  uint8_t *sRaw = sV + kKvBuffers * C::KV_TILE;      // [kKvRawSlots]
  // S, P and the products with P: by row tile and buffer
  __shared__ __align__(8) uint64_t raw_full[kKvRawSlots], raw_empty[kKvRawSlots],
      k_full[kKvBuffers], k_empty[kKvBuffers], v_full[kKvBuffers], v_empty[kKvBuffers],
      s_full[2][2], p_full[2][2], pv_done[2][2], drain[2];
  __shared__ uint32_t missing[kKvMasks];  // strips that the cache lacks, a bit each
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  __shared__ int s_item[2];  // request (-1: none), block and head within it
  volatile int *abort_flag = &abort_word;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kKvRawSlots; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], 4);
    }
    for (int s = 0; s < kKvBuffers; ++s) {
      mbar_init(&k_full[s], 4);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 4);
      mbar_init(&v_empty[s], 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&s_full[s / 2][s % 2], 1);
      mbar_init(&p_full[s / 2][s % 2], 4);
      mbar_init(&pv_done[s / 2][s % 2], 1);
    }
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    abort_word = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  pdl_launch_dependents();
  pdl_wait();
  const int item = static_cast<int>(blockIdx.x) / a.splits;
  const int split = static_cast<int>(blockIdx.x) - item * a.splits;
  if (warp == 0) {  // this block's request
    int64_t before = 0;
    int found = -1, local = 0;
    for (int b0 = 0; b0 < a.batch && found < 0; b0 += 32) {
      const int b = b0 + lane;
      const int64_t mine = b < a.batch ? kv_tile_items(a, b) : 0;
      int64_t n = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t m = __shfl_up_sync(0xFFFFFFFFu, n, d);
        if (lane >= d) n += m;
      }
      const uint32_t past = __ballot_sync(0xFFFFFFFFu, before + n > item);
      if (past) {
        const int src = __ffs(past) - 1;
        found = b0 + src;
        local = static_cast<int>(item - (before + __shfl_sync(0xFFFFFFFFu, n - mine, src)));
      }
      before += __shfl_sync(0xFFFFFFFFu, n, 31);
    }
    if (lane == 0) {
      s_item[0] = found;
      s_item[1] = local;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int b = s_item[0];
  if (b < 0) {  // more blocks than work
    if (a.splits > 1 && split == 0 && threadIdx.x == 0) a.meta[item] = make_int4(-1, 0, 0, 0);
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, 512);
    return;
  }
  const KvRequest req = kv_request(a, b);
  const int total_rows = req.q_len * a.group;
  const int blocks = (total_rows + kKvTileRows - 1) / kKvTileRows;
  const int head = s_item[1] % a.cache.heads;
  // the last rows, which see the most tokens, come first
  const int row0 = (blocks - 1 - s_item[1] / a.cache.heads) * kKvTileRows;
  const int rows = min(kKvTileRows, total_rows - row0);
  const int row_tiles = rows > 128 ? 2 : 1;
  // tokens that some row of the block sees, and that all of them see
  const int most = kv_limit(req, (row0 + rows - 1) / a.group, a.causal);
  // this block's chunks of them
  const int all_chunks = (most + kKvChunk - 1) / kKvChunk;
  const int per_split = (all_chunks + a.splits - 1) / a.splits;
  const int chunk0 = min(split * per_split, all_chunks);
  const int chunks = min(per_split, all_chunks - chunk0);
  if (a.splits > 1 && split == 0 && threadIdx.x == 0)
    a.meta[item] = make_int4(b, head, row0, rows);

  // A wait of the whole warp, and what follows when it runs out.
  auto wait = [&](uint64_t *bar, int n) {
    if (mbar_wait_polled_warp(bar, n & 1, abort_flag, timeout_ns)) return true;
    if (lane == 0) {
      record_timeout(kSiteKvTiles);
      *abort_flag = 1;
    }
    return false;
  };

  // The issuing warps' waits; and every MMA has retired before they go on.
  auto wait_mma = [&](uint64_t *bar, int n) {
    const bool ok = wait(bar, n);
    tc_fence_after();
    return ok;
  };
  auto finish = [&](uint32_t leader, int which) {
    umma_commit_by(leader, &drain[which]);
    int zero = 0;
    if (!mbar_wait_polled_warp(&drain[which], 0, &zero, timeout_ns) && lane == 0)
      record_timeout(kSiteKvTiles);
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const int32_t *table = a.table + static_cast<int64_t>(b) * a.width;
    const int strips = min((most + kStripTokens - 1) / kStripTokens,
                           (chunk0 + chunks) * kKvChunkStrips);
    auto page_of = [&](int strip) {
      return lane < kKvChunkStrips && strip < strips
                 ? table[(strip * kStripTokens) >> a.cache.page_shift]
                 : -1;
    };
    int page = page_of(chunk0 * kKvChunkStrips + lane);
    int i = 0;
    for (; i < chunks; ++i) {
      const int slot = i % kKvRawSlots;
      if (!wait(&raw_empty[slot], i / kKvRawSlots + 1)) break;
      const int strip = (chunk0 + i) * kKvChunkStrips + lane;
      const bool there = page >= 0 && page < a.cache.pages;
      const uint32_t mask = __ballot_sync(0xFFFFFFFFu, there);
      if (lane == 0) {
        missing[i % kKvMasks] = ~mask & ((1u << kKvChunkStrips) - 1);
        mbar_arrive_expect_tx(&raw_full[slot], __popc(mask) * strip_bytes(D));
      }
      __syncwarp();
      if (there) {
        const int64_t at = ((static_cast<int64_t>(page) * a.cache.heads + head)
                            << (a.cache.page_shift - 4)) +
                           (strip & ((1 << (a.cache.page_shift - 4)) - 1));
        bulk_load_1d(sRaw + slot * C::RAW + lane * strip_bytes(D),
                     a.cache.data + at * strip_bytes(D), strip_bytes(D), &raw_full[slot],
                     l2_policy_evict_normal());
      }
      page = page_of(strip + kKvChunkStrips);
    }
    if (i < chunks) {  // copies in flight land before the block may end
      int zero = 0;
      for (int k = max(i - kKvRawSlots, 0); k < i; ++k)
        mbar_wait_polled_warp(&raw_full[k % kKvRawSlots], k / kKvRawSlots & 1, &zero, timeout_ns);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ scores
    asm volatile("bar.sync 1, 288;" ::: "memory");  // Q is there
    // (a broadcast value is known to be the same for the whole warp)
    const int n = __shfl_sync(0xFFFFFFFFu, chunks, 0);
    const int n_t = __shfl_sync(0xFFFFFFFFu, row_tiles, 0);
    const uint32_t base = __shfl_sync(0xFFFFFFFFu, tmem, 0);
    const uint32_t leader = elect_one();
    constexpr uint32_t idesc = idesc_f16_f32(128, kKvChunk, false);
    const uint32_t q_desc = desc_k_major(smem_u32(sQ)), k_desc = desc_k_major(smem_u32(sK));
    bool ok = true;
    for (int i = 0; i < n && ok; ++i) {
      const int buf = i % kKvBuffers;
      ok = wait_mma(&k_full[buf], i / kKvBuffers);
      for (int t = 0; t < n_t && ok; ++t) {  // S = Q_t K^T
        // P of two chunks before lies there
        if (i >= 2) ok = wait_mma(&pv_done[t][i & 1], (i - 2) >> 1);
        if (!ok) break;
        const uint32_t q = q_desc + t * (C::Q_TILE >> 4), k = k_desc + buf * (C::KV_TILE >> 4);
        const uint32_t d = base + t * 128 + (i & 1) * 64;
        umma_f16_ss<false>(leader, d, q, k, idesc);
#pragma unroll
        for (int x = 1; x < D / 16; ++x)
          umma_f16_ss<true>(leader, d, q + ((x / 4 * C::Q_ATOM + x % 4 * 32) >> 4),
                            k + ((x / 4 * C::KV_ATOM + x % 4 * 32) >> 4), idesc);
        umma_commit_by(leader, &s_full[t][i & 1]);
      }
      if (ok) umma_commit_by(leader, &k_empty[buf]);
    }
    finish(leader, 0);
  } else if (warp == 2) {
    // ------------------------------------------------------------ sums
    const int n = __shfl_sync(0xFFFFFFFFu, chunks, 0);
    const int n_t = __shfl_sync(0xFFFFFFFFu, row_tiles, 0);
    const uint32_t base = __shfl_sync(0xFFFFFFFFu, tmem, 0);
    const uint32_t leader = elect_one();
    constexpr uint32_t idesc = idesc_f16_f32(128, D, true);
    const uint32_t v_desc = desc_mn_major(smem_u32(sV), C::KV_ATOM);
    bool ok = true;
    for (int i = 0; i < n && ok; ++i) {
      const int buf = i % kKvBuffers;
      ok = wait_mma(&v_full[buf], i / kKvBuffers);
      for (int t = 0; t < n_t && ok; ++t) {  // O_t += P_t V
        ok = wait_mma(&p_full[t][i & 1], i >> 1);
        if (!ok) break;
        const uint32_t v = v_desc + buf * (C::KV_TILE >> 4);
        const uint32_t d = base + C::O_COL + t * 128, p = base + t * 128 + (i & 1) * 64;
#pragma unroll
        for (int x = 0; x < kKvChunk / 16; ++x)
          umma_f16_ts(leader, d, p + x * 8, v + x * (2048 >> 4), idesc, x != 0 || i != 0);
        umma_commit_by(leader, &pv_done[t][i & 1]);
      }
      if (ok) umma_commit_by(leader, &v_empty[buf]);
    }
    finish(leader, 1);
  } else if (warp >= 12) {
    // ------------------------------------------------------------ codes to FP16
    const int w = warp - 12;  // this warp's strip of a chunk
    bool ok = true;
    constexpr int LANES = D / 32;              // lanes of a row, 32 elements (16 bytes of codes) each
    constexpr int ROWS = 32 / LANES;           // rows of a round
    constexpr int ROUNDS = kStripTokens / ROWS;
    const int part = lane % LANES;
    // 32 codes and their two scales to FP16, to a row of an FP16 tile
    auto convert = [&](const uint4 &codes, uint32_t scales, uint8_t *tile, int row) {
      const uint32_t sh = cvt_f16_e4m3x2(scales);
      const __half2 s = *reinterpret_cast<const __half2 *>(&sh);
      const __half2 s0 = __low2half2(s), s1 = __high2half2(s);
      uint32_t h[4][4];
      cvt_f16_e2m1x8(codes.x, h[0]);
      cvt_f16_e2m1x8(codes.y, h[1]);
      cvt_f16_e2m1x8(codes.z, h[2]);
      cvt_f16_e2m1x8(codes.w, h[3]);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
#pragma unroll
        for (int z = 0; z < 4; ++z) h[y][z] = scaled(h[y][z], y < 2 ? s0 : s1);
      }
      // 16-byte units 4 (part % 2) + y of the row's 128 bytes in atom part / 2,
      // swizzled; the second atom's lanes go in another order, which keeps the
      // eight lanes of a store phase on eight different units
      uint8_t *to = tile + part / 2 * C::KV_ATOM + row * 128;
      const int turn = part / 2 * 2;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int unit = part % 2 * 4 + (y ^ turn);
        const uint4 v = turn ? make_uint4(h[y ^ 2][0], h[y ^ 2][1], h[y ^ 2][2], h[y ^ 2][3])
                             : make_uint4(h[y][0], h[y][1], h[y][2], h[y][3]);
        *reinterpret_cast<uint4 *>(to + ((unit ^ (row & 7)) << 4)) = v;
      }
    };
    for (int i = 0; i < chunks && ok; ++i) {
      const int slot = i % kKvRawSlots, buf = i % kKvBuffers, use = i / kKvBuffers;
      const uint8_t *strip = sRaw + slot * C::RAW + w * strip_bytes(D);
      ok = wait(&raw_full[slot], i / kKvRawSlots);
      if (!ok) break;
      const bool gone = missing[i % kKvMasks] >> w & 1u;
      uint4 kc[ROUNDS], vc[ROUNDS];
      uint32_t ks[ROUNDS], vs[ROUNDS];
#pragma unroll
      for (int x = 0; x < ROUNDS; ++x) {
        const int in = x * ROWS + lane / LANES;
        kc[x] = *reinterpret_cast<const uint4 *>(strip + in * (D / 2) + part * 16);
        vc[x] = *reinterpret_cast<const uint4 *>(strip + strip_v(D) + in * (D / 2) + part * 16);
        ks[x] = *reinterpret_cast<const uint16_t *>(strip + strip_ks(D) + in * (D / 16) + part * 2);
        vs[x] = *reinterpret_cast<const uint16_t *>(strip + strip_vs(D) + in * (D / 16) + part * 2);
        // V of tokens that are not there has to be finite: rows weigh it with 0
        if (gone || (chunk0 + i) * kKvChunk + w * kStripTokens + in >= req.kv) vs[x] = 0;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&raw_empty[slot]);
      // the products with what the buffers held before are done
      ok = wait(&k_empty[buf], use + 1) && wait(&v_empty[buf], use + 1);
      if (!ok) break;
#pragma unroll
      for (int x = 0; x < ROUNDS; ++x)
        convert(kc[x], ks[x], sK + buf * C::KV_TILE, w * kStripTokens + x * ROWS + lane / LANES);
#pragma unroll
      for (int x = 0; x < ROUNDS; ++x)
        convert(vc[x], vs[x], sV + buf * C::KV_TILE, w * kStripTokens + x * ROWS + lane / LANES);
      fence_async_shared();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&k_full[buf]);
        mbar_arrive(&v_full[buf]);
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax
    const int tile = (warp - 4) / 4, quarter = warp & 3;
    const int r = tile * 128 + quarter * 32 + lane;  // this thread's row of the block
    const bool live = r < rows;
    const int i = live ? (row0 + r) / a.group : 0;
    const int64_t at = (static_cast<int64_t>(req.q0 + i) * a.cache.heads + head) * a.group +
                       (row0 + r) % a.group;
    const int lim = live ? kv_limit(req, i, a.causal) : most;
    const float factor = a.scale * 1.4426950408889634f * __ldg(a.s_k);
    float c = 0.0f;  // scores to log2 units, never negative
    {
      uint4 q[D / 8];
      uint32_t top = 0;
#pragma unroll
      for (int x = 0; x < D / 8; ++x) {
        q[x] = live ? __ldg(reinterpret_cast<const uint4 *>(a.q + at * D) + x)
                    : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {q[x].x, q[x].y, q[x].z, q[x].w};
#pragma unroll
        for (int y = 0; y < 4; ++y) top = max(top, max(w[y] & 0x7FFFu, (w[y] >> 16) & 0x7FFFu));
      }
      const int e = top == 0 ? 0 : min(max(static_cast<int>(top >> 7) - 127, -126), 126);
      // (not 0 either: -inf, a score not seen, stays -inf)
      c = fmaxf(fabsf(factor) * __uint_as_float(static_cast<uint32_t>(127 + e) << 23), 0x1p-126f);
      const float down =
          copysignf(__uint_as_float(static_cast<uint32_t>(127 - e) << 23), factor);
      uint8_t *to = sQ + tile * C::Q_TILE + (quarter * 32 + lane) * 128;
#pragma unroll
      for (int x = 0; x < D / 8; ++x) {
        const uint4 h = make_uint4(pack_f16(bf16_lo(q[x].x) * down, bf16_hi(q[x].x) * down),
                                   pack_f16(bf16_lo(q[x].y) * down, bf16_hi(q[x].y) * down),
                                   pack_f16(bf16_lo(q[x].z) * down, bf16_hi(q[x].z) * down),
                                   pack_f16(bf16_lo(q[x].w) * down, bf16_hi(q[x].w) * down));
        *reinterpret_cast<uint4 *>(to + x / 8 * C::Q_ATOM + (((x % 8) ^ (lane & 7)) << 4)) = h;
      }
      fence_async_shared();
    }
    asm volatile("bar.sync 1, 288;" ::: "memory");  // with the warp that reads it
    const bool used = tile < row_tiles;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_o = tmem + lanes + C::O_COL + tile * 128;
    float neg_m = INFINITY, l = 0.0f;  // kKvLift - m, the sum of the weights
    bool ok = true;
    for (int i = 0; used && i < chunks; ++i) {
      ok = wait(&s_full[tile][i & 1], i >> 1);
      if (!ok) break;
      tc_fence_after();
      const uint32_t t_s = tmem + lanes + tile * 128 + (i & 1) * 64;
      uint32_t s0[32], s1[32];  // the scores of 32 tokens each
      tmem_ld_32x32b_x32(t_s, s0);
      tmem_ld_32x32b_x32(t_s + 32, s1);
      const int tok0 = (chunk0 + i) * kKvChunk;
      const uint32_t gone = missing[i % kKvMasks];
      const bool edge = __any_sync(0xFFFFFFFFu, tok0 + kKvChunk > lim) || gone != 0;
      tmem_ld_wait();
      if (edge) {  // a score that the row does not see is -inf
        auto mask = [&](uint32_t (&s)[32], int tok, uint32_t gone) {
          const int n0 = gone & 1u ? 0 : lim - tok, n1 = gone & 2u ? 0 : lim - tok;
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (x >= (x < kStripTokens ? n0 : n1)) s[x] = 0xFF800000u;
        };
        mask(s0, tok0, gone);
        mask(s1, tok0 + 32, gone >> 2);
      }
      float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int x = 0; x < 32; x += 2) {
        tops[x / 2 % 2] = max3(tops[x / 2 % 2], s0[x], s0[x + 1]);
        tops[2 + x / 2 % 2] = max3(tops[2 + x / 2 % 2], s1[x], s1[x + 1]);
      }
      const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
      const float now = top == -INFINITY ? -INFINITY : top * c;
      if (__any_sync(0xFFFFFFFFu, now + neg_m > kKvTop)) {
        // move the maxima (at first from -inf); O must not be in use
        const float next = fminf(neg_m, kKvLift - now);
        const float by = next == INFINITY ? 1.0f : ex2_approx(next - neg_m);
        neg_m = next;
        l *= by;
        if (i > 0) {
          ok = wait(&pv_done[tile][(i - 1) & 1], (i - 1) >> 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int col = 0; col < D; col += 16) {
            uint32_t o[16];
            tmem_ld_32x32b_x16(t_o + col, o);
            tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * by);
            tmem_st_32x32b_x16(t_o + col, o);
          }
        }
      }
      // a row that has seen nothing yet has no maximum: any, for weights of 0
      const float shift = neg_m == INFINITY ? 0.0f : neg_m;
      const uint64_t c2 = pair(c, c), shift2 = pair(shift, shift);
      uint64_t sums = pair(0.0f, 0.0f);
      // weights, rounded to FP16 (see kKvLift) for the second product
      auto weigh = [&](const uint32_t (&s)[32], uint32_t col) {
        uint32_t p[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const float2 v = unpair(fma2(pair(s[2 * x], s[2 * x + 1]), c2, shift2));
          const float e0 = ex2_approx(v.x), e1 = ex2_approx(v.y);
          sums = add2(sums, pair(e0, e1));
          p[x] = pack_f16(e0, e1);
        }
        tmem_st_32x32b_x16(col, p);
      };
      weigh(s0, t_s);
      weigh(s1, t_s + 16);
      l += unpair(sums).x + unpair(sums).y;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[tile][i & 1]);
    }
    if (used && ok && chunks > 0) {
      ok = wait(&pv_done[tile][(chunks - 1) & 1], (chunks - 1) >> 1);
      tc_fence_after();
    }
    if (used && ok && a.splits > 1) {  // sums as they are, [D / 4][256 rows][4]
      const int64_t slot = static_cast<int64_t>(blockIdx.x) * kKvTileRows + r;
      float *to = a.part + static_cast<int64_t>(blockIdx.x) * kKvTileRows * D + 4 * r;
#pragma unroll 1
      for (int col = 0; chunks > 0 && col < D; col += 32) {
        uint32_t o[32];
        tmem_ld_32x32b_x32(t_o + col, o);
        tmem_ld_wait();
        if (!live) continue;
#pragma unroll
        for (int x = 0; x < 32; x += 4)
          *reinterpret_cast<uint4 *>(to + (col + x) * kKvTileRows) =
              make_uint4(o[x], o[x + 1], o[x + 2], o[x + 3]);
      }
      float *ml = a.part + static_cast<int64_t>(kKvTileSlots) * kKvTileRows * D;
      if (live) *reinterpret_cast<float2 *>(ml + 2 * slot) = make_float2(-neg_m, l);
    } else if (used && ok) {
      const float s_v = a.s_out ? __ldg(a.s_v) / __ldg(a.s_out) : __ldg(a.s_v);
      const float by = l != 0.0f ? s_v / l : 0.0f;
#pragma unroll 1
      for (int col = 0; col < D; col += 32) {
        uint32_t o[32];
        if (chunks > 0) {
          tmem_ld_32x32b_x32(t_o + col, o);
          tmem_ld_wait();
        }
        float v[32];
#pragma unroll
        for (int x = 0; x < 32; ++x)
          v[x] = chunks > 0 && l != 0.0f ? __uint_as_float(o[x]) * by : 0.0f;
        if (!live) continue;
        if (a.s_out) {
          uint4 *to = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(a.out) + at * D + col);
#pragma unroll
          for (int x = 0; x < 32; x += 16) {
            uint32_t h[4];
#pragma unroll
            for (int y = 0; y < 4; ++y)
              h[y] = pack4(cvt_e4m3x2(v[x + 4 * y], v[x + 4 * y + 1]),
                           cvt_e4m3x2(v[x + 4 * y + 2], v[x + 4 * y + 3]));
            to[x / 16] = make_uint4(h[0], h[1], h[2], h[3]);
          }
        } else {
          uint4 *to = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + at * D + col);
#pragma unroll
          for (int x = 0; x < 32; x += 8) {
            uint32_t h[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const __nv_bfloat162 z = __floats2bfloat162_rn(v[x + 2 * y], v[x + 2 * y + 1]);
              h[y] = *reinterpret_cast<const uint32_t *>(&z);
            }
            to[x / 8] = make_uint4(h[0], h[1], h[2], h[3]);
          }
        }
      }
      if (a.lse && live) a.lse[at] = (log2f(l) - neg_m) * 0.6931471805599453f;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Adds the partial sums of a row block's splits, in order: 8 rows a block (16
// where D = 64), 4 of a row's values a thread.
constexpr int kKvTileMergeThreads = 256;

template <int D>
__global__ void __launch_bounds__(kKvTileMergeThreads)
    fp4_kv_tiles_merge_kernel(const KvAttnArgs a) {
  constexpr int LANES = D / 4;
  constexpr int ROWS = kKvTileMergeThreads / LANES;
  constexpr int BLOCKS = kKvTileRows / ROWS;
  pdl_launch_dependents();
  pdl_wait();
  const int item = static_cast<int>(blockIdx.x) / BLOCKS;
  const int4 w = a.meta[item];
  // neighbouring threads: the block's rows, then the next four values
  const int r = static_cast<int>(blockIdx.x) % BLOCKS * ROWS + static_cast<int>(threadIdx.x) % ROWS;
  if (w.x < 0 || r >= w.w) return;
  const int lane = threadIdx.x / ROWS;
  const float2 *ml = reinterpret_cast<const float2 *>(
      a.part + static_cast<int64_t>(kKvTileSlots) * kKvTileRows * D);
  float top = -INFINITY, sum = 0.0f;
  float4 val = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int s = 0; s < a.splits; ++s) {
    const int64_t slot = static_cast<int64_t>(item * a.splits + s) * kKvTileRows;
    const float2 p = ml[slot + r];
    const float4 v = *reinterpret_cast<const float4 *>(a.part + slot * D +
                                                       4 * (lane * kKvTileRows + r));
    // nothing seen there, and nothing written where it had no chunk; but a NaN sum counts
    if (p.x == -INFINITY && p.y == 0.0f) continue;
    const float now = fmaxf(top, p.x);
    const float base = now == -INFINITY ? 0.0f : now;
    const float x = ex2_approx(top - base), y = p.x == -INFINITY ? 1.0f : ex2_approx(p.x - base);
    sum = sum * x + p.y * y;
    val.x = val.x * x + v.x * y;
    val.y = val.y * x + v.y * y;
    val.z = val.z * x + v.z * y;
    val.w = val.w * x + v.w * y;
    top = now;
  }
  const KvRequest req = kv_request(a, w.x);
  const int i = (w.z + r) / a.group;
  const int64_t at = (static_cast<int64_t>(req.q0 + i) * a.cache.heads + w.y) * a.group +
                     (w.z + r) % a.group;
  const float out_by = a.s_out ? __ldg(a.s_v) / __ldg(a.s_out) : __ldg(a.s_v);
  const float by = sum != 0.0f ? out_by / sum : 0.0f;
  kv_store4(a, at * D + 4 * lane, make_float4(val.x * by, val.y * by, val.z * by, val.w * by));
  if (a.lse && lane == 0) a.lse[at] = (top + log2f(sum)) * 0.6931471805599453f;
}

}  // namespace fp8ws
