// The FP8 Linear with a fused epilogue (gemm_epilogue_sm100.cuh) for few rows
// (a decode step's tokens), for sm_100a.
//
// Bound by the weight's bytes: every SM has to stream a share of W from the
// first microsecond, and there is no second use of a tile.  So the WEIGHT's
// rows are the 128 rows of the MMA and the tokens its N = 32, 64 or 128 columns
// (Y^T = W X^T; an activation of 17 rows fills 17 of 32 columns instead of 17
// of 256 rows), and K is split over the S = 1, 2, 4 or 8 blocks of a cluster, so
// that N / 128 x S blocks cover the SMs (more rows than 128, where N is small,
// are further tiles).  Each block sums its K range in TMEM;
// the ranges' sums meet in shared memory across the cluster, each block
// finishing NTOK / S of the tokens: the others' shares come by bulk copies (a
// store of each lane into the other block took 0.2 us a token), it adds the S
// partial sums in rank order (the same bits every time) and applies bias,
// activation, residual and output type.  A lane is a weight row, so a warp's accesses to Y and R are 32
// neighbouring columns.
//   warp 0 TMA producer, warp 1 MMA issue and TMEM, warps 2..9 epilogue
#pragma once

#include "common.cuh"
#include "gemm_epilogue_sm100.cuh"

namespace fp8ws {

constexpr int kRowsEpiWarps = 8;
constexpr int kRowsThreads = 64 + 32 * kRowsEpiWarps;

template <int NTOK_>
struct RowsCfg {
  static constexpr int NTOK = NTOK_;
  static constexpr int W_BYTES = 128 * kGemmBK;
  static constexpr int X_BYTES = NTOK * kGemmBK;
  static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
  static constexpr int STAGES = NTOK == 32 ? 8 : (NTOK == 64 ? 6 : 4);
  static constexpr int SUM_BYTES = NTOK * 128 * 4;  // [rank][NTOK / S][128] partial sums
  static_assert(SUM_BYTES <= STAGES * STAGE_BYTES, "this block's sums take the ring's place");
  static constexpr int BAR_BYTES = 256;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + SUM_BYTES + BAR_BYTES + 1024;
  static_assert((2 * STAGES + 2) * 8 + 8 <= BAR_BYTES, "barrier area");
  static_assert(SMEM_BYTES <= 232448, "shared memory");
};

// `bytes` bytes from this block's shared memory to another block's of the
// cluster, counted on a barrier there (cluster addresses; multiples of 16).
__device__ __forceinline__ void bulk_copy_cluster(uint32_t dst, const void *src, uint32_t bytes,
                                                  uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, "
      "[%3];" ::"r"(dst),
      "r"(smem_u32(src)), "r"(bytes), "r"(bar)
      : "memory");
}

template <int NTOK>
__global__ void __launch_bounds__(kRowsThreads, 1)
    fp8_gemm_rows_kernel(const __grid_constant__ CUtensorMap tm_w,
                         const __grid_constant__ CUtensorMap tm_x, const EpilogueArgs E,
                         const uint16_t *residual, void *out, int all_rows, int N, int K,
                         int row_tiles, int kb_per_block, uint64_t timeout_ns) {
  using C = RowsCfg<NTOK>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *sW = smem;
  uint8_t *sX = sW + C::STAGES * C::W_BYTES;
  float *sums = reinterpret_cast<float *>(sX + C::STAGES * C::X_BYTES);
  uint64_t *full = reinterpret_cast<uint64_t *>(reinterpret_cast<uint8_t *>(sums) + C::SUM_BYTES);
  uint64_t *empty = full + C::STAGES;
  uint64_t *done = empty + C::STAGES;
  uint64_t *met = done + 1;  // the other blocks' sums landed
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(met + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t S;  // blocks of the cluster
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(S));
  const uint32_t rank = cluster_ctarank();
  const int tile = static_cast<int>(blockIdx.x / S);
  const int n0 = tile / row_tiles * 128, row0 = tile % row_tiles * NTOK;
  const int M = min(NTOK, all_rows - row0);  // tokens of this tile
  const int num_kb = (K + kGemmBK - 1) / kGemmBK;
  const int kb0 = static_cast<int>(rank) * kb_per_block;
  const int kb1 = min(kb0 + kb_per_block, num_kb);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    mbar_init(met, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, NTOK);
    tmem_relinquish();
  }
  pdl_launch_dependents();
  pdl_wait();  // the previous kernel's outputs (our inputs) are complete from here on
  tc_fence_before();
  cluster_sync();  // every block of the cluster runs: its shared memory may be written
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int slice = NTOK / static_cast<int>(S);  // tokens that a block finishes
  const int m0 = static_cast<int>(rank) * slice;
  const int mine = max(min(slice, M - m0), 0);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int s = it % C::STAGES;
        if (!mbar_wait_bounded(&empty[s], (it / C::STAGES & 1) ^ 1, abort_flag, timeout_ns)) {
          record_timeout(kSiteProducerEmpty);
          *abort_flag = 1;
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&full[s], C::STAGE_BYTES);
        tma_load_2d(sW + s * C::W_BYTES, &tm_w, &full[s], kb * kGemmBK, n0);
        tma_load_2d(sX + s * C::X_BYTES, &tm_x, &full[s], kb * kGemmBK, row0);
      }
      if (!ok) {  // loads in flight land before the block may end
        int zero = 0;
        for (int k = it > C::STAGES ? it - C::STAGES : 0; k < it; ++k)
          mbar_wait_bounded(&full[k % C::STAGES], k / C::STAGES & 1, &zero, timeout_ns);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_e4m3_f32(128, NTOK);
      int it = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int s = it % C::STAGES;
        if (!mbar_wait_bounded(&full[s], it / C::STAGES & 1, abort_flag, timeout_ns)) {
          record_timeout(kSiteMmaFull);
          *abort_flag = 1;
          break;
        }
        tc_fence_after();
        const uint32_t w_addr = smem_u32(sW + s * C::W_BYTES);
        const uint32_t x_addr = smem_u32(sX + s * C::X_BYTES);
#pragma unroll
        for (int k = 0; k < kGemmBK / 32; ++k)
          umma_f8(tmem, smem_desc_k_sw128(w_addr + k * 32), smem_desc_k_sw128(x_addr + k * 32),
                  idesc, (it | k) != 0 ? 1u : 0u);
        umma_commit(&empty[s]);
      }
      umma_commit(done);
      int zero = 0;
      if (!mbar_wait_bounded(done, 0, &zero, timeout_ns)) record_timeout(kSiteDrain);
    }
    __syncwarp();
  } else {
    // ------------------------------------- this block's sums to the cluster
    constexpr int RUN = 8;  // tokens of a thread at a time
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;  // weight row n0 + row
    const int n = n0 + row;
    const int count = n < N ? mine : 0;
    float *own = reinterpret_cast<float *>(smem);  // [token][128], over the ring
    if (threadIdx.x == 64 && S > 1)
      mbar_arrive_expect_tx(met, (S - 1) * static_cast<uint32_t>(mine) * 512);
    const int half = (warp - 2) >> 2;  // of two warps with the same rows
    float res[RUN];
    auto load_residual = [&](float (&res)[RUN], int x0) {
#pragma unroll
      for (int y = 0; y < RUN; ++y)
        res[y] = residual && x0 + y < count
                     ? __uint_as_float(static_cast<uint32_t>(
                                           residual[static_cast<int64_t>(row0 + m0 + x0 + y) * N + n])
                                       << 16)
                     : 0.0f;
    };
    load_residual(res, half * RUN);  // the first ones are on their way during the products
    const float scale = __ldg(E.s_in) * __ldg(E.s_w);
    const float inv_out = E.s_out ? __frcp_rn(__ldg(E.s_out)) : 1.0f;
    const float bias =
        E.bias && n < N ? __uint_as_float(static_cast<uint32_t>(__ldg(E.bias + n)) << 16) : 0.0f;
    // (`done`: every product has read the ring, so every load has landed)
    if (mbar_wait_bounded_warp(done, 0, abort_flag, timeout_ns)) {
      tc_fence_after();
#pragma unroll 1
      for (int c = 32 * half; c < NTOK && c < M; c += 64) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + c, r);
        tmem_ld_wait();
#pragma unroll
        for (int x = 0; x < 32; ++x) own[(c + x) * 128 + row] = __uint_as_float(r[x]);
      }
      tc_fence_before();
    } else if (lane == 0) {
      record_timeout(kSiteEpiTmemFull);
      *abort_flag = 1;
    }
    fence_async_shared();
    asm volatile("bar.sync 1, 256;" ::: "memory");  // the epilogue warps
    const uint32_t owner = threadIdx.x - 64;
    if (owner < S && owner != rank) {
      const int tokens = min(slice, M - static_cast<int>(owner) * slice);
      if (tokens > 0)
        bulk_copy_cluster(map_shared_rank(smem_u32(sums + rank * slice * 128), owner),
                          own + owner * slice * 128, tokens * 512,
                          map_shared_rank(smem_u32(met), owner));
    }
    bool ok = true;
    if (S > 1 && !mbar_wait_bounded_warp(met, 0, abort_flag, timeout_ns)) {
      if (lane == 0) {
        record_timeout(kSiteEpiTmemFull);
        *abort_flag = 1;
      }
      ok = false;
    }
    // ------------------------------------------------------------ epilogue
    for (int x0 = half * RUN; ok && x0 < count; x0 += 2 * RUN) {
      // the next ones' loads go before this run's stores (R may be Y)
      float next[RUN];
      load_residual(next, x0 + 2 * RUN);
      float v[RUN];
#pragma unroll
      for (int y = 0; y < RUN; ++y) v[y] = 0.0f;
      for (uint32_t k = 0; k < S; ++k) {
        const float *from = k == rank ? own + m0 * 128 : sums + k * slice * 128;
#pragma unroll
        for (int y = 0; y < RUN; ++y)
          if (x0 + y < count) v[y] += from[(x0 + y) * 128 + row];
      }
#pragma unroll
      for (int y = 0; y < RUN; ++y) {
        v[y] = fmaf(v[y], scale, bias);
        switch (E.act) {
          case kActRelu: v[y] = activate<kActRelu>(v[y]); break;
          case kActSilu: v[y] = activate<kActSilu>(v[y]); break;
          case kActGelu: v[y] = activate<kActGelu>(v[y]); break;
          default: break;
        }
        v[y] += res[y];
        if (x0 + y < count) {
          const int64_t at = static_cast<int64_t>(row0 + m0 + x0 + y) * N + n;
          if (E.s_out)
            static_cast<uint8_t *>(out)[at] =
                static_cast<uint8_t>(cvt_e4m3x2(v[y] * inv_out, 0.0f));
          else
            static_cast<__nv_bfloat16 *>(out)[at] = __float2bfloat16_rn(v[y]);
        }
        res[y] = next[y];
      }
    }
  }
  // no block leaves while another may still copy from or to its shared memory
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, NTOK);
  }
}

}  // namespace fp8ws
