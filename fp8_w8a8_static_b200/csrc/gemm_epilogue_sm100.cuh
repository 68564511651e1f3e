// FP8 E4M3 W8A8 Linear with bias, activation and residual in its epilogue, on
// CTA pairs (tcgen05 cta_group::2), for sm_100a.
//
//   Y[M,N] = out( act( (s_in s_w) Xq[M,K] . Wq[N,K]^T + bias[N] ) + R[M,N] )
//
// in fp32 up to one rounding: out = BF16, or E4M3 codes of the value over
// s_out.  The main loop is fp8_gemm_pair_kernel's for one problem: 256 x 256
// tiles, both CTAs loading 128 rows of A and of B per 128-byte K step, the
// last ragged wave as 256 x 128 halves.
//   warp 0      TMA producer (both CTAs; no cluster multicast)
//   warp 1      TMEM allocation (both CTAs); MMA issue (leader)
//   warps 2..9  epilogue (both CTAs): two warps per TMEM lane quarter, each on
//               half of the tile's columns, 32 columns at a time
// What the epilogue adds to a plain one is traffic (2 bytes an element for R)
// and issue slots (an activation is 8 to 14 instructions and two of the
// special function unit an element).  Both stay behind the next tile's main
// loop: R comes by TMA into two 32 x 32 boxes a warp, the first two asked for
// before the accumulator is awaited, and eight warps halve the last tile's
// exposed epilogue.  Y leaves through 64-byte-swizzled boxes by TMA stores.
// R may be Y itself: a warp's box is read before the same box is stored.
#pragma once

#include "common.cuh"
#include "elementwise.cuh"
#include "gemm_pair_sm100.cuh"

namespace fp8ws {

constexpr int kEpiWarps = 8;
constexpr int kEpiThreads = 64 + 32 * kEpiWarps;

enum EpiAct : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3 };

struct EpilogueArgs {
  const float *s_in;
  const float *s_w;
  const uint16_t *bias;  // may be null
  const float *s_out;    // FP8 output only
  int act;
};

template <bool FP8, bool RES>
struct EpiCfg {
  static constexpr int STAGES = RES ? 5 : 6;
  static constexpr int A_BYTES = 128 * kGemmBK;
  static constexpr int B_BYTES = 128 * kGemmBK;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int TX_BYTES = 2 * STAGE_BYTES;
  static constexpr int TX_HALF_BYTES = 2 * (A_BYTES + B_BYTES / 2);
  static constexpr int BOX_BYTES = 32 * 64;  // 32 rows of 64 bytes
  static constexpr int STORE_COLS = FP8 ? 64 : 32;
  static constexpr int OUT_BYTES = kEpiWarps * 2 * BOX_BYTES;
  static constexpr int RES_BYTES = RES ? kEpiWarps * 2 * BOX_BYTES : 0;
  static constexpr int BAR_BYTES = 512;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + OUT_BYTES + RES_BYTES + BAR_BYTES + 1024;
  static constexpr uint32_t TMEM_COLS = 512;  // two 256-column accumulators
  static_assert((2 * STAGES + 5 + 2 * kEpiWarps) * 8 + 8 <= BAR_BYTES, "barrier area");
  static_assert(SMEM_BYTES <= 232448, "shared memory");
};

// silu(x) = x / (1 + e^-x); gelu(x) = x / (1 + e^-2u) with u = sqrt(2/pi)
// (x + 0.044715 x^3), the tanh form (0.5 (1 + tanh u) = 1 / (1 + e^-2u), which
// keeps its relative accuracy where the value is small).  NaN passes through
// all of them.  The exponential's argument a is rounded, so the relative error
// grows with it: |a| 2^-24 for each of its roundings (two of SiLU's, up to four of
// GELU's, their constants' among them) beside some 2^-21 of ex2 and rcp.
template <int ACT>
__device__ __forceinline__ float activate(float x) {
  if constexpr (ACT == kActRelu) {
    return x < 0.0f ? 0.0f : x;
  } else if constexpr (ACT == kActSilu) {
    return x * rcp_approx(1.0f + ex2_approx(x * -1.4426950408889634f));
  } else if constexpr (ACT == kActGelu) {
    // -2 sqrt(2/pi) log2(e) (x + 0.044715 x^3)
    const float u = x * fmaf(x * x, -0.10294324f, -2.3022082f);
    return x * rcp_approx(1.0f + ex2_approx(u));
  } else {
    return x;
  }
}

// v = act(acc scale + bias) of 32 columns of one row.
template <int ACT>
__device__ __forceinline__ void activate32(const uint32_t (&r)[32], float scale,
                                           const float (&bias)[32], float (&v)[32]) {
#pragma unroll
  for (int e = 0; e < 32; ++e)
    v[e] = activate<ACT>(fmaf(__uint_as_float(r[e]), scale, bias[e]));
}

template <bool FP8, bool RES>
__global__ void __launch_bounds__(kEpiThreads, 1)
    fp8_gemm_epilogue_kernel(const __grid_constant__ CUtensorMap tm_a,
                             const __grid_constant__ CUtensorMap tm_b,
                             const __grid_constant__ CUtensorMap tm_bh,
                             const __grid_constant__ CUtensorMap tm_r,
                             const __grid_constant__ CUtensorMap tm_d, const PairGroup G,
                             const EpilogueArgs E, int K, uint64_t timeout_ns, SplitPlan plan) {
  using C = EpiCfg<FP8, RES>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *sA = smem;
  uint8_t *sB = smem + STAGES * C::A_BYTES;
  uint8_t *sOut = sB + STAGES * C::B_BYTES;
  uint8_t *sRes = sOut + C::OUT_BYTES;
  uint64_t *bars = reinterpret_cast<uint64_t *>(sRes + C::RES_BYTES);
  uint64_t *full = bars;              // leader: both CTAs' loads of a stage landed
  uint64_t *empty = bars + STAGES;    // both: the leader's MMAs finished with a stage
  uint64_t *tfull = bars + 2 * STAGES;  // both: an accumulator is complete
  uint64_t *tempty = tfull + 2;       // leader: both CTAs' epilogues read an accumulator
  uint64_t *drain = tempty + 2;       // leader: every MMA retired
  uint64_t *rfull = drain + 1;        // a warp's residual box landed
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(rfull + 2 * kEpiWarps);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cluster = blockIdx.x >> 1;
  const int nclusters = gridDim.x >> 1;
  const int num_kb = (K + kGemmBK - 1) / kGemmBK;
  const int num_units = plan_units(plan);
  const int M = G.M[0], N = G.N[0];

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    for (int i = 0; i < 2 * kEpiWarps; ++i) mbar_init(&rfull[i], 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(plan.halves == 2 ? &tm_bh : &tm_b);
    tma_prefetch_desc(&tm_d);
    if (RES) tma_prefetch_desc(&tm_r);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, C::TMEM_COLS);
    tmem_relinquish_pair();
  }
  pdl_launch_dependents();
  pdl_wait();  // the previous kernel's outputs (our inputs) are complete from here on
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      uint32_t issued_mask = 0, issued_parity = 0;
      bool ok = true;
      const uint64_t pol_first = l2_policy_evict_first();
      const uint64_t pol_normal = l2_policy_evict_normal();
      const uint64_t pol_a = G.hint[0] == kHintAFirst ? pol_first : pol_normal;
      const uint64_t pol_b = G.hint[0] == kHintBFirst ? pol_first : pol_normal;
      for (int u = cluster; u < num_units && ok; u += nclusters) {
        const UnitRange ur = unit_range(u, plan, num_kb);
        const GroupTile gt = group_tile(ur.tile, G);
        if (!unit_live(ur, gt, G)) continue;
        const bool half = ur.half >= 0;
        const int a_row = gt.tc.m * kPairTile + static_cast<int>(rank) * 128;
        const int b_row = unit_col0(ur, gt) + static_cast<int>(rank) * (half ? 64 : 128);
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag, timeout_ns)) {
            record_timeout(kSiteProducerEmpty);
            *abort_flag = 1;
            ok = false;
            break;
          }
          const uint32_t full_leader = map_shared_rank(smem_u32(&full[stage]), 0);
          if (leader) mbar_arrive_expect_tx(&full[stage], half ? C::TX_HALF_BYTES : C::TX_BYTES);
          tma_load_2d_pair_hint(sA + stage * C::A_BYTES, &tm_a, full_leader, kb * kGemmBK, a_row,
                                pol_a);
          tma_load_2d_pair_hint(sB + stage * C::B_BYTES, half ? &tm_bh : &tm_b, full_leader,
                                kb * kGemmBK, b_row, pol_b);
          issued_mask |= 1u << stage;
          issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && leader) {
        // Let the loads of the rounds this CTA started land before leaving.
        int zero = 0;
        for (int s = 0; s < STAGES; ++s)
          if (issued_mask & (1u << s))
            mbar_wait_bounded(&full[s], (issued_parity >> s) & 1u, &zero, timeout_ns);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------- MMA issue (leader)
    if (lane == 0 && leader) {
      constexpr uint32_t idesc_full = idesc_e4m3_f32(kPairTile, kPairTile);
      constexpr uint32_t idesc_half = idesc_e4m3_f32(kPairTile, kPairTile / 2);
      uint32_t stage = 0, phase = 0;
      uint32_t it = 0;
      bool ok = true;
      for (int u = cluster; u < num_units && ok; u += nclusters) {
        const UnitRange ur = unit_range(u, plan, num_kb);
        if (!unit_live(ur, group_tile(ur.tile, G), G)) continue;
        const uint32_t idesc = ur.half >= 0 ? idesc_half : idesc_full;
        const uint32_t acc = it & 1u;
        const uint32_t acc_phase = (it >> 1) & 1u;
        if (!mbar_wait_bounded(&tempty[acc], acc_phase ^ 1u, abort_flag, timeout_ns)) {
          record_timeout(kSiteMmaTmemEmpty);
          *abort_flag = 1;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * kPairTile;
        for (int kb = 0; kb < num_kb; ++kb) {
          if (!mbar_wait_bounded(&full[stage], phase, abort_flag, timeout_ns)) {
            record_timeout(kSiteMmaFull);
            *abort_flag = 1;
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(sA + stage * C::A_BYTES);
          const uint32_t b_addr = smem_u32(sB + stage * C::B_BYTES);
#pragma unroll
          for (int k = 0; k < kGemmBK / 32; ++k) {
            umma_f8_pair(d_tmem, smem_desc_k_sw128(a_addr + k * 32),
                         smem_desc_k_sw128(b_addr + k * 32), idesc, (kb | k) != 0 ? 1u : 0u);
          }
          umma_commit_pair(&empty[stage], 0x3);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) umma_commit_pair(&tfull[acc], 0x3);
        ++it;
      }
      umma_commit_pair(drain, 0x1);
      int zero = 0;
      if (!mbar_wait_bounded(drain, 0, &zero, timeout_ns)) record_timeout(kSiteDrain);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ epilogue (both CTAs)
    const int ew = warp - 2;
    const int quarter = warp & 3;  // the TMEM lanes this warp may read
    const float scale = __ldg(E.s_in) * __ldg(E.s_w);
    const float inv_out = FP8 ? __frcp_rn(__ldg(E.s_out)) : 1.0f;
    const int sw = (lane >> 1) & 3;  // 64-byte swizzle: unit k of row r lies at (k ^ sw)
    uint8_t *out_buf = sOut + ew * 2 * C::BOX_BYTES;
    uint8_t *res_buf = sRes + ew * 2 * C::BOX_BYTES;
    uint64_t *rbar = rfull + 2 * ew;
    uint32_t it = 0, stored = 0;
    uint32_t rphase = 0, rpending = 0;  // bit per residual box
    for (int u = cluster; u < num_units; u += nclusters) {
      const UnitRange ur = unit_range(u, plan, num_kb);
      const GroupTile gt = group_tile(ur.tile, G);
      if (!unit_live(ur, gt, G)) continue;
      const int nchunk = ur.half >= 0 ? 2 : 4;  // 32-column chunks of this warp
      const int cbase = (ew >> 2) * nchunk * 32;
      const int row0 = gt.tc.m * kPairTile + static_cast<int>(rank) * 128 + quarter * 32;
      const int col0 = unit_col0(ur, gt) + cbase;
      const uint32_t acc = it & 1u;
      const uint32_t acc_phase = (it >> 1) & 1u;
      ++it;
      auto ask = [&](int c) {  // residual box of chunk c
        if (RES && c < nchunk && col0 + c * 32 < N && row0 < M) {
          const int s = c & 1;
          if (lane == 0) {
            mbar_arrive_expect_tx(&rbar[s], C::BOX_BYTES);
            tma_load_2d(res_buf + s * C::BOX_BYTES, &tm_r, &rbar[s], col0 + c * 32, row0);
          }
          rpending |= 1u << s;
        }
      };
      ask(0);
      ask(1);
      if (!mbar_wait_bounded_warp(&tfull[acc], acc_phase, abort_flag, timeout_ns)) {
        if (lane == 0) {
          record_timeout(kSiteEpiTmemFull);
          *abort_flag = 1;
        }
        break;
      }
      tc_fence_after();
      const uint32_t t_acc =
          tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * kPairTile + cbase;
      bool ok = true;
#pragma unroll 1
      for (int c = 0; c < nchunk; ++c) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(t_acc + c * 32, r);
        const int col = col0 + c * 32;
        float bias[32];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint4 w = make_uint4(0, 0, 0, 0);
          if (E.bias && col + 8 * j < N)
            w = __ldg(reinterpret_cast<const uint4 *>(E.bias + col + 8 * j));
          bias[8 * j] = bf16_lo(w.x);
          bias[8 * j + 1] = bf16_hi(w.x);
          bias[8 * j + 2] = bf16_lo(w.y);
          bias[8 * j + 3] = bf16_hi(w.y);
          bias[8 * j + 4] = bf16_lo(w.z);
          bias[8 * j + 5] = bf16_hi(w.z);
          bias[8 * j + 6] = bf16_lo(w.w);
          bias[8 * j + 7] = bf16_hi(w.w);
        }
        tmem_ld_wait();
        if (c == nchunk - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(map_shared_rank(smem_u32(&tempty[acc]), 0));
        }
        if (col >= N || row0 >= M) {  // wholly outside Y
          // an FP8 box whose first half holds columns is stored below
          if (!(FP8 && (c & 1) && col - 32 < N && row0 < M)) continue;
        }
        float v[32];
        switch (E.act) {
          case kActRelu: activate32<kActRelu>(r, scale, bias, v); break;
          case kActSilu: activate32<kActSilu>(r, scale, bias, v); break;
          case kActGelu: activate32<kActGelu>(r, scale, bias, v); break;
          default: activate32<kActNone>(r, scale, bias, v); break;
        }
        if (RES && (rpending >> (c & 1) & 1u)) {
          const int s = c & 1;
          if (!mbar_wait_bounded_warp(&rbar[s], rphase >> s & 1u, abort_flag, timeout_ns)) {
            if (lane == 0) {
              record_timeout(kSiteEpiResidual);
              *abort_flag = 1;
            }
            ok = false;
            break;
          }
          rphase ^= 1u << s;
          rpending &= ~(1u << s);
          const uint8_t *row = res_buf + s * C::BOX_BYTES + lane * 64;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 w = *reinterpret_cast<const uint4 *>(row + ((j ^ sw) << 4));
            v[8 * j] += bf16_lo(w.x);
            v[8 * j + 1] += bf16_hi(w.x);
            v[8 * j + 2] += bf16_lo(w.y);
            v[8 * j + 3] += bf16_hi(w.y);
            v[8 * j + 4] += bf16_lo(w.z);
            v[8 * j + 5] += bf16_hi(w.z);
            v[8 * j + 6] += bf16_lo(w.w);
            v[8 * j + 7] += bf16_hi(w.w);
          }
          __syncwarp();  // the box is read: it may be filled again
          ask(c + 2);
        }
        uint8_t *box = out_buf + (stored & 1u) * C::BOX_BYTES;
        if (!FP8 || (c & 1) == 0) {
          if (lane == 0) tma_store_wait_read<1>();  // this box's previous store has read it
          __syncwarp();
        }
        uint8_t *row = box + lane * 64;
        if constexpr (FP8) {
          uint32_t q[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            q[j] = pack4(cvt_e4m3x2(v[4 * j] * inv_out, v[4 * j + 1] * inv_out),
                         cvt_e4m3x2(v[4 * j + 2] * inv_out, v[4 * j + 3] * inv_out));
          const int k = 2 * (c & 1);
          *reinterpret_cast<uint4 *>(row + ((k ^ sw) << 4)) = make_uint4(q[0], q[1], q[2], q[3]);
          *reinterpret_cast<uint4 *>(row + (((k + 1) ^ sw) << 4)) =
              make_uint4(q[4], q[5], q[6], q[7]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __nv_bfloat162 b =
                  __floats2bfloat162_rn(v[8 * j + 2 * e], v[8 * j + 2 * e + 1]);
              h[e] = *reinterpret_cast<const uint32_t *>(&b);
            }
            *reinterpret_cast<uint4 *>(row + ((j ^ sw) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
          }
        }
        if (!FP8 || (c & 1)) {
          fence_async_shared();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tm_d, box, FP8 ? col - 32 : col, row0);
            tma_store_commit();
          }
          ++stored;
        }
      }
      if (!ok) break;
    }
    if (RES) {  // after a wait that ran out: boxes in flight land first
      int zero = 0;
      for (int s = 0; s < 2; ++s)
        if (rpending >> s & 1u) mbar_wait_bounded_warp(&rbar[s], rphase >> s & 1u, &zero, timeout_ns);
    }
    if (lane == 0) tma_store_wait_all<0>();
  }

  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
  }
}

}  // namespace fp8ws
