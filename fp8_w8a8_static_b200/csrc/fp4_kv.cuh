// The 4-bit paged K/V cache: its format, the kernels that write it, read it
// back and lay out its pages.
//
// A cache is [pages][kv heads][page / 16][18 D] bytes.  16 tokens of one head
// are one strip of 18 D bytes:
//   K codes [16][D/2] | V codes [16][D/2] | K scales [16][D/16] | V scales [16][D/16]
// A code is E2M1 (sign, 2 exponent bits, 1 mantissa bit: 0, .5, 1, 1.5, 2, 3, 4, 6),
// element 2i in the low nibble of byte i.  A scale is one E4M3 value for 16
// elements.  With s the tensor's static fp32 scale:
//   scale = E4M3_satRNE( max16 |x| / fl32(6 s) ),  code = E2M1_satRNE( x / fl32(scale s) )
//   value = code scale s
// code x scale has at most 6 significant bits: it is exact in FP16 and BF16.
// The strip is the unit the attention kernels copy and multiply (16 tokens are
// one K step of the second product), so a page of any size is a whole number
// of contiguous copies, and a 64-token run of a page is one contiguous block.
//
// A NaN in the K or V of a token's head makes that head's 16 K scales of the
// token NaN: every row that attends to the token reads NaN, rows that do not
// are untouched (V, which a masked row multiplies by 0, stays finite).
#pragma once

#include "common.cuh"
#include "elementwise.cuh"

namespace fp8ws {

constexpr int kStripTokens = 16;
constexpr int kKvThreads = 256;

__host__ __device__ constexpr int strip_bytes(int D) { return 18 * D; }
__host__ __device__ constexpr int strip_v(int D) { return 8 * D; }
__host__ __device__ constexpr int strip_ks(int D) { return 16 * D; }
__host__ __device__ constexpr int strip_vs(int D) { return 17 * D; }

// Eight fp32 values -> eight E2M1 codes, value 0 in the lowest nibble
// (nearest, ties to even, saturating at +-6).
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Four bytes of codes -> eight values as four FP16 pairs.
__device__ __forceinline__ void cvt_f16_e2m1x8(uint32_t codes, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
}

// Two E4M3 codes (the low 16 bits) -> an FP16 pair.
__device__ __forceinline__ uint32_t cvt_f16_e4m3x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<unsigned short>(codes)));
  return r;
}

__device__ __forceinline__ float e4m3_to_float(uint32_t code) {
  const uint32_t h = cvt_f16_e4m3x2(code);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

struct KvCache {
  uint8_t *data;
  int64_t pages;
  int heads;
  int page_shift;  // log2 of the tokens of a page
};

// Byte offset of the strip of `slot` (= page * page size + place) for a head,
// in 64 bits: a cache may exceed 4 GB.
template <int D>
__device__ __forceinline__ int64_t strip_offset(const KvCache &c, int64_t slot, int head) {
  const int64_t page = slot >> c.page_shift;
  const int strip = static_cast<int>(slot & ((int64_t(1) << c.page_shift) - 1)) / kStripTokens;
  return (((page * c.heads + head) << (c.page_shift - 4)) + strip) * strip_bytes(D);
}

// ------------------------------------------------------------------ append
// One token's head takes D/4 lanes: D/8 for K, D/8 for V, 8 values each, so
// that K's and V's loads of a warp are whole 128-byte lines.  A pair of lanes
// owns the 16 values of a scale.
template <int D>
__global__ void __launch_bounds__(kKvThreads)
    fp4_kv_append_kernel(const uint16_t *__restrict__ k, const uint16_t *__restrict__ v,
                         const int64_t *__restrict__ slots, int64_t units, const float *s_k,
                         const float *s_v, const KvCache c) {
  constexpr int LANES = D / 4;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x % LANES;
  const bool is_v = lane >= LANES / 2;
  const int part = lane % (LANES / 2);  // which 8 values
  const float s = __ldg(is_v ? s_v : s_k);
  const float s6 = __fmul_rn(6.0f, s);
  const int64_t n_slots = c.pages << c.page_shift;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (kKvThreads / LANES);
  const int64_t warp_units = 32 / LANES;
  // every lane of a warp runs the same number of rounds (the shuffles below)
  for (int64_t u0 = static_cast<int64_t>(blockIdx.x) * (kKvThreads / LANES) +
                    (threadIdx.x / 32) * warp_units;
       u0 < units; u0 += stride) {
    const int64_t u = u0 + (threadIdx.x % 32) / LANES;
    const bool live = u < units;
    const int64_t token = live ? u / c.heads : 0;
    const int head = live ? static_cast<int>(u - token * c.heads) : 0;
    const int64_t slot = live ? __ldg(slots + token) : -1;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (live) w = ld_stream(reinterpret_cast<const uint4 *>((is_v ? v : k) + u * D) + part);
    float x[8] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y),
                  bf16_lo(w.z), bf16_hi(w.z), bf16_lo(w.w), bf16_hi(w.w)};
    float amax = 0.0f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (x[i] != x[i]) {
        nan = true;
        x[i] = 0.0f;
      }
      amax = fmaxf(amax, fabsf(x[i]));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    const uint32_t nans = __ballot_sync(0xFFFFFFFFu, nan);
    const uint32_t mine = (LANES == 32 ? 0xFFFFFFFFu : ((1u << LANES) - 1u))
                          << ((threadIdx.x % 32) / LANES * LANES);
    uint32_t scale = cvt_e4m3x2(__fdiv_rn(amax, s6), 0.0f) & 0xFFu;
    const float by = __fmul_rn(e4m3_to_float(scale), s);
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = by > 0.0f ? __fdiv_rn(x[i], by) : 0.0f;
    const uint32_t codes = cvt_e2m1x8(t);
    if (!is_v && (nans & mine)) scale = 0x7Fu;
    if (slot < 0 || slot >= n_slots) continue;
    uint8_t *strip = c.data + strip_offset<D>(c, slot, head);
    const int row = static_cast<int>(slot & (kStripTokens - 1));
    *reinterpret_cast<uint32_t *>(strip + (is_v ? strip_v(D) : 0) + row * (D / 2) + part * 4) =
        codes;
    if (!(part & 1))
      strip[(is_v ? strip_vs(D) : strip_ks(D)) + row * (D / 16) + part / 2] =
          static_cast<uint8_t>(scale);
  }
}

// ------------------------------------------------------------------ gather
template <int D>
__global__ void __launch_bounds__(kKvThreads)
    fp4_kv_gather_kernel(const int64_t *__restrict__ slots, int64_t units, const float *s_k,
                         const float *s_v, const KvCache c, uint16_t *__restrict__ k,
                         uint16_t *__restrict__ v) {
  constexpr int LANES = D / 4;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x % LANES;
  const bool is_v = lane >= LANES / 2;
  const int part = lane % (LANES / 2);
  const float s = __ldg(is_v ? s_v : s_k);
  const int64_t n_slots = c.pages << c.page_shift;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (kKvThreads / LANES);
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kKvThreads / LANES) + threadIdx.x / LANES;
       u < units; u += stride) {
    const int64_t token = u / c.heads;
    const int head = static_cast<int>(u - token * c.heads);
    const int64_t slot = __ldg(slots + token);
    uint4 out = make_uint4(0, 0, 0, 0);
    if (slot >= 0 && slot < n_slots) {
      const uint8_t *strip = c.data + strip_offset<D>(c, slot, head);
      const int row = static_cast<int>(slot & (kStripTokens - 1));
      const uint32_t codes = *reinterpret_cast<const uint32_t *>(
          strip + (is_v ? strip_v(D) : 0) + row * (D / 2) + part * 4);
      const float scale =
          e4m3_to_float(strip[(is_v ? strip_vs(D) : strip_ks(D)) + row * (D / 16) + part / 2]);
      uint32_t h[4], r[4];
      cvt_f16_e2m1x8(codes, h);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<__half2 *>(&h[i]));
        // code x scale is exact; two roundings, to fp32 and to BF16
        const __nv_bfloat162 b =
            __floats2bfloat162_rn((f.x * scale) * s, (f.y * scale) * s);
        r[i] = *reinterpret_cast<const uint32_t *>(&b);
      }
      out = make_uint4(r[0], r[1], r[2], r[3]);
    }
    st_stream(reinterpret_cast<uint4 *>((is_v ? v : k) + u * D) + part, out);
  }
}

// ------------------------------------------------------------------ tables
// Block tables, row offsets and slots of one step, in one cluster: its first
// block scans the requests' lengths (each thread one request, a running sum
// from one 512-request round to the next), writes the row offsets, the new
// lengths and the table entries of the new pages; after a cluster barrier
// every thread of the cluster finds the slots of its tokens by a search in the
// row offsets.  All of it is latency: a few dependent reads of a few KB.
constexpr int kTableThreads = 512;
constexpr int kTableMaxBlocks = 8;  // the portable cluster size

struct TableArgs {
  const int32_t *lens;
  const int32_t *added;
  int batch;
  int page_shift;
  int32_t *table;
  int64_t width;
  const int32_t *free_pages;
  int64_t n_free;
  const int32_t *used;
  int32_t *pool;
  int32_t *cu_q;
  int32_t *kv_lens;
  int64_t *slots;
  int n_slots;
};

__device__ __forceinline__ int64_t pages_of(int64_t tokens, int shift, int64_t width) {
  const int64_t p = (tokens + (int64_t(1) << shift) - 1) >> shift;
  return p < width ? p : width;
}

__global__ void __launch_bounds__(kTableThreads) fp4_kv_tables_kernel(const TableArgs a) {
  __shared__ int64_t warp_rows[kTableThreads / 32], warp_pages[kTableThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  if (cluster_ctarank() == 0) {
    const int64_t used = max(0, *a.used);
    int64_t rows = 0, pages = 0;  // of the requests before this round
    if (threadIdx.x == 0) a.cu_q[0] = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kTableThreads) {
      const int b = b0 + static_cast<int>(threadIdx.x);
      int64_t old = 0, add = 0;
      if (b < a.batch) {
        old = max(0, a.lens[b]);
        add = max(0, a.added[b]);
      }
      const int64_t held = pages_of(old, a.page_shift, a.width);
      const int64_t need = pages_of(old + add, a.page_shift, a.width) - held;
      int64_t r = add, p = need;  // inclusive sums over the warp, then the block
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t r2 = __shfl_up_sync(0xFFFFFFFFu, r, d);
        const int64_t p2 = __shfl_up_sync(0xFFFFFFFFu, p, d);
        if (lane >= d) {
          r += r2;
          p += p2;
        }
      }
      if (lane == 31) {
        warp_rows[warp] = r;
        warp_pages[warp] = p;
      }
      __syncthreads();
      int64_t all_rows = 0, all_pages = 0;
#pragma unroll
      for (int w = 0; w < kTableThreads / 32; ++w) {
        if (w < warp) {
          r += warp_rows[w];
          p += warp_pages[w];
        }
        all_rows += warp_rows[w];
        all_pages += warp_pages[w];
      }
      __syncthreads();
      if (b < a.batch) {
        a.cu_q[b + 1] = static_cast<int32_t>(min(rows + r, static_cast<int64_t>(INT32_MAX)));
        a.kv_lens[b] = static_cast<int32_t>(min(old + add, static_cast<int64_t>(INT32_MAX)));
      }
      // the new pages of the warp's requests, one request after the other
      const int64_t first = used + pages + p - need;
      uint32_t todo = __ballot_sync(0xFFFFFFFFu, need > 0);
      while (todo) {
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        const int64_t n = __shfl_sync(0xFFFFFFFFu, need, src);
        const int64_t from = __shfl_sync(0xFFFFFFFFu, first, src);
        const int64_t to = __shfl_sync(0xFFFFFFFFu, held, src);
        int32_t *row = a.table + static_cast<int64_t>(b0 + warp * 32 + src) * a.width;
        for (int64_t i = lane; i < n; i += 32)
          row[to + i] = from + i < a.n_free ? a.free_pages[from + i] : -1;
      }
      rows += all_rows;
      pages += all_pages;
    }
    __syncthreads();  // pool may be the buffer that `used` was read from
    if (threadIdx.x == 0) {
      const int64_t left = max(int64_t(0), a.n_free - used);
      const int64_t got = min(pages, left);
      a.pool[0] = static_cast<int32_t>(min(used + got, static_cast<int64_t>(INT32_MAX)));
      a.pool[1] = static_cast<int32_t>(min(pages - got, static_cast<int64_t>(INT32_MAX)));
    }
  }
  cluster_sync();  // the writes above are visible to the whole cluster
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kTableThreads + threadIdx.x; t < a.n_slots;
       t += static_cast<int64_t>(gridDim.x) * kTableThreads) {
    int lo = 0, hi = a.batch;  // the first request whose rows end after t
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (a.cu_q[mid + 1] > t)
        hi = mid;
      else
        lo = mid + 1;
    }
    int64_t slot = -1;
    if (lo < a.batch) {
      const int64_t start = a.cu_q[lo];
      // the request's new tokens are its last ones (lens may be kv_lens by now)
      const int64_t at = a.kv_lens[lo] - static_cast<int64_t>(max(0, a.added[lo])) + t - start;
      const int64_t j = at >> a.page_shift;
      if (j < a.width) {
        const int64_t page = a.table[static_cast<int64_t>(lo) * a.width + j];
        if (page >= 0)
          slot = (page << a.page_shift) + (at & ((int64_t(1) << a.page_shift) - 1));
      }
    }
    a.slots[t] = slot;
  }
}

}  // namespace fp8ws
