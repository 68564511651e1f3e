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
// Blocks an SM of the append and gather kernels: 48 registers a thread.  Their
// rounds are chains of slot, values, codes and store, so it is the warps that
// hide them (8191 x 8 x 128, both: 24.7 us with 54 registers and four blocks, 22.8
// with five, 23.5 with six or eight).
constexpr int kKvBlocks = 5;

__host__ __device__ constexpr int strip_bytes(int D) { return 18 * D; }
__host__ __device__ constexpr int strip_v(int D) { return 8 * D; }
__host__ __device__ constexpr int strip_ks(int D) { return 16 * D; }
__host__ __device__ constexpr int strip_vs(int D) { return 17 * D; }

__device__ __forceinline__ void halves(uint64_t v, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

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

// The (token, head) of a thread's units, which lie `stride` apart: one division
// for all of them.
struct UnitWalk {
  int64_t token, d_token;
  int head, d_head, heads;
  __device__ UnitWalk(int64_t u, int64_t stride, int64_t units, int n) : heads(n) {
    const bool small = units <= INT32_MAX && stride <= INT32_MAX;
    token = small ? static_cast<uint32_t>(u) / static_cast<uint32_t>(n) : u / n;
    d_token = small ? static_cast<uint32_t>(stride) / static_cast<uint32_t>(n) : stride / n;
    head = static_cast<int>(u - token * n);
    d_head = static_cast<int>(stride - d_token * n);
  }
  __device__ void next() {
    token += d_token;
    head += d_head;
    if (head >= heads) {
      head -= heads;
      ++token;
    }
  }
};

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
// A lane owns the 16 values of a scale, so nothing is exchanged but the NaN
// ballot: D/16 lanes for a token's K of one head, D/16 for its V.  Bound by the
// values' bytes (2 read, 0.56 written).  An IEEE division per value would cost
// more than the stream (append and gather of 8191 x 8 x 128: 35 us with it, 22.8
// without), so a code is first bracketed: with r = fl32(1 / by), x fl32(r (1 -
// 2^-20)) and x fl32(r (1 + 2^-20)) lie on either side of fl32(x / by) (each of
// their two roundings, and the quotient's, is 2^-24); where both have one code
// it is the quotient's, and only lanes with a code that differs divide.  Two or
// four units of a lane in flight were not faster: they cost resident blocks.

// Codes of the 8 BF16 values of w over `by`, the IEEE quotient's.  r is 1 / by, 0
// to divide at once.
__device__ __forceinline__ uint32_t quotient_codes(const uint32_t *w, float by, float r) {
  const float l = __fmul_rn(r, 1.0f - 0x1p-20f), h = __fmul_rn(r, 1.0f + 0x1p-20f);
  const uint64_t lo = f32x2(l, l), hi = f32x2(h, h);
  float p[8], q[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t x = f32x2(bf16_lo(w[i]), bf16_hi(w[i]));
    halves(mul_f32x2(x, lo), p[2 * i], p[2 * i + 1]);
    halves(mul_f32x2(x, hi), q[2 * i], q[2 * i + 1]);
  }
  const uint32_t a = cvt_e2m1x8(p), b = cvt_e2m1x8(q);
  if (a == b && r != 0.0f) return a;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    p[2 * i] = __fdiv_rn(bf16_lo(w[i]), by);
    p[2 * i + 1] = __fdiv_rn(bf16_hi(w[i]), by);
  }
  return cvt_e2m1x8(p);
}

// One token's K or V of 16 values (two 16-byte vectors) -> 8 bytes of codes and
// the scale's code.  NaN values count as 0 (`nan` tells).
__device__ __forceinline__ uint2 quantize16(const uint4 (&w)[2], float s, float s6,
                                            uint32_t &scale, bool &nan) {
  uint32_t raw[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
  auto largest = [&] {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = __vmaxu2(top, raw[i] & 0x7FFF7FFFu);
    return max(top & 0xFFFFu, top >> 16);
  };
  uint32_t top = largest();
  nan = top > 0x7F80u;
  if (nan) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if ((raw[i] & 0x7FFFu) > 0x7F80u) raw[i] &= 0xFFFF0000u;
      if ((raw[i] >> 16 & 0x7FFFu) > 0x7F80u) raw[i] &= 0x0000FFFFu;
    }
    top = largest();
  }
  scale = cvt_e4m3x2(__fdiv_rn(__uint_as_float(top << 16), s6), 0.0f) & 0xFFu;
  const float by = __fmul_rn(e4m3_to_float(scale), s);
  if (!(by > 0.0f)) return make_uint2(0, 0);
  const float r = by > 0x1p-120f && by < 0x1p120f ? __frcp_rn(by) : 0.0f;
  return make_uint2(quotient_codes(raw, by, r), quotient_codes(raw + 4, by, r));
}

template <int D>
__global__ void __launch_bounds__(kKvThreads, kKvBlocks)
    fp4_kv_append_kernel(const uint16_t *__restrict__ k, const uint16_t *__restrict__ v,
                         const int64_t *__restrict__ slots, int64_t units, const float *s_k,
                         const float *s_v, const KvCache c) {
  constexpr int LANES = D / 8;             // lanes of a unit: one token of one head
  constexpr int UNITS = kKvThreads / LANES;  // units of a block's round
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x % LANES;
  const bool is_v = lane >= LANES / 2;
  const int part = lane % (LANES / 2);  // which 16 values
  const float s = __ldg(is_v ? s_v : s_k);
  const float s6 = __fmul_rn(6.0f, s);
  const int64_t n_slots = c.pages << c.page_shift;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * UNITS;
  const uint32_t mine = ((1u << LANES) - 1u) << (threadIdx.x % 32 / LANES * LANES);
  const uint16_t *from = is_v ? v : k;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * UNITS;
  UnitWalk at(first + threadIdx.x / LANES, stride, units + UNITS, c.heads);
  // every lane of a warp runs the same number of rounds (the ballot below)
  for (int64_t u0 = first; u0 < units; u0 += stride, at.next()) {
    const int64_t u = u0 + threadIdx.x / LANES;
    uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    int64_t slot = -1;
    if (u < units) {
      const uint4 *src = reinterpret_cast<const uint4 *>(from + u * D) + 2 * part;
      w[0] = ld_stream(src);
      w[1] = ld_stream(src + 1);
      slot = __ldg(slots + at.token);
    }
    uint32_t scale;
    bool nan;
    const uint2 codes = quantize16(w, s, s6, scale, nan);
    const uint32_t nans = __ballot_sync(0xFFFFFFFFu, nan);
    if (!is_v && (nans & mine)) scale = 0x7Fu;
    if (slot < 0 || slot >= n_slots) continue;
    uint8_t *strip = c.data + strip_offset<D>(c, slot, at.head);
    const int row = static_cast<int>(slot & (kStripTokens - 1));
    *reinterpret_cast<uint2 *>(strip + (is_v ? strip_v(D) : 0) + row * (D / 2) + part * 8) = codes;
    strip[(is_v ? strip_vs(D) : strip_ks(D)) + row * (D / 16) + part] = static_cast<uint8_t>(scale);
  }
}

// ------------------------------------------------------------------ gather
template <int D>
__global__ void __launch_bounds__(kKvThreads, kKvBlocks)
    fp4_kv_gather_kernel(const int64_t *__restrict__ slots, int64_t units, const float *s_k,
                         const float *s_v, const KvCache c, uint16_t *__restrict__ k,
                         uint16_t *__restrict__ v) {
  constexpr int LANES = D / 8;
  constexpr int UNITS = kKvThreads / LANES;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x % LANES;
  const bool is_v = lane >= LANES / 2;
  const int part = lane % (LANES / 2);
  const float s = __ldg(is_v ? s_v : s_k);
  const int64_t n_slots = c.pages << c.page_shift;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * UNITS;
  uint16_t *to = is_v ? v : k;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * UNITS + threadIdx.x / LANES;
  UnitWalk at(first, stride, units + UNITS, c.heads);
  for (int64_t u = first; u < units; u += stride, at.next()) {
    uint2 codes = make_uint2(0, 0);
    uint32_t scale = 0;  // zeros for a slot outside the cache
    const int64_t slot = __ldg(slots + at.token);
    if (slot >= 0 && slot < n_slots) {
      const uint8_t *strip = c.data + strip_offset<D>(c, slot, at.head);
      const int row = static_cast<int>(slot & (kStripTokens - 1));
      codes = *reinterpret_cast<const uint2 *>(strip + (is_v ? strip_v(D) : 0) + row * (D / 2) +
                                               part * 8);
      scale = strip[(is_v ? strip_vs(D) : strip_ks(D)) + row * (D / 16) + part];
    }
    const float f = e4m3_to_float(scale);
    uint32_t h[2][4], r[2][4];
    cvt_f16_e2m1x8(codes.x, h[0]);
    cvt_f16_e2m1x8(codes.y, h[1]);
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 e = __half22float2(*reinterpret_cast<__half2 *>(&h[y][i]));
        // code x scale is exact; two roundings, to fp32 and to BF16
        const __nv_bfloat162 b = __floats2bfloat162_rn((e.x * f) * s, (e.y * f) * s);
        r[y][i] = *reinterpret_cast<const uint32_t *>(&b);
      }
    uint4 *dst = reinterpret_cast<uint4 *>(to + u * D) + 2 * part;
    st_stream(dst, make_uint4(r[0][0], r[0][1], r[0][2], r[0][3]));
    st_stream(dst + 1, make_uint4(r[1][0], r[1][1], r[1][2], r[1][3]));
  }
}

// ------------------------------------------------------------------ tables
// Block tables, row offsets and slots of one step, in one cluster.  Every
// block scans the requests' lengths, a thread a request and THREADS at a time
// (the same few KB, so no block waits for another's sums), and fills the new
// pages of its share of the requests, a warp a request.  After a cluster
// barrier the warps take 256 slots at a time: the requests of the first and the
// last of them bound the search of the others (one request, or two or three,
// for prompts).  The row offsets are searched in shared memory where one round
// covers the batch.  All of it is latency, not bytes: dependent reads and the
// instructions of a few SMs are what it counts (300 prompts, 80 thousand
// tokens: 12.7 us, 36 with a full search per slot and one block filling the
// pages; 32 requests of one token: 3.4 us).
constexpr int kTableMaxBlocks = 8;  // the portable cluster size
constexpr int kTableUnroll = 8;     // slots of a thread in flight

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

__device__ __forceinline__ int32_t saturate_i32(int64_t v) {
  return static_cast<int32_t>(v < INT32_MAX ? v : INT32_MAX);
}

// The first of requests [lo, hi) whose rows end after t (hi: none).
__device__ __forceinline__ int request_of(const int32_t *cu, int t, int lo, int hi) {
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (cu[mid + 1] > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// NEAR: at most THREADS requests, one turn; the offsets stay in shared memory.
template <int THREADS, bool NEAR>
__global__ void __launch_bounds__(THREADS) fp4_kv_tables_kernel(const TableArgs a) {
  constexpr int WARPS = THREADS / 32;
  __shared__ int64_t warp_rows[WARPS], warp_pages[WARPS];
  __shared__ int64_t s_from[THREADS];  // a request's first new page in free_pages
  __shared__ int32_t s_held[THREADS], s_need[THREADS];
  __shared__ int32_t s_cu[THREADS + 1], s_old[THREADS];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int rank = blockIdx.x, ranks = gridDim.x;
  const int64_t used = max(0, *a.used);
  // lengths that the slots still need are replaced only after them (kv_lens - added
  // would not do: kv_lens saturates)
  const bool lens_later = !NEAR && a.kv_lens == a.lens;
  int64_t rows = 0, pages = 0;  // of the requests before this turn
  for (int b0 = 0; b0 < a.batch; b0 += THREADS) {
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
    // also: every block has read this turn's lengths, which kv_lens may replace
    cluster_sync();
    int64_t all_rows = 0, all_pages = 0;
#pragma unroll 8
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) {
        r += warp_rows[w];
        p += warp_pages[w];
      }
      all_rows += warp_rows[w];
      all_pages += warp_pages[w];
    }
    s_from[threadIdx.x] = used + pages + p - need;
    s_held[threadIdx.x] = static_cast<int32_t>(held);
    s_need[threadIdx.x] = static_cast<int32_t>(need);
    s_cu[threadIdx.x + 1] = saturate_i32(rows + r);
    s_old[threadIdx.x] = static_cast<int32_t>(old);
    if (rank == 0 && b < a.batch) {
      a.cu_q[b + 1] = saturate_i32(rows + r);
      if (!lens_later) a.kv_lens[b] = saturate_i32(old + add);
    }
    __syncthreads();
    const int here = min(THREADS, a.batch - b0);
    for (int x = rank * WARPS + warp; x < here; x += ranks * WARPS) {
      const int n = s_need[x];
      if (n == 0) continue;
      const int64_t from = s_from[x];
      int32_t *row = a.table + static_cast<int64_t>(b0 + x) * a.width + s_held[x];
#pragma unroll 4
      for (int i = lane; i < n; i += 32)
        row[i] = from + i < a.n_free ? __ldg(a.free_pages + from + i) : -1;
    }
    rows += all_rows;
    pages += all_pages;
    __syncthreads();  // the shared arrays may be written again
  }
  if (threadIdx.x == 0) {
    s_cu[0] = 0;
    if (rank == 0) {
      const int64_t left = max(int64_t(0), a.n_free - used);
      const int64_t got = min(pages, left);
      a.cu_q[0] = 0;
      a.pool[0] = saturate_i32(used + got);
      a.pool[1] = saturate_i32(pages - got);
    }
  }
  cluster_sync();  // the entries and offsets above are visible to the whole cluster
  const int32_t *cu = NEAR ? s_cu : a.cu_q;
  const int last = min(a.n_slots, cu[a.batch]);  // slots behind have no token
  constexpr int RUN = 32 * kTableUnroll;
  for (int64_t base = static_cast<int64_t>(rank * WARPS + warp) * RUN; base < a.n_slots;
       base += static_cast<int64_t>(ranks) * WARPS * RUN) {
    const int t0 = static_cast<int>(base);
    const int end = min(last - t0, RUN);  // slots of the run that have a token
    // lane 0 the first slot's request, the others the last one's
    int edge = 0;
    if (end > 0) edge = request_of(cu, lane == 0 ? t0 : t0 + end - 1, 0, a.batch - 1);
    const int b_first = __shfl_sync(0xFFFFFFFFu, edge, 0);
    const int b_last = __shfl_sync(0xFFFFFFFFu, edge, 1);
    int b[kTableUnroll];
    int64_t at[kTableUnroll];
    int32_t page[kTableUnroll];
#pragma unroll
    for (int x = 0; x < kTableUnroll; ++x) {
      const int i = x * 32 + lane;
      at[x] = -1;
      b[x] = b_first;
      if (i < end) {
        b[x] = request_of(cu, t0 + i, b_first, b_last);
        // (lens may be kv_lens by now where there was one turn)
        const int64_t old = NEAR ? s_old[b[x]] : max(0, a.lens[b[x]]);
        at[x] = old + (t0 + i - cu[b[x]]);
      }
    }
#pragma unroll
    for (int x = 0; x < kTableUnroll; ++x) {
      const int64_t j = at[x] >> a.page_shift;
      page[x] = at[x] >= 0 && j < a.width ? a.table[static_cast<int64_t>(b[x]) * a.width + j] : -1;
    }
#pragma unroll
    for (int x = 0; x < kTableUnroll; ++x)
      if (base + x * 32 + lane < a.n_slots)
        a.slots[base + x * 32 + lane] =
            page[x] < 0 ? -1
                        : (static_cast<int64_t>(page[x]) << a.page_shift) +
                              (at[x] & ((int64_t(1) << a.page_shift) - 1));
  }
  if (lens_later) {
    cluster_sync();  // every block has read the lengths
    if (rank == 0)
      for (int b = threadIdx.x; b < a.batch; b += THREADS)
        a.kv_lens[b] = saturate_i32(static_cast<int64_t>(max(0, a.lens[b])) + max(0, a.added[b]));
  }
}

}  // namespace fp8ws
