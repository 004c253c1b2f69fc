// Device helpers of the paged 8-bit cache kernels: where a position's row
// lives, and codes as pairs of f16.
//
// A page holds page_tokens (P, a power of two from 16 to 128) consecutive
// positions of one sequence for every kv head, K and V apart; each (page, kv
// head) has one fp32 scale for its K codes and one for its V codes, and a row
// reads as code * scale.  P >= 16, so 16 positions that start at a multiple
// of 16 lie in one page, under one scale.
#pragma once
#include <cuda_fp8.h>

#include "kvq_common.cuh"
#include "kvq_paged.h"

namespace kvq {
namespace {

// A page's scale below this is stored as 0 (all codes 0); readers may take
// log2 and the reciprocal of every other scale.
constexpr float kSmallestScale = 9.094947017729282e-13f;   // 2^-40

// A V scale of 0 counts as this in a read's reference and sum: 2^20 below the
// smallest scale, so that a page of zeros sets the reference only where its keys
// weigh 2^20 times the others' (counted as 1, it pushed the others' probabilities
// below f16's range); and not so small that a weight of 2^-30 beside values of
// scale 2^40 leaves fp32's range before it is summed (2^(-30 - 60 - 40)).
constexpr float kZeroScale = 8.673617379884035e-19f;       // 2^-60

// The largest i in [0, n) with key(i) <= x, for non-decreasing keys with key(0)
// <= x, by a whole warp: 32 keys at a time, so that up to 1024 take two loads one
// after the other in the place of ten.
template <typename T, typename Key>
__device__ __forceinline__ int warp_search(int n, T x, Key key) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  while (n > 1) {
    const int step = (n + 31) / 32, i = lane * step;
    const uint32_t b = __ballot_sync(0xffffffffu, i < n && key(lo + i) <= x);
    const int at = max(0, 31 - __clz(b)) * step;          // (lane 0's key is)
    lo += at;
    n = min(step, n - at);
  }
  return lo;
}

// The sequence of a packed row: the largest s with off[s] <= row.
__device__ __forceinline__ int paged_seq_of(const PagedRows& r, int row) {
  if (r.row_offsets == nullptr) return row;
  int lo = 0, hi = r.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(r.row_offsets + mid) <= row) lo = mid; else hi = mid - 1;
  }
  return lo;
}

struct SeqRows { int s, off, rows, start; };
__device__ __forceinline__ SeqRows paged_seq_rows(const PagedRows& r, int s) {
  if (r.row_offsets == nullptr) return {s, s, 1, __ldg(r.start + s)};
  const int o = __ldg(r.row_offsets + s);
  return {s, o, __ldg(r.row_offsets + s + 1) - o, __ldg(r.start + s)};
}

constexpr int kNoPage = -2;          // of a read, in the place of a page: rows see the keys, but the table names no page

// The page of position p of sequence s, or -1 when the table names none.
__device__ __forceinline__ int paged_page(const PagedArgs& pg, int s, int p) {
  const int id = __ldg(pg.tables + (size_t)s * pg.max_pages + (p >> pg.p_shift));
  return (unsigned)id < (unsigned)pg.n_pages ? id : -1;
}

// Four codes (bytes 0..3 of w) as two pairs of f16: (0, 1) and (2, 3).
//   int8: a code with its sign bit flipped under the exponent of 1024 is 1024 +
//   128 + code; the subtraction of 1152 is exact.
//   e4m3: the hardware's conversion (three logic operations a pair, which
//   rebias the exponent, took 7 % longer in the decode read).
__device__ __forceinline__ uint32_t h2_sub_1152(uint32_t x) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&x), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <bool E4M3>
__device__ __forceinline__ void codes_to_h2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (E4M3) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
  } else {
    w ^= 0x80808080u;
    lo = h2_sub_1152(prmt(w, 0x64646464u, 0x4140u));
    hi = h2_sub_1152(prmt(w, 0x64646464u, 0x4342u));
  }
}

// x / s as a code byte, rounded half to even: fl32(x / s) for s > 0.
template <bool E4M3>
__device__ __forceinline__ uint32_t encode_q(float q) {
  if constexpr (E4M3) return (uint32_t)__nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
  return (uint32_t)min(max(__float2int_rn(q), -127), 127) & 0xFFu;
}
template <bool E4M3>
__device__ __forceinline__ float decode_byte(uint32_t b) {
  if constexpr (E4M3) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b, __NV_E4M3);
    return __half2float(__half(h));
  }
  return (float)(int)(int8_t)b;
}

}  // namespace
}  // namespace kvq
