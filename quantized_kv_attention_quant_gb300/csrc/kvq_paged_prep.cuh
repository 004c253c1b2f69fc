// The rows' prep of the paged calls: RMSNorm and RoPE of 256 / D rows (one of
// 256 or 512) at a time by one warp, at least 8 consecutive elements a lane, each
// rounded to the bf16 nearest to the exact result (the precision contract of
// kvq_common.cuh).
//
// The float-float arithmetic that decides every rounding is needed only where
// a plain fp32 result lies near a tie.  So the row is formed in fp32 with a
// bound on its error, rounded from both ends of the interval, and only where
// the two differ in bf16 is the exact form taken: for the norm the whole row
// (its sum of squares), for the rotation the element.
//   Norm.  x^2 is exact; a lane's 8 or 16 squares are summed in two chains, so
//   that at most 8 + 1 + 5 (lanes) additions and one of eps round: <= 15 * 2^-24
//   of the sum, half of it in 1/sqrt, whose approximation is within 2^-22.9 (2.2 *
//   2^-24), and the product with x w (exact) rounds once: below 11 * 2^-24; 12 *
//   2^-24 are taken.
//   Rotation.  r = fl(x c + fl(y s)) with c, s the leading floats of the angle.
//   What they leave out is at most 2^-25 each, the product rounds by 2^-24 |y|, r
//   and the two ends by 2^-24 |r| each, and |r| <= |x| + |y|: 3.5 * 2^-24 (|x| +
//   |y|) in all; 2^-22 are taken.
// 2^-140 more on each side covers what underflows; it also sends exact zeros to
// the exact forms, which keep their sign.
// About 1 row in 30 of 128 dims takes the norm's exact form, and an element in
// some 1000 the rotation's.
#pragma once
#include "kvq_common.cuh"

namespace kvq {
namespace {

__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// E 16-bit values as pairs, 16 bytes an access.
template <int E>
__device__ __forceinline__ void load_pairs(uint32_t (&v)[E / 2], const uint16_t* p) {
#pragma unroll
  for (int i = 0; i < E / 8; ++i) {
    const uint4 x = reinterpret_cast<const uint4*>(p)[i];
    v[4 * i] = x.x;
    v[4 * i + 1] = x.y;
    v[4 * i + 2] = x.z;
    v[4 * i + 3] = x.w;
  }
}
template <int E>
__device__ __forceinline__ void store_pairs(uint16_t* p, const uint32_t (&v)[E / 2]) {
#pragma unroll
  for (int i = 0; i < E / 8; ++i)
    reinterpret_cast<uint4*>(p)[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

// A row's lanes, and rows of a warp.
template <int D>
struct PrepLanes {
  static constexpr int E = D < 256 ? 8 : D / 32;          // elements a lane
  static constexpr int N = D / E;                         // lanes a row
  static constexpr int ROWS = 32 / N;                     // rows a warp
};

// Item i of n rows (r) by heads (h), i < 2^16; inv = ceil(2^32 / heads) gives
// i / heads exactly (for one head it passes 32 bits).
struct PrepItem { int r, h; };
__device__ __forceinline__ uint32_t prep_inv(int heads) { return 0xFFFFFFFFu / (uint32_t)heads + 1u; }
__device__ __forceinline__ PrepItem prep_item(int i, int heads, uint32_t inv) {
  const int r = heads == 1 ? i : (int)__umulhi((uint32_t)i, inv);
  return {r, i - r * heads};
}

// Angles of a block's rows: the leading floats (cos, sin) and the rest apart,
// R/2 pairs a row.  Under full rotation lane l of a row's first half and its
// partner in the second rotate elements l E .. with the pairs l E .., two of them
// 16 bytes apart from the next lane's: pair j = l E + 2 i + e is entry
// N i + 2 l + e.
struct Angles {
  float2* hi;
  float2* lo;
};
template <int D>
__device__ __forceinline__ int angle_at(int R, int j) {
  constexpr int E = PrepLanes<D>::E;
  return R == D ? (j % E / 2) * PrepLanes<D>::N + j / E * 2 + (j & 1) : j;
}
template <int D>
__device__ __forceinline__ void put_angle(const Angles& t, int row, int R, int j, int p, const float (&f)[3]) {
  ff c, s;
  rope_cos_sin(p, f[0], f[1], f[2], c, s);
  const int at = row * (R >> 1) + angle_at<D>(R, j);
  t.hi[at] = make_float2(c.hi, s.hi);
  t.lo[at] = make_float2(c.lo, s.lo);
}

constexpr float kUnder = 7.17464813734306e-43f;           // 2^-140
constexpr float kRotEnds = 2.384185791015625e-7f;         // 2^-22

// The two ends of x c + y s.
__device__ __forceinline__ float2 rot_ends(float x, float y, float c, float s) {
  const float r = __fmaf_rn(x, c, __fmul_rn(y, s)), b = fabsf(x) + fabsf(y);
  return make_float2(__fmaf_rn(b, kRotEnds, r) + kUnder, __fmaf_rn(b, -kRotEnds, r) - kUnder);
}

// raw: the lane's E bf16 in pairs; w: its weights; row: the row's place in the
// angles; nr: two shared rows [D] of the row's own (0 < R < D).  Returns the
// prepped elements in pairs.  All lanes of the warp call it.
template <int D, int E = PrepLanes<D>::E>
__device__ __forceinline__ void prep_row(const uint32_t (&raw)[E / 2], const float (&w)[E], const float eps,
                                         const int R, const Angles& ang, const int row, uint16_t* nr,
                                         uint32_t (&y)[E / 2]) {
  constexpr int N = PrepLanes<D>::N;
  const int lane = threadIdx.x & (N - 1), half = R >> 1;
  float s0 = 0.f, s1 = 0.f;
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    s0 = __fmaf_rn(bf16lo_to_f(raw[i]), bf16lo_to_f(raw[i]), s0);
    s1 = __fmaf_rn(bf16hi_to_f(raw[i]), bf16hi_to_f(raw[i]), s1);
  }
  float ss = s0 + s1;
#pragma unroll
  for (int m = N / 2; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
  const float ms = __fadd_rn(__fmul_rn(ss, 1.f / D), eps);
  float inv;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(ms));
  const float eb = inv * (12.f / 16777216.f);
  bool same = ms > 1e-30f && ms < 1e30f;                  // (no subnormals, no overflow in the bound)
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    const float a = __fmul_rn(bf16lo_to_f(raw[i]), w[2 * i]), b = __fmul_rn(bf16hi_to_f(raw[i]), w[2 * i + 1]);
    const float da = __fmaf_rn(fabsf(a), eb, kUnder), db = __fmaf_rn(fabsf(b), eb, kUnder);
    y[i] = bf16x2_rn(__fmaf_rn(a, inv, da), __fmaf_rn(b, inv, db));
    same &= y[i] == bf16x2_rn(__fmaf_rn(a, inv, -da), __fmaf_rn(b, inv, -db));
  }
  if (!__all_sync(0xffffffffu, same)) {
    ff t0 = {0.f, 0.f}, t1 = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      ff_acc_sq(t0, bf16lo_to_f(raw[i]));
      ff_acc_sq(t1, bf16hi_to_f(raw[i]));
    }
    t0 = ff_add(t0, t1);
#pragma unroll
    for (int m = N / 2; m >= 1; m >>= 1)
      t0 = ff_add(t0, ff{__shfl_xor_sync(0xffffffffu, t0.hi, m), __shfl_xor_sync(0xffffffffu, t0.lo, m)});
    const ff ex = rms_inv(t0, D, eps);
#pragma unroll
    for (int i = 0; i < E / 2; ++i)
      y[i] = (uint32_t)norm_scale_bf16(bf16lo_to_f(raw[i]), w[2 * i], ex) |
             ((uint32_t)norm_scale_bf16(bf16hi_to_f(raw[i]), w[2 * i + 1], ex) << 16);
  }
  if (R == D) {
    // x_e c - x_(e+D/2) s in the row's first lanes, x_e c + x_(e-D/2) s in the others
    const float4* t = reinterpret_cast<const float4*>(ang.hi + row * half) + (lane & (N / 2 - 1));
    const uint32_t flip = lane < N / 2 ? 0x80008000u : 0u;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const uint32_t o = __shfl_xor_sync(0xffffffffu, y[i], N / 2) ^ flip;
      const float4 a = t[N / 2 * i];                        // (cos, sin) of both elements
      const float2 r0 = rot_ends(bf16lo_to_f(y[i]), bf16lo_to_f(o), a.x, a.y);
      const float2 r1 = rot_ends(bf16hi_to_f(y[i]), bf16hi_to_f(o), a.z, a.w);
      uint32_t r = bf16x2_rn(r0.x, r1.x);
      if (r != bf16x2_rn(r0.y, r1.y)) {
        const float4 b = (reinterpret_cast<const float4*>(ang.lo + row * half) + (lane & (N / 2 - 1)))[N / 2 * i];
        r = (uint32_t)rot_bf16(bf16lo_to_f(y[i]), bf16lo_to_f(o), ff{a.x, b.x}, ff{-a.y, -b.y}) |
            ((uint32_t)rot_bf16(bf16hi_to_f(y[i]), bf16hi_to_f(o), ff{a.z, b.z}, ff{-a.w, -b.w}) << 16);
      }
      y[i] = r;
    }
  } else if (R > 0) {
    // the normed row to shared memory; the rotated dims are then spread over
    // all its lanes (dim e = lane + N k), whatever share of the row they are
    uint32_t* nw = reinterpret_cast<uint32_t*>(nr) + lane * (E / 2);
    uint16_t* rt = nr + D;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) nw[i] = y[i];
    __syncwarp();
    for (int e = lane; e < R; e += N) {
      const bool low = e < half;
      const int j = low ? e : e - half;
      const float2 a = ang.hi[row * half + j];
      const float xe = bf16_to_f(nr[e]), xp = bf16_to_f(nr[low ? e + half : j]);
      const float2 ends = rot_ends(xe, xp, a.x, low ? -a.y : a.y);
      const uint32_t two = bf16x2_rn(ends.x, ends.y);
      uint32_t r = two & 0xFFFFu;
      if (r != two >> 16) {
        const float2 b = ang.lo[row * half + j];
        r = rot_bf16(xe, xp, ff{a.x, b.x}, low ? ff{a.y, b.y} : ff{-a.y, -b.y});
      }
      rt[e] = (uint16_t)r;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const int e = lane * E + 2 * i;                     // R is even: e and e + 1 on the same side
      if (e < R) y[i] = *reinterpret_cast<const uint32_t*>(rt + e);
    }
    __syncwarp();                                         // both rows read before the next item writes them
  }
}

}  // namespace
}  // namespace kvq
