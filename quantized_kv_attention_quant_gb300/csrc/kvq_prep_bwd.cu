// kvq_train_prep_backward: the gradient of the training read's preps, the
// per-head RMS norms of q, k and v with the rotation of q and k in the same
// pass.  For a raw row x of D elements, weight w, r = 1 / sqrt(mean(x^2) + eps):
//   forward   y = x r w,  z = R_p y   (R_p turns the first rope_dims dims)
//   backward  dy = R_p^T dz,  g = w dy,
//             dx = r g - x r^3 / D sum(g x),   dw = sum over rows of dy x r
// v has w = 1 and no rotation; on a K = V layer both norms read the same raw
// row and their dx are added before the one rounding to bf16.  The forward's
// roundings pass the gradient through.
//
// One pass over memory: x, dz in, dx out (6 bytes an element with bf16 dz).  Long
// calls are bound by the latency of those loads at 16 warps an SM (16384 rows of 8 +
// 2 + 2 heads of 256, fp32 gradients of keys and values: 84 us, 0.59 of the measured
// copy rate), short ones by the angles and the chain of shuffles of a row (2048 such
// rows in 18 us, 0.31; issue slots 47 % busy): the layout is for loads in flight and
// few instructions.  80 registers, for 24 warps an SM, spilled (125 us); a block
// barrier and a shared table of angles per row took 182.
// Every warp works alone on runs of (row, head) pairs, a row's heads as a rule (q
// heads on some of a block's warps, a donor's keys and values on the others): it
// evaluates a row's angles once, keeps the (cos, sin) of its own dims in registers for all
// heads, and holds the next heads' x and dz in flight.  VEC
// consecutive dims of a lane per 16-byte access; the rotation's partner of a dim
// sits a fixed number of lanes away (one shuffle).  dw stays in registers over
// all rows of a warp, goes to one partial row per block and is summed over the
// blocks in block order by a second small kernel.
#include <algorithm>

#include "kvq_common.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr int kPbWarps = 8;

// cos and sin of p f (f the exact sum of three floats, 0 <= p < 2^24) to
// about 1e-7: p f and its distance r to the nearest multiple of pi/2 in
// float-float (two_prod exact, pi/2 in three floats), then the Taylor series of
// sine and cosine (|r| <= pi/4: the terms left out are below 2e-9 and 6e-10).
__device__ __forceinline__ float2 rope_cos_sin_f32(int p, float f1, float f2, float f3) {
  const float P = (float)p;
  const ff a1 = two_prod(P, f1), a2 = two_prod(P, f2);
  const float k = rintf(__fmul_rn(a1.hi, KVQ_TWO_OVER_PI));
  const ff b1 = two_prod(k, KVQ_PIO2_1), b2 = two_prod(k, KVQ_PIO2_2);
  ff r = {__fsub_rn(a1.hi, b1.hi), 0.f};      // exact
  ff_accum(r, a1.lo);
  ff_accum(r, -b1.lo);
  ff_accum(r, a2.hi);
  ff_accum(r, -b2.hi);
  const float x = r.hi + (r.lo + (fmaf(P, f3, a2.lo) - fmaf(k, KVQ_PIO2_3, b2.lo)));
  const float z = x * x;
  const float s = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), x);
  const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f),
                               -0.5f), 1.f);
  const int q = (int)k & 3;
  const float cc = q & 1 ? s : c, ss = q & 1 ? c : s;
  return make_float2(q == 1 || q == 2 ? -cc : cc, q >= 2 ? -ss : ss);
}

template <int D>
struct Pb {
  static constexpr int E = D / 32;                    // elements per lane
  static constexpr int VEC = E < 8 ? E : 8;           // consecutive ones
  static constexpr int NC = E / VEC;                  // chunks of 32 * VEC dims
  __host__ __device__ static constexpr int dim(int c, int lane) { return (c * 32 + lane) * VEC; }
};

// a lane's E bf16 of a row as they are stored, two to a word
template <int D>
__device__ __forceinline__ void load_raw(const uint16_t* row, int lane, uint32_t (&w)[D / 64]) {
  using T = Pb<D>;
#pragma unroll
  for (int c = 0; c < T::NC; ++c) {
    const uint16_t* p = row + (c * 32 + lane) * T::VEC;
    if constexpr (T::VEC == 8) *reinterpret_cast<uint4*>(w + 4 * c) = *reinterpret_cast<const uint4*>(p);
    else if constexpr (T::VEC == 4) *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
    else w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}
template <int D>
__device__ __forceinline__ void unpack(const uint32_t (&w)[D / 64], float (&v)[D / 32]) {
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    v[2 * i] = bf16lo_to_f(w[i]);
    v[2 * i + 1] = bf16hi_to_f(w[i]);
  }
}
template <int D>
__device__ __forceinline__ void load_bf16(const uint16_t* row, int lane, float (&v)[D / 32]) {
  uint32_t w[D / 64];
  load_raw<D>(row, lane, w);
  unpack<D>(w, v);
}
template <int D>
__device__ __forceinline__ void load_f32(const float* row, int lane, float (&v)[D / 32]) {
  using T = Pb<D>;
#pragma unroll
  for (int c = 0; c < T::NC; ++c) {
    const float* p = row + (c * 32 + lane) * T::VEC;
    if constexpr (T::VEC >= 4) {
#pragma unroll
      for (int i = 0; i < T::VEC; i += 4) {
        const float4 u = __ldg(reinterpret_cast<const float4*>(p + i));
        v[c * T::VEC + i] = u.x; v[c * T::VEC + i + 1] = u.y;
        v[c * T::VEC + i + 2] = u.z; v[c * T::VEC + i + 3] = u.w;
      }
    } else {
      const float2 u = __ldg(reinterpret_cast<const float2*>(p));
      v[0] = u.x; v[1] = u.y;
    }
  }
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
template <int D>
__device__ __forceinline__ void store_bf16(uint16_t* row, int lane, const float (&v)[D / 32]) {
  using T = Pb<D>;
#pragma unroll
  for (int c = 0; c < T::NC; ++c) {
    uint32_t w[T::VEC / 2];
#pragma unroll
    for (int i = 0; i < T::VEC / 2; ++i)
      w[i] = bf16_pair(v[c * T::VEC + 2 * i], v[c * T::VEC + 2 * i + 1]);
    uint16_t* p = row + (c * 32 + lane) * T::VEC;
    if constexpr (T::VEC == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (T::VEC == 4) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
  }
}

// How a lane finds the partners of its dims in the rotation of `rope` dims.
enum : int { kNoRope, kLanes, kChunks, kAny };   // none; whole lanes apart in chunk 0; chunk 0 with chunk 1; else

template <int D>
__device__ __forceinline__ int rope_kind(int rope) {
  using T = Pb<D>;
  const int half = rope >> 1;
  if (half == 0) return kNoRope;
  if (half % T::VEC == 0 && 2 * (half / T::VEC) <= 32) return kLanes;
  if (T::NC == 2 && half == 32 * T::VEC) return kChunks;
  return kAny;
}

// dz -> R^T dz in place: of a pair (j, j + half) at angle (c, s),
//   dy_j = dz_j c + dz_(j+half) s,  dy_(j+half) = dz_(j+half) c - dz_j s.
// cs: the (c, s) of this lane's dims, s with its sign (kLanes, kChunks);
// table, scratch: the row's pairs and D floats of this warp (kAny).
template <int D>
__device__ __forceinline__ void unrotate(float (&z)[D / 32], int lane, int rope, int kind,
                                         const float2 (&cs)[Pb<D>::VEC], const float2* table, float* scratch) {
  using T = Pb<D>;
  if (kind == kLanes) {                               // (lanes past the rotated dims hold c = 1, s = 0)
    const int s = (rope >> 1) / T::VEC, other = lane < s ? lane + s : lane < 2 * s ? lane - s : lane;
#pragma unroll
    for (int i = 0; i < T::VEC; ++i) z[i] = fmaf(z[i], cs[i].x, __shfl_sync(0xffffffffu, z[i], other) * cs[i].y);
  } else if (kind == kChunks) {
    if constexpr (T::NC == 2) {
#pragma unroll
      for (int i = 0; i < T::VEC; ++i) {
        const float a = z[i], b = z[T::VEC + i];
        z[i] = fmaf(a, cs[i].x, b * cs[i].y);
        z[T::VEC + i] = fmaf(b, cs[i].x, -a * cs[i].y);
      }
    }
  } else if (kind == kAny) {
    const int half = rope >> 1;
#pragma unroll
    for (int i = 0; i < T::E; ++i) scratch[T::dim(i / T::VEC, lane) + i % T::VEC] = z[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < T::E; ++i) {
      const int e = T::dim(i / T::VEC, lane) + i % T::VEC;
      if (e < rope) {
        const bool lo = e < half;
        const float y = scratch[lo ? e + half : e - half];
        const float2 t = table[lo ? e : e - half];
        z[i] = fmaf(z[i], t.x, lo ? y * t.y : -y * t.y);
      }
    }
    __syncwarp();
  }
}

template <int NW>
__device__ __forceinline__ float weight(const uint32_t (&w)[NW], int i) {
  return i & 1 ? bf16hi_to_f(w[i / 2]) : bf16lo_to_f(w[i / 2]);
}

// dx of one row from x and dy; adds the row's part of dw.
template <int D, bool WEIGHT>
__device__ __forceinline__ void norm_backward(const float (&x)[D / 32], const float (&dy)[D / 32],
                                              const uint32_t (&w)[D / 64], float eps, float (&dx)[D / 32],
                                              float (&dw)[D / 32]) {
  constexpr int E = D / 32;
  float ss = 0.f, gx = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    ss = fmaf(x[i], x[i], ss);
    gx = fmaf(WEIGHT ? dy[i] * weight(w, i) : dy[i], x[i], gx);
  }
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) {
    ss += __shfl_xor_sync(0xffffffffu, ss, m);
    gx += __shfl_xor_sync(0xffffffffu, gx, m);
  }
  const float ms = fmaf(ss, 1.f / D, eps), r0 = rsqrtf(ms);
  const float r = r0 * fmaf(-0.5f * ms * r0, r0, 1.5f);     // one Newton step: within 2^-23
  // r^3 gx / D as r (r (r gx / D)): no intermediate of r^3's size
  const float back = r * (r * (r * gx * (1.f / D)));
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const float g = WEIGHT ? dy[i] * weight(w, i) : dy[i];
    dx[i] = fmaf(r, g, -x[i] * back);
    if (WEIGHT) dw[i] = fmaf(dy[i], x[i] * r, dw[i]);
  }
}

struct PbWs {
  uint32_t* status;
  float* part;          // [blocks][2][D]: q and k weight gradients
};

// The share of a call's work: qw of a block's warps take q heads, the others keys
// and values, in runs of q_run or kv_run consecutive (row, head) pairs.
struct PbShare { int qw, q_run, kv_run; };

template <int D>
__global__ void __launch_bounds__(kPbWarps * 32, 2)
prep_bwd_kernel(const PrepBwdArgs a, const RopeFreqs freqs, const PbWs ws, const PbShare sh) {
  using T = Pb<D>;
  constexpr int E = T::E, NW = D / 64;
  extern __shared__ __align__(16) uint8_t pb_smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int R = a.L.rope_dims, half = R >> 1, Hq = a.L.n_q, Hkv = a.L.n_kv;
  float (*freq)[3] = reinterpret_cast<float (*)[3]>(pb_smem);
  float* rows = reinterpret_cast<float*>(pb_smem + 16 * ((3 * half + 3) / 4));                  // [warps][D]
  float2* table = reinterpret_cast<float2*>(rows + kPbWarps * D) + warp * half;                 // [warps][half]
  if (R > 0) stage_freqs(freqs.f, half, freq);
  pdl_wait();
  pdl_launch();
  // the layout rules; every block looks at all of them, so that a layout that
  // breaks one leaves every output as it was
  bool bad = false;
  const int P = __ldg(a.off + 1);
  for (int b = tid; b < a.n_blocks; b += kPbWarps * 32) {
    const int o0 = __ldg(a.off + b), o1 = __ldg(a.off + b + 1);
    bad |= !(o0 >= 0 && o0 <= o1 && o1 <= a.n_rows && P >= 0 && (b == 0 ? o0 == 0 : o0 >= P) &&
             (b + 1 < a.n_blocks || o1 == a.n_rows));
  }
  bad = __syncthreads_or(bad);
  if (blockIdx.x == 0 && tid == 0) *ws.status = bad ? 1u << KVQ_DEV_BADSEQ : 0u;
  if (bad) return;

  const int qw = sh.qw;
  const bool is_q = warp < qw;
  const int heads = is_q ? Hq : Hkv, n_warps = (is_q ? qw : kPbWarps - qw) * gridDim.x, run = is_q ? sh.q_run : sh.kv_run;
  const int me = is_q ? (int)blockIdx.x * qw + warp : (int)blockIdx.x * (kPbWarps - qw) + warp - qw;
  const int kind = rope_kind<D>(R);
  float dw[E];
  uint32_t w[NW];                                     // the weights (only 2-byte aligned), two to a word
  {
    const uint16_t* src = is_q ? a.q_w : a.k_w;
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      const int e = T::dim(i / T::VEC, lane) + i % T::VEC;
      w[i / 2] = (uint32_t)__ldg(src + e) | ((uint32_t)__ldg(src + e + 1) << 16);
      dw[i] = dw[i + 1] = 0.f;
    }
  }
  // this warp's runs me, me + n_warps, ... of the (row, head) pairs
  struct At { int row, h, left; };
  const long long first = (long long)me * run, jump = (long long)(n_warps - 1) * run;
  const int jump_rows = (int)(jump / heads), jump_heads = (int)(jump % heads);
  At at = {(int)min((long long)a.n_rows, first / heads), (int)(first % heads), run};
  auto step = [&](At& p) {
    if (--p.left == 0) {
      p.left = run;
      p.row += jump_rows;
      p.h += jump_heads;
      if (p.h >= heads) {
        p.h -= heads;
        ++p.row;
      }
    }
    if (++p.h == heads) {
      p.h = 0;
      ++p.row;
    }
  };
  float2 cs[T::VEC];
  int at_row = -1;
  auto angles = [&](int row) {                        // the row's rotation: table, and this lane's part of it
    if (R == 0 || row == at_row) return;
    at_row = row;
    int lo = 0, hi = a.n_blocks - 1;                  // largest block starting at or before the row
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(a.off + mid) <= row) lo = mid; else hi = mid - 1;
    }
    const int pos = lo == 0 ? row : P + (row - __ldg(a.off + lo));
    __syncwarp();
    for (int j = lane; j < half; j += 32) table[j] = rope_cos_sin_f32(pos, freq[j][0], freq[j][1], freq[j][2]);
    __syncwarp();
    if (kind == kLanes) {
      const int s = half / T::VEC, j0 = (lane < s ? lane : lane - s) * T::VEC;
#pragma unroll
      for (int i = 0; i < T::VEC; ++i) {
        cs[i] = lane < 2 * s ? table[j0 + i] : make_float2(1.f, 0.f);
        if (lane >= s) cs[i].y = -cs[i].y;
      }
    } else if (kind == kChunks) {
#pragma unroll
      for (int i = 0; i < T::VEC; ++i) cs[i] = table[lane * T::VEC + i];
    }
  };
  if (is_q) {
    // x and dz of the next AHEAD heads in flight
    constexpr int AHEAD = D <= 256 ? 2 : 0;           // (head_dim 512: no registers for it)
    uint32_t xr[AHEAD + 1][NW], zr[AHEAD + 1][NW];
    At ahead = at;
    auto fetch = [&](uint32_t (&x)[NW], uint32_t (&z)[NW]) {
      if (ahead.row >= a.n_rows) return;
      const size_t o = ((size_t)ahead.row * heads + ahead.h) * D;
      load_raw<D>(a.q_raw + o, lane, x);
      load_raw<D>(a.dq_hat + o, lane, z);
      step(ahead);
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) fetch(xr[i], zr[i]);
    while (at.row < a.n_rows) {
#pragma unroll
      for (int b = 0; b < AHEAD + 1; ++b) {
        if (at.row >= a.n_rows) break;
        fetch(xr[(b + AHEAD) % (AHEAD + 1)], zr[(b + AHEAD) % (AHEAD + 1)]);
        angles(at.row);
        float x[E], z[E], dx[E];
        unpack<D>(xr[b], x);
        unpack<D>(zr[b], z);
        unrotate<D>(z, lane, R, kind, cs, table, rows + warp * D);
        norm_backward<D, true>(x, z, w, a.L.eps, dx, dw);
        store_bf16<D>(a.dq_raw + ((size_t)at.row * heads + at.h) * D, lane, dx);
        step(at);
      }
    }
  } else {
    auto gradient = [&](const void* g, size_t o, float (&z)[E]) {
      if (a.dkv_f32) load_f32<D>(static_cast<const float*>(g) + o, lane, z);
      else load_bf16<D>(static_cast<const uint16_t*>(g) + o, lane, z);
    };
    for (; at.row < a.n_rows; step(at)) {
      const size_t o = ((size_t)at.row * heads + at.h) * D;
      // all four rows in flight at once; at head_dim 512 v's after k's
      constexpr bool EARLY = D <= 256;
      float z[E], y[E], dx[E];
      uint32_t xr[NW], vr[NW];
      auto load_v = [&]() {
        if (!a.L.k_eq_v) load_raw<D>(a.v_raw + o, lane, vr);
        gradient(a.dv_hat, o, y);
      };
      load_raw<D>(a.k_raw + o, lane, xr);
      gradient(a.dk_hat, o, z);
      if (EARLY) load_v();
      angles(at.row);
      {
        float x[E];
        unpack<D>(xr, x);
        unrotate<D>(z, lane, R, kind, cs, table, rows + warp * D);
        norm_backward<D, true>(x, z, w, a.L.eps, dx, dw);
      }
      if (!a.L.k_eq_v) store_bf16<D>(a.dk_raw + o, lane, dx);
      if (!EARLY) load_v();
      float x[E], dv[E];
      unpack<D>(a.L.k_eq_v ? xr : vr, x);
      norm_backward<D, false>(x, y, w, a.L.eps, dv, dw);
      if (a.L.k_eq_v) {
#pragma unroll
        for (int i = 0; i < E; ++i) dx[i] += dv[i];
        store_bf16<D>(a.dk_raw + o, lane, dx);
      } else {
        store_bf16<D>(a.dv_raw + o, lane, dv);
      }
    }
  }
  // the block's weight gradients: over its warps in warp order
  __syncwarp();
#pragma unroll
  for (int i = 0; i < E; ++i) rows[warp * D + T::dim(i / T::VEC, lane) + i % T::VEC] = dw[i];
  __syncthreads();
  for (int i = tid; i < 2 * D; i += kPbWarps * 32) {
    const int kv = i / D, e = i % D, w0 = kv ? qw : 0, w1 = kv ? kPbWarps : qw;
    if (w0 == w1) continue;
    float s = 0.f;
    for (int x = w0; x < w1; ++x) s += rows[x * D + e];
    if (gridDim.x == 1) (kv ? a.dk_w : a.dq_w)[e] = s;
    else ws.part[((size_t)blockIdx.x * 2 + kv) * D + e] = s;
  }
}

// Sums the blocks' weight gradients: block x takes 32 columns of one kind,
// warp w the partial rows w, w + 32, ...; the sums join in warp order.
constexpr int kPbSumWarps = 32;
__global__ void __launch_bounds__(kPbSumWarps * 32)
prep_bwd_weights_kernel(const PrepBwdArgs a, const PbWs ws, const int blocks, const int D) {
  __shared__ float sums[kPbSumWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch();
  const int kind = blockIdx.y, e = blockIdx.x * 32 + lane;
  float* dst = kind == 0 ? a.dq_w : a.dk_w;
  if (*ws.status != 0 || !dst) return;
  float s = 0.f;
#pragma unroll 10
  for (int b = warp; b < blocks; b += kPbSumWarps) s += ws.part[((size_t)b * 2 + kind) * D + e];
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int w = 1; w < kPbSumWarps; ++w) s += sums[w][lane];
    dst[e] = s;
  }
}

// Most blocks of a grid (their partial rows are kept): two per SM, as many as are resident.
constexpr int kPbMaxBlocks = 304;

template <int D>
cudaError_t launch_t(const PrepBwdArgs& a, const RopeFreqs& f, void* wsp, int num_sms, cudaStream_t st) {
  PbWs ws;
  ws.status = static_cast<uint32_t*>(wsp);
  ws.part = reinterpret_cast<float*>(static_cast<uint8_t*>(wsp) + 256);
  const int half = a.L.rope_dims / 2, nq = a.q_raw ? a.L.n_q : 0, nkv = a.k_raw ? a.L.n_kv : 0;
  // warps in proportion to the bytes of a row
  const long long q_bytes = 6LL * nq, kv_bytes = (long long)nkv * ((a.L.k_eq_v ? 4 : 8) + (a.dkv_f32 ? 8 : 4));
  const int qw = nkv == 0 ? kPbWarps
                 : nq == 0 ? 0
                           : (int)std::max<long long>(1, std::min<long long>(kPbWarps - 1, (kPbWarps * q_bytes + (q_bytes + kv_bytes) / 2) / (q_bytes + kv_bytes)));
  // blocks: enough that no warp has more than one head, two per SM at most
  const int kw = kPbWarps - qw;
  const long long want = std::max(qw ? ((long long)a.n_rows * nq + qw - 1) / qw : 0,
                                  kw ? ((long long)a.n_rows * nkv + kw - 1) / kw : 0);
  // (a handful of heads goes to one block, which needs no second kernel)
  const int blocks = want <= 3 ? 1 : (int)std::min<long long>(std::min(kPbMaxBlocks, 2 * num_sms), want);
  // a row's heads in one run (its angles are evaluated once: 2048 rows of 8 heads of
  // 256 took 18.2 us so, 20.3 in runs of 4, 22.9 in one run per warp, 16384 rows 84.7,
  // 107 and 111), fewer where there are not as many pairs for every warp
  auto run_of = [&](int warps, int heads) {
    const long long all = (long long)a.n_rows * heads, n = std::max(1LL, (long long)warps * blocks);
    return (int)std::max(1LL, std::min<long long>(heads, (all + n - 1) / n));
  };
  const PbShare sh = {qw, run_of(qw, nq), run_of(kw, nkv)};
  const size_t smem = 16 * ((3 * half + 3) / 4) + (size_t)kPbWarps * (D * 4 + half * 8);      // at most 35 KB
  cudaError_t e;
  if ((e = launch_pdl(prep_bwd_kernel<D>, dim3(blocks), dim3(kPbWarps * 32), smem, st, a, f, ws, sh)) != cudaSuccess)
    return e;
  if (blocks == 1) return cudaSuccess;
  return launch_pdl(prep_bwd_weights_kernel, dim3(D / 32, 2), dim3(kPbSumWarps * 32), 0, st, a, ws, blocks, D);
}

}  // namespace

size_t prep_bwd_ws_bytes(const LayerArgs& L) { return 256 + (size_t)kPbMaxBlocks * 2 * L.D * 4; }

cudaError_t launch_prep_bwd(const PrepBwdArgs& a, const RopeFreqs& f, void* ws, int num_sms, cudaStream_t st) {
  switch (a.L.D) {
    case 64: return launch_t<64>(a, f, ws, num_sms, st);
    case 128: return launch_t<128>(a, f, ws, num_sms, st);
    case 256: return launch_t<256>(a, f, ws, num_sms, st);
    case 512: return launch_t<512>(a, f, ws, num_sms, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
