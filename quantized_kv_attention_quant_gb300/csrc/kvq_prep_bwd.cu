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
// One pass over memory: x, dz in, dx out (6 bytes an element with bf16 dz).
// A block takes `rb` rows at a time: it evaluates the rows' rotation angles
// once for all heads into shared memory, then each warp takes one (row, head)
// at a time, VEC consecutive dims of a lane per 16-byte access.  The rotation's
// partner of a dim sits a fixed number of lanes away (one shuffle).  dw stays
// in registers over all rows of a warp, goes to one partial row per block and
// is summed over the blocks in block order by a second small kernel.
#include <algorithm>

#include "kvq_common.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr int kPbWarps = 8;
constexpr int kPbMaxRows = 16;          // rows of a block per step

// cos and sin of p f (f the exact sum of three floats, 0 <= p < 2^24) to
// about 1e-7: p f and its distance to the nearest multiple of pi/2 in
// float-float (two_prod exact, pi/2 in three floats), then the library's
// sine and cosine of the remainder.
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
  const float rr = r.hi + (r.lo + (fmaf(P, f3, a2.lo) - fmaf(k, KVQ_PIO2_3, b2.lo)));
  float s, c;
  sincosf(rr, &s, &c);
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

template <int D>
__device__ __forceinline__ void load_bf16(const uint16_t* row, int lane, float (&v)[D / 32]) {
  using T = Pb<D>;
#pragma unroll
  for (int c = 0; c < T::NC; ++c) {
    const uint16_t* p = row + (c * 32 + lane) * T::VEC;
    uint32_t w[T::VEC / 2];
    if constexpr (T::VEC == 8) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
      w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    } else if constexpr (T::VEC == 4) {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
      w[0] = u.x; w[1] = u.y;
    } else {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    }
#pragma unroll
    for (int i = 0; i < T::VEC / 2; ++i) {
      v[c * T::VEC + 2 * i] = bf16lo_to_f(w[i]);
      v[c * T::VEC + 2 * i + 1] = bf16hi_to_f(w[i]);
    }
  }
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
template <int D>
__device__ __forceinline__ void store_bf16(uint16_t* row, int lane, const float (&v)[D / 32]) {
  using T = Pb<D>;
#pragma unroll
  for (int c = 0; c < T::NC; ++c) {
    uint32_t w[T::VEC / 2];
#pragma unroll
    for (int i = 0; i < T::VEC / 2; ++i)
      w[i] = (uint32_t)f_to_bf16_rn(v[c * T::VEC + 2 * i]) | ((uint32_t)f_to_bf16_rn(v[c * T::VEC + 2 * i + 1]) << 16);
    uint16_t* p = row + (c * 32 + lane) * T::VEC;
    if constexpr (T::VEC == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (T::VEC == 4) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
  }
}

// dz -> R^T dz in place: of a pair (j, j + half) at angle (c, s),
//   dy_j = dz_j c + dz_(j+half) s,  dy_(j+half) = dz_(j+half) c - dz_j s.
// cs: the row's half (cos, sin) pairs; scratch: D floats of this warp, used
// when the pairs do not sit whole lanes apart inside one chunk.
template <int D>
__device__ __forceinline__ void unrotate(float (&z)[D / 32], int lane, int rope, const float2* cs, float* scratch) {
  using T = Pb<D>;
  const int half = rope >> 1, s = half / T::VEC;
  if (half % T::VEC == 0 && 2 * s <= 32) {            // pairs s lanes apart in chunk 0
    const bool in = lane < 2 * s, lo = lane < s;
    const int other = !in ? lane : lo ? lane + s : lane - s;
    const int j0 = (lo ? lane : lane - s) * T::VEC;
#pragma unroll
    for (int i = 0; i < T::VEC; ++i) {
      const float y = __shfl_sync(0xffffffffu, z[i], other);
      if (in) {
        const float2 t = cs[j0 + i];
        z[i] = fmaf(z[i], t.x, lo ? y * t.y : -y * t.y);
      }
    }
  } else if (T::NC == 2 && s == 32) {                 // chunk 0 with chunk 1, in the lane
    if constexpr (T::NC == 2) {
#pragma unroll
      for (int i = 0; i < T::VEC; ++i) {
        const float2 t = cs[lane * T::VEC + i];
        const float a = z[i], b = z[T::VEC + i];
        z[i] = fmaf(a, t.x, b * t.y);
        z[T::VEC + i] = fmaf(b, t.x, -a * t.y);
      }
    }
  } else {                                            // any other even rope_dims
#pragma unroll
    for (int i = 0; i < T::E; ++i) scratch[T::dim(i / T::VEC, lane) + i % T::VEC] = z[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < T::E; ++i) {
      const int e = T::dim(i / T::VEC, lane) + i % T::VEC;
      if (e < rope) {
        const bool lo = e < half;
        const float y = scratch[lo ? e + half : e - half];
        const float2 t = cs[lo ? e : e - half];
        z[i] = fmaf(z[i], t.x, lo ? y * t.y : -y * t.y);
      }
    }
    __syncwarp();
  }
}

// dx of one row from x and dy; adds the row's part of dw.
template <int D, bool WEIGHT>
__device__ __forceinline__ void norm_backward(const float (&x)[D / 32], const float (&dy)[D / 32],
                                              const float (&w)[D / 32], float eps, float (&dx)[D / 32],
                                              float (&dw)[D / 32]) {
  constexpr int E = D / 32;
  float ss = 0.f, gx = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    ss = fmaf(x[i], x[i], ss);
    gx = fmaf(WEIGHT ? dy[i] * w[i] : dy[i], x[i], gx);
  }
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) {
    ss += __shfl_xor_sync(0xffffffffu, ss, m);
    gx += __shfl_xor_sync(0xffffffffu, gx, m);
  }
  const float r = 1.f / sqrtf(ss * (1.f / D) + eps);
  // r^3 gx / D as r (r (r gx / D)): no intermediate of r^3's size
  const float back = r * (r * (r * gx * (1.f / D)));
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const float g = WEIGHT ? dy[i] * w[i] : dy[i];
    dx[i] = fmaf(r, g, -x[i] * back);
    if (WEIGHT) dw[i] = fmaf(dy[i], x[i] * r, dw[i]);
  }
}

struct PbWs {
  uint32_t* status;
  float* part;          // [blocks][2][D]: q and k weight gradients
};

template <int D>
__global__ void __launch_bounds__(kPbWarps * 32)
prep_bwd_kernel(const PrepBwdArgs a, const RopeFreqs freqs, const PbWs ws, const int rb) {
  constexpr int E = D / 32;
  extern __shared__ __align__(16) uint8_t pb_smem[];
  __shared__ int rpos[kPbMaxRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int R = a.L.rope_dims, half = R >> 1, Hq = a.L.n_q, Hkv = a.L.n_kv;
  float2* cs = reinterpret_cast<float2*>(pb_smem);                              // [rb][half]
  float (*freq)[3] = reinterpret_cast<float (*)[3]>(pb_smem + ((size_t)rb * half * 8 + 15) / 16 * 16);
  float* rows = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(freq) + 16 * ((3 * half + 3) / 4));   // [warps][D]
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

  float wq[E], wk[E], dwq[E], dwk[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int e = Pb<D>::dim(i / Pb<D>::VEC, lane) + i % Pb<D>::VEC;
    wq[i] = a.q_raw ? bf16_to_f(__ldg(a.q_w + e)) : 0.f;
    wk[i] = a.k_raw ? bf16_to_f(__ldg(a.k_w + e)) : 0.f;
    dwq[i] = dwk[i] = 0.f;
  }
  const int nq = a.q_raw ? Hq : 0, per_row = nq + (a.k_raw ? Hkv : 0);
  for (long long row0 = (long long)blockIdx.x * rb; row0 < a.n_rows; row0 += (long long)gridDim.x * rb) {
    const int n = (int)min((long long)rb, a.n_rows - row0);
    __syncthreads();                                  // the last step's angles are read
    if (R > 0) {
      if (tid < n) {
        const int row = (int)row0 + tid;
        int lo = 0, hi = a.n_blocks - 1;              // largest block starting at or before the row
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (__ldg(a.off + mid) <= row) lo = mid; else hi = mid - 1;
        }
        rpos[tid] = lo == 0 ? row : P + (row - __ldg(a.off + lo));
      }
      __syncthreads();
      for (int i = tid; i < n * half; i += kPbWarps * 32) {
        const int j = i % half;
        cs[i] = rope_cos_sin_f32(rpos[i / half], freq[j][0], freq[j][1], freq[j][2]);
      }
      __syncthreads();
    }
    for (int it = warp; it < n * per_row; it += kPbWarps) {
      const int rl = it / per_row, h = it % per_row;
      const size_t row = (size_t)row0 + rl;
      float x[E], z[E], dx[E];
      if (h < nq) {
        const size_t o = (row * Hq + h) * D;
        load_bf16<D>(a.q_raw + o, lane, x);
        load_bf16<D>(a.dq_hat + o, lane, z);
        if (R > 0) unrotate<D>(z, lane, R, cs + rl * half, rows + warp * D);
        norm_backward<D, true>(x, z, wq, a.L.eps, dx, dwq);
        store_bf16<D>(a.dq_raw + o, lane, dx);
      } else {
        const size_t o = (row * Hkv + (h - nq)) * D;
        float y[E], dv[E];
        load_bf16<D>(a.k_raw + o, lane, x);
        if (a.dkv_f32) {
          load_f32<D>(static_cast<const float*>(a.dk_hat) + o, lane, z);
          load_f32<D>(static_cast<const float*>(a.dv_hat) + o, lane, y);
        } else {
          load_bf16<D>(static_cast<const uint16_t*>(a.dk_hat) + o, lane, z);
          load_bf16<D>(static_cast<const uint16_t*>(a.dv_hat) + o, lane, y);
        }
        if (R > 0) unrotate<D>(z, lane, R, cs + rl * half, rows + warp * D);
        norm_backward<D, true>(x, z, wk, a.L.eps, dx, dwk);
        if (!a.L.k_eq_v) {
          store_bf16<D>(a.dk_raw + o, lane, dx);
          load_bf16<D>(a.v_raw + o, lane, x);
        }
        norm_backward<D, false>(x, y, wk, a.L.eps, dv, dwk);
        if (a.L.k_eq_v) {
#pragma unroll
          for (int i = 0; i < E; ++i) dx[i] += dv[i];
          store_bf16<D>(a.dk_raw + o, lane, dx);
        } else {
          store_bf16<D>(a.dv_raw + o, lane, dv);
        }
      }
    }
  }
  // the block's weight gradients: over its warps in warp order
  for (int kind = 0; kind < 2; ++kind) {
    if (kind == 0 ? !a.q_raw : !a.k_raw) continue;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < E; ++i)
      rows[warp * D + Pb<D>::dim(i / Pb<D>::VEC, lane) + i % Pb<D>::VEC] = kind == 0 ? dwq[i] : dwk[i];
    __syncthreads();
    for (int e = tid; e < D; e += kPbWarps * 32) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kPbWarps; ++w) s += rows[w * D + e];
      if (gridDim.x == 1) (kind == 0 ? a.dq_w : a.dk_w)[e] = s;
      else ws.part[((size_t)blockIdx.x * 2 + kind) * D + e] = s;
    }
  }
}

// Sums the blocks' weight gradients: block x takes 32 columns of one kind,
// warp w the partial rows w, w + 8, ...; the eight sums join in warp order.
__global__ void __launch_bounds__(kPbWarps * 32)
prep_bwd_weights_kernel(const PrepBwdArgs a, const PbWs ws, const int blocks, const int D) {
  __shared__ float sums[kPbWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch();
  const int kind = blockIdx.y, e = blockIdx.x * 32 + lane;
  float* dst = kind == 0 ? a.dq_w : a.dk_w;
  if (*ws.status != 0 || !dst) return;
  float s = 0.f;
  for (int b = warp; b < blocks; b += kPbWarps) s += ws.part[((size_t)b * 2 + kind) * D + e];
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int w = 1; w < kPbWarps; ++w) s += sums[w][lane];
    dst[e] = s;
  }
}

// Blocks of the grid: two per SM's worth of work at most, so that a call's
// partial rows stay few.
constexpr int kPbMaxBlocks = 608;

template <int D>
cudaError_t launch_t(const PrepBwdArgs& a, const RopeFreqs& f, void* wsp, cudaStream_t st) {
  PbWs ws;
  ws.status = static_cast<uint32_t*>(wsp);
  ws.part = reinterpret_cast<float*>(static_cast<uint8_t*>(wsp) + 256);
  const int per_row = (a.q_raw ? a.L.n_q : 0) + (a.k_raw ? a.L.n_kv : 0), half = a.L.rope_dims / 2;
  // four items a warp per step; angle tables of at most 16 KB
  int rb = std::max(1, std::min(kPbMaxRows, 4 * kPbWarps / per_row));
  if (half > 0) rb = std::max(1, std::min(rb, 2048 / half));
  const size_t smem = ((size_t)rb * half * 8 + 15) / 16 * 16 + 16 * ((3 * half + 3) / 4) + (size_t)kPbWarps * D * 4;
  const int blocks = std::min(kPbMaxBlocks, (a.n_rows + rb - 1) / rb);
  cudaError_t e;
  if ((e = launch_pdl(prep_bwd_kernel<D>, dim3(blocks), dim3(kPbWarps * 32), smem, st, a, f, ws, rb)) != cudaSuccess)
    return e;
  if (blocks == 1) return cudaSuccess;
  return launch_pdl(prep_bwd_weights_kernel, dim3(D / 32, 2), dim3(kPbWarps * 32), 0, st, a, ws, blocks, D);
}

}  // namespace

size_t prep_bwd_ws_bytes(const LayerArgs& L) { return 256 + (size_t)kPbMaxBlocks * 2 * L.D * 4; }

cudaError_t launch_prep_bwd(const PrepBwdArgs& a, const RopeFreqs& f, void* ws, cudaStream_t st) {
  switch (a.L.D) {
    case 64: return launch_t<64>(a, f, ws, st);
    case 128: return launch_t<128>(a, f, ws, st);
    case 256: return launch_t<256>(a, f, ws, st);
    case 512: return launch_t<512>(a, f, ws, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
