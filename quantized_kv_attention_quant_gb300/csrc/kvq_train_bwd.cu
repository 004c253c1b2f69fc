// attn_train_backward: the gradient of the training read (kvq_train.cu) by
// q_hat, k_hat and v_hat under the prefix-shared layout.  With the row's
// log-sum-exp from the forward,
//   P = exp(S - lse), S = q k;  dP = dO v;  dS = P (dP - delta), delta = dO . O
//   dq = dS k,  dk = dS^T q,  dv = P^T dO   (dk, dv over the kv head's q heads)
// A row that sees one key has P = 1 whatever its score: its dS is 0 exactly.
//
// Plain kernels: one warp per (row, head) walks the keys it sees for dq, one
// warp per (key, kv head) walks the rows that see it for dk and dv, all in
// fp32 with the head dims spread over the lanes.
#include "kvq_common.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr int kWarps = 8;

struct BwdWs {
  uint32_t* status;     // status word; word 1: 1 when the layout is valid
  float* delta;         // [n_rows][n_q]
};

BwdWs bwd_carve(void* ws) {
  BwdWs w;
  w.status = static_cast<uint32_t*>(ws);
  w.delta = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 256);
  return w;
}

// One block: the layout rules of include/kvq.h.
__global__ void __launch_bounds__(256) layout_kernel(const TrainBwdArgs a, BwdWs w) {
  __shared__ int bad;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  const int P = a.off[1];
  for (int b = threadIdx.x; b < a.n_blocks; b += blockDim.x) {
    const int o0 = a.off[b], o1 = a.off[b + 1];
    const bool ok = o0 >= 0 && o0 <= o1 && o1 <= a.n_rows && P >= 0 && (b == 0 ? o0 == 0 : o0 >= P) &&
                    (b + 1 < a.n_blocks || o1 == a.n_rows) && o1 - o0 <= a.max_block_rows;
    if (!ok) atomicOr(&bad, 1);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    w.status[0] = bad ? 1u << KVQ_DEV_BADSEQ : 0u;
    w.status[1] = bad ? 0u : 1u;
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// block of packed row r (largest b with off[b] <= r and a non-empty block)
__device__ __forceinline__ int find_block(const int32_t* off, int n, int r) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(off + mid) <= r) lo = mid; else hi = mid - 1;
  }
  return lo;
}

template <int E>
__device__ __forceinline__ void load_row(const uint16_t* p, int lane, float (&v)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i) v[i] = bf16_to_f(__ldg(p + i * 32 + lane));
}
template <int E>
__device__ __forceinline__ float dot(const float (&x)[E], const float (&y)[E]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) s = fmaf(x[i], y[i], s);
  return warp_sum(s);
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) dq_kernel(const TrainBwdArgs a, BwdWs w) {
  constexpr int E = D / 32;
  if (w.status[1] == 0) return;
  const int lane = threadIdx.x & 31;
  const long long it = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (it >= (long long)a.n_rows * a.L.n_q) return;
  const int r = (int)(it / a.L.n_q), h = (int)(it % a.L.n_q), kvh = h / a.L.G;
  const int b = find_block(a.off, a.n_blocks, r), P = a.off[1], o0 = a.off[b];
  const int pos = b == 0 ? r : P + (r - o0), lo = a.L.window > 0 ? max(0, pos - a.L.window + 1) : 0;
  float q[E], dO[E], acc[E];
  load_row<E>(a.q + (size_t)it * D, lane, q);
  load_row<E>(a.d_out + (size_t)it * D, lane, dO);
  float dl = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const size_t o = (size_t)it * D + i * 32 + lane;
    const float ov = a.out_f32 ? static_cast<const float*>(a.out)[o] : bf16_to_f(static_cast<const uint16_t*>(a.out)[o]);
    dl = fmaf(dO[i], ov, dl);
    acc[i] = 0.f;
  }
  dl = warp_sum(dl);
  if (lane == 0) w.delta[it] = dl;
  const float lse = a.lse[it];
  for (int p = lo; p <= pos && lo != pos; ++p) {
    const int j = b == 0 || p < P ? p : o0 + (p - P);
    float k[E], v[E];
    load_row<E>(a.k + ((size_t)j * a.L.n_kv + kvh) * D, lane, k);
    load_row<E>(a.v + ((size_t)j * a.L.n_kv + kvh) * D, lane, v);
    const float ds = expf(dot(q, k) - lse) * (dot(dO, v) - dl);
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = fmaf(ds, k[i], acc[i]);
  }
#pragma unroll
  for (int i = 0; i < E; ++i) a.dq[(size_t)it * D + i * 32 + lane] = f_to_bf16_rn(acc[i]);
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) dkv_kernel(const TrainBwdArgs a, BwdWs w) {
  constexpr int E = D / 32;
  if (w.status[1] == 0) return;
  const int lane = threadIdx.x & 31;
  const long long it = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (it >= (long long)a.n_rows * a.L.n_kv) return;
  const int j = (int)(it / a.L.n_kv), kvh = (int)(it % a.L.n_kv);
  const int bj = find_block(a.off, a.n_blocks, j), P = a.off[1];
  const int pj = bj == 0 ? j : P + (j - a.off[bj]);
  const int hi = a.L.window > 0 ? pj + a.L.window - 1 : 1 << 30;    // the newest position that sees the key
  float k[E], v[E], dk[E], dv[E];
  load_row<E>(a.k + (size_t)it * D, lane, k);
  load_row<E>(a.v + (size_t)it * D, lane, v);
#pragma unroll
  for (int i = 0; i < E; ++i) dk[i] = dv[i] = 0.f;
  // the key's own block from the key on, then (a prefix key) every branch
  for (int b = bj; b < (bj == 0 ? a.n_blocks : bj + 1); ++b) {
    const int o0 = a.off[b], o1 = a.off[b + 1];
    for (int r = b == bj ? j : o0; r < o1; ++r) {
      const int pos = b == 0 ? r : P + (r - o0);
      if (pos > hi) break;
      const bool one = pos == 0 || a.L.window == 1;
      for (int h = kvh * a.L.G; h < (kvh + 1) * a.L.G; ++h) {
        const size_t rh = (size_t)r * a.L.n_q + h;
        float q[E], dO[E];
        load_row<E>(a.q + rh * D, lane, q);
        load_row<E>(a.d_out + rh * D, lane, dO);
        const float p = expf(dot(q, k) - a.lse[rh]);
        const float ds = one ? 0.f : p * (dot(dO, v) - w.delta[rh]);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          dk[i] = fmaf(ds, q[i], dk[i]);
          dv[i] = fmaf(p, dO[i], dv[i]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const size_t o = (size_t)it * D + i * 32 + lane;
    if (a.dkv_f32) {
      float* pk = static_cast<float*>(a.dk) + o;
      float* pv = static_cast<float*>(a.dv) + o;
      *pk = a.accumulate ? *pk + dk[i] : dk[i];
      *pv = a.accumulate ? *pv + dv[i] : dv[i];
    } else {
      static_cast<uint16_t*>(a.dk)[o] = f_to_bf16_rn(dk[i]);
      static_cast<uint16_t*>(a.dv)[o] = f_to_bf16_rn(dv[i]);
    }
  }
}

template <int D>
cudaError_t launch_t(const TrainBwdArgs& a, BwdWs w, cudaStream_t st) {
  const long long nq = ((long long)a.n_rows * a.L.n_q + kWarps - 1) / kWarps;
  const long long nk = ((long long)a.n_rows * a.L.n_kv + kWarps - 1) / kWarps;
  if (nq > 0x7fffffffLL || nk > 0x7fffffffLL) return cudaErrorInvalidValue;
  layout_kernel<<<1, 256, 0, st>>>(a, w);
  dq_kernel<D><<<(unsigned)nq, kWarps * 32, 0, st>>>(a, w);
  dkv_kernel<D><<<(unsigned)nk, kWarps * 32, 0, st>>>(a, w);
  return cudaGetLastError();
}

}  // namespace

size_t train_bwd_ws_bytes(const LayerArgs& L, int n_blocks, int n_rows, int max_block_rows) {
  return 256 + (size_t)n_rows * L.n_q * 4;
}

cudaError_t launch_train_bwd(const TrainBwdArgs& a, void* ws, cudaStream_t st) {
  const BwdWs w = bwd_carve(ws);
  switch (a.L.D) {
    case 64: return launch_t<64>(a, w, st);
    case 128: return launch_t<128>(a, w, st);
    case 256: return launch_t<256>(a, w, st);
    case 512: return launch_t<512>(a, w, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
