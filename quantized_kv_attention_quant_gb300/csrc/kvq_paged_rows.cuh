// The first kernel of the paged reads: q prep of every row, the outputs of
// rows that read nothing, and the plan of the calls that cut their keys into
// equal shares.
#pragma once
#include "kvq_paged.cuh"
#include "kvq_qrows.cuh"

namespace kvq {
namespace {

// Rows of a read are taken in groups of at most TG consecutive rows of one
// sequence.  Group u of sequence s with base(s) = floor(row_offsets[s] / TG) + s
// is its rows TG (u - base(s)) ..; groups past a sequence's rows are empty.
struct PagedGroup {
  int s;        // sequence
  int row0;     // first row (packed)
  int nt;       // rows whose position the table can hold
  int bad;      // rows past it
  int p0;       // position of the first row
  int lo, hi;   // oldest and newest position that a row of the group sees
  int kt0;      // lo rounded down to 64
  int tiles;    // key tiles of KT from there (0: nothing to read)
};

__device__ __forceinline__ PagedGroup paged_group(const PagedRows& r, const PagedArgs& pg, int window, int TG, int KT,
                                                  int u) {
  PagedGroup g;
  int t0 = 0, take;
  if (r.row_offsets == nullptr) {
    g.s = u;
    g.row0 = u;
    g.p0 = __ldg(r.start + u);
    take = 1;
  } else {
    int lo = 0, hi = r.n_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(r.row_offsets + mid) / TG + mid <= u) lo = mid; else hi = mid - 1;
    }
    const SeqRows sr = paged_seq_rows(r, lo);
    g.s = lo;
    t0 = (u - (sr.off / TG + lo)) * TG;
    take = sr.off >= 0 && sr.off + sr.rows <= r.n_rows ? max(0, min(TG, sr.rows - t0)) : 0;
    g.row0 = sr.off + t0;
    g.p0 = sr.start >= 0 ? sr.start + t0 : -1;
  }
  if (g.p0 < 0) take = 0;                                 // an idle sequence
  g.nt = min(take, max(0, pg.limit - g.p0));
  g.bad = take - g.nt;
  g.hi = g.p0 + g.nt - 1;
  g.lo = window > 0 ? max(0, g.p0 - window + 1) : 0;
  g.kt0 = g.lo & ~63;
  g.tiles = g.nt > 0 ? (g.hi - g.kt0) / KT + 1 : 0;
  return g;
}

inline int paged_groups(const PagedRows& r, int TG) {
  return r.row_offsets ? r.n_rows / TG + r.n_seqs : r.n_rows;
}

// Rows without keys: an idle sequence's are zeros, those past the table NaN.
template <int D>
__device__ __forceinline__ void paged_fill_rows(const DecodeArgs& a, const PagedArgs& pg, int rb, int bx) {
  const int limit = pg.limit;
  for (int row = bx * rb; row < min(a.n_rows, bx * rb + rb); ++row) {
    int p, start;
    if (a.row_offsets == nullptr) {
      start = p = __ldg(a.pos + row);
    } else {
      const RowInfo ri = row_info(a, row);
      start = __ldg(a.pos + ri.s);
      p = ri.p;
    }
    if (start >= 0 && p >= 0 && p < limit) continue;
    const float v = start < 0 ? 0.f : __int_as_float(0x7FC00000);
    const size_t n = (size_t)a.L.n_q * D, at = (size_t)row * n;
    for (size_t i = threadIdx.x; i < n; i += kQrWarps * 32) {
      if (a.out_f32) reinterpret_cast<float*>(a.out)[at + i] = v;
      else reinterpret_cast<uint16_t*>(a.out)[at + i] = start < 0 ? 0 : 0x7FC0;
    }
  }
}

// prefix[u] = key tiles of the groups before u (one block), and the call's
// status word.
__device__ __forceinline__ void paged_plan_block(const PagedRows& r, const PagedArgs& pg, int window, int TG, int KT,
                                                 int n_groups, long long* prefix, uint32_t* status) {
  __shared__ int wsum[kQrWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  long long base = 0;
  bool bad = false;
  for (int u0 = 0; u0 < n_groups; u0 += kQrWarps * 32) {
    const int u = u0 + tid;
    int t = 0;
    if (u < n_groups) {
      const PagedGroup g = paged_group(r, pg, window, TG, KT, u);
      t = g.tiles;
      bad |= g.bad > 0;
    }
    int inc = t;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, inc, m);
      if (lane >= m) inc += o;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    long long before = base, total = 0;
    for (int w = 0; w < kQrWarps; ++w) {
      if (w < warp) before += wsum[w];
      total += wsum[w];
    }
    if (u < n_groups) prefix[u] = before + inc - t;
    base += total;
    __syncthreads();
  }
  const bool any = __syncthreads_or(bad);
  if (tid == 0) {
    prefix[n_groups] = base;
    *status = any ? (1u << KVQ_DEV_BADSEQ) : 0u;
  }
}

// order = the groups, those with the most key tiles first (one block): a
// counting sort over the tile counts; the order of equal ones is open (it
// decides only which CTA takes a group).
constexpr int kOrderBins = 2048;
__device__ __forceinline__ void paged_order_block(const PagedRows& r, const PagedArgs& pg, int window, int TG, int KT,
                                                  int n_groups, int32_t* order, uint32_t* status) {
  __shared__ int bins[kOrderBins];
  __shared__ int wsum[kQrWarps];
  constexpr int PER = kOrderBins / (kQrWarps * 32);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < kOrderBins; i += kQrWarps * 32) bins[i] = 0;
  __syncthreads();
  bool bad = false;
  auto bin_of = [](int tiles) { return kOrderBins - 1 - min(tiles, kOrderBins - 1); };   // most first
  for (int u = tid; u < n_groups; u += kQrWarps * 32) {
    const PagedGroup g = paged_group(r, pg, window, TG, KT, u);
    bad |= g.bad > 0;
    atomicAdd(&bins[bin_of(g.tiles)], 1);
  }
  __syncthreads();
  int mine[PER], sum = 0;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    mine[k] = sum;
    sum += bins[PER * tid + k];
  }
  int inc = sum;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, inc, m);
    if (lane >= m) inc += o;
  }
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  int before = inc - sum;
  for (int w = 0; w < warp; ++w) before += wsum[w];
#pragma unroll
  for (int k = 0; k < PER; ++k) bins[PER * tid + k] = before + mine[k];
  const bool any = __syncthreads_or(bad);
  for (int u = tid; u < n_groups; u += kQrWarps * 32) {
    const PagedGroup g = paged_group(r, pg, window, TG, KT, u);
    order[atomicAdd(&bins[bin_of(g.tiles)], 1)] = u;
  }
  if (tid == 0) *status = any ? (1u << KVQ_DEV_BADSEQ) : 0u;
}

// Block 0 makes the plan (the tile prefix, or the order of the groups) and
// writes the status word, the others prep rb rows each.
template <int D>
__global__ void __launch_bounds__(kQrWarps * 32)
paged_prep_kernel(const DecodeArgs a, const PagedArgs pg, const RopeFreqs freqs, const int rb, const int TG,
                  const int KT, const int n_groups, long long* prefix, int32_t* order, uint32_t* status) {
  if (blockIdx.x == 0) {
    pdl_wait();
    pdl_launch();
    PagedRows r = {a.row_offsets, a.pos, a.n_seqs, a.n_rows};
    if (prefix) paged_plan_block(r, pg, a.L.window, TG, KT, n_groups, prefix, status);
    else paged_order_block(r, pg, a.L.window, TG, KT, n_groups, order, status);
  } else {
    qprep_rows_block<D>(a, freqs, rb, blockIdx.x - 1);
    paged_fill_rows<D>(a, pg, rb, blockIdx.x - 1);
  }
}

// q_hat as f16 to q16 [n_rows][n_q][D]; `spare`: a word that qprep_rows_block
// may clear in the place of a status word.
template <int D>
cudaError_t launch_paged_prep(const PagedReadArgs& a, const RopeFreqs& f, int TG, int KT, int n_groups, uint16_t* q16,
                              long long* prefix, int32_t* order, uint32_t* status, uint32_t* spare,
                              cudaStream_t st) {
  DecodeArgs d = {};
  d.L = a.L;
  d.n_seqs = a.r.n_seqs;
  d.n_rows = a.r.n_rows;
  d.row_offsets = a.r.row_offsets;
  d.pos = a.r.start;
  d.q_raw = a.q_raw;
  d.q_w = a.q_w;
  d.out = a.out;
  d.out_f32 = a.out_f32;
  d.q_prepped = a.q_prepped;
  d.ws.status = spare;
  d.ws.q16 = q16;
  const int rb = qprep_rows_rb(a.L);
  const int nq = (a.r.n_rows + rb - 1) / rb;
  return launch_pdl(paged_prep_kernel<D>, dim3(nq + 1), dim3(kQrWarps * 32), qprep_rows_smem(a.L, rb), st, d, a.pg, f,
                    rb, TG, KT, n_groups, prefix, order, status);
}

}  // namespace
}  // namespace kvq
