// The first kernel of the paged reads: q prep of every row, the outputs of
// rows that read nothing, and the plan of the calls that cut their keys into
// equal shares.
#pragma once
#include <algorithm>

#include "kvq_paged.cuh"
#include "kvq_paged_prep.cuh"

namespace kvq {
namespace {

constexpr int kPrWarps = 8;           // of the prep kernel's blocks
constexpr int kNoSeq = -2;            // in the place of a start: the row lies behind the last sequence

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

// Group u, which belongs to sequence s.
__device__ __forceinline__ PagedGroup paged_group_of(const PagedRows& r, const PagedArgs& pg, int window, int TG, int KT,
                                                     int u, int s) {
  PagedGroup g;
  int t0 = 0, take;
  g.s = s;
  if (r.row_offsets == nullptr) {
    g.row0 = u;
    g.p0 = __ldg(r.start + u);
    take = 1;
  } else {
    const SeqRows sr = paged_seq_rows(r, s);
    t0 = (u - (sr.off / TG + s)) * TG;
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

// Group u; WARP: u is the same in all lanes, which search its sequence together.
template <bool WARP>
__device__ __forceinline__ PagedGroup paged_group(const PagedRows& r, const PagedArgs& pg, int window, int TG, int KT,
                                                  int u) {
  int s = u;
  if (r.row_offsets != nullptr) {
    const auto base = [&](int i) { return __ldg(r.row_offsets + i) / TG + i; };
    s = 0;
    if constexpr (WARP) {
      s = warp_search(r.n_seqs, u, base);
    } else {
      int hi = r.n_seqs - 1;
      while (s < hi) {
        const int mid = (s + hi + 1) >> 1;
        if (base(mid) <= u) s = mid; else hi = mid - 1;
      }
    }
  }
  return paged_group_of(r, pg, window, TG, KT, u, s);
}

inline int paged_groups(const PagedRows& r, int TG) {
  return r.row_offsets ? r.n_rows / TG + r.n_seqs : r.n_rows;
}

// The width of a group in a call's shares of work: its key tiles, and one more
// for what a unit costs however short it is (look-ups, its first copies, its
// results).  Without it a CTA with ten short units of a ragged batch ended
// 27 us after one with a single long one (of 115).
__device__ __forceinline__ int paged_width(int tiles) { return tiles > 0 ? tiles + 1 : 0; }

// prefix[u] = widths of the groups before u, by a block of WARPS warps (wsum:
// WARPS ints of shared memory); true in every thread if a row is past its table.
template <int WARPS, typename T>
__device__ __forceinline__ bool paged_plan(const PagedRows& r, const PagedArgs& pg, int window, int TG, int KT,
                                           int n_groups, T* prefix, int* wsum) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  T base = 0;
  bool bad = false;
  for (int u0 = 0; u0 < n_groups; u0 += WARPS * 32) {
    const int u = u0 + tid;
    int t = 0;
    if (u < n_groups) {
      const PagedGroup g = paged_group<false>(r, pg, window, TG, KT, u);
      t = paged_width(g.tiles);
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
    T before = base, total = 0;
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) before += wsum[w];
      total += wsum[w];
    }
    if (u < n_groups) prefix[u] = before + inc - t;
    base += total;
    __syncthreads();
  }
  if (tid == 0) prefix[n_groups] = base;
  return __syncthreads_or(bad);
}

// order[rank] = the groups, those with the most key tiles first (one block): a
// counting sort over the tile counts; the order of equal ones is open (it
// decides only which CTA takes a group).  A group of t tiles is cut into min(t, s)
// pieces along its keys, and those of more than one piece get places for their
// results, one behind the other.  s is the largest number up to `most` whose pieces,
// `per` places each, fit `places`: with ge(x) groups of at least x tiles, the groups
// of more than one tile have ge(2) - ge(1) + sum of ge(1 .. s) pieces, and those before rank r, which
// has m = min(t, s) itself, r m + sum of ge(m + 1 .. s).
struct PagedOrder {
  int4* order;     // group, sequence, first piece, pieces
  int per, most, places;
};
constexpr int kOrderBins = 2048;
constexpr int kMostPieces = 64;       // of a group
__device__ __forceinline__ void paged_order_block(const PagedRows& r, const PagedArgs& pg, int window, int TG, int KT,
                                                  int n_groups, const PagedOrder& o, uint32_t* status) {
  __shared__ int bins[kOrderBins];
  __shared__ int wsum[kPrWarps];
  __shared__ int ge[kMostPieces + 1];
  __shared__ long long upto[kMostPieces + 1];             // sum of ge(1 .. x)
  __shared__ int s_sh;
  constexpr int PER = kOrderBins / (kPrWarps * 32);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < kOrderBins; i += kPrWarps * 32) bins[i] = 0;
  __syncthreads();
  bool bad = false;
  auto bin_of = [](int tiles) { return kOrderBins - 1 - min(tiles, kOrderBins - 1); };   // most first
  for (int u = tid; u < n_groups; u += kPrWarps * 32) {
    const PagedGroup g = paged_group<false>(r, pg, window, TG, KT, u);
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
  for (int k = 0; k < PER; ++k) {
    bins[PER * tid + k] = before + mine[k];
    const int x = kOrderBins - (PER * tid + k);           // these have at least x tiles
    if (x <= kMostPieces) ge[x] = before + mine[k];
  }
  const bool any = __syncthreads_or(bad);
  if (warp == 0) {
    long long a = ge[lane + 1], b = ge[lane + 33];
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, a, m), y = __shfl_up_sync(0xffffffffu, b, m);
      if (lane >= m) {
        a += x;
        b += y;
      }
    }
    b += __shfl_sync(0xffffffffu, a, 31);
    upto[lane + 1] = a;
    upto[lane + 33] = b;
    const long long more = (long long)ge[2] - ge[1];
    const bool fit_a = lane + 1 <= o.most && (lane == 0 || (a + more) * o.per <= o.places);
    const bool fit_b = lane + 33 <= o.most && (b + more) * o.per <= o.places;
    const int fit = __popc(__ballot_sync(0xffffffffu, fit_a)) + __popc(__ballot_sync(0xffffffffu, fit_b));
    if (lane == 0) s_sh = max(1, fit);
  }
  __syncthreads();
  const int s = s_sh;
  for (int u = tid; u < n_groups; u += kPrWarps * 32) {
    const PagedGroup g = paged_group<false>(r, pg, window, TG, KT, u);
    const int rank = atomicAdd(&bins[bin_of(g.tiles)], 1), m = min(g.tiles, s);
    o.order[rank] = make_int4(u, g.s, m > 1 ? (int)((long long)rank * m + upto[s] - upto[m]) : 0, m);
  }
  if (tid == 0) *status = any ? (1u << KVQ_DEV_BADSEQ) : 0u;
}

// Block 0 makes the plan (the groups' widths added up, or the order of the
// groups) and writes the status word; the others each prep rb rows of hpb heads:
// q_hat as f16 to q16 [n_rows][n_q][D] (exact for bf16 in f16's normal range) and
// as bf16 to q_prepped.  Rows that read nothing get their outputs here: zeros for
// an idle sequence, NaN past the table; rows behind the last sequence get none.
// 6374 rows of 32 heads of 128: 45 us, instructions (384 for two rows of a warp,
// issue 76 %; the bytes would take 15); one token of 64 sequences 5, of 8
// sequences with heads of 512 7: angles, norm and rotation in turn.
template <int D>
__global__ void __launch_bounds__(kPrWarps * 32)
paged_prep_kernel(const PagedReadArgs a, const RopeFreqs freqs, const int rb, const int hpb, const int TG, const int KT,
                  const int n_groups, uint16_t* q16, long long* prefix, const PagedOrder order, uint32_t* status) {
  using PL = PrepLanes<D>;
  constexpr int E = PL::E;
  extern __shared__ __align__(16) uint8_t pr_buf[];
  __shared__ int rpos[16], rstart[16];
  const int tid = threadIdx.x, sub = tid / PL::N, lane = tid & (PL::N - 1);   // (sub: the row's lanes in the block)
  if (blockIdx.x == 0) {
    pdl_wait();
    pdl_launch();
    if (prefix) {
      __shared__ int wsum[kPrWarps];
      const bool bad = paged_plan<kPrWarps>(a.r, a.pg, a.L.window, TG, KT, n_groups, prefix, wsum);
      if (tid == 0) *status = bad ? (1u << KVQ_DEV_BADSEQ) : 0u;
    } else paged_order_block(a.r, a.pg, a.L.window, TG, KT, n_groups, order, status);
    return;
  }
  const int R = a.L.rope_dims, half = R >> 1, n_q = a.L.n_q;
  Angles ang = {reinterpret_cast<float2*>(pr_buf), reinterpret_cast<float2*>(pr_buf) + rb * half};
  float (*freq)[3] = reinterpret_cast<float (*)[3]>(pr_buf + (size_t)rb * half * 16);
  uint16_t* nr = reinterpret_cast<uint16_t*>(pr_buf + (size_t)rb * half * 16 + 16 * ((3 * half + 3) / 4)) + sub * 2 * D;
  const int hb = (n_q + hpb - 1) / hpb;
  const int row0 = (blockIdx.x - 1) / hb * rb, h0 = (blockIdx.x - 1) % hb * hpb;
  const int n = min(rb, a.r.n_rows - row0), nh = min(hpb, n_q - h0);
  // until the stream's previous kernel is complete only the frequency table is read
  if (R > 0) stage_freqs(freqs.f, half, freq);
  pdl_wait();
  pdl_launch();
  // (row, head) items, kPrWarps PL::ROWS of them at a time, one round ahead (past the last: the last again)
  const int items = n * nh;
  const uint32_t inv = prep_inv(nh);
  const uint16_t* base = a.q_raw + ((size_t)row0 * n_q + h0) * D + lane * E;
  uint32_t nx[E / 2] = {};
  const auto fetch = [&](int i) {
    const PrepItem it = prep_item(min(i, items - 1), nh, inv);
    load_pairs<E>(nx, base + ((size_t)it.r * n_q + it.h) * D);
  };
  fetch(sub);
  float w[E];
#pragma unroll
  for (int i = 0; i < E; ++i) w[i] = bf16_to_f(__ldg(a.q_w + lane * E + i));
  for (int r = tid >> 5; r < n; r += kPrWarps) {
    const int row = row0 + r;
    const int s = a.r.row_offsets == nullptr
                      ? row
                      : warp_search(a.r.n_seqs, row, [&](int i) { return __ldg(a.r.row_offsets + i); });
    const SeqRows sr = paged_seq_rows(a.r, s);
    if ((tid & 31) == 0) {
      rstart[r] = row - sr.off < sr.rows ? max(sr.start, -1) : kNoSeq;
      rpos[r] = sr.start < 0 ? 0 : sr.start + (row - sr.off);
    }
  }
  __syncthreads();
  for (int idx = tid; idx < n * half; idx += kPrWarps * 32) {
    const int r = idx / half, j = idx - r * half;
    put_angle<D>(ang, r, R, j, min(max(rpos[r], 0), (1 << 24) - 1), freq[j]);
  }
  __syncthreads();
  // (the rounds of a warp: it has PL::ROWS items in each)
  for (int i0 = sub & ~(PL::ROWS - 1); i0 < items; i0 += kPrWarps * PL::ROWS) {
    const int ii = i0 + (sub & (PL::ROWS - 1));
    const PrepItem at = prep_item(min(ii, items - 1), nh, inv);
    const int r = at.r;
    uint32_t raw[E / 2], y[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) raw[i] = nx[i];
    if (i0 + kPrWarps * PL::ROWS < items) fetch(ii + kPrWarps * PL::ROWS);
    prep_row<D>(raw, w, a.L.eps, R, ang, r, nr, y);
    const size_t o = ((size_t)(row0 + r) * n_q + h0 + at.h) * D + lane * E;
    uint32_t f[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) f[i] = pack_h2(bf16lo_to_f(y[i]), bf16hi_to_f(y[i]));
    store_pairs<E>(q16 + o, f);
    if (a.q_prepped && rstart[r] != kNoSeq) {             // (only 2-byte alignment is asked of it)
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        a.q_prepped[o + 2 * i] = (uint16_t)(y[i] & 0xFFFFu);
        a.q_prepped[o + 2 * i + 1] = (uint16_t)(y[i] >> 16);
      }
    }
    if (rstart[r] != kNoSeq && (rstart[r] < 0 || rpos[r] < 0 || rpos[r] >= a.pg.limit)) {
      const bool idle = rstart[r] < 0;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (a.out_f32) reinterpret_cast<float*>(a.out)[o + i] = idle ? 0.f : __int_as_float(0x7FC00000);
        else reinterpret_cast<uint16_t*>(a.out)[o + i] = idle ? 0 : 0x7FC0;
      }
    }
  }
}

template <int D>
cudaError_t launch_paged_prep(const PagedReadArgs& a, const RopeFreqs& f, int TG, int KT, int n_groups, uint16_t* q16,
                              long long* prefix, const PagedOrder& order, uint32_t* status, int num_sms,
                              cudaStream_t st) {
  // few rows: a block takes what its warps prep at once (latency); many: all heads of
  // up to 16 rows, which share their angles (16 KB of them at most)
  const int n_q = a.L.n_q, half = a.L.rope_dims / 2;
  const bool few = (long long)a.r.n_rows * n_q <= 16ll * num_sms;
  const int at_once = kPrWarps * PrepLanes<D>::ROWS;
  const int hpb = few ? std::min(n_q, at_once) : n_q;
  int rb = few ? std::max(1, std::min(16, at_once / hpb)) : std::max(1, std::min(16, a.r.n_rows / (6 * num_sms)));
  rb = std::max(1, std::min(rb, 32768 / n_q));            // (items of a block: prep_item)
  if (half > 0) rb = std::max(1, std::min(rb, 1024 / half));
  const size_t smem = (size_t)rb * half * 16 + 16 * ((3 * half + 3) / 4) + (size_t)at_once * 2 * D * 2;
  const long long blocks = (long long)((a.r.n_rows + rb - 1) / rb) * ((n_q + hpb - 1) / hpb) + 1;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_pdl(paged_prep_kernel<D>, dim3((unsigned)blocks), dim3(kPrWarps * 32), smem, st, a, f, rb, hpb, TG, KT,
                    n_groups, q16, prefix, order, status);
}

}  // namespace
}  // namespace kvq
