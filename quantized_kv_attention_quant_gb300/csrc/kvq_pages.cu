// The upkeep of a pool of pages: kvq_pages_free, kvq_pages_fork,
// kvq_pages_reserve, kvq_pages_compact.
//
// The pool's whole state is three device arrays (page tables, lengths,
// references per page); a page is free when its references are 0, and free
// pages are always taken lowest number first, so the results depend on the
// state alone and every call can be captured in a graph.
//
// Free and fork touch one sequence per block.  Reserve and compact need ranks
// among the pool's free or live pages: one cluster of eight blocks (256 warps)
// counts them, each warp over a contiguous run of pages by ballots, meets at
// the cluster's barrier, and every warp adds up the counts before its own; the
// pages' positions follow from a second pass.  A single block would need a
// block barrier per 1024 pages; a grid would need a launch per pass.  The copies
// of whole pages (codes and scales of every cache) follow in a grid over the
// GPU, warp by warp in runs of 8 KB, the pairs read from the workspace; they are
// bound by memory traffic (each byte read and written once).
//
// Measured: free and fork of 48 sequences 3.5 us each, reserve 9 (half of it the
// two passes' loads, half barriers and the cluster), compact's marking 7, the copies
// of 295 MB of pages (900 pages, 20 layers) 91 us of a call's 102, 6.5 TB/s.
#include <algorithm>

#include "kvq_common.cuh"
#include "kvq_paged.h"
#include "kvq_tc.cuh"

namespace kvq {

namespace {

constexpr int kPgThreads = 1024, kPgCluster = 8;
constexpr int kPgWarps = kPgCluster * kPgThreads / 32;    // 256
constexpr uint32_t kRun = 8192;                           // bytes of a page copied by one warp at a time

// counts per warp, then the lists, in the caller's workspace
struct PagesWs {
  int32_t* n_pairs;     // 1
  int32_t* counts;      // [2][kPgWarps]
  int32_t* src;         // [n_pages]
  int32_t* dst;         // [n_pages]
  int32_t* list;        // [n_pages]: free pages (reserve), the pages' new numbers (compact)
};
size_t pages_ws_layout(const PoolArgs& p, void* base, PagesWs* w) {
  const size_t n = ((size_t)p.n_pages * 4 + 255) / 256 * 256, head = 256 + 2 * kPgWarps * 4;
  if (w) {
    uint8_t* b = static_cast<uint8_t*>(base);
    w->n_pairs = reinterpret_cast<int32_t*>(b);
    w->counts = reinterpret_cast<int32_t*>(b + 256);
    w->src = reinterpret_cast<int32_t*>(b + head);
    w->dst = reinterpret_cast<int32_t*>(b + head + n);
    w->list = reinterpret_cast<int32_t*>(b + head + 2 * n);
  }
  return head + 3 * n;
}

// pages that a sequence of `len` tokens holds
__device__ __forceinline__ int pages_of(const PoolArgs& p, int len) {
  return len <= 0 ? 0 : min(((len - 1) >> p.p_shift) + 1, p.max_pages);
}
__device__ __forceinline__ bool is_page(const PoolArgs& p, int id) { return (unsigned)id < (unsigned)p.n_pages; }

__global__ void __launch_bounds__(256)
pages_free_kernel(const PoolArgs p, const int32_t* seqs, const int32_t* keep) {
  pdl_wait();
  pdl_launch();
  const int i = blockIdx.x, s = __ldg(seqs + i);
  bool again = (unsigned)s >= (unsigned)p.n_seqs;         // no such sequence, or listed before
  for (int j = threadIdx.x; j < i; j += 256) again |= __ldg(seqs + j) == s;
  if (__syncthreads_or(again)) return;
  const int len = p.lens[s], left = min(len, keep ? max(__ldg(keep + i), 0) : 0);
  __syncthreads();                                        // every thread has the length
  int32_t* t = p.tables + (size_t)s * p.max_pages;
  for (int k = pages_of(p, left) + threadIdx.x; k < pages_of(p, len); k += 256) {
    const int id = t[k];
    if (is_page(p, id)) atomicSub(p.refs + id, 1);
    t[k] = -1;
  }
  if (threadIdx.x == 0 && left < len) p.lens[s] = left;
}

__global__ void __launch_bounds__(256)
pages_fork_kernel(const PoolArgs p, const int32_t* parents, const int32_t* children, int n, int32_t* granted) {
  pdl_wait();
  pdl_launch();
  const int i = blockIdx.x, from = __ldg(parents + i), to = __ldg(children + i);
  bool no = (unsigned)from >= (unsigned)p.n_seqs || (unsigned)to >= (unsigned)p.n_seqs;
  for (int j = threadIdx.x; j < n; j += 256) {
    const int c = __ldg(children + j);
    no |= c == from || (j < i && c == to);
  }
  // the child's length is read only where this block alone may write it
  no = __syncthreads_or(no);
  if (!no) no = p.lens[to] != 0;
  no = __syncthreads_or(no);
  if (threadIdx.x == 0 && granted) granted[i] = no ? 0 : 1;
  if (no) return;
  const int len = p.lens[from];
  const int32_t* a = p.tables + (size_t)from * p.max_pages;
  int32_t* b = p.tables + (size_t)to * p.max_pages;
  for (int k = threadIdx.x; k < pages_of(p, len); k += 256) {
    const int id = a[k];
    b[k] = id;
    if (is_page(p, id)) atomicAdd(p.refs + id, 1);
  }
  if (threadIdx.x == 0) p.lens[to] = len;
}

// The run of pages (or sequences) of cluster warp gw.
__device__ __forceinline__ void run_of(int n, int gw, int& lo, int& hi) {
  const int per = ((n + kPgWarps - 1) / kPgWarps + 31) / 32 * 32;
  lo = (int)min((long long)n, (long long)per * gw);
  hi = (int)min((long long)n, (long long)lo + per);
}

// Sum of counts[0 .. gw) and of all.
__device__ __forceinline__ int before_of(const int32_t* counts, int gw, int& total) {
  const int lane = threadIdx.x & 31;
  int b = 0, t = 0;
#pragma unroll
  for (int k = 0; k < kPgWarps / 32; ++k) {
    const int w = 32 * k + lane, c = __ldcg(counts + w);
    t += c;
    if (w < gw) b += c;
  }
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) {
    b += __shfl_xor_sync(0xffffffffu, b, m);
    t += __shfl_xor_sync(0xffffffffu, t, m);
  }
  total = t;
  return b;
}

// The cluster's barrier: what was written before it, all warps see after it
// (read past L1).
__device__ __forceinline__ void meet() {
  __syncwarp();
  tc::cluster_sync();
}

// What a sequence asks for.
struct Need { int len, grown, have, want, shared; bool fits; };
__device__ __forceinline__ Need need_of(const PoolArgs& p, const int32_t* n_new, int s) {
  Need d;
  d.len = max(0, __ldcg(p.lens + s));
  const int more = max(0, __ldg(n_new + s));
  const long long to = (long long)d.len + more;
  d.fits = to <= (long long)p.max_pages << p.p_shift && to <= (1 << 24);
  d.grown = d.fits ? (int)to : d.len;
  d.have = pages_of(p, d.len);
  d.want = pages_of(p, d.grown);
  d.shared = -1;
  if (d.grown > d.len && (d.len & (p.P - 1))) {           // the last page will be written
    const int id = __ldcg(p.tables + (size_t)s * p.max_pages + d.have - 1);
    if (is_page(p, id) && __ldcg(p.refs + id) > 1) d.shared = id;
  }
  return d;
}

__global__ void __cluster_dims__(kPgCluster, 1, 1) __launch_bounds__(kPgThreads)
pages_reserve_kernel(const PoolArgs p, const int32_t* n_new, int32_t* start_pos, int32_t* granted, const PagesWs w) {
  pdl_wait();
  pdl_launch();
  const int lane = threadIdx.x & 31, gw = (int)tc::cta_rank() * (kPgThreads / 32) + (threadIdx.x >> 5);
  int p_lo, p_hi, s_lo, s_hi;
  run_of(p.n_pages, gw, p_lo, p_hi);
  run_of(p.n_seqs, gw, s_lo, s_hi);
  // ---- free pages and pages asked for, per warp ----
  int n_free = 0, n_need = 0;
  for (int i0 = p_lo; i0 < p_hi; i0 += 32) {
    const int i = i0 + lane;
    n_free += __popc(__ballot_sync(0xffffffffu, i < p_hi && __ldcg(p.refs + i) <= 0));
  }
  for (int i = s_lo + lane; i < s_hi; i += 32) {
    const Need d = need_of(p, n_new, i);
    n_need += d.want - d.have + (d.shared >= 0 ? 1 : 0);
  }
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) n_need += __shfl_xor_sync(0xffffffffu, n_need, m);
  if (lane == 0) {
    w.counts[gw] = n_free;
    w.counts[kPgWarps + gw] = n_need;
  }
  if (gw == 0 && lane == 0) *w.n_pairs = 0;
  meet();
  // ---- the free pages that will be taken, in ascending order ----
  int all_free, all_need;
  int at = before_of(w.counts, gw, all_free), asked = before_of(w.counts + kPgWarps, gw, all_need);
  for (int i0 = p_lo; i0 < p_hi && at < all_need; i0 += 32) {
    const int i = i0 + lane;
    const bool f = i < p_hi && __ldcg(p.refs + i) <= 0;
    const uint32_t b = __ballot_sync(0xffffffffu, f);
    if (f) w.list[at + __popc(b & ((1u << lane) - 1u))] = i;
    at += __popc(b);
  }
  // what each sequence of the warp's run gets is fixed before any reference changes
  // (a warp has at most 32 sequences at a time; longer runs are walked again below)
  meet();
  for (int i0 = s_lo; i0 < s_hi; i0 += 32) {
    const int s = i0 + lane;
    Need d = {};
    int need = 0;
    if (s < s_hi) {
      d = need_of(p, n_new, s);
      need = d.want - d.have + (d.shared >= 0 ? 1 : 0);
    }
    int upto = need;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, upto, m);
      if (lane >= m) upto += o;
    }
    const int sum = __shfl_sync(0xffffffffu, upto, 31);
    // parked in the outputs until every warp has read the references
    if (s < s_hi) {
      const bool ok = d.fits && (need == 0 || asked + upto <= all_free);
      start_pos[s] = asked + upto - need;
      granted[s] = ok ? (d.shared >= 0 ? 2 : 1) : 0;
    }
    asked += sum;
  }
  meet();
  // ---- a warp per sequence: its pages, length, and the copy of a shared last page ----
  for (int s = gw; s < p.n_seqs; s += kPgWarps) {
    const int first = __ldcg(start_pos + s), ok = __ldcg(granted + s);
    const int len = max(0, __ldcg(p.lens + s)), more = max(0, __ldg(n_new + s));
    __syncwarp();                                         // every lane has them
    const int have = pages_of(p, len);
    int32_t* t = p.tables + (size_t)s * p.max_pages;
    if (ok) {
      const int want = pages_of(p, len + more);
      for (int k = have + lane; k < want; k += 32) {
        const int id = __ldcg(w.list + first + (ok == 2 ? 1 : 0) + k - have);
        t[k] = id;
        p.refs[id] = 1;
      }
      if (lane == 0) {
        if (ok == 2) {
          const int old = t[have - 1], id = __ldcg(w.list + first), k = atomicAdd(w.n_pairs, 1);
          w.src[k] = old;
          w.dst[k] = id;
          t[have - 1] = id;
          p.refs[id] = 1;
          atomicSub(p.refs + old, 1);
        }
        p.lens[s] = len + more;
      }
    }
    if (lane == 0) {
      start_pos[s] = len;
      granted[s] = ok ? 1 : 0;
    }
  }
}

__global__ void __cluster_dims__(kPgCluster, 1, 1) __launch_bounds__(kPgThreads)
pages_compact_kernel(const PoolArgs p, int32_t* page_map, int32_t* n_live, const PagesWs w) {
  pdl_wait();
  pdl_launch();
  const int lane = threadIdx.x & 31, gw = (int)tc::cta_rank() * (kPgThreads / 32) + (threadIdx.x >> 5);
  int lo, hi;
  run_of(p.n_pages, gw, lo, hi);
  int live = 0;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    live += __popc(__ballot_sync(0xffffffffu, i < hi && __ldcg(p.refs + i) > 0));
  }
  if (lane == 0) w.counts[gw] = live;
  if (gw == 0 && lane == 0) *w.n_pairs = 0;
  meet();
  // L live pages: a hole is a free page below L, and a live page at or past L moves
  int L;
  int at = before_of(w.counts, gw, L), holes = 0;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    const bool f = i < hi && __ldcg(p.refs + i) > 0;
    const uint32_t b = __ballot_sync(0xffffffffu, f);
    const int rank = at + __popc(b & ((1u << lane) - 1u));   // live pages before i
    if (i < hi) {
      w.list[i] = f ? i : -1;
      if (!f && i < L) {
        w.dst[i - rank] = i;
        ++holes;
      }
      if (f && i >= L) w.src[L - 1 - rank] = i;           // counted from the last one
    }
    at += __popc(b);
  }
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) holes += __shfl_xor_sync(0xffffffffu, holes, m);
  if (lane == 0 && holes) atomicAdd(w.n_pairs, holes);
  meet();
  const int m = __ldcg(w.n_pairs);
  const int tid = gw * 32 + lane;
  // hole k (ascending) takes the k-th page that moves
  for (int k = tid; k < m; k += kPgWarps * 32) {
    const int from = __ldcg(w.src + m - 1 - k), to = __ldcg(w.dst + k);
    p.refs[to] = __ldcg(p.refs + from);
    p.refs[from] = 0;
    w.list[from] = to;
  }
  if (tid == 0) *n_live = L;
  if (page_map) {
    meet();
    for (int i = tid; i < p.n_pages; i += kPgWarps * 32) page_map[i] = __ldcg(w.list + i);
  }
}

struct CopyPlan {
  PoolCaches c;
  uint32_t run0[KVQ_MAX_PAGED_CACHES + 1];                // runs of a page before cache i (K, then V)
};

// Runs of the page pairs, a warp each; `renumber`: also the tables, by the
// pages' new numbers, and pair k's source is src[n - 1 - k].
__global__ void __launch_bounds__(256)
pages_copy_kernel(const PoolArgs p, const __grid_constant__ CopyPlan plan, const PagesWs w, const int renumber) {
  pdl_wait();
  pdl_launch();
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * 8, gw = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (renumber) {
    for (long long s = gw; s < p.n_seqs; s += warps) {
      int32_t* t = p.tables + (size_t)s * p.max_pages;
      const int n = pages_of(p, p.lens[s]);
      for (int k = lane; k < n; k += 32) {
        const int id = t[k];
        if (is_page(p, id)) t[k] = __ldcg(w.list + id);
      }
    }
  }
  const int n_pairs = __ldcg(w.n_pairs);
  const uint32_t per = plan.run0[plan.c.n];
  for (long long it = gw; it < (long long)n_pairs * per; it += warps) {
    const int pair = (int)(it / per);
    const uint32_t run = (uint32_t)(it - (long long)pair * per);
    int a = 0, b = plan.c.n - 1;                          // the last cache with run0 <= run
    while (a < b) {
      const int mid = (a + b + 1) >> 1;
      if (plan.run0[mid] <= run) a = mid; else b = mid - 1;
    }
    const PoolCaches::Cache& c = plan.c.c[a];
    const uint32_t half = (plan.run0[a + 1] - plan.run0[a]) / 2, in = run - plan.run0[a];
    const bool v = in >= half;
    const uint32_t off = (v ? in - half : in) * kRun, bytes = min(kRun, c.page_bytes - off);
    const int from = __ldcg(w.src + (renumber ? n_pairs - 1 - pair : pair)), to = __ldcg(w.dst + pair);
    uint8_t* base = v ? c.v : c.k;
    const uint4* src = reinterpret_cast<const uint4*>(base + (size_t)from * c.page_bytes + off);
    uint4* dst = reinterpret_cast<uint4*>(base + (size_t)to * c.page_bytes + off);
    const int n16 = (int)(bytes / 16);                    // 64 .. 512
    int i = lane;
    for (; i + 7 * 32 < n16; i += 8 * 32) {
      uint4 x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = __ldcs(src + i + 32 * k);
#pragma unroll
      for (int k = 0; k < 8; ++k) __stcs(dst + i + 32 * k, x[k]);
    }
    for (; i < n16; i += 32) dst[i] = src[i];
    if (off == 0) {
      float* sc = v ? c.vs : c.ks;
      for (int h = lane; h < c.n_kv; h += 32) sc[(size_t)to * c.n_kv + h] = sc[(size_t)from * c.n_kv + h];
    }
  }
}

cudaError_t launch_copy(const PoolArgs& p, const PoolCaches& c, const PagesWs& w, int renumber, int num_sms,
                        cudaStream_t st) {
  CopyPlan plan;
  plan.c = c;
  uint32_t at = 0;
  for (int i = 0; i < c.n; ++i) {
    plan.run0[i] = at;
    at += 2 * ((c.c[i].page_bytes + kRun - 1) / kRun);
  }
  for (int i = c.n; i <= KVQ_MAX_PAGED_CACHES; ++i) plan.run0[i] = at;
  return launch_pdl(pages_copy_kernel, dim3(num_sms * 8), dim3(256), 0, st, p, plan, w, renumber);
}

}  // namespace

size_t pages_ws_bytes(const PoolArgs& p) { return pages_ws_layout(p, nullptr, nullptr); }

cudaError_t launch_pages_free(const PoolArgs& p, const int32_t* seqs, const int32_t* keep, int n, cudaStream_t st) {
  return launch_pdl(pages_free_kernel, dim3(n), dim3(256), 0, st, p, seqs, keep);
}

cudaError_t launch_pages_fork(const PoolArgs& p, const int32_t* parents, const int32_t* children, int n,
                              int32_t* granted, cudaStream_t st) {
  return launch_pdl(pages_fork_kernel, dim3(n), dim3(256), 0, st, p, parents, children, n, granted);
}

cudaError_t launch_pages_reserve(const PoolArgs& p, const PoolCaches& c, const int32_t* n_new, int32_t* start_pos,
                                 int32_t* granted, void* ws, int num_sms, cudaStream_t st) {
  PagesWs w;
  pages_ws_layout(p, ws, &w);
  const cudaError_t e = launch_pdl(pages_reserve_kernel, dim3(kPgCluster), dim3(kPgThreads), 0, st, p, n_new, start_pos,
                                   granted, w);
  return e != cudaSuccess ? e : launch_copy(p, c, w, 0, num_sms, st);
}

cudaError_t launch_pages_compact(const PoolArgs& p, const PoolCaches& c, int32_t* page_map, int32_t* n_live, void* ws,
                                 int num_sms, cudaStream_t st) {
  PagesWs w;
  pages_ws_layout(p, ws, &w);
  const cudaError_t e = launch_pdl(pages_compact_kernel, dim3(kPgCluster), dim3(kPgThreads), 0, st, p, page_map, n_live,
                                   w);
  return e != cudaSuccess ? e : launch_copy(p, c, w, 1, num_sms, st);
}

}  // namespace kvq
