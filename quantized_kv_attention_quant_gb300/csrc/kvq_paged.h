// Launch interfaces of the paged 8-bit cache: append, read-back, attention
// over pages, and the pages' upkeep (kvq_paged_append.cu, kvq_paged_decode.cu,
// kvq_paged_prefill.cu, kvq_pages.cu).
#pragma once
#include <atomic>

#include "kvq_internal.h"

namespace kvq {

// Allows a kernel `bytes` of dynamic shared memory, once per device (`done`:
// the kernel's own, a bit per device).
template <typename Kernel>
inline cudaError_t allow_smem(Kernel* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// One layer's pages (kvq_paged_cache) with the table of a call's sequences.
struct PagedArgs {
  uint8_t* k_codes;       // [n_pages][n_kv][P][D]
  uint8_t* v_codes;
  float* k_scales;        // [n_pages][n_kv]
  float* v_scales;
  const int32_t* tables;  // [n_seqs][max_pages]
  int n_pages, max_pages, P, p_shift, e4m3;
  int limit;              // positions at or past it are no rows of the call
};

// Rows of a call: sequence s has rows row_offsets[s] .. row_offsets[s+1]-1 at
// positions start[s] ..; row_offsets == nullptr: one row per sequence.
struct PagedRows {
  const int32_t* row_offsets;
  const int32_t* start;
  int n_seqs, n_rows;
};

struct PagedAppendArgs {
  LayerArgs L;
  PagedArgs pg;
  PagedRows r;
  const uint16_t* k_raw;
  const uint16_t* v_raw;
  const uint16_t* k_w;
  uint16_t* prepped;
};
cudaError_t launch_paged_append(const PagedAppendArgs& a, const RopeFreqs& f, int num_sms, cudaStream_t st);

struct PagedGatherArgs {
  PagedArgs pg;
  PagedRows r;
  int n_kv, D;
  uint16_t* k_rows;
  uint16_t* v_rows;
};
cudaError_t launch_paged_gather(const PagedGatherArgs& a, int num_sms, cudaStream_t st);

struct PagedReadArgs {
  LayerArgs L;
  PagedArgs pg;
  PagedRows r;
  const uint16_t* q_raw;
  const uint16_t* q_w;
  void* out;
  int out_f32;
  uint16_t* q_prepped;
};
// The read on mma.sync: 16 (token, q head) rows of a kv head a unit, the keys
// of all units cut into equal shares.  max_pos: host bound of the rows'
// positions.
size_t paged_decode_ws_bytes(const LayerArgs& L, int n_seqs, int n_rows, int max_pos, int num_sms);
cudaError_t launch_paged_decode(const PagedReadArgs& a, const RopeFreqs& f, int max_pos, void* ws, int num_sms,
                                cudaStream_t st);

// The read on tcgen05: prompt rows, G dividing 128, more than a few rows.
bool paged_prefill_supported(const LayerArgs& L, int max_rows_per_seq);
size_t paged_prefill_ws_bytes(const LayerArgs& L, int n_seqs, int n_rows, int max_pos, int num_sms);
cudaError_t launch_paged_prefill(const PagedReadArgs& a, const RopeFreqs& f, int max_pos, void* ws, int num_sms,
                                 cudaStream_t st);

// The pool of pages (kvq_page_pool) and the caches whose pages it manages.
struct PoolArgs {
  int32_t* tables;
  int32_t* lens;
  int32_t* refs;
  int n_seqs, max_pages, n_pages, P, p_shift;
};
struct PoolCaches {
  int n;
  struct Cache {
    uint8_t* k;
    uint8_t* v;
    float* ks;
    float* vs;
    int32_t n_kv;
    uint32_t page_bytes;  // of one of k, v
  } c[KVQ_MAX_PAGED_CACHES];
};
size_t pages_ws_bytes(const PoolArgs& p);
cudaError_t launch_pages_free(const PoolArgs& p, const int32_t* seqs, const int32_t* keep, int n, cudaStream_t st);
cudaError_t launch_pages_fork(const PoolArgs& p, const int32_t* parents, const int32_t* children, int n,
                              int32_t* granted, cudaStream_t st);
cudaError_t launch_pages_reserve(const PoolArgs& p, const PoolCaches& c, const int32_t* n_new, int32_t* start_pos,
                                 int32_t* granted, void* ws, int num_sms, cudaStream_t st);
cudaError_t launch_pages_compact(const PoolArgs& p, const PoolCaches& c, int32_t* page_map, int32_t* n_live, void* ws,
                                 int num_sms, cudaStream_t st);

}  // namespace kvq
