// attn_train_backward: the gradient of the training read (kvq_train.cu) by
// q_hat, k_hat and v_hat under the prefix-shared layout, on the tensor cores.
// With each row's log-sum-exp from the forward, over the keys j that row i sees,
//   P = exp(S - lse), S = q k;  dP = dO v;  dS = P (dP - delta), delta = dO . O
//   dq = dS k,  dk = dS^T q,  dv = P^T dO   (dk, dv over the kv head's q heads)
// A row that sees one key has P = 1 whatever its score: its dS is 0 exactly.
//
// Five products per (row, head, key), each computed once.  At head_dim 256 and
// 512 the accumulators of dk and dv fill tensor memory by themselves, so a
// kernel that keeps S and dP beside them would have to split the head dims and
// recompute both (8 or 9 products instead of 5).  Instead P and dS go through
// the workspace as bf16 tiles of 128 rows x 128 keys, a chunk of the tile list at
// a time (1 GB, or four row tiles' whole lists where that is more: it does not grow
// with rows x keys, past some 524,000 visible keys it does with the keys):
//   prep     delta per (row, head); one block lists the row tiles, key tiles
//            and chunks of the layout
//   scores   S and dP of one chunk's tiles (tcgen05, fp32 in tensor memory),
//            softmax and dS in registers, P and dS tiles out
//   products dq of the chunk's row tiles, dk and dv of every key tile over the
//            chunk's row tiles: one kernel, out = sum_t A_t B_t in tensor memory
//   finish   dk and dv joined over splits (fixed order) into the outputs
//            (left out when one chunk and one split write them directly)
// Each is a programmatic dependent of the one before.  Measured on 2048 rows of a
// prefix of 1024 and four branches of 256, 16 heads of 512 on one kv head: 168 us,
// 0.44 of the measured bf16 rate (one by one: prep 20 us, scores 63, products 78,
// finish 13);
// on 4096 rows of a prefix of 2048 and two branches of 1024 508 us, 0.63; on 8192
// rows of twice those blocks, in several chunks, 1.84 ms, 0.70.
//
// A row tile is 128 (token, head) pairs of one block that share a kv head (128/G
// tokens times G heads, pair r = token r / G, head r % G), a key tile 128 keys of
// one block counted from the block's start.  P and dS tiles are stored as 8 x
// 16-byte core matrices, [16 key groups of 8][128 rows][8 keys]: a warp of the
// scores kernel (lane = row) writes 512 contiguous bytes per store, and the
// same image is a K-major operand without swizzle for dq (M = rows, K = keys)
// and, read transposed, an MN-major one for dk and dv (M = keys, K = rows).  The
// other operands (k, q, dO) are MN-major too: rows of 64 dims straight from
// TMA (128-byte swizzle), no transposition anywhere.
#include "kvq_common.cuh"
#include "kvq_internal.h"
#include "kvq_tc.cuh"
#include "kvq_tma.cuh"

#include <algorithm>
#include <atomic>
#include <mutex>
#include <type_traits>

namespace kvq {

namespace {

constexpr int kT = 128;                     // rows and keys of a tile
constexpr uint32_t kTileBytes = kT * kT * 2;
constexpr int kMaxSplits = 8;
constexpr int kMaxPairs = 128;              // CTA pairs of a grid
constexpr float kL2E = 1.4426950408889634f;

// A row tile: tokens row0 .. row0 + nt - 1 (packed), the first at position
// pos0; its P and dS tiles are base .. base + nA + nB - 1 of its kv head's list:
// the prefix's key tiles a0 .. (keys at positions below kend), then its own
// block's key tiles b0 .. (block 0's own keys are the prefix).
struct alignas(16) RowTile {
  int row0, nt, pos0, base;
  int a0, nA, b0, nB;
  int off0, block, kend, pad;
};
// A key tile: keys row0 .. row0 + n - 1 (packed), tile idx of its block; the row
// tiles that may see it are lo .. hi - 1 (a branch's: its own, from there on; with a
// window, up to the last whose window reaches back to it.  The products' lists look
// at each of them, for every item: without that end the listing grew with rows x rows,
// 19.3 instead of 11.5 ms on 524288 rows with a window of 512, 8 heads of 256).
struct alignas(16) KeyTile { int row0, n, block, idx, lo, hi, pad[2]; };

// The key tiles that either of two row tiles sees: prefix tiles a0 .., own-block
// tiles b0 .. of both (one block) or of the first and then c0 .. of the second.
struct Merged {
  int a0, nA, b0, nB, c0, nC;
  __device__ __forceinline__ int n() const { return nA + nB + nC; }
};
__device__ __forceinline__ Merged merged(const RowTile& r0, const RowTile& r1, bool two) {
  Merged u = {r0.a0, r0.nA, r0.b0, r0.nB, 0, 0};
  if (!two) return u;
  auto hull = [](int& lo, int& n, int lo1, int n1) {
    if (n1 == 0) return;
    const int l = n ? min(lo, lo1) : lo1, h = n ? max(lo + n, lo1 + n1) : lo1 + n1;
    lo = l;
    n = h - l;
  };
  hull(u.a0, u.nA, r1.a0, r1.nA);
  if (r0.block == r1.block) {
    hull(u.b0, u.nB, r1.b0, r1.nB);
  } else {
    u.c0 = r1.b0;
    u.nC = r1.nB;
  }
  return u;
}
// Key tile j of a merged list: its first key's packed row and position, and its
// place in each row tile's own list (-1: not there).
struct MergedTile { int pk, lp, j0, j1; bool prefix; };
__device__ __forceinline__ MergedTile merged_at(const Merged& u, const RowTile& r0, const RowTile& r1, bool two, int j) {
  MergedTile t;
  auto in = [](int x, int lo, int n, int base) { return x >= lo && x < lo + n ? base + x - lo : -1; };
  t.prefix = j < u.nA;
  if (t.prefix) {
    const int x = u.a0 + j;
    t.pk = t.lp = x * kT;
    t.j0 = in(x, r0.a0, r0.nA, 0);
    t.j1 = two ? in(x, r1.a0, r1.nA, 0) : -1;
  } else if (j < u.nA + u.nB) {
    const int x = u.b0 + j - u.nA;
    t.pk = r0.off0 + x * kT;
    t.lp = r0.kend + x * kT;                          // a branch: its first row is at position P = kend
    t.j0 = in(x, r0.b0, r0.nB, r0.nA);
    t.j1 = two && r1.block == r0.block ? in(x, r1.b0, r1.nB, r1.nA) : -1;
  } else {
    const int x = u.c0 + j - u.nA - u.nB;
    t.pk = r1.off0 + x * kT;
    t.lp = r1.kend + x * kT;
    t.j0 = -1;
    t.j1 = r1.nA + x - r1.b0;
  }
  return t;
}

struct alignas(16) Head {
  uint32_t status;
  int ok, nrt, nkt;             // layout valid; row and key tiles of one kv head
  int ntiles;                   // (row tile, key tile) pairs of one kv head
  int npieces;                  // entries of the piece list
  int nunits;                   // units of the scores kernel, of one kv head
  int pad;
};

struct Ws {
  Head* head;
  int* chunk;                   // [nl + 1]: chunk c is pairs of row tiles chunk[c] .. chunk[c + 1] - 1 (kv head major)
  int* units;                   // [pairs of row tiles]: units of the scores kernel before each
  int* counts;                  // [nkt]: row tiles that see a key tile; then [key pairs]: pieces of its lists
  int* next;                    // [nl]: the products' items drawn so far
  int* list;                    // the (key pair, piece) of every dk and dv item: pair * kMaxSplits + piece
  int4* begin;                  // [pairs]: a CTA pair's units, and the kv head, row tile pair and key tile of its first
  int* starts;                  // [2][n_blocks + 1]: row and key tiles before each block
  RowTile* rt;
  KeyTile* kt;
  float* delta;                 // [n_rows][n_q]
  float* acc;                   // [splits][2][n_rows][n_kv][D]: dk, dv
  uint8_t* p;                   // [cap + 1] tiles, the last of zeros
  uint8_t* ds;
};

// Sizes of a call, from what the host knows (block offsets are in device memory).
struct Plan {
  int nrt, nkt;                 // bounds of row and key tiles of a kv head
  int cap;                      // tiles of a chunk
  int nl;                       // chunk launches
  int splits, piece;            // of a key pair's row tiles: most pieces; row tiles of one
  int direct;                   // one chunk, one split: dk and dv need no sums beside the outputs
  bool fits;                    // tile counts fit 32 bits (else nothing else is set)
  size_t chunk_o, next_o, begin_o, units_o, counts_o, list_o, starts_o, rt_o, kt_o, delta_o, acc_o, p_o, ds_o, bytes;
};

inline long long cdiv(long long a, long long b) { return (a + b - 1) / b; }

// Output columns per CTA of the products kernel.
__host__ __device__ constexpr int prod_n(int D) { return D > 256 ? 256 : D; }

// Tiles of a chunk (1 GB of workspace; more only where a row tile sees over 4096 key
// tiles, as a chunk ends before a pair of row tiles that does not fit).  Larger is faster: 4096 rows of 16
// heads of 512 took 1016 us in chunks of 1024 (64 MB, within L2), 751 of 2048, 612
// in one: longer sums for each output beat L2 hits.
constexpr int kChunkTiles = 16384;
// Least row tiles of a piece: 6 and 8 took 27.4 and 30.3 us on 739 rows in ragged
// blocks, 54.8 and 53.5 on 2048 rows with a window of 512 (head_dim 256, 8 heads).
constexpr int kMinPiece = 6;

Plan make_plan(const LayerArgs& L, int n_blocks, int n_rows, int max_block_rows, int num_sms) {
  Plan p = {};
  const int TQ = kT / L.G, W = L.window;
  p.nrt = std::min(n_rows, n_rows / TQ + n_blocks);
  p.nkt = std::min(n_rows, n_rows / kT + n_blocks);
  // most key tiles of a row tile: prefix and own block, both at or before it
  const long long per_block = cdiv(max_block_rows, kT), pfx = n_blocks > 1 ? per_block : 0, n128 = n_rows / kT;
  long long tmax = std::min(pfx + per_block, n128 + 3);
  if (W > 0) tmax = std::min(tmax, ((long long)W + TQ + kT - 3) / kT + 2);   // a span of W + TQ - 1 positions
  // all pairs of a kv head: a block's own part grows from 1 tile to per_block
  // (half of it on average); or, by packed order, half of all keys for the
  // full row tiles and all of them for each block's last, ragged one
  const long long by_block = p.nrt * std::min(tmax, pfx + max_block_rows / (2 * kT) + 3);
  const long long by_order = n_rows / TQ * std::min(tmax, n128 / 2 + 4) + n_blocks * tmax;
  const long long total = std::min(by_block, by_order) * L.n_kv;
  if (total > 0x7fffffffLL || L.n_kv > 0xffff) return Plan{};
  p.fits = true;
  const long long cap = std::min<long long>(total, std::max<long long>(kChunkTiles, 4 * tmax));
  p.cap = (int)cap;
  // a chunk ends before a pair of row tiles that does not fit: more than cap - 2 tmax tiles each
  p.nl = cap >= total ? 1 : (int)cdiv(total, cap - 2 * tmax + 1);
  // Splits: the list of row tiles of a key pair is cut into pieces, so that no
  // CTA's item is long beside an SM's share of the products (in steps of a pair
  // of tiles); a piece costs its output once more, so it is not cut short.
  // With one chunk each list is cut by its own length (`piece` row tiles at
  // least), with several every list into the same number of pieces.
  const int H = L.D / prod_n(L.D);
  const long long share = std::min(total, cap) * 3 * H / 2 / num_sms;
  p.piece = (int)std::max<long long>(kMinPiece, share / 2);
  p.splits = p.nl == 1 ? (int)std::min<long long>(kMaxSplits, cdiv(p.nrt, p.piece))
                       : (int)std::min<long long>(kMaxSplits, std::max(1LL, std::min<long long>(p.nrt, 2 * cap / tmax) / std::max(1LL, share)));
  // and have room: 256 MB of partial sums, or one set
  const size_t plane = 2 * (size_t)n_rows * L.n_kv * L.D * 4;
  const size_t acc = std::max(plane, std::min<size_t>(kMaxSplits * plane, (size_t)256 << 20));
  p.splits = (int)std::min<size_t>(p.splits, acc / plane);
  p.direct = p.nl == 1 && p.splits == 1;
  size_t o = 256;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += (bytes + 255) / 256 * 256;
    return at;
  };
  p.chunk_o = take(((size_t)p.nl + 1) * 4);
  p.next_o = take((size_t)p.nl * 4);
  p.begin_o = take(kMaxPairs * sizeof(int4));
  p.units_o = take(((size_t)p.nrt + 1) / 2 * 4);
  p.counts_o = take(((size_t)p.nkt + (p.nkt + 1) / 2) * 4);
  p.list_o = take(((size_t)p.nkt + 1) / 2 * kMaxSplits * 4);
  p.starts_o = take(((size_t)n_blocks + 1) * 8);
  p.rt_o = take((size_t)p.nrt * sizeof(RowTile));
  p.kt_o = take((size_t)p.nkt * sizeof(KeyTile));
  p.delta_o = take((size_t)n_rows * L.n_q * 4);
  p.acc_o = take(acc);
  p.p_o = take(((size_t)p.cap + 1) * kTileBytes);      // the last tile holds zeros
  p.ds_o = take(((size_t)p.cap + 1) * kTileBytes);
  p.bytes = o;
  return p;
}

Ws carve(void* base, const Plan& p) {
  uint8_t* b = static_cast<uint8_t*>(base);
  Ws w;
  w.head = reinterpret_cast<Head*>(b);
  w.chunk = reinterpret_cast<int*>(b + p.chunk_o);
  w.next = reinterpret_cast<int*>(b + p.next_o);
  w.counts = reinterpret_cast<int*>(b + p.counts_o);
  w.list = reinterpret_cast<int*>(b + p.list_o);
  w.units = reinterpret_cast<int*>(b + p.units_o);
  w.begin = reinterpret_cast<int4*>(b + p.begin_o);
  w.starts = reinterpret_cast<int*>(b + p.starts_o);
  w.rt = reinterpret_cast<RowTile*>(b + p.rt_o);
  w.kt = reinterpret_cast<KeyTile*>(b + p.kt_o);
  w.delta = reinterpret_cast<float*>(b + p.delta_o);
  w.acc = reinterpret_cast<float*>(b + p.acc_o);
  w.p = b + p.p_o;
  w.ds = b + p.ds_o;
  return w;
}

// ---------------------------------------------------------------------------
// prep: the layout's tiles (block 0) and delta (the other blocks)
// ---------------------------------------------------------------------------
// Bound by reading out and d_out once: 101 MB of 2048 rows x 16 heads of 512 in
// 20 us, 0.74 of the measured copy rate.  In short calls the plan's chain of
// dependent steps counts instead (3.5 us for one row tile).
constexpr int kPrepThreads = 256;

// Exclusive prefix sum over the block's threads; *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, s, m);
    if (lane >= m) s += o;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kPrepThreads / 32; ++w) {
    const int x = warp_sums[w];
    before += w < warp ? x : 0;
    all += x;
  }
  *total = all;
  return before + s - v;
}

// Largest i in [0, n) with a[i] <= x (a[0] <= x, a non-decreasing).
__device__ __forceinline__ int last_le(const int* a, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// What the plan needs of the host's: tiles of a chunk, chunks, and how lists are cut.
struct PlanArgs { int cap, nl, splits, piece, pairs; };       // pairs: CTA pairs of the scores kernel

__device__ void plan_block(const TrainBwdArgs& a, const Ws& w, const PlanArgs pl) {
  // what later steps look up again stays in shared memory where it is small (the
  // chain of dependent loads is the whole time of a short call)
  constexpr int kS = kPrepThreads;
  __shared__ int sums[kPrepThreads / 32], s_off[kS + 1], s_rs[kS], s_ks[kS], s_counts[kS], s_units[kS];
  __shared__ RowTile s_rt[kS];
  const int tid = threadIdx.x, nb = a.n_blocks, TQ = kT / a.L.G, W = a.L.window, cap = pl.cap, nl = pl.nl;
  const int32_t* off = a.off;
  if (nb <= kS) {
    for (int b = tid; b <= nb; b += kPrepThreads) s_off[b] = a.off[b];
    __syncthreads();
    off = s_off;
  }
  for (int c = tid; c < nl; c += kPrepThreads) w.next[c] = 0;
  const int P = off[1];
  bool bad = false;
  for (int b = tid; b < nb; b += kPrepThreads) {
    const int o0 = off[b], o1 = off[b + 1];
    bad |= !(o0 >= 0 && o0 <= o1 && o1 <= a.n_rows && P >= 0 && (b == 0 ? o0 == 0 : o0 >= P) &&
             (b + 1 < nb || o1 == a.n_rows) && o1 - o0 <= a.max_block_rows);
  }
  bad = __syncthreads_or(bad);
  if (bad) {                                // no tiles: nothing is written
    for (int c = tid; c <= nl; c += kPrepThreads) w.chunk[c] = 0;
    if (tid == 0) *w.head = Head{1u << KVQ_DEV_BADSEQ, 0, 0, 0, 0, 0, 0, 0};
    return;
  }
  int* rs = nb <= kS ? s_rs : w.starts;
  int* ks = nb <= kS ? s_ks : w.starts + nb + 1;
  int nrt = 0, nkt = 0;
  for (int b0 = 0; b0 < nb; b0 += kPrepThreads) {
    const int b = b0 + tid, rows = b < nb ? off[b + 1] - off[b] : 0;
    int tr, tk;
    const int r = block_scan((rows + TQ - 1) / TQ, sums, &tr), k = block_scan((rows + kT - 1) / kT, sums, &tk);
    if (b < nb) {
      rs[b] = nrt + r;
      ks[b] = nkt + k;
    }
    nrt += tr;
    nkt += tk;
  }
  int* counts = nkt <= kS ? s_counts : w.counts;
  RowTile* rt = nrt <= kS ? s_rt : w.rt;
  __syncthreads();
  for (int i = tid; i < nkt; i += kPrepThreads) {
    const int b = last_le(ks, nb, i), idx = i - ks[b], o0 = off[b];
    const int n = min(kT, off[b + 1] - o0 - idx * kT), lo = rs[b] + idx * kT / TQ;
    int hi = b == 0 || b + 1 == nb ? nrt : rs[b + 1];
    if (W > 0) {
      // the last row of its block, from the block's start, whose window holds the tile's
      // last key; a prefix tile is seen by branches (from position P on) only if that is P or later
      const long long last = (long long)idx * kT + n - 1 + W - 1;
      if (b > 0 || last < P) hi = (int)min((long long)(b == 0 && nb > 1 ? rs[1] : hi), rs[b] + last / TQ + 1);
    }
    w.kt[i] = KeyTile{o0 + idx * kT, n, b, idx, lo, hi, {0, 0}};
    counts[i] = 0;
  }
  __syncthreads();
  int ntiles = 0;
  for (int i0 = 0; i0 < nrt; i0 += kPrepThreads) {
    const int i = i0 + tid;
    RowTile t = {};
    if (i < nrt) {
      const int b = last_le(rs, nb, i), o0 = off[b], rows = off[b + 1] - o0, t0 = (i - rs[b]) * TQ;
      const int first = b == 0 ? 0 : P;
      t.row0 = o0 + t0;
      t.nt = min(TQ, rows - t0);
      t.pos0 = first + t0;
      t.off0 = o0;
      t.block = b;
      t.kend = b == 0 ? 0x7fffffff : P;
      const int last = t.pos0 + t.nt - 1, lo = W > 0 ? max(0, t.pos0 - W + 1) : 0;
      const int a_hi = b == 0 ? last : P - 1;
      if (a_hi >= lo) {
        t.a0 = lo / kT;
        t.nA = a_hi / kT - t.a0 + 1;
      }
      if (b > 0) {
        t.b0 = (max(lo, P) - P) / kT;
        t.nB = (last - P) / kT - t.b0 + 1;
      }
    }
    int tot;
    t.base = ntiles + block_scan(t.nA + t.nB, sums, &tot);
    ntiles += tot;
    if (i < nrt) {
      w.rt[i] = t;
      if (nrt <= kS) s_rt[i] = t;
      if (pl.splits > 1 && nl == 1) {                  // (whole numbers: their order does not matter)
        for (int j = 0; j < t.nA; ++j) atomicAdd(counts + t.a0 + j, 1);
        for (int j = 0; j < t.nB; ++j) atomicAdd(counts + ks[t.block] + t.b0 + j, 1);
      }
    }
  }
  __syncthreads();
  // the pieces of every key pair's list: `piece` row tiles or more each with one
  // chunk (by the longer of the two tiles' lists), `splits` with several
  const int nkp = (nkt + 1) / 2;
  int npieces = 0;
  for (int i0 = 0; i0 < nkp; i0 += kPrepThreads) {
    const int i = i0 + tid;
    int cuts = 0;
    if (i < nkp) {
      const volatile int* c = counts;
      const int n = max(c[2 * i], 2 * i + 1 < nkt ? c[2 * i + 1] : 0);
      cuts = nl == 1 ? max(1, min(pl.splits, n / pl.piece)) : pl.splits;
      w.counts[nkt + i] = cuts;
    }
    int tot;
    const int at = npieces + block_scan(cuts, sums, &tot);
    npieces += tot;
    for (int c = 0; c < cuts; ++c) w.list[at + c] = i * kMaxSplits + c;
  }
  // the units of every pair of row tiles
  const int rp = (nrt + 1) / 2;
  int* units = rp <= kS ? s_units : w.units;
  int nunits = 0;
  for (int m0 = 0; m0 < rp; m0 += kPrepThreads) {
    const int m = m0 + tid;
    int n = 0;
    if (m < rp) n = (merged(rt[2 * m], rt[min(2 * m + 1, nrt - 1)], 2 * m + 1 < nrt).n() + 1) / 2;
    int tot;
    const int at = nunits + block_scan(n, sums, &tot);
    nunits += tot;
    if (m < rp) {
      w.units[m] = at;
      if (rp <= kS) s_units[m] = at;
    }
  }
  const int all = rp * a.L.n_kv;
  if (nl == 1) {
    // one chunk, which make_plan's bound holds (were it not to, nothing is written);
    // where each CTA pair of the scores kernel begins
    const bool fits = (long long)ntiles * a.L.n_kv <= cap;
    __syncthreads();
    for (int c = tid; c < pl.pairs && fits; c += kPrepThreads) {
      const long long n = (long long)nunits * a.L.n_kv, u0 = n * c / pl.pairs, u1 = n * (c + 1) / pl.pairs;
      const int rem = (int)(u0 % nunits), m = last_le(units, rp, rem);
      w.begin[c] = make_int4((int)(u1 - u0), (int)(u0 / nunits), m, 2 * (rem - units[m]));
    }
    if (tid == 0) {
      w.chunk[0] = 0;
      w.chunk[1] = fits ? all : 0;
      *w.head = fits ? Head{0u, 1, nrt, nkt, ntiles, npieces, nunits, 0} : Head{1u << KVQ_DEV_BADSEQ, 0, 0, 0, 0, 0, 0, 0};
    }
    return;
  }
  if (tid == 0) {
    // chunks: as many whole pairs of row tiles as fit in cap tiles
    auto before = [&](int x) -> long long {            // tiles before pair x (kv head major)
      return (long long)(x / rp) * ntiles + (x % rp ? w.rt[x % rp * 2].base : 0);
    };
    int x = 0, c = 0;
    w.chunk[0] = 0;
    while (x < all && c < nl) {
      const long long room = before(x) + cap;
      if (before(x + 1) > room) break;
      int lo = x + 1, hi = all;                        // largest end with before(end) <= room
      while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (before(mid) <= room) lo = mid; else hi = mid - 1;
      }
      x = lo;
      w.chunk[++c] = x;
    }
    // make_plan's bounds hold every valid layout; were one to break them, nothing is written
    const bool fits = x == all;
    while (c < nl) w.chunk[++c] = x;
    if (!fits)
      for (int i = 0; i <= nl; ++i) w.chunk[i] = 0;
    *w.head = fits ? Head{0u, 1, nrt, nkt, ntiles, npieces, nunits, 0} : Head{1u << KVQ_DEV_BADSEQ, 0, 0, 0, 0, 0, 0, 0};
  }
}

template <int D>
__global__ void __launch_bounds__(kPrepThreads)
bwd_prep_kernel(const TrainBwdArgs a, const Ws w, const PlanArgs pl) {
  pdl_wait();
  pdl_launch();
  if (blockIdx.x == 0) {
    plan_block(a, w, pl);
    return;
  }
  // the tiles of zeros, 4 KB a block
  for (int i = blockIdx.x - 1; i < (int)(2 * kTileBytes / 4096); i += gridDim.x - 1) {
    uint8_t* z = (i & 1 ? w.ds : w.p) + (size_t)pl.cap * kTileBytes + (i >> 1) * 4096;
    reinterpret_cast<uint4*>(z)[threadIdx.x] = make_uint4(0, 0, 0, 0);
  }
  // delta: one warp per (row, head)
  constexpr int E = D / 32, VEC = E < 8 ? E : 8;
  const int lane = threadIdx.x & 31;
  const long long n = (long long)a.n_rows * a.L.n_q, step = (long long)(gridDim.x - 1) * (kPrepThreads / 32);
  const bool vec = (reinterpret_cast<uintptr_t>(a.out) & 15u) == 0;
  auto partial = [&](long long it) {                  // this lane's part of dO . O
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < E / VEC; ++c) {
      const size_t o = (size_t)it * D + (c * 32 + lane) * VEC;
      float g[VEC], x[VEC];
      uint32_t u[VEC / 2];
      if constexpr (VEC == 8) *reinterpret_cast<uint4*>(u) = __ldg(reinterpret_cast<const uint4*>(a.d_out + o));
      else if constexpr (VEC == 4) *reinterpret_cast<uint2*>(u) = __ldg(reinterpret_cast<const uint2*>(a.d_out + o));
      else u[0] = __ldg(reinterpret_cast<const uint32_t*>(a.d_out + o));
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) {
        g[2 * i] = bf16lo_to_f(u[i]);
        g[2 * i + 1] = bf16hi_to_f(u[i]);
      }
      if (a.out_f32) {
        const float* p = static_cast<const float*>(a.out) + o;
        if (vec && VEC >= 4) {
#pragma unroll
          for (int i = 0; i < VEC; i += 4) *reinterpret_cast<float4*>(x + i) = __ldg(reinterpret_cast<const float4*>(p + i));
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i) x[i] = __ldg(p + i);
        }
      } else {
        const uint16_t* p = static_cast<const uint16_t*>(a.out) + o;
        if (vec && VEC == 8) {
          *reinterpret_cast<uint4*>(u) = __ldg(reinterpret_cast<const uint4*>(p));
#pragma unroll
          for (int i = 0; i < VEC / 2; ++i) {
            x[2 * i] = bf16lo_to_f(u[i]);
            x[2 * i + 1] = bf16hi_to_f(u[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i) x[i] = bf16_to_f(__ldg(p + i));
        }
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) s = fmaf(g[i], x[i], s);
    }
    return s;
  };
  // two of them at a time, for twice the loads in flight
  for (long long it = (long long)(blockIdx.x - 1) * (kPrepThreads / 32) + (threadIdx.x >> 5); it < n; it += 2 * step) {
    const bool both = it + step < n;
    float s0 = partial(it), s1 = both ? partial(it + step) : 0.f;
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) {
      s0 += __shfl_xor_sync(0xffffffffu, s0, m);
      s1 += __shfl_xor_sync(0xffffffffu, s1, m);
    }
    if (lane == 0) {
      w.delta[it] = s0;
      if (both) w.delta[it + step] = s1;
    }
  }
}

// ---------------------------------------------------------------------------
// tensor-core pieces
// ---------------------------------------------------------------------------

// Descriptor of a shared-memory operand without swizzle (8 x 16-byte core
// matrices) or MN-major with rows of 128 or 64 swizzled bytes.
//   K-major, no swizzle:  lbo = next 8 elements of K, sbo = next 8 rows of M
//   MN-major, no swizzle: lbo = next 8 of K, sbo = next 8 elements of M
//   MN-major, swizzled:   lbo = next row's worth of elements of N, sbo = next 8 of K
constexpr int kPlain = 0, kSw128 = 2, kSw64 = 4;
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo, int swizzle) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)swizzle << 61);
}
constexpr uint32_t kTransA = 1u << 15, kTransB = 1u << 16;   // instruction descriptor: MN-major operand

__device__ __forceinline__ void ld_x32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
               "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
               "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                 "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                 "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
                 "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
                 "=r"(r[30]), "=r"(r[31])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// 2^x; a result below the smallest normal float is 0 (no P that small counts)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Two f16, finite: where scores are so large (10^6) that their own rounding takes
// P = exp(S - lse) past 2, it stays below 2 instead of becoming an infinity.
__device__ __forceinline__ uint32_t pack_h2_sat(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// A wait by a whole warp.  One that gives up (kvq_common.cuh) flags the status
// word once and lets the warp run on without waiting, all lanes alike.
struct Waiter {
  uint32_t* status;
  bool dead = false;
  __device__ __forceinline__ void operator()(uint64_t* bar, int parity) {
    const bool ok = !dead && mbar_wait(bar, parity);
    if (__any_sync(0xffffffffu, !ok)) {
      if (!dead) flag_error(status, KVQ_DEV_TIMEOUT);
      dead = true;
    }
  }
  // by one thread alone
  __device__ __forceinline__ void one(uint64_t* bar, int parity) {
    if (!dead && !mbar_wait(bar, parity)) {
      dead = true;
      flag_error(status, KVQ_DEV_TIMEOUT);
    }
  }
};

// ---------------------------------------------------------------------------
// scores: P and dS of one chunk's tiles
// ---------------------------------------------------------------------------

// A pair of CTAs (a cluster of two) works on a pair of row tiles, one each, with
// MMAs of 256 rows x 256 keys: a unit is two of the key tiles that either row
// tile sees, each CTA bringing one of them and its own q and dO.  Shared memory
// is then read and written at 128 bytes a cycle for MMAs at their full rate (a
// CTA alone needs 256 for 128 x 128 and 192 for 128 x 256 and ran at 0.5 and 0.67
// of the rate), and L2 delivers half as much.  S and dP of a unit fill tensor
// memory; the two halves alternate: while the epilogue turns S into P, dP is
// multiplied, and while it turns dP into dS, the next unit's S.  Measured at
// head_dim 512 (2048 rows, 16 heads): 63 us, tensor pipe 47 % busy, operands at 7.9
// of some 9.5 TB/s that L2 delivers: q and dO pass again for every unit, as there
// is no room to keep them (kept, with stages of half the size, 10 % slower).  At 256
// and less they stay, and the epilogue's chain of a unit bounds it.
template <int D>
struct Sc {
  static constexpr int NG = D / 64;
  static constexpr bool RES = D <= 256;               // q and dO of the row tile stay in shared memory
  static constexpr int STAGE = RES ? 16384 : 32768;   // 64 dims of k or v, a tile (with q's or dO's behind)
  static constexpr int NS = D <= 128 ? 8 : 6;
  static constexpr int A_OFF = 0;                     // q, then dO: NG blocks each of [128 rows x 128 B]
  static constexpr int R_OFF = RES ? 2 * NG * 16384 : 0;
  static constexpr int C_OFF = R_OFF + NS * STAGE;
  static constexpr int BYTES = C_OFF + 512 + 1024;    // + room to align the base
};
// Sixteen epilogue warps, a key tile of the unit per eight; a thread's 64 P wait
// for dP as pairs of f16 times 2^15: 11 bits of every P above 2^-29 (8 times finer
// than the bf16 dS they end in), in half the registers of fp32.  Columns come 16
// at a time, so that next to nothing spills: shared memory leaves so little L1
// that reloads go to L2 (with P in fp32 and 32 columns at a time the epilogue took
// 10k cycles a unit for them, now 3k).
constexpr int kScEpi = 16;
constexpr int kScThreads = (kScEpi + 2) * 32;
constexpr float kPScale = 32768.f;

// What the copies tell the other warps of their CTA about a unit.
enum : int { kUnitFresh = 1, kUnitEnd = 2, kUnitLast = 4 };      // another pair of row tiles; no more; another pair follows
constexpr int kUnits = 4;                             // units told ahead
struct alignas(16) Unit {
  int flags, slot[2], lp[2];                          // this CTA's tile slots (-1: not in its list), first positions
  int prefix;                                         // bit t: tile t holds keys of the prefix
  int row0, nt, pos0, kend, kvh, pad;                 // this CTA's row tile
};

// Largest i in [0, n) with a[i] <= x, by the whole warp, 32 probes a step.
__device__ __forceinline__ int find_last_le(const int* a, int n, int x) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = n;                                // the answer is in [lo, lo + len)
  while (len > 1) {
    const int step = (len + 31) / 32;
    const bool le = lane * step < len && __ldg(a + lo + lane * step) <= x;
    const int k = __popc(__ballot_sync(0xffffffffu, le)) - 1;   // probes are non-decreasing, probe 0 holds
    len = min(step, len - k * step);
    lo += k * step;
  }
  return lo;
}
// The plan's records, from L2 (they may be read before the grid below has waited).
template <typename R>
__device__ __forceinline__ R load_plan(const R* src) {
  static_assert(sizeof(R) % 16 == 0 && alignof(R) == 16, "whole 16-byte words");
  R t;
  const int4* s = reinterpret_cast<const int4*>(src);
  int4* d = reinterpret_cast<int4*>(&t);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(R) / 16); ++i) d[i] = __ldcg(s + i);
  return t;
}

template <int D>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kScThreads, 1)
bwd_scores_kernel(const TrainBwdArgs a, const Ws w, const int chunk, const int one_chunk, const __grid_constant__ CUtensorMap tmq,
                  const __grid_constant__ CUtensorMap tmo, const __grid_constant__ CUtensorMap tmk,
                  const __grid_constant__ CUtensorMap tmv) {
  using T = Sc<D>;
  constexpr int NG = T::NG;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ Unit units[kUnits];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* sm = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const uint32_t sb = smem_u32(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)tc::cta_rank();
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + T::C_OFF);      // CTA 0's: both CTAs' copies landed
  uint64_t* empty = full + T::NS;
  uint64_t* a_full = empty + T::NS;                   // [2] CTA 0's: q, dO landed
  uint64_t* a_free = a_full + 2;                      // [2] the row tiles' S, dP are done
  uint64_t* acc_full = a_free + 2;                    // [2] a unit's S, its dP done
  uint64_t* acc_free = acc_full + 2;                  // [2] CTA 0's: read by both epilogues
  uint64_t* unit_full = acc_free + 2;                 // [kUnits]
  uint64_t* unit_empty = unit_full + kUnits;          // [kUnits]
  uint32_t* tslot = reinterpret_cast<uint32_t*>(unit_empty + kUnits);
  if (tid == 0) {
    for (int s = 0; s < T::NS; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(a_full + s, 1);
      mbar_init(a_free + s, 1);
      mbar_init(acc_full + s, 1);
      mbar_init(acc_free + s, 2 * kScEpi);
    }
    for (int s = 0; s < kUnits; ++s) {
      mbar_init(unit_full + s, 1);
      mbar_init(unit_empty + s, kScEpi + (rank == 0 ? 1 : 0));      // the epilogue, and CTA 0's MMA warp
    }
    fence_mbar_init();
  }
  if (warp == 0) {
    tc::tmem_alloc2(tslot, 512);
    tc::tmem_relinquish2();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();                                 // both CTAs' barriers and tensor memory are there
  tc::fence_after_sync();
  const uint32_t tmem = *tslot;
  // the plan and delta; the last chunk's tiles are read.  The next kernel is let
  // go only then, so that it may read the plan before it waits.
  if (warp == kScEpi && lane == 0)
    for (const CUtensorMap* m : {&tmq, &tmo, &tmk, &tmv}) prefetch_map(m);
  if (warp >= kScEpi) {
    pdl_wait();
    pdl_launch();
  }

  const int G = a.L.G;
  Waiter wait{&w.head->status};
  if (warp == kScEpi) {
    // ================= the walk, and copies: this CTA's row tile and one key tile of a unit =================
    const Head hd = *w.head;
    const int x0 = w.chunk[chunk], x1 = w.chunk[chunk + 1], rp = (hd.nrt + 1) / 2;
    int count = 0, kvh = 0, m = 0, j = 0;             // this pair's units; kv head, pair of row tiles, next key tile of its list
    long long c0 = 0;                                 // tiles before the chunk
    if (one_chunk) {                                  // (one round of loads: the chain below counts in a short call)
      const int4 b = w.begin[blockIdx.x / 2];
      count = x0 < x1 ? b.x : 0;
      kvh = b.y;
      m = b.z;
      j = b.w;
    } else if (x0 < x1) {
      auto before = [&](int x) { return (long long)(x / rp) * hd.nunits + (x % rp ? __ldg(w.units + x % rp) : 0); };
      const long long b0 = before(x0), n = before(x1) - b0;
      const long long u0 = b0 + n * (blockIdx.x / 2) / (gridDim.x / 2), u1 = b0 + n * (blockIdx.x / 2 + 1) / (gridDim.x / 2);
      count = (int)(u1 - u0);
      c0 = (long long)(x0 / rp) * hd.ntiles + (x0 % rp ? __ldg(&w.rt[x0 % rp * 2].base) : 0);
      kvh = (int)(u0 / hd.nunits);
      const int rem = (int)(u0 % hd.nunits);
      if (count > 0) {
        m = find_last_le(w.units, rp, rem);
        j = 2 * (rem - __ldg(w.units + m));
      }
    }
    if (lane == 0) {
      const uint32_t full0 = tc::in_cta0(full), a_full0 = tc::in_cta0(a_full);
      int st = 0, ph = 0, pairs = 0, n = 0;
      bool fresh = true, two = false;
      RowTile r0 = {}, r1 = {};
      Merged u = {};
      for (; n < count; ++n) {
        if (fresh) {
          r0 = load_plan(w.rt + 2 * m);
          two = 2 * m + 1 < hd.nrt;
          r1 = load_plan(w.rt + (two ? 2 * m + 1 : 2 * m));
          u = merged(r0, r1, two);
        }
        const bool more = j + 1 < u.n();
        const MergedTile t0 = merged_at(u, r0, r1, two, j), t1 = merged_at(u, r0, r1, two, more ? j + 1 : j);
        const int k0 = rank == 0 ? t0.j0 : t0.j1, k1 = !more ? -1 : rank == 0 ? t1.j0 : t1.j1;
        const int base = (int)((long long)kvh * hd.ntiles - c0 + (rank == 0 ? r0.base : r1.base));
        const int row0 = rank == 0 ? r0.row0 : r1.row0, pk = rank == 0 ? t0.pk : t1.pk, e = n % kUnits;
        wait.one(unit_empty + e, (n / kUnits & 1) ^ 1);
        Unit& un = units[e];
        un.flags = (fresh ? kUnitFresh : 0) | (j + 2 >= u.n() && n + 1 < count ? kUnitLast : 0);
        un.slot[0] = k0 < 0 ? -1 : base + k0;
        un.slot[1] = k1 < 0 ? -1 : base + k1;
        un.lp[0] = t0.lp;
        un.lp[1] = t1.lp;
        un.prefix = (t0.prefix ? 1 : 0) | (t1.prefix ? 2 : 0);
        un.row0 = row0;
        un.nt = rank == 0 ? r0.nt : two ? r1.nt : 0;
        un.pos0 = rank == 0 ? r0.pos0 : r1.pos0;
        un.kend = rank == 0 ? r0.kend : r1.kend;
        un.kvh = kvh;
        mbar_arrive(unit_full + e);
        for (int c = 0; c < 2 * NG; ++c) {
          if (T::RES && fresh && c % NG == 0) {       // q before k, dO before v
            const int half = c / NG;
            if (pairs > 0) wait.one(a_free + half, (pairs - 1) & 1);
            if (rank == 0) mbar_arrive_expect_tx(a_full + half, 2 * NG * 16384);
            for (int b = 0; b < NG; ++b)
              tc::tma2_load_3d(sb + T::A_OFF + (c + b) * 16384, half ? &tmo : &tmq, 64 * b, kvh * G, row0, a_full0 + 8 * half);
            pairs += half;
          }
          wait.one(empty + st, ph ^ 1);
          const int dim = 64 * (c < NG ? c : c - NG);
          const uint32_t dst = sb + T::R_OFF + st * T::STAGE, bar = full0 + 8 * st;
          if (rank == 0) mbar_arrive_expect_tx(full + st, 2 * T::STAGE);
          tc::tma2_load_3d(dst, c < NG ? &tmk : &tmv, dim, kvh, pk, bar);
          if (!T::RES) tc::tma2_load_3d(dst + 16384, c < NG ? &tmq : &tmo, dim, kvh * G, row0, bar);
          if (++st == T::NS) {
            st = 0;
            ph ^= 1;
          }
        }
        j += 2;
        fresh = j >= u.n();
        if (fresh) {
          j = 0;
          if (++m == rp) {
            m = 0;
            ++kvh;
          }
        }
      }
      wait.one(unit_empty + n % kUnits, (n / kUnits & 1) ^ 1);
      units[n % kUnits].flags = kUnitEnd;
      mbar_arrive(unit_full + n % kUnits);
      // every stage consumed, in both CTAs, before either may leave
      for (int i = 0; i < T::NS; ++i) {
        wait.one(empty + st, ph ^ 1);
        if (++st == T::NS) {
          st = 0;
          ph ^= 1;
        }
      }
    }
    __syncwarp();
  } else if (warp == kScEpi + 1) {
    // ================= S = q k^T, dP = dO v^T (CTA 0, for both) =================
    constexpr uint32_t ID = tc::idesc_bf16_f32(2 * kT, 2 * kT);
    int st = 0, ph = 0, pairs = 0;
    for (int n = 0; rank == 0; ++n) {
      const int e = n % kUnits;
      wait(unit_full + e, n / kUnits & 1);
      const int flags = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&units[e].flags), 0);
      if (lane == 0) mbar_arrive(unit_empty + e);
      if ((flags & kUnitEnd) || wait.dead) break;
      for (int c = 0; c < 2 * NG; ++c) {
        const int half = c >= NG;
        if (T::RES && (flags & kUnitFresh) && c % NG == 0) {
          wait(a_full + half, pairs & 1);
          pairs += half;
        }
        if (n > 0 && (c == 0 || c == NG)) wait(acc_free + half, (n - 1) & 1);
        wait(full + st, ph);
        tc::fence_after_sync();
        if (lane == 0) {
          const uint32_t bs = sb + T::R_OFF + st * T::STAGE;
          const uint32_t as = T::RES ? sb + T::A_OFF + c * 16384 : bs + 16384;
#pragma unroll
          for (int s = 0; s < 4; ++s)
            tc::mma2_f16(tmem + 256 * half, tc::desc_kmajor_sw128(as + 32 * s, 1024),
                         tc::desc_kmajor_sw128(bs + 32 * s, 1024), ID, (c != 0 && c != NG) || s != 0);
          tc::commit2(empty + st);
          if (c == NG - 1 || c == 2 * NG - 1) {
            if (T::RES && (flags & kUnitLast)) tc::commit2(a_free + half);
            tc::commit2(acc_full + half);
          }
        }
        __syncwarp();
        if (++st == T::NS) {
          st = 0;
          ph ^= 1;
        }
      }
    }
  } else {
    // ================= P and dS: thread = row, half hh of one key tile of the unit =================
    const int r = 32 * (warp & 3) + lane, mine = warp >> 3, hh = warp >> 2 & 1, W = a.L.window;
    const int tq = r / G, h = r % G;
    const uint32_t ts = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + kT * mine + 64 * hh;
    float lse2 = 0.f, delta = 0.f;                    // log2(e) lse, delta / 2^15
    int lo = 0, hi = -1, cut = -1;                    // visible positions: lo .. hi, in prefix tiles lo .. cut
    // Round -1 is a rehearsal on whatever tensor memory holds, with nothing waited
    // for, told or stored: the straight-line code below (15 KB) then comes from the
    // instruction cache, while the plan and the first copies are still on their way
    // (a first unit took 10k cycles instead of 5k).
    for (int n = -1;; ++n) {
      const bool real = n >= 0;
      if (n == 0) {                                   // delta; the last chunk's tiles are read
        pdl_wait();
        pdl_launch();
      }
      Unit un = {};
      if (real) {
        const int e = n % kUnits;
        wait(unit_full + e, n / kUnits & 1);
        un = units[e];
        __syncwarp();
        if (lane == 0) mbar_arrive(unit_empty + e);
        if ((un.flags & kUnitEnd) || wait.dead) break;
      }
      if (un.flags & kUnitFresh) {
        const bool valid = tq < un.nt;
        const int pos = un.pos0 + tq;
        lo = W > 0 ? max(0, pos - W + 1) : 0;
        hi = valid ? pos : -1;
        cut = valid ? min(pos, un.kend - 1) : -1;
        if (valid) {
          const size_t o = (size_t)(un.row0 + tq) * a.L.n_q + un.kvh * G + h;
          lse2 = __ldg(a.lse + o) * kL2E;
          delta = w.delta[o] * (1.f / kPScale);
        }
      }
      const int slot = mine ? un.slot[1] : un.slot[0], lp = (mine ? un.lp[1] : un.lp[0]) + 64 * hh;
      const bool busy = slot >= 0;
      const int top = un.prefix >> mine & 1 ? cut : hi;
      // (a row that sees one key does not see 64: it always takes the masked form)
      const bool whole = __all_sync(0xffffffffu, lp >= lo && lp + 63 <= top);
      const size_t at = (size_t)(busy ? slot : 0) * kTileBytes + hh * 16384 + r * 16;
      uint32_t ph[32];
      if (real) wait(acc_full, n & 1);
      tc::fence_after_sync();
      __syncwarp();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float p[16];
        if (busy) {
          tc::ld_x16(ts + 16 * q, p);
          tc::wait_ld();
        }
        if (q == 3) {                       // S is read
          tc::fence_before_sync();
          __syncwarp();
          if (real && lane == 0) tc::arrive_cta0(acc_free);
        }
        if (busy) {
#pragma unroll
          for (int i = 0; i < 16; ++i) p[i] = ex2(fmaf(p[i], kL2E, -lse2));
          if (!whole) {
#pragma unroll
            for (int i = 0; i < 16; ++i) p[i] = lp + 16 * q + i >= lo && lp + 16 * q + i <= top ? p[i] : 0.f;
          }
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (real) *reinterpret_cast<uint4*>(w.p + at + (2 * q + c) * 2048) =
                make_uint4(pack_bf2(p[8 * c], p[8 * c + 1]), pack_bf2(p[8 * c + 2], p[8 * c + 3]),
                           pack_bf2(p[8 * c + 4], p[8 * c + 5]), pack_bf2(p[8 * c + 6], p[8 * c + 7]));
#pragma unroll
          for (int i = 0; i < 8; ++i) ph[8 * q + i] = pack_h2_sat(p[2 * i] * kPScale, p[2 * i + 1] * kPScale);
        }
      }
      if (!whole && lo >= hi) {                       // one key: dS = 0
#pragma unroll
        for (int i = 0; i < 32; ++i) ph[i] = 0u;
      }
      if (real) wait(acc_full + 1, n & 1);
      tc::fence_after_sync();
      __syncwarp();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float d[16];
        if (busy) {
          tc::ld_x16(ts + 256 + 16 * q, d);
          tc::wait_ld();
        }
        if (q == 3) {                       // dP is read
          tc::fence_before_sync();
          __syncwarp();
          if (real && lane == 0) tc::arrive_cta0(acc_free + 1);
        }
        if (busy) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&ph[8 * q + i]));
            d[2 * i] = p.x * fmaf(d[2 * i], 1.f / kPScale, -delta);
            d[2 * i + 1] = p.y * fmaf(d[2 * i + 1], 1.f / kPScale, -delta);
          }
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (real) *reinterpret_cast<uint4*>(w.ds + at + (2 * q + c) * 2048) =
                make_uint4(pack_bf2(d[8 * c], d[8 * c + 1]), pack_bf2(d[8 * c + 2], d[8 * c + 3]),
                           pack_bf2(d[8 * c + 4], d[8 * c + 5]), pack_bf2(d[8 * c + 6], d[8 * c + 7]));
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();                                 // neither CTA's memory is written or read any more
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc2(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// products: out[128 x N] = sum over steps of A_t (128 x 64) B_t (64 x N)
// ---------------------------------------------------------------------------
// An item is a pair of tiles (two row tiles for dq, two key tiles for dk or dv)
// times N head dims, and a pair of CTAs (a cluster of two) works on it with
// MMAs of 256 rows: each CTA brings its own tile's A and half of B, so that
// shared memory is read at half the rate one CTA's MMA needs (bound by that and
// by what L2 delivers, a CTA alone reached 0.6 of the rate) and the accumulators
// fit tensor memory twice: an item's output runs under the next item's products.
// The list of row tiles of a key pair is cut into pieces, each with its own
// sums.  A tile that a step's other tile sees alone is a tile of zeros.  The CTA
// pairs stay resident and draw the items from a counter (in turn, the last of them
// ended 18 us after the first).  Measured at head_dim 512 (2048 rows, 16 heads): 78
// us, tensor pipe 53 % busy, L2 at 9.5 TB/s, which bounds it with the items' ends.
// At 128 P and dS are two thirds of what it reads and come from DRAM where they
// are more than L2 holds.

// A step is a whole tile: 128 rows (or keys) of K in one stage, three copies (a
// copy takes the issuing thread some 150 cycles; with stages of 64 the copies
// took longer than their MMAs).
constexpr int kBatches = 2, kBatch = 4;                       // of steps listed ahead, and steps of one
constexpr int kItems = 4;                                     // items told to the epilogue ahead
template <int N>
struct Pr {
  static constexpr int A_BYTES = kTileBytes;                  // 128 x 128 of P or dS
  static constexpr int DIMS = N / 2;                          // of B per CTA
  static constexpr int BOX = DIMS < 64 ? DIMS : 64;           // per copy
  static constexpr int B_BYTES = DIMS * 256;                  // 128 rows
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int NS = N == 256 ? 3 : 4;
  static constexpr int E_OFF = NS * STAGE;                    // 4 KB per output warp
  static constexpr int L_OFF = E_OFF + 8 * 4096;              // the copies' list
  static constexpr int C_OFF = L_OFF + kBatches * kBatch * 16;
  static constexpr int BYTES = C_OFF + 512 + 1024;
};
constexpr int kPrEpi = 8;
constexpr int kPrThreads = (kPrEpi + 3) * 32;

// What the copies tell the MMA warp about a stage.
enum : int { kFirst = 1, kLast = 2, kKeys = 4, kEnd = 8, kQ = 16 };   // kKeys: dk or dv, with kQ dk

struct Item {
  bool dkv;
  int kind, half, kvh, split;   // kind 0: dk = dS^T q, 1: dv = P^T dO
  int t0, n;                    // first tile of the pair (key tile, or row tile of the kv head) and tiles (1, 2)
};

struct ProdArgs {
  int chunk;
  int zero;                     // slot of a tile of zeros
  int direct;                   // 1: dk and dv go straight to the outputs
};

template <int D>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPrThreads, 1)
bwd_products_kernel(const TrainBwdArgs a, const Ws w, const ProdArgs pa, const __grid_constant__ CUtensorMap tmq,
                    const __grid_constant__ CUtensorMap tmo, const __grid_constant__ CUtensorMap tmk,
                    const __grid_constant__ CUtensorMap tmp, const __grid_constant__ CUtensorMap tmd) {
  constexpr int N = prod_n(D), H = D / N;
  using T = Pr<N>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* sm = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const uint32_t sb = smem_u32(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)tc::cta_rank();
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + T::C_OFF);      // CTA 0's: both CTAs' copies landed
  uint64_t* empty = full + T::NS;
  uint64_t* done = empty + T::NS;                     // [2] an item's products are in tensor memory
  uint64_t* acc_free = done + 2;                      // [2] CTA 0's: and read from it, in both CTAs
  uint64_t* item_full = acc_free + 2;                 // [kItems]
  uint64_t* item_empty = item_full + kItems;          // [kItems]
  uint64_t* list_full = item_empty + kItems;          // [kBatches]
  uint64_t* list_empty = list_full + kBatches;        // [kBatches]
  uint64_t* mail_full = list_empty + kBatches;        // [2] CTA 1's: the next item's number
  uint64_t* mail_empty = mail_full + 2;               // [2] CTA 0's
  uint32_t* tslot = reinterpret_cast<uint32_t*>(mail_empty + 2);
  volatile int* info = reinterpret_cast<volatile int*>(tslot + 1);   // [NS] stage flags (CTA 0)
  volatile int* items = info + T::NS;                 // [kItems][2]: item (-1: no more), its steps
  volatile int* list_n = items + 2 * kItems;          // [kBatches] steps of a batch (0: no more)
  volatile int* mail = list_n + kBatches;             // [2] (CTA 1)
  int4* list = reinterpret_cast<int4*>(sm + T::L_OFF);
  if (tid == 0) {
    for (int s = 0; s < T::NS; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(done + s, 1);
      mbar_init(acc_free + s, 2 * kPrEpi);
      mbar_init(mail_full + s, 1);
      mbar_init(mail_empty + s, 1);
    }
    for (int s = 0; s < kItems; ++s) {
      mbar_init(item_full + s, 1);
      mbar_init(item_empty + s, kPrEpi);
    }
    for (int s = 0; s < kBatches; ++s) {
      mbar_init(list_full + s, 1);
      mbar_init(list_empty + s, 1);
    }
    fence_mbar_init();
  }
  if (warp == 0) {
    tc::tmem_alloc2(tslot, 512);
    tc::tmem_relinquish2();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();                                 // both CTAs' barriers and tensor memory are there
  tc::fence_after_sync();
  const uint32_t tmem = *tslot;
  // (the warp that lists the items needs the plan alone, which the scores kernel
  // has waited for before this one could start: the lists of a CTA's first items
  // are there when P and dS are, 4 to 7 us sooner)
  if (warp == kPrEpi && lane == 0)
    for (const CUtensorMap* m : {&tmq, &tmo, &tmk, &tmp, &tmd}) prefetch_map(m);
  if (warp != kPrEpi + 2) pdl_wait();
  pdl_launch();

  const Head hd = load_plan(w.head);
  const int G = a.L.G, nkv = a.L.n_kv;
  const int x0 = __ldcg(w.chunk + pa.chunk), x1 = __ldcg(w.chunk + pa.chunk + 1);
  // Items kv head by kv head, the last first: its tiles are the newest in L2, and dq
  // meets the dS that dk has just read.  Of a head dk and dv come first (the longest
  // sums).  An empty chunk (or layout) has no items.
  const int rp = (hd.nrt + 1) / 2, n_dkv = hd.npieces * 2 * H;       // (of one kv head)
  const int n_items = x0 < x1 ? n_dkv * nkv + (x1 - x0) * H : 0;
  const long long c0 = x0 < x1 ? (long long)(x0 / rp) * hd.ntiles + __ldcg(&w.rt[x0 % rp * 2].base) : 0;
  auto decode = [&](int id) {
    Item t;
    auto above = [&](int h) { return n_dkv * (nkv - 1 - h) + H * max(0, x1 - max(x0, (h + 1) * rp)); };
    int lo = 0, hi = nkv - 1;                         // the least head with no more items above it than id
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (above(mid) <= id) hi = mid; else lo = mid + 1;
    }
    id -= above(lo);
    t.kvh = lo;
    t.dkv = id < n_dkv;
    if (!t.dkv) id -= n_dkv;
    t.half = id % H;
    id /= H;
    t.kind = t.split = 0;
    if (t.dkv) {
      t.kind = id % 2;
      id = __ldcg(w.list + id / 2);
      t.split = id % kMaxSplits;
      t.t0 = id / kMaxSplits * 2;
      t.n = min(2, hd.nkt - t.t0);
    } else {
      t.t0 = (max(x0 - lo * rp, 0) + id) * 2;
      t.n = min(2, hd.nrt - t.t0);
    }
    return t;
  };
  Waiter wait{&w.head->status};

  if (warp == kPrEpi + 2) {
    // ================= the items' steps, listed ahead for the copies =================
    // (a list costs several dependent loads, as long as a few steps' products)
    int e = 0, eph = 0, b = 0, bph = 0;
    auto publish = [&](int id, int n) {
      wait(item_empty + e, eph ^ 1);
      if (lane == 0) {
        items[2 * e] = id;
        items[2 * e + 1] = n;
        mbar_arrive(item_full + e);
      }
      __syncwarp();
      if (++e == kItems) {
        e = 0;
        eph ^= 1;
      }
    };
    auto hand_over = [&](int n) {
      __syncwarp();
      if (lane == 0) {
        list_n[b] = n;
        mbar_arrive(list_full + b);
      }
      __syncwarp();
      if (++b == kBatches) {
        b = 0;
        bph ^= 1;
      }
    };
    // The items are taken from a counter, the longest first: CTA 0 draws one as soon
    // as the last's final steps are listed (four to eight of them still to copy) and
    // sends its number to CTA 1.  Who takes an item does not show in the results.
    auto draw = [&](int k) {
      const int slot = k & 1, parity = k >> 1 & 1;
      int id = 0;
      if (rank == 0) {
        wait(mail_empty + slot, parity ^ 1);
        if (lane == 0) {
          id = (int)(gridDim.x / 2) + atomicAdd(w.next + pa.chunk, 1);
          tc::send_cta1(const_cast<int*>(mail + slot), id, mail_full + slot);
        }
        id = __shfl_sync(0xffffffffu, id, 0);
      } else {
        if (lane == 0) mbar_arrive_expect_tx(mail_full + slot, 4);
        __syncwarp();
        wait(mail_full + slot, parity);
        id = mail[slot];
        __syncwarp();
        if (lane == 0) tc::arrive_cta0_release(mail_empty + slot);
      }
      return wait.dead ? n_items : id;
    };
    for (int id = blockIdx.x / 2, k = 0; id < n_items; id = draw(k++)) {
      const Item it = decode(id);
      const long long slot0 = (long long)it.kvh * hd.ntiles - c0;    // slot of the kv head's first tile
      const int place = it.kvh << 10 | (it.half * N + rank * T::DIMS), kind = it.dkv ? kKeys | (it.kind == 0 ? kQ : 0) : 0;
      int at = 0, n = 0;                              // steps listed, steps of the item
      // steps, one a lane where `see`: s0 and s1 (-1: not there) are the tiles
      // of the pair, `row` the first of the 128 rows of B that they meet
      auto batch = [&](bool see, int s0, int s1, int row) {
        const uint32_t m = __ballot_sync(0xffffffffu, see);
        const int x = __popc(m & ((1u << lane) - 1)), mine = rank == 0 ? s0 : s1, steps = __popc(m);
        for (int from = 0; from < steps; from += kBatch) {
          wait(list_empty + b, bph ^ 1);
          if (see && x >= from && x < from + kBatch)
            list[kBatch * b + x - from] = make_int4(mine >= 0 ? mine : pa.zero, row, place,
                                                    kind | (at + x == 0 ? kFirst : 0) | (at + x == n - 1 ? kLast : 0));
          hand_over(min(kBatch, steps - from));
        }
        at += steps;
      };
      if (it.dkv) {
        // the chunk's row tiles that see either key tile; this piece's share of them by count
        const KeyTile ka = load_plan(w.kt + it.t0), kb = load_plan(w.kt + it.t0 + it.n - 1);
        const int cuts = __ldcg(w.counts + hd.nkt + it.t0 / 2);
        const int xs = max(2 * (x0 - it.kvh * rp), min(ka.lo, kb.lo));
        const int xe = min(2 * (x1 - it.kvh * rp), max(ka.hi, kb.hi));
        auto tile_of = [&](const KeyTile& t, const RowTile& r) -> int {      // its place in the row tile's list
          if (t.block == 0) return t.idx >= r.a0 && t.idx < r.a0 + r.nA ? t.idx - r.a0 : -1;
          return t.block == r.block && t.idx >= r.b0 && t.idx < r.b0 + r.nB ? r.nA + t.idx - r.b0 : -1;
        };
        int all = 0, count = 0;                       // lane g: of the g-th 32 row tiles
        RowTile r = {}, head = {};                    // (the first 32 are kept: in a short call they are all)
#pragma unroll 4
        for (int i = xs; i < xe; i += 32) {
          bool see = false;
          if (i + lane < xe) {
            r = load_plan(w.rt + i + lane);
            see = tile_of(ka, r) >= 0 || tile_of(kb, r) >= 0;
            if (i == xs) head = r;
          }
          const int c = __popc(__ballot_sync(0xffffffffu, see));
          if ((i - xs) / 32 == lane) count = c;
          all += c;
        }
        const int v0 = (int)((long long)all * it.split / cuts), v1 = (int)((long long)all * (it.split + 1) / cuts);
        n = v1 - v0;
        publish(id, n);
        int seen = 0;
        for (int i = xs, g = 0; i < xe && seen < v1; i += 32, ++g) {
          if (g < 32) {                               // all of another piece
            const int c = __shfl_sync(0xffffffffu, count, g);
            if (seen + c <= v0) {
              seen += c;
              continue;
            }
          }
          int j0 = -1, j1 = -1, row = 0;
          if (i + lane < xe) {
            if (g == 0) r = head;
            else r = load_plan(w.rt + i + lane);
            j0 = tile_of(ka, r);
            j1 = it.n == 2 ? tile_of(kb, r) : -1;
            const int base = (int)(slot0 + r.base);
            j0 += j0 >= 0 ? base : 0;
            j1 += j1 >= 0 ? base : 0;
            row = r.row0;
          }
          const uint32_t m = __ballot_sync(0xffffffffu, j0 >= 0 || j1 >= 0);
          const int mine = seen + __popc(m & ((1u << lane) - 1));
          batch((m >> lane & 1) && mine >= v0 && mine < v1, j0, j1, row);
          seen += __popc(m);
        }
      } else {
        // the key tiles that either row tile sees
        const bool two = it.n == 2;
        const RowTile r0 = load_plan(w.rt + it.t0), r1 = load_plan(w.rt + it.t0 + it.n - 1);
        const Merged u = merged(r0, r1, two);
        const int base0 = (int)(slot0 + r0.base), base1 = (int)(slot0 + r1.base);
        auto sees = [&](int j, MergedTile& t) {
          if (j >= u.n()) return false;
          t = merged_at(u, r0, r1, two, j);
          return t.j0 >= 0 || t.j1 >= 0;
        };
        MergedTile t = {};
        for (int j = 0; j < u.n(); j += 32) n += __popc(__ballot_sync(0xffffffffu, sees(j + lane, t)));
        publish(id, n);
        for (int j = 0; j < u.n(); j += 32) {
          const bool see = sees(j + lane, t);
          batch(see, t.j0 < 0 ? -1 : base0 + t.j0, t.j1 < 0 ? -1 : base1 + t.j1, t.pk);
        }
      }
    }
    publish(-1, 0);
    wait(list_empty + b, bph ^ 1);
    hand_over(0);
  } else if (warp == kPrEpi) {
    // ================= copies: this CTA's tile of A and half of B =================
    if (lane == 0) {
      int st = 0, ph = 0;
      const uint32_t bar0 = tc::in_cta0(full);
      for (int b = 0, bph = 0;;) {
        wait.one(list_full + b, bph);
        const int n = wait.dead ? 0 : list_n[b];
        if (n == 0) break;
        for (int x = 0; x < n; ++x) {
          const int4 s = list[kBatch * b + x];            // tile, first row of B, kv head and dims, flags
          wait.one(empty + st, ph ^ 1);
          const uint32_t dst = sb + st * T::STAGE, bar = bar0 + 8 * st;
          if (rank == 0) {
            info[st] = s.w;
            mbar_arrive_expect_tx(full + st, 2 * T::STAGE);
          }
          const bool keys = s.w & kKeys, of_q = s.w & kQ;
          const int kvh = s.z >> 10, dim = s.z & 1023;
          tc::tma2_load_4d(dst, keys && !of_q ? &tmp : &tmd, 0, 0, 0, s.x, bar);
#pragma unroll
          for (int i = 0; i < T::DIMS / T::BOX; ++i)
            tc::tma2_load_3d(dst + T::A_BYTES + i * 16384, !keys ? &tmk : of_q ? &tmq : &tmo, dim + T::BOX * i,
                             keys ? kvh * G : kvh, s.y, bar);
          if (++st == T::NS) {
            st = 0;
            ph ^= 1;
          }
        }
        mbar_arrive(list_empty + b);
        if (++b == kBatches) {
          b = 0;
          bph ^= 1;
        }
      }
      // every stage consumed, in both CTAs, before either may leave
      const int st1 = st;
      for (int i = 0; i < T::NS; ++i) {
        wait.one(empty + st, ph ^ 1);
        if (++st == T::NS) {
          st = 0;
          ph ^= 1;
        }
      }
      if (rank == 0) {
        info[st1] = kEnd;
        mbar_arrive(full + st1);
      }
    }
    __syncwarp();
  } else if (warp == kPrEpi + 1) {
    // ================= products (CTA 0, for both) =================
    int st = 0, ph = 0, use = 0;
    bool started = false;
    while (rank == 0) {
      wait(full + st, ph);
      const int f = __shfl_sync(0xffffffffu, info[st], 0);   // (every lane is here before lane 0 goes on)
      if ((f & kEnd) || wait.dead) break;
      const int buf = use & 1;
      if (f & kFirst) {
        if (use >= 2) wait(acc_free + buf, ((use >> 1) - 1) & 1);
        started = false;
      }
      tc::fence_after_sync();
      if (lane == 0) {
        const uint32_t ID = tc::idesc_bf16_f32(2 * kT, N) | kTransB | (f & kKeys ? kTransA : 0u);
        const uint32_t as = sb + st * T::STAGE, bs = as + T::A_BYTES;
        constexpr uint32_t ROW = T::BOX * 2;          // bytes of a row of B
#pragma unroll
        for (int s = 0; s < 8; ++s)
          tc::mma2_f16(tmem + buf * N,
                       f & kKeys ? smem_desc(as + 256 * s, 128, 2048, kPlain) : smem_desc(as + 4096 * s, 2048, 128, kPlain),
                       smem_desc(bs + 16 * ROW * s, 16384, 8 * ROW, T::BOX == 64 ? kSw128 : kSw64), ID, started || s > 0);
        tc::commit2(empty + st);
        if (f & kLast) tc::commit2(done + buf);
      }
      __syncwarp();
      started = true;
      if (f & kLast) ++use;
      if (++st == T::NS) {
        st = 0;
        ph ^= 1;
      }
    }
  } else {
    // ================= out: warp = 32 rows of this CTA's tile, half of the columns =================
    uint8_t* stg = sm + T::E_OFF + warp * 4096;
    int e = 0, eph = 0, use = 0;
    const size_t plane = (size_t)a.n_rows * nkv * D;
    for (;;) {
      wait(item_full + e, eph);
      const int id = items[2 * e], steps = items[2 * e + 1];
      if (id < 0 || wait.dead) break;
      const Item it = decode(id);
      const int buf = use & 1;
      const bool has = steps > 0;
      if (has) {
        wait(done + buf, (use >> 1) & 1);
        tc::fence_after_sync();
      }
      __syncwarp();
      // where the tile's rows go: row r at o + (r >> sh) * big + (r & ((1 << sh) - 1)) * D
      size_t o = 0, big;
      int rows = 0, sh;
      if (it.dkv) {
        sh = 0;
        big = (size_t)nkv * D;
        if (rank < it.n) {
          const KeyTile k = load_plan(w.kt + it.t0 + rank);
          rows = k.n;
          o = ((size_t)k.row0 * nkv + it.kvh) * D;
        }
      } else {
        sh = 31 - __clz(G);
        big = (size_t)a.L.n_q * D;
        if (rank < it.n) {
          const RowTile r = load_plan(w.rt + it.t0 + rank);
          rows = r.nt * G;
          o = ((size_t)r.row0 * a.L.n_q + it.kvh * G) * D;
        }
      }
      o += it.half * N;
      auto at = [&](int r) { return o + (size_t)(r >> sh) * big + (size_t)(r & ((1 << sh) - 1)) * D; };
      void* out = it.dkv ? (it.kind == 0 ? a.dk : a.dv) : a.dq;
      const bool part = it.dkv && !pa.direct, f32 = part || (it.dkv && a.dkv_f32);
      const bool add = it.dkv && (pa.direct ? a.accumulate != 0 : pa.chunk > 0);
      if (part) out = w.acc + ((size_t)it.split * 2 + it.kind) * plane;
      const bool vec = (reinterpret_cast<uintptr_t>(out) & 15u) == 0;
      const int r0 = 32 * (warp & 3), n0 = (warp >> 2) * (N / 2);
      const uint32_t ta = tmem + ((uint32_t)r0 << 16) + buf * N;
      const bool write = rows > r0 && (has || !add);
      for (int c = n0; c < n0 + N / 2 && write; c += 32) {
        float v[32];
        if (has) {
          ld_x32(ta + c, v);
          tc::wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0.f;
        }
        if (!vec) {                                   // an output that is only aligned to its elements
          if (r0 + lane < rows) {
            const size_t p = at(r0 + lane) + c;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (f32) static_cast<float*>(out)[p + i] = add ? static_cast<float*>(out)[p + i] + v[i] : v[i];
              else static_cast<uint16_t*>(out)[p + i] = f_to_bf16_rn(v[i]);
            }
          }
          continue;
        }
        // through shared memory, so that 8 (4) lanes write a row's 128 (64) bytes
        if (f32) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<float4*>(stg + lane * 128 + ((q ^ (lane & 7)) << 4)) =
                make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
          __syncwarp();
          const int q = lane & 7;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3);
            float4 x = *reinterpret_cast<const float4*>(stg + r * 128 + ((q ^ (r & 7)) << 4));
            if (r0 + r < rows) {
              float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + at(r0 + r) + c + 4 * q);
              if (add) {
                const float4 y = *p;
                x = make_float4(y.x + x.x, y.y + x.y, y.z + x.z, y.w + x.w);
              }
              *p = x;
            }
          }
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint4*>(stg + lane * 64 + ((q ^ (lane >> 1 & 3)) << 4)) =
                make_uint4(pack_bf2(v[8 * q], v[8 * q + 1]), pack_bf2(v[8 * q + 2], v[8 * q + 3]),
                           pack_bf2(v[8 * q + 4], v[8 * q + 5]), pack_bf2(v[8 * q + 6], v[8 * q + 7]));
          __syncwarp();
          const int q = lane & 3;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 8 * i + (lane >> 2);
            const uint4 x = *reinterpret_cast<const uint4*>(stg + r * 64 + ((q ^ (r >> 1 & 3)) << 4));
            if (r0 + r < rows) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at(r0 + r) + c + 8 * q) = x;
          }
        }
        __syncwarp();
      }
      if (has) {
        tc::fence_before_sync();
        ++use;
      }
      __syncwarp();
      if (lane == 0) {
        if (has) tc::arrive_cta0(acc_free + buf);
        mbar_arrive(item_empty + e);
      }
      if (++e == kItems) {
        e = 0;
        eph ^= 1;
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();                                 // neither CTA's memory is written or read any more
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc2(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// finish: dk and dv over the splits, in split order
// ---------------------------------------------------------------------------
// Reads the pieces' sums from L2 (up to 8 x 8 MB at 2048 rows of 512) and writes the
// outputs: 13 us there, latency; four rows a block, all pieces of a word in flight
// (two at a time, and larger shares: 14 to 19 us), read as data that no one reads
// again (the whole call on 2048 rows with a window of 512: 54.4 us, else 55.4).
__global__ void __launch_bounds__(256) bwd_finish_kernel(const TrainBwdArgs a, const Ws w) {
  pdl_wait();
  pdl_launch();
  const int nkt = w.head->nkt;                        // (0 for a layout that breaks the rules)
  const size_t plane = (size_t)a.n_rows * a.L.n_kv * a.L.D;
  const int kind = blockIdx.z, D = a.L.D;
  void* out = kind == 0 ? a.dk : a.dv;
  const bool vec = (reinterpret_cast<uintptr_t>(out) & 15u) == 0;
  // block (x, y): key tiles x, x + grid, ..., a share y of their rows
  for (int t = blockIdx.x; t < nkt; t += gridDim.x) {
    const KeyTile k = w.kt[t];
    const int pieces = w.counts[nkt + t / 2];
    const int per = kT / gridDim.y, r0 = blockIdx.y * per, quads = min(per, k.n - r0) * a.L.n_kv * (D / 4);
    for (int q = threadIdx.x; q < quads; q += 256) {
      const size_t e = ((size_t)(k.row0 + r0) * a.L.n_kv * (D / 4) + q) * 4;
      float4 s = __ldcs(reinterpret_cast<const float4*>(w.acc + kind * plane + e));
#pragma unroll 7
      for (int i = 1; i < pieces; ++i) {
        const float4 y = __ldcs(reinterpret_cast<const float4*>(w.acc + ((size_t)i * 2 + kind) * plane + e));
        s = make_float4(s.x + y.x, s.y + y.y, s.z + y.z, s.w + y.w);
      }
      const float v[4] = {s.x, s.y, s.z, s.w};
      if (a.dkv_f32) {
        float* p = static_cast<float*>(out) + e;
        if (vec) {
          float4 x = s;
          if (a.accumulate) {
            const float4 y = *reinterpret_cast<float4*>(p);
            x = make_float4(y.x + x.x, y.y + x.y, y.z + x.z, y.w + x.w);
          }
          *reinterpret_cast<float4*>(p) = x;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) p[i] = a.accumulate ? p[i] + v[i] : v[i];
        }
      } else {
        uint16_t* p = static_cast<uint16_t*>(out) + e;
        if (vec) {
          *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) p[i] = f_to_bf16_rn(v[i]);
        }
      }
    }
  }
}

// ---- host side ----

bool map_bf16(CUtensorMap* m, const void* base, int D, int heads, int rows, int box_h, int box_r, int box_d = 64) {
  return rows_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, D, heads, rows, box_h, box_r, box_d);
}

template <int D>
cudaError_t launch_t(const TrainBwdArgs& a, void* wsp, int num_sms, cudaStream_t st) {
  constexpr int N = prod_n(D), H = D / N;
  static_assert(Sc<D>::BYTES <= 227 * 1024 && Pr<N>::BYTES <= 227 * 1024, "shared memory");
  cudaError_t e;
  static std::atomic<bool> attr_set[64];
  static std::mutex attr_mu;
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    std::lock_guard<std::mutex> lock(attr_mu);
    if (!attr_set[dev].load(std::memory_order_relaxed)) {
      e = cudaFuncSetAttribute(bwd_scores_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sc<D>::BYTES);
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(bwd_products_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Pr<N>::BYTES);
      if (e != cudaSuccess) return e;
      attr_set[dev].store(true, std::memory_order_release);
    }
  }
  const LayerArgs& L = a.L;
  const Plan p = make_plan(L, a.n_blocks, a.n_rows, a.max_block_rows, num_sms);
  if (!p.fits) return cudaErrorInvalidValue;
  const Ws w = carve(wsp, p);
  const int TQ = kT / L.G;
  // boxes of 128 (token, head) pairs or keys
  CUtensorMap q1, o1, k1, v1, q2, o2, k2, pm, dm;
  constexpr int BOX = Pr<N>::BOX;
  if (!map_bf16(&q1, a.q, D, L.n_q, a.n_rows, L.G, TQ) || !map_bf16(&o1, a.d_out, D, L.n_q, a.n_rows, L.G, TQ) ||
      !map_bf16(&k1, a.k, D, L.n_kv, a.n_rows, 1, kT) || !map_bf16(&v1, a.v, D, L.n_kv, a.n_rows, 1, kT) ||
      !map_bf16(&q2, a.q, D, L.n_q, a.n_rows, L.G, TQ, BOX) || !map_bf16(&o2, a.d_out, D, L.n_q, a.n_rows, L.G, TQ, BOX) ||
      !map_bf16(&k2, a.k, D, L.n_kv, a.n_rows, 1, kT, BOX) ||
      !runs_map(&pm, w.p, 2, kT / 8, p.cap + 1, 2, kT / 8) || !runs_map(&dm, w.ds, 2, kT / 8, p.cap + 1, 2, kT / 8))
    return cudaErrorInvalidValue;
  const int pairs = std::max(1, std::min({num_sms / 2, kMaxPairs, p.cap}));
  const int prep_blocks = 1 + (int)std::min<long long>(cdiv((long long)a.n_rows * L.n_q, kPrepThreads / 32), 8LL * num_sms);
  if ((e = launch_pdl(bwd_prep_kernel<D>, dim3(prep_blocks), dim3(kPrepThreads), 0, st, a, w,
                      PlanArgs{p.cap, p.nl, p.splits, p.piece, pairs})) !=
      cudaSuccess)
    return e;
  const long long items = cdiv(p.nkt, 2) * p.splits * L.n_kv * 2 * H + std::min<long long>((long long)p.nrt * L.n_kv, p.cap) * H;
  if (items > 0x7fffffffLL) return cudaErrorInvalidValue;
  for (int c = 0; c < p.nl; ++c) {
    if ((e = launch_pdl(bwd_scores_kernel<D>, dim3(2 * pairs), dim3(kScThreads), (size_t)Sc<D>::BYTES, st,
                        a, w, c, (int)(p.nl == 1), q1, o1, k1, v1)) != cudaSuccess)
      return e;
    if ((e = launch_pdl(bwd_products_kernel<D>, dim3(2 * (unsigned)std::min<long long>(std::max(1, num_sms / 2), items)), dim3(kPrThreads),
                        (size_t)Pr<N>::BYTES, st, a, w, ProdArgs{c, p.cap, p.direct}, q2, o2, k2, pm, dm)) != cudaSuccess)
      return e;
  }
  if (p.direct) return cudaSuccess;
  return launch_pdl(bwd_finish_kernel, dim3(std::min(p.nkt, 4 * num_sms), 32, 2), dim3(256), 0, st, a, w);
}

}  // namespace

size_t train_bwd_ws_bytes(const LayerArgs& L, int n_blocks, int n_rows, int max_block_rows) {
  return make_plan(L, n_blocks, n_rows, max_block_rows, 1).bytes;      // (the SM count sets the splits alone; 0: too large)
}

cudaError_t launch_train_bwd(const TrainBwdArgs& a, void* ws, int num_sms, cudaStream_t st) {
  switch (a.L.D) {
    case 64: return launch_t<64>(a, ws, num_sms, st);
    case 128: return launch_t<128>(a, ws, num_sms, st);
    case 256: return launch_t<256>(a, ws, num_sms, st);
    case 512: return launch_t<512>(a, ws, num_sms, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
