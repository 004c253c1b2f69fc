// attn_paged_prefill on the tensor cores (tcgen05): prompt rows over pages of
// 8-bit codes.
//
// One CTA takes MT tiles of 128 (token, q head) rows of one sequence and kv
// head (row r = token r / G, head r % G) and walks the keys they see in tiles
// of KT.  Mathematics as in kvq_paged_decode.cu: products of f16 q and codes
// are exact, the value scale goes into the probability,
//   t_j = (q . ck_j) sk log2 e + log2 sv,  p_j = 2^(t_j - ref) as f16,
//   O += p_j cv_j,  l += p_j / sv,  out = O / l,
// so codes enter both products as the exact f16 values they stand for.
//
// Roles (one barrier pair per buffer, no block barrier in the loop):
//   - converters: 16-byte loads of codes (the next tile's K or V in flight in
//     registers while this one is converted), code pairs to f16, stored to the
//     128-byte-swizzled rows of 64 dims that the MMA reads: K as a K-major
//     operand, V as an MN-major one (rows are keys in both, so one layout serves
//     both).  Positions that no row sees are stored as zeros and not read.
//   - one MMA thread: S = q K^T into a score slot of tensor memory, O += P V with
//     P from tensor memory.  MT = 2 (head_dim <= 128): the two row tiles
//     alternate, one's products run under the other's softmax.  MT = 1: two score
//     slots, the next tile's S runs under this one's softmax.
//   - softmax: MT = 2: a thread per row; MT = 1: two threads per row, each half
//     of the tile's keys, which exchange the row maximum through shared memory.
//     P (f16) overwrites the scores it comes from.  ref is renewed (and O
//     rescaled) only where a tile exceeds it by 2^8.
// MMAs of one thread execute in issue order, so S of the next tile may be
// issued right behind the P V that reads the slot it overwrites.
//
// head_dim 512: two CTAs per row tile, each 256 of the output dims (tensor
// memory holds 512 columns: 256 of O, 2 KT of scores).
//
// Row tiles are taken longest first (sorted by the prep kernel), and cut along
// the keys when there are too few of them to fill the GPU; paged_join_kernel
// joins the pieces in order.
#include <algorithm>

#include "kvq_paged.cuh"
#include "kvq_paged_rows.cuh"
#include "kvq_tc.cuh"

namespace kvq {

namespace {

template <int D>
struct Pf {
  static constexpr int MT = D <= 128 ? 2 : 1;           // row tiles per CTA
  static constexpr int DO = D > 256 ? 256 : D;          // output dims per CTA
  static constexpr int NSPLIT = D / DO;
  static constexpr int KT = D == 512 ? 64 : 128;        // keys per tile
  static constexpr int SUB = KT / 16;                   // scales per tile
  static constexpr int KST = D <= 128 ? 2 : 1;          // K and V stages
  static constexpr int NC = 224;                        // converter threads
  static constexpr int THREADS = 256 + NC + 32;         // 512: 128 registers each
  static constexpr int Q_BYTES = 128 * D * 2;           // of a row tile
  static constexpr int K_BYTES = KT * D * 2, V_BYTES = KT * DO * 2;
  static constexpr int K_OFF = MT * Q_BYTES;
  static constexpr int V_OFF = K_OFF + KST * K_BYTES;
  static constexpr int SC_OFF = V_OFF + KST * V_BYTES;  // float4 [4][SUB]: sk log2 e, log2 sv, 1 / sv
  static constexpr int X_OFF = SC_OFF + 4 * SUB * 16;   // MT == 1: row maxima [2][2][128]
  static constexpr int B_OFF = X_OFF + (MT == 1 ? 2048 : 0);
  static constexpr int USED = B_OFF + 160;
  // (one CTA per SM: each takes all of tensor memory)
  static constexpr int BYTES = USED > 120 * 1024 ? USED : 120 * 1024;
  static constexpr int KN = KT * D / 16, VN = KT * DO / 16;        // 16-byte loads of a tile
  static constexpr int KV = (KN + NC - 1) / NC, VV = (VN + NC - 1) / NC;   // per converter thread
  static constexpr int C_S = MT * DO;                   // tensor-memory columns: O, then two score slots
  static_assert(C_S + 2 * KT <= 512, "tensor memory");
  static_assert(BYTES <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ float pf_ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint4 ldg_codes(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// MN-major operand, 128-byte swizzle: lbo to the next 64 elements of N, sbo to the next 8 of K
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
constexpr uint32_t kMnMajorB = 1u << 16;                // instruction descriptor: B is MN-major

__device__ __forceinline__ void pf_ld32(uint32_t taddr, float (&v)[32]) {
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
__device__ __forceinline__ void pf_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
               "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
               :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
                  "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
               : "memory");
}

// The pieces that a unit of n key tiles is cut into, and piece z's tiles.
__device__ __forceinline__ int pf_pieces(int n, int splits) { return min(n, splits); }
__device__ __forceinline__ int pf_tile0(int n, int pieces, int z) { return (int)((long long)n * z / pieces); }

template <int D, bool E4M3>
__global__ void __launch_bounds__(Pf<D>::THREADS, 1)
paged_prefill_kernel(const PagedReadArgs a, const int TQ, const int splits, const int32_t* order, const uint16_t* q16,
                     float* part_o, float* part_ml, uint32_t* status) {
  using S = Pf<D>;
  constexpr int MT = S::MT, DO = S::DO, KT = S::KT, SUB = S::SUB, KST = S::KST, NC = S::NC;
  constexpr float L2E = 1.4426950408889634f;
  constexpr float kSlack = 8.f, kTop = 7.f;
  extern __shared__ __align__(1024) uint8_t sm[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.L.G, n_kv = a.L.n_kv, W = a.L.window, P = a.pg.P, sh = a.pg.p_shift;
  pdl_launch();
  pdl_wait();                                             // q16, the order and the status word are written
  // ---- the CTA's rows and keys ----
  const int per = n_kv * S::NSPLIT, z = blockIdx.y;
  const int rank = blockIdx.x / per, hx = blockIdx.x - rank * per;
  const int u = __ldg(order + rank), h = hx / S::NSPLIT, d_base = (hx % S::NSPLIT) * DO;
  const PagedGroup g = paged_group(a.r, a.pg, W, TQ, KT, u);
  if (g.tiles == 0) return;
  const int n_all = g.tiles;
  const int pieces = pf_pieces(n_all, splits);
  if (z >= pieces) return;
  const int t_a = pf_tile0(n_all, pieces, z), n = pf_tile0(n_all, pieces, z + 1) - t_a;
  const int k0 = g.kt0 + KT * t_a;
  const int rows = g.nt * G;

  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + S::B_OFF);
  uint64_t* k_full = bars;                                // [2] (converter warps)
  uint64_t* k_empty = bars + 2;                           // [2]
  uint64_t* v_full = bars + 4;                            // [2]
  uint64_t* v_empty = bars + 6;                           // [2]
  uint64_t* s_full = bars + 8;                            // [2] scores of a slot written
  uint64_t* p_full = bars + 10;                           // [2] P of a slot written (softmax warps)
  uint64_t* o_full = bars + 12;                           // [1]
  volatile uint32_t* ctl = reinterpret_cast<volatile uint32_t*>(bars + 14);   // tensor memory, bad page
  const uint32_t sb = smem_u32(sm);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + i, NC / 32);
      mbar_init(v_full + i, NC / 32);
      mbar_init(k_empty + i, 1);
      mbar_init(v_empty + i, 1);
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, MT == 2 ? 4 : 8);
    }
    mbar_init(o_full, 1);
    fence_mbar_init();
    ctl[1] = 0;
  }
  if (warp == 0) {
    tc::tmem_alloc(const_cast<uint32_t*>(ctl), 512);
    tc::tmem_relinquish();
  }
  // ---- q into shared memory: blocks of 64 dims [128 rows x 128 B], swizzled ----
  for (int i = tid; i < MT * 128 * (D / 8); i += S::THREADS) {
    const int r = i / (D / 8), c = i - r * (D / 8);       // row, 16-byte chunk of it
    uint4 v = {0u, 0u, 0u, 0u};
    if (r < rows) v = *reinterpret_cast<const uint4*>(q16 + ((size_t)(g.row0 + r / G) * a.L.n_q + h * G + r % G) * D + 8 * c);
    *reinterpret_cast<uint4*>(sm + (r >> 7) * S::Q_BYTES + (c >> 3) * 16384 + tc::sw128_off(r & 127, c & 7)) = v;
  }
  fence_proxy_async();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = ctl[0];
  bool dead = false;
  auto wait = [&](uint64_t* bar, int parity) {
    if (!dead && !mbar_wait(bar, parity)) {
      dead = true;
      flag_error(status, KVQ_DEV_TIMEOUT);
    }
  };

  if (warp == 8 + NC / 32) {
    // ================= products =================
    constexpr uint32_t ID_QK = tc::idesc_f16_f32(128, KT), ID_PV = tc::idesc_f16_f32(128, DO) | kMnMajorB;
    const bool leader = lane == 0;
    auto qk = [&](int m, int i) {                         // slot: MT == 2: m, else i & 1
      const int slot = MT == 2 ? m : i & 1, st = i % KST;
      if (leader) {
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
          tc::mma_f16(tmem + S::C_S + KT * slot,
                      tc::desc_kmajor_sw128(sb + m * S::Q_BYTES + (s >> 2) * 16384 + 32 * (s & 3), 1024),
                      tc::desc_kmajor_sw128(sb + S::K_OFF + st * S::K_BYTES + (s >> 2) * (KT * 128) + 32 * (s & 3), 1024),
                      ID_QK, s != 0);
        tc::commit(s_full + slot);
      }
      __syncwarp();
    };
    auto pv = [&](int m, int i) {
      const int slot = MT == 2 ? m : i & 1, st = i % KST;
      if (leader) {
#pragma unroll
        for (int s = 0; s < KT / 16; ++s) {
          const int col = MT == 2 ? 8 * s : (s / (KT / 32)) * (KT / 2) + 8 * (s % (KT / 32));
          tc::mma_f16_ts(tmem + m * DO, tmem + S::C_S + KT * slot + col,
                         desc_mn_sw128(sb + S::V_OFF + st * S::V_BYTES + 2048 * s, KT * 128, 1024), ID_PV,
                         i > 0 || s > 0);
        }
      }
      __syncwarp();
    };
    auto done = [&](uint64_t* bar) {
      if (leader) tc::commit(bar);
      __syncwarp();
    };
    wait(k_full, 0);
    tc::fence_after_sync();
    for (int m = 0; m < MT; ++m) qk(m, 0);
    done(k_empty);
    for (int i = 0; i < n; ++i) {
      const int nx = i + 1;
      if (MT == 1 && nx < n) {                            // the next scores before this P V
        wait(k_full + nx % KST, (nx / KST) & 1);
        tc::fence_after_sync();
        qk(0, nx);
        done(k_empty + nx % KST);
      }
      wait(v_full + i % KST, (i / KST) & 1);
      if (MT == 2 && nx < n) wait(k_full + nx % KST, (nx / KST) & 1);
      for (int m = 0; m < MT; ++m) {
        if (MT == 2) wait(p_full + m, i & 1);
        else wait(p_full + (i & 1), (i >> 1) & 1);
        tc::fence_after_sync();
        pv(m, i);
        if (m == MT - 1) done(v_empty + i % KST);
        if (MT == 2 && nx < n) qk(m, nx);
      }
      if (MT == 2 && nx < n) done(k_empty + nx % KST);
    }
    done(o_full);
  } else if (warp >= 8) {
    // ================= converters =================
    const int ct = tid - 256, cw = warp - 8;
    constexpr int CK = D / 16, CV = DO / 16;              // 16-byte chunks of a key
    const int32_t* table = a.pg.tables + (size_t)g.s * a.pg.max_pages;
    // lane s < SUB: the page of 16 positions s of tile t (-2: none is seen)
    auto look_up = [&](int t) {
      const int key = k0 + KT * t + 16 * lane;
      int id = -2;
      if (lane < SUB && t < n && key <= g.hi && key + 15 >= g.lo) id = __ldg(table + (key >> sh));
      return id;
    };
    auto checked = [&](int id) {
      if (id == -2) return -1;
      if ((unsigned)id < (unsigned)a.pg.n_pages) return id;
      ctl[1] = 1;
      return -1;
    };
    auto load = [&](const uint8_t* codes, int t, int pid, int key_l, int c) {   // chunk c of key key_l of tile t
      const int id = __shfl_sync(0xffffffffu, pid, key_l >> 4);
      const int key = k0 + KT * t + key_l;
      uint4 v = {0u, 0u, 0u, 0u};
      if (id >= 0 && key >= g.lo && key <= g.hi)
        v = ldg_codes(codes + ((((size_t)id * n_kv + h) << sh) + (key & (P - 1))) * D + 16 * c);
      return v;
    };
    // chunk c (16 dims) of row key_l: two swizzled 16-byte chunks of f16; odd
    // 64-dim blocks write theirs in the other order, so that the lanes of a key
    // meet all banks
    auto store = [&](uint32_t base, int key_l, int c, uint4 v) {
      uint32_t o[8];
      codes_to_h2<E4M3>(v.x, o[0], o[1]);
      codes_to_h2<E4M3>(v.y, o[2], o[3]);
      codes_to_h2<E4M3>(v.z, o[4], o[5]);
      codes_to_h2<E4M3>(v.w, o[6], o[7]);
      uint8_t* row = sm + base + (c >> 2) * (KT * 128);
      const int c0 = 2 * (c & 3), odd = (c >> 2) & 1;
      const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
      *reinterpret_cast<uint4*>(row + tc::sw128_off(key_l, c0 + odd)) = odd ? hi : lo;
      *reinterpret_cast<uint4*>(row + tc::sw128_off(key_l, c0 + 1 - odd)) = odd ? lo : hi;
    };
    uint4 ka[S::KV], va[S::VV];
    float sk = 0.f, sv = 0.f;
    auto load_k = [&](int t, int pid) {
#pragma unroll
      for (int j = 0; j < S::KV; ++j) {
        const int x = min(j * NC + ct, S::KN - 1);
        ka[j] = load(a.pg.k_codes, t, pid, x / CK, x % CK);
      }
      if (cw == 0) {                                      // lane s: the scales of its 16 positions
        sk = sv = 0.f;
        if (lane < SUB && pid >= 0) {
          sk = __ldg(a.pg.k_scales + (size_t)pid * n_kv + h);
          sv = __ldg(a.pg.v_scales + (size_t)pid * n_kv + h);
        }
      }
    };
    auto load_v = [&](int t, int pid) {
#pragma unroll
      for (int j = 0; j < S::VV; ++j) {
        const int x = min(j * NC + ct, S::VN - 1);
        va[j] = load(a.pg.v_codes, t, pid, x / CV, d_base / 16 + x % CV);
      }
    };
    auto store_k = [&](int t) {
      const int st = t % KST;
      wait(k_empty + st, ((t / KST) & 1) ^ 1);
      if (cw == 0 && lane < SUB) {
        const float one = sv > 0.f ? sv : 1.f;
        *reinterpret_cast<float4*>(sm + S::SC_OFF + ((t & 3) * SUB + lane) * 16) =
            make_float4(sk * L2E, __log2f(one), __fdividef(1.f, one), 0.f);
      }
#pragma unroll
      for (int j = 0; j < S::KV; ++j) {
        const int x = j * NC + ct;
        if (x < S::KN) store(S::K_OFF + st * S::K_BYTES, x / CK, x % CK, ka[j]);
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(k_full + st);
    };
    // K runs a tile ahead of V: K(0), K(1), V(0), K(2), V(1), .., each loaded
    // while the one before it waits or is stored
    int pid1 = checked(look_up(0)), raw = look_up(1);
    load_k(0, pid1);
    load_v(0, pid1);
    store_k(0);
    pid1 = checked(raw);
    raw = look_up(2);
    if (n > 1) load_k(1, pid1);
    for (int i = 0; i < n; ++i) {
      const int st = i % KST;
      const int pid2 = checked(raw);                      // of tile i + 2 (pid1: of i + 1)
      raw = look_up(i + 3);
      if (i + 1 < n) store_k(i + 1);
      if (i + 2 < n) load_k(i + 2, pid2);
      wait(v_empty + st, ((i / KST) & 1) ^ 1);
#pragma unroll
      for (int j = 0; j < S::VV; ++j) {
        const int x = j * NC + ct;
        if (x < S::VN) store(S::V_OFF + st * S::V_BYTES, x / CV, x % CV, va[j]);
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(v_full + st);
      if (i + 1 < n) load_v(i + 1, pid1);
      pid1 = pid2;
    }
  } else {
    // ================= softmax =================
    constexpr int NK = MT == 2 ? KT : KT / 2;             // keys of a tile per thread
    const int wg = warp >> 2;                             // row tile, or half of the keys
    const int m = MT == 2 ? wg : 0;
    const int r = 32 * (warp & 3) + lane, rg = 128 * m + r;
    const int t_r = min(rg / G, g.nt - 1);
    const int p_r = g.p0 + t_r, lo_r = W > 0 ? p_r - W + 1 : 0;
    const bool valid = rg < rows;
    // what every row of the row tile sees
    const int t_first = min(128 * m / G, g.nt - 1), t_last = min((128 * m + 127) / G, g.nt - 1);
    const int p_min = g.p0 + t_first, lo_max = W > 0 ? g.p0 + t_last - W + 1 : 0;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t t_o = lanes + m * DO;
    float ref = -INFINITY, l = 0.f;
    float* xm = reinterpret_cast<float*>(sm + S::X_OFF);
    for (int i = 0; i < n; ++i) {
      const int slot = MT == 2 ? m : i & 1;
      const uint32_t t_s = lanes + S::C_S + KT * slot + (MT == 2 ? 0 : (KT / 2) * wg);
      if (MT == 2) wait(s_full + m, i & 1);
      else wait(s_full + slot, (i >> 1) & 1);
      tc::fence_after_sync();
      __syncwarp();
      const float4* sc = reinterpret_cast<const float4*>(sm + S::SC_OFF) + (i & 3) * SUB + (MT == 2 ? 0 : (SUB / 2) * wg);
      const int key0 = k0 + KT * i + (MT == 2 ? 0 : (KT / 2) * wg);
      const bool whole = key0 >= lo_max && key0 + NK - 1 <= p_min;
      // ---- the tile's largest t ----
      float top = -INFINITY;
#pragma unroll
      for (int c = 0; c < NK / 32; ++c) {
        float v[32];
        pf_ld32(t_s + 32 * c, v);
        tc::wait_ld();
        if (!whole) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int key = key0 + 32 * c + e;
            v[e] = key <= p_r && key >= lo_r ? v[e] : -INFINITY;
          }
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float x = v[16 * b];
#pragma unroll
          for (int e = 1; e < 16; ++e) x = fmaxf(x, v[16 * b + e]);
          const float4 f = sc[2 * c + b];
          // (a masked subtile of scale 0 would read -inf * 0)
          top = fmaxf(top, x == -INFINITY ? x : fmaf(x, f.x, f.y));
        }
      }
      if constexpr (MT == 1) {                            // the other half's
        xm[((i & 1) * 2 + wg) * 128 + r] = top;
        named_bar(1, 256);
        top = fmaxf(top, xm[((i & 1) * 2 + (wg ^ 1)) * 128 + r]);
      }
      const bool renew = top > ref + kSlack || (ref == -INFINITY && top > -INFINITY);
      const bool again = renew && ref != -INFINITY;
      const float alpha = again ? pf_ex2(ref - top) : 1.f;
      if (renew) {
        ref = top;
        l *= alpha;
      }
      if (__any_sync(0xffffffffu, again)) {
        // O is settled: MT == 2: S of this tile came after the last P V; MT == 1: wait for it
        if (MT == 1) {
          wait(v_empty + (i - 1) % KST, ((i - 1) / KST) & 1);
          tc::fence_after_sync();
          __syncwarp();
        }
        constexpr int OC = MT == 2 ? DO : DO / 2;
#pragma unroll 1
        for (int c = 0; c < OC / 16; ++c) {
          const uint32_t at = t_o + (MT == 2 ? 0 : OC * wg) + 16 * c;
          float v[16];
          tc::ld_x16(at, v);
          tc::wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] *= alpha;
          tc::st_x16(at, v);
        }
      }
      // ---- P ----
      const float base = ref == -INFINITY ? 0.f : ref - kTop;
#pragma unroll
      for (int c = 0; c < NK / 32; ++c) {
        float v[32];
        pf_ld32(t_s + 32 * c, v);
        tc::wait_ld();
        if (!whole) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int key = key0 + 32 * c + e;
            v[e] = key <= p_r && key >= lo_r ? v[e] : -INFINITY;
          }
        }
        uint32_t pw[16];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const float4 f = sc[2 * c + b];
          const float off = f.y - base;
          float s0 = 0.f, s1 = 0.f;
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            float x0 = fmaf(v[16 * b + e], f.x, off), x1 = fmaf(v[16 * b + e + 1], f.x, off);
            if (!whole) {                                 // (-inf * 0)
              x0 = v[16 * b + e] == -INFINITY ? -INFINITY : x0;
              x1 = v[16 * b + e + 1] == -INFINITY ? -INFINITY : x1;
            }
            const float p0 = pf_ex2(x0), p1 = pf_ex2(x1);
            s0 += p0;
            s1 += p1;
            pw[8 * b + e / 2] = pack_h2(p0, p1);
          }
          l = fmaf(s0 + s1, f.z, l);
        }
        pf_st16(t_s + 16 * c, pw);
      }
      tc::wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full + slot);
    }
    // ---- out ----
    if constexpr (MT == 1) {                              // l of both halves
      named_bar(1, 256);                                  // the last maxima are read
      xm[wg * 128 + r] = l;
      named_bar(1, 256);
      l += xm[(wg ^ 1) * 128 + r];
    }
    wait(o_full, 0);
    tc::fence_after_sync();
    __syncwarp();
    if (ctl[1]) {
      l = __int_as_float(0x7FC00000);
      if (tid == 0) flag_error(status, KVQ_DEV_BADSEQ);
    }
    const float inv = 1.f / l;
    constexpr int OC = MT == 2 ? DO : DO / 2;
    const int o0 = MT == 2 ? 0 : OC * wg;
    const size_t unit = (size_t)u * per + hx;
    const size_t prow = (unit * splits + z) * (MT * 128) + rg;
    const size_t at = ((size_t)(g.row0 + rg / G) * a.L.n_q + h * G + rg % G) * D + d_base + o0;
    const bool vec = (reinterpret_cast<uintptr_t>(a.out) & 15u) == 0;
#pragma unroll 1
    for (int c = 0; c < OC / 16; ++c) {
      float v[16];
      tc::ld_x16(t_o + o0 + 16 * c, v);
      tc::wait_ld();
      if (!valid) continue;
      if (pieces > 1) {
        float4* d = reinterpret_cast<float4*>(part_o + prow * DO + o0 + 16 * c);
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        continue;
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] *= inv;
      if (a.out_f32) {
        float* d = reinterpret_cast<float*>(a.out) + at + 16 * c;
        if (vec) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            reinterpret_cast<float4*>(d)[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) d[e] = v[e];
        }
      } else {
        uint16_t* d = reinterpret_cast<uint16_t*>(a.out) + at + 16 * c;
        if (vec) {
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            w[e] = (uint32_t)f_to_bf16_rn(v[2 * e]) | ((uint32_t)f_to_bf16_rn(v[2 * e + 1]) << 16);
          reinterpret_cast<uint4*>(d)[0] = make_uint4(w[0], w[1], w[2], w[3]);
          reinterpret_cast<uint4*>(d)[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) d[e] = f_to_bf16_rn(v[e]);
        }
      }
    }
    if (pieces > 1 && valid && (MT == 2 || wg == 0)) {
      part_ml[prow * 2] = ref;
      part_ml[prow * 2 + 1] = l;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// The units that were cut along the keys: each thread four dims of one row
// over its pieces, in order.
template <int D>
__global__ void __launch_bounds__(256)
paged_join_kernel(const PagedReadArgs a, const int TQ, const int splits, const float* part_o, const float* part_ml) {
  using S = Pf<D>;
  constexpr int DO = S::DO, ROWS = S::MT * 128;
  pdl_launch();
  pdl_wait();
  const int per = a.L.n_kv * S::NSPLIT, G = a.L.G;
  const int u = blockIdx.x / per, hx = blockIdx.x - u * per;
  const PagedGroup g = paged_group(a.r, a.pg, a.L.window, TQ, S::KT, u);
  if (g.tiles == 0) return;
  const int pieces = pf_pieces(g.tiles, splits);
  if (pieces == 1) return;
  const int i = blockIdx.y * 256 + threadIdx.x;
  const int r = i / (DO / 4), d = (i - r * (DO / 4)) * 4;
  if (r >= g.nt * G) return;
  const size_t row0 = ((size_t)blockIdx.x * splits) * ROWS + r;
  float M = -INFINITY;
  for (int z = 0; z < pieces; ++z) M = fmaxf(M, __ldg(part_ml + (row0 + (size_t)z * ROWS) * 2));
  float l = 0.f;
  float4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int z = 0; z < pieces; ++z) {
    const size_t row = row0 + (size_t)z * ROWS;
    const float mz = __ldg(part_ml + row * 2), lz = __ldg(part_ml + row * 2 + 1);
    const float4 v = __ldg(reinterpret_cast<const float4*>(part_o + row * DO + d));
    const float f = mz == -INFINITY ? 0.f : pf_ex2(mz - M);
    l = fmaf(lz, f, l);
    o.x = fmaf(v.x, f, o.x);
    o.y = fmaf(v.y, f, o.y);
    o.z = fmaf(v.z, f, o.z);
    o.w = fmaf(v.w, f, o.w);
  }
  const float inv = 1.f / l;
  const int h = hx / S::NSPLIT;
  const size_t at = ((size_t)(g.row0 + r / G) * a.L.n_q + h * G + r % G) * D + (hx % S::NSPLIT) * DO + d;
  const float w[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (a.out_f32) reinterpret_cast<float*>(a.out)[at + e] = w[e];
    else reinterpret_cast<uint16_t*>(a.out)[at + e] = f_to_bf16_rn(w[e]);
  }
}

struct PfPlan { int TQ, n_groups, splits; long long units; };
template <int D>
PfPlan pf_plan(const LayerArgs& L, int n_seqs, int n_rows, int max_pos, int num_sms) {
  using S = Pf<D>;
  PfPlan p;
  p.TQ = S::MT * 128 / L.G;
  static const int32_t some = 0;
  p.n_groups = paged_groups(PagedRows{&some, nullptr, n_seqs, n_rows}, p.TQ);
  p.units = (long long)p.n_groups * L.n_kv * S::NSPLIT;
  // as many pieces as fill the GPU once (one CTA per SM), of at least two tiles
  long long keys = (long long)max_pos + 1;
  if (L.window > 0) keys = std::min<long long>(keys, (long long)L.window + p.TQ);
  const long long tiles = (keys + S::KT - 1) / S::KT;
  // (groups are counted with room for one short one per sequence)
  const long long real = std::max(1ll, ((long long)n_rows / p.TQ + (n_rows % p.TQ != 0)) * L.n_kv * S::NSPLIT);
  p.splits = (int)std::max(1ll, std::min<long long>({num_sms / real, tiles / 2, 64ll}));
  return p;
}

// status (256 B), q16, order, part_o, part_ml
struct PfWs { size_t q16, order, part_o, part_ml, total; };
template <int D>
PfWs pf_ws(const LayerArgs& L, int n_rows, const PfPlan& p) {
  using S = Pf<D>;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t prows = p.splits > 1 ? (size_t)p.units * p.splits * S::MT * 128 : 0;
  PfWs w;
  w.q16 = 256;
  w.order = up(w.q16 + (size_t)n_rows * L.n_q * D * 2);
  w.part_o = up(w.order + (size_t)p.n_groups * 4);
  w.part_ml = up(w.part_o + prows * S::DO * 4);
  w.total = up(w.part_ml + prows * 8);
  return w;
}

template <int D, bool E4M3>
cudaError_t launch_t(const PagedReadArgs& a, const RopeFreqs& f, int max_pos, void* ws, int num_sms, cudaStream_t st) {
  using S = Pf<D>;
  const PfPlan p = pf_plan<D>(a.L, a.r.n_seqs, a.r.n_rows, max_pos, num_sms);
  const PfWs w = pf_ws<D>(a.L, a.r.n_rows, p);
  if (p.units > 0x7fffffffLL) return cudaErrorInvalidValue;
  uint8_t* b = static_cast<uint8_t*>(ws);
  uint32_t* status = reinterpret_cast<uint32_t*>(b);
  uint16_t* q16 = reinterpret_cast<uint16_t*>(b + w.q16);
  int32_t* order = reinterpret_cast<int32_t*>(b + w.order);
  float* part_o = reinterpret_cast<float*>(b + w.part_o);
  float* part_ml = reinterpret_cast<float*>(b + w.part_ml);
  cudaError_t e = launch_paged_prep<D>(a, f, p.TQ, S::KT, p.n_groups, q16, nullptr, order, status, num_sms, st);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(paged_prefill_kernel<D, E4M3>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::BYTES);
  if (e != cudaSuccess) return e;
  if ((e = prof_before(st)) != cudaSuccess) return e;
  e = launch_pdl(paged_prefill_kernel<D, E4M3>, dim3((unsigned)p.units, p.splits), dim3(S::THREADS), S::BYTES, st, a,
                 p.TQ, p.splits, order, q16, part_o, part_ml, status);
  if (e != cudaSuccess) return e;
  if ((e = prof_after(st)) != cudaSuccess || p.splits == 1) return e;
  return launch_pdl(paged_join_kernel<D>, dim3((unsigned)p.units, S::MT * 128 * (S::DO / 4) / 256), dim3(256), 0, st, a,
                    p.TQ, p.splits, part_o, part_ml);
}

template <int D>
cudaError_t launch_d(const PagedReadArgs& a, const RopeFreqs& f, int max_pos, void* ws, int num_sms, cudaStream_t st) {
  return a.pg.e4m3 ? launch_t<D, true>(a, f, max_pos, ws, num_sms, st)
                   : launch_t<D, false>(a, f, max_pos, ws, num_sms, st);
}

}  // namespace

bool paged_prefill_supported(const LayerArgs& L, int max_rows_per_seq) {
  return 128 % L.G == 0 && max_rows_per_seq * L.G > 32;
}

size_t paged_prefill_ws_bytes(const LayerArgs& L, int n_seqs, int n_rows, int max_pos, int num_sms) {
  switch (L.D) {
    case 64: return pf_ws<64>(L, n_rows, pf_plan<64>(L, n_seqs, n_rows, max_pos, num_sms)).total;
    case 128: return pf_ws<128>(L, n_rows, pf_plan<128>(L, n_seqs, n_rows, max_pos, num_sms)).total;
    case 256: return pf_ws<256>(L, n_rows, pf_plan<256>(L, n_seqs, n_rows, max_pos, num_sms)).total;
    default: return pf_ws<512>(L, n_rows, pf_plan<512>(L, n_seqs, n_rows, max_pos, num_sms)).total;
  }
}

cudaError_t launch_paged_prefill(const PagedReadArgs& a, const RopeFreqs& f, int max_pos, void* ws, int num_sms,
                                 cudaStream_t st) {
  switch (a.L.D) {
    case 64: return launch_d<64>(a, f, max_pos, ws, num_sms, st);
    case 128: return launch_d<128>(a, f, max_pos, ws, num_sms, st);
    case 256: return launch_d<256>(a, f, max_pos, ws, num_sms, st);
    default: return launch_d<512>(a, f, max_pos, ws, num_sms, st);
  }
}

}  // namespace kvq
