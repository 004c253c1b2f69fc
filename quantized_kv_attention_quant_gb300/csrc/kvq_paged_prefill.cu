// attn_paged_prefill on the tensor cores (tcgen05): prompt rows over pages of
// 8-bit codes.
//
// A pair of CTAs (a cluster of two, cta_group::2 MMAs) takes 2 MT tiles of 128
// (token, q head) rows of one sequence and kv head (row r = token r / G, head r %
// G), CTA c the rows 128 MT c .., and walks the keys they see in tiles of KT.
// Mathematics as in kvq_paged_decode.cu: products of f16 q and codes are exact,
// the value scale goes into the probability,
//   t_j = (q . ck_j) sk log2 e + log2 sv,  p_j = 2^(t_j - ref) as f16,
//   O += p_j cv_j,  l += p_j / sv,  out = O / l
// (sv = 0: kZeroScale in t and l, the codes as zeros; keys whose page is not
// named: scores of 0 at sk = infinity, NaN for the rows that see them and -inf for
// the others), so codes enter both products as the exact f16 values they stand for.  An MMA
// of the pair reads half of its B operand from each CTA's shared memory: CTA c
// converts the keys KT / 2 c .. of K and the output dims DO / 2 c .. of V, so the
// codes are converted once for twice the rows (a CTA for itself spent as long
// on the conversion as on everything else).
//
// Roles (one barrier pair per buffer, no block barrier in the loop):
//   - four converter warps: 16-byte loads of codes, a tile ahead in registers, code
//     pairs to f16, stored to the swizzled rows that the MMA reads: K as a K-major
//     operand, V as an MN-major one (rows are keys in both).  A warp's keys lie 16
//     by 16 in one page.  Eight lanes take four chunks of two neighbouring rows,
//     whose swizzles meet all banks.  Positions that no row sees are stored as
//     zeros and not read.  K runs a tile ahead of V.
//   - one MMA warp of CTA 0, for both: S = q K^T into a score slot of tensor memory,
//     O += P V with P from tensor memory.
//   - eight softmax warps.  MT = 2 (head_dim <= 128): a thread per row, four warps
//     per row tile; the two row tiles take turns on the tensor cores, one's products
//     under the other's softmax, and P V begins with the first half of the keys while
//     the second is formed.  MT = 1: two threads per row, each half of the
//     tile's keys, which exchange the row maximum through shared memory; two score
//     slots, the next tile's S runs under this one's softmax.  P (f16) overwrites
//     the scores it comes from.  ref is renewed (and O rescaled) only where a tile
//     exceeds it by 2^8.
// MMAs of one thread execute in issue order, so S of the next tile may be
// issued right behind the P V that reads the slot it overwrites.
//
// head_dim 512: two pairs per row tile, each 256 of the output dims (tensor
// memory holds 512 columns: 256 of O, 2 KT of scores).
//
// Row tiles are taken longest first (sorted by the prep kernel), and cut along
// the keys when there are too few of them to fill the GPU; paged_join_kernel
// joins the pieces in order.
//
// Measured (8 q heads a pair of CTAs, GB300): 6374 packed rows of 32 q heads on 8
// kv heads, D 128, 161 GFLOP: this kernel 172 us alone (0.48 of the measured bf16
// rate), its prep 45; 500 rows behind 16300 keys, 8 q heads on 2, D 256, 68 GFLOP:
// 67 us (0.52), join 7.  What bounds it: at D <= 128 the chain of a row tile (scores
// loaded 110, maxima 670, P 1200, its products and the next scores some 1000 of
// about 4200 cycles; the tensor cores take 2048 of them for both row tiles), and a
// CTA's ends, some 9 us of its 40: q and the first keys 4, the first scores 1, the
// results 2, the next CTA's start 2.  Left out, as measured (us, the first case):
// P through shared memory, which frees the score slot at once (226 against 226,
// 78.5 against 75.2 at D 256, which has two slots anyway); one MMA warp per row
// tile (the two fall into step); a CTA for itself instead of a pair (276 / 103).
#include <algorithm>
#include <atomic>

#include "kvq_paged.cuh"
#include "kvq_paged_rows.cuh"
#include "kvq_tc.cuh"

namespace kvq {

namespace {

template <int D>
struct Pf {
  static constexpr int MT = D <= 128 ? 2 : 1;           // row tiles per CTA
  static constexpr int ROWS = 2 * MT * 128;             // rows of a pair
  static constexpr int DO = D > 256 ? 256 : D;          // output dims per pair
  static constexpr int NSPLIT = D / DO;
  static constexpr int KT = D == 512 ? 64 : 128;        // keys per tile
  static constexpr int SUB = KT / 16;                   // scales per tile
  static constexpr int KST = D <= 128 ? 3 : 2;          // K and V stages
  static constexpr int THREADS = 512;                   // 8 softmax, 4 converter, 1 MMA warp (and 3 to fill a warpgroup)
  // a converter warp per tile: 16 keys x KD dims of K, VU times 16 keys x VD dims of V
  static constexpr int KHALVES = 8 / SUB;               // warps that share 16 keys of K (halves of the dims)
  static constexpr int KD = D / KHALVES, KJ = KD / 32;  // KJ 16-byte loads per lane
  static constexpr int VU = SUB / 4, VD = DO / 2, VJ = VD / 32;
  static constexpr int Q_BYTES = 128 * D * 2;           // of a row tile
  static constexpr int K_BYTES = KT / 2 * D * 2, V_BYTES = KT * VD * 2;    // of a CTA's half tile
  static constexpr int K_BLK = KT / 2 * 128;            // 64 dims of K
  static constexpr int V_ROW = VD < 64 ? VD * 2 : 128;  // bytes of a key in a block of V
  static constexpr int V_BLK = KT * V_ROW;
  static constexpr int K_OFF = MT * Q_BYTES;
  static constexpr int V_OFF = K_OFF + KST * K_BYTES;
  static constexpr int SC_OFF = V_OFF + KST * V_BYTES;  // float4 [4][SUB]: sk log2 e, log2 sv, 1 / sv
  static constexpr int X_OFF = SC_OFF + 4 * SUB * 16;   // MT == 1: row maxima [2][2][128]
  static constexpr int B_OFF = X_OFF + (MT == 1 ? 2048 : 0);
  static constexpr int USED = B_OFF + 200;
  // (one CTA per SM: each takes all of tensor memory)
  static constexpr int BYTES = USED > 120 * 1024 ? USED : 120 * 1024;
  static constexpr int C_S = MT * DO;                   // tensor-memory columns: O, then two score slots
  static_assert(C_S + 2 * KT <= 512, "tensor memory");
  static_assert(BYTES <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ float pf_ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// pairs of floats in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)),
        "l"(*reinterpret_cast<uint64_t*>(&c)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(r) : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint4 ldg_codes(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// MN-major operand, rows of 128 or 64 swizzled bytes: lbo to the next row's worth of N, sbo to the next 8 of K
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t lbo, uint32_t sbo, int row) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)(row == 128 ? 2 : 4) << 61);
}
// D (+)= A[tmem of both CTAs] * B[half of N in each CTA's smem]
__device__ __forceinline__ void mma2_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            bool accumulate) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
               :: "r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u) : "memory");
}
// An arrival at CTA 0's barrier after this CTA's shared memory was written and
// fenced for the tensor cores, which read it where it is: a release within the
// CTA (one over the cluster took 1000 cycles).
__device__ __forceinline__ void arrive_pair(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(tc::in_cta0(bar)) : "memory");
}
// One thread of the warp, always the same, known to the compiler as one: the
// operands of what it issues stay in uniform registers (27 cycles an MMA; 65, more
// than the MMA takes, under a test of the lane number).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
constexpr uint32_t kMnMajorB = 1u << 16;                // instruction descriptor: B is MN-major

__device__ __forceinline__ void pf_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
               "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
               "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                 "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                 "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
                 "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
                 "=r"(r[30]), "=r"(r[31])
               : "r"(taddr));
}
// the loads of r are complete (its uses stay behind the wait)
__device__ __forceinline__ void pf_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}
__device__ __forceinline__ void pf_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
               "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
               :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
                  "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
               : "memory");
}

// The first tile of piece z of a unit of n key tiles.
__device__ __forceinline__ int pf_tile0(int n, int pieces, int z) { return (int)((long long)n * z / pieces); }

template <int D, bool E4M3>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Pf<D>::THREADS, 1)
paged_prefill_kernel(const PagedReadArgs a, const int TQ, const int4* order, const uint16_t* q16, float* part_o,
                     float* part_ml, uint32_t* status) {
  using S = Pf<D>;
  constexpr int MT = S::MT, DO = S::DO, KT = S::KT, SUB = S::SUB, KST = S::KST;
  constexpr float L2E = 1.4426950408889634f;
  constexpr float kSlack = 8.f, kTop = 7.f;
  extern __shared__ __align__(1024) uint8_t sm[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.L.G, n_kv = a.L.n_kv, W = a.L.window, P = a.pg.P, sh = a.pg.p_shift;
  pdl_launch();
  pdl_wait();                                             // q16, the order and the status word are written
  // ---- the CTA's rows and keys ----
  const int per = n_kv * S::NSPLIT, z = blockIdx.y;
  const int cta = (int)tc::cta_rank();                    // of the pair
  const int rank = (blockIdx.x >> 1) / per, hx = (blockIdx.x >> 1) - rank * per;
  const int4 us = __ldg(order + rank);
  const int u = us.x, h = hx / S::NSPLIT, d_base = (hx % S::NSPLIT) * DO;
  const PagedGroup g = paged_group_of(a.r, a.pg, W, TQ, KT, u, us.y);
  if (g.tiles == 0) return;
  const int n_all = g.tiles;
  const int pieces = us.w;
  if (z >= pieces) return;
  const int t_a = pf_tile0(n_all, pieces, z), n = pf_tile0(n_all, pieces, z + 1) - t_a;
  const int k0 = g.kt0 + KT * t_a;
  const int rows = g.nt * G, row0 = cta * MT * 128;       // of the pair; the CTA's first

  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + S::B_OFF);
  // in CTA 0: K, V converted and P written in both CTAs; in each CTA: the rest
  uint64_t* k_full = bars;                                // [3] (converter warps of both)
  uint64_t* v_full = bars + 3;                            // [3]
  uint64_t* p_full = bars + 6;                            // [2] (softmax warps of both)
  uint64_t* k_empty = bars + 8;                           // [3] (the MMA warp)
  uint64_t* v_empty = bars + 11;                          // [3]
  uint64_t* s_full = bars + 14;                           // [2] scores of a slot written
  uint64_t* o_full = bars + 16;                           // [2] a row tile's last product
  uint64_t* sc_full = bars + 18;                          // [4] a tile's scales (the CTA's converter warps)
  uint64_t* p_half = bars + 22;                           // [2] as p_full, MT == 2: the first half of the keys
  volatile uint32_t* ctl = reinterpret_cast<volatile uint32_t*>(bars + 24);   // tensor memory
  const uint32_t sb = smem_u32(sm);
  if (tid == 0) {
    for (int i = 0; i < 3; ++i) {
      mbar_init(k_full + i, 8);
      mbar_init(v_full + i, 8);
      mbar_init(k_empty + i, 1);
      mbar_init(v_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(p_full + i, MT == 2 ? 8 : 16);
      mbar_init(p_half + i, 8);
      mbar_init(s_full + i, 1);
      mbar_init(o_full + i, 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(sc_full + i, 4);
    fence_mbar_init();
  }
  if (warp == 0) {
    tc::tmem_alloc2(const_cast<uint32_t*>(ctl), 512);
    tc::tmem_relinquish2();
  }
  // ---- q into shared memory: blocks of 64 dims [128 rows x 128 B], swizzled; the converter warps fetch their
  // first codes meanwhile ----
  constexpr int QT = S::THREADS - 128, QN = MT * 128 * (D / 8), QB = 11;   // (QB loads in flight)
  if (warp < 8 || warp >= 12) {
    const int g_shift = __ffs(G) - 1;                     // (G divides 128)
    for (int i0 = warp < 8 ? tid : tid - 128; i0 < QN; i0 += QB * QT) {
      uint4 v[QB];
#pragma unroll
      for (int k = 0; k < QB; ++k) {
        const int i = i0 + k * QT, r = i / (D / 8), c = i - r * (D / 8), rg = row0 + r;   // row, 16-byte chunk of it
        v[k] = make_uint4(0u, 0u, 0u, 0u);
        if (i < QN && rg < rows)
          v[k] = __ldg(reinterpret_cast<const uint4*>(
              q16 + ((size_t)(g.row0 + (rg >> g_shift)) * a.L.n_q + h * G + (rg & (G - 1))) * D + 8 * c));
      }
#pragma unroll
      for (int k = 0; k < QB; ++k) {
        const int i = i0 + k * QT, r = i / (D / 8), c = i - r * (D / 8);
        if (i < QN)
          *reinterpret_cast<uint4*>(sm + (r >> 7) * S::Q_BYTES + (c >> 3) * 16384 + tc::sw128_off(r & 127, c & 7)) = v[k];
      }
    }
  }
  auto meet = [&]() {                                     // barriers, tensor memory and q of both CTAs
    fence_proxy_async();
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync();
    tc::fence_after_sync();
    return ctl[0];
  };
  bool dead = false;
  auto wait = [&](uint64_t* bar, int parity) {
    if (!dead && !mbar_wait(bar, parity)) {
      dead = true;
      flag_error(status, KVQ_DEV_TIMEOUT);
    }
  };

  // MT == 2: a row of 128 scores stays in registers: 168 for the softmax threads,
  // 88 for the others (256 threads each of the launch's 512 x 128)
  if (warp >= 8) {
    if constexpr (MT == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp >= 12) {
      const uint32_t tmem = __shfl_sync(0xffffffffu, meet(), 0);
      // ================= products of both CTAs (CTA 0) =================
      if (cta == 0 && warp == 12) {
        constexpr uint32_t ID_QK = tc::idesc_f16_f32(256, KT), ID_PV = tc::idesc_f16_f32(256, DO) | kMnMajorB;
        // descriptors of the first steps; an address step of b bytes adds b / 16
        const uint64_t q_desc = tc::desc_kmajor_sw128(sb, 1024), k_desc = tc::desc_kmajor_sw128(sb + S::K_OFF, 1024),
                       v_desc = desc_mn(sb + S::V_OFF, S::V_BLK, 8 * S::V_ROW, S::V_ROW);
        auto qk = [&](int m, int i) {                     // scores of tile i
          const int slot = MT == 2 ? m : i & 1, st = i % KST;
          if (elect_one()) {
            const uint64_t qd = q_desc + m * (S::Q_BYTES / 16), kd = k_desc + st * (S::K_BYTES / 16);
            const uint32_t d = tmem + S::C_S + KT * slot;
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
              tc::mma2_f16(d, qd + (s >> 2) * 1024 + 2 * (s & 3), kd + (s >> 2) * (S::K_BLK / 16) + 2 * (s & 3), ID_QK,
                           s != 0);
            tc::commit2(s_full + slot);
            if (m == MT - 1) tc::commit2(k_empty + st);
          }
          __syncwarp();
        };
        auto pv = [&](int m, int i) {                     // O += P V of tile i
          const int slot = MT == 2 ? m : i & 1, st = i % KST;
          const uint64_t vd = v_desc + st * (S::V_BYTES / 16);
          const uint32_t p = tmem + S::C_S + KT * slot, d = tmem + m * DO;
          if constexpr (MT == 2) {
            wait(p_half + m, i & 1);
            tc::fence_after_sync();
            if (elect_one()) {
#pragma unroll
              for (int s = 0; s < KT / 32; ++s) mma2_f16_ts(d, p + 8 * s, vd + s * S::V_ROW, ID_PV, i > 0 || s > 0);
            }
            __syncwarp();
          }
          wait(p_full + slot, MT == 2 ? i & 1 : (i >> 1) & 1);
          tc::fence_after_sync();
          if (elect_one()) {
#pragma unroll
            for (int s = MT == 2 ? KT / 32 : 0; s < KT / 16; ++s) {
              const int col = MT == 2 ? 8 * s : (s / (KT / 32)) * (KT / 2) + 8 * (s % (KT / 32));
              mma2_f16_ts(d, p + col, vd + s * S::V_ROW, ID_PV, i > 0 || s > 0);
            }
            if (m == MT - 1) tc::commit2(v_empty + st);
            if (i == n - 1) tc::commit2(o_full + m);
          }
          __syncwarp();
        };
        const int n_u = __shfl_sync(0xffffffffu, n, 0);
        wait(k_full, 0);
        tc::fence_after_sync();
        for (int m = 0; m < MT; ++m) qk(m, 0);
        for (int i = 0; i < n_u; ++i) {
          const int nx = i + 1;
          // MT == 1: the next scores under this tile's softmax; MT == 2: each row tile's right behind its P V, in
          // turn, so that one row tile's products run under the other's softmax
          if (MT == 1 && nx < n_u) {
            wait(k_full + nx % KST, (nx / KST) & 1);
            tc::fence_after_sync();
            qk(0, nx);
          }
          wait(v_full + i % KST, (i / KST) & 1);
          if (MT == 2 && nx < n_u) wait(k_full + nx % KST, (nx / KST) & 1);
          for (int m = 0; m < MT; ++m) {
            pv(m, i);
            if (MT == 2 && nx < n_u) qk(m, nx);
          }
        }
      }
    } else {
      // ================= converters =================
      constexpr int KJ = S::KJ, VJ = S::VJ, VU = S::VU, NKW = SUB / 2;   // K's 16-key runs of this CTA
      const int cw = warp - 8;
      // the warp's 16 keys of K (16-key run cta * NKW + cw % NKW of a tile, half cw / NKW of the dims) and its
      // runs cw, cw + 4 .. of V; with VU == 2 the K run is one of them
      const int run_k = cta * NKW + cw % NKW, half = cw / NKW;
      const int32_t* table = a.pg.tables + (size_t)g.s * a.pg.max_pages;
      const size_t page_bytes = ((size_t)n_kv << sh) * D;
      // the lane's first row and 16-dim chunk of 64 dims; load j: row + 8 (j / blocks), block j % blocks
      // (32 dims of V: one chunk of one row)
      const int r0 = 2 * (lane >> 3) + ((lane >> 2) & 1), c0 = lane & 3;
      const uint32_t s_lane = tc::sw128_off(r0, 2 * c0);
      const int rv = S::VD < 64 ? lane >> 1 : r0, cv = S::VD < 64 ? lane & 1 : c0;
      const uint32_t v_at = S::VD < 64 ? rv * 64 + ((2 * cv ^ ((rv >> 1) & 3)) << 4) : s_lane;
      const uint8_t* k_lane = a.pg.k_codes + ((size_t)h << sh) * D + r0 * D + 16 * c0 + half * S::KD;
      const uint8_t* v_lane = a.pg.v_codes + ((size_t)h << sh) * D + rv * D + 16 * cv + d_base + cta * S::VD;
      auto seen = [&](int t, int run) {
        const int key = k0 + KT * t + 16 * run;
        return t < n && key <= g.hi && key + 15 >= g.lo;
      };
      auto look_up = [&](int t, int run) {
        return seen(t, run) ? __ldg(table + ((k0 + KT * t + 16 * run) >> sh)) : -1;
      };
      bool bad = false;
      // the page of a looked-up entry of tile t (which may hold any number), -1 where no row sees the keys, kNoPage
      // where the entry names none
      auto checked = [&](int t, int run, int id) {
        if (!seen(t, run)) return -1;
        if ((unsigned)id < (unsigned)a.pg.n_pages) return id;
        bad = true;
        return kNoPage;
      };
      // J loads of run `run` of tile t, rows r + 8 (j / nb)
      auto load = [&](auto& v, const uint8_t* codes, int nb, int r, int t, int run, int id) {
        constexpr int J = sizeof(v) / 16;
        const int key = k0 + KT * t + 16 * run;
        const uint8_t* src = codes + max(id, 0) * page_bytes + (key & (P - 1)) * D;
        if (id >= 0 && key >= g.lo && key + 15 <= g.hi) {
#pragma unroll
          for (int j = 0; j < J; ++j) v[j] = ldg_codes(src + 8 * (j / nb) * D + 64 * (j % nb));
        } else {
#pragma unroll
          for (int j = 0; j < J; ++j) {
            const int k = key + r + 8 * (j / nb);
            v[j] = make_uint4(0u, 0u, 0u, 0u);
            if (id >= 0 && k >= g.lo && k <= g.hi) v[j] = ldg_codes(src + 8 * (j / nb) * D + 64 * (j % nb));
          }
        }
      };
      auto put = [&](const auto& v, uint32_t at, uint32_t at1, int nb, uint32_t blk) {
        constexpr int J = sizeof(v) / 16;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          uint32_t o[8];
          codes_to_h2<E4M3>(v[j].x, o[0], o[1]);
          codes_to_h2<E4M3>(v[j].y, o[2], o[3]);
          codes_to_h2<E4M3>(v[j].z, o[4], o[5]);
          codes_to_h2<E4M3>(v[j].w, o[6], o[7]);
          const uint32_t d = 1024 * (j / nb) + blk * (j % nb);
          *reinterpret_cast<uint4*>(sm + at + d) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(sm + at1 + d) = make_uint4(o[4], o[5], o[6], o[7]);
        }
      };
      auto full = [&](uint64_t* bar) {                    // (in CTA 0)
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) arrive_pair(bar);
      };
      uint4 kb[KJ], vb[VU][VJ];
      float sk[VU], sv[VU];
      auto load_k = [&](int t, const int (&id)[VU], int idk) {
        load(kb, k_lane, S::KD / 64, r0, t, run_k, idk);
#pragma unroll
        for (int e = 0; e < VU; ++e) {
          sk[e] = id[e] == kNoPage ? INFINITY : 0.f;
          if (id[e] >= 0) sk[e] = __ldg(a.pg.k_scales + (size_t)id[e] * n_kv + h);
          sv[e] = id[e] >= 0 ? __ldg(a.pg.v_scales + (size_t)id[e] * n_kv + h) : 0.f;
        }
      };
      auto load_v = [&](int t, const int (&id)[VU]) {
#pragma unroll
        for (int e = 0; e < VU; ++e) load(vb[e], v_lane, S::VD < 64 ? 1 : S::VD / 64, rv, t, cw + 4 * e, id[e]);
      };
      auto put_k = [&](int t) {
        const int st = t % KST;
        wait(k_empty + st, ((t / KST) & 1) ^ 1);
        if (lane == 0) {
#pragma unroll
          for (int e = 0; e < VU; ++e) {
            const float s = sv[e] > 0.f ? sv[e] : kZeroScale;
            *reinterpret_cast<float4*>(sm + S::SC_OFF + ((t & 3) * SUB + cw + 4 * e) * 16) =
                make_float4(fmaxf(sk[e] * L2E, 1e-30f), __log2f(s), __fdividef(1.f, s), 0.f);
          }
          mbar_arrive(sc_full + (t & 3));
        }
        const uint32_t at = S::K_OFF + st * S::K_BYTES + half * (S::KD / 64) * S::K_BLK + (cw % NKW) * 2048;
        put(kb, at + s_lane, at + (s_lane ^ 16u), S::KD / 64, S::K_BLK);
        full(k_full + st);
      };
      // page numbers of tiles: id0 of the first, id1 of i + 1 (its V comes next), raw ahead
      int id0[VU], id1[VU], raw[VU];
      auto idk_of = [&](const int (&id)[VU], int t) {     // the K run's
        return VU == 2 ? (run_k < 4 ? id[0] : id[VU - 1]) : checked(t, run_k, look_up(t, run_k));
      };
#pragma unroll
      for (int e = 0; e < VU; ++e) {
        id0[e] = checked(0, cw + 4 * e, look_up(0, cw + 4 * e));
        id1[e] = checked(1, cw + 4 * e, look_up(1, cw + 4 * e));
        raw[e] = look_up(2, cw + 4 * e);
      }
      load_k(0, id0, idk_of(id0, 0));
      load_v(0, id0);
      meet();
      // (values of scale 0 are stored as zeros: here, and below by not reading them)
#pragma unroll
      for (int e = 0; e < VU; ++e)
        if (!(sv[e] > 0.f))
#pragma unroll
          for (int j = 0; j < VJ; ++j) vb[e][j] = make_uint4(0u, 0u, 0u, 0u);
      put_k(0);
      load_k(1, id1, idk_of(id1, 1));
      for (int i = 0; i < n; ++i) {
        const int st = i % KST;
        int id2[VU];
#pragma unroll
        for (int e = 0; e < VU; ++e) {
          id2[e] = checked(i + 2, cw + 4 * e, raw[e]);
          raw[e] = look_up(i + 3, cw + 4 * e);
        }
        if (i + 1 < n) put_k(i + 1);
#pragma unroll
        for (int e = 0; e < VU; ++e)
          if (!(sv[e] > 0.f)) id1[e] = -1;
        load_k(i + 2, id2, idk_of(id2, i + 2));
        wait(v_empty + st, ((i / KST) & 1) ^ 1);
#pragma unroll
        for (int e = 0; e < VU; ++e) {
          const uint32_t at = S::V_OFF + st * S::V_BYTES + (cw + 4 * e) * 16 * S::V_ROW;
          put(vb[e], at + v_at, at + (v_at ^ 16u), S::VD < 64 ? 1 : S::VD / 64, S::V_BLK);
        }
        full(v_full + st);
        load_v(i + 1, id1);
#pragma unroll
        for (int e = 0; e < VU; ++e) id1[e] = id2[e];
      }
      if (bad && lane == 0) flag_error(status, KVQ_DEV_BADSEQ);
    }
  } else {
    // ================= softmax =================
    const uint32_t tmem = meet();
    if constexpr (MT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    constexpr int NK = MT == 2 ? KT : KT / 2;             // keys of a tile per thread
    const int wg = warp >> 2;                             // row tile, or half of the keys
    const int m = MT == 2 ? wg : 0;
    const int r = 32 * (warp & 3) + lane, rg = row0 + 128 * m + r;
    const int t_r = min(rg / G, g.nt - 1);
    const int p_r = g.p0 + t_r, lo_r = W > 0 ? p_r - W + 1 : 0;
    const bool valid = rg < rows;
    // what every row of the row tile sees
    const int t_first = min((row0 + 128 * m) / G, g.nt - 1), t_last = min((row0 + 128 * m + 127) / G, g.nt - 1);
    const int p_min = g.p0 + t_first, lo_max = W > 0 ? g.p0 + t_last - W + 1 : 0;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t t_o = lanes + m * DO;
    float ref = -INFINITY, l = 0.f;
    float* xm = reinterpret_cast<float*>(sm + S::X_OFF);
    for (int i = 0; i < n; ++i) {
      const int slot = MT == 2 ? m : i & 1;
      const uint32_t t_s = lanes + S::C_S + KT * slot + (MT == 2 ? 0 : (KT / 2) * wg);
      wait(sc_full + (i & 3), (i >> 2) & 1);
      if (MT == 2) wait(s_full + m, i & 1);
      else wait(s_full + slot, (i >> 1) & 1);
      tc::fence_after_sync();
      __syncwarp();
      const float4* sc = reinterpret_cast<const float4*>(sm + S::SC_OFF) + (i & 3) * SUB + (MT == 2 ? 0 : (SUB / 2) * wg);
      const int key0 = k0 + KT * i + (MT == 2 ? 0 : (KT / 2) * wg);
      const bool whole = key0 >= lo_max && key0 + NK - 1 <= p_min;
      // ---- the scores, and the tile's largest t ----
      // (a masked score is -inf; the scales in shared memory are above 0)
      constexpr int NCH = NK / 32;
      uint32_t v[NCH][32];
#pragma unroll
      for (int c = 0; c < NCH; ++c) pf_ld32(t_s + 32 * c, v[c]);
#pragma unroll
      for (int c = 0; c < NCH; ++c) pf_wait(v[c]);
      if (!whole) {
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int key = key0 + 32 * c + e;
            v[c][e] = key <= p_r && key >= lo_r ? v[c][e] : 0xFF800000u;
          }
      }
      float top = -INFINITY;
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float x0 = __uint_as_float(v[c][16 * b]), x1 = __uint_as_float(v[c][16 * b + 1]);
#pragma unroll
          for (int e = 2; e < 14; e += 4) {
            x0 = max3(x0, __uint_as_float(v[c][16 * b + e]), __uint_as_float(v[c][16 * b + e + 1]));
            x1 = max3(x1, __uint_as_float(v[c][16 * b + e + 2]), __uint_as_float(v[c][16 * b + e + 3]));
          }
          x0 = max3(x0, __uint_as_float(v[c][16 * b + 14]), __uint_as_float(v[c][16 * b + 15]));
          const float4 f = sc[2 * c + b];
          top = fmaxf(top, fmaf(fmaxf(x0, x1), f.x, f.y));
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
      for (int c = 0; c < NCH; ++c) {
        uint32_t pw[16];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const float4 f = sc[2 * c + b];
          const float off = f.y - base;
          float2 s0 = {0.f, 0.f}, s1 = {0.f, 0.f};
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            float2 x = fma2(make_float2(__uint_as_float(v[c][16 * b + e]), __uint_as_float(v[c][16 * b + e + 1])),
                            make_float2(f.x, f.x), make_float2(off, off));
            float2 y = fma2(make_float2(__uint_as_float(v[c][16 * b + e + 2]), __uint_as_float(v[c][16 * b + e + 3])),
                            make_float2(f.x, f.x), make_float2(off, off));
            x = make_float2(pf_ex2(x.x), pf_ex2(x.y));
            y = make_float2(pf_ex2(y.x), pf_ex2(y.y));
            s0 = add2(s0, x);
            s1 = add2(s1, y);
            pw[8 * b + e / 2] = pack_h2(x.x, x.y);
            pw[8 * b + e / 2 + 1] = pack_h2(y.x, y.y);
          }
          s0 = add2(s0, s1);
          l = fmaf(s0.x + s0.y, f.z, l);
        }
        pf_st16(t_s + 16 * c, pw);
        if (MT == 2 && c == NCH / 2 - 1) {
          tc::wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::arrive_cta0(p_half + m);
        }
      }
      tc::wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::arrive_cta0(p_full + slot);   // (only tensor memory is passed on)
    }
    // ---- out ----
    if constexpr (MT == 1) {                              // l of both halves
      named_bar(1, 256);                                  // the last maxima are read
      xm[wg * 128 + r] = l;
      named_bar(1, 256);
      l += xm[(wg ^ 1) * 128 + r];
    }
    wait(o_full + m, 0);
    tc::fence_after_sync();
    __syncwarp();
    const float inv = 1.f / l;
    constexpr int OC = MT == 2 ? DO : DO / 2;
    const int o0 = MT == 2 ? 0 : OC * wg;
    const size_t prow = ((size_t)__ldg(order + rank).z * per + hx * pieces + z) * S::ROWS + rg;
    const size_t at = ((size_t)(g.row0 + rg / G) * a.L.n_q + h * G + rg % G) * D + d_base + o0;
    const bool vec = (reinterpret_cast<uintptr_t>(a.out) & 15u) == 0;
#pragma unroll 1
    for (int c = 0; c < OC / 32; ++c) {
      uint32_t w[32];
      pf_ld32(t_o + o0 + 32 * c, w);
      pf_wait(w);
      if (!valid) continue;
      if (pieces > 1) {
        uint4* d = reinterpret_cast<uint4*>(part_o + prow * DO + o0 + 32 * c);
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
        continue;
      }
#pragma unroll
      for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * inv);
      if (a.out_f32) {
        uint32_t* d = reinterpret_cast<uint32_t*>(a.out) + at + 32 * c;
        if (vec) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            reinterpret_cast<uint4*>(d)[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) d[e] = w[e];
        }
      } else {
        uint16_t* d = reinterpret_cast<uint16_t*>(a.out) + at + 32 * c;
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = bf16x2_rn(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1]));
        if (vec) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            reinterpret_cast<uint4*>(d)[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            d[2 * e] = (uint16_t)(w[e] & 0xFFFFu);
            d[2 * e + 1] = (uint16_t)(w[e] >> 16);
          }
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
  tc::cluster_sync();                                     // neither CTA's memory is used any more
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc2(ctl[0], 512);
  }
}

// The units that were cut along the keys: each thread four dims of one row
// over its pieces, in order.
template <int D>
__global__ void __launch_bounds__(256)
paged_join_kernel(const PagedReadArgs a, const int TQ, const int4* order, const float* part_o, const float* part_ml) {
  using S = Pf<D>;
  constexpr int DO = S::DO, ROWS = S::ROWS;
  pdl_launch();
  pdl_wait();
  const int per = a.L.n_kv * S::NSPLIT, G = a.L.G;
  const int rank = blockIdx.x / per, hx = blockIdx.x - rank * per;
  const int4 us = __ldg(order + rank);
  const int pieces = us.w;
  if (pieces < 2) return;
  const PagedGroup g = paged_group_of(a.r, a.pg, a.L.window, TQ, S::KT, us.x, us.y);
  const int i = blockIdx.y * 256 + threadIdx.x;
  const int r = i / (DO / 4), d = (i - r * (DO / 4)) * 4;
  if (r >= g.nt * G) return;
  const size_t row0 = ((size_t)us.z * per + hx * pieces) * ROWS + r;
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

// setmaxnreg hands out the registers that the block was launched with: a build
// that needs fewer than 128 a thread would wait forever, so it is refused.
template <int D, bool E4M3>
cudaError_t check_registers() {
  if (Pf<D>::MT != 2) return cudaSuccess;
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes at;
    const cudaError_t e = cudaFuncGetAttributes(&at, paged_prefill_kernel<D, E4M3>);
    if (e != cudaSuccess) return e;
    regs.store(at.numRegs, std::memory_order_relaxed);
  }
  return regs.load(std::memory_order_relaxed) == 128 ? cudaSuccess : cudaErrorLaunchOutOfResources;
}

// most: pieces of a unit; places: for the pieces of units that are cut (of this
// call or any of fewer rows, which may cut more)
struct PfPlan { int TQ, n_groups, most; long long units, places; };
template <int D>
PfPlan pf_plan(const LayerArgs& L, int n_seqs, int n_rows, int max_pos, int num_sms) {
  using S = Pf<D>;
  PfPlan p;
  p.TQ = S::ROWS / L.G;
  static const int32_t some = 0;
  p.n_groups = paged_groups(PagedRows{&some, nullptr, n_seqs, n_rows}, p.TQ);
  p.units = (long long)p.n_groups * L.n_kv * S::NSPLIT;
  // as many pieces as fill the GPU once (one pair per two SMs), of at least two tiles; where the units are
  // more than their rows would fill, as many as fit places for twice the pairs (once: 2 chunks of 40 rows
  // behind 16,000 keys with 3 behind 2,000, 32q/8kv D 128, 202 us for 101; 32 windows of 32 rows, 8q/2kv
  // D 256, window 512, 32 for 51)
  long long keys = (long long)max_pos + 1;
  if (L.window > 0) keys = std::min<long long>(keys, (long long)L.window + p.TQ);
  const long long tiles = (keys + S::KT - 1) / S::KT;
  // (groups are counted with room for one short one per sequence)
  const long long real = std::max(1ll, ((long long)n_rows / p.TQ + (n_rows % p.TQ != 0)) * L.n_kv * S::NSPLIT);
  const long long cut = std::max(1ll, std::min<long long>(tiles / 2, kMostPieces));
  p.most = (int)std::max(1ll, std::min<long long>(num_sms / 2 / real, cut));
  p.places = cut > 1 ? std::min<long long>(num_sms / 2 * 2, p.units * cut) : 0;
  return p;
}

// status (256 B), q16, order, part_o, part_ml
struct PfWs { size_t q16, order, part_o, part_ml, total; };
template <int D>
PfWs pf_ws(const LayerArgs& L, int n_rows, const PfPlan& p) {
  using S = Pf<D>;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t prows = (size_t)p.places * S::ROWS;
  PfWs w;
  w.q16 = 256;
  w.order = up(w.q16 + (size_t)n_rows * L.n_q * D * 2);
  w.part_o = up(w.order + (size_t)p.n_groups * 16);
  w.part_ml = up(w.part_o + prows * S::DO * 4);
  w.total = up(w.part_ml + prows * 8);
  return w;
}

template <int D, bool E4M3>
cudaError_t launch_t(const PagedReadArgs& a, const RopeFreqs& f, int max_pos, void* ws, int num_sms, cudaStream_t st) {
  using S = Pf<D>;
  const PfPlan p = pf_plan<D>(a.L, a.r.n_seqs, a.r.n_rows, max_pos, num_sms);
  const PfWs w = pf_ws<D>(a.L, a.r.n_rows, p);
  if (p.units > 0x3fffffffLL) return cudaErrorInvalidValue;
  uint8_t* b = static_cast<uint8_t*>(ws);
  uint32_t* status = reinterpret_cast<uint32_t*>(b);
  uint16_t* q16 = reinterpret_cast<uint16_t*>(b + w.q16);
  int4* order = reinterpret_cast<int4*>(b + w.order);
  float* part_o = reinterpret_cast<float*>(b + w.part_o);
  float* part_ml = reinterpret_cast<float*>(b + w.part_ml);
  cudaError_t e = check_registers<D, E4M3>();
  if (e != cudaSuccess) return e;
  const PagedOrder po = {order, a.L.n_kv * S::NSPLIT, p.most, (int)p.places};
  e = launch_paged_prep<D>(a, f, p.TQ, S::KT, p.n_groups, q16, nullptr, po, status, num_sms, st);
  if (e != cudaSuccess) return e;
  static std::atomic<uint64_t> allowed{0};
  e = allow_smem(paged_prefill_kernel<D, E4M3>, S::BYTES, allowed);
  if (e != cudaSuccess) return e;
  if ((e = prof_before(st)) != cudaSuccess) return e;
  e = launch_pdl(paged_prefill_kernel<D, E4M3>, dim3((unsigned)p.units * 2, p.most), dim3(S::THREADS), S::BYTES, st, a,
                 p.TQ, order, q16, part_o, part_ml, status);
  if (e != cudaSuccess) return e;
  if ((e = prof_after(st)) != cudaSuccess || p.most == 1) return e;
  // (units that are cut are the first of the order, and have two places at least)
  const long long cut = std::min(p.units, p.places / 2);
  return launch_pdl(paged_join_kernel<D>, dim3((unsigned)cut, S::ROWS * (S::DO / 4) / 256), dim3(256), 0, st, a, p.TQ,
                    order, part_o, part_ml);
}

template <int D>
cudaError_t launch_d(const PagedReadArgs& a, const RopeFreqs& f, int max_pos, void* ws, int num_sms, cudaStream_t st) {
  return a.pg.e4m3 ? launch_t<D, true>(a, f, max_pos, ws, num_sms, st)
                   : launch_t<D, false>(a, f, max_pos, ws, num_sms, st);
}

}  // namespace

// The rows of a call go to one kernel, by those of its longest sequence.  32 (token, head) rows, two units
// of the row kernel, for which it walks the keys twice, is where the two cross at the latest when the GPU is
// full: us a call of this kernel / the row kernel, 64 sequences behind 4000 keys (one behind 16,000):
//   (token, head) rows        16             32             64             128            256
//   D 64, 8q/2kv      125 / 35       113 / 58       115 / 98       116 / 181      117 / 410
//                    (28 / 13)      (30 / 14)      (31 / 17)      (33 / 20)      (34 / 27)
//   D 128, 32q/8kv    401 / 143      393 / 238      401 / 425      410 / 792      436 / 1513
//                    (39 / 23)      (40 / 27)      (41 / 36)      (43 / 59)      (46 / 104)
//   D 256, 8q/2kv     124 / 86       125 / 149      130 / 254      130 / 443      138 / 817
//                    (32 / 18)      (33 / 22)      (34 / 27)      (37 / 38)      (40 / 61)
//   D 512, 16q/1kv    208 / 93       210 / 149      214 / 261      222 / 472      234 / 796
//                    (44 / 21)      (46 / 24)      (48 / 31)      (52 / 39)      (49 / 60)
//   D 256, window 512, 32 sequences: 34 / 30   36 / 41   40 / 62   51 / 100   32 / 131
// G = 3, 5, 6, .. rows of a token do not divide a row tile, whose places are formed by shifts: such layers
// take the row kernel at any length (6374 prompt rows of 24q/8kv D 128 1170 us, of 32q/8kv 206 here).
bool paged_prefill_supported(const LayerArgs& L, int max_rows_per_seq) {
  return 128 % L.G == 0 && max_rows_per_seq > 32 / L.G;   // (their product may pass 32 bits)
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
