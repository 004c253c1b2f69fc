// attn_paged_decode (and few-row windows of attn_paged_prefill): attention of
// single tokens over pages of 8-bit codes, on mma.sync.
//
// A unit is one kv head of a group of up to 16 / G rows of one sequence: its
// 16 (token, q head) rows are the M rows of m16n8k16 (row r = token r / G, head
// r % G), so a window of drafted rows reads its keys once.  The key tiles (64 or
// 128 positions) of all units, in (group, kv head, tile) order, and a place per unit
// for what it costs however short it is, are cut into equal contiguous shares,
// one per CTA (long and short sequences mixed leave no CTA idle); a share that
// holds part of a unit leaves its softmax state and sums in the workspace and
// paged_merge_kernel joins the parts in order.
//
// Mathematics, per key j of a page with scales sk, sv and codes ck_j, cv_j:
//   y_j = (q . ck_j) sk log2 e          (products of f16 q and codes are exact)
//   t_j = y_j + log2 sv
//   p_j = 2^(t_j - ref)                 rounded to f16 for the product with cv
//   O += p_j cv_j,   l += p_j / sv      out = O / l
// The value scale goes into the probability, not the codes, so both products
// take codes as exact f16 values, and ref follows the largest t_j, so p_j <=
// 2^15 whatever the scales are (renewed when a tile exceeds it by 2^8).  A value
// scale of 0 (rows of zeros, whatever numbers the codes are) counts as kZeroScale
// in t and l, and its p enters the product as 0.  Keys whose page is not named have
// a K scale of NaN: so have the scores of the rows that see them, and those rows alone.
//
// A CTA is four warps; with D >= 256, WD = D / 128 of them form a team that
// shares the output: each keeps 128 dims of O (64 registers) for the keys of
// all of them, and they exchange P and the row maxima through shared memory,
// one barrier a tile (the next tile's scores are formed before it, so it also
// publishes their maxima).  With D <= 128 a warp works alone, on 32 keys of a
// tile of 128.
//
// Codes come by the tensor memory accelerator in boxes of 16 keys x 128 dims
// (one page, one scale) into a ring that is the warp's own: no barrier between
// warps, and a box is refilled as soon as the warp has read it.  The boxes are
// 128-byte swizzled; which key an MMA column stands for is chosen (key_of) so
// that neither the K reads (two keys, four 16-byte chunks a quarter warp) nor
// the V reads (four keys, two chunks) meet a bank twice.  The order of dims
// inside an MMA's k range and of output columns is free too, so a lane takes 16
// consecutive bytes.  Page numbers are looked up a tile ahead of the copies.
// (16-byte asynchronous copies by every lane, in the place of the accelerator,
// spent a third of the instructions on addresses and bounds.)
//
// What bounds it, measured on GB300: 64 ragged sequences of up to 16,000 keys, 32 q
// heads on 8 of 128, e4m3 (577 MB): 113 us with prep and merge, 86 of them the walk
// at the copy rate, 5 until the first tile is there, 9 until the last CTA ends;
// 8 x 32,700 keys, 16 q heads on one of 512, int8 (268 MB): 69 us, the walk 46 (0.87 of
// the copy rate), the prep before it 7, results and merge 9.  Rings of K and V
// apart, q in shared memory at D 128 and a fourth CTA per SM gained nothing.
#include <algorithm>

#include "kvq_paged.cuh"
#include "kvq_paged_rows.cuh"
#include "kvq_tc.cuh"
#include "kvq_tma.cuh"

namespace kvq {

namespace {

constexpr int kPdThreads = 128;
constexpr int kPdMinKeys = 128;          // shortest share of a CTA, keys
// Groups that a CTA plans itself, one a thread, in the place of waiting for the
// prep kernel's plan: 16 single rows 10.5 us a call for 12.5, 64 14.8 for 15.6; beyond
// that it costs more than the wait (600 rows 52.7 for 51.7, 400 groups of windows 63 for 60).
constexpr int kPdPlan = kPdThreads;

template <int D>
struct Pd {
  static constexpr int WD = D >= 128 ? D / 128 : 1;     // warps that share a tile's output dims
  static constexpr int TEAMS = 4 / WD;
  static constexpr int SW = WD == 1 ? 2 : 1;            // 16-key subtiles per warp and tile
  static constexpr int SUBS = 4 * SW;                   // per tile
  static constexpr int KT = 16 * SUBS;                  // keys per tile
  static constexpr int SV = SW * WD;                    // subtiles whose V a warp multiplies
  static constexpr int DS = D / WD;                     // output dims per warp
  static constexpr int NT = DS / 8;                     // 8-dim MMA columns per warp
  static constexpr int VB = DS / 8;                     // V bytes of a key per lane (8 or 16)
  static constexpr int KS = D / 16;                     // MMA steps of QK
  static constexpr bool QREG = D <= 128;                // q fragments in registers
  // a warp's ring: boxes of 16 keys x ROW bytes; per tile NK of K, then SV of V
  static constexpr int ROW = D < 128 ? D : 128;
  static constexpr int BOX = 16 * ROW;
  static constexpr int KBX = D < 128 ? 1 : D / 128;     // K boxes of a subtile
  static constexpr int NK = SW * KBX;
  static constexpr int NB = NK + SV;
  static constexpr int DEP = D == 512 ? 1 : 2;          // tiles in the ring
  static constexpr int CPS = D == 64 ? 4 : D == 128 ? 3 : 2;       // CTAs per SM
  static constexpr int RING = 4 * DEP * NB * BOX;
  static constexpr int Q_OFF = RING;                    // q fragments [KS][32] x 16 B
  static constexpr int P_OFF = Q_OFF + (QREG ? 0 : KS * 512);      // P fragments [2][4 warps][32] x 16 B
  static constexpr int M_OFF = P_OFF + (WD > 1 ? 4096 : 0);        // row maxima [2][4 warps][16]
  static constexpr int S_OFF = M_OFF + 512;             // scales [4 warps][4 tiles][SW][2]
  static constexpr int B_OFF = S_OFF + 4 * 4 * 2 * 2 * 4;          // barriers [4 warps][DEP][NB]
  static constexpr int PLAN_OFF = B_OFF + 4 * DEP * NB * 8;       // a small call's plan, and 4 sums
  static constexpr int BYTES = PLAN_OFF + (kPdPlan + 1 + 4) * 4;
  static constexpr int OSTR = D + 4;                    // floats of a merged row (a row's start moves by 4 banks)
  static_assert(TEAMS * 16 * OSTR * 4 + 128 * 4 <= RING, "the merge of a CTA's warps reuses the ring");
};

// The key of a subtile's 8 that column i of an MMA stands for.
__device__ __forceinline__ int key_of(int i) { return i & 1 ? (i - 1) ^ 5 : i; }
// Byte offset of 16-byte chunk c of key k in a box (the accelerator's swizzle).
template <int ROW>
__device__ __forceinline__ uint32_t box_off(int k, int c) {
  return ROW == 128 ? k * 128 + ((c ^ (k & 7)) << 4) : k * 64 + ((c ^ ((k >> 1) & 3)) << 4);
}

__device__ __forceinline__ void cp4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(m)) : "memory");
}
__device__ __forceinline__ uint4 lds128(const void* p) { return *reinterpret_cast<const uint4*>(p); }

// The shares of a call: a line of T places (a unit has one for what it costs at
// all, then one per key tile) over nc CTAs, CTA c taking those from
// ceil(T c / nc) to before ceil(T (c + 1) / nc).
struct PdShares {
  long long T;
  int nc;
  __device__ long long begin(int c) const { return (T * c + nc - 1) / nc; }
  __device__ int cta_of(long long x) const { return (int)(x * nc / T); }
};
template <int D>
__device__ __forceinline__ PdShares pd_shares(long long T, int ctas) {
  return {T, (int)max(1ll, min((long long)ctas, T * Pd<D>::KT / kPdMinKeys))};
}

// part_o [2 ctas][16][D], part_ml [2 ctas][2][16]: slot 2 c of CTA c is the
// piece that begins its share, 2 c + 1 the piece that ends it.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kPdThreads, Pd<D>::CPS)
paged_decode_kernel(const PagedReadArgs a, const __grid_constant__ CUtensorMap tmk,
                    const __grid_constant__ CUtensorMap tmv, const int TG, const int n_groups, const uint16_t* q16,
                    const long long* prefix, float* part_o, float* part_ml, uint32_t* status) {
  using S = Pd<D>;
  constexpr int WD = S::WD, NT = S::NT, VB = S::VB, KS = S::KS, SW = S::SW, SV = S::SV, NK = S::NK, NB = S::NB,
                DEP = S::DEP, KT = S::KT;
  constexpr float L2E = 1.4426950408889634f;
  constexpr float kSlack = 8.f;      // how far a tile may exceed ref, log2
  constexpr float kTop = 7.f;        // p of a key at ref is 2^kTop
  extern __shared__ __align__(1024) uint8_t sm[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rr = lane >> 2, cc = lane & 3;
  const int team = warp / WD, wd = warp % WD;
  const int G = a.L.G, n_kv = a.L.n_kv, P = a.pg.P, sh = a.pg.p_shift, W = a.L.window;
  uint8_t* ring = sm + warp * (DEP * NB * S::BOX);
  float* scale = reinterpret_cast<float*>(sm + S::S_OFF) + warp * 4 * SW * 2;
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + S::B_OFF) + warp * DEP * NB;
  if (lane == 0) {
    prefetch_map(&tmk);
    prefetch_map(&tmv);
    for (int i = 0; i < DEP * NB; ++i) mbar_init(full + i, 1);
    fence_mbar_init();
  }
  __syncwarp();
  pdl_launch();
  // The prep kernel lets this one start when the kernels before both are
  // complete, so up to kPdPlan groups are planned here, and the first keys asked
  // for, while it runs; q16 and the status word are waited for before their use.
  const bool own = n_groups <= kPdPlan;
  int* const plan = reinterpret_cast<int*>(sm + S::PLAN_OFF);
  if (own) paged_plan<4>(a.r, a.pg, W, TG, KT, n_groups, plan, plan + kPdPlan + 1);
  else pdl_wait();
  bool waited = !own;
  const auto width_before = [=](int i) { return own ? (long long)plan[i] : __ldg(prefix + i); };
  const PdShares shares = pd_shares<D>(width_before(n_groups) * n_kv, gridDim.x);
  if (shares.T == 0 || (int)blockIdx.x >= shares.nc) {
    if (own) pdl_wait();                                  // (whoever waits for this kernel waits for that one)
    return;
  }
  long long x = shares.begin(blockIdx.x);
  const long long x_begin = x, x_end = shares.begin(blockIdx.x + 1);
  int used = 0;                                           // tiles the ring has held
  bool dead = false;
  auto wait = [&](uint64_t* bar, int parity) {
    if (!dead && !mbar_wait(bar, parity)) {
      dead = true;
      flag_error(status, KVQ_DEV_TIMEOUT);
    }
  };

  while (x < x_end) {
    // ---- the unit of place x: group u, kv head h, n of its key tiles from t_a ----
    const auto first_place = [=](int i) { return width_before(i) * n_kv; };
    const int u = warp_search(n_groups, x, first_place);
    const long long w0 = width_before(u);
    const int width = (int)(width_before(u + 1) - w0);
    const PagedGroup g = paged_group<true>(a.r, a.pg, W, TG, KT, u);
    const int in_u = (int)(x - w0 * n_kv);
    const int h = in_u / width, at = in_u - h * width;
    const int t_a = max(at - 1, 0);
    const int places = (int)min((long long)(width - at), x_end - x);
    const int n = places - (at == 0 ? 1 : 0);
    if (n == 0) {                                         // the share ends before the unit's first tile
      x += places;
      continue;
    }
    const int k0 = g.kt0 + KT * t_a;                      // first position of the piece
    const int rows = g.nt * G;

    // ---- page numbers: lane i < SUBS looks up the page of 16 positions i of a tile ----
    bool bad = false;
    const int32_t* table = a.pg.tables + (size_t)g.s * a.pg.max_pages;
    auto seen = [&](int t) {
      const int key = k0 + KT * t + 16 * lane;
      return lane < S::SUBS && t < n && key <= g.hi && key + 15 >= g.lo;
    };
    auto look_up = [&](int t) { return seen(t) ? __ldg(table + ((k0 + KT * t + 16 * lane) >> sh)) : -1; };
    // the page of a looked-up entry of tile t (which may hold any number), -1 where no row sees it, kNoPage where the
    // entry names none
    auto checked = [&](int t, int id) {
      if (!seen(t)) return -1;
      if ((unsigned)id < (unsigned)a.pg.n_pages) return id;
      bad = true;
      return kNoPage;
    };
    // copies of a box: 16 positions from key0, bytes x .. of their rows, of page id (zeros, from outside the pages,
    // where there is none)
    auto copy = [&](int box, const CUtensorMap* map, int id, int key0, int xb) {
      mbar_arrive_expect_tx(full + box, S::BOX);
      tc::tma_load_3d(smem_u32(ring + box * S::BOX), map, xb, key0 & (P - 1), id < 0 ? -1 : id * n_kv + h,
                      smem_u32(full + box));
    };
    auto issue_k = [&](int t, int pid) {                  // K and the scales of tile t
      const int slot = (used + t) % DEP;
      int ids[SW];
#pragma unroll
      for (int e = 0; e < SW; ++e) ids[e] = __shfl_sync(0xffffffffu, pid, SW * warp + e);
      const int key0 = k0 + KT * t + 16 * SW * warp;
      if (lane == 0) {
#pragma unroll
        for (int e = 0; e < SW; ++e)
#pragma unroll
          for (int b = 0; b < S::KBX; ++b) copy(slot * NB + e * S::KBX + b, &tmk, ids[e], key0 + 16 * e, 128 * b);
      }
      if (lane < 2 * SW) {
        // (keys without a page: a K scale of NaN)
        const int id = SW == 2 && lane >= 2 ? ids[SW - 1] : ids[0];
        float* at = scale + ((used + t) & 3) * SW * 2 + lane;
        if (id == kNoPage) *at = lane & 1 ? 0.f : __int_as_float(0x7FC00000);
        else cp4(smem_u32(at), (lane & 1 ? a.pg.v_scales : a.pg.k_scales) + (size_t)max(id, 0) * n_kv + h,
                 id >= 0 ? 4u : 0u);
      }
    };
    auto issue_v = [&](int t, int pid) {                  // V of tile t: the team's keys, the warp's dims
      const int slot = (used + t) % DEP;
#pragma unroll
      for (int e = 0; e < SV; ++e) {
        const int sub = team * SV + e, id = __shfl_sync(0xffffffffu, pid, sub);
        if (lane == 0) copy(slot * NB + NK + e, &tmv, id, k0 + KT * t + 16 * sub, wd * S::DS);
      }
    };
    // pages of tile j + DEP (V comes next) and j + DEP + 1 (K)
    int pid_v = checked(0, look_up(0)), pid_k, raw;
    if (DEP == 2) {
      pid_k = checked(1, look_up(1));
      raw = look_up(2);
      issue_k(0, pid_v);
      cp_commit();
      issue_v(0, pid_v);
      if (n > 1) issue_k(1, pid_k);
      cp_commit();
      if (n > 1) issue_v(1, pid_k);
      pid_v = checked(2, raw);
      raw = look_up(3);
    } else {
      raw = look_up(1);
      issue_k(0, pid_v);
      cp_commit();
      issue_v(0, pid_v);
      pid_v = checked(1, raw);
      raw = look_up(2);
    }
    pid_k = pid_v;

    if (!waited) {
      pdl_wait();
      waited = true;
    }

    // ---- q fragments of the unit: step 4 b + t takes dims 64 b + 16 c + 4 t .. +3 of lane column c ----
    uint32_t qf[S::QREG ? KS : 1][4];
    {
      auto q_row = [&](int r) {
        return q16 + ((size_t)(g.row0 + r / G) * a.L.n_q + h * G + r % G) * D;
      };
      // (a team's warps fill the fragments that all of them read, every fourth block of 64 dims each)
      constexpr int STEP = S::QREG ? 1 : 4, NBL = D / 64 / STEP;
      const int b0 = S::QREG ? 0 : warp;
      uint4 v[NBL][2][2];
#pragma unroll
      for (int i = 0; i < NBL; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          v[i][e][0] = v[i][e][1] = make_uint4(0, 0, 0, 0);
          if (rr + 8 * e < rows) {
            const uint4* src = reinterpret_cast<const uint4*>(q_row(rr + 8 * e) + 64 * (b0 + STEP * i) + 16 * cc);
            v[i][e][0] = src[0];
            v[i][e][1] = src[1];
          }
        }
#pragma unroll
      for (int i = 0; i < NBL; ++i) {
        const uint32_t* w0 = reinterpret_cast<const uint32_t*>(v[i][0]);
        const uint32_t* w1 = reinterpret_cast<const uint32_t*>(v[i][1]);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          if constexpr (S::QREG) {
            qf[4 * i + t][0] = w0[2 * t];
            qf[4 * i + t][1] = w1[2 * t];
            qf[4 * i + t][2] = w0[2 * t + 1];
            qf[4 * i + t][3] = w1[2 * t + 1];
          } else {
            reinterpret_cast<uint4*>(sm + S::Q_OFF)[(4 * (b0 + STEP * i) + t) * 32 + lane] =
                make_uint4(w0[2 * t], w1[2 * t], w0[2 * t + 1], w1[2 * t + 1]);
          }
        }
      }
      if constexpr (!S::QREG) __syncthreads();
    }

    // what the thread's two rows see, and what all of them do
    const int pr0 = g.p0 + min(rr / G, g.nt - 1), pr1 = g.p0 + min((rr + 8) / G, g.nt - 1);
    const int lo0 = W > 0 ? pr0 - W + 1 : 0, lo1 = W > 0 ? pr1 - W + 1 : 0;
    const int lo_last = W > 0 ? g.hi - W + 1 : 0;
    const int kc0 = key_of(2 * cc), kc1 = key_of(2 * cc + 1);      // keys of the thread's columns

    float O[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) O[i][e] = 0.f;
    float ref0 = -INFINITY, ref1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float sc[SW][2][4];                                   // raw scores of the tile to come: subtile, 8 keys, MMA element
    float sk[SW], lsv[SW], isv[SW];

    // scores of tile j, its boxes refilled, its scales; the maxima of the thread's rows over the warp's keys
    auto scores = [&](int j, float& m0, float& m1) {
      const int tt = used + j, slot = tt % DEP, par = (tt / DEP) & 1;
      m0 = m1 = -INFINITY;
      cp_wait<DEP - 1>();
      __syncwarp();
#pragma unroll
      for (int e = 0; e < SW; ++e) {
        constexpr int CH = D >= 256 ? 2 : 1;              // accumulation chains per 8 keys
        float acc[CH][2][4];
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int f = 0; f < 2; ++f)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[c][f][i] = 0.f;
#pragma unroll
        for (int b = 0; b < D / 64; ++b) {
          const int box = slot * NB + e * S::KBX + b / 2;
          if (b % 2 == 0) wait(full + box, par);
          const uint8_t* bx = ring + box * S::BOX;
          const uint4 ka = lds128(bx + box_off<S::ROW>(key_of(rr), 4 * (b & 1) + cc));
          const uint4 kb = lds128(bx + box_off<S::ROW>(8 + key_of(rr), 4 * (b & 1) + cc));
          const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            uint32_t q[4];
            if constexpr (S::QREG) {
#pragma unroll
              for (int i = 0; i < 4; ++i) q[i] = qf[4 * b + t][i];
            } else {
              const uint4 v = lds128(sm + S::Q_OFF + ((4 * b + t) * 32 + lane) * 16);
              q[0] = v.x; q[1] = v.y; q[2] = v.z; q[3] = v.w;
            }
            uint32_t b0, b1;
            codes_to_h2<E4M3>(wa[t], b0, b1);
            mma_f16(acc[t % CH][0], q, b0, b1);
            codes_to_h2<E4M3>(wb[t], b0, b1);
            mma_f16(acc[t % CH][1], q, b0, b1);
          }
        }
        const float2 s2 = *reinterpret_cast<const float2*>(scale + ((tt & 3) * SW + e) * 2);
        // (a K scale of 0: scores of 0, by a factor that keeps a masked -inf what it is)
        sk[e] = fmaxf(s2.x * L2E, 1e-30f);
        const float sv = s2.y > 0.f ? s2.y : kZeroScale;
        lsv[e] = __log2f(sv);
        isv[e] = __fdividef(1.f, sv);
        const int key0 = k0 + KT * j + 16 * (SW * warp + e);
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[e][f][i] = CH == 2 ? acc[0][f][i] + acc[CH - 1][f][i] : acc[0][f][i];
        // a row does not see all 16 keys, or they have no page (NaN for the rows that see one)
        if (key0 < lo_last || key0 + 15 > g.p0 || s2.x != s2.x) {
          const float add = s2.x - s2.x;
#pragma unroll
          for (int f = 0; f < 2; ++f)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int key = key0 + 8 * f + (i & 1 ? kc1 : kc0);
              const bool see = (i >> 1) ? key <= pr1 && key >= lo1 : key <= pr0 && key >= lo0;
              sc[e][f][i] = see ? sc[e][f][i] + add : -INFINITY;
            }
        }
        m0 = fmaxf(m0, fmaf(fmaxf(fmaxf(sc[e][0][0], sc[e][0][1]), fmaxf(sc[e][1][0], sc[e][1][1])), sk[e], lsv[e]));
        m1 = fmaxf(m1, fmaf(fmaxf(fmaxf(sc[e][0][2], sc[e][0][3]), fmaxf(sc[e][1][2], sc[e][1][3])), sk[e], lsv[e]));
      }
      __syncwarp();                                       // the boxes and scales are read
      if (j + DEP < n) issue_k(j + DEP, pid_k);
      cp_commit();
#pragma unroll
      for (int m = 1; m <= 2; m <<= 1) {
        m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, m));
        m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, m));
      }
    };
    float* mbuf = reinterpret_cast<float*>(sm + S::M_OFF);
    auto post_max = [&](int j, float m0, float m1) {
      if (cc == 0) {
        mbuf[((j & 1) * 4 + warp) * 16 + rr] = m0;
        mbuf[((j & 1) * 4 + warp) * 16 + rr + 8] = m1;
      }
    };
    auto team_sync = [&]() {
      if constexpr (WD == 4) __syncthreads();
      else if constexpr (WD == 2) named_bar(1 + team, 64);
    };

    // ---- tile by tile ----
    float m0, m1;
    scores(0, m0, m1);
    if constexpr (WD > 1) {
      post_max(0, m0, m1);
      team_sync();
    }
    for (int j = 0; j < n; ++j) {
      // (pid_k served K of tile j + DEP: the same pages hold its V)
      pid_v = pid_k;
      pid_k = checked(j + DEP + 1, raw);
      raw = look_up(j + DEP + 2);
      if constexpr (WD > 1) {
#pragma unroll
        for (int w = 0; w < WD; ++w) {
          m0 = fmaxf(m0, mbuf[((j & 1) * 4 + team * WD + w) * 16 + rr]);
          m1 = fmaxf(m1, mbuf[((j & 1) * 4 + team * WD + w) * 16 + rr + 8]);
        }
      }
      // a renewed reference: what was summed so far is rescaled
      const bool new0 = m0 > ref0 + kSlack || (ref0 == -INFINITY && m0 > -INFINITY);
      const bool new1 = m1 > ref1 + kSlack || (ref1 == -INFINITY && m1 > -INFINITY);
      if (__any_sync(0xffffffffu, new0 || new1)) {
        const float a0 = new0 ? ex2(ref0 - m0) : 1.f, a1 = new1 ? ex2(ref1 - m1) : 1.f;
        if (new0) ref0 = m0;
        if (new1) ref1 = m1;
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          O[i][0] *= a0;
          O[i][1] *= a0;
          O[i][2] *= a1;
          O[i][3] *= a1;
        }
      }
      uint32_t pf[SW][4];
      const float r0 = ref0 == -INFINITY ? 0.f : ref0 - kTop, r1 = ref1 == -INFINITY ? 0.f : ref1 - kTop;
#pragma unroll
      for (int e = 0; e < SW; ++e) {
        const float c0 = lsv[e] - r0, c1 = lsv[e] - r1;
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const float p0 = ex2(fmaf(sc[e][f][0], sk[e], c0)), p1 = ex2(fmaf(sc[e][f][1], sk[e], c0));
          const float p2 = ex2(fmaf(sc[e][f][2], sk[e], c1)), p3 = ex2(fmaf(sc[e][f][3], sk[e], c1));
          s0 += p0 + p1;
          s1 += p2 + p3;
          pf[e][2 * f] = pack_h2(p0, p1);
          pf[e][2 * f + 1] = pack_h2(p2, p3);
        }
        l0 = fmaf(s0, isv[e], l0);
        l1 = fmaf(s1, isv[e], l1);
        if (lsv[e] < -50.f) {                             // values of scale 0 (the smallest other: -40)
#pragma unroll
          for (int i = 0; i < 4; ++i) pf[e][i] = 0u;
        }
      }
      if constexpr (WD > 1)
        *reinterpret_cast<uint4*>(sm + S::P_OFF + ((j & 1) * 4 + warp) * 512 + lane * 16) =
            make_uint4(pf[0][0], pf[0][1], pf[0][2], pf[0][3]);
      if (j + 1 < n) {
        scores(j + 1, m0, m1);
        if constexpr (WD > 1) post_max(j + 1, m0, m1);
      }
      team_sync();
      const int slot = (used + j) % DEP, par = ((used + j) / DEP) & 1;
#pragma unroll
      for (int e = 0; e < SV; ++e) {
        uint32_t p[4];
        if constexpr (WD > 1) {
          const uint4 v = lds128(sm + S::P_OFF + ((j & 1) * 4 + team * WD + e) * 512 + lane * 16);
          p[0] = v.x; p[1] = v.y; p[2] = v.z; p[3] = v.w;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) p[i] = pf[e][i];
        }
        const int box = slot * NB + NK + e;
        wait(full + box, par);
        const uint8_t* bx = ring + box * S::BOX;
        uint32_t vw[4][VB / 4];
#pragma unroll
        for (int f = 0; f < 4; ++f) {                     // the keys of P's columns
          const int k = (f & 1 ? kc1 : kc0) + 8 * (f >> 1);
          if constexpr (VB == 16) {
            const uint4 v = lds128(bx + box_off<S::ROW>(k, rr));
            vw[f][0] = v.x; vw[f][1] = v.y; vw[f][2] = v.z; vw[f][3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(bx + box_off<S::ROW>(k, rr >> 1) + 8 * (rr & 1));
            vw[f][0] = v.x; vw[f][1] = v.y;
          }
        }
        if constexpr (E4M3) {
          // bytes that no row sees may read as NaN, which a weight of 0 does not hide
          const int key0 = k0 + KT * j + 16 * (team * SV + e);
          if (key0 < g.lo || key0 + 15 > g.hi) {
#pragma unroll
            for (int f = 0; f < 4; ++f) {
              const int key = key0 + (f & 1 ? kc1 : kc0) + 8 * (f >> 1);
              if (key < g.lo || key > g.hi)
#pragma unroll
                for (int w = 0; w < VB / 4; ++w) vw[f][w] = 0u;
            }
          }
        }
#pragma unroll
        for (int w = 0; w < VB / 4; ++w) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {                // dims 4 w + 2 hf, + 1 of the lane's
            const uint32_t sel = hf ? 0x7362u : 0x5140u;  // bytes (key, next key) of two dims
            uint32_t a0, a1, b0, b1;
            codes_to_h2<E4M3>(prmt(vw[0][w], vw[1][w], sel), a0, a1);
            codes_to_h2<E4M3>(prmt(vw[2][w], vw[3][w], sel), b0, b1);
            mma_f16(O[4 * w + 2 * hf], p, a0, b0);
            mma_f16(O[4 * w + 2 * hf + 1], p, a1, b1);
          }
        }
      }
      __syncwarp();                                       // V is read
      if (j + DEP < n) issue_v(j + DEP, pid_v);
    }
    used += n;

    // ---- join the warps, in shared memory ----
    cp_wait<0>();
    bad = __syncthreads_or(bad);
    if (bad && tid == 0) flag_error(status, KVQ_DEV_BADSEQ);
#pragma unroll
    for (int m = 1; m <= 2; m <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, m);
      l1 += __shfl_xor_sync(0xffffffffu, l1, m);
    }
    float* ob = reinterpret_cast<float*>(sm);             // [TEAMS][16][OSTR]
    float* lb = ob + S::TEAMS * 16 * S::OSTR;             // [4 warps][16] l, then [4 warps][16] ref
    if (cc == 0) {
      lb[warp * 16 + rr] = l0;
      lb[warp * 16 + rr + 8] = l1;
      lb[64 + warp * 16 + rr] = ref0;
      lb[64 + warp * 16 + rr + 8] = ref1;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (rr + 8 * e < rows) {
#pragma unroll
        for (int cn = 0; cn < 2; ++cn) {
          float* dst = ob + (team * 16 + rr + 8 * e) * S::OSTR + wd * S::DS + VB * (2 * cc + cn);
#pragma unroll
          for (int i = 0; i < NT; i += 4)
            *reinterpret_cast<float4*>(dst + i) = make_float4(O[i][2 * e + cn], O[i + 1][2 * e + cn],
                                                              O[i + 2][2 * e + cn], O[i + 3][2 * e + cn]);
        }
      }
    }
    __syncthreads();
    const bool whole = n == width - 1;
    const int slot = 2 * blockIdx.x + (x == x_begin ? 0 : 1);
    for (int i = tid; i < rows * (D / 4); i += kPdThreads) {
      const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
      float M = -INFINITY, l = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) M = fmaxf(M, lb[64 + w * 16 + r]);
      float4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int t = 0; t < S::TEAMS; ++t) {
        const float rf = lb[64 + t * WD * 16 + r], f = rf == -INFINITY ? 0.f : ex2(rf - M);
        const float4 v = *reinterpret_cast<const float4*>(ob + (t * 16 + r) * S::OSTR + d);
        o.x = fmaf(v.x, f, o.x);
        o.y = fmaf(v.y, f, o.y);
        o.z = fmaf(v.z, f, o.z);
        o.w = fmaf(v.w, f, o.w);
#pragma unroll
        for (int w = 0; w < WD; ++w) l = fmaf(lb[(t * WD + w) * 16 + r], f, l);
      }
      if (whole) {
        const float inv = 1.f / l;
        const size_t at = ((size_t)(g.row0 + r / G) * a.L.n_q + h * G + r % G) * D + d;
        const float w[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (a.out_f32) reinterpret_cast<float*>(a.out)[at + e] = w[e];
          else reinterpret_cast<uint16_t*>(a.out)[at + e] = f_to_bf16_rn(w[e]);
        }
      } else {
        *reinterpret_cast<float4*>(part_o + ((size_t)slot * 16 + r) * D + d) = o;
        if (d == 0) {
          part_ml[(size_t)slot * 32 + r] = M;
          part_ml[(size_t)slot * 32 + 16 + r] = l;
        }
      }
    }
    fence_proxy_async();                                  // (the accelerator writes there next)
    __syncthreads();
    x += places;
  }
  if (!waited) pdl_wait();
}

// The units that were cut: one block per (unit, 128 outputs of it), or, where
// there are more units than twice the shares, per (cut between two shares, 128
// outputs); eight threads share four dims of one row, each every eighth piece (a
// unit may have dozens), and add up in a fixed order.  38 pieces a unit (D 512):
// 6.4 us, the latency of a few dependent loads (with one thread for all of a unit's
// pieces, and look-ups by single threads, that call took 93 us in the place of 76).
constexpr int kMergeWays = 8;
template <int D, bool BY_CUT>
__global__ void __launch_bounds__(256)
paged_merge_kernel(const PagedReadArgs a, const int TG, const int n_groups, const int ctas, const long long* prefix,
                   const float* part_o, const float* part_ml) {
  pdl_launch();
  const int n_kv = a.L.n_kv, G = a.L.G;
  int u = blockIdx.x / n_kv, h = blockIdx.x - u * n_kv;
  PagedGroup g;
  if constexpr (!BY_CUT)                                  // (of the call's inputs alone)
    g = paged_group<true>(a.r, a.pg, a.L.window, TG, Pd<D>::KT, u);
  pdl_wait();
  const long long T = __ldg(prefix + n_groups) * n_kv;
  const PdShares shares = pd_shares<D>(T, ctas);
  const int cut = blockIdx.x + 1;
  if constexpr (BY_CUT) {
    if (T == 0 || cut >= shares.nc) return;
    const auto first_place = [=](int i) { return __ldg(prefix + i) * n_kv; };
    u = warp_search(n_groups, shares.begin(cut), first_place);
  }
  const long long pu = __ldg(prefix + u);
  const int width = (int)(__ldg(prefix + u + 1) - pu);
  if (width == 0) return;
  if constexpr (BY_CUT) h = (int)((shares.begin(cut) - pu * n_kv) / width);
  const long long x0 = pu * n_kv + (long long)h * width, x1 = x0 + width;
  const int c0 = shares.cta_of(x0 + 1), c1 = shares.cta_of(x1 - 1);
  if (c0 == c1) return;                                   // one CTA had it whole
  if constexpr (BY_CUT) {
    if (cut != c0 + 1) return;                            // not the unit's first cut
    g = paged_group<true>(a.r, a.pg, a.L.window, TG, Pd<D>::KT, u);
  }
  __shared__ float4 so[kMergeWays][32];
  __shared__ float2 sl[kMergeWays][32];
  const int way = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = blockIdx.y * 32 + lane, r = i / (D / 4), d = (i - r * (D / 4)) * 4;
  const bool valid = r < g.nt * G;
  const int first = 2 * c0 + (shares.begin(c0) >= x0 ? 0 : 1);
  // the way's pieces, four at a time, relative to the largest reference so far
  float M = -INFINITY, l = 0.f;
  float4 o = {0.f, 0.f, 0.f, 0.f};
  if (valid) {
    for (int c = c0 + way; c <= c1; c += 4 * kMergeWays) {
      float m[4], lp[4];
      float4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int at = c + k * kMergeWays;
        m[k] = -INFINITY;
        if (at <= c1) {
          const size_t slot = at == c0 ? first : 2 * at;
          m[k] = __ldg(part_ml + slot * 32 + r);
          lp[k] = __ldg(part_ml + slot * 32 + 16 + r);
          v[k] = __ldg(reinterpret_cast<const float4*>(part_o + (slot * 16 + r) * D + d));
        }
      }
      const float M1 = fmaxf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), M);
      const float f0 = M == -INFINITY ? 0.f : ex2(M - M1);
      M = M1;
      l *= f0;
      o.x *= f0;
      o.y *= f0;
      o.z *= f0;
      o.w *= f0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (c + k * kMergeWays <= c1) {
          const float f = m[k] == -INFINITY ? 0.f : ex2(m[k] - M);
          l = fmaf(lp[k], f, l);
          o.x = fmaf(v[k].x, f, o.x);
          o.y = fmaf(v[k].y, f, o.y);
          o.z = fmaf(v[k].z, f, o.z);
          o.w = fmaf(v[k].w, f, o.w);
        }
      }
    }
  }
  so[way][lane] = o;
  sl[way][lane] = make_float2(M, l);
  __syncthreads();
  if (way != 0 || !valid) return;
#pragma unroll
  for (int w = 1; w < kMergeWays; ++w) M = fmaxf(M, sl[w][lane].x);
  l = 0.f;
  o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kMergeWays; ++w) {
    const float2 ml = sl[w][lane];
    const float4 v = so[w][lane];
    const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
    l = fmaf(ml.y, f, l);
    o.x = fmaf(v.x, f, o.x);
    o.y = fmaf(v.y, f, o.y);
    o.z = fmaf(v.z, f, o.z);
    o.w = fmaf(v.w, f, o.w);
  }
  const float inv = 1.f / l;
  const size_t at = ((size_t)(g.row0 + r / G) * a.L.n_q + h * G + r % G) * D + d;
  const float w[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (a.out_f32) reinterpret_cast<float*>(a.out)[at + e] = w[e];
    else reinterpret_cast<uint16_t*>(a.out)[at + e] = f_to_bf16_rn(w[e]);
  }
}

int pd_kt(int D) { return D <= 128 ? Pd<128>::KT : Pd<256>::KT; }
int pd_cps(int D) { return D == 64 ? Pd<64>::CPS : D == 128 ? Pd<128>::CPS : D == 256 ? Pd<256>::CPS : Pd<512>::CPS; }

// rows of a group, groups and CTAs of a call
struct PdPlan { int TG, n_groups, max_tiles, ctas; };
PdPlan pd_plan(const LayerArgs& L, const PagedRows& r, int max_pos, int num_sms) {
  PdPlan p;
  p.TG = r.row_offsets ? std::max(1, 16 / L.G) : 1;
  p.n_groups = paged_groups(r, p.TG);
  // a group sees at most max_pos + 1 positions, or its window's
  long long keys = (long long)max_pos + 1;
  if (L.window > 0) keys = std::min<long long>(keys, (long long)L.window + p.TG - 1);
  // (a window's keys begin anywhere in a tile, a whole sequence's at 0)
  const int kt = pd_kt(L.D);
  p.max_tiles = (int)(keys == (long long)max_pos + 1 ? (keys + kt - 1) / kt : (keys + kt + 62) / kt + 1);
  const long long most = (long long)p.n_groups * L.n_kv * p.max_tiles;
  p.ctas = (int)std::max(1ll, std::min<long long>((long long)num_sms * pd_cps(L.D), most));
  return p;
}

// status (256 B), q16, prefix, part_o, part_ml
struct PdWs { size_t q16, prefix, part_o, part_ml, total; };
PdWs pd_ws(const LayerArgs& L, const PagedRows& r, const PdPlan& p) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  PdWs w;
  w.q16 = 256;
  w.prefix = up(w.q16 + (size_t)r.n_rows * L.n_q * L.D * 2);
  w.part_o = up(w.prefix + ((size_t)p.n_groups + 1) * 8);
  w.part_ml = up(w.part_o + (size_t)p.ctas * 2 * 16 * L.D * 4);
  w.total = up(w.part_ml + (size_t)p.ctas * 2 * 32 * 4);
  return w;
}

template <int D, bool E4M3>
cudaError_t launch_t(const PagedReadArgs& a, const RopeFreqs& f, int max_pos, void* ws, int num_sms, cudaStream_t st) {
  using S = Pd<D>;
  const PdPlan p = pd_plan(a.L, a.r, max_pos, num_sms);
  const PdWs w = pd_ws(a.L, a.r, p);
  uint8_t* b = static_cast<uint8_t*>(ws);
  uint32_t* status = reinterpret_cast<uint32_t*>(b);
  uint16_t* q16 = reinterpret_cast<uint16_t*>(b + w.q16);
  long long* prefix = reinterpret_cast<long long*>(b + w.prefix);
  float* part_o = reinterpret_cast<float*>(b + w.part_o);
  float* part_ml = reinterpret_cast<float*>(b + w.part_ml);
  cudaError_t e = launch_paged_prep<D>(a, f, p.TG, S::KT, p.n_groups, q16, prefix, PagedOrder{}, status, num_sms, st);
  if (e != cudaSuccess) return e;
  CUtensorMap tmk, tmv;
  if (!pages_map(&tmk, a.pg.k_codes, D, a.pg.P, (long long)a.pg.n_pages * a.L.n_kv) ||
      !pages_map(&tmv, a.pg.v_codes, D, a.pg.P, (long long)a.pg.n_pages * a.L.n_kv))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> allowed{0};
  e = allow_smem(paged_decode_kernel<D, E4M3>, S::BYTES, allowed);
  if (e != cudaSuccess) return e;
  if ((e = prof_before(st)) != cudaSuccess) return e;
  e = launch_pdl(paged_decode_kernel<D, E4M3>, dim3(p.ctas), dim3(kPdThreads), S::BYTES, st, a, tmk, tmv, p.TG, p.n_groups,
                 q16, prefix, part_o, part_ml, status);
  if (e != cudaSuccess) return e;
  if ((e = prof_after(st)) != cudaSuccess) return e;
  if (p.max_tiles < 2) return cudaSuccess;                // a single tile is never cut
  const long long units = (long long)p.n_groups * a.L.n_kv;
  // (finding a cut's unit takes two loads more, 256 rows of 2 kv heads 31.8 us a call for 28.7; but most of many
  // units are not cut: 480 windows of 4 rows, 1920 units, 76 for 128, 1000 rows 77 for 84)
  const bool by_cut = units > 2ll * p.ctas;
  const int slices = (p.TG * a.L.G * (D / 4) + 31) / 32;
  return launch_pdl(by_cut ? paged_merge_kernel<D, true> : paged_merge_kernel<D, false>,
                    dim3((unsigned)(by_cut ? std::max(1, p.ctas - 1) : units), slices), dim3(32 * kMergeWays), 0, st, a,
                    p.TG, p.n_groups, p.ctas, prefix, part_o, part_ml);
}

template <int D>
cudaError_t launch_d(const PagedReadArgs& a, const RopeFreqs& f, int max_pos, void* ws, int num_sms, cudaStream_t st) {
  return a.pg.e4m3 ? launch_t<D, true>(a, f, max_pos, ws, num_sms, st)
                   : launch_t<D, false>(a, f, max_pos, ws, num_sms, st);
}

}  // namespace

size_t paged_decode_ws_bytes(const LayerArgs& L, int n_seqs, int n_rows, int max_pos, int num_sms) {
  // (a call of single tokens has no row offsets; windows may have more groups)
  static const int32_t some = 0;
  const PagedRows one = {nullptr, nullptr, n_seqs, n_rows}, many = {&some, nullptr, n_seqs, n_rows};
  return std::max(pd_ws(L, one, pd_plan(L, one, max_pos, num_sms)).total,
                  pd_ws(L, many, pd_plan(L, many, max_pos, num_sms)).total);
}

cudaError_t launch_paged_decode(const PagedReadArgs& a, const RopeFreqs& f, int max_pos, void* ws, int num_sms,
                                cudaStream_t st) {
  switch (a.L.D) {
    case 64: return launch_d<64>(a, f, max_pos, ws, num_sms, st);
    case 128: return launch_d<128>(a, f, max_pos, ws, num_sms, st);
    case 256: return launch_d<256>(a, f, max_pos, ws, num_sms, st);
    default: return launch_d<512>(a, f, max_pos, ws, num_sms, st);
  }
}

}  // namespace kvq
