// kvq_paged_append and kvq_paged_gather: new K/V rows into 8-bit pages, and
// pages read back as bf16 rows.
//
// Append.  The rows are prepped as by kv_quant_append (k: RMSNorm, bf16, RoPE,
// bf16; v: un-scaled RMSNorm, bf16).  A page has one scale per kv head for K
// and one for V, so what one block does is what one page takes: block (unit,
// head group, K or V) preps every new row of the page for its heads, keeps the
// bf16 rows in shared memory, takes their largest magnitude per head, and with
//   s_new = largest / 127 (int8) or / 448 (e4m3), 0 below 2^-40,
//   s     = max(s_new, s_old) if the page already holds rows, else s_new,
// writes code = round(x / s) for the new rows; where s grew, the rows that
// were there become round(code * s_old / s).  All in IEEE fp32 (products with
// the reciprocal, a little more and a little less, decide where they round to
// the same code, else a division).  Units: rows row_offsets[s] .. of sequence s
// touch at most floor(rows / P) + 2 pages, so unit u of sequence s with base(s) =
// floor(row_offsets[s] / P) + 2 s is its page number u - base(s); units past the
// sequence's last page leave at once.  One warp preps 256 / D rows at a time (one
// of 256 or 512), with the rotation angles of up to rb rows at a time computed
// once for all heads of the block.
//
// What bounds it: instructions, of the prep (two thirds) and the codes, not the
// few bytes per row.  The heads of a block share a row's angles; more heads a
// block mean fewer angles, fewer blocks and more shared memory.  Measured: 8008
// rows of 8 kv heads of 128, 50 us (33 MB in, 16 out; issue 71 %); 64 rows of 2
// heads of 256 in 64 sequences 8.4 us (latency).
//
// Gather.  A thread takes 16 codes of one row; 8008 rows of 8 kv heads of 128 in
// 13 us (16 MB in, 33 out).
#include <algorithm>

#include "kvq_paged.cuh"
#include "kvq_paged_prep.cuh"

namespace kvq {

namespace {

constexpr int kPaWarps = 8;
constexpr int kPaMaxHeads = 16;      // heads per block

// bytes of shared memory: bf16 rows of hb heads, then the K blocks' angles,
// frequencies and each warp's two rows
struct PaSmem { size_t cs, freq, nrm, total; };
__host__ __device__ inline PaSmem pa_smem(int D, int half, int hb, int cap, int rb) {
  PaSmem m;
  m.cs = ((size_t)hb * cap * D * 2 + 15) / 16 * 16;
  m.freq = m.cs + (size_t)rb * half * 16;
  m.nrm = m.freq + 16 * (size_t)((3 * half + 3) / 4);
  m.total = m.nrm + (size_t)kPaWarps * 2 * (D < 256 ? 256 : D) * 2;
  return m;
}

// Codes of E bf16 values (pairs in src) at scale s.  x times the rounded
// reciprocal is within 2^-23 of x / s, and fl32(x / s) within 2^-24: where both
// ends of 2^-21 around the product give one code, that is round(fl32(x / s)).
template <int E, bool E4M3>
__device__ __forceinline__ void encode_row(const uint32_t (&src)[E / 2], float s, uint32_t (&o)[E / 4]) {
  constexpr float kRound = 12582912.f;                    // 1.5 * 2^23: the sum's last bit is 1
#pragma unroll
  for (int i = 0; i < E / 4; ++i) o[i] = 0u;
  if (!(s > 0.f)) return;
  const float rcp = __frcp_rn(s), up = rcp * (1.f + 4.76837158203125e-7f), dn = rcp * (1.f - 4.76837158203125e-7f);
  bool same = true;
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    const float x0 = bf16lo_to_f(src[i]), x1 = bf16hi_to_f(src[i]);
    uint32_t two;
    if constexpr (E4M3) {
      uint16_t a, b;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(a) : "f"(x1 * up), "f"(x0 * up));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(x1 * dn), "f"(x0 * dn));
      same &= a == b;
      two = a;
    } else {
      const uint32_t a0 = __float_as_uint(__fmaf_rn(x0, up, kRound)), a1 = __float_as_uint(__fmaf_rn(x1, up, kRound));
      same &= a0 == __float_as_uint(__fmaf_rn(x0, dn, kRound)) && a1 == __float_as_uint(__fmaf_rn(x1, dn, kRound));
      two = prmt(a0, a1, 0x4440u) & 0xFFFFu;              // (|x / s| < 127.5: no code leaves its byte)
    }
    o[i / 2] |= two << (16 * (i & 1));
  }
  if (same) return;
#pragma unroll
  for (int i = 0; i < E / 4; ++i) o[i] = 0u;
#pragma unroll
  for (int i = 0; i < E; ++i)
    o[i / 4] |= encode_q<E4M3>(__fdiv_rn((i & 1) ? bf16hi_to_f(src[i / 2]) : bf16lo_to_f(src[i / 2]), s)) << (8 * (i & 3));
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kPaWarps * 32)
paged_append_kernel(const PagedAppendArgs a, const RopeFreqs freqs, const int hb, const int cap, const int rb) {
  using PL = PrepLanes<D>;
  constexpr int E = PL::E, ROUND = kPaWarps * PL::ROWS;   // items of a round
  extern __shared__ __align__(16) uint8_t pa_buf[];
  __shared__ uint32_t amax[kPaMaxHeads];
  __shared__ float s_was[kPaMaxHeads], s_now[kPaMaxHeads];
  const int tid = threadIdx.x, sub = tid / PL::N, lane = tid & (PL::N - 1);   // (sub: the row's lanes in the block)
  const int kind = blockIdx.z;                            // 0: K, 1: V
  const int R = kind == 0 ? a.L.rope_dims : 0, half = R >> 1, n_kv = a.L.n_kv;
  const PaSmem m = pa_smem(D, a.L.rope_dims >> 1, hb, cap, rb);
  uint16_t* rows = reinterpret_cast<uint16_t*>(pa_buf);   // [hb][cap][D]
  const Angles ang = {reinterpret_cast<float2*>(pa_buf + m.cs), reinterpret_cast<float2*>(pa_buf + m.cs) + rb * half};
  float (*freq)[3] = reinterpret_cast<float (*)[3]>(pa_buf + m.freq);
  uint16_t* nr = reinterpret_cast<uint16_t*>(pa_buf + m.nrm) + sub * 2 * D;
  if (R > 0) stage_freqs(freqs.f, half, freq);
  pdl_wait();
  pdl_launch();

  // ---- the block's page: its sequence, positions and rows ----
  const int u = blockIdx.x, P = a.pg.P, sh = a.pg.p_shift;
  const int lo = warp_search(a.r.n_seqs, u, [&](int s) { return (__ldg(a.r.row_offsets + s) >> sh) + 2 * s; });
  const SeqRows sr = paged_seq_rows(a.r, lo);
  if (sr.rows <= 0 || sr.start < 0 || sr.off < 0 || sr.off + sr.rows > a.r.n_rows) return;
  const int page_i = (sr.start >> sh) + u - ((sr.off >> sh) + 2 * lo);
  const int limit = a.pg.limit;
  const int p_lo = max(sr.start, page_i << sh);
  const int p_hi = min(min(sr.start + sr.rows, limit), (page_i + 1) << sh);
  if (p_lo >= p_hi) return;
  const int page = paged_page(a.pg, sr.s, p_lo);
  if (page < 0) return;
  const int n = p_hi - p_lo, slot0 = p_lo & (P - 1), row0 = sr.off + (p_lo - sr.start);
  const int h0 = blockIdx.y * hb, nh = min(hb, n_kv - h0);
  if (n > cap) return;                                    // (cap >= the rows of any page)
  if (tid < nh) amax[tid] = 0u;

  float w[E];
#pragma unroll
  for (int i = 0; i < E; ++i) w[i] = kind == 0 ? bf16_to_f(__ldg(a.k_w + lane * E + i)) : 1.f;
  const uint16_t* raw = (kind == 0 || a.L.k_eq_v) ? a.k_raw : a.v_raw;

  const uint32_t inv = prep_inv(nh);
  const int sub0 = sub & ~(PL::ROWS - 1), in_warp = sub & (PL::ROWS - 1);
  // ---- prep, rb rows at a time ----
  for (int c0 = 0; c0 < n; c0 += rb) {
    const int cnt = min(rb, n - c0);
    if (R > 0) {
      __syncthreads();                                    // the frequencies; the last rows' angles are read
      for (int idx = tid; idx < cnt * half; idx += kPaWarps * 32) {
        const int r = idx / half, j = idx - r * half;
        put_angle<D>(ang, r, R, j, p_lo + c0 + r, freq[j]);
      }
    }
    __syncthreads();
    // (row, head) items, one round ahead (past the last: the last again)
    const int items = cnt * nh;
    uint32_t nx[E / 2] = {};
    const auto fetch = [&](int i) {
      const PrepItem it = prep_item(min(i, items - 1), nh, inv);
      load_pairs<E>(nx, raw + ((size_t)(row0 + c0 + it.r) * n_kv + h0 + it.h) * D + lane * E);
    };
    fetch(sub);
    for (int i0 = sub0; i0 < items; i0 += ROUND) {
      const PrepItem at = prep_item(min(i0 + in_warp, items - 1), nh, inv);
      const int r = at.r, hh = at.h;
      uint32_t x[E / 2], y[E / 2];
#pragma unroll
      for (int i = 0; i < E / 2; ++i) x[i] = nx[i];
      if (i0 + ROUND < items) fetch(i0 + ROUND + in_warp);
      prep_row<D>(x, w, a.L.eps, R, ang, r, nr, y);
      store_pairs<E>(rows + (hh * cap + c0 + r) * D + lane * E, y);
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < E / 2; ++i)
        top = fmaxf(top, fmaxf(fabsf(bf16lo_to_f(y[i])), fabsf(bf16hi_to_f(y[i]))));
#pragma unroll
      for (int k = PL::N / 2; k >= 1; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
      if (lane == 0) atomicMax(&amax[hh], __float_as_uint(top));   // (of magnitudes: ordered as their bits)
      if (a.prepped) {
        uint16_t* d = a.prepped + (((size_t)kind * a.r.n_rows + row0 + c0 + r) * n_kv + h0 + hh) * D + lane * E;
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
          d[2 * i] = (uint16_t)(y[i] & 0xFFFFu);
          d[2 * i + 1] = (uint16_t)(y[i] >> 16);
        }
      }
    }
  }
  __syncthreads();

  // ---- the page's scale per head ----
  if (tid < nh) {
    float* sp = (kind == 0 ? a.pg.k_scales : a.pg.v_scales) + (size_t)page * n_kv + h0 + tid;
    float s = __fdiv_rn(__uint_as_float(amax[tid]), E4M3 ? 448.f : 127.f);
    if (!(s >= kSmallestScale)) s = 0.f;
    float was = s;
    if (slot0 > 0) {
      was = *sp;
      s = fmaxf(s, was);
    }
    s_was[tid] = was;
    s_now[tid] = s;
    *sp = s;
  }
  __syncthreads();

  // ---- rows that were there move to a grown scale ----
  uint8_t* codes = (kind == 0 ? a.pg.k_codes : a.pg.v_codes) + (((size_t)page * n_kv + h0) << sh) * D;
  if (slot0 > 0) {
    for (int hh = 0; hh < nh; ++hh) {
      const float was = s_was[hh], now = s_now[hh];
      if (!(now > was)) continue;
      uint4* c = reinterpret_cast<uint4*>(codes + (((size_t)hh) << sh) * D);
      for (int i = tid; i < slot0 * (D / 16); i += kPaWarps * 32) {
        uint4 v = c[i];
        uint32_t* vw = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t o = 0;
#pragma unroll
          for (int b = 0; b < 4; ++b)
            o |= encode_q<E4M3>(__fdiv_rn(__fmul_rn(decode_byte<E4M3>((vw[k] >> (8 * b)) & 0xFFu), was), now)) << (8 * b);
          vw[k] = o;
        }
        c[i] = v;
      }
    }
  }

  // ---- the new rows' codes ----
  for (int i = sub; i < n * nh; i += ROUND) {
    const PrepItem at = prep_item(i, nh, inv);
    const int r = at.r, hh = at.h;
    uint32_t src[E / 2];
    load_pairs<E>(src, rows + (hh * cap + r) * D + lane * E);
    uint32_t o[E / 4];
    encode_row<E, E4M3>(src, s_now[hh], o);
    uint8_t* dst = codes + ((((size_t)hh) << sh) + slot0 + r) * D + lane * E;
    if constexpr (E == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(o[0], o[1]);
    if constexpr (E == 16) *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// One thread reads 16 codes of a row and writes them as bf16.
template <bool E4M3>
__global__ void __launch_bounds__(256)
paged_gather_kernel(const PagedGatherArgs a, const long long items) {
  pdl_wait();
  pdl_launch();
  const int kind = blockIdx.y, per = a.n_kv * (a.D / 16);
  const uint8_t* codes = kind == 0 ? a.pg.k_codes : a.pg.v_codes;
  const float* scales = kind == 0 ? a.pg.k_scales : a.pg.v_scales;
  uint16_t* out = kind == 0 ? a.k_rows : a.v_rows;
  const int limit = a.pg.limit;
  for (long long it = (long long)blockIdx.x * 256 + threadIdx.x; it < items; it += (long long)gridDim.x * 256) {
    const int row = (int)(it / per), in = (int)(it - (long long)row * per);
    const int h = in / (a.D / 16), d0 = (in - h * (a.D / 16)) * 16;
    const SeqRows sr = paged_seq_rows(a.r, paged_seq_of(a.r, row));
    if (row - sr.off >= sr.rows) continue;                // behind the last sequence
    const int p = sr.start + (row - sr.off);
    const int page = sr.start >= 0 && p >= 0 && p < limit ? paged_page(a.pg, sr.s, p) : -1;
    uint32_t o[8];
    if (page < 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = 0x7FC07FC0u;
    } else {
      const size_t ph = (size_t)page * a.n_kv + h;
      const float s = __ldg(scales + ph);
      const uint4 v = *reinterpret_cast<const uint4*>(codes + ((ph << a.pg.p_shift) + (p & (a.pg.P - 1))) * a.D + d0);
      const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float f[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) f[b] = __fmul_rn(decode_byte<E4M3>((vw[k] >> (8 * b)) & 0xFFu), s);
        o[2 * k] = (uint32_t)f_to_bf16_rn(f[0]) | ((uint32_t)f_to_bf16_rn(f[1]) << 16);
        o[2 * k + 1] = (uint32_t)f_to_bf16_rn(f[2]) | ((uint32_t)f_to_bf16_rn(f[3]) << 16);
      }
    }
    uint4* dst = reinterpret_cast<uint4*>(out + ((size_t)row * a.n_kv + h) * a.D + d0);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// a head's rows of the largest page, angles of 512 pairs, frequencies, the warps' rows
constexpr size_t kPaMostSmem = 128 * 512 * 2 + 512 * 16 + 256 * 12 + kPaWarps * 2 * 512 * 2 + 64;

template <int D, bool E4M3>
cudaError_t launch_append_t(const PagedAppendArgs& a, const RopeFreqs& f, int num_sms, cudaStream_t st) {
  const int P = a.pg.P, half = a.L.rope_dims / 2, n_kv = a.L.n_kv;
  const int cap = std::min(P, a.r.n_rows);
  const int rb = half > 0 ? std::max(1, std::min(8, 512 / half)) : 8;     // (16 and 1024: 61.6 us for 59.4)
  // the heads of a block share its angles; as many as 32 KB of rows hold, fewer
  // while there are less than four blocks per SM
  int hb = std::max(1, std::min({n_kv, kPaMaxHeads, 32768 / (cap * D * 2)}));
  const long long pages = (long long)a.r.n_rows / P + a.r.n_seqs;
  while (hb > 1 && pages * ((n_kv + hb - 1) / hb) * 2 < 4ll * num_sms) hb = (hb + 1) / 2;
  const size_t smem = pa_smem(D, half, hb, cap, rb).total;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(paged_append_kernel<D, E4M3>, (int)kPaMostSmem, allowed);
  if (e != cudaSuccess) return e;
  const long long units = (long long)(a.r.n_rows >> a.pg.p_shift) + 2ll * a.r.n_seqs;
  if (units > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_pdl(paged_append_kernel<D, E4M3>, dim3((unsigned)units, (n_kv + hb - 1) / hb, 2), dim3(kPaWarps * 32),
                    smem, st, a, f, hb, cap, rb);
}

template <int D>
cudaError_t launch_append_d(const PagedAppendArgs& a, const RopeFreqs& f, int num_sms, cudaStream_t st) {
  return a.pg.e4m3 ? launch_append_t<D, true>(a, f, num_sms, st) : launch_append_t<D, false>(a, f, num_sms, st);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, const RopeFreqs& f, int num_sms, cudaStream_t st) {
  switch (a.L.D) {
    case 64: return launch_append_d<64>(a, f, num_sms, st);
    case 128: return launch_append_d<128>(a, f, num_sms, st);
    case 256: return launch_append_d<256>(a, f, num_sms, st);
    default: return launch_append_d<512>(a, f, num_sms, st);
  }
}

cudaError_t launch_paged_gather(const PagedGatherArgs& a, int num_sms, cudaStream_t st) {
  const long long items = (long long)a.r.n_rows * a.n_kv * (a.D / 16);
  const unsigned blocks = (unsigned)std::min<long long>((items + 255) / 256, 8ll * num_sms);
  return a.pg.e4m3 ? launch_pdl(paged_gather_kernel<true>, dim3(blocks, 2), dim3(256), 0, st, a, items)
                   : launch_pdl(paged_gather_kernel<false>, dim3(blocks, 2), dim3(256), 0, st, a, items);
}

}  // namespace kvq
