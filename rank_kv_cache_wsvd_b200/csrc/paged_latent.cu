// Decode attention over per-head low-rank latents (int8 / int4 codes with an
// fp16 scale per row) that lie in pages, for sm_100a: the operation of
// wsvd_decode_attention, reassociated the same way
//   q' = B_Kh . q,  s_l = s^K_l (code^K_l . q') * softmax_scale,
//   o = sum_l p_l s^V_l code^V_l,  out = (o / sum_l p_l) . B_Vh,
// with both products over the rows as integer matrix instructions on the codes
// as they are stored:
//   scores  m16n8k32: 16 rows x 32 codes against q' as a fixed-point number in
//           three signed base-256 digits (24 bits), a digit per column;
//   values  m16n8k32: 16 latent columns x 32 rows (ldmatrix transposes the
//           bytes) against w_l = p_l s^V_l, cut into three digits the same way
//           relative to the strip's largest weight (22 bits).
// Both sums are exact; int4 codes enter as 16 times their value, so that one
// mask or shift unpacks them.  Against one dp4a chain and one conversion per
// code (the contiguous decode) this takes most of the per-row work off the
// issue slots, which bound that kernel for short rows.
//
// Strips of rows are dealt evenly to warps.  Every warp is a worker of its own:
// its cp.async pipeline, its running maximum and sum, its partial results, and
// where it arrives last at a head, the join and the product with B_Vh.  Nothing
// waits for a CTA, so one warp's joins are hidden by the others' strips (a
// ragged int4 batch of 16 x 32 heads: 20.6 us; with the same pipelines joined per
// CTA 30.0).  A warp projects q' itself at the start of a segment while its first
// strips arrive: with a q' kernel ahead of this one the ragged batch took 20.6 us
// against 18.9, long caches 1 to 3 us less, and every call a second launch (2.5 us
// of host time).  Measured, 32 heads: 4 x 32768 rows 34.5 / 51.9 / 91.5 / 175 us for
// int8 r 16 / 32 / 64 / 128 (4.4 / 5.5 / 6.1 / 6.2 TB/s) and 42.1 / 56.1 / 100 for
// int4 r 32 / 64 / 128; one sequence of 1600 rows 9.3 us.  Bound by HBM from 64-byte
// rows on; shorter rows by the instructions a row costs whatever its length.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "paged.cuh"
#include "paged_rows.cuh"
#include "wsvd_internal.h"

using namespace wsvd;

namespace {

constexpr int kDigitMax = 127 * 65536 + 127 * 256 + 127;  // largest number of three signed digits
constexpr int kDigitBias = 0x808080;  // x + bias holds the digits + 128, a byte each

// BITS per code, RB bytes per row.
template <int BITS, int RB>
struct LatCfg {
  static constexpr int kR = RB * 8 / BITS;                // codes per row
  static constexpr int kTS = RB <= 32 ? 128 : (RB == 64 ? 64 : 32);  // rows per strip
  static constexpr int kBlocks = kTS / 32;                // of 32 rows, one per lane
  static constexpr int kGroups = kTS / 16;                // of 16 rows, within one page each
  static constexpr int kHalf = kTS * RB;
  static constexpr int kStage = 2 * kHalf + 2 * kTS * 2;  // K codes, V codes, K scales, V scales
  // Strips of 8 KB (4 KB for 16-byte rows): with strips of 64 rows instead of
  // 128, 4 x 32768 rows of r 32 took 53.0 us (int8) and 46.3 (int4) against 50.9
  // and 40.0.  A segment counts as two strips more (a ragged int4 batch of 16:
  // 21.1 / 20.7 / 21.5 us with 1 / 2 / 4).
  static constexpr int kWarps = 12, kStages = 2, kLead = 2;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kKS = kR >= 32 ? kR / 32 : 1;      // k steps of the score product
  static constexpr int kChunks = RB / 16;                 // 16-byte chunks of a row
  static constexpr int kDG = kR / 16;                     // groups of 16 latent columns
  static constexpr size_t kSmem = (size_t)kWarps * kStages * kStage;
};

struct LatDecodeArgs {
  PagedSeqs seqs;  // a unit: a head
  int H, Hd, page_shift, num_pages, max_pages, ctas;
  const int32_t* block_table;
  const uint8_t *lat_k, *lat_v;
  const __half *scale_k, *scale_v;
  const uint16_t* q;     // [B][H][Hd]
  int q_dtype;
  const __half *Bk, *Bv; // [H][r][Hd]
  float* out;
  float* partials;       // [kMaxDecodeCtas + B * H][r + 2]: o, then m, l
  int32_t* counters;     // [kMaxDecodeCtas], by the first worker of a cut head
  int32_t* err;
  float qscale;
};

__device__ __forceinline__ void imma32(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void imma16(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm("mma.sync.aligned.m16n8k16.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(b0));
}
// Two transposed 16 x 16 byte blocks: lanes 0-15 give the rows of the first,
// 16-31 of the second; the registers are the row operand of m16n8k32 for the
// blocks' columns (16) x rows (32).
__device__ __forceinline__ void ldsm_bytes_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ int warp_max_s32(int v) {
  int r;
  asm volatile("redux.sync.max.s32 %0, %1, 0xffffffff;" : "=r"(r) : "r"(v));
  return r;
}

// Order of floats as integers, and back (NaN above infinity).
__device__ __forceinline__ int float_key(float x) {
  const int b = __float_as_int(x);
  return b >= 0 ? b : b ^ 0x7fffffff;
}
__device__ __forceinline__ float key_float(int k) { return __int_as_float(k >= 0 ? k : k ^ 0x7fffffff); }

// Offset of 16-byte chunk c of row r: rows that share a bank column at one
// chunk index are turned apart.
template <int RB>
__device__ __forceinline__ uint32_t lat_off(int r, int c) {
  constexpr int kTurn = RB == 16 ? 0 : (RB == 32 ? 2 : (RB == 64 ? 1 : 0));
  return (uint32_t)(r * RB + ((c ^ ((r >> kTurn) & (RB / 16 - 1))) << 4));
}

// Four bytes, byte `k` of each of four words.
__device__ __forceinline__ uint32_t bytes_of(const uint4& w, uint32_t sel) {
  return __byte_perm(__byte_perm(w.x, w.y, sel), __byte_perm(w.z, w.w, sel), 0x5410);
}

// A warp's q' = bk . q, bk [R][Hd] fp16, Hd <= 64 N: eight lanes to a row, four
// rows at a time.  Returns the lane's largest |q'| as bits (a NaN above all).
template <int R, int N>
__device__ __forceinline__ int project_query(const uint16_t* q, int dtype, const __half* bk, int Hd, float* out,
                                               int lane) {
  const int sub = lane & 7, part = lane >> 3;
  float x[N][8];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int d = (i * 8 + sub) * 8;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (d < Hd) w = __ldg(reinterpret_cast<const uint4*>(q + d));
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = dtype == WSVD_DTYPE_BF16
                           ? make_float2(__uint_as_float(ws[k] << 16), __uint_as_float(ws[k] & 0xffff0000u))
                           : h2_pair(ws[k]);
      x[i][2 * k] = f.x;
      x[i][2 * k + 1] = f.y;
    }
  }
  int amax = 0;
  constexpr int kFly = R / 4 < 8 ? R / 4 : (N == 4 ? 4 : 8);  // turns whose loads are in flight together
#pragma unroll 1
  for (int j0 = 0; j0 < R; j0 += 4 * kFly) {
    uint4 w[kFly][N];
#pragma unroll
    for (int j = 0; j < kFly; ++j)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int d = (i * 8 + sub) * 8;
        w[j][i] = make_uint4(0, 0, 0, 0);
        if (d < Hd) w[j][i] = __ldg(reinterpret_cast<const uint4*>(bk + (size_t)(j0 + 4 * j + part) * Hd + d));
      }
#pragma unroll
    for (int j = 0; j < kFly; ++j) {
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t ws[4] = {w[j][i].x, w[j][i].y, w[j][i].z, w[j][i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = h2_pair(ws[k]);
          v = fmaf(f.x, x[i][2 * k], v);
          v = fmaf(f.y, x[i][2 * k + 1], v);
        }
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (sub == 0) out[j0 + 4 * j + part] = v;
      amax = max(amax, __float_as_int(fabsf(v)));
    }
  }
  return amax;
}

// A warp's out[0 .. 32 N) = (o . inv) . bv, bv [R][32 N] fp16; lane i columns N i ..
template <int R, int N>
__device__ __forceinline__ void up_project(const float* o, float inv, const __half* bv, float* out, int lane) {
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
  constexpr int kFly = N == 8 ? 8 : 16;  // rows whose loads are in flight together
#pragma unroll 1
  for (int j0 = 0; j0 < R; j0 += kFly) {
    __align__(16) __half x[kFly][N];
#pragma unroll
    for (int j = 0; j < kFly; ++j) {
      const __half* p = bv + (size_t)(j0 + j) * 32 * N + lane * N;
      if constexpr (N == 8) *reinterpret_cast<uint4*>(x[j]) = *reinterpret_cast<const uint4*>(p);
      else if constexpr (N == 4) *reinterpret_cast<uint2*>(x[j]) = *reinterpret_cast<const uint2*>(p);
      else if constexpr (N == 2) *reinterpret_cast<uint32_t*>(x[j]) = *reinterpret_cast<const uint32_t*>(p);
      else x[j][0] = *p;
    }
#pragma unroll
    for (int j = 0; j < kFly; ++j)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = fmaf(o[j0 + j], __half2float(x[j][i]), v[i]);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) out[lane * N + i] = v[i] * inv;
}

template <int BITS, int RB>
__global__ void __launch_bounds__(LatCfg<BITS, RB>::kThreads, 1) lat_decode_kernel(const LatDecodeArgs a) {
  using C = LatCfg<BITS, RB>;
  constexpr int TS = C::kTS, S = C::kStages, NW = C::kWarps, R = C::kR, KS = C::kKS, NBL = C::kBlocks, DG = C::kDG;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(16) float sm_q[NW][R];      // q', then the result
  __shared__ __align__(16) uint32_t sm_w[NW][TS];  // the strip's weights as digits
  __shared__ int sm_valid[NW][S];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c4 = lane & 3;
  const int H = a.H, Hd = a.Hd;
  const PagedSeqs& seqs = a.seqs;
  // Worker: one warp.  Few workers are spread over the SMs.
  const int me = warp * gridDim.x + blockIdx.x;
  griddep_wait();

  for (int b = blockIdx.x; b < seqs.B; b += gridDim.x)
    if (seqs.rows(b) == 0)
      for (int i = tid; i < H * Hd; i += C::kThreads) a.out[(size_t)b * H * Hd + i] = 0.f;
  Strips<TS> share;
  typename Strips<TS>::Segment seg;
  const auto plan = [&](int, int) {
    return typename Strips<TS>::Plan{me, min((int)gridDim.x * NW, kMaxDecodeCtas), 1, C::kLead};
  };
  if (!share.deal(seqs, plan, a.err, &seg)) return;

  // ---- the warp's copies: cursor `ld`; lane i holds the page of 16-row group i
  const uint32_t my_ring = smem_u32(ring) + (uint32_t)warp * S * C::kStage;
  auto ld = seg;
  int ls = ld.s;
  bool more = true;
  int pg = -1;
  const int page_mask = (1 << a.page_shift) - 1;
  auto settle = [&]() {  // the next strip of this warp, and its pages
    while (more && ls >= ld.e) {
      more = ld.next(seqs);
      ls = ld.s;
    }
    if (more) {
      const int l = ls * TS + lane % C::kGroups * 16;
      pg = lane < C::kGroups && l < ld.n ? __ldg(a.block_table + (size_t)ld.b * a.max_pages + (l >> a.page_shift)) : -1;
    }
  };
  auto issue = [&](int stage) {
    if (more) {
      const uint32_t dst = my_ring + (uint32_t)stage * C::kStage;
      const int l0 = ls * TS;
      const bool in = pg >= 0 && pg < a.num_pages;
      if (lane < C::kGroups && !in && l0 + lane * 16 < ld.n) set_err(a.err, WSVD_DEVERR_PAGE_RANGE);
      const int valid = (int)(__ballot_sync(0xffffffffu, in) & ((1u << C::kGroups) - 1));
      // Codes: whole groups of 16 rows (rows past the length lie in the same
      // page; they are masked later).
      constexpr int kRowsPer = 512 / RB;  // rows of one copy instruction
#pragma unroll
      for (int j = 0; j < TS / kRowsPer; ++j) {
        const int r = j * kRowsPer + lane / C::kChunks, ch = lane % C::kChunks, grp = r / 16;
        const int p = __shfl_sync(0xffffffffu, pg, grp);
        const bool there = (valid >> grp) & 1;
        const size_t row = (((size_t)(there ? p : 0) * H + ld.u) << a.page_shift) + ((l0 + r) & page_mask);
        const size_t src = there ? row * RB + ch * 16 : 0;
        const uint32_t off = lat_off<RB>(r, ch);
        cp_async16(dst + off, a.lat_k + src, there ? 16u : 0u);
        cp_async16(dst + C::kHalf + off, a.lat_v + src, there ? 16u : 0u);
      }
      {  // scales: 8 rows a copy, K then V
        constexpr int kPer = TS / 8;
        const int i = lane % kPer, grp = i / 2;
        const int p = __shfl_sync(0xffffffffu, pg, grp);
        if (lane < 2 * kPer) {
          const bool there = (valid >> grp) & 1;
          const size_t row = (((size_t)(there ? p : 0) * H + ld.u) << a.page_shift) + ((l0 + i * 8) & page_mask);
          cp_async16(dst + 2 * C::kHalf + lane * 16, (lane < kPer ? a.scale_k : a.scale_v) + (there ? row : 0),
                     there ? 16u : 0u);
        }
      }
      if (lane == 0) sm_valid[warp][stage] = valid;
      ++ls;
      settle();
    }
    cp_commit();
  };
  settle();
  for (int i = 0; i < S - 1; ++i) issue(i);
  int stage = 0;

  // A lane's row within a block of 32, in the score product's order of rows.
  const int tok = ((c4 >> 1) << 4) | ((c4 & 1) << 3) | g;
  // Weight digits: column g takes byte 2 - g (the high digit first); columns
  // from 3 on are zero.
  const uint32_t wsel = g < 3 ? (uint32_t)((2 - g) | ((6 - g) << 4)) : 0u, wmask = g < 3 ? 0xffffffffu : 0u;

  for (bool go = true; go; go = seg.next(seqs)) {
    if (seg.s == seg.e) continue;
    const int h = seg.u;
    const size_t bh = (size_t)seg.b * H + h;

    // ---- q' as signed digits in the score product's column operand: even
    // columns the high digit, odd ones the middle; a second operand the low.
    uint32_t qhm[KS][2], qlo[KS][2];
    float qstep;
    {
      const uint16_t* q = a.q + bh * Hd;
      const __half* bk = a.Bk + (size_t)h * R * Hd;
      const int most = Hd == 128  ? project_query<R, 2>(q, a.q_dtype, bk, Hd, sm_q[warp], lane)
                       : Hd == 256 ? project_query<R, 4>(q, a.q_dtype, bk, Hd, sm_q[warp], lane)
                                   : project_query<R, 1>(q, a.q_dtype, bk, Hd, sm_q[warp], lane);
      const float amax = __int_as_float(warp_max_s32(most));
      __syncwarp();
      const float inv = amax > 0.f ? (float)kDigitMax / amax : 0.f;
      qstep = amax / (float)kDigitMax * a.qscale * (BITS == 4 ? 0.0625f : 1.f);
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t hm = 0, lo = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = BITS == 8 ? k * 32 + x * 16 + 4 * c4 + i : k * 32 + 8 * c4 + 2 * i + x;
            int v = 0;
            if (R >= 32 || x == 0) v = max(-kDigitMax, min(kDigitMax, __float2int_rn(sm_q[warp][e] * inv)));
            const uint32_t y = (uint32_t)(v + kDigitBias);
            hm |= ((y >> (g & 1 ? 8 : 16)) & 0xffu) << (8 * i);
            lo |= (y & 0xffu) << (8 * i);
          }
          qhm[k][x] = hm ^ 0x80808080u;
          qlo[k][x] = lo ^ 0x80808080u;
        }
    }

    float m = kNegInf, l = 0.f, o[DG][4];
#pragma unroll
    for (int d = 0; d < DG; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;

    for (int s = seg.s; s < seg.e; ++s) {
      cp_wait<S - 2>();
      __syncwarp();
      issue(stage == 0 ? S - 1 : stage - 1);
      const uint32_t kb = my_ring + (uint32_t)stage * C::kStage, vb = kb + C::kHalf, sb = vb + C::kHalf;
      const int valid = sm_valid[warp][stage];
      const bool masked = s * TS > seg.n - TS || valid != (1 << C::kGroups) - 1;

      // ---- scores: lane `lane` ends with row tok of every block
      float sc[NBL];
#pragma unroll
      for (int blk = 0; blk < NBL; ++blk) {
        int hm[2][4] = {}, lo[2][4] = {};
        if constexpr (RB == 16) {  // 32 rows of one chunk in one load
          uint32_t f[4];
          ldsm4(f, kb + lat_off<RB>(blk * 32 + lane, 0));
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if constexpr (BITS == 8) {
              imma16(hm[t], f[2 * t], f[2 * t + 1], qhm[0][0]);
              imma16(lo[t], f[2 * t], f[2 * t + 1], qlo[0][0]);
            } else {
              const uint32_t e0 = (f[2 * t] << 4) & 0xf0f0f0f0u, e1 = (f[2 * t + 1] << 4) & 0xf0f0f0f0u;
              const uint32_t d0 = f[2 * t] & 0xf0f0f0f0u, d1 = f[2 * t + 1] & 0xf0f0f0f0u;
              imma32(hm[t], e0, e1, d0, d1, qhm[0][0], qhm[0][1]);
              imma32(lo[t], e0, e1, d0, d1, qlo[0][0], qlo[0][1]);
            }
          }
        } else {
#pragma unroll
          for (int cp = 0; cp < C::kChunks / 2; ++cp)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              uint32_t f[4];
              ldsm4(f, kb + lat_off<RB>(blk * 32 + t * 16 + (lane & 15), 2 * cp + (lane >> 4)));
              if constexpr (BITS == 8) {
                imma32(hm[t], f[0], f[1], f[2], f[3], qhm[cp][0], qhm[cp][1]);
                imma32(lo[t], f[0], f[1], f[2], f[3], qlo[cp][0], qlo[cp][1]);
              } else {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  const uint32_t e0 = (f[2 * x] << 4) & 0xf0f0f0f0u, e1 = (f[2 * x + 1] << 4) & 0xf0f0f0f0u;
                  const uint32_t d0 = f[2 * x] & 0xf0f0f0f0u, d1 = f[2 * x + 1] & 0xf0f0f0f0u;
                  imma32(hm[t], e0, e1, d0, d1, qhm[2 * cp + x][0], qhm[2 * cp + x][1]);
                  imma32(lo[t], e0, e1, d0, d1, qlo[2 * cp + x][0], qlo[2 * cp + x][1]);
                }
              }
            }
        }
        const bool t1 = c4 & 2, r1 = c4 & 1;
        const int ih = t1 ? (r1 ? hm[1][2] : hm[1][0]) : (r1 ? hm[0][2] : hm[0][0]);
        const int im = t1 ? (r1 ? hm[1][3] : hm[1][1]) : (r1 ? hm[0][3] : hm[0][1]);
        const int il = t1 ? (r1 ? lo[1][2] : lo[1][0]) : (r1 ? lo[0][2] : lo[0][0]);
        const float dot = fmaf((float)ih, 65536.f, fmaf((float)im, 256.f, (float)il));
        sc[blk] = dot * (lds_half_as_float(sb + 2u * (blk * 32 + tok)) * qstep);
        if (masked) {
          const int r = blk * 32 + tok;
          if (s * TS + r >= seg.n || !((valid >> (r / 16)) & 1)) sc[blk] = kNegInf;
        }
      }

      // ---- running maximum, weights, and their digits
      int top = float_key(sc[0]);
#pragma unroll
      for (int blk = 1; blk < NBL; ++blk) top = max(top, float_key(sc[blk]));
      const float mn = fmaxf(m, key_float(warp_max_s32(top)));
      const float ref = mn == kNegInf ? 0.f : mn;
      const float alpha = ex2(m - ref);
      m = mn;
      l *= alpha;
      float wt[NBL], big = 0.f;
#pragma unroll
      for (int blk = 0; blk < NBL; ++blk) {
        const float p = ex2(sc[blk] - ref);
        l += p;
        // a row that is masked weighs nothing whatever its scale holds
        const float w = p * lds_half_as_float(sb + (uint32_t)TS * 2u + 2u * (blk * 32 + tok));
        wt[blk] = p > 0.f ? w : 0.f;
        big = __int_as_float(max(__float_as_int(big), __float_as_int(fabsf(wt[blk]))));
      }
      // Power-of-two scale that brings the largest weight to [2^21, 2^22).
      const int bits = warp_max_s32(__float_as_int(big)), ex = max(22, bits >> 23);
      const float up = __int_as_float((275 - ex) << 23);
      // step; an infinite or NaN weight makes the result NaN
      const float step = bits >= 0x7f800000 ? __int_as_float(0x7fffffff)
                                            : __int_as_float((ex - 21) << 23) * (BITS == 4 ? 0.0625f : 1.f);
#pragma unroll
      for (int blk = 0; blk < NBL; ++blk)
        sm_w[warp][blk * 32 + tok] = (uint32_t)(__float2int_rn(wt[blk] * up) + kDigitBias);
      __syncwarp();

      // ---- values
      int acc[DG][4];
#pragma unroll
      for (int d = 0; d < DG; ++d) acc[d][0] = acc[d][1] = acc[d][2] = acc[d][3] = 0;
#pragma unroll
      for (int blk = 0; blk < NBL; ++blk) {
        const uint4 w0 = *reinterpret_cast<const uint4*>(&sm_w[warp][blk * 32 + 4 * c4]);
        const uint4 w1 = *reinterpret_cast<const uint4*>(&sm_w[warp][blk * 32 + 16 + 4 * c4]);
        const uint32_t b0 = (bytes_of(w0, wsel) ^ 0x80808080u) & wmask, b1 = (bytes_of(w1, wsel) ^ 0x80808080u) & wmask;
#pragma unroll
        for (int ch = 0; ch < C::kChunks; ++ch) {
          uint32_t f[4];
          ldsm_bytes_t(f, vb + lat_off<RB>(blk * 32 + lane, ch));
          if constexpr (BITS == 8) {
            imma32(acc[ch], f[0], f[1], f[2], f[3], b0, b1);
          } else {
            imma32(acc[2 * ch], (f[0] << 4) & 0xf0f0f0f0u, (f[1] << 4) & 0xf0f0f0f0u, (f[2] << 4) & 0xf0f0f0f0u,
                   (f[3] << 4) & 0xf0f0f0f0u, b0, b1);
            imma32(acc[2 * ch + 1], f[0] & 0xf0f0f0f0u, f[1] & 0xf0f0f0f0u, f[2] & 0xf0f0f0f0u, f[3] & 0xf0f0f0f0u, b0,
                   b1);
          }
        }
      }
#pragma unroll
      for (int d = 0; d < DG; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[d][i] = fmaf((float)acc[d][i], step, o[d][i] * alpha);
      __syncwarp();  // every lane has read this stage and the weights
      stage = stage == S - 1 ? 0 : stage + 1;
    }

    // ---- the segment's result: digits joined (lanes c4 = 0 hold high and
    // middle, 1 the low), lane j the latent columns j, j + 32, ...
#pragma unroll
    for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    __syncwarp();
#pragma unroll
    for (int d = 0; d < DG; ++d)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float low = __shfl_down_sync(0xffffffffu, o[d][2 * half], 1);
        const float v = fmaf(o[d][2 * half], 65536.f, fmaf(o[d][2 * half + 1], 256.f, low));
        // latent column of operand row g + 8 half: int4 groups hold the even and the odd codes of a chunk
        const int row = g + 8 * half;
        const int j = BITS == 8 ? d * 16 + row : (d >> 1) * 32 + 2 * row + (d & 1);
        if (c4 == 0) sm_q[warp][j] = v;
      }
    __syncwarp();
    constexpr int NJ = (R + 31) / 32, kSlot = R + 2;
    if (seg.s != 0 || seg.e != seg.strips()) {
      // Part of a unit: slot me + bh is this warp's alone, as workers and units
      // both only rise along the shares.  The last to arrive joins the parts in
      // the order of the workers, so the result does not depend on who that is.
      int wf, np;
      share.holders(seg, &wf, &np);
      float* part = a.partials + ((size_t)me + bh) * kSlot;
#pragma unroll
      for (int j0 = 0; j0 < R; j0 += 32)
        if (j0 + lane < R) __stcg(part + j0 + lane, sm_q[warp][j0 + lane]);
      if (lane == 0) __stcg(reinterpret_cast<float2*>(part + R), make_float2(m, l));
      __threadfence();
      __syncwarp();
      int last = 0;
      if (lane == 0) last = atom_add_acq_rel_gpu(a.counters + wf, 1) == np - 1;
      if (!__shfl_sync(0xffffffffu, last, 0)) continue;
      __threadfence();
      const float* from = a.partials + ((size_t)wf + bh) * kSlot;
      constexpr int kJoin = 8;  // partials whose loads are in flight together
      float sum[NJ];
#pragma unroll
      for (int k = 0; k < NJ; ++k) sum[k] = 0.f;
      m = kNegInf;
      l = 0.f;
      for (int i0 = 0; i0 < np; i0 += kJoin) {
        float2 ml[kJoin];
        float x[kJoin][NJ], mx = m;
#pragma unroll
        for (int i = 0; i < kJoin; ++i) {
          const float* p = from + (size_t)(i0 + i) * kSlot;
          const bool in = i0 + i < np;
          ml[i] = in ? __ldcg(reinterpret_cast<const float2*>(p + R)) : make_float2(kNegInf, 0.f);
#pragma unroll
          for (int k = 0; k < NJ; ++k) x[i][k] = in && k * 32 + lane < R ? __ldcg(p + k * 32 + lane) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kJoin; ++i) mx = fmaxf(mx, ml[i].x);
        const float ref = mx == kNegInf ? 0.f : mx, f0 = ex2(m - ref);
        l *= f0;
#pragma unroll
        for (int k = 0; k < NJ; ++k) sum[k] *= f0;
#pragma unroll
        for (int i = 0; i < kJoin; ++i) {
          const float f = ex2(ml[i].x - ref);
          l = fmaf(ml[i].y, f, l);
#pragma unroll
          for (int k = 0; k < NJ; ++k) sum[k] = fmaf(x[i][k], f, sum[k]);
        }
        m = mx;
      }
      if (lane == 0) st_relaxed_gpu(a.counters + wf, 0);
#pragma unroll
      for (int k = 0; k < NJ; ++k)
        if (k * 32 + lane < R) sm_q[warp][k * 32 + lane] = sum[k];
      __syncwarp();
    }

    // ---- out = (o / L) . B_Vh
    const float inv = 1.f / l;
    const __half* bv = a.Bv + (size_t)h * R * Hd;
    float* out = a.out + bh * Hd;
    if (Hd == 128) up_project<R, 4>(sm_q[warp], inv, bv, out, lane);
    else if (Hd == 64) up_project<R, 2>(sm_q[warp], inv, bv, out, lane);
    else if (Hd == 32) up_project<R, 1>(sm_q[warp], inv, bv, out, lane);
    else up_project<R, 8>(sm_q[warp], inv, bv, out, lane);
    __syncwarp();
  }
  cp_wait<0>();
}

struct LatKernel {
  void (*fn)(const LatDecodeArgs);
  size_t smem;
  int threads;
};
template <int BITS, int RB>
LatKernel lat_kernel() {
  using C = LatCfg<BITS, RB>;
  return LatKernel{&lat_decode_kernel<BITS, RB>, C::kSmem, C::kThreads};
}
bool pick_lat(int bits, int rowbytes, LatKernel* k) {
  if (bits == 8) {
    switch (rowbytes) {
      case 16: *k = lat_kernel<8, 16>(); return true;
      case 32: *k = lat_kernel<8, 32>(); return true;
      case 64: *k = lat_kernel<8, 64>(); return true;
      case 128: *k = lat_kernel<8, 128>(); return true;
    }
  } else {
    switch (rowbytes) {
      case 16: *k = lat_kernel<4, 16>(); return true;
      case 32: *k = lat_kernel<4, 32>(); return true;
      case 64: *k = lat_kernel<4, 64>(); return true;
    }
  }
  return false;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Bytes in front of the prefill's scratch in the paged append's workspace: the
// one-token append's completion counter, which every call leaves zero.
constexpr size_t kPagedCounterBytes = 256;

// Whether one token of each of B sequences takes the append's GEMV (fp32 FMAs, up
// to four tokens per pass over the weights) rather than the tensor-core GEMM.
// Measured, GEMV / GEMM in us, 32 heads, E 4096: r 32, 1 / 2 / 4 / 5 sequences 6.9 /
// 7.6 / 12.3 / 17.1 against 15.5; r 64, 1 / 3 / 4 9.4 / 16.0 / 22.5 against 17.4; r 128, 1
// / 2 / 3 14.5 / 19.6 / 34.2 against 21.8; 16 sequences of r 32 78 against 16.0.
inline bool prefers_gemv(int B, int r) { return B <= 4 && B * r <= 192; }

}  // namespace

extern "C" int wsvd_decode_attention_paged(int B, int H, int Hd, int r, int bits, int page_size, int num_pages,
                                           int max_pages, const int32_t* seq_lens, const int32_t* block_table,
                                           const void* q, int q_dtype, const uint8_t* lat_k, const uint8_t* lat_v,
                                           const void* scale_k, const void* scale_v, const void* B_k, const void* B_v,
                                           float softmax_scale, float* out, void* workspace, size_t workspace_bytes,
                                           int32_t* err, void* stream) {
  if (B < 0 || H < 1 || num_pages < 0 || max_pages < 0) return WSVD_ERR_INVALID_ARG;
  if (B == 0) return WSVD_OK;
  if (bits != 8 && bits != 4) return WSVD_ERR_INVALID_ARG;
  if (r < 1 || (r * bits) % 8) return WSVD_ERR_INVALID_ARG;
  if (q_dtype != WSVD_DTYPE_FP16 && q_dtype != WSVD_DTYPE_BF16) return WSVD_ERR_INVALID_ARG;
  if (B > 4096 || H > (1 << 20) || (Hd != 32 && Hd != 64 && Hd != 128 && Hd != 256)) return WSVD_ERR_UNSUPPORTED;
  const int shift = page_shift_of(page_size);
  LatKernel kern;
  if (shift < 0 || !pick_lat(bits, r * bits / 8, &kern)) return WSVD_ERR_UNSUPPORTED;
  if ((long long)max_pages << shift > 0x7fffffffLL || (long long)B * H > 0x7fffffffLL) return WSVD_ERR_UNSUPPORTED;
  if (!seq_lens || !block_table || !q || !lat_k || !lat_v || !scale_k || !scale_v || !B_k || !B_v || !out || !workspace)
    return WSVD_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(lat_k) || !aligned16(lat_v) || !aligned16(scale_k) || !aligned16(scale_v) ||
      !aligned16(B_k) || !aligned16(B_v) || !aligned16(out) || !aligned16(workspace))
    return WSVD_ERR_INVALID_ARG;
  // The workspace of wsvd_decode_attention: the counters where that call has
  // them, so that calls of both, of any sizes, may use it in turn.
  const size_t need = wsvd_decode_workspace_size(B, H, r), heads = (size_t)B * H, up = (size_t)H * r * Hd * 2;
  size_t codes, scales;
  if (!pool_bytes(num_pages, H, shift, (size_t)r * bits / 8, &codes) || !pool_bytes(num_pages, H, shift, 2, &scales))
    return WSVD_ERR_UNSUPPORTED;
  const Span read[] = {{seq_lens, (size_t)B * 4}, {block_table, (size_t)B * max_pages * 4}, {q, heads * Hd * 2},
                       {lat_k, codes}, {lat_v, codes}, {scale_k, scales}, {scale_v, scales}, {B_k, up}, {B_v, up}};
  const Span written[] = {{out, heads * Hd * 4}, {workspace, need}, {err, 4}};
  if (clash(written, read)) return WSVD_ERR_INVALID_ARG;
  if (workspace_bytes < need) return WSVD_ERR_WORKSPACE_TOO_SMALL;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  LatDecodeArgs a{};
  a.seqs = PagedSeqs{B, H, max_pages << shift, seq_lens};
  a.H = H; a.Hd = Hd; a.page_shift = shift; a.num_pages = num_pages; a.max_pages = max_pages;
  a.block_table = block_table;
  a.lat_k = lat_k; a.lat_v = lat_v;
  a.scale_k = static_cast<const __half*>(scale_k); a.scale_v = static_cast<const __half*>(scale_v);
  a.Bv = static_cast<const __half*>(B_v);
  a.out = out;
  a.counters = reinterpret_cast<int32_t*>(w);
  a.partials = reinterpret_cast<float*>(w + kSplitCounterBytes);
  a.q = static_cast<const uint16_t*>(q);
  a.q_dtype = q_dtype;
  a.Bk = static_cast<const __half*>(B_k);
  a.err = err;
  a.qscale = (softmax_scale != 0.f ? softmax_scale : (float)(1.0 / sqrt((double)Hd))) * kLog2e;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  (void)cudaGetLastError();
  if (paged_resident_ctas(reinterpret_cast<const void*>(kern.fn), kern.threads, kern.smem, &a.ctas) != cudaSuccess) return WSVD_ERR_CUDA;
  return launch_behind(kern.fn, dim3((unsigned)a.ctas), kern.threads, kern.smem, s, a) == cudaSuccess ? WSVD_OK
                                                                                                       : WSVD_ERR_CUDA;
}

extern "C" size_t wsvd_latent_append_paged_workspace_size(int B, int T, int E) {
  return kPagedCounterBytes + (B < 1 || T < 1 || E < 1 ? 0 : paged_block_scratch(B, T, E));
}

extern "C" int wsvd_latent_append_paged(int B, int T, int H, int E, int r, int bits, int page_size, int num_pages,
                                        int max_pages, int hadamard_block, const void* x, int x_dtype, const void* A_k,
                                        const void* A_v, const int32_t* seq_lens, int32_t* seq_lens_out,
                                        const int32_t* block_table, uint8_t* lat_k, uint8_t* lat_v, void* scale_k,
                                        void* scale_v, void* workspace, size_t workspace_bytes, int32_t* err,
                                        void* stream) {
  if (B < 0 || T < 0 || H < 1 || E < 1 || r < 1 || num_pages < 0 || max_pages < 0) return WSVD_ERR_INVALID_ARG;
  if (B == 0) return WSVD_OK;
  if (bits != 8 && bits != 4) return WSVD_ERR_INVALID_ARG;
  if (x_dtype != WSVD_DTYPE_FP16 && x_dtype != WSVD_DTYPE_BF16) return WSVD_ERR_INVALID_ARG;
  if (hadamard_block < 1 || hadamard_block > 1024 || (hadamard_block & (hadamard_block - 1)) || E % hadamard_block)
    return WSVD_ERR_INVALID_ARG;
  const int shift = page_shift_of(page_size);
  LatKernel reader;  // rows that the paged decode can read
  if (shift < 0 || (r * bits) % 8 || !pick_lat(bits, r * bits / 8, &reader)) return WSVD_ERR_UNSUPPORTED;
  if ((long long)max_pages << shift > 0x7fffffffLL) return WSVD_ERR_UNSUPPORTED;
  if (!seq_lens || !seq_lens_out || !block_table || !workspace) return WSVD_ERR_INVALID_ARG;
  if (T > 0 && (!x || !A_k || !A_v || !lat_k || !lat_v || !scale_k || !scale_v)) return WSVD_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(A_k) || !aligned16(A_v) || !aligned16(lat_k) || !aligned16(lat_v) ||
      !aligned16(scale_k) || !aligned16(scale_v) || !aligned16(workspace))
    return WSVD_ERR_INVALID_ARG;
  const int ranks = append_cluster_size(E, hadamard_block);
  const bool gemm = paged_block_takes(B, T, H, E, r);
  const bool gemv = T == 1 && B <= 16 && E <= 65536 && 2LL * H <= 65535 && ranks > 0 &&
                    append_smem_bytes(B, E, r, ranks) <= 200 * 1024;  // K and V of a head are grid rows
  if (T > 0 && !gemm && !gemv) return WSVD_ERR_UNSUPPORTED;
  const size_t need = wsvd_latent_append_paged_workspace_size(B, T, E), lb = (size_t)B * 4;
  const size_t xb = (size_t)B * T * E * 2, down = (size_t)H * E * r * 2;
  size_t codes, scales;
  if (!pool_bytes(num_pages, H, shift, (size_t)r * bits / 8, &codes) || !pool_bytes(num_pages, H, shift, 2, &scales))
    return WSVD_ERR_UNSUPPORTED;
  const Span read[] = {{seq_lens_out == seq_lens ? nullptr : seq_lens, lb}, {block_table, (size_t)B * max_pages * 4},
                       {x, xb}, {A_k, down}, {A_v, down}};
  const Span written[] = {{seq_lens_out, lb}, {lat_k, codes}, {lat_v, codes}, {scale_k, scales}, {scale_v, scales},
                          {workspace, need}, {err, 4}};
  if (clash(written, read)) return WSVD_ERR_INVALID_ARG;
  if (workspace_bytes < need) return WSVD_ERR_WORKSPACE_TOO_SMALL;

  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) {
    if (seq_lens_out != seq_lens &&
        cudaMemcpyAsync(seq_lens_out, seq_lens, (size_t)B * 4, cudaMemcpyDeviceToDevice, s) != cudaSuccess)
      return WSVD_ERR_CUDA;
    return WSVD_OK;
  }
  const PagedRows place{block_table, max_pages, shift, num_pages, seq_lens_out};
  AppendArgs a{};
  a.B = B; a.H = H; a.E = E; a.r = r; a.bits = bits; a.L_cap = max_pages << shift; a.blk = hadamard_block;
  a.cluster = ranks;
  a.hnorm = (float)(1.0 / sqrt((double)hadamard_block));
  a.x = x; a.x_dtype = x_dtype; a.Ak = A_k; a.Av = A_v;
  a.seq_lens = const_cast<int32_t*>(seq_lens);  // read only: PagedRows writes seq_lens_out
  a.lat_k = lat_k; a.lat_v = lat_v;
  a.scale_k = static_cast<__half*>(scale_k); a.scale_v = static_cast<__half*>(scale_v);
  a.counter = static_cast<int32_t*>(workspace); a.err = err;
  (void)cudaGetLastError();
  // One token of few sequences, and of up to 16 where E does not suit the GEMM:
  // the append's GEMV, bound by reading A once; all else the tensor-core GEMM.
  const cudaError_t e = gemv && (prefers_gemv(B, r) || !gemm)
                            ? launch_append_paged(a, place, s)
                            : launch_paged_block(a, T, place, static_cast<uint8_t*>(workspace) + kPagedCounterBytes, s);
  return e == cudaSuccess ? WSVD_OK : WSVD_ERR_CUDA;
}
