// A block of new tokens into latent pages, for sm_100a: each token rotated with
// the block Hadamard S1, projected through A_Kh / A_Vh and quantised (the
// operation of wsvd_latent_prefill, rows placed through the page table).
//
//   1. block_rotate_kernel: one CTA a token: rotation in registers and lane
//      exchanges, an exact power-of-two scale that brings the largest value to
//      [2^14, 2^15), and the split of every value into fp16 hi + lo (22 bits);
//   2. block_gemm_kernel: [tokens x E] . [E x 2 H r] on the tcgen05 tensor cores
//      with the quantiser in its epilogue; the last CTA to finish advances the
//      lengths.
//
// A tile is TOK tokens x BN columns (whole heads of K or of V).  64 tokens: the hi rows
// and the lo rows stand one above the other in one 128-row operand, so one MMA makes
// both products.  128 tokens, where there are many: the products are made in turn, lo
// then hi, into one accumulator, over the same weights.  Warps of a tile of 128 columns
// (of 256: warps 0-7 sum, two threads a row, then the producer and the issuer):
//   warp 4     TMA producer: per 64-wide k-tile hi [TOK x 64], lo [TOK x 64] and
//              the weights [64 x BN], a ring of mbarrier stages;
//   warp 5     allocates tensor memory and issues four k16 MMAs per k-tile into a
//              fresh accumulator of NH;
//   warps 0-3  thread <-> operand row: adds every k-tile's sum to fp32 registers,
//              rounding to nearest (the tensor cores' own sums do not).
// Where there are few tiles a cluster of up to 8 CTAs splits E for one tile; the
// ranks' sums are read through the cluster's shared memory in rank order, each
// rank quantising its share of the tokens.  The k-loop is bound by the operand tiles'
// way from L2 (75 to 92 GB/s a SM whatever the tile).  32 heads of r 32, E 4096, both
// kernels: 576 tokens 31 us, of which 16.7 are 32 k-tiles a CTA (221 MB of tiles; the
// products alone, hi and lo, 11.7) and 14.4 do not grow with E (rotation, start, the
// clusters' join, quantiser); 4096 tokens 160 (1.0 GB; 83), 16 tokens 14.5 (11.6 at E 1024).
#include <cooperative_groups.h>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math.h>

#include <algorithm>
#include <map>
#include <mutex>
#include <tuple>

#include "common.cuh"
#include "paged.cuh"
#include "paged_rows.cuh"
#include "tc05.cuh"

namespace cg = cooperative_groups;

namespace wsvd {

namespace {

// ------------------------------------------------------------------ 1. rotate + split
// EPT consecutive values a thread (a power of two, 32 EPT >= blk), loaded and stored
// eight at a time: whole sectors, and fewer lane exchanges per value than with four
// (1728 tokens of E 4096: four at a time 16 us, eight 13; calls of 1728 tokens with
// E 2048 38.8 us with EPT 4, 36.1 with 8, with E 4096 75.3 with 8 and with 16).
template <int EPT>
__global__ void __launch_bounds__(512) block_rotate_kernel(const uint16_t* x, int dtype, int E, int blk, float hnorm,
                                                           __half* xhi, __half* xlo, float* inv_p) {
  __shared__ float wmax[16];
  griddep_wait();
  griddep_launch_dependents();  // the GEMM may set up (it waits for this grid before it reads)
  const int tid = threadIdx.x, lane = tid & 31, e = tid * EPT;
  const size_t at = (size_t)blockIdx.x * E + e;
  float v[EPT];
#pragma unroll
  for (int i = 0; i < EPT; i += 8) {
    uint4 w = make_uint4(0, 0, 0, 0);
    if (e + i < E) w = *reinterpret_cast<const uint4*>(x + at + i);
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = dtype == WSVD_DTYPE_BF16
                           ? make_float2(__uint_as_float(ws[k] << 16), __uint_as_float(ws[k] & 0xffff0000u))
                           : h2_pair(ws[k]);
      v[i + 2 * k] = f.x;
      v[i + 2 * k + 1] = f.y;
    }
  }
  // Sylvester butterflies; blocks of blk values never cross E's end.
#pragma unroll
  for (int hh = 1; hh < EPT; hh <<= 1) {
    if (hh >= blk) break;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      if (i & hh) continue;
      const float u = v[i], w = v[i + hh];
      v[i] = u + w;
      v[i + hh] = u - w;
    }
  }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    if (d * EPT >= blk) break;
    const bool upper = lane & d;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const float w = __shfl_xor_sync(0xffffffffu, v[i], d);
      v[i] = upper ? w - v[i] : v[i] + w;
    }
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < EPT; ++i) {
    v[i] *= hnorm;
    amax = fmaxf(amax, fabsf(v[i]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (lane == 0) wmax[tid >> 5] = amax;
  __syncthreads();
  amax = 0.f;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) amax = fmaxf(amax, wmax[w]);
  int k = 0;  // clamped so that 2^k and 2^-k are normal floats
  if (amax > 0.f) k = max(-126, min(126, 14 - ((int)((__float_as_uint(amax) >> 23) & 0xffu) - 127)));
  const float p = __uint_as_float((uint32_t)(127 + k) << 23);
#pragma unroll
  for (int i = 0; i < EPT; i += 8) {
    if (e + i >= E) break;
    uint32_t hw[4], lw[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float a = v[i + 2 * q] * p, b = v[i + 2 * q + 1] * p;
      const __half2 h = __floats2half2_rn(a, b);
      const float2 f = __half22float2(h);
      const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
      hw[q] = *reinterpret_cast<const uint32_t*>(&h);
      lw[q] = *reinterpret_cast<const uint32_t*>(&l);
    }
    *reinterpret_cast<uint4*>(xhi + at + i) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
    *reinterpret_cast<uint4*>(xlo + at + i) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
  }
  if (tid == 0) inv_p[blockIdx.x] = __uint_as_float((uint32_t)(127 - k) << 23);
}

// ------------------------------------------------------------------ 2. GEMM + quantise
constexpr int kBK = 64, kSMs = 148;

// TOK tokens a tile, 64 (hi above lo) or 128 (hi and lo products in turn).  Tiles of 256 columns have two epilogue threads a row, 128 columns each.
template <int R, int BN_, int TOK_>
struct BlockCfg {
  static constexpr int BN = BN_, TOK = TOK_;
  static constexpr int CG = BN == 256 ? 2 : 1, COLS = BN / CG;   // column groups; columns a thread sums
  static constexpr int kEpi = 128 * CG;                           // epilogue threads
  static constexpr int kThreads = kEpi + 64;
  static constexpr int NG = R <= 64 ? R : 64;                    // columns per weight box
  static constexpr int SW = NG == 16 ? 6 : (NG == 32 ? 4 : 2);   // descriptor swizzle: 32 / 64 / 128 bytes
  static constexpr int HALF = TOK * kBK * 2;                      // hi (or lo) rows of a stage
  static constexpr int STAGE = 2 * HALF + kBK * BN * 2;
  static constexpr int S = 196608 / STAGE < 6 ? 196608 / STAGE : 6;
  static constexpr int NH = 512 / BN;                             // accumulators: all 512 columns
  static constexpr int PITCH = BN + 4;                            // floats per row of the sums
  // The sums reuse the ring: 128 operand rows, and behind them a rank's share of the tokens.
  static constexpr int SUMS = (128 + TOK / 2) * PITCH * 4;
  static constexpr int RING = SUMS > S * STAGE ? SUMS : S * STAGE;
  static constexpr int SMEM = RING + 1024 + 256;
  static_assert(R <= BN && STAGE % 1024 == 0, "whole heads; stages keep the swizzle atoms' alignment");
  static_assert(TOK == 64 || TOK == 128, "operand rows");
};

struct BlockArgs {
  int M, T, B, H, bits, cap, KT, ranks, ctas;
  const float* inv_p;
  const int32_t* seq_lens;
  uint8_t *lat_k, *lat_v;
  __half *scale_k, *scale_v;
  int32_t* counter;
  int32_t* err;
};

// TMA tile loads, warp-level: a converged warp calls them, one elected lane issues.
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* tm, int c0, int c1, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      "\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* tm, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}

// a += x, b += y, rounding to nearest.
__device__ __forceinline__ void add2(float& a, float& b, uint32_t x, uint32_t y) {
  asm("{\n\t.reg .b64 s, t;\n\t"
      "mov.b64 s, {%0, %1};\n\tmov.b64 t, {%2, %3};\n\t"
      "add.rn.f32x2 s, s, t;\n\tmov.b64 {%0, %1}, s;\n\t}"
      : "+f"(a), "+f"(b)
      : "r"(x), "r"(y));
}

// grid (token tiles x ranks, column tiles of K then V)
template <int R, int BN_, int TOK_>
__global__ void __launch_bounds__(BlockCfg<R, BN_, TOK_>::kThreads, 1)
    block_gemm_kernel(const __grid_constant__ CUtensorMap tm_xhi, const __grid_constant__ CUtensorMap tm_xlo,
                      const __grid_constant__ CUtensorMap tm_wk, const __grid_constant__ CUtensorMap tm_wv,
                      const BlockArgs a, const PagedRows place) {
  using C = BlockCfg<R, BN_, TOK_>;
  constexpr int BN = C::BN, TOK = C::TOK, NG = C::NG, S = C::S, NH = C::NH, kThreads = C::kThreads;
  constexpr int kProducer = C::kEpi / 32, kIssuer = kProducer + 1;  // warps
  extern __shared__ __align__(128) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // swizzle atoms need 1024-byte alignment
  uint8_t* smem = smem_raw + (base - raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::RING);
  uint64_t* empty = full + S;
  uint64_t* hfull = empty + S;   // [NH] a k-tile's sums are in tensor memory
  uint64_t* hfree = hfull + NH;  // [NH] they have been read (an arrival per warp)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(hfree + NH);
  __shared__ int sm_pos[TOK], sm_why[TOK];  // of the tile's tokens: first row of its block, refusal
  const int tid = threadIdx.x, warp = tid >> 5;
  const int ranks = a.ranks, rank = (int)blockIdx.x % ranks;
  const int m0 = (int)blockIdx.x / ranks * TOK;
  const int side = (int)gridDim.y / 2, kv = (int)blockIdx.y >= side, nl = ((int)blockIdx.y - kv * side) * BN;
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < NH; ++i) {
      mbar_init(&hfull[i], 1);
      mbar_init(&hfree[i], C::kEpi / 32);
    }
    fence_mbar_init();
  }
  if (warp == kIssuer) tc05::alloc(tmem_slot, 512);
  tc05::fence_before_sync();
  __syncthreads();
  tc05::fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  bool timed_out = false;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!mbar_wait_bounded(bar, parity, timed_out ? 0ull : kWaitLimitNs)) {
      if (!timed_out) set_err(a.err, WSVD_DEVERR_PIPE_TIMEOUT);
      timed_out = true;
    }
  };
  const int kt0 = a.KT * rank / ranks, KT = a.KT * (rank + 1) / ranks - kt0;  // this rank's k-tiles

  if (warp == kProducer) {  // ---------------------------------------------- TMA producer
    const CUtensorMap* wmap = kv ? &tm_wv : &tm_wk;
    bool waited = false;
    for (int kt = 0; kt < KT; ++kt) {
      const int s = kt % S;
      if (kt >= S) wait(&empty[s], (uint32_t)(((kt / S) - 1) & 1));
      __syncwarp();
      const uint32_t st = base + (uint32_t)(s * C::STAGE);
      const int k0 = (kt0 + kt) * kBK;
      mbar_arrive_expect_tx_warp(&full[s], C::STAGE);
      // The weights first: they do not wait for the rotation.
#pragma unroll
      for (int g = 0; g < BN / NG; ++g) {
        const int col = nl + g * NG;  // heads past the last are filled with zeros
        tma_3d(st + 2 * C::HALF + g * (kBK * NG * 2), wmap, col % R, k0, col / R, &full[s]);
      }
      if (!waited) griddep_wait();
      waited = true;
      tma_2d(st, &tm_xhi, k0, m0, &full[s]);  // tokens past the last are filled with zeros
      tma_2d(st + C::HALF, &tm_xlo, k0, m0, &full[s]);
    }
    for (int kt = std::max(0, KT - S); kt < KT; ++kt) wait(&full[kt % S], (uint32_t)((kt / S) & 1));
    __syncwarp();
  } else if (warp == kIssuer) {  // ----------------------------------------- MMA issuer
    constexpr uint32_t idesc = tc05::instr_desc(1, 0, 0, 0, 1, 128, BN);
    for (int kt = 0; kt < KT; ++kt) {
      const int s = kt % S, hb = kt % NH;
      wait(&full[s], (uint32_t)((kt / S) & 1));
      if (kt >= NH) wait(&hfree[hb], (uint32_t)(((kt / NH) - 1) & 1));
      __syncwarp();
      tc05::fence_after_sync();
      const uint32_t st = base + (uint32_t)(s * C::STAGE), d = tmem + (uint32_t)(hb * BN);
#pragma unroll
      for (int op = TOK == 64 ? 0 : 1; op >= 0; --op)  // lo first: the sum grows last
#pragma unroll
        for (int kk = 0; kk < kBK / 16; ++kk)
          tc05::mma_f16_warp(d, tc05::smem_desc_sw(st + op * C::HALF + kk * 32, 16, 1024, 2),
                             tc05::smem_desc_sw(st + 2 * C::HALF + kk * 32 * NG, 128 * NG, 16 * NG, C::SW), idesc,
                             kk > 0 || (TOK == 128 && op == 0));
      tc05::commit_warp(&empty[s]);
      tc05::commit_warp(&hfull[hb]);
    }
    // every MMA has completed before the ring is reused and the allocation released
    for (int kt = std::max(0, KT - NH); kt < KT; ++kt) wait(&hfull[kt % NH], (uint32_t)((kt / NH) & 1));
    __syncwarp();
  } else {  // ---------------------------------------------------------------- thread = operand row
    constexpr int COLS = C::COLS;
    const int col0 = (tid >> 7) * COLS;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)col0;
    const int token = tid & (TOK - 1), m = m0 + token;
    if (tid < TOK && m < a.M) {  // while the first tiles arrive
      const int b = m / a.T, pos = ld_relaxed_gpu(a.seq_lens + b);
      sm_pos[token] = pos;
      sm_why[token] = place.refused(b, pos, a.T, a.cap);
    }
    __syncwarp();
    float tot[COLS];
#pragma unroll
    for (int c = 0; c < COLS; ++c) tot[c] = 0.f;
    for (int kt = 0; kt < KT; ++kt) {
      const int hb = kt % NH;
      wait(&hfull[hb], (uint32_t)((kt / NH) & 1));
      tc05::fence_after_sync();
#pragma unroll
      for (int c0 = 0; c0 < COLS; c0 += 64) {  // two loads in flight per wait
        uint32_t va[32], vb[32];
        tc05::ld32(lane_base + (uint32_t)(hb * BN + c0), va);
        tc05::ld32(lane_base + (uint32_t)(hb * BN + c0 + 32), vb);
        tc05::wait_ld();
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          add2(tot[c0 + c], tot[c0 + c + 1], va[c], va[c + 1]);
          add2(tot[c0 + 32 + c], tot[c0 + 33 + c], vb[c], vb[c + 1]);
        }
      }
      tc05::fence_before_sync();
      __syncwarp();
      if ((tid & 31) == 0) mbar_arrive(&hfree[hb]);
    }
    griddep_wait();  // 1 / p comes from the rotation grid
    const float ip = m < a.M ? a.inv_p[m] : 0.f;
    float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(smem) +
                                            (size_t)(tid & 127) * C::PITCH + col0);
#pragma unroll
    for (int c = 0; c < COLS; c += 4)
      dst[c / 4] = make_float4(tot[c] * ip, tot[c + 1] * ip, tot[c + 2] * ip, tot[c + 3] * ip);
  }

  // ---- the rank's share of the tokens: hi and lo of all ranks, in order
  cg::cluster_group cluster = cg::this_cluster();
  float* part = reinterpret_cast<float*>(smem);  // [hi 64, lo 64] or [128][PITCH]
  // The joined tokens [PITCH]: behind the parts that other ranks read, else over the hi rows.
  float* sums = ranks > 1 ? part + 128 * C::PITCH : part;
  const int r0 = TOK * rank / ranks, rows = TOK * (rank + 1) / ranks - r0;
  if (ranks > 1) cluster.sync();
  else __syncthreads();
  for (int i = tid; i < rows * (BN / 4); i += kThreads) {
    const int row = i / (BN / 4), c = i % (BN / 4) * 4;
    if (m0 + r0 + row >= a.M) break;
    const size_t at = (size_t)(r0 + row) * C::PITCH + c;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    float4 x[8], y[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < ranks) {
        const float* p = (ranks > 1 ? cluster.map_shared_rank(part, q) : part) + at;
        x[q] = *reinterpret_cast<const float4*>(p);
        y[q] = TOK == 64 ? *reinterpret_cast<const float4*>(p + 64 * C::PITCH) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < ranks)
        v = make_float4(v.x + (x[q].x + y[q].x), v.y + (x[q].y + y[q].y), v.z + (x[q].z + y[q].z),
                        v.w + (x[q].w + y[q].w));
    *reinterpret_cast<float4*>(sums + (size_t)row * C::PITCH + c) = v;
  }
  if (ranks > 1) cluster.sync();  // the ranks' sums have been read: a rank may leave
  else __syncthreads();

  // ---- quantise: LPU threads to a (token, head) row, QCOLS of its columns each
  constexpr int HEADS = BN / R, LPU = R > 32 ? R / 32 : 1, QCOLS = R / LPU;
  const int Q = a.bits == 8 ? 127 : 7, RB = R * a.bits / 8;
  const int units = rows * HEADS * LPU;
  for (int u = tid; u < (units + 31) / 32 * 32; u += kThreads) {  // whole warps: the maximum crosses lanes
    const int row = u / (HEADS * LPU), hh = u / LPU % HEADS, sub = u % LPU, m = m0 + r0 + row, h = nl / R + hh;
    const bool real = u < units && m < a.M && h < a.H;
    const float4* src = reinterpret_cast<const float4*>(sums + (size_t)(u < units ? row : 0) * C::PITCH + hh * R + sub * QCOLS);
    float v[QCOLS], amax = 0.f;
#pragma unroll
    for (int c = 0; c < QCOLS / 4; ++c) {
      const float4 x = src[c];
      v[4 * c] = x.x; v[4 * c + 1] = x.y; v[4 * c + 2] = x.z; v[4 * c + 3] = x.w;
      amax = max_abs(max_abs(max_abs(max_abs(amax, x.x), x.y), x.z), x.w);
    }
#pragma unroll
    for (int o = LPU / 2; o > 0; o >>= 1) amax = max_abs(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (!real) continue;
    const int b = m / a.T, t = m - b * a.T, pos = sm_pos[r0 + row], why = sm_why[r0 + row];
    if (why) {
      if (blockIdx.y == 0 && hh == 0 && sub == 0 && t == 0) set_err(a.err, why);
      continue;
    }
    const __half sh = __float2half_rn(__fdiv_rn(amax, (float)Q));
    const float sc = __half2float(sh);
    const size_t at = place.row(b, h, a.H, pos + t, a.cap);
    auto code = [&](int j) { return sc > 0.f ? max(-Q, min(Q, __float2int_rn(__fdiv_rn(v[j], sc)))) : 0; };
    uint32_t* dst = reinterpret_cast<uint32_t*>((kv ? a.lat_v : a.lat_k) + at * RB + sub * (QCOLS * a.bits / 8));
    if (a.bits == 8) {
#pragma unroll
      for (int w = 0; w < QCOLS / 4; ++w) {
        uint32_t x = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) x |= ((uint32_t)code(4 * w + k) & 0xFFu) << (8 * k);
        dst[w] = x;
      }
    } else {
#pragma unroll
      for (int w = 0; w < QCOLS / 8; ++w) {
        uint32_t x = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) x |= ((uint32_t)code(8 * w + k) & 0xFu) << (4 * k);
        dst[w] = x;
      }
    }
    if (sub == 0) (kv ? a.scale_v : a.scale_k)[at] = sh;
  }
  tc05::fence_before_sync();
  __syncthreads();
  if (warp == kIssuer) {
    tc05::fence_after_sync();
    tc05::dealloc(tmem, 512);
  }

  // ---- the new lengths, by the last CTA to come here (every CTA has read the old ones)
  if (tid < 32) {
    int last = 0;
    if (tid == 0) last = atom_add_acq_rel_gpu(a.counter, 1) == a.ctas - 1;
    if (__shfl_sync(0xffffffffu, last, 0)) {
      for (int b = tid; b < a.B; b += 32) {
        const int pos = ld_relaxed_gpu(a.seq_lens + b);
        place.advance(nullptr, b, pos, a.T, place.refused(b, pos, a.T, a.cap) == 0);
      }
      if (tid == 0) st_relaxed_gpu(a.counter, 0);
    }
  }
}

// ------------------------------------------------------------------ host
// Tensor maps are encoded through the driver's entry point (no link-time
// dependence on the driver library).
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Tokens [M][E] fp16: boxes of 64 columns x a tile's rows, 128-byte swizzle.
bool token_map(CUtensorMap* tm, const void* base, int M, int E, int rows) {
  auto enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)E, (cuuint64_t)M};
  const cuuint64_t strides[1] = {(cuuint64_t)E * 2};
  const cuuint32_t box[2] = {(cuuint32_t)kBK, (cuuint32_t)rows}, es[2] = {1, 1};
  return enc(tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Weights [H][E][r] fp16 as (j, e, h): boxes of NG columns x 64 rows of one head.
bool weight_map(CUtensorMap* tm, const void* base, int H, int E, int r, int NG) {
  auto enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)r, (cuuint64_t)E, (cuuint64_t)H};
  const cuuint64_t strides[2] = {(cuuint64_t)r * 2, (cuuint64_t)E * r * 2};
  const cuuint32_t box[3] = {(cuuint32_t)NG, (cuuint32_t)kBK, 1}, es[3] = {1, 1, 1};
  const CUtensorMapSwizzle sw = NG == 16   ? CU_TENSOR_MAP_SWIZZLE_32B
                                : NG == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                           : CU_TENSOR_MAP_SWIZZLE_128B;
  return enc(tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters of c CTAs of a kernel that the current device runs at once (the
// shared-memory opt-in is made on the way; asked once per device, kernel and
// size; 0 on failure).
int resident_clusters(const void* kern, int threads, size_t smem, int c) {
  static std::mutex mu;
  static std::map<std::tuple<int, const void*, int>, int> known;
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lock(mu);
  const auto key = std::make_tuple(dev, kern, c);
  auto it = known.find(key);
  if (it != known.end()) return it->second;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)c);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    return 0;  // asked again next time
  }
  return known[key] = n;
}

// CTAs that split E for one tile: the most whose clusters all run at once, at
// least two k-tiles each.
template <int R, int BN, int TOK>
int tile_ranks(int tiles, int KT) {
  using C = BlockCfg<R, BN, TOK>;
  const void* fn = reinterpret_cast<const void*>(block_gemm_kernel<R, BN, TOK>);
  for (int c = 8; c > 1; --c)
    if (2 * c <= KT && tiles * (long long)c <= kSMs && tiles <= resident_clusters(fn, C::kThreads, C::SMEM, c)) return c;
  return 1;
}

template <int R, int BN, int TOK>
cudaError_t launch_tiles(BlockArgs a, const __half* xhi, const __half* xlo, int E, const void* A_k, const void* A_v,
                         const PagedRows& place, cudaStream_t s) {
  using C = BlockCfg<R, BN, TOK>;
  auto kern = block_gemm_kernel<R, BN, TOK>;
  const void* fn = reinterpret_cast<const void*>(kern);
  CUtensorMap mh, ml, mk, mv;
  if (!token_map(&mh, xhi, a.M, E, TOK) || !token_map(&ml, xlo, a.M, E, TOK) || !weight_map(&mk, A_k, a.H, E, R, C::NG) ||
      !weight_map(&mv, A_v, a.H, E, R, C::NG))
    return cudaErrorInvalidValue;
  if (resident_clusters(fn, C::kThreads, C::SMEM, 1) < 1) return cudaErrorInvalidConfiguration;
  const int mt = (a.M + TOK - 1) / TOK, nt = 2 * ((a.H * R + BN - 1) / BN);
  a.KT = E / kBK;
  a.ranks = tile_ranks<R, BN, TOK>(mt * nt, a.KT);
  a.ctas = mt * a.ranks * nt;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)a.ranks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(mt * a.ranks), (unsigned)nt);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, mh, ml, mk, mv, a, place);
}

// Which tile: 64 tokens x 128 columns, 64 x 256 or 128 x 256.  The operand tiles come
// from L2 and bound the kernel once the CTAs fill the device: 32, 48 and 64 KB a
// k-tile for 1, 2 and 4 times the products.
//   Columns.  With half a wave of tiles or fewer the narrow ones keep more SMs at work.
// Measured, 128 / 256 columns in us (32 heads, E 4096): r 32, 16 tokens 15.4 / 16.6, 128
// 18.2 / 22.3, 320 33.8 / 29.5, 576 36.6 / 32.8, 1728 102 / 95; r 64, 128 23.1 / 23.9,
// 256 34.7 / 28.9, 576 68.1 / 44.9, 1728 195 / 127; r 128, 128 34.5 / 29.8; r 16, 576
// 30.0 / 29.8, 1728 79.5 / 69.  Columns past a side's last head are idle: at most a
// quarter of them.
//   Tokens.  Of the wide tiles, those whose waves end sooner: a k-tile takes 0.53 us of
// 64 tokens, 0.86 of 128 (weighed 5 : 8).  Measured, 64 / 128 tokens: r 32, 400 tokens
// 29.1 / 27.9, 576 30.7 / 35.0, 800 46.8 / 43.5, 1152 50.6 / 46.5, 1728 91 / 75, 4096
// 195 / 160; r 64, 576 44.3 / 69, 1152 84 / 74, 1728 125 / 139, 4096 308 / 290; r 128,
// 320 85 / 69, 576 84 / 124, 1152 163 / 141, 4096 627 / 510.
//   Dropped: pairs of CTAs of 128 tokens that share their weight tile (cta_group::2):
// a fresh accumulator per k-tile has to be read by both before the next but one, 1.37
// us a k-tile; accumulators of four k-tiles, 0.9.  Sums of two k-tiles an accumulator
// changed the single CTAs by less than 2 %.
template <int R>
cudaError_t launch_block(const BlockArgs& a, const __half* xhi, const __half* xlo, int E, const void* A_k,
                         const void* A_v, const PagedRows& place, cudaStream_t s) {
  const int hr = a.H * R, KT = E / kBK, mt = (a.M + 63) / 64, n256 = 2 * ((hr + 255) / 256);
  if ((long long)mt * 2 * ((hr + 127) / 128) > kSMs / 2 && 2 * n256 * 256 <= 5 * hr) {
    const int few = mt * n256, tall = (mt + 1) / 2 * n256;  // tiles of 64, of 128 tokens
    const auto span = [&](int tiles, int ranks) {
      return (long long)((tiles * ranks + kSMs - 1) / kSMs) * ((KT + ranks - 1) / ranks);
    };
    if (8 * span(tall, tile_ranks<R, 256, 128>(tall, KT)) < 5 * span(few, tile_ranks<R, 256, 64>(few, KT)))
      return launch_tiles<R, 256, 128>(a, xhi, xlo, E, A_k, A_v, place, s);
    return launch_tiles<R, 256, 64>(a, xhi, xlo, E, A_k, A_v, place, s);
  }
  if constexpr (R <= 64)
    if (hr <= 64) return launch_tiles<R, 64, 64>(a, xhi, xlo, E, A_k, A_v, place, s);
  return launch_tiles<R, 128, 64>(a, xhi, xlo, E, A_k, A_v, place, s);
}

inline size_t align16(size_t v) { return (v + 15) / 16 * 16; }

}  // namespace

size_t paged_block_scratch(int B, int T, int E) {
  const size_t M = (size_t)B * T;
  return 2 * align16(M * E * 2) + align16(M * 4);
}

bool paged_block_takes(int B, int T, int H, int E, int r) {
  const long long M = (long long)B * T;
  return E % 64 == 0 && E <= 16384 && M <= (1LL << 24) && (long long)H * r <= (1LL << 21) &&
         M * H * r <= (1LL << 42) &&  // tiles in an int
         (r == 16 || r == 32 || r == 64 || r == 128);
}

cudaError_t launch_paged_block(const AppendArgs& p, int T, const PagedRows& place, void* scratch, cudaStream_t s) {
  const int M = p.B * T;
  uint8_t* w = static_cast<uint8_t*>(scratch);
  const size_t xbytes = align16((size_t)M * p.E * 2);
  __half *xhi = reinterpret_cast<__half*>(w), *xlo = reinterpret_cast<__half*>(w + xbytes);
  float* inv = reinterpret_cast<float*>(w + 2 * xbytes);
  const uint16_t* x = static_cast<const uint16_t*>(p.x);
  int ept = 8;
  while (ept * 32 < p.blk || ept * 512 < p.E) ept *= 2;
  const unsigned nt = (unsigned)((p.E / ept + 31) / 32 * 32);
  const auto rotate = ept == 8 ? block_rotate_kernel<8>
                      : ept == 16 ? block_rotate_kernel<16> : block_rotate_kernel<32>;
  const cudaError_t e = launch_behind(rotate, dim3((unsigned)M), (int)nt, 0, s, x, p.x_dtype, p.E, p.blk, p.hnorm, xhi,
                                      xlo, inv);
  if (e != cudaSuccess) return e;
  BlockArgs a{};
  a.M = M; a.T = T; a.B = p.B; a.H = p.H; a.bits = p.bits; a.cap = p.L_cap;
  a.inv_p = inv; a.seq_lens = p.seq_lens;
  a.lat_k = p.lat_k; a.lat_v = p.lat_v; a.scale_k = p.scale_k; a.scale_v = p.scale_v;
  a.counter = p.counter; a.err = p.err;
  switch (p.r) {
    case 16: return launch_block<16>(a, xhi, xlo, p.E, p.Ak, p.Av, place, s);
    case 32: return launch_block<32>(a, xhi, xlo, p.E, p.Ak, p.Av, place, s);
    case 64: return launch_block<64>(a, xhi, xlo, p.E, p.Ak, p.Av, place, s);
    case 128: return launch_block<128>(a, xhi, xlo, p.E, p.Ak, p.Av, place, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace wsvd
