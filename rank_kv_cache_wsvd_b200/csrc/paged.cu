// Dense 16-bit key-value cache in pages, for sm_100a: appending new keys and
// values with the rotary position rotation, and attention of the newest
// token(s) over the pages.
//
// A cache is a pool of pages [num_pages][Hkv][page_size][Hd] shared by all
// sequences; block_table[b][i] names the page that holds rows
// i * page_size .. of sequence b, so row l of head h lies at
//   pool + ((block_table[b][l / page_size] * Hkv + h) * page_size + l % page_size) * Hd.
#include <algorithm>
#include <map>
#include <mutex>
#include <tuple>
#include <type_traits>

#include "common.cuh"
#include "paged.cuh"
#include "wsvd_internal.h"

using namespace wsvd;

namespace {

// ------------------------------------------------------------------ append
struct KvAppendArgs {
  int T, Hq, Hkv, Hd, rot, inter, page_shift, num_pages, max_pages, cap;
  int row_slots;  // threads that share a token's rows, per unit (a power of two)
  const uint16_t *k, *v, *q;
  long long k_stride, v_stride, q_stride;
  const float* cos_sin;
  const int32_t* new_lens;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int32_t* seq_lens_out;
  uint16_t *k_pages, *v_pages, *q_out;
  int32_t* counters;
  int32_t* err;
};

// Small CTAs, since each waits out its length and page loads: 8 x 2048 tokens of
// 32 + 2 x 8 heads of 128 take 64.7 us with 128 threads, 67.5 with 256, 73.5 with
// 512; 576 tokens of 96 heads 5.8, 7.5 and 12.3 us; one token 3.06, 2.93 and 3.2.
constexpr int kAppendCta = 128;

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return h2_pair(w);
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (BF16) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// The next 16-bit part of two weights, which keep what is left: bf16 the upper
// halves, so that three parts carry all 24 bits; fp16 rounded, two parts 22 bits.
template <bool BF16>
__device__ __forceinline__ uint32_t take_part(float& p0, float& p1) {
  if constexpr (BF16) {
    const uint32_t a = __float_as_uint(p0), b = __float_as_uint(p1);
    p0 -= __uint_as_float(a & 0xffff0000u);
    p1 -= __uint_as_float(b & 0xffff0000u);
    return __byte_perm(a, b, 0x7632);
  } else {
    const uint32_t x = pack2<BF16>(p0, p1);
    const float2 f = unpack2<BF16>(x);
    p0 -= f.x;
    p1 -= f.y;
    return x;
  }
}

// The rotation of 8 pairs (a_i, b_i): a' = a cos - b sin, b' = b cos + a sin,
// in fp32, rounded once to the 16-bit type of the cache.  x, y: the two
// 16-byte chunks of a unit.  Split pairs: a_i in x, b_i in y; interleaved: the
// pairs lie side by side, the first four in x, the others in y.
template <bool BF16>
__device__ __forceinline__ void rotate_unit(uint4& x, uint4& y, const float4* cs, const float4* sn, bool inter) {
  uint32_t* xw = reinterpret_cast<uint32_t*>(&x);
  uint32_t* yw = reinterpret_cast<uint32_t*>(&y);
  const float* c = reinterpret_cast<const float*>(cs);
  const float* s = reinterpret_cast<const float*>(sn);
  if (inter) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 u = unpack2<BF16>(xw[i]), w = unpack2<BF16>(yw[i]);
      xw[i] = pack2<BF16>(u.x * c[i] - u.y * s[i], u.y * c[i] + u.x * s[i]);
      yw[i] = pack2<BF16>(w.x * c[4 + i] - w.y * s[4 + i], w.y * c[4 + i] + w.x * s[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 u = unpack2<BF16>(xw[i]), w = unpack2<BF16>(yw[i]);
      const float c0 = c[2 * i], c1 = c[2 * i + 1], s0 = s[2 * i], s1 = s[2 * i + 1];
      xw[i] = pack2<BF16>(u.x * c0 - w.x * s0, u.y * c1 - w.y * s1);
      yw[i] = pack2<BF16>(w.x * c0 + u.x * s0, w.y * c1 + u.y * s1);
    }
  }
}

// grid (token tiles, B).  A unit is 32 bytes of one head's row: 16-byte chunks i
// and i + rot/16 of the rotated values (which split pairs need together), or
// two chunks half of the rest apart, so that the threads of a row always touch
// neighbouring chunks.  A thread keeps one token and one unit, so it reads its
// cosines and sines and the token's page once, and walks the token's rows (Hq
// of q, Hkv of k, Hkv of v) kAppendRows at a time, their loads in flight
// together; the first of them leave before the length and the page table, which
// they do not depend on, are known.  Bound by the bytes for prompts (8 x 2048
// tokens, 32 + 2 x 8 heads of 128: 64.7 us, 6.35 TB/s), by three dependent loads
// (length, page, angle) for one token (3 us).  Six rows at a time: with three the
// same prompts took 69.6, with four, which leave a part-filled second turn, 82.2.
constexpr int kAppendRows = 6;

template <bool BF16>
__global__ void __launch_bounds__(kAppendCta) kv_append_kernel(const KvAppendArgs a) {
  griddep_wait();
  const int b = blockIdx.y, tid = threadIdx.x;
  const int units = a.Hd / 16, rows = a.Hq + 2 * a.Hkv, ru = a.rot / 16;
  const int unit = tid & (units - 1), slot = tid / units;
  const int step = a.row_slots, t = blockIdx.x * (kAppendCta / units / step) + slot / step;
  // A padded block's counts come first: its padding is not read.
  const int n = a.new_lens ? a.new_lens[b] : a.T;
  const bool turned = unit < ru;
  const int c0 = turned ? unit : ru + unit, c1 = turned ? unit + ru : units + unit;
  uint4 x[kAppendRows], y[kAppendRows];
  const size_t tok = (size_t)b * a.T + min(t, a.T - 1);
  auto fetch = [&](int row0) {
#pragma unroll
    for (int i = 0; i < kAppendRows; ++i) {
      const int row = row0 + i * step;
      if (t >= min(n, a.T) || row >= rows) continue;
      const int kr = row - a.Hq, vr = kr - a.Hkv;
      const uint16_t* src = kr < 0   ? a.q + tok * a.q_stride + (size_t)row * a.Hd
                            : vr < 0 ? a.k + tok * a.k_stride + (size_t)kr * a.Hd
                                     : a.v + tok * a.v_stride + (size_t)vr * a.Hd;
      x[i] = reinterpret_cast<const uint4*>(src)[c0];
      y[i] = reinterpret_cast<const uint4*>(src)[c1];
    }
  };
  const int row_first = slot & (step - 1);
  fetch(row_first);

  const int pos = a.seq_lens[b];
  // The whole block of a sequence is refused together, so every CTA of the
  // sequence comes to the same answer before it writes.
  const bool len_ok = n >= 0 && n <= a.T;
  bool ok = len_ok && pos >= 0 && (long long)pos + n <= a.cap;
  const int32_t* table = a.block_table + (size_t)b * a.max_pages;
  bool bad_page = false;
  if (ok && n > 0) {
    const int p1 = (pos + n - 1) >> a.page_shift;
    for (int p = (pos >> a.page_shift) + tid; p <= p1; p += kAppendCta) {
      const int pg = table[p];
      bad_page |= pg < 0 || pg >= a.num_pages;
    }
  }
  bad_page = __syncthreads_or(bad_page);
  if (tid == 0 && blockIdx.x == 0) {
    if (!len_ok) set_err(a.err, WSVD_DEVERR_LEN_RANGE);
    else if (!ok) set_err(a.err, WSVD_DEVERR_CACHE_FULL);
    else if (bad_page) set_err(a.err, WSVD_DEVERR_PAGE_RANGE);
  }
  ok = ok && !bad_page;
  const int there = ok ? n : 0;

  if (t < a.T) {
    const bool stored = t < there;
    const int l = stored ? pos + t : 0;
    float4 c[2], s[2];
    size_t page_row = 0;  // of head 0; a head further lies a page further
    if (stored) {
      page_row = (((size_t)table[l >> a.page_shift] * a.Hkv) << a.page_shift) + (l & ((1 << a.page_shift) - 1));
      if (turned) {
        const float4* cs = reinterpret_cast<const float4*>(a.cos_sin + (size_t)l * a.rot);
        const float4* sn = cs + a.rot / 8;
        const int i0 = a.inter ? unit : 2 * unit, i1 = a.inter ? unit + ru : 2 * unit + 1;
        c[0] = cs[i0]; c[1] = cs[i1];
        s[0] = sn[i0]; s[1] = sn[i1];
      }
    }
    for (int row0 = row_first; row0 < rows; row0 += kAppendRows * step) {
      if (row0 != row_first) fetch(row0);
#pragma unroll
      for (int i = 0; i < kAppendRows; ++i) {
        const int row = row0 + i * step;
        if (row >= rows) break;
        const int kr = row - a.Hq, vr = kr - a.Hkv;
        if (!stored) {  // padding: nothing is cached, q_out is zero
          if (kr >= 0) break;
          x[i] = y[i] = make_uint4(0, 0, 0, 0);
        } else if (turned && vr < 0) {
          rotate_unit<BF16>(x[i], y[i], c, s, a.inter);
        }
        uint16_t* out = kr < 0   ? a.q_out + (tok * a.Hq + row) * a.Hd
                        : vr < 0 ? a.k_pages + (page_row + ((size_t)kr << a.page_shift)) * a.Hd
                                 : a.v_pages + (page_row + ((size_t)vr << a.page_shift)) * a.Hd;
        reinterpret_cast<uint4*>(out)[c0] = x[i];
        reinterpret_cast<uint4*>(out)[c1] = y[i];
      }
    }
  }

  // The new length.  Written in place it must not be seen by a CTA of this
  // sequence that has not read the old one: the last CTA to arrive writes it.
  if (tid == 0) {
    const int len = there ? pos + there : pos;
    if (a.seq_lens_out != a.seq_lens) {
      if (blockIdx.x == 0) a.seq_lens_out[b] = len;
    } else if (gridDim.x == 1) {
      a.seq_lens_out[b] = len;
    } else if (atom_add_acq_rel_gpu(a.counters + b, 1) == (int)gridDim.x - 1) {
      st_relaxed_gpu(a.seq_lens_out + b, len);
      st_relaxed_gpu(a.counters + b, 0);
    }
  }
}

// ------------------------------------------------------------------ decode
// For each sequence b, KV head h and chunk of its G * Tq queries the rows are
// cut into strips of TS rows.  All strips of all (b, h, chunk) units, in that
// order, are dealt evenly to a grid of CTAs; a CTA's share of one unit is a
// segment, whose strips its warps take in turn.  Each warp is a pipeline of its
// own: it copies its strips with cp.async into its ring in shared memory
// (16-byte chunks, swizzled so that ldmatrix reads no bank twice) and needs no
// barrier until the segment ends.
//
// Per strip, with m16n8k16 products (up to 8 queries as their columns, up to 16 as
// their rows, so GQA reads the rows once for all of them):
//   S = K q^T (or q K^T)       the queries held in registers
//   p = 2^(S * scale * log2 e - m), m the running maximum of the warp's rows
//   O^T += V^T p^T (or P V)    V by transposed ldmatrix
// p is not rounded to the 16-bit type: it is cut into parts whose sum carries
// 22 (two fp16 parts) or 24 bits (three bf16 parts), each its own product.
// The products cost less than the rows' bytes for up to 16 queries.
template <bool BF16, int HD, int NB>
struct DecCfg {
  // Rows per strip, warps per CTA and stages per warp: strips of 8 KB (16 KB at
  // head size 256), a ring of 192 KB per SM.  A warp reads one stage while the others
  // are on their way: 96 KB an SM with two stages.  Twelve warps of two stages beat
  // eight of three (4 x 32768 rows of 8 heads of 128: 84.7 us against 87.3) except with
  // 16 queries of head size 128 and their registers (16 sequences of 1024 .. 4096 rows
  // of 8 heads 41.5 against 38.8, 4 x 32768 rows 92.7 against 94.5).  Strips of half the
  // size need more warps for the same bytes and lose (16 queries of head size 64 as
  // columns, 9 x 32768 rows: sixteen warps of three 66.0 against 56.6).
  static constexpr bool kWide = HD == 128 && NB == 2;
  static constexpr int kTS = HD >= 128 ? 16 : (HD == 64 ? 32 : 64);
  static constexpr int kWarps = HD == 256 ? 6 : kWide ? 8 : 12;
  static constexpr int kStages = kWide ? 3 : 2;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kMT = kTS / 16;
  static constexpr int kHalf = kTS * HD * 2;      // bytes of a strip's K (or V)
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kChunks = HD / 8;          // 16-byte chunks of a row
  static constexpr int kParts = BF16 ? 3 : 2;
  static constexpr int kQ = 8 * NB;               // queries of a chunk
  static constexpr size_t kSmem = (size_t)kWarps * kStages * kStage;
  static_assert(kQ * HD * 4 <= kStage, "a warp's merge scratch is one stage");
};

// Floats of one partial result: O [queries][Hd], then (m, l) per query, a
// multiple of four so that every O row can be read in 16-byte pieces.
__host__ __device__ constexpr int partial_floats(int queries, int Hd) { return queries * Hd + (2 * queries + 3) / 4 * 4; }

struct KvDecodeArgs {
  PagedSeqs seqs;  // a unit: a KV head and a chunk of its queries
  int Tq, Hq, Hkv, G, nq, chunks, page_shift, num_pages, max_pages, ctas;
  const int32_t* block_table;
  const uint16_t *q, *k, *v;
  float* out;
  float* partials;  // two a worker: O [min(nq, kQ)][HD], then (m, l) per query
  int32_t* counters;  // by the first worker of a cut unit
  int32_t* err;
  float qscale;
};

__device__ __forceinline__ uint32_t movm_t(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF16)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte chunk c of row r in a strip: eight rows at one chunk
// index lie in eight different 16-byte columns of the banks.
template <int HD>
__device__ __forceinline__ uint32_t strip_off(int r, int c) {
  if (HD == 32) return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
  return (uint32_t)(r * HD * 2 + ((c ^ (r & 7)) << 4));
}

// The same product into D = 0 + A B.
template <bool BF16>
__device__ __forceinline__ void mma16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF16)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// (x0, x1) = (x0, x1) f + (y0, y1), one instruction.
__device__ __forceinline__ void fma2(float& x0, float& x1, float f, float y0, float y1) {
  asm("{\n\t.reg .b64 x, f, y;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 f, {%2, %2};\n\tmov.b64 y, {%3, %4};\n\t"
      "fma.rn.f32x2 x, x, f, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(f), "f"(y0), "f"(y1));
}

// Whether a strip of `bytes` at vb holds an infinity or a NaN (the whole warp asks).
template <bool BF16>
__device__ __forceinline__ bool any_wild(uint32_t vb, int bytes, int lane) {
  bool wild = false;
  for (int i = lane; i < bytes / 16; i += 32) {
    const uint4 w = lds128(vb + (uint32_t)i * 16);
    const uint32_t e = BF16 ? 0x7f80u : 0x7c00u, e2 = e << 16;
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) wild |= (ws[k] & e) == e || (ws[k] & e2) == e2;
  }
  return __any_sync(0xffffffffu, wild);
}

// Up to eight queries of a warp, as the columns of the products: S = K q^T, O^T += V^T p^T.
template <bool BF16, int HD>
struct Queries8 {
  using C = DecCfg<BF16, HD, 1>;
  static constexpr int TS = C::kTS, MT = C::kMT, KS = HD / 16, NP = C::kParts;
  static constexpr float kBias = BF16 ? 0.f : 12.f;
  uint32_t q[KS][2];
  int lim[2], lim_min;              // rows that query 2 c4 + i sees
  float scale, m[2], l[2], o[KS][4];  // o: dims 16 d + g, then + 8, of queries 2 c4 + {0, 1}

  __device__ __forceinline__ void begin(const KvDecodeArgs& a, int b, int n, int h, int j0, int nq, int lane) {
    const int g = lane >> 2, c4 = lane & 3;
    lim_min = n - a.Tq + 1;
    scale = a.qscale;
    const int jq = j0 + (g < nq ? g : 0);
    const uint16_t* qr = a.q + (((size_t)b * a.Tq + jq / a.G) * a.Hq + h * a.G + jq % a.G) * HD + 2 * c4;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      q[k][0] = g < nq ? __ldg(reinterpret_cast<const uint32_t*>(qr + 16 * k)) : 0u;
      q[k][1] = g < nq ? __ldg(reinterpret_cast<const uint32_t*>(qr + 16 * k + 8)) : 0u;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      lim[i] = lim_min + min(j0 + 2 * c4 + i, a.nq - 1) / a.G;
      m[i] = kNegInf;
      l[i] = 0.f;
    }
#pragma unroll
    for (int d = 0; d < KS; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
  }

  __device__ __forceinline__ void strip(const KvDecodeArgs& a, uint32_t kb, uint32_t vb, int l0, int valid, int lane) {
    const int g = lane >> 2, c4 = lane & 3;
    // Two sums (even and odd steps of 16 values), so that consecutive products
    // do not wait for one another.
    float sc[MT][4], sc2[MT][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[t][i] = sc2[t][i] = 0.f;
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        uint32_t kf[4];
        ldsm4(kf, kb + strip_off<HD>(t * 16 + (lane & 15), 2 * k + (lane >> 4)));
        mma16816<BF16>(k & 1 ? sc2[t] : sc[t], kf, q[k][0], q[k][1]);
      }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[t][i] = (sc[t][i] + sc2[t][i]) * scale;
    const bool masked = l0 > lim_min - TS || valid != (1 << MT) - 1;
    if (masked) {
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = l0 + t * 16 + g + (i >> 1) * 8;
          if (row >= lim[i & 1] || !((valid >> t) & 1)) sc[t][i] = kNegInf;
        }
    }
    // Running maximum and sum; columns (queries) of sc and o are the same.
    float alpha[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float mx = kNegInf;
#pragma unroll
      for (int t = 0; t < MT; ++t) mx = fmaxf(mx, fmaxf(sc[t][i], sc[t][i + 2]));
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      const float mn = fmaxf(m[i], mx);
      const float ref = mn == kNegInf ? 0.f : mn;
      alpha[i] = ex2(m[i] - ref);
      m[i] = mn;
      float add = 0.f;
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int r = 0; r < 4; r += 2) {
          const float p = ex2(sc[t][i + r] - ref + kBias);
          sc[t][i + r] = p;
          add += p;
        }
      l[i] = l[i] * alpha[i] + add;
    }
    if (masked && a.Tq > 1 && any_wild<BF16>(vb, C::kHalf, lane)) {  // as for 16 queries, row by row
#pragma unroll
      for (int d = 0; d < KS; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[d][i] *= alpha[i & 1];
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll 1
        for (int r = 0; r < 16; ++r) {
          const int row = l0 + t * 16 + r, from = (r & 7) * 4 + c4;
          const float p00 = __shfl_sync(0xffffffffu, sc[t][0], from);
          const float p01 = __shfl_sync(0xffffffffu, sc[t][1], from);
          const float p10 = __shfl_sync(0xffffffffu, sc[t][2], from);
          const float p11 = __shfl_sync(0xffffffffu, sc[t][3], from);
          const float p[2] = {r < 8 ? p00 : p10, r < 8 ? p01 : p11};
#pragma unroll
          for (int d = 0; d < KS; ++d)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint16_t w;
              asm volatile("ld.shared.u16 %0, [%1];"
                           : "=h"(w)
                           : "r"(vb + strip_off<HD>(t * 16 + r, 2 * d + half) + 2u * g)
                           : "memory");
              const float v = BF16 ? __uint_as_float((uint32_t)w << 16) : __half2float(__ushort_as_half(w));
#pragma unroll
              for (int i = 0; i < 2; ++i)
                if (row < lim[i]) o[d][2 * half + i] = fmaf(p[i], v, o[d][2 * half + i]);
            }
        }
      return;
    }
    uint32_t pf[MT][NP][2];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      float r0 = sc[t][0], r1 = sc[t][1], r2 = sc[t][2], r3 = sc[t][3];
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        pf[t][k][0] = movm_t(take_part<BF16>(r0, r1));
        pf[t][k][1] = movm_t(take_part<BF16>(r2, r3));
      }
    }
    constexpr int DG = 4 < KS ? 4 : KS;  // sums that start at zero, as for 16 queries
#pragma unroll
    for (int d0 = 0; d0 < KS; d0 += DG) {
      float part[DG][4];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        uint32_t vf[DG][4];
#pragma unroll
        for (int d = 0; d < DG; ++d)
          ldsm4_t(vf[d], vb + strip_off<HD>(t * 16 + ((lane >> 4) << 3) + (lane & 7), 2 * (d0 + d) + ((lane >> 3) & 1)));
#pragma unroll
        for (int k = 0; k < NP; ++k)
#pragma unroll
          for (int d = 0; d < DG; ++d) {
            if (t == 0 && k == 0) mma16816_first<BF16>(part[d], vf[d], pf[t][k][0], pf[t][k][1]);
            else mma16816<BF16>(part[d], vf[d], pf[t][k][0], pf[t][k][1]);
          }
      }
#pragma unroll
      for (int d = 0; d < DG; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[d0 + d][i] = fmaf(o[d0 + d][i], alpha[i & 1], part[d][i]);
    }
  }

  __device__ __forceinline__ void leave(float* scratch, float* sm_m, float* sm_l, int lane) const {
    const int g = lane >> 2, c4 = lane & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float v = l[i];
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) v += __shfl_xor_sync(0xffffffffu, v, x);
      const int j = 2 * c4 + i;
      if (g == 0) {
        sm_m[j] = m[i];
        sm_l[j] = v;
      }
#pragma unroll
      for (int d = 0; d < KS; ++d) {
        scratch[j * HD + ((d * 16 + g) ^ (c4 << 3))] = o[d][i];
        scratch[j * HD + ((d * 16 + 8 + g) ^ (c4 << 3))] = o[d][2 + i];
      }
    }
  }
};

// Up to 16 queries of a warp, as the rows of the products: S = q K^T, O += P V.
// The scores' registers are the second product's operand as they lie (no
// movmatrix), and a query's maximum crosses four lanes: 561 instructions a strip (32
// rows, head size 64), 762 as two column blocks of the form for eight.  28 queries
// of 4 heads of 64, 9 x 32768 rows: 81 us against 101; 16 of 8 heads of 128, 4 x 32768
// rows: 93 against 95.6.
template <bool BF16, int HD>
struct Queries16 {
  using C = DecCfg<BF16, HD, 2>;
  static constexpr int TS = C::kTS, MT = C::kMT, KS = HD / 16, NP = C::kParts;
  // 2^bias keeps the low fp16 part of small weights out of the denormals.
  static constexpr float kBias = BF16 ? 0.f : 12.f;
  uint32_t q[KS][4];
  int lim[2], lim_min;             // rows that query g + 8 i sees
  float scale, m[2], l[2], o[HD / 8][4];  // o: dims 8 n + 2 c4 + {0, 1} of query g, then of g + 8

  __device__ __forceinline__ void begin(const KvDecodeArgs& a, int b, int n, int h, int j0, int nq, int lane) {
    const int g = lane >> 2, c4 = lane & 3;
    lim_min = n - a.Tq + 1;
    scale = fabsf(a.qscale);  // its sign goes into the queries
    const uint32_t flip = a.qscale < 0.f ? 0x80008000u : 0u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = g + 8 * i, jq = j0 + (j < nq ? j : 0);
      const uint16_t* qr = a.q + (((size_t)b * a.Tq + jq / a.G) * a.Hq + h * a.G + jq % a.G) * HD + 2 * c4;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        q[k][i] = j < nq ? __ldg(reinterpret_cast<const uint32_t*>(qr + 16 * k)) ^ flip : 0u;
        q[k][2 + i] = j < nq ? __ldg(reinterpret_cast<const uint32_t*>(qr + 16 * k + 8)) ^ flip : 0u;
      }
      lim[i] = lim_min + min(j0 + j, a.nq - 1) / a.G;
      m[i] = kNegInf;
      l[i] = 0.f;
    }
#pragma unroll
    for (int d = 0; d < HD / 8; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
  }

  // The strip of rows l0 .. at kb and vb; bit t of valid: 16 rows whose page is in the pool.
  __device__ __forceinline__ void strip(const KvDecodeArgs& a, uint32_t kb, uint32_t vb, int l0, int valid, int lane) {
    const int c4 = lane & 3;
    float sc[2 * MT][4];
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        uint32_t f[4];
        ldsm4(f, kb + strip_off<HD>(t * 16 + ((lane >> 4) << 3) + (lane & 7), 2 * k + ((lane >> 3) & 1)));
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (k == 0) mma16816_first<BF16>(sc[2 * t + x], q[k], f[2 * x], f[2 * x + 1]);
          else mma16816<BF16>(sc[2 * t + x], q[k], f[2 * x], f[2 * x + 1]);
        }
      }
    const bool masked = l0 > lim_min - TS || valid != (1 << MT) - 1;
    if (masked) {
#pragma unroll
      for (int t = 0; t < 2 * MT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (l0 + t * 8 + 2 * c4 + (i & 1) >= lim[i >> 1] || !((valid >> (t / 2)) & 1)) sc[t][i] = kNegInf;
    }
    float alpha[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float mx = kNegInf;
#pragma unroll
      for (int t = 0; t < 2 * MT; ++t) mx = fmaxf(mx, fmaxf(sc[t][2 * i], sc[t][2 * i + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m[i], mx * scale);
      const float ref = mn == kNegInf ? 0.f : mn;
      alpha[i] = ex2(m[i] - ref);
      m[i] = mn;
      float add0 = 0.f, add1 = 0.f;
      const float sub = kBias - ref;
#pragma unroll
      for (int t = 0; t < 2 * MT; ++t) {
        fma2(sc[t][2 * i], sc[t][2 * i + 1], scale, sub, sub);
        sc[t][2 * i] = ex2(sc[t][2 * i]);
        sc[t][2 * i + 1] = ex2(sc[t][2 * i + 1]);
        add0 += sc[t][2 * i];
        add1 += sc[t][2 * i + 1];
      }
      l[i] = fmaf(l[i], alpha[i], add0 + add1);
    }
    // A later token's value may be infinite or NaN; it must not reach the
    // queries that do not see it (0 * NaN), so such a strip is summed row by
    // row.  Rows past the length are zero already.
    if (masked && a.Tq > 1 && any_wild<BF16>(vb, C::kHalf, lane)) {
#pragma unroll
      for (int d = 0; d < HD / 8; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[d][i] *= alpha[i >> 1];
#pragma unroll
      for (int t = 0; t < 2 * MT; ++t)
#pragma unroll 1
        for (int r = 0; r < 8; ++r) {
          float p[4];  // query g and g + 8 of row r: even and odd rows lie in different registers
#pragma unroll
          for (int i = 0; i < 4; ++i) p[i] = __shfl_sync(0xffffffffu, sc[t][i], (lane & ~3) | (r >> 1));
          const float w[2] = {r & 1 ? p[1] : p[0], r & 1 ? p[3] : p[2]};
          const int row = t * 8 + r;
#pragma unroll
          for (int d = 0; d < HD / 8; ++d) {
            const float2 v = unpack2<BF16>(lds32(vb + strip_off<HD>(row, d) + 4u * c4));
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (l0 + row < lim[i]) {
                o[d][2 * i] = fmaf(w[i], v.x, o[d][2 * i]);
                o[d][2 * i + 1] = fmaf(w[i], v.y, o[d][2 * i + 1]);
              }
          }
        }
      return;
    }
    uint32_t pf[MT][NP][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int x = 0; x < 4; ++x) {  // query g (x even) or g + 8, rows 2 c4 + {0, 1} (x < 2) or eight on
        float p0 = sc[2 * t + x / 2][2 * (x & 1)], p1 = sc[2 * t + x / 2][2 * (x & 1) + 1];
#pragma unroll
        for (int k = 0; k < NP; ++k) pf[t][k][x] = take_part<BF16>(p0, p1);
      }
    // Each strip's product starts at zero and joins O in fp32: the tensor
    // cores' own sums do not round to nearest, and over a long cache that
    // bias would show (3e-6 of the output at 32768 rows, 4e-7 this way).
    // Several dim blocks at a time, for products that do not wait for one another.
    constexpr int DG = 2;
#pragma unroll
    for (int d0 = 0; d0 < KS; d0 += DG) {
      float part[2 * DG][4];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        uint32_t f[DG][4];
#pragma unroll
        for (int d = 0; d < DG; ++d) ldsm4_t(f[d], vb + strip_off<HD>(t * 16 + (lane & 15), 2 * (d0 + d) + (lane >> 4)));
#pragma unroll
        for (int k = 0; k < NP; ++k)
#pragma unroll
          for (int d = 0; d < 2 * DG; ++d) {
            if (t == 0 && k == 0) mma16816_first<BF16>(part[d], pf[t][k], f[d / 2][2 * (d & 1)], f[d / 2][2 * (d & 1) + 1]);
            else mma16816<BF16>(part[d], pf[t][k], f[d / 2][2 * (d & 1)], f[d / 2][2 * (d & 1) + 1]);
          }
      }
#pragma unroll
      for (int d = 0; d < 2 * DG; ++d)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          fma2(o[2 * d0 + d][2 * i], o[2 * d0 + d][2 * i + 1], alpha[i], part[d][2 * i], part[d][2 * i + 1]);
    }
  }

  // O as [query][dim] with bits 3 and 4 of dim turned by the query, and the statistics.
  __device__ __forceinline__ void leave(float* scratch, float* sm_m, float* sm_l, int lane) const {
    const int g = lane >> 2, c4 = lane & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float v = l[i];
      v += __shfl_xor_sync(0xffffffffu, v, 1);
      v += __shfl_xor_sync(0xffffffffu, v, 2);
      const int j = g + 8 * i;
      if (c4 == 0) {
        sm_m[j] = m[i];
        sm_l[j] = v;
      }
#pragma unroll
      for (int d = 0; d < HD / 8; ++d)
        *reinterpret_cast<float2*>(scratch + j * HD + ((d * 8 + 2 * c4) ^ (((j >> 1) & 3) << 3))) =
            make_float2(o[d][2 * i], o[d][2 * i + 1]);
    }
  }
};

// Strips that a segment's fixed cost counts as.  Measured, 0 / 8 / 16 / 24 / 32 / 48 strips
// in us: nine ragged sequences with 28 queries of 4 heads of 64 24.0 / 22.1 / 21.5 / 20.8 /
// 20.6 / 21.2; with 7 queries 16.0 / 15.4 / 14.5 / 13.3 / 13.6 / 13.6; 32 heads of 1600 rows
// 13.3 / 14.0 / 11.8 / 11.1 / 11.2 / 11.3.
constexpr int kLead = 24;

// Up to 8 queries a head, many units and sequences of few strips: every warp is a
// worker with segments of its own, nothing waits for a CTA, and most units end in
// one warp's registers.  Measured with CTAs / warps as workers (us, head size 128):
// 256 sequences x 128 rows of 8 heads, 4 queries each 56.4 / 36.5; 64 x 200 rows of 32
// heads 68.4 / 42.9, 64 x 500 95.7 / 88.4, 32 x 1000 87.9 / 86.9; 8 heads with 4 queries,
// 64 x 500 33.8 / 33.7, 256 x 500 99.7 / 96.6, 256 x 1000 168 / 172, 32 x 1000 30.2 / 33.8;
// with 8 queries 64 x 300 28.4 / 30.0; one sequence of 300 rows, whose few units warps
// would have to join, 7.8 / 15.
constexpr int kSoloStrips = 40, kSoloUnits = 512, kSoloLead = 4;
constexpr int kMaxSolo = 2016;  // workers that way at most

// MANY: many units, so that their sequences may be short (kSoloUnits); a kernel of
// its own, as the code alone costs a small call half a microsecond.
template <bool BF16, int HD, int NB, bool MANY>
__global__ void __launch_bounds__(DecCfg<BF16, HD, NB>::kThreads, 1) kv_decode_kernel(const KvDecodeArgs a) {
  using C = DecCfg<BF16, HD, NB>;
  constexpr int TS = C::kTS, MT = C::kMT, S = C::kStages, NW = C::kWarps;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float sm_m[NW][C::kQ], sm_l[NW][C::kQ];
  __shared__ int sm_valid[NW][S];
  __shared__ int sm_slot[NW], sm_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c4 = lane & 3;
  const int c = blockIdx.x;
  const PagedSeqs& seqs = a.seqs;
  griddep_wait();

  // Sequences without rows: zeros, spread over the CTAs.
  for (int b = c; b < seqs.B; b += gridDim.x)
    if (seqs.rows(b) == 0)
      for (int i = tid; i < a.Tq * a.Hq * HD; i += C::kThreads) a.out[(size_t)b * a.Tq * a.Hq * HD + i] = 0.f;
  Strips<TS> share;
  typename Strips<TS>::Segment seg;
  bool solo = false;  // short sequences: every warp a worker of its own
  int me = c;
  const auto plan = [&](int mean, int live) {
    solo = MANY && mean < kSoloStrips && live * (long long)seqs.units >= kSoloUnits;
    if (!solo) return typename Strips<TS>::Plan{c, a.ctas, NW, kLead};
    me = warp * (int)gridDim.x + c;
    return typename Strips<TS>::Plan{me, min((int)gridDim.x * NW, kMaxSolo), 1, kSoloLead};
  };
  if (!share.deal(seqs, plan, a.err, &seg)) return;
  const int first = MANY && solo ? 0 : warp, stride = MANY && solo ? 1 : NW;  // of a segment's strips, this warp's

  // ---- the warp's copies: cursor `ld`, page ids one strip ahead
  const uint32_t my_ring = smem_u32(ring) + (uint32_t)warp * S * C::kStage;
  auto ld = seg;
  int ls = ld.s + first;
  int lh = 0;  // its KV head
  bool more = true, moved = true;
  int pg[MT];
  const int page_mask = (1 << a.page_shift) - 1;
  auto settle = [&]() {  // the next strip of this warp, and its pages
    while (more && ls >= ld.e) {
      more = ld.next(seqs);
      ls = ld.s + first;
      moved = true;
    }
    if (more) {
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int l = ls * TS + i * 16;
        pg[i] = l < ld.n ? __ldg(a.block_table + (size_t)ld.b * a.max_pages + (l >> a.page_shift)) : 0;
      }
      if (moved) lh = ld.u / a.chunks;  // while the page ids arrive
      moved = false;
    }
  };
  auto issue = [&](int stage) {
    if (more) {
      const uint32_t dst = my_ring + (uint32_t)stage * C::kStage;
      int valid = 0;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int l0 = ls * TS + i * 16;
        const bool in = pg[i] >= 0 && pg[i] < a.num_pages;
        if (!in && lane == 0 && l0 < ld.n) set_err(a.err, WSVD_DEVERR_PAGE_RANGE);
        valid |= (in ? 1 : 0) << i;
        const size_t row0 = (((size_t)(in ? pg[i] : 0) * a.Hkv + lh) << a.page_shift) + (l0 & page_mask);
        const int rows = in ? ld.n - l0 : 0;  // rows at and past the length are zero-filled, not read
        constexpr int kPer = 16 * C::kChunks / 32;
        const uint16_t *ks = a.k + row0 * HD + lane * 8, *vs = a.v + row0 * HD + lane * 8;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int idx = j * 32 + lane, r = idx / C::kChunks, ch = idx % C::kChunks;
          const uint32_t to = dst + strip_off<HD>(i * 16 + r, ch), bytes = r < rows ? 16u : 0u;
          cp_async16(to, ks + j * 256, bytes);
          cp_async16(to + C::kHalf, vs + j * 256, bytes);
        }
      }
      if (lane == 0) sm_valid[warp][stage] = valid;
      ls += stride;
      settle();
    }
    cp_commit();
  };
  settle();
  for (int i = 0; i < S - 1; ++i) issue(i);
  int stage = 0;  // of the next strip to read

  // ---- segment by segment
  for (bool go = true; go; go = seg.next(seqs)) {
    if (seg.s == seg.e) continue;
    const int h = seg.u / a.chunks, j0 = (seg.u % a.chunks) * C::kQ;
    const int nq = min(C::kQ, a.nq - j0);
    const int lim_min = seg.n - a.Tq + 1;
    typename std::conditional<NB == 1, Queries8<BF16, HD>, Queries16<BF16, HD>>::type acc;
    acc.begin(a, seg.b, seg.n, h, j0, nq, lane);

    int last_stage = stage == 0 ? S - 1 : stage - 1;  // a stage with nothing in it or on its way
    for (int s = seg.s + first; s < seg.e; s += stride) {
      cp_wait<S - 2>();
      __syncwarp();
      issue(stage == 0 ? S - 1 : stage - 1);
      const uint32_t kb = my_ring + (uint32_t)stage * C::kStage;
      acc.strip(a, kb, kb + C::kHalf, s * TS, sm_valid[warp][stage], lane);
      __syncwarp();  // every lane has read this stage before it is filled again
      last_stage = stage;
      stage = stage == S - 1 ? 0 : stage + 1;
    }

    const bool whole = seg.s == 0 && seg.e == seg.strips();
    const int qmax = min(C::kQ, a.nq);  // queries per partial slot
    const int slot = partial_floats(qmax, HD);
    // A worker has at most one unit that it begins within, and one that it only begins.
    float* part = a.partials + (size_t)(2 * me + (seg.s == 0 ? 1 : 0)) * slot;
    auto store = [&](int j, int d, float4 v, float L) {
      const int jq = j0 + j, t = jq / a.G;
      const float f = lim_min + t > 0 ? 1.f / L : 0.f;
      if (f == 0.f) v = make_float4(0.f, 0.f, 0.f, 0.f);
      *reinterpret_cast<float4*>(a.out + (((size_t)seg.b * a.Tq + t) * a.Hq + h * a.G + jq % a.G) * HD + d) =
          make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
    };
    // Joins the partials of a unit's workers, in their order; idx0, step: the
    // caller's threads.
    auto join = [&](int idx0, int step) {
      int wf, np;
      share.holders(seg, &wf, &np);
      const float* from = a.partials + (size_t)2 * wf * slot;
      constexpr int kJoin = 8;  // partials whose loads are in flight together
      for (int idx = idx0; idx < nq * (HD / 4); idx += step) {
        const int j = idx / (HD / 4), d = idx % (HD / 4) * 4;
        float M = kNegInf, L = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = 0; i0 < np; i0 += kJoin) {
          float2 ml[kJoin];
          float4 x[kJoin];
          float top = M;
#pragma unroll
          for (int i = 0; i < kJoin; ++i) {
            const float* p = from + (size_t)2 * (i0 + i) * slot + (i0 + i == 0 ? slot : 0);  // slot 1 of the first
            const bool in = i0 + i < np;
            ml[i] = in ? __ldcg(reinterpret_cast<const float2*>(p + qmax * HD + 2 * j)) : make_float2(kNegInf, 0.f);
            x[i] = in ? __ldcg(reinterpret_cast<const float4*>(p + j * HD + d)) : make_float4(0.f, 0.f, 0.f, 0.f);
          }
#pragma unroll
          for (int i = 0; i < kJoin; ++i) top = fmaxf(top, ml[i].x);
          const float ref = top == kNegInf ? 0.f : top, f0 = ex2(M - ref);
          L *= f0;
          v = make_float4(v.x * f0, v.y * f0, v.z * f0, v.w * f0);
#pragma unroll
          for (int i = 0; i < kJoin; ++i) {
            const float f = ex2(ml[i].x - ref);
            L = fmaf(ml[i].y, f, L);
            v.x = fmaf(x[i].x, f, v.x);
            v.y = fmaf(x[i].y, f, v.y);
            v.z = fmaf(x[i].z, f, v.z);
            v.w = fmaf(x[i].w, f, v.w);
          }
          M = top;
        }
        store(j, d, v, L);
      }
    };

    if constexpr (MANY) if (solo) {  // ---- one warp's result: straight to out, or to its partial slot
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float L = acc.l[i];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) L += __shfl_xor_sync(0xffffffffu, L, x);
        const int j = 2 * c4 + i;
        if (j >= nq) continue;
        const int jq = j0 + j, t = jq / a.G;
        float* to = whole ? a.out + (((size_t)seg.b * a.Tq + t) * a.Hq + h * a.G + jq % a.G) * HD : part + j * HD;
        const bool sees = lim_min + t > 0;
        const float f = whole ? 1.f / L : 1.f;
#pragma unroll
        for (int d = 0; d < HD / 16; ++d) {
          __stcg(to + d * 16 + g, whole && !sees ? 0.f : acc.o[d][i] * f);
          __stcg(to + d * 16 + 8 + g, whole && !sees ? 0.f : acc.o[d][2 + i] * f);
        }
        if (!whole && g == 0) __stcg(reinterpret_cast<float2*>(part + qmax * HD + 2 * j), make_float2(acc.m[i], L));
      }
      if (whole) continue;
      int wf, np, last = 0;
      share.holders(seg, &wf, &np);
      __threadfence();
      __syncwarp();
      if (lane == 0) last = atom_add_acq_rel_gpu(a.counters + wf, 1) == np - 1;
      if (!__shfl_sync(0xffffffffu, last, 0)) continue;
      __threadfence();
      join(lane, 32);
      if (lane == 0) st_relaxed_gpu(a.counters + wf, 0);
      continue;
    }

    // ---- the warps' results of this segment, joined.  Each warp leaves O in
    // its free stage, [query][dim] with bits 3 and 4 of dim turned by the query
    // so that the stores meet no bank twice and float4 reads stay whole.
    float* scratch = reinterpret_cast<float*>(ring) + (size_t)(warp * S + last_stage) * (C::kStage / 4);
    acc.leave(scratch, sm_m[warp], sm_l[warp], lane);
    if (lane == 0) sm_slot[warp] = warp * S + last_stage;
    __syncthreads();
    for (int idx = tid; idx < nq * (HD / 4); idx += C::kThreads) {
      const int j = idx / (HD / 4), d = idx % (HD / 4) * 4;
      float M = kNegInf, L = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < NW; ++w) M = fmaxf(M, sm_m[w][j]);
      const float ref = M == kNegInf ? 0.f : M;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float f = ex2(sm_m[w][j] - ref);
        const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(ring) +
                                                          (size_t)sm_slot[w] * (C::kStage / 4) + j * HD +
                                                          (d ^ (((j >> 1) & 3) << 3)));
        L = fmaf(sm_l[w][j], f, L);
        v.x = fmaf(x.x, f, v.x);
        v.y = fmaf(x.y, f, v.y);
        v.z = fmaf(x.z, f, v.z);
        v.w = fmaf(x.w, f, v.w);
      }
      if (whole) {
        store(j, d, v, L);
      } else {
        __stcg(reinterpret_cast<float4*>(part + j * HD + d), v);
        if (d == 0) __stcg(reinterpret_cast<float2*>(part + qmax * HD + 2 * j), make_float2(M, L));
      }
    }

    // ---- a unit cut over several CTAs: the last to arrive joins the partials
    // in the order of the CTAs, so the result does not depend on who that is.
    if (!whole) {
      int wf, np;
      share.holders(seg, &wf, &np);
      __threadfence();
      __syncthreads();
      if (tid == 0) sm_last = atom_add_acq_rel_gpu(a.counters + wf, 1) == np - 1;
      __syncthreads();
      if (sm_last) {
        __threadfence();
        join(tid, C::kThreads);
        if (tid == 0) st_relaxed_gpu(a.counters + wf, 0);
      }
    }
    __syncthreads();  // the scratch and the statistics are free again
  }
  cp_wait<0>();
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t align16(size_t v) { return (v + 15) / 16 * 16; }
inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

// Queries per chunk: 16, at head size 256 eight (registers).
// Two sixteens over one copy of the rows at head sizes 32 and 64 (eight warps, three
// stages) gain for long sequences what they lose for short ones: 28 queries of 4 heads
// of 64, 9 x 32768 rows 78.5 us against 86.5 (81 since), 9 ragged sequences 21.3 / 21.0, of 64
// rows 7.6 / 6.5.
inline int chunk_queries(int nq, int Hd) { return nq > 8 && Hd != 256 ? 16 : 8; }

using DecodeFn = void (*)(const KvDecodeArgs);
struct DecodeKernel {
  DecodeFn fn;
  size_t smem;
  int threads;
};
template <bool BF16, int HD, int NB>
DecodeKernel decode_kernel_of(bool many = false) {
  using C = DecCfg<BF16, HD, NB>;
  return DecodeKernel{many ? &kv_decode_kernel<BF16, HD, NB, NB == 1> : &kv_decode_kernel<BF16, HD, NB, false>, C::kSmem,
                      C::kThreads};
}
template <bool BF16>
DecodeKernel pick_decode(int Hd, int qc, bool many) {
  switch (Hd) {
    case 32: return qc == 16 ? decode_kernel_of<BF16, 32, 2>() : decode_kernel_of<BF16, 32, 1>(many);
    case 64: return qc == 16 ? decode_kernel_of<BF16, 64, 2>() : decode_kernel_of<BF16, 64, 1>(many);
    case 128: return qc == 16 ? decode_kernel_of<BF16, 128, 2>() : decode_kernel_of<BF16, 128, 1>(many);
    default: return decode_kernel_of<BF16, 256, 1>(many);
  }
}

// The workspace: the counters (kSplitCounterBytes, in front, so that no size of call
// moves them), then two partial results a worker.  Its size is that of 2048 warps
// or 592 CTAs and a counter per unit; the workers that a call never has make room
// for the counters.
constexpr int kSoloSlots = 2048, kCtaSlots = 592;
static_assert(kMaxSolo * sizeof(int32_t) <= kSplitCounterBytes && kMaxPagedCtas <= kMaxSolo, "a counter a worker");
static_assert((kSoloSlots - kMaxSolo) * 2 * partial_floats(1, 32) * sizeof(float) >= kSplitCounterBytes &&
                  (kCtaSlots - kMaxPagedCtas) * 2 * partial_floats(9, 32) * sizeof(float) >= kSplitCounterBytes,
              "the counters take the place of partial results that no worker has");
size_t decode_ws(int B, int Tq, int Hq, int Hkv, int Hd) {
  const int nq = Hq / Hkv * Tq, qc = chunk_queries(nq, Hd), chunks = (nq + qc - 1) / qc;
  return align16((size_t)2 * (qc == 8 ? kSoloSlots : kCtaSlots) * partial_floats(std::min(nq, qc), Hd) * sizeof(float)) +
         align16((size_t)B * Hkv * chunks * sizeof(int32_t));
}

}  // namespace

cudaError_t wsvd::paged_resident_ctas(const void* fn, int threads, size_t smem, int* ctas) {
  static std::mutex mu;
  static std::map<std::pair<int, const void*>, int> known;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  const auto key = std::make_pair(dev, fn);
  auto it = known.find(key);
  if (it == known.end()) {
    int sms = 0, occ = 0;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
        (e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess ||
        (e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, fn, threads, smem)) != cudaSuccess)
      return e;
    it = known.emplace(key, std::min(kMaxPagedCtas, sms * std::max(1, occ))).first;
  }
  *ctas = it->second;
  return cudaSuccess;
}

extern "C" {

size_t paged_kv_append_workspace_size(int B) { return B < 0 ? 0 : std::max<size_t>(16, align16((size_t)B * 4)); }

int paged_kv_append(int B, int T, int Hq, int Hkv, int Hd, int rot_dim, int interleaved, int page_size, int num_pages,
                    int max_pages, int max_pos, const void* k, long long k_stride, const void* v, long long v_stride,
                    const void* q, long long q_stride, int dtype, const float* cos_sin, const int32_t* new_lens,
                    const int32_t* block_table, const int32_t* seq_lens, int32_t* seq_lens_out, void* k_pages,
                    void* v_pages, void* q_out, void* workspace, size_t workspace_bytes, int32_t* err, void* stream) {
  if (B < 0 || T < 0 || Hq < 0 || Hkv < 1 || num_pages < 0 || max_pages < 0 || max_pos < 0) return WSVD_ERR_INVALID_ARG;
  if (B == 0) return WSVD_OK;
  if (dtype != WSVD_DTYPE_FP16 && dtype != WSVD_DTYPE_BF16) return WSVD_ERR_INVALID_ARG;
  if (rot_dim < 0 || rot_dim > Hd) return WSVD_ERR_INVALID_ARG;
  if (Hd != 32 && Hd != 64 && Hd != 128 && Hd != 256) return WSVD_ERR_UNSUPPORTED;
  if (rot_dim % 16) return WSVD_ERR_UNSUPPORTED;
  const int shift = page_shift_of(page_size);
  if (shift < 0 || B > 65535 || (long long)Hq + 2LL * Hkv > (1 << 20)) return WSVD_ERR_UNSUPPORTED;
  if ((long long)max_pages << shift > 0x7fffffffLL) return WSVD_ERR_UNSUPPORTED;
  if (!block_table || !seq_lens || !seq_lens_out || !k_pages || !v_pages || !workspace) return WSVD_ERR_INVALID_ARG;
  if (T > 0 && (!k || !v || (Hq > 0 && (!q || !q_out)))) return WSVD_ERR_INVALID_ARG;
  if (rot_dim > 0 && !cos_sin) return WSVD_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(q) || !aligned16(q_out) || !aligned16(k_pages) ||
      !aligned16(v_pages) || !aligned16(cos_sin) || !aligned16(workspace))
    return WSVD_ERR_INVALID_ARG;
  if (k_stride < (long long)Hkv * Hd || v_stride < (long long)Hkv * Hd || k_stride % 8 || v_stride % 8 ||
      (Hq > 0 && (q_stride < (long long)Hq * Hd || q_stride % 8)))
    return WSVD_ERR_INVALID_ARG;
  // Nothing that is written may share a byte with what is read, but for the
  // two that may be updated in place: the lengths, and a dense q.
  const size_t tok = (size_t)B * T, lb = (size_t)B * 4;
  size_t pool;
  if (!pool_bytes(num_pages, Hkv, shift, (size_t)Hd * 2, &pool)) return WSVD_ERR_UNSUPPORTED;
  bool wide = false;  // a stride whose last token lies past any address
  auto span = [&](const void* p, long long stride, int heads) {
    size_t n = 0;
    if (tok && heads)
      wide |= __builtin_mul_overflow(tok - 1, (size_t)stride, &n) || __builtin_add_overflow(n, (size_t)heads * Hd, &n) ||
              __builtin_mul_overflow(n, (size_t)2, &n);
    return Span{p, n};
  };
  const bool q_in_place = q_out == q && q_stride == (long long)Hq * Hd, lens_in_place = seq_lens_out == seq_lens;
  const Span read[] = {span(k, k_stride, Hkv), span(v, v_stride, Hkv), span(q_in_place ? nullptr : q, q_stride, Hq),
                       {block_table, (size_t)B * max_pages * 4}, {rot_dim ? cos_sin : nullptr, (size_t)max_pos * rot_dim * 4},
                       {new_lens, lb}, {lens_in_place ? nullptr : seq_lens, lb}};
  const Span written[] = {{k_pages, pool}, {v_pages, pool}, {q_out, tok * Hq * Hd * 2}, {seq_lens_out, lb},
                          {workspace, paged_kv_append_workspace_size(B)}, {err, 4}};
  if (wide || clash(written, read)) return WSVD_ERR_INVALID_ARG;
  if (workspace_bytes < paged_kv_append_workspace_size(B)) return WSVD_ERR_WORKSPACE_TOO_SMALL;

  KvAppendArgs a{};
  a.T = T; a.Hq = Hq; a.Hkv = Hkv; a.Hd = Hd; a.rot = rot_dim; a.inter = interleaved != 0;
  a.page_shift = shift; a.num_pages = num_pages; a.max_pages = max_pages;
  a.cap = max_pages << shift;
  if (rot_dim > 0) a.cap = std::min(a.cap, max_pos);
  a.k = static_cast<const uint16_t*>(k); a.v = static_cast<const uint16_t*>(v); a.q = static_cast<const uint16_t*>(q);
  a.k_stride = k_stride; a.v_stride = v_stride; a.q_stride = q_stride;
  a.cos_sin = cos_sin; a.new_lens = new_lens; a.block_table = block_table;
  a.seq_lens = seq_lens; a.seq_lens_out = seq_lens_out;
  a.k_pages = static_cast<uint16_t*>(k_pages); a.v_pages = static_cast<uint16_t*>(v_pages);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.counters = static_cast<int32_t*>(workspace); a.err = err;
  // Threads enough on a token's rows that each has all of its own in flight at
  // once; more of them when the tokens would not fill the SMs.
  const int slots = kAppendCta / (Hd / 16);
  a.row_slots = 1;
  while (a.row_slots < slots && a.row_slots * kAppendRows < Hq + 2 * Hkv) a.row_slots *= 2;
  while (a.row_slots < slots && tok * a.row_slots / slots < 148 * 4) a.row_slots *= 2;
  const int tokens = slots / a.row_slots;
  const dim3 grid((unsigned)std::max(1, (T + tokens - 1) / tokens), (unsigned)B);
  (void)cudaGetLastError();
  const auto kern = dtype == WSVD_DTYPE_BF16 ? kv_append_kernel<true> : kv_append_kernel<false>;
  return launch_behind(kern, grid, kAppendCta, 0, as_stream(stream), a) == cudaSuccess ? WSVD_OK : WSVD_ERR_CUDA;
}

size_t paged_decode_workspace_size(int B, int Tq, int Hq, int Hkv, int Hd) {
  if (B < 0 || Tq < 1 || Hkv < 1 || Hq < Hkv || Hq % Hkv || Hd < 1) return 0;
  return decode_ws(B, Tq, Hq, Hkv, Hd);
}

int paged_decode_attention(int B, int Tq, int Hq, int Hkv, int Hd, int page_size, int num_pages, int max_pages,
                           const int32_t* seq_lens, const int32_t* block_table, const void* q, const void* k_pages,
                           const void* v_pages, int dtype, float softmax_scale, float* out, void* workspace,
                           size_t workspace_bytes, int32_t* err, void* stream) {
  if (B < 0 || Tq < 1 || Hkv < 1 || Hq < Hkv || Hq % Hkv || num_pages < 0 || max_pages < 0) return WSVD_ERR_INVALID_ARG;
  if (B == 0) return WSVD_OK;
  if (dtype != WSVD_DTYPE_FP16 && dtype != WSVD_DTYPE_BF16) return WSVD_ERR_INVALID_ARG;
  if (Hd != 32 && Hd != 64 && Hd != 128 && Hd != 256) return WSVD_ERR_UNSUPPORTED;
  const int shift = page_shift_of(page_size);
  const long long nq = (long long)(Hq / Hkv) * Tq;
  if (shift < 0 || B > 65535 || nq > 64 || (long long)Tq * Hq * Hd > 0x7fffffffLL) return WSVD_ERR_UNSUPPORTED;
  if ((long long)max_pages << shift > 0x7fffffffLL) return WSVD_ERR_UNSUPPORTED;
  if (!seq_lens || !block_table || !q || !k_pages || !v_pages || !out || !workspace) return WSVD_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out) || !aligned16(workspace))
    return WSVD_ERR_INVALID_ARG;
  const size_t need = decode_ws(B, Tq, Hq, Hkv, Hd), queries = (size_t)B * Tq * Hq * Hd;
  size_t pool;
  if (!pool_bytes(num_pages, Hkv, shift, (size_t)Hd * 2, &pool)) return WSVD_ERR_UNSUPPORTED;
  const Span read[] = {{seq_lens, (size_t)B * 4}, {block_table, (size_t)B * max_pages * 4}, {q, queries * 2},
                       {k_pages, pool}, {v_pages, pool}};
  const Span written[] = {{out, queries * 4}, {workspace, need}, {err, 4}};
  if (clash(written, read)) return WSVD_ERR_INVALID_ARG;
  if (workspace_bytes < need) return WSVD_ERR_WORKSPACE_TOO_SMALL;
  const int qc = chunk_queries((int)nq, Hd);
  const bool many = (long long)B * Hkv * ((nq + qc - 1) / qc) >= kSoloUnits;
  const DecodeKernel kern = dtype == WSVD_DTYPE_BF16 ? pick_decode<true>(Hd, qc, many) : pick_decode<false>(Hd, qc, many);
  KvDecodeArgs a{};
  a.Tq = Tq; a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv; a.nq = (int)nq; a.chunks = (int)((nq + qc - 1) / qc);
  a.seqs = PagedSeqs{B, Hkv * a.chunks, max_pages << shift, seq_lens};
  a.page_shift = shift; a.num_pages = num_pages; a.max_pages = max_pages; a.block_table = block_table;
  a.q = static_cast<const uint16_t*>(q); a.k = static_cast<const uint16_t*>(k_pages);
  a.v = static_cast<const uint16_t*>(v_pages);
  a.out = out;
  a.counters = static_cast<int32_t*>(workspace);
  a.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kSplitCounterBytes);
  a.err = err;
  a.qscale = (softmax_scale != 0.f ? softmax_scale : (float)(1.0 / sqrt((double)Hd))) * kLog2e;
  (void)cudaGetLastError();
  if (paged_resident_ctas(reinterpret_cast<const void*>(kern.fn), kern.threads, kern.smem, &a.ctas) != cudaSuccess) return WSVD_ERR_CUDA;
  return launch_behind(kern.fn, dim3((unsigned)a.ctas), kern.threads, kern.smem, as_stream(stream), a) == cudaSuccess
             ? WSVD_OK
             : WSVD_ERR_CUDA;
}

}  // extern "C"
