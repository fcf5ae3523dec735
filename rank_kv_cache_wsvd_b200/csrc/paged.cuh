// Shared by the paged kernels: how the strips of ragged sequences are dealt to
// CTAs, the warp's copies, and host helpers of the entry points.
#pragma once

#include <utility>

#include "common.cuh"

namespace wsvd {

// ------------------------------------------------------------------ dealing strips to workers
// The sequences of a call and their units: every sequence has `units` of them
// (a head, or a head and a group of queries), each over all of its rows.
struct PagedSeqs {
  int B, units, cap;  // cap: rows the page table has room for
  const int32_t* seq_lens;
  __device__ __forceinline__ int rows(int b) const {  // a length out of range counts as none
    const int n = seq_lens[b];
    return n < 0 || n > cap ? 0 : n;
  }
};

// A unit's rows are cut into strips of TS rows, and counts as its strips plus a
// lead (what a segment costs beside its strips: queries, joins) when the shares
// of the workers (CTAs or warps) are cut, else a worker that meets many short
// sequences would finish last.
template <int TS>
struct Strips {
  // Unsigned: a length may be as large as an int holds.
  static __device__ __forceinline__ int strips_of(int n) { return (int)(((uint32_t)n + (TS - 1)) / TS); }
  // A worker's share of one unit: strips [s, e) of unit u of sequence b (n
  // rows); none when the share ends within the lead.
  struct Segment {
    int b, u, n, s, e, lead;
    int at, taken;   // where the share begins in the unit (lead included), and how much of the unit it takes
    long long left;  // of the worker's share from here on
    __device__ __forceinline__ int strips() const { return strips_of(n); }
    __device__ __forceinline__ void enter(int place) {
      at = place;
      taken = (int)min((long long)(strips() + lead - at), left);
      s = max(0, at - lead);
      e = max(0, at + taken - lead);
    }
    __device__ __forceinline__ bool next(const PagedSeqs& q) {
      left -= taken;
      if (left <= 0) return false;
      if (++u == q.units) {
        u = 0;
        do n = q.rows(++b);
        while (n == 0);
      }
      enter(0);
      return true;
    }
  };

  long long total, base, extra, end;  // strips in all; per worker; workers with one more; this worker's end
  int workers;                        // workers that have a share

  __device__ __forceinline__ long long begin_of(int c) const { return base * c + min((long long)c, extra); }
  __device__ __forceinline__ int worker_of(long long strip) const {  // whose share holds a strip
    const long long big = extra * (base + 1);
    return (int)(strip < big ? strip / (base + 1) : extra + (strip - big) / base);
  }
  // The workers that hold strips of the segment's unit: the first, and how many.
  __device__ __forceinline__ void holders(const Segment& g, int* first, int* count) const {
    const long long u0 = end - g.left - g.at + g.lead;  // the unit's first strip in the whole order
    *first = worker_of(u0);
    *count = worker_of(u0 + g.strips() - 1) - *first + 1;
  }

  // How the strips are dealt: this worker of `count`, `least` strips a worker at
  // least (so that a small problem is not cut too finely), a unit's lead.
  struct Plan {
    int me, count, least, lead;
  };

  // This worker's share and its first segment; false when it has none.  Every
  // warp finds it for itself (all lanes take part).  plan(mean, live): the Plan
  // for `live` sequences that have rows, whose units have `mean` strips on average.
  template <class F>
  __device__ __forceinline__ bool deal(const PagedSeqs& q, F plan, int32_t* err, Segment* seg) {
    const int lane = threadIdx.x & 31;
    const int per = (q.B + 31) / 32;
    const int b0 = min(q.B, lane * per), b1 = min(q.B, b0 + per);
    long long sum = 0;
    int live = 0;
#pragma unroll 4
    for (int b = b0; b < b1; ++b) {
      const int raw = q.seq_lens[b], n = raw < 0 || raw > q.cap ? 0 : raw;
      if (n != raw && blockIdx.x == 0) set_err(err, WSVD_DEVERR_LEN_RANGE);
      sum += strips_of(n);
      live += n > 0;
    }
    long long incl = sum;
    int lives = live;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      const int w = __shfl_up_sync(0xffffffffu, lives, o);
      if (lane >= o) {
        incl += v;
        lives += w;
      }
    }
    total = __shfl_sync(0xffffffffu, incl, 31);
    const int all_live = __shfl_sync(0xffffffffu, lives, 31);
    if (all_live == 0) return false;
    const Plan p = plan(total < 0x80000000ll ? (int)((uint32_t)total / (uint32_t)all_live) : 0x7fffffff, all_live);
    total = (total + (long long)all_live * p.lead) * q.units;
    const long long most = (total + p.least - 1) / p.least;
    workers = (int)(most < p.count ? most : p.count);
    if (p.me >= workers) return false;
    base = (unsigned long long)total < 0x80000000ull ? (uint32_t)total / (uint32_t)workers : total / workers;
    extra = total - base * workers;
    const long long begin = begin_of(p.me);
    end = begin + base + (p.me < extra ? 1 : 0);
    const long long before = (incl - sum + (long long)(lives - live) * p.lead) * q.units;
    const long long mine = (sum + (long long)live * p.lead) * q.units;
    const bool here = begin >= before && begin < before + mine;
    long long rem = begin - before;
    int sb = b0;
    if (here)
      for (;; ++sb) {
        const int n = q.rows(sb);
        const long long ns = n > 0 ? (long long)(strips_of(n) + p.lead) * q.units : 0;
        if (rem < ns) break;
        rem -= ns;
      }
    const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    seg->b = __shfl_sync(0xffffffffu, sb, src);
    rem = __shfl_sync(0xffffffffu, rem, src);
    seg->n = q.rows(seg->b);
    seg->left = end - begin;
    seg->lead = p.lead;
    const int unit = seg->strips() + p.lead;
    seg->u = (int)(rem / unit);
    seg->enter((int)(rem % unit));
    return true;
  }
};

// ------------------------------------------------------------------ warp copies and fragments
// 16 bytes to shared memory; `bytes` 0 reads nothing and fills with zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// ------------------------------------------------------------------ host
// Launches a kernel that begins with griddep_wait: its CTAs may be placed while
// the stream's preceding kernel drains, and touch no memory before that one has
// completed (two calls in a row 2 us sooner than with an ordinary launch).
template <class... P, class... A>
cudaError_t launch_behind(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A&&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<A>(args)...);
}

// Upper bound of the paged decodes' grids.
constexpr int kMaxPagedCtas = 588;

// log2 of a page size the paged caches take (16 .. 256), else -1.
inline int page_shift_of(int page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

// The bytes of an argument.
struct Span {
  const void* p;
  size_t n;
};
inline bool overlap(const Span& x, const Span& y) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
  return x.p && y.p && x.n && y.n && a < b + y.n && b < a + x.n;
}
// Whether something that is written shares a byte with something that is read or
// with another thing that is written.
template <int W, int R>
bool clash(const Span (&written)[W], const Span (&read)[R]) {
  for (int i = 0; i < W; ++i) {
    for (const Span& r : read)
      if (overlap(written[i], r)) return true;
    for (int j = i + 1; j < W; ++j)
      if (overlap(written[i], written[j])) return true;
  }
  return false;
}
// *bytes = num_pages * heads * page_size rows of row_bytes; false past 2^63.
inline bool pool_bytes(int num_pages, int heads, int page_shift, size_t row_bytes, size_t* bytes) {
  return !__builtin_mul_overflow((size_t)num_pages * (size_t)heads, row_bytes << page_shift, bytes) &&
         *bytes <= (size_t)1 << 63;
}

// CTAs of a kernel that the current device holds at once, at most
// kMaxPagedCtas (its shared-memory opt-in is made on the way); asked once per
// device and kernel.
cudaError_t paged_resident_ctas(const void* fn, int threads, size_t smem, int* ctas);

}  // namespace wsvd
