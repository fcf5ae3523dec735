// Device helpers shared by the sm_100a kernels: mbarrier + 1-D bulk-copy (TMA)
// staging with bounded waits, and exact integer -> float32 code conversion.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "wsvd_internal.h"

namespace wsvd {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_huge_valf();

// ---------------------------------------------------------------- shared memory / mbarrier
__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void fence_mbar_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
               : "memory");
}

// Adds expected transaction bytes without arriving (the phase cannot complete
// before the owner's arrive, which may come later with more bytes).
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ uint64_t globaltimer_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// Wait for phase `parity` of an mbarrier, giving up after `limit_ns` of wall
// time.  Returns false on timeout; the caller records WSVD_DEVERR_PIPE_TIMEOUT
// and leaves the pipeline instead of spinning forever.
__device__ __forceinline__ bool mbar_wait_bounded(uint64_t* bar, uint32_t parity,
                                                  uint64_t limit_ns = kWaitLimitNs) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (globaltimer_ns() - t0 > limit_ns) return false;
  }
}

// Address of `p` (this CTA's shared memory) in the shared window of cluster
// CTA `rank`, as a shared::cluster address.
__device__ __forceinline__ uint32_t mapa_shared(const void* p, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}

// 4-byte store into another cluster CTA's shared memory that completes 4
// bytes of transaction count on that CTA's mbarrier (both shared::cluster
// addresses).  Once the barrier phase completes the value is visible to the
// waiting CTA; no fence is needed on either side.
__device__ __forceinline__ void st_async_f32(uint32_t remote_addr, float v, uint32_t remote_bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(remote_addr),
               "r"(__float_as_uint(v)), "r"(remote_bar)
               : "memory");
}

// Bounded wait (cluster-scope acquire) for phase `parity` of a barrier that
// other CTAs of the cluster complete.  Returns false on timeout.
__device__ __forceinline__ bool mbar_wait_cluster_bounded(uint64_t* bar, uint32_t parity,
                                                          uint64_t limit_ns = kWaitLimitNs) {
  const uint32_t addr = smem_u32(bar);
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(addr), "r"(parity)
        : "memory");
    if (done) return true;
    if (globaltimer_ns() - t0 > limit_ns) return false;
  }
}

// 1-D bulk copy global -> this CTA's shared memory, completing `bytes` of
// transaction count on `bar`.  Both addresses 16-byte aligned, bytes % 16 == 0.
// No multicast: the destination is this CTA only.
__device__ __forceinline__ void bulk_g2s(void* smem_dst, const void* gsrc, uint32_t bytes, uint64_t* bar,
                                         uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
          smem_u32(smem_dst)),
      "l"(gsrc), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// Warp-level forms of the two calls above: every lane of a converged warp
// executes the call with the same operands and one elected lane issues it
// (issued from a lone lane behind a divergent branch, each costs far more).
__device__ __forceinline__ void mbar_arrive_expect_tx_warp(uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "r"(bytes)
      : "memory");
}
__device__ __forceinline__ void bulk_g2s_warp(void* smem_dst, const void* gsrc, uint32_t bytes, uint64_t* bar,
                                              uint64_t policy) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], "
      "%4;\n\t}" ::"r"(smem_u32(smem_dst)),
      "l"(gsrc), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// L2 policy for data read exactly once (latent / KV streams): evict first, so
// the small reused operands (B matrices, q) stay resident.
__device__ __forceinline__ uint64_t l2_evict_first_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// L2 policy for small operands many CTAs re-read (B matrices, q): keep them.
__device__ __forceinline__ uint64_t l2_evict_last_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// Programmatic dependent launch.  griddep_wait: returns once the grid this
// one was launched behind (programmatic stream serialisation) has completed
// and its memory is visible; a no-op for a normal launch.
// griddep_launch_dependents: lets the dependent grid be scheduled before this
// one completes (it still waits in griddep_wait for the data).
__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void griddep_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Explicit shared-memory loads (32-bit shared addresses).  volatile: they stay
// after the mbarrier waits that make the staged bytes visible.
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ float lds_half_as_float(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return __half2float(__ushort_as_half(v));
}

// Cluster-wide barrier in two halves.  The arrive is relaxed: it only orders
// the mbarrier initialisations, which fence_mbar_init has already released
// at cluster scope; the wait acquires.
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

__device__ __forceinline__ void named_barrier_sync(int id, int nthreads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

// The larger of amax and |x|, as integers: a NaN lies above infinity and stays,
// where fmaxf drops it.  For the largest latent of a row, whose scale then is NaN.
__device__ __forceinline__ float max_abs(float amax, float x) {
  return __int_as_float(max(__float_as_int(amax), __float_as_int(fabsf(x))));
}

// gpu-scope acquire load (a completion counter that other CTAs bump after a
// release of their data).
__device__ __forceinline__ int ld_acquire_gpu(const int32_t* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ int ld_relaxed_gpu(const int32_t* p) {
  int v;
  asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_relaxed_gpu(int32_t* p, int v) {
  asm volatile("st.relaxed.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// Returns the previous value; release orders this thread's (and, after a CTA
// barrier, the CTA's) earlier accesses before the add, acquire the later ones.
__device__ __forceinline__ int atom_add_acq_rel_gpu(int32_t* p, int v) {
  int old;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

__device__ __forceinline__ void set_err(int32_t* err, int32_t bits) {
  if (err) atomicOr(err, bits);
}

// 2^x on the MUFU unit (flushes denormal results to zero; 2^-inf = 0).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 4-way byte dot products with 32-bit accumulate: d = c + sum_i a.byte_i * b.byte_i.
// Suffixes give the signedness of the bytes of a, then b.
__device__ __forceinline__ int dp4a_ss(uint32_t a, uint32_t b, int c) {
  int d;
  asm("dp4a.s32.s32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ int dp4a_su(uint32_t a, uint32_t b, int c) {
  int d;
  asm("dp4a.s32.u32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ int dp4a_us(uint32_t a, uint32_t b, int c) {
  int d;
  asm("dp4a.u32.s32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ int dp4a_uu(uint32_t a, uint32_t b, int c) {
  int d;
  asm("dp4a.u32.u32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// ---------------------------------------------------------------- code conversion
// int8 codes -> float32, exact.  Each byte is moved into the low mantissa byte
// of 2^23 (after flipping its sign bit, so it reads as c + 128); subtracting
// 2^23 + 128 leaves c exactly (IEEE-754 layout: integers below 2^24 are exact).
__device__ __forceinline__ float2 i8_pair(uint32_t xflip, int first) {
  const uint32_t sel0 = 0x7540u | (uint32_t)first;
  const uint32_t sel1 = 0x7540u | (uint32_t)(first + 1);
  float2 f;
  f.x = __uint_as_float(__byte_perm(xflip, 0x4B000000u, sel0));
  f.y = __uint_as_float(__byte_perm(xflip, 0x4B000000u, sel1));
  return __fadd2_rn(f, make_float2(-8388736.f, -8388736.f));
}

// int4 codes (two's complement nibbles, element k in bits 4k..4k+3 of the word)
// -> float32, exact.  Same mantissa trick with offset 8.
__device__ __forceinline__ float2 i4_pair(uint32_t xflip, int k) {
  float2 f;
  f.x = __uint_as_float(((xflip >> (4 * k)) & 0xFu) | 0x4B000000u);
  f.y = __uint_as_float(((xflip >> (4 * k + 4)) & 0xFu) | 0x4B000000u);
  return __fadd2_rn(f, make_float2(-8388616.f, -8388616.f));
}

// Element idx of a B matrix stored as fp16 or (w8) as int8, as float32 (exact).
__device__ __forceinline__ float bmat_elem(const void* base, int w8, size_t idx) {
  return w8 ? (float)static_cast<const int8_t*>(base)[idx] : __half2float(static_cast<const __half*>(base)[idx]);
}

__device__ __forceinline__ float2 h2_pair(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

__device__ __forceinline__ float load_q_elem(const void* q, int dtype, size_t i) {
  const uint16_t u = reinterpret_cast<const uint16_t*>(q)[i];
  if (dtype == WSVD_DTYPE_BF16) return __uint_as_float(((uint32_t)u) << 16);
  return __half2float(__ushort_as_half(u));
}

}  // namespace wsvd
