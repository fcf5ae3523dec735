// Where the latent append and prefill put their rows: the contiguous cache
// [B][H][L_cap], or pages of a pool.
#pragma once

#include "common.cuh"
#include "wsvd_internal.h"

namespace wsvd {

struct ContiguousRows {
  static constexpr bool kSplits = false;  // the prefill's tiles are never split over E: its rows keep their bits
  // 0, or the WSVD_DEVERR_* bit for which rows pos .. pos + n - 1 of sequence b are refused.
  __device__ __forceinline__ int refused(int, int pos, int n, int L_cap) const {
    return pos >= 0 && (long long)pos + n <= L_cap ? 0 : WSVD_DEVERR_CACHE_FULL;
  }
  // Row l of sequence b, head h, in the arrays of codes and scales.
  __device__ __forceinline__ size_t row(int b, int h, int H, int l, int L_cap) const {
    return ((size_t)b * H + h) * L_cap + l;
  }
  // The new length of sequence b (pos unless its n rows were written).
  __device__ __forceinline__ void advance(int32_t* seq_lens, int b, int pos, int n, bool written) const {
    if (written) st_relaxed_gpu(seq_lens + b, pos + n);
  }
};

// L_cap is the page table's capacity max_pages << page_shift.
struct PagedRows {
  static constexpr bool kSplits = true;
  const int32_t* block_table;  // [B][max_pages]
  int max_pages, page_shift, num_pages;
  int32_t* seq_lens_out;       // receives every length
  __device__ __forceinline__ int refused(int b, int pos, int n, int L_cap) const {
    if (pos < 0 || (long long)pos + n > L_cap) return WSVD_DEVERR_CACHE_FULL;
    const int32_t* t = block_table + (size_t)b * max_pages;
    bool bad = false;
    const int last = (pos + n - 1) >> page_shift;
#pragma unroll 4
    for (int p = pos >> page_shift; p <= last; ++p) bad |= (uint32_t)t[p] >= (uint32_t)num_pages;
    return bad ? WSVD_DEVERR_PAGE_RANGE : 0;
  }
  __device__ __forceinline__ size_t row(int b, int h, int H, int l, int) const {
    const size_t page = (size_t)block_table[(size_t)b * max_pages + (l >> page_shift)];
    return ((page * H + h) << page_shift) + (l & ((1 << page_shift) - 1));
  }
  __device__ __forceinline__ void advance(int32_t*, int b, int pos, int n, bool written) const {
    st_relaxed_gpu(seq_lens_out + b, written ? pos + n : pos);
  }
};

// The append of launch_append into pages (fp16 weights); a.L_cap is the page
// table's capacity.
cudaError_t launch_append_paged(const AppendArgs& a, const PagedRows& place, cudaStream_t stream);
// wsvd_latent_prefill's checks and launches for rows in pages (a wsvd_status).
int prefill_paged(const PagedRows& place, int B, int T, int H, int E, int r, int bits, int L_cap, int hadamard_block,
                  const void* x, int x_dtype, const void* A_k, const void* A_v, int32_t* seq_lens, uint8_t* lat_k,
                  uint8_t* lat_v, void* scale_k, void* scale_v, void* workspace, size_t workspace_bytes, int32_t* err,
                  void* stream);

}  // namespace wsvd
