// Where an append puts its rows: the contiguous cache [B][H][L_cap], or pages of
// a pool.
#pragma once

#include "common.cuh"
#include "wsvd_internal.h"

namespace wsvd {

struct ContiguousRows {
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
// A block of T tokens per sequence into pages (paged_prefill.cu): whether it
// takes these sizes, its scratch, and its launches (a.L_cap as above, a.counter
// zero and left zero).
bool paged_block_takes(int B, int T, int H, int E, int r);
size_t paged_block_scratch(int B, int T, int E);
cudaError_t launch_paged_block(const AppendArgs& a, int T, const PagedRows& place, void* scratch, cudaStream_t stream);

}  // namespace wsvd
