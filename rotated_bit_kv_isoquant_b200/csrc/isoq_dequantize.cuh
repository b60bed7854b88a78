// Shared by the read-back kernels: a listed token's page, and one token's codes out of a
// group of the 3-bit V tile layout.
#pragma once

#include "isoq_common.cuh"
#include "isoq_internal.h"
#include "isoq_ptx.cuh"

namespace isoq {

// Index of the page-table entry of (sequence s, position pos), or -1 with the reason's
// status bit in `bad`.
__device__ __forceinline__ long long page_entry(const DequantizeArgs& a, int s, int pos,
                                                uint32_t& bad) {
  bad = 0;
  if (s < 0 || s >= a.n_seqs) bad = ISOQ_ST_SEQ_RANGE;
  else if (pos < 0 || pos / kPage >= a.max_pages || (a.rope && pos >= a.rope_max_pos))
    bad = ISOQ_ST_POS_RANGE;
  return bad ? -1 : (long long)s * a.max_pages + pos / kPage;
}

// The page itself, or -1 with the status bit.
__device__ __forceinline__ int valid_page(const DequantizeArgs& a, int phys, uint32_t& bad) {
  if (phys >= 0 && phys < a.n_pages) return phys;
  bad = ISOQ_ST_PAGE_RANGE;
  return -1;
}

// The unit word (nibble e = the code of dim 8u + e) of member j of a group W0 W1 W2: dims 2b,
// 2b + 1 are the nibbles j and j + 4 of word b, the spare unit's for b = 3.
__device__ __forceinline__ uint32_t member_unit(uint32_t W0, uint32_t W1, uint32_t W2, int j) {
  W0 >>= 4 * j;
  W1 >>= 4 * j;
  W2 >>= 4 * j;
  auto pair = [](uint32_t x) { return (x & 7u) | ((x >> 12) & 0x70u); };
  return pair(W0) | pair(W1) << 8 | pair(W2) << 16 | pair(ptx::spare_codes(W0, W1, W2)) << 24;
}

}  // namespace isoq
