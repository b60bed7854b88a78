// Sliding-window attention with sinks: which tokens a query row sees, and which pages of a
// sequence a CTA has to read for its rows.
//
// A row whose causal limit is lim (it sits at position lim - 1) sees the tokens
//   t in [max(0, lim - W), lim)   its window of W tokens, itself among them
//   t in [0, min(S, lim))         the first S tokens of the sequence, the sinks.
// A CTA's rows have limits lim_lo .. lim_hi, so the tokens that any of them sees lie in
// the pages of [0, min(S, lim_hi)) and of [max(0, lim_lo - W), lim_hi).  The pages between
// the two runs are never read and their page-table entries never used: a caller may have
// recycled them.  A CTA numbers the pages it has to visit 0 .. n-1 (slots); page() gives
// the sequence's page of a slot.
#pragma once

#include <stdint.h>

#include "isoq_common.cuh"
#include "isoq_internal.h"

namespace isoq {

// By value to the kernels compiled with WIN; ignored by the others.
struct WinArgs {
  int window;     // W >= 1
  int n_sinks;    // S >= 0
  int max_len;    // the host's bound of the sequence lengths (the split plan's)
  int out_dtype;  // element type of the output rows (ISOQ_F32, ISOQ_BF16, ISOQ_F16)
};

inline WinArgs win_args(const DecodeArgs& a) {
  return WinArgs{a.window, a.n_sinks, a.max_len, a.out_dtype};
}

template <bool WIN>
struct WinPages {
  int sink_pages = 0, skip = 0;  // slots before the gap, pages in the gap
  int n_slots;                   // pages to visit
  int lo_min = 0, lo_max = 0;    // first window token of the first / last row
  __device__ WinPages(const WinArgs& w, int lim_lo, int lim_hi) {
    n_slots = (lim_hi + kPage - 1) / kPage;
    if constexpr (WIN) {
      lo_min = max(0, lim_lo - w.window);
      lo_max = max(0, lim_hi - w.window);
      sink_pages = (min(w.n_sinks, lim_hi) + kPage - 1) / kPage;
      skip = max(0, lo_min / kPage - sink_pages);
      n_slots -= skip;
    }
  }
  __device__ __forceinline__ int page(int slot) const {
    return !WIN || slot < sink_pages ? slot : slot + skip;
  }
  // every row sees all 64 tokens of the page that starts at tok0 (the causal side of the
  // test is the caller's)
  __device__ __forceinline__ bool page_full(const WinArgs& w, int tok0) const {
    return !WIN || tok0 >= lo_max || kPage <= w.n_sinks - tok0;
  }
  // some row sees token t (causal side: the caller's)
  __device__ __forceinline__ bool any_sees(const WinArgs& w, int t) const {
    return !WIN || t >= lo_min || t < w.n_sinks;
  }
};

// The first window token of a row with causal limit lim.
template <bool WIN>
__device__ __forceinline__ int win_lo(const WinArgs& w, int lim) {
  return WIN ? max(0, lim - w.window) : 0;
}
// The row with first window token lo sees token t (causal side: the caller's).
template <bool WIN>
__device__ __forceinline__ bool win_sees(const WinArgs& w, int lo, int t) {
  return !WIN || t >= lo || t < w.n_sinks;
}

// A sequence's length as the kernels use it: clamped to the page table, and with a window
// to the bound that the split plan was made for and to 2^31 - 64, up to which the positions of
// its last page and the one behind it are ints (each sets ISOQ_ST_LEN_RANGE).
template <bool WIN>
__device__ __forceinline__ int clamp_len(int len, int max_pages, const WinArgs& w, bool report,
                                         uint32_t* status) {
  int most = max_pages * kPage;
  if constexpr (WIN)
    most = (int)min((long long)min(w.max_len, 0x7FFFFFFF - (kPage - 1)), (long long)max_pages * kPage);
  if (len > most) {
    if (report) set_status(status, ISOQ_ST_LEN_RANGE);
    len = most;
  }
  return WIN ? max(len, 0) : len;
}

// One output element in the caller's type (rounded to nearest once).
__device__ __forceinline__ void store_typed(void* out, size_t i, float v, int dtype) {
  if (dtype == ISOQ_F32) static_cast<float*>(out)[i] = v;
  else if (dtype == ISOQ_BF16) static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(out)[i] = __float2half_rn(v);
}

}  // namespace isoq
