// End of a windowed decode whose context chunks are the CTAs of one cluster (or one CTA): each
// CTA leaves the merged state of its rows in shared memory, the cluster's CTAs share the rows
// out, and the one that has a row merges its states by log-sum-exp over distributed shared
// memory, divides, rotates back and writes it.  No partial results in global memory and no
// second kernel.
#pragma once

#include <math_constants.h>

#include "isoq_check.cuh"
#include "isoq_common.cuh"
#include "isoq_ptx.cuh"
#include "isoq_window.cuh"

namespace isoq {

// Floats of a row's state in shared memory: acc[D] relative to the maximum, l, the maximum in
// log2 units (-inf: no token), padding to 16 bytes.
template <int D>
constexpr int finish_stride() { return D + 4; }

__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return (int)r;
}

// All threads of the cluster's CTAs; orders their shared-memory accesses.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// The address of this CTA's shared-memory address in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// fin: [nh][finish_stride] in shared memory, complete for this CTA up to a barrier.  n_parts
// CTAs (1: no cluster).  Every thread of every CTA calls this.
template <int D, int NW>
__device__ __forceinline__ void finish_rows(const float* fin, int nh, int n_parts,
                                            const int* row_off, const float* __restrict__ head_mats,
                                            void* __restrict__ out, size_t seq_row,
                                            [[maybe_unused]] size_t out_rows, int out_dtype,
                                            uint32_t* status) {
  constexpr int E = D / 32, NB = E / 4, FS = finish_stride<D>();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = n_parts > 1 ? cluster_rank() : 0;
  float M[NB][16];
  if (warp * n_parts + rank < nh) {
#pragma unroll
    for (int k = 0; k < NB; ++k) load_block_mat(head_mats, lane * NB + k, M[k]);
  }
  if (n_parts > 1) cluster_sync();
  else __syncthreads();
  for (int h = warp * n_parts + rank; h < nh; h += NW * n_parts) {
    const uint32_t at = ptx::smem_u32(fin + h * FS);
    float top = -CUDART_INF_F, l = 0.f, o[E];
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = 0.f;
#pragma unroll 2
    for (int p = 0; p < n_parts; ++p) {
      const uint32_t a = n_parts > 1 ? in_cta(at, p) : at;
      const float2 lm = ld_cluster2(a + D * 4);
      float4 v[NB];
#pragma unroll
      for (int k = 0; k < NB; ++k) v[k] = ld_cluster4(a + (lane * E + 4 * k) * 4);
      if (lm.y == -CUDART_INF_F) continue;
      const float now = fmaxf(top, lm.y);
      const float r = ptx::ex2(top - now), f = ptx::ex2(lm.y - now);  // top = -inf: 0
      top = now;
      l = fmaf(l, r, lm.x * f);
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        o[4 * k] = fmaf(o[4 * k], r, v[k].x * f);
        o[4 * k + 1] = fmaf(o[4 * k + 1], r, v[k].y * f);
        o[4 * k + 2] = fmaf(o[4 * k + 2], r, v[k].z * f);
        o[4 * k + 3] = fmaf(o[4 * k + 3], r, v[k].w * f);
      }
    }
    float y[E];
#pragma unroll
    for (int k = 0; k < NB; ++k) mat_inv(M[k], o + 4 * k, y + 4 * k);
    wht_warp<E>(y, lane);
    // divided by l, the WHT's and the levels' 1 / sqrt(d) each
    const float f = l > 0.f ? 1.f / (l * (float)D) : 0.f;
    const size_t row = seq_row + row_off[h];
    if (!in_bounds(row < out_rows, status)) continue;
    const size_t ob = row * D + lane * E;
#pragma unroll
    for (int i = 0; i < E; ++i) store_typed(out, ob + i, y[i] * f, out_dtype);
  }
  if (n_parts > 1) cluster_sync();  // no CTA leaves while its rows are read
}

}  // namespace isoq
