// Read-back of cached vectors: the packed codes of listed tokens turned back into K and V.
//
//   x = (n / sqrt(d)) R^T L[c],  R^T = (orthonormal WHT) (block-diagonal M^T),
// i.e. per vector the level of every code, the transposed 4x4 blocks, an unnormalised WHT and
// one factor n / d.  With a rotary table, the embedding that the append applied to K is taken
// off again: (a, b) = dims (i, i + d/2) -> (a cos + b sin, b cos - a sin).
#include "isoq_check.cuh"
#include "isoq_common.cuh"
#include "isoq_dequantize.cuh"
#include "isoq_internal.h"
#include "isoq_ptx.cuh"
#include "isoq_vtile.cuh"

namespace isoq {
using namespace ptx;
namespace {

template <typename T, int E>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[E]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < E; i += 4)
      *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
    uint32_t w[E / 2];
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      if constexpr (sizeof(T) == 2 && __is_same(T, __half)) {
        w[i / 2] = pack_f16x2(v[i], v[i + 1]);
      } else {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[i], v[i + 1]);
        w[i / 2] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
    if constexpr (E == 4) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// One warp per (token, KV head): K, then V; lane l holds dims l E .. l E + E-1.
constexpr int kDqWarps = 8;
template <int D, int BITS, typename T>
__global__ void __launch_bounds__(kDqWarps * 32) dequantize_warp_kernel(const DequantizeArgs a) {
  constexpr int E = D / 32, NB = E / 4, CB = code_bytes(D, BITS), BB = block_bytes(D, BITS);
  __shared__ float level[16];  // by the stored field: the code, or the 4-bit sign-magnitude
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid < (1 << BITS))
    level[tid] = BITS == 4 ? (tid < 8 ? mag_f32(4, tid) : -mag_f32(4, tid - 8)) : level_f32(BITS, tid);
  __syncthreads();
  const int h = blockIdx.y, i = blockIdx.x * kDqWarps + (tid >> 5);
  if (i >= a.n_tokens) return;
  uint32_t bad;
  const int pos = __ldg(a.positions + i);
  const long long entry = page_entry(a, __ldg(a.seq_ids + i), pos, bad);
  const int phys = entry < 0 ? -1 : valid_page(a, __ldg(a.page_table + entry), bad);
  if (phys < 0) {
    if (lane == 0 && h == 0) set_status(a.status, bad);
    return;
  }
  const int slot = pos & (kPage - 1);
  const uint8_t* blk = a.blocks + ((size_t)phys * a.n_kv_heads + h) * BB;
  float M[NB][16];
#pragma unroll
  for (int k = 0; k < NB; ++k)
    if (in_bounds(lane * NB + k < D / 4, a.status))
      load_block_mat(a.mats + (size_t)h * D * 4, lane * NB + k, M[k]);
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    T* out = static_cast<T*>(side ? a.V : a.K);
    if (out == nullptr) continue;
    const uint8_t* codes = blk + (side ? v_codes_off(D, BITS) : 0);
    const float n = half_at(blk + (side ? v_norm_off(D, BITS) : k_norm_off(D, BITS)) + 2 * slot);
    // the lane's fields, E nibbles of f
    uint32_t f = 0;
    const int dim = lane * E;
    if (BITS == 3 && side) {
      int B, t, j;
      vt_slot(slot, B, t, j);
      const int go = vt_group_off(D, B, t, dim / 8);
      if (!in_bounds(go + 12 <= kPage * CB, a.status)) continue;
      const uint32_t* g = reinterpret_cast<const uint32_t*>(codes + go);
      const uint32_t U = member_unit(__ldg(g), __ldg(g + 1), __ldg(g + 2), j);
      f = U >> (E == 4 ? 16 * (lane & 1) : 0);
    } else if (BITS == 3) {
      const int go = slot * CB + dim / 32 * 12;
      if (!in_bounds(go + 12 <= kPage * CB, a.status)) continue;
      const uint32_t* g = reinterpret_cast<const uint32_t*>(codes + go);
      const uint32_t w0 = __ldg(g), w1 = __ldg(g + 1), w2 = __ldg(g + 2);
      const int u = dim / 8 % 4;
      f = u == 0 ? w0 : u == 1 ? w1 : w2;
      f = u == 3 ? spare_codes(w0, w1, w2) : f & 0x77777777u;
      if (E == 4) f >>= 16 * (lane & 1);
    } else if (BITS == 4) {
      const int go = slot * CB + dim / 8 * 4;
      if (!in_bounds(go + 4 <= kPage * CB, a.status)) continue;
      f = __ldg(reinterpret_cast<const uint32_t*>(codes + go));
      if (E == 4) f >>= 16 * (lane & 1);
    } else {
      const int go = slot * CB + dim / 16 * 4;
      if (!in_bounds(go + 4 <= kPage * CB, a.status)) continue;
      // slots: dims 2i of the half-word's 8 are slot i, dims 2i + 1 slot i + 4
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(codes + go)) >> (16 * (dim / 8 & 1));
      const int i0 = (lane & 1) * 2;  // E = 4: dims 4 (lane & 1) .. + 3
      f = (w >> (2 * i0) & 3u) | (w >> (2 * i0 + 8) & 3u) << 4 | (w >> (2 * i0 + 2) & 3u) << 8 |
          (w >> (2 * i0 + 10) & 3u) << 12;
    }
    float z[E], y[E];
#pragma unroll
    for (int e = 0; e < E; ++e) z[e] = level[f >> (4 * e) & 15u];
#pragma unroll
    for (int k = 0; k < NB; ++k) mat_inv(M[k], z + 4 * k, y + 4 * k);
    wht_warp<E>(y, lane);
    const float c = n * (1.0f / D);
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] *= c;
    if (a.rope && side == 0) {  // lanes 0-15 hold the first halves of the pairs
      const float* cs = a.rope + ((size_t)pos * (D / 2) + (lane & 15) * E) * 2;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float other = __shfl_xor_sync(kFull, y[e], 16);
        const float2 r = __ldg(reinterpret_cast<const float2*>(cs) + e);
        y[e] = fmaf(lane < 16 ? other : -other, r.y, y[e] * r.x);
      }
    }
    store_vec<T, E>(out + ((size_t)i * a.n_kv_heads + h) * D + dim, y);
  }
}

template <int D, int BITS, typename T>
cudaError_t launch_warp(const DequantizeArgs& a, cudaStream_t stream) {
  dim3 grid((unsigned)(((long long)a.n_tokens + kDqWarps - 1) / kDqWarps), a.n_kv_heads);
  dequantize_warp_kernel<D, BITS, T><<<grid, kDqWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int D, int BITS>
cudaError_t launch_t(const DequantizeArgs& a, cudaStream_t stream) {
  switch (a.dtype) {
    case ISOQ_F32: return launch_warp<D, BITS, float>(a, stream);
    case ISOQ_BF16: return launch_warp<D, BITS, __nv_bfloat16>(a, stream);
    case ISOQ_F16: return launch_warp<D, BITS, __half>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_dequantize(const DequantizeArgs& a, cudaStream_t stream, int n_sm) {
  if (use_dequantize_tc(a)) return launch_dequantize_tc(a, stream, n_sm);
  if (a.d == 256) return launch_t<256, 3>(a, stream);
  switch (a.bits) {
    case 2: return launch_t<128, 2>(a, stream);
    case 3: return launch_t<128, 3>(a, stream);
    case 4: return launch_t<128, 4>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace isoq
