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

// One warp per KV head and run of `tokens` <= 32 listed tokens: K, then V of each; lane l holds
// dims l E .. l E + E-1 and the head's blocks of them.  The run's pages are looked up at once, a
// token a lane, and the next token's words are loaded while one is computed.  The shuffles of
// the WHT bound it (20 a vector at d = 128, with the loads ~30 of the load-store pipe's cycles):
// 32768 tokens x 8 heads to fp32 in 107 us (2.8 TB/s), at d = 256 in 208 (2.8 TB/s); 188 with a
// token a warp, which the lookups bounded, 158 with four heads of a token a warp, whose blocks
// were loaded again for each.
constexpr int kDqWarps = 8;
struct HeadWords {  // what a lane needs of a token's K and V codes, and the norms
  uint32_t k[3], v[3];
  uint16_t kn, vn;
  int slot;
  bool live;
};

template <int D, int BITS, typename T, bool ROPE>
__global__ void __launch_bounds__(kDqWarps * 32) dequantize_warp_kernel(const DequantizeArgs a, int tokens) {
  constexpr int E = D / 32, NB = E / 4, CB = code_bytes(D, BITS), BB = block_bytes(D, BITS);
  __shared__ float level[16];  // by the stored field: the code, or the 4-bit sign-magnitude
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid < (1 << BITS))
    level[tid] = BITS == 4 ? (tid < 8 ? mag_f32(4, tid) : -mag_f32(4, tid - 8)) : level_f32(BITS, tid);
  __syncthreads();
  const int h = blockIdx.y, dim = lane * E;
  const long long i0 = ((long long)blockIdx.x * kDqWarps + (tid >> 5)) * tokens;
  const int count = (int)min((long long)tokens, a.n_tokens - i0);
  if (count <= 0) return;
  int my_pos = 0, my_page = -1;  // of token i0 + lane
  if (lane < count) {
    uint32_t bad;
    my_pos = __ldg(a.positions + i0 + lane);
    const long long entry = page_entry(a, __ldg(a.seq_ids + i0 + lane), my_pos, bad);
    if (entry >= 0) my_page = valid_page(a, __ldg(a.page_table + entry), bad);
    if (my_page < 0 && h == 0) set_status(a.status, bad);
  }
  float M[NB][16];
#pragma unroll
  for (int k = 0; k < NB; ++k)
    if (in_bounds(lane * NB + k < D / 4, a.status))
      load_block_mat(a.mats + (size_t)h * D * 4, lane * NB + k, M[k]);
  constexpr int kWords = BITS == 3 ? 3 : 1;
  auto load = [&](int t, HeadWords& w) {
    const int page = __shfl_sync(kFull, my_page, t), slot = __shfl_sync(kFull, my_pos, t) & (kPage - 1);
    w.slot = slot;
    w.live = page >= 0;
    if (page < 0) return;
    // byte offsets of the lane's words in a record (K, and V of 2 and 4 bits) or V tile group
    int B, q, j;
    vt_slot(slot, B, q, j);
    const int k_off = slot * CB + (BITS == 3 ? dim / 32 * 12 : BITS == 4 ? dim / 8 * 4 : dim / 16 * 4);
    const int v_off = BITS == 3 ? vt_group_off(D, B, q, dim / 8) : k_off;
    const uint8_t* blk = a.blocks + ((size_t)page * a.n_kv_heads + h) * BB;
    w.live = in_bounds(k_off + 4 * kWords <= kPage * CB && v_off + 4 * kWords <= kPage * CB, a.status);
    if (!w.live) return;
    if (a.K != nullptr) {
#pragma unroll
      for (int x = 0; x < kWords; ++x) w.k[x] = __ldg(reinterpret_cast<const uint32_t*>(blk + k_off) + x);
      w.kn = __ldg(reinterpret_cast<const uint16_t*>(blk + k_norm_off(D, BITS) + 2 * slot));
    }
    if (a.V != nullptr) {
      const uint8_t* g = blk + v_codes_off(D, BITS) + v_off;
#pragma unroll
      for (int x = 0; x < kWords; ++x) w.v[x] = __ldg(reinterpret_cast<const uint32_t*>(g) + x);
      w.vn = __ldg(reinterpret_cast<const uint16_t*>(blk + v_norm_off(D, BITS) + 2 * slot));
    }
  };
  float sgn[5];  // the lane's side of each cross-lane stage of the WHT
#pragma unroll
  for (int s = 0; s < 5; ++s) sgn[s] = ((lane >> s) & 1) ? -1.f : 1.f;

  HeadWords now, next;
  load(0, now);
#pragma unroll 1
  for (int t = 0; t < count; ++t, now = next) {
    if (t + 1 < count) load(t + 1, next);
    if (!now.live) continue;  // its rows stay as they were
    const int pos = __shfl_sync(kFull, my_pos, t);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      T* out = static_cast<T*>(side ? a.V : a.K);
      if (out == nullptr) continue;
      const uint32_t* w = side ? now.v : now.k;
      const float n = __half2float(__ushort_as_half(side ? now.vn : now.kn));
      // the lane's fields, E nibbles of f
      uint32_t f = 0;
      if (BITS == 3 && side) {
        f = member_unit(w[0], w[1], w[2], (now.slot & 1) | ((now.slot >> 2) & 2)) >> (E == 4 ? 16 * (lane & 1) : 0);
      } else if (BITS == 3) {
        const int u = dim / 8 % 4;
        f = u == 0 ? w[0] : u == 1 ? w[1] : w[2];
        f = u == 3 ? spare_codes(w[0], w[1], w[2]) : f & 0x77777777u;
        if (E == 4) f >>= 16 * (lane & 1);
      } else if (BITS == 4) {
        f = E == 4 ? w[0] >> (16 * (lane & 1)) : w[0];
      } else {
        // slots: dims 2i of the half-word's 8 are slot i, dims 2i + 1 slot i + 4
        const uint32_t x = w[0] >> (16 * (dim / 8 & 1));
        const int i0 = (lane & 1) * 2;  // E = 4: dims 4 (lane & 1) .. + 3
        f = (x >> (2 * i0) & 3u) | (x >> (2 * i0 + 8) & 3u) << 4 | (x >> (2 * i0 + 2) & 3u) << 8 |
            (x >> (2 * i0 + 10) & 3u) << 12;
      }
      float z[E], y[E];
#pragma unroll
      for (int e = 0; e < E; ++e) z[e] = level[f >> (4 * e) & 15u];
#pragma unroll
      for (int k = 0; k < NB; ++k) mat_inv(M[k], z + 4 * k, y + 4 * k);
      wht_signed<E>(y, sgn);
      const float c = n * (1.0f / D);
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] *= c;
      if (ROPE && side == 0) {  // lanes 0-15 hold the first halves of the pairs
        const float4* cs = reinterpret_cast<const float4*>(
            a.rope + ((size_t)pos * (D / 2) + (lane & 15) * E) * 2);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float4 r = __ldg(cs + e / 2);  // (cos, sin) of two pairs
          const float p0 = __shfl_xor_sync(kFull, y[e], 16), p1 = __shfl_xor_sync(kFull, y[e + 1], 16);
          y[e] = fmaf(lane < 16 ? p0 : -p0, r.y, y[e] * r.x);
          y[e + 1] = fmaf(lane < 16 ? p1 : -p1, r.w, y[e + 1] * r.z);
        }
      }
      store_vec<T, E>(out + ((size_t)(i0 + t) * a.n_kv_heads + h) * D + dim, y);
    }
  }
}

template <int D, int BITS, typename T>
cudaError_t launch_warp(const DequantizeArgs& a, cudaStream_t stream, int n_sm) {
  // several tokens a warp as far as that leaves every SM its 32 warps
  const long long pairs = (long long)a.n_tokens * a.n_kv_heads;
  long long tokens = pairs / ((long long)n_sm * 32);
  tokens = tokens < 1 ? 1 : tokens > 16 ? 16 : tokens;
  const long long per_cta = tokens * kDqWarps;
  dim3 grid((unsigned)((a.n_tokens + per_cta - 1) / per_cta), a.n_kv_heads);
  if (a.rope) dequantize_warp_kernel<D, BITS, T, true><<<grid, kDqWarps * 32, 0, stream>>>(a, (int)tokens);
  else dequantize_warp_kernel<D, BITS, T, false><<<grid, kDqWarps * 32, 0, stream>>>(a, (int)tokens);
  return cudaGetLastError();
}

template <int D, int BITS>
cudaError_t launch_t(const DequantizeArgs& a, cudaStream_t stream, int n_sm) {
  switch (a.dtype) {
    case ISOQ_F32: return launch_warp<D, BITS, float>(a, stream, n_sm);
    case ISOQ_BF16: return launch_warp<D, BITS, __nv_bfloat16>(a, stream, n_sm);
    case ISOQ_F16: return launch_warp<D, BITS, __half>(a, stream, n_sm);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_dequantize(const DequantizeArgs& a, cudaStream_t stream, int n_sm) {
  if (use_dequantize_tc(a)) return launch_dequantize_tc(a, stream, n_sm);
  if (a.d == 256) return launch_t<256, 3>(a, stream, n_sm);
  switch (a.bits) {
    case 2: return launch_t<128, 2>(a, stream, n_sm);
    case 3: return launch_t<128, 3>(a, stream, n_sm);
    case 4: return launch_t<128, 4>(a, stream, n_sm);
  }
  return cudaErrorInvalidValue;
}

}  // namespace isoq
