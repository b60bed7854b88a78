// One page of a (page, KV head) block at d = 128 dequantised by NT threads into the tensor cores'
// no-swizzle shared-memory operand of 64 tokens x 128 dims in binary16.
#pragma once

#include "isoq_check.cuh"
#include "isoq_common.cuh"
#include "isoq_ptx.cuh"
#include "isoq_vtile.cuh"

namespace isoq {
using namespace ptx;

constexpr int kPageTile = 64 * 128 * 2;  // bytes

__device__ __forceinline__ void st_v4(uint32_t addr, const uint32_t (&o)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(o[0]), "r"(o[1]),
               "r"(o[2]), "r"(o[3])
               : "memory");
}

// blk: the block in shared memory; tid 0 .. NT-1, whole warps.  kv = 0: K_hat, K-major (B of the scores, N = 64
// tokens): (dim/8) 1024 + (tok/8) 128 + (tok%8) 16 + (dim%8) 2.  kv = 1: V_hat, MN-major (B of
// the value product, K = 64 tokens): (tok/8) 2048 + (dim/8) 128 + (tok%8) 16 + (dim%8) 2.
// Values are ALPHA times the levels; tl0 .. th1 are the format's level tables.
template <int BITS, int NT = 128>
__device__ __forceinline__ void page_tile(const uint8_t* blk, int kv, int tid, uint32_t tile,
                                          uint32_t tl0, uint32_t tl1, uint32_t th0, uint32_t th1,
                                          uint32_t* status) {
  constexpr int D = 128, CB = code_bytes(D, BITS), W = BITS;
#pragma unroll
  for (int hf = 0; hf < (256 + NT - 1) / NT; ++hf) {
    const int u = tid + NT * hf;
    if (256 % NT != 0 && u >= 256) break;
    if (BITS == 3 && kv == 1) {
      // V tile layout: u = (block, quad, 8-dim unit) group of four tokens.  Lanes 4m ..
      // 4m+3 take quads 0-3 of one unit, so a warp's 12-byte group loads hit 32 distinct
      // banks.  A member's 16-byte tile row sits at chunk (2 quad + member bit 0) % 8 of
      // a 128-byte line, the same line for every member of a unit; lanes with an odd unit
      // store their members in the order 1 0 3 2 (nibbles swapped within each byte of
      // the words), so each quarter-warp's stores cover the 8 chunks once.
      const int t4 = u & 3, un = (u >> 2) & 15, B = u >> 6, jf = un & 1;
      const uint32_t* wp = reinterpret_cast<const uint32_t*>(
          blk + v_codes_off(D, BITS) + vt_group_off(D, B, t4, un));
      if (!in_bounds(vt_group_off(D, B, t4, un) + 12 <= kPage * CB, status)) continue;
      const int sh = 4 * jf;
      uint32_t w3[3];
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const uint32_t x = wp[i];
        w3[i] = ((x >> sh) & 0x0F0F0F0Fu) | ((x << sh) & 0xF0F0F0F0u);
      }
      uint32_t o[4][4];
      vdeq_group(w3[0], w3[1], w3[2], tl0, tl1, th0, th1, o);  // o[j]: member j ^ jf
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int tkj = vt_member_slot(B, t4, j ^ jf);
        const int vo = (tkj >> 3) * 2048 + un * 128 + (tkj & 7) * 16;
        if (!in_bounds(vo + 16 <= kPageTile, status)) continue;
        st_v4(tile + vo, o[j]);
      }
      continue;
    }
    // token, 32-dim group: a warp takes 8 tokens x 4 groups, so its 32-bit code loads
    // (word 12 tk + 3 q + i) hit 32 distinct banks and each quarter-warp's 16-byte tile
    // stores 8 distinct bank groups (tk % 8)
    const int tk = 8 * (u >> 5) + (u & 7), q = (u >> 3) & 3;
    const uint32_t* wp = reinterpret_cast<const uint32_t*>(
                             blk + (kv ? v_codes_off(D, BITS) : 0) + tk * CB) + W * q;
    if (!in_bounds(tk * CB + 4 * W * (q + 1) <= kPage * CB, status)) continue;
    uint32_t w[W];
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = wp[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t o[4];
      kdeq<BITS>(w, j, tl0, tl1, th0, th1, o);  // dims 32q + 8j .. +7 of token tk
      const int c = 4 * q + j;
      const uint32_t to = kv ? (tk >> 3) * 2048 + c * 128 + (tk & 7) * 16
                             : c * 1024 + (tk >> 3) * 128 + (tk & 7) * 16;
      if (!in_bounds(to + 16 <= kPageTile, status))
        continue;
      st_v4(tile + to, o);
    }
  }
}

}  // namespace isoq
