// Sliding-window attention of a chunk of query tokens with many rows per KV head (d = 128) on
// the 5th-generation tensor cores, its steps on warps of their own.
//
// As in the other attention kernels the queries are rotated once, scores and value sum run on
// codebook levels in the rotated space, and a row is a (query token, query head) pair; what a
// row sees is isoq_window.cuh's.  One CTA per SM of 16 warps works on one context chunk of one
// KV head:
//   warps 8-11   take the page blocks from a 2-stage ring (1-D bulk copies), dequantise K_hat into
//                f16 operand tiles and give the page's norms
//   warps 13-15  dequantise V_hat
//   warp 12      one thread issues the products: scores S = Q~hi K_hat^T + Q~lo K_hat^T and
//                O += P' V_hat, accumulators in tensor memory
//   warps 0-3,   softmax: thread r owns row r of its half (tensor-memory lane r), reads its 64
//   warps 4-7    scores, keeps its running maximum and sum, writes P' = p |v| / sigma, sigma the
//                largest |v| that a row of the CTA sees; lift_bits says what is done for a row that
//                sees much smaller ones
// With more than 128 rows per KV head the two softmax halves hold two blocks of 128 rows and
// share every page's tiles (256 rows for one dequantisation); with fewer both hold the same
// rows and take the pages in turn, and their states are merged at the end.  So one half's
// softmax runs while the other half's products do, and the next page is dequantised
// meanwhile; all hand-offs are mbarriers with bounded waits, none a CTA barrier.
//
// The score queries keep an f16 high and low part, the weights P' are f16 with f32
// accumulators, statistics are f32 (as in the multi-token kernel, whose error bounds hold).
// A call whose rows' pages fit one chunk divides, rotates back and writes its output here.
// Otherwise partial states go to the combine.
//
// Measured (64 query / 8 KV heads, window 4096): 2048 query tokens of one sequence 540 us (509
// TFLOP/s of scores and values, the low query part not counted), 574 where most norms are a
// twentieth of the first ones and rows are lifted; 16 tokens of 8 sequences 71 us.
// A page of 256 rows takes ~3900 cycles, of which a softmax warp computes ~2500: its latency
// bounds the kernel (issue 48% of the cycles, tensor pipe 35%, exponent unit 25%).  Why this
// split: one CTA of 128 threads doing the steps in turn, two per SM, took 1266 us; the score
// products read A and B from shared memory (48 cycles of its bandwidth for 32 of the tensor
// core), so 256 rows share a page's tiles, and the next page's scores are issued before this
// page's value products.
#include <math_constants.h>

#include <type_traits>

#include "isoq_check.cuh"
#include "isoq_common.cuh"
#include "isoq_internal.h"
#include "isoq_pagetile.cuh"
#include "isoq_ptx.cuh"
#include "isoq_tc.cuh"
#include "isoq_window.cuh"

namespace isoq {
using namespace ptx;
namespace {

constexpr int kWD = 128;
constexpr int kWWarps = 16, kWThreads = kWWarps * 32;
constexpr int kWK = 128, kWV = 96;  // threads that dequantise K_hat (and the norms), V_hat
// tensor-memory columns: S 64, P' 32 and O 128 of each half
constexpr uint32_t kWCols = 512;
__device__ __forceinline__ constexpr uint32_t col_s(int w) { return 64 * w; }
__device__ __forceinline__ constexpr uint32_t col_p(int w) { return 128 + 32 * w; }
__device__ __forceinline__ constexpr uint32_t col_o(int w) { return 256 + 128 * w; }

// The weights p |v| / sigma go to the value product as binary16, whose subnormals below 2^-14 cost
// them bits, and sigma is the largest |v| of the tokens that any row of the CTA sees.  For a row
// that sees much smaller ones the reference is sigma / 2^bits instead, near the row's own largest,
// by keeping p 2^bits for p: its running maximum is `bits` lower, sums and outputs divide by it.
// Weights reach 2^(kLazy + kLift) kSigmaSlack = 2^15 at most, and a subnormal's half step is at
// most 2^-25 of the row's largest |v| times its largest p: kLift pays for norms down to sigma / 8,
// which need no lift.
constexpr float kLift = 3.f;
constexpr float kSpreadNorms = 8.f;  // 2^kLift
// The bits for a tile or page whose tokens that the row sees have norms of at most v (0: none);
// `bits` as before, if it still does.
__device__ __forceinline__ float lift_bits(float v, float sigma, float bits) {
  const float ref = sigma * ex2(-bits);
  if (v > 0.f && ref <= kSpreadNorms * v && v <= kSigmaSlack * ref) return bits;
  // a power of two above sigma / v, by the exponents
  const int over = (int)(__float_as_uint(sigma) >> 23) - (int)(__float_as_uint(v) >> 23) + 1;
  return v > 0.f && sigma > kSpreadNorms * v ? (float)over : 0.f;
}

// A page as the softmax takes it: it has data; some row may need a lift on it (lift_bits: a token
// that some row sees has |v| < sigma / kSpreadNorms); none does, but on the half's page before.
enum PageState { kValid = 1, kSpread = 2, kLevel = 4 };
enum Bar {  // mbarriers: of the ring (2), the tile stages (up to 4), the softmax halves (2)
  kRing = 0, kKFull = 2, kVFull = 6, kKFree = 10, kVFree = 14,
  kSFull = 18, kSRead = 20, kPFull = 22, kPvDone = 24, kDrain = 26, kBars = 27
};

template <int BITS>
struct WinSmem {
  static constexpr int kBB = block_bytes(kWD, BITS);
  // at 0: the queries, [2 halves][hi, lo], at the end the halves' merge
  // (k-groups 2048 + 16 bytes apart, so that a row's 8-byte stores spread over the banks)
  static constexpr int kQGroup = 2064, kQPart = 16 * kQGroup;
  static_assert(kQPart % 256 == 0, "the tiles behind the queries start on 256 bytes");
  static constexpr int kOffK = 4 * kQPart;              // [2] K_hat tiles
  static constexpr int kOffV = kOffK + 2 * kPageTile;   // [2] V_hat tiles
  static constexpr int kOffRing = kOffV + 2 * kPageTile;
  static constexpr int kOffNorm = kOffRing + 2 * kBB;   // float [4 stages][64 K | 64 V]
  static constexpr int kOffMeta = kOffNorm + 4 * 128 * 4;  // float [4] sigma, int [4] PageState,
                                                        // float [4] largest |v| that a row sees
  static constexpr int kOffRed = kOffMeta + 48;         // float2 [2]
  static constexpr int kOffMl = kOffRed + 16;           // float2 [2 halves][128]: m, l
  static constexpr int kOffRow = kOffMl + 256 * 8;      // int [256]: output row of each row
  static constexpr int kOffUnit = kOffRow + 256 * 4;    // float [256]: query_exponent's 2^e by softmax thread
  static constexpr int kOffBar = kOffUnit + 256 * 4;
  static constexpr int kOffTmem = kOffBar + kBars * 8 + 8;
  static constexpr int kBytes = kOffTmem + 16;
  static_assert(kOffRing % 16 == 0 && kBB % 16 == 0 && kOffBar % 8 == 0 && kOffNorm % 16 == 0, "");
  static_assert(kBytes <= 227 * 1024, "shared memory");
  // one row block leaves the second half's query tiles free: two more tile stages
  static_assert(4 * kPageTile <= 2 * kQPart, "stages 2 and 3");
};

template <typename TQ, int BITS>
__global__ void __launch_bounds__(kWThreads, 1)
    window_tc_kernel(const float* __restrict__ params, const uint8_t* __restrict__ blocks,
                     const int32_t* __restrict__ page_table, int n_pages, int max_pages, int H,
                     const TQ* __restrict__ Q, int n_q_heads, int n_q,
                     const int32_t* __restrict__ seq_lens, float scale, int pages_per_split,
                     int n_splits, float* __restrict__ partials, void* __restrict__ out,
                     uint32_t* status, const WinArgs win) {
  using SM = WinSmem<BITS>;
  constexpr int D = kWD, E = D / 32, PS = D + 4, BB = SM::kBB;
  constexpr float ALPHA = alpha_of<BITS>();
  constexpr uint32_t kIdS = tc::idesc_f16(128, 64, false, false);  // scores
  constexpr uint32_t kIdO = tc::idesc_f16(128, 128, false, true);  // value product
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SM::kOffBar);
  float* nrm = reinterpret_cast<float*>(smem + SM::kOffNorm);
  float* sig = reinterpret_cast<float*>(smem + SM::kOffMeta);
  int* valid = reinterpret_cast<int*>(smem + SM::kOffMeta) + 4;
  float* top = reinterpret_cast<float*>(smem + SM::kOffMeta) + 8;
  float2* red = reinterpret_cast<float2*>(smem + SM::kOffRed);
  float2* ml = reinterpret_cast<float2*>(smem + SM::kOffMl);
  int* row_off = reinterpret_cast<int*>(smem + SM::kOffRow);
  float* unit = reinterpret_cast<float*>(smem + SM::kOffUnit);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM::kOffTmem);
  const uint32_t sQ = smem_u32(smem), sK = smem_u32(smem + SM::kOffK), sV = smem_u32(smem + SM::kOffV);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = blockIdx.x, s = blockIdx.z;
  const int G = n_q_heads / H;
  const int n_rows = n_q * G;
  const bool two = n_rows > 128;                 // two row blocks that share the pages
  const int rows_cta = two ? 256 : 128;
  const int n_groups = (n_rows + rows_cta - 1) / rows_cta;
  const int hk = blockIdx.y / n_groups, row0 = (blockIdx.y - hk * n_groups) * rows_cta;
  const int nh = min(rows_cta, n_rows - row0);   // rows handled here
  auto row_index = [&](int r) {                  // row of the sequence's output / partials
    const int R = row0 + r;
    return (R / G) * n_q_heads + hk * G + R % G;
  };

  const int len = clamp_len<true>(__ldg(seq_lens + s), max_pages, win,
                                  tid == 0 && split == 0 && blockIdx.y == 0, status);
  auto lim_of = [&](int r) { return max(0, min(len, len - n_q + 1 + (row0 + r) / G)); };
  const int lim_lo = lim_of(0), lim_hi = lim_of(nh - 1);
  const WinPages<true> wp(win, lim_lo, lim_hi);
  const int p_begin = split * pages_per_split;   // slots of the pages to visit
  const int n = min(wp.n_slots, p_begin + pages_per_split) - p_begin;
  float* out_base = partials + ((size_t)s * n_q * n_q_heads) * n_splits * PS + (size_t)split * PS;
  const size_t seq_row = (size_t)s * n_q * n_q_heads;
  if (n <= 0) {  // empty: zero rows, or m = -inf, l = 0, acc = 0
    if (out != nullptr) {
      for (int i = tid; i < nh * D; i += kWThreads) {
        const int r = row_index(i / D);
        if (in_bounds(r < n_q * n_q_heads, status))
          store_typed(out, (seq_row + r) * D + i % D, 0.f, win.out_dtype);
      }
    } else {
      for (int i = tid; i < nh * PS; i += kWThreads) {
        const int r = row_index(i / PS), c = i % PS;
        if (in_bounds(r < n_q * n_q_heads, status))
          out_base[(size_t)r * n_splits * PS + c] = c == D ? -CUDART_INF_F : 0.f;
      }
    }
    return;
  }
  const int* pt_row = page_table + (size_t)s * max_pages;
  auto entry_of = [&](int k) {  // page-table entry of page k of the chunk, as it is
    const int pg = wp.page(p_begin + k);
    return k < n && in_bounds(pg < max_pages, status) ? __ldg(pt_row + pg) : -1;
  };

  // ---- tensor memory, barriers, the first two pages ------------------------------------
  if (warp == 12) tc::alloc(tmem_slot, kWCols);
  auto issue = [&](int k, int ph) {  // one thread
    const int st = k & 1;
    if (ph >= 0 && ph < n_pages) {
      mbar_expect_tx(bars + kRing + st, BB);
      bulk_copy(smem + SM::kOffRing + st * BB, blocks + ((size_t)ph * H + hk) * BB, BB, bars + kRing + st);
    } else {
      set_status(status, ISOQ_ST_PAGE_RANGE);
      mbar_arrive(bars + kRing + st);  // complete the phase without data; the page is masked
    }
  };
  if (tid == 256) {
    for (int i = 0; i < kBars; ++i) {
      // arrivals: the K threads; theirs (norms) and the V threads; a softmax half; else one
      mbar_init(bars + i, i >= kKFull && i < kVFull   ? kWK
                          : i >= kVFull && i < kKFree ? kWK + kWV
                          : i >= kSRead && i < kPvDone ? 128 : 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    issue(0, entry_of(0));
    if (n > 1) issue(1, entry_of(1));
  }

  if (tid < 256) {
    row_off[tid] = tid < nh ? row_index(tid) : n_q * n_q_heads;
    unit[tid] = 1.f;
  }
  float sgn[5];  // the lane's side of each cross-lane stage of the WHT
#pragma unroll
  for (int i = 0; i < 5; ++i) sgn[i] = ((lane >> i) & 1) ? -1.f : 1.f;
  __syncthreads();  // the rows' places
  // ---- a6: rotate the rows' queries into the A tiles (f16 high and low parts) ------------
  {
    float M[16];
    load_block_mat(params + (size_t)hk * D * 4, lane, M);
    const int k0 = lane * E;  // dims 4 lane .. + 3: half of one 16-byte core-matrix row
    constexpr int kAt = 4;  // rows at a time; the next four's loads run meanwhile
    auto load = [&](int r0, float (&v)[kAt][E]) {
#pragma unroll
      for (int j = 0; j < kAt; ++j) {
        const int r = r0 + kWWarps * j;
#pragma unroll
        for (int i = 0; i < E; ++i) v[j][i] = 0.f;
        if (r < nh && in_bounds(row_off[r] < n_q * n_q_heads, status))
          load_vec<TQ, E>(Q + (seq_row + row_off[r]) * D + k0, v[j]);
      }
    };
    float nx[kAt][E];
    load(warp, nx);
#pragma unroll 1
    for (int r0 = warp; r0 < rows_cta; r0 += kWWarps * kAt) {
      float v[kAt][E];
#pragma unroll
      for (int j = 0; j < kAt; ++j)
#pragma unroll
        for (int i = 0; i < E; ++i) v[j][i] = nx[j][i];
      load(r0 + kWWarps * kAt, nx);
#pragma unroll
      for (int j = 0; j < kAt; ++j) wht_signed<E>(v[j], sgn);
      // z, and whether a row's largest element lies outside the range that needs no division
      uint32_t sizes = 0;  // bit j: row j has an element >= 2^-3 (or is none), bit 4 + j: >= 2^15
#pragma unroll
      for (int j = 0; j < kAt; ++j) {
        float z[E];
        mat_fwd(M, v[j], z);
        float big = r0 + kWWarps * j < nh ? 0.f : 1.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          v[j][e] = z[e];
          big = fmaxf(big, fabsf(z[e]));
        }
        sizes |= (big >= kQueryMin ? 1u << j : 0u) | (big >= kQueryMax ? 16u << j : 0u);
      }
      if (__reduce_or_sync(kFull, sizes) != 15u) {  // out of line: code that does not run is not fetched
#pragma unroll
        for (int j = 0; j < kAt; ++j) {
          const int r = r0 + kWWarps * j, ex = query_exponent<E>(v[j]);
#pragma unroll
          for (int e = 0; e < E; ++e) v[j][e] *= pow2i(-ex);
          if (lane == 0 && in_bounds(r < rows_cta, status)) {
            unit[r] = pow2i(ex);
            if (!two) unit[128 + r] = pow2i(ex);  // both halves hold the row
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kAt; ++j) {
        const int r = r0 + kWWarps * j;
        const float (&z)[E] = v[j];
        float hi[E];
#pragma unroll
        for (int e = 0; e < E; ++e) hi[e] = __half2float(__float2half_rn(z[e]));
        const uint32_t at = sQ + (r >> 7) * 2 * SM::kQPart + (k0 >> 3) * SM::kQGroup +
                            ((r & 127) >> 3) * 128 + (r & 7) * 16 + (k0 & 7) * 2;
        if (r >= rows_cta || !in_bounds(at + SM::kQPart + 8 <= sK, status)) continue;
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(pack_f16x2(hi[0], hi[1])),
                     "r"(pack_f16x2(hi[2], hi[3])) : "memory");
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at + SM::kQPart),
                     "r"(pack_f16x2(z[0] - hi[0], z[1] - hi[1])),
                     "r"(pack_f16x2(z[2] - hi[2], z[3] - hi[3])) : "memory");
      }
    }
  }
  fence_proxy_async();
  tc::fence_before();
  __syncthreads();  // barriers initialised, tensor memory allocated, query tiles written
  tc::fence_after();
  const uint32_t tmem = __shfl_sync(kFull, *tmem_slot, 0);
  const int role = __shfl_sync(kFull, warp, 0);  // warp-uniform to the compiler as well
  // tile stages: 2, or 4 with one row block; page k takes stage k % stages, phase k / stages
  const int st_mask = two ? 1 : 3, st_log = two ? 1 : 2;
  auto tile_k = [&](int st) { return st < 2 ? sK + st * kPageTile : sQ + 2 * SM::kQPart + (st - 2) * 2 * kPageTile; };
  auto tile_v = [&](int st) { return st < 2 ? sV + st * kPageTile : tile_k(st) + kPageTile; };
  // jobs of softmax half w: page k = i with two row blocks, else k = 2 i + w
  auto jobs = [&](int w) { return two ? n : (n - w + 1) / 2; };
  bool ok = true;
  // this thread's row state (softmax warps)
  const int w = (warp >> 2) & 1, r_tid = tid & 127;
  const int my_r = two ? 128 * w + r_tid : r_tid;
  float m2 = -CUDART_INF_F, lsum = 0.f, sigma = 0.f;
  const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);

  // the ring stage has been read by the K and V threads; whether one of them gave up
  auto ring_read = [&]() {
    uint32_t gave_up;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 2, %2, p;\n"
        " selp.u32 %0, 1, 0, q;\n}"
        : "=r"(gave_up) : "r"((uint32_t)!ok), "n"(kWK + kWV) : "memory");
    return gave_up != 0;
  };
  if (role >= 8 && role != 12) {
    // ================ dequantisation ======================================================
    const bool k_side = role < 12;
    const int t = tid - (k_side ? 256 : 416);
    uint32_t tl0, tl1, th0, th1;
    level_tables<BITS>(tl0, tl1, th0, th1);
    const float kf = scale * kLog2e / (ALPHA * (float)D);  // log2 score per (dot * nK)
    int spreads = 0;  // bit 0: the page before of the same softmax half was spread
    int issued = min(n, 2), k = 0;
    // page-table entries of pages k .. k + 2, each loaded three pages ahead of its use
    int ph0 = entry_of(0), ph1 = entry_of(1), ph2 = entry_of(2);
    for (; k < n; ++k) {
      const int st = k & st_mask;
      const int before = k - st_mask - 1;  // the page that had the stage
      const int ph_before = (before >> st_log) & 1;
      const uint8_t* blk = smem + SM::kOffRing + (k & 1) * BB;
      const int ph3 = entry_of(k + 3);
      ok = mbar_wait(bars + kRing + (k & 1), (k >> 1) & 1);
      if (k_side) {
        ok = ok && (before < 0 || mbar_wait(bars + kKFree + st, ph_before));
        if (ok) page_tile<BITS, kWK>(blk, 0, t, tile_k(st), tl0, tl1, th0, th1, status);
        fence_proxy_async();  // the generic-proxy tile writes, before the tensor core reads
        if (ok) mbar_arrive(bars + kKFull + st);
      }
      // the V tile, the norms and sigma of the page before have been used once its value product
      // is done
      ok = ok && (before < 0 || mbar_wait(bars + kVFree + st, ph_before));
      if (!k_side) {
        if (ok) page_tile<BITS, kWV>(blk, 1, t, tile_v(st), tl0, tl1, th0, th1, status);
        fence_proxy_async();
      } else {
        // nrm[j] = |k_j| kf; nrm[64 + j] = |v_j| / sigma with the CTA's V-norm reference sigma (it
        // only scales the weights), raised when a token some row sees has |v| > kSigmaSlack sigma
        const int tok0 = wp.page(p_begin + k) * kPage;
        const bool page_ok = ph0 >= 0 && ph0 < n_pages;
        if (t < 64) {
          if (ok) nrm[st * 128 + t] = half_at(blk + k_norm_off(D, BITS) + 2 * t) * kf;
        } else {
          const int j = t - 64;
          float nv = half_at(blk + v_norm_off(D, BITS) + 2 * j);
          const bool seen = page_ok && tok0 + j < lim_hi && wp.any_sees(win, tok0 + j);
          nv = seen ? nv : 0.f;
          // largest and smallest (norms, >= 0, order as their bits do)
          const uint32_t pm2 = __reduce_max_sync(kFull, __float_as_uint(nv));
          const uint32_t pl2 = __reduce_min_sync(kFull, __float_as_uint(seen ? nv : CUDART_INF_F));
          if (lane == 0) red[warp - 10] = make_float2(__uint_as_float(pm2), __uint_as_float(pl2));
          asm volatile("bar.sync 1, 64;" ::: "memory");  // warps 10 and 11
          const float4 both = *reinterpret_cast<const float4*>(red);
          const float pm = fmaxf(both.x, both.z), pl = fminf(both.y, both.w);
          sigma = pm > sigma * kSigmaSlack ? pm : sigma;
          const bool spread = sigma > kSpreadNorms * pl, before_spread = spreads & 1;
          spreads = two ? spread : spreads >> 1 | (spread ? 2 : 0);
          if (ok) {
            nrm[st * 128 + t] = sigma > 0.f ? nv * (1.f / sigma) : 0.f;
            if (t == 64) {
              sig[st] = sigma;
              top[st] = pm;
              valid[st] = (page_ok ? kValid : 0) | (spread ? kSpread : before_spread ? kLevel : 0);
            }
          }
        }
      }
      if (ok) mbar_arrive(bars + kVFull + st);
      if (ring_read()) break;
      if (tid == 256 && k + 2 < n) {
        fence_proxy_async();
        issue(k + 2, ph2);
      }
      if (k + 2 < n) issued = k + 3;
      ph0 = ph1;
      ph1 = ph2;
      ph2 = ph3;
    }
    if (k < n) {  // gave up: wait (bounded) for the copies in flight
      ok = false;
      if (tid == 256)
        for (int kk = k; kk < issued; ++kk) mbar_wait(bars + kRing + (kk & 1), (kk >> 1) & 1);
    }
  } else if (role == 12) {
    // ================ products ============================================================
    // the whole warp runs the loop, one lane issues (tc::elect_one says why)
    const bool one = tc::elect_one();
    auto wait = [&](int bar, int phase) { return __all_sync(kFull, mbar_wait(bars + bar, phase & 1)) != 0; };
    auto commit = [&](int bar) {
      if (one) tc::commit(bars + bar);
    };
    // a7: S_h(k), 8 k-steps of 16 dims, the high and the low part
    auto scores = [&](int h, int k) {
      const uint64_t q = tc::sdesc(sQ + (two ? h : 0) * 2 * SM::kQPart, SM::kQGroup, 128);
      const uint64_t kt = tc::sdesc(tile_k(k & st_mask), 1024, 128);
      tc::fence_after();
      if (one) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {  // descriptors count 16 bytes
          tc::mma_ss(tmem + col_s(h), q + kk * (2 * SM::kQGroup / 16), kt + kk * 128, kIdS, kk > 0);
          tc::mma_ss(tmem + col_s(h), q + (SM::kQPart + kk * 2 * SM::kQGroup) / 16, kt + kk * 128, kIdS, 1);
        }
      }
      commit(kSFull + h);
    };
    // a8: O_h += P'_h . V_hat(k), 4 k-steps of 16 tokens; i = the half's job number
    auto values = [&](int h, int k, int i) {
      const uint64_t vt = tc::sdesc(tile_v(k & st_mask), 2048, 128);
      tc::fence_after();
      if (one) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          tc::mma_ts(tmem + col_o(h), tmem + col_p(h) + 8 * j, vt + j * 256, kIdO,
                     (i > 0 || j > 0) ? 1u : 0u);
      }
      commit(kPvDone + h);
    };
    if (two) {
      if ((ok = wait(kKFull, 0))) {
        scores(0, 0);
        scores(1, 0);
        commit(kKFree);
      }
      for (int k = 0; ok && k < n; ++k) {
        const int st = k & 1, st1 = st ^ 1;
        // the next page's scores as soon as this page's have been read: a half that has
        // written its weights goes straight on
        if (k + 1 < n) {
          if (!(ok = wait(kKFull + st1, (k + 1) >> 1) && wait(kSRead, k))) break;
          scores(0, k + 1);
          if (!(ok = wait(kSRead + 1, k))) break;
          scores(1, k + 1);
          commit(kKFree + st1);
        }
        if (!(ok = wait(kVFull + st, k >> 1) && wait(kPFull, k))) break;
        values(0, k, k);
        if (!(ok = wait(kPFull + 1, k))) break;
        values(1, k, k);
        commit(kVFree + st);
      }
    } else {
      for (int k = 0; ok && k < 2 && k < n; ++k) {
        if (!(ok = wait(kKFull + k, 0))) break;
        scores(k, k);
        commit(kKFree + k);
      }
      for (int k = 0; ok && k < n; ++k) {
        const int h = k & 1, i = k >> 1, st = k & 3, st2 = (k + 2) & 3;
        if (k + 2 < n) {
          if (!(ok = wait(kKFull + st2, (k + 2) >> 2) && wait(kSRead + h, i))) break;
          scores(h, k + 2);
          commit(kKFree + st2);
        }
        if (!(ok = wait(kVFull + st, k >> 2) && wait(kPFull + h, i))) break;
        values(h, k, i);
        commit(kVFree + st);
      }
    }
    if (!ok) {  // gave up: wait (bounded) for the products in flight
      commit(kDrain);
      mbar_wait(bars + kDrain, 0);
    }
    __syncwarp();
  } else {
    // ================ softmax of this thread's row ==========================================
    const int my_lim = my_r < nh ? lim_of(my_r) : lim_hi;
    const int my_lo = win_lo<true>(win, my_lim);
    const uint32_t t_s = t_lane + col_s(w), t_p = t_lane + col_p(w), t_o = t_lane + col_o(w);
    const int n_jobs = jobs(w);
    // a warp with a divided row (query_exponent) has no page that goes unmasked: the common path is
    // without its multiplication (as a branch of every page it cost 1.6% of a long chunk)
    const int full_to = __any_sync(kFull, unit[tid] != 1.f) ? -1 : lim_lo;
    float lim = kLazy + kLift;  // of an exponent: kLazy plus the row's lift
    for (int i = 0; i < n_jobs; ++i) {
      const int k = two ? i : 2 * i + w, st = k & st_mask;
      // the page's scores (warp-uniform: collective loads follow), then its norms
      ok = __all_sync(kFull, mbar_wait(bars + kSFull + w, i & 1));
      if (!ok) break;
      tc::fence_after();
      float x[64];
      {
        uint32_t sr[64];
        tc::ld64(t_s, sr);
#pragma unroll
        for (int j = 0; j < 64; ++j) x[j] = __uint_as_float(sr[j]);
      }
      tc::fence_before();
      mbar_arrive(bars + kSRead + w);
      ok = __all_sync(kFull, mbar_wait(bars + kVFull + st, (k >> st_log) & 1));
      if (!ok) break;
      const float* nk = nrm + st * 128;
      const int state = valid[st];
      const bool page_ok = (state & kValid) != 0;
      const int tok0 = wp.page(p_begin + k) * kPage;
      const float sg = sig[st];
      const float vr = sg > sigma ? sigma / sg : 1.f;  // 0 on the first valid page
      sigma = sg;
      // exponents a_j = s_j |k_j| - m2 from one FMA each; m2, the row's running maximum less its lift,
      // moves only when some a_j > lim, kLazy above that maximum (or on the row's first scores), and
      // then O is rescaled in place, factor resc
      float resc = vr;
      bool moved = vr != 1.f;
      auto sees = [&](int tok) { return page_ok && tok < my_lim && win_sees<true>(win, my_lo, tok); };
      const bool all = page_ok && tok0 + kPage <= full_to && wp.page_full(win, tok0);
      if (state & (kSpread | kLevel)) {  // the row's lift
        float bits = 0.f;
        if (state & kSpread) {
          float v = top[st];
          if (!all) {
            v = 0.f;
#pragma unroll 4
            for (int j = 0; j < 64; ++j) v = fmaxf(v, sees(tok0 + j) ? nk[64 + j] : 0.f);
            v *= sg;
          }
          bits = lift_bits(v, sg, lim - (kLazy + kLift));
        }
        const float up = lim - (kLazy + kLift + bits);  // what m2 rises by
        if (up != 0.f) {
          lim -= up;
          m2 += up;
          lsum *= ex2(-up);
          resc *= ex2(-up);
          moved = true;
        }
      }
      auto exponents = [&](auto full_c) {
        constexpr bool FULL = decltype(full_c)::value;
        if (!FULL && __any_sync(kFull, unit[threadIdx.x] != 1.f)) {
          const float mul = unit[threadIdx.x];
#pragma unroll
          for (int j = 0; j < 64; ++j) x[j] *= mul;
        }
        const bool fresh = m2 == -CUDART_INF_F;
        const float2 nm2 = fresh ? make_float2(0.f, 0.f) : make_float2(-m2, -m2);
        float am[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
        for (int j4 = 0; j4 < 64; j4 += 4) {
          const float4 k4 = *reinterpret_cast<const float4*>(nk + j4);
          const float2 a01 = f2_fma(make_float2(x[j4], x[j4 + 1]), make_float2(k4.x, k4.y), nm2);
          const float2 a23 = f2_fma(make_float2(x[j4 + 2], x[j4 + 3]), make_float2(k4.z, k4.w), nm2);
          const float av[4] = {a01.x, a01.y, a23.x, a23.y};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float a = av[e];
            if constexpr (!FULL) a = sees(tok0 + j4 + e) ? a : -CUDART_INF_F;
            x[j4 + e] = a;
            am[e] = fmaxf(am[e], a);
          }
        }
        const float amax = fmaxf(fmaxf(am[0], am[1]), fmaxf(am[2], am[3]));
        if (fresh ? amax != -CUDART_INF_F : amax > lim) {
          const float up = amax - (lim - kLazy);
          const float f = fresh ? 0.f : ex2(-up);  // fresh: nothing accumulated yet
          resc *= f;
          lsum *= f;
          m2 = fresh ? up : m2 + up;
          moved = true;
#pragma unroll
          for (int j = 0; j < 64; ++j) x[j] -= up;
        }
      };
      if (all) exponents(std::true_type{});
      else exponents(std::false_type{});
      uint32_t pw[32];
      float2 ls01 = make_float2(0.f, 0.f), ls23 = make_float2(0.f, 0.f);
#pragma unroll
      for (int j4 = 0; j4 < 64; j4 += 4) {
        const float4 v4 = *reinterpret_cast<const float4*>(nk + 64 + j4);
        const float2 p01 = make_float2(ex2(x[j4]), ex2(x[j4 + 1]));  // -inf: 0
        const float2 p23 = make_float2(ex2(x[j4 + 2]), ex2(x[j4 + 3]));
        ls01 = f2_add(ls01, p01);
        ls23 = f2_add(ls23, p23);
        const float2 w01 = f2_mul(p01, make_float2(v4.x, v4.y));
        const float2 w23 = f2_mul(p23, make_float2(v4.z, v4.w));
        pw[j4 / 2] = pack_f16x2(w01.x, w01.y);
        pw[j4 / 2 + 1] = pack_f16x2(w23.x, w23.y);
      }
      lsum += (ls01.x + ls01.y) + (ls23.x + ls23.y);
      // P' and O are this thread's again once the half's last value product is done
      ok = __all_sync(kFull, i == 0 || mbar_wait(bars + kPvDone + w, (i - 1) & 1));
      if (!ok) break;
      tc::fence_after();
      if (i > 0 && __any_sync(kFull, moved)) {  // collective: the other rows with factor 1
        uint32_t ov[32];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tc::ld32(t_o + 32 * c, ov);
#pragma unroll
          for (int j = 0; j < 32; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * resc);
          tc::st32(t_o + 32 * c, ov);
        }
      }
      tc::st32(t_p, pw);
      tc::wait_st();
      tc::fence_before();
      mbar_arrive(bars + kPFull + w);
    }
    if (ok && n_jobs > 0) ok = mbar_wait(bars + kPvDone + w, (n_jobs - 1) & 1);
  }

  // ---- every role is through: the rows' results ------------------------------------------
  tc::fence_before();
  const bool failed = __syncthreads_or(!ok);
  tc::fence_after();
  if (failed) {
    if (tid == 0) set_status(status, ISOQ_ST_TIMEOUT);
  } else {
    // The rows' accumulators go through the query tiles' memory, one 512-byte row of 32 chunks
    // each (chunk index xor the row's low bits), and a warp finishes a row: rolled loops, since
    // straight-line code that runs once per CTA costs its fetches (a register-resident inverse
    // rotation, one thread a row, took 80 us a CTA).
    auto at = [&](int r, int c) { return reinterpret_cast<float4*>(smem + r * 512 + ((c ^ (r & 7)) << 4)); };
    if (role < 8) {
      const float f = jobs(w) > 0 ? sigma / ALPHA : 0.f;  // O holds sum p |v| ALPHA L / sigma
      const int r = 128 * w + r_tid;
      ml[r] = make_float2(m2, lsum);
#pragma unroll 1
      for (int c = 0; c < 4 && jobs(w) > 0; ++c) {
        uint32_t ov[32];
        tc::ld32(t_lane + col_o(w) + 32 * c, ov);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *at(r, 8 * c + j) =
              make_float4(__uint_as_float(ov[4 * j]) * f, __uint_as_float(ov[4 * j + 1]) * f,
                          __uint_as_float(ov[4 * j + 2]) * f, __uint_as_float(ov[4 * j + 3]) * f);
      }
    }
    __syncthreads();
    {
      float M[16];
      load_block_mat(params + (size_t)hk * D * 4, lane, M);
      constexpr int kAt = 4;  // rows at a time
#pragma unroll 1
      for (int r0 = role; r0 < nh; r0 += kWWarps * kAt) {
        float y[kAt][E], m[kAt], l[kAt];
#pragma unroll
        for (int j = 0; j < kAt; ++j) {
          const int r = min(r0 + kWWarps * j, nh - 1);
          const float2 a = ml[r];
          const float4 v = *at(r, lane);
          m[j] = a.x;
          float fa = 1.f, fb = 0.f;
          float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
          l[j] = a.y;
          if (!two && jobs(1) > 0) {  // the halves' states of the same row meet
            const float2 b = ml[128 + r];
            u = *at(128 + r, lane);
            m[j] = fmaxf(a.x, b.x);
            fa = a.x == -CUDART_INF_F ? 0.f : ex2(a.x - m[j]);
            fb = b.x == -CUDART_INF_F ? 0.f : ex2(b.x - m[j]);
            l[j] = a.y * fa + b.y * fb;
          }
          const float o[E] = {fmaf(u.x, fb, v.x * fa), fmaf(u.y, fb, v.y * fa), fmaf(u.z, fb, v.z * fa),
                              fmaf(u.w, fb, v.w * fa)};
          if (out != nullptr) {
            mat_inv(M, o, y[j]);
          } else {
#pragma unroll
            for (int i = 0; i < E; ++i) y[j][i] = o[i];
          }
        }
        if (out != nullptr) {
#pragma unroll
          for (int j = 0; j < kAt; ++j) wht_signed<E>(y[j], sgn);
        }
#pragma unroll
        for (int j = 0; j < kAt; ++j) {
          const int r = r0 + kWWarps * j;
          if (r >= nh) continue;
          const int ri = row_off[r];
          if (!in_bounds(ri < n_q * n_q_heads, status)) continue;
          if (out != nullptr) {  // divided by l, the WHT's and the levels' 1 / sqrt(d) each
            const float f = l[j] > 0.f ? 1.f / (l[j] * (float)D) : 0.f;
            const size_t at0 = (seq_row + ri) * D + lane * E;
            const float4 v = make_float4(y[j][0] * f, y[j][1] * f, y[j][2] * f, y[j][3] * f);
            if (win.out_dtype == ISOQ_F32) {
              *reinterpret_cast<float4*>(static_cast<float*>(out) + at0) = v;
            } else if (win.out_dtype == ISOQ_F16) {
              *reinterpret_cast<uint2*>(static_cast<__half*>(out) + at0) =
                  make_uint2(pack_f16x2(v.x, v.y), pack_f16x2(v.z, v.w));
            } else {
              __nv_bfloat162* p = reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(out) + at0);
              p[0] = __floats2bfloat162_rn(v.x, v.y);
              p[1] = __floats2bfloat162_rn(v.z, v.w);
            }
          } else {
            float* p = out_base + (size_t)ri * n_splits * PS;
            *reinterpret_cast<float4*>(p + lane * E) = make_float4(y[j][0], y[j][1], y[j][2], y[j][3]);
            if (lane == 0) {
              p[D] = m[j] == -CUDART_INF_F ? -CUDART_INF_F : m[j] / kLog2e;  // natural-log units
              p[D + 1] = l[j];
            }
          }
        }
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 12) {
    tc::fence_after();
    tc::dealloc(tmem, kWCols);
  }
}

template <typename TQ, int BITS>
cudaError_t launch_window_t(const DecodeArgs& a, cudaStream_t stream) {
  using SM = WinSmem<BITS>;
  static unsigned long long attr_set = 0;  // the shared-memory opt-in, per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !((attr_set >> dev) & 1ull)) {
    e = cudaFuncSetAttribute(window_tc_kernel<TQ, BITS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             SM::kBytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_set |= 1ull << dev;
  }
  const int rows = a.n_q * (a.n_q_heads / a.n_kv_heads), per = window_tc_rows(rows);
  dim3 grid(a.n_splits, a.n_kv_heads * ((rows + per - 1) / per), a.n_seqs);
  window_tc_kernel<TQ, BITS><<<grid, kWThreads, SM::kBytes, stream>>>(
      a.params, a.blocks, a.page_table, a.n_pages, a.max_pages, a.n_kv_heads,
      static_cast<const TQ*>(a.Q), a.n_q_heads, a.n_q, a.seq_lens, a.scale, a.pages_per_split,
      a.n_splits, a.partials, a.n_splits == 1 ? a.out : nullptr, a.status, win_args(a));
  return cudaGetLastError();
}

template <int BITS>
cudaError_t launch_window_b(const DecodeArgs& a, cudaStream_t stream) {
  switch (a.q_dtype) {
    case ISOQ_F32: return launch_window_t<float, BITS>(a, stream);
    case ISOQ_BF16: return launch_window_t<__nv_bfloat16, BITS>(a, stream);
    case ISOQ_F16: return launch_window_t<__half, BITS>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_window_tc(const DecodeArgs& a, cudaStream_t stream) {
  switch (a.bits) {
    case 2: return launch_window_b<2>(a, stream);
    case 3: return launch_window_b<3>(a, stream);
    case 4: return launch_window_b<4>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace isoq
