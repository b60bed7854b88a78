// Read-back to 16-bit types with the inverse rotation on the tensor cores.
//
//   X[128 vectors x 128 dims] = Z[128 x d] . R  per KV head,  x = (n / sqrt d) (Z R)
// Z holds the levels of the vectors' codes as binary16 (ALPHA times the level: relative
// error < 2e-5 at 3 bits, 0 at 2, < 6e-5 at 4), R the head's rotation (WHT and 4x4 blocks
// in one matrix, made here from the blocks in doubled binary32) as one or two binary16 parts, the
// sums in the tensor core's binary32.  Rounding: with both parts (fp16 outputs) R keeps 22
// bits, so the levels' 2e-5 leads, 1/24 of the output's own half step.  bf16 outputs take
// the high part alone: an entry's relative error of at most 2^-12 to 2^-11 gives elements
// ~1.5e-4 of the vector's rms off, a tenth of the rms error of rounding to bf16.
//
// Work: a CTA keeps R of one head (and, at d = 256, one 128-column half) in shared memory
// and walks over tiles of 128 vectors: 64 listed tokens' K and V, or 128 tokens of one
// side.  Per tile the threads turn the code words that they loaded one tile ahead into the
// operand tile (byte permutes, as in the attention kernels), one thread issues the d/16
// products per part into tensor memory, and while they run the next tile's words are
// loaded; then each thread scales its row's share of the accumulator, takes the rotary
// embedding off, rounds, and writes it out in whole 32-byte sectors.  A 16-row block whose
// tokens are one 16-slot block of a page in order (any run that starts at a multiple of 16)
// reads the V tile layout's groups as they are, four tokens at a time; other tokens pick
// their own nibbles out of the groups.
//
// Measured (32768 consecutive tokens, 8 KV heads, K and V): d = 128 to bf16 47 us (3.4 TB/s of
// codes read and values written), to fp16 53 us, with the rotary embedding 72 and 107 us;
// d = 256 to bf16 134 us, with the embedding 231.  ncu on the first: ALU pipe 55% busy, issue
// 55% of the cycles, DRAM 27%, tensor pipe 20%: bound by the instructions of the fill and the
// write-out (44 a vector) and by the chain of one tile's steps.  R made by every CTA (~0.3 us)
// instead of read from a copy kept with the parameters: bf16 1.4 us longer, the others 0.6 to 7
// shorter.  Tried, with 45 us for the first: the
// output staged in shared memory and sent as one bulk copy a row, 57-70 (the copy engine takes
// ~33 cycles a row), or written by 16 lanes a row, 57; each thread writing its own row's
// columns, 56 (32 lines an instruction); the page lookups not pipelined, 70; twice the threads
// a CTA, 61.  The accumulator is therefore read as 16-row fragments whose columns are ordered
// so that a quad writes 128 contiguous bytes.
#include "isoq_check.cuh"
#include "isoq_common.cuh"
#include "isoq_dequantize.cuh"
#include "isoq_internal.h"
#include "isoq_ptx.cuh"
#include "isoq_tc.cuh"
#include "isoq_vtile.cuh"

namespace isoq {
using namespace ptx;
namespace {

constexpr int kTile = 128;  // vectors per tile = rows of the product = tensor-memory lanes
constexpr uint32_t kTileCols = 128;
// A listed token of a tile: its (page, head) block (null: nothing to read or write), position.
struct TileRow {
  const uint8_t* blk;
  int pos, pad;
};

template <int D, bool LO, bool ROPE>
struct ReadSmem {
  static constexpr int kPart = D * 128 * 2;          // one binary16 part of R
  static constexpr int kOffA = (LO ? 2 : 1) * kPart; // operand tile
  static constexpr int kTileBytes = kTile * D * 2;
  // of three tiles: the one being written out, the next, and the one whose rows come in
  static constexpr int kOffRow = kOffA + kTileBytes;                           // TileRow [3][128]
  static constexpr int kOffNorm = kOffRow + 3 * kTile * (int)sizeof(TileRow);  // float [3][128]
  static constexpr int kOffWhole = kOffNorm + 3 * kTile * 4;  // int [3][8]: 16-row blocks in order
  static constexpr int kOffBar = kOffWhole + 3 * 8 * 4;
  static constexpr int kOffTmem = kOffBar + 8 + 8;
  // the rotary table's 64 pairs of the tile's 64 keys, 512 bytes a row
  static constexpr int kOffTable = (kOffTmem + 16 + 127) / 128 * 128;
  static constexpr int kBytes = ROPE ? kOffTable + 64 * 512 : kOffTmem + 16;
  static_assert(kBytes <= 227 * 1024, "shared memory");
  static_assert(kOffA % 1024 == 0 && kOffBar % 8 == 0 && kOffRow % 16 == 0, "alignment");
};

// CTAs per SM: what the shared memory (R in one or two parts, a tile) and the registers let in.
template <int D, bool LO>
constexpr int read_ctas(bool rope) { return D == 256 || (LO && rope) ? 1 : LO || rope ? 2 : 3; }

__device__ __forceinline__ void st_chunk(uint32_t addr, uint32_t x, uint32_t y, uint32_t z,
                                         uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z),
               "r"(w)
               : "memory");
}

// 32 bytes of a row at p: one full sector in one instruction where p allows it.
__device__ __forceinline__ void st_sector(void* p, const uint32_t (&o)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(o[0]),
                 "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(o[0], o[1], o[2], o[3]);
    static_cast<uint4*>(p)[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float2 v) {
  if constexpr (__is_same(T, __half)) {
    return pack_f16x2(v.x, v.y);
  } else {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
}

// (u + v) (a + b + c + d) as x + y to twice binary32's bits, |v| <= ulp(u) / 2: the sums' and the
// product's rounding errors are kept (Knuth's two-sum, and a fused multiply-add).
__device__ __forceinline__ float2 scaled_sum(float a, float b, float c, float d, float u, float v) {
  float s = a, e = 0.f;
  auto add = [&](float t) {
    const float r = s + t, w = r - s;
    e += (s - (r - w)) + (t - w);
    s = r;
  };
  add(b);
  add(c);
  add(d);
  const float p = s * u, err = fmaf(s, u, -p) + fmaf(s, v, e * u), x = p + err;
  return make_float2(x, (p - x) + err);
}

// 2 d threads: each takes, of either item (64 rows), one 32-dim group of a row or one group
// of the V tile layout.
template <int D, int BITS, typename T, bool LO, bool ROPE>
__global__ void __launch_bounds__(2 * D, read_ctas<D, LO>(ROPE))
    dequantize_tc_kernel(const DequantizeArgs a, int units, int n_tiles) {
  using SM = ReadSmem<D, LO, ROPE>;
  constexpr int NT = 2 * D, CB = code_bytes(D, BITS), BB = block_bytes(D, BITS), W = BITS;
  constexpr int NU = D / 8;                // 8-dim units
  // A warp reads 16 rows of the accumulator at a time: at d = 128 the 8 warps cover the 128
  // rows and take both 64-column halves, at d = 256 16 warps take one half each.
  constexpr int kHalves = D == 128 ? 2 : 1;
  constexpr uint32_t kId = tc::idesc_f16(128, 128, false, false);
  extern __shared__ __align__(1024) uint8_t smem[];
  TileRow* rows = reinterpret_cast<TileRow*>(smem + SM::kOffRow);  // [3 tiles][128]
  float* nrm = reinterpret_cast<float*>(smem + SM::kOffNorm);
  int* whole = reinterpret_cast<int*>(smem + SM::kOffWhole);
  uint64_t* done = reinterpret_cast<uint64_t*>(smem + SM::kOffBar);  // the products
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM::kOffTmem);
  const uint32_t sB = smem_u32(smem), sA = smem_u32(smem + SM::kOffA);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int unit = blockIdx.x % units, first = blockIdx.x / units, step = gridDim.x / units;
  const int h = unit / (D / 128), q = unit - h * (D / 128);
  // with a rotary table a tile is always 64 tokens, the V rows empty where V is not wanted
  const bool both = ROPE || (a.K != nullptr && a.V != nullptr);
  const int per_tile = both ? 64 : 128;    // tokens per tile
  auto side_of = [&](int item) { return both ? item : a.K == nullptr; };  // 0: K, 1: V
  auto out_of = [&](int item) { return side_of(item) ? a.V : a.K; };
  // token of row r (0..127) of a tile; its two items are 64 rows each
  auto token_of = [&](int tile, int r) { return (long long)tile * per_tile + (both ? r & 63 : r); };

  // The tiles' tokens come in three dependent loads (list, page table, codes), each issued a
  // whole tile before its result is used.  Thread r < 128 follows row r:
  //   fetch_token   sequence and position            (tile k + 3)
  //   fetch_page    the page-table entry             (tile k + 2)
  //   put_row       block and position to stage st   (tile k + 1)
  int tok_s = 0, tok_p = 0, pg_p = 0, pg = -1;  // token of the next fetch_page, entry of put_row
  uint32_t pg_bad = 0;
  bool tok_live = false;
  auto fetch_token = [&](long long tile) {
    const long long i = tile * per_tile + (both ? tid & 63 : tid);
    tok_live = tid < kTile && tile < n_tiles && i < a.n_tokens && (!ROPE || out_of(tid >> 6) != nullptr);
    if (tok_live) {
      tok_s = __ldg(a.seq_ids + i);
      tok_p = __ldg(a.positions + i);
    }
  };
  auto fetch_page = [&]() {
    pg_bad = 0;
    pg_p = tok_p;
    long long entry = -1;
    if (tok_live) entry = page_entry(a, tok_s, tok_p, pg_bad);
    pg = entry < 0 ? -1 : __ldg(a.page_table + entry);
    if (tok_live && entry >= 0) pg_bad = ISOQ_ST_PAGE_RANGE;  // if the entry is not a page
  };
  auto put_row = [&](int st) {
    if (tid < kTile) {
      const bool ok = pg >= 0 && pg < a.n_pages;
      // one report a token: with both sides in the tile, of the K row, or of the V row without K
      const bool mine = !both || (tid < 64) == (a.K != nullptr);
      if (!ok && pg_bad && h == 0 && q == 0 && mine) set_status(a.status, pg_bad);
      TileRow r;
      r.blk = ok ? a.blocks + ((size_t)pg * a.n_kv_heads + h) * BB : nullptr;
      r.pos = pg_p;
      r.pad = 0;
      rows[st * kTile + tid] = r;
      const int p0 = __shfl_sync(kFull, pg_p, lane & 16), x0 = __shfl_sync(kFull, pg, lane & 16);
      const bool in_order = ok && pg == x0 && pg_p == p0 + (lane & 15) && (p0 & 15) == 0;
      const unsigned all = __ballot_sync(kFull, in_order);
      if ((lane & 15) == 0) whole[st * 8 + (tid >> 4)] = ((all >> (lane & 16)) & 0xFFFFu) == 0xFFFFu;
    }
  };
  // this thread's place in the 64 rows of an item: row and 32-dim group, ...
  const int my_row = 8 * (warp & 7) + (lane & 7), my_q = (lane >> 3) + 4 * (warp >> 3);
  const uint32_t my_chunk = sA + 4 * my_q * 2048 + (my_row >> 3) * 128 + (my_row & 7) * 16;
  // ... or, of the V tile layout, a group of four tokens: lanes 4m .. 4m + 3 take the quads of
  // one unit, and odd units their members in the order 1 0 3 2, so that the 16-byte stores
  // of 8 lanes cover the 8 chunks of a 128-byte line once
  const int my_quad = tid & 3, my_unit = (tid >> 2) & (NU - 1), my_block = tid >> (D == 128 ? 6 : 7);
  const int my_swap = 4 * (my_unit & 1);
  const uint32_t my_group = sA + my_unit * 2048 + 2 * my_block * 128 + 2 * my_quad * 16;
  const uint32_t my_even = my_group + 4 * my_swap, my_odd = my_group + 16 - 4 * my_swap;
  uint32_t w[2][W];
  uint16_t my_norm = 0;  // as loaded: converted a tile later
  // an item's words are groups of the V tile layout (else records of one token)
  auto grouped = [&](int item) { return BITS == 3 && side_of(item); };
  auto load_words = [&](int st) {
#pragma unroll
    for (int item = 0; item < 2; ++item) {
      const bool gr = grouped(item);
      const TileRow t = rows[st * kTile + 64 * item + (gr ? 16 * my_block : my_row)];
      if (gr ? whole[st * 8 + 4 * item + my_block] == 0 : t.blk == nullptr) continue;
      const int slot = t.pos & (kPage - 1);
      const int go = gr ? vt_group_off(D, slot >> 4, my_quad, my_unit) : slot * CB + 4 * W * my_q;
      const uint8_t* p = t.blk + (side_of(item) ? v_codes_off(D, BITS) : 0) + go;
      if (!in_bounds(go + 4 * W <= kPage * CB, a.status)) continue;
      if constexpr (W == 4) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
        w[item][0] = v.x, w[item][1] = v.y, w[item][2] = v.z, w[item][3] = v.w;
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) w[item][i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
      }
    }
    if (tid < kTile) {
      const TileRow t = rows[st * kTile + tid];
      if (t.blk != nullptr)
        my_norm = __ldg(reinterpret_cast<const uint16_t*>(
            t.blk + (side_of(tid >> 6) ? v_norm_off(D, BITS) : k_norm_off(D, BITS)) +
            2 * (t.pos & (kPage - 1))));
    }
  };

  uint32_t tl0, tl1, th0, th1;
  level_tables<BITS>(tl0, tl1, th0, th1);
  const uint32_t a_end = sA + SM::kTileBytes;
  auto put = [&](uint32_t addr, const uint32_t (&o)[4]) {
    if (in_bounds(addr >= sA && addr + 16 <= a_end, a.status)) st_chunk(addr, o[0], o[1], o[2], o[3]);
  };
  auto fill_tile = [&](int st) {
#pragma unroll
    for (int item = 0; item < 2; ++item) {
      const bool gr = grouped(item);
      const uint32_t at = item * 8 * 128;  // rows 64 item ..
      if (gr && whole[st * 8 + 4 * item + my_block]) {
        uint32_t x[3];
#pragma unroll
        for (int i = 0; i < 3; ++i)
          x[i] = ((w[item][i] >> my_swap) & 0x0F0F0F0Fu) | ((w[item][i] << my_swap) & 0xF0F0F0F0u);
        uint32_t o[4][4];
        vdeq_group(x[0], x[1], x[2], tl0, tl1, th0, th1, o);  // o[j]: member j, swapped in pairs
        put(at + my_even, o[0]);
        put(at + my_odd, o[1]);
        put(at + my_even + 128, o[2]);
        put(at + my_odd + 128, o[3]);
      }
      if (gr && whole[st * 8 + 4 * item + (my_row >> 4)]) continue;
      const TileRow r = rows[st * kTile + 64 * item + my_row];
      if (r.blk == nullptr) continue;
      if (gr) {
        int B, t, j;
        vt_slot(r.pos & (kPage - 1), B, t, j);
#pragma unroll
        for (int p = 0; p < 4; p += 2) {  // units 4 my_q + p, + 1: 24 bytes, 8-byte aligned
          const int go = vt_group_off(D, B, t, 4 * my_q + p);
          if (!in_bounds(go + 24 <= kPage * CB, a.status)) continue;
          const uint2* g = reinterpret_cast<const uint2*>(r.blk + v_codes_off(D, 3) + go);
          const uint2 x = __ldg(g), y = __ldg(g + 1), z = __ldg(g + 2);
          uint32_t o[4];
          deq8(member_unit(x.x, x.y, y.x, j), tl0, tl1, th0, th1, o);
          put(at + my_chunk + p * 2048, o);
          deq8(member_unit(y.y, z.x, z.y, j), tl0, tl1, th0, th1, o);
          put(at + my_chunk + (p + 1) * 2048, o);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t o[4];
          kdeq<BITS>(w[item], j, tl0, tl1, th0, th1, o);
          put(at + my_chunk + j * 2048, o);
        }
      }
    }
    if (tid < kTile) nrm[st * kTile + tid] = __half2float(__ushort_as_half(my_norm));
  };

  // ---- R into shared memory, tensor memory, the first tiles' rows and words -------------
  if (warp == 0) tc::alloc(tmem_slot, kTileCols);
  if (tid == 0) {
    mbar_init(done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // Column n of R is (-1)^popc(k & dim) times one of four sums of block k / 4's row, by dim % 4 (the
  // Sylvester matrix's rows 4 kb + j, j = 0..3): 4 d values in all, two a thread.  They go to the
  // operand tile's place, [k / 8][dim % 4][k % 8], the second part behind the first.
  static_assert(4 * D == 2 * NT, "two values a thread");
  const float4* mat = reinterpret_cast<const float4*>(a.mats + (size_t)h * D * 4);
  float4 m[2];  // row x % 4 of block x / 16, x = tid, tid + NT
#pragma unroll
  for (int y = 0; y < 2; ++y) m[y] = __ldg(mat + ((tid + y * NT) >> 4) * 4 + (tid & 3));
  fetch_token(first);
  fetch_page();
  constexpr double kUnit = kRotScale / (D == 256 ? 16.0 : 11.313708498984761);  // / sqrt(d)
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const int kb = (tid + y * NT) >> 4, row = tid & 3, odd = (tid >> 2) & 3;
    const float2 r = scaled_sum(m[y].x, (odd & 1) ? -m[y].y : m[y].y, (odd & 2) ? -m[y].z : m[y].z,
                                (odd == 1 || odd == 2) ? -m[y].w : m[y].w, (float)kUnit,
                                (float)(kUnit - (double)(float)kUnit));
    const int at = (kb >> 1) * 32 + odd * 8 + (kb & 1) * 4 + row;
    if (!in_bounds(at < 4 * D, a.status)) continue;
    __half* t = reinterpret_cast<__half*>(smem + SM::kOffA) + at;
    t[0] = __float2half_rn(r.x);
    if constexpr (LO) t[4 * D] = __float2half_rn((r.x - __half2float(t[0])) + r.y);
  }
  fetch_token(first + step);
  put_row(0);
  fetch_page();
  fetch_token(first + 2ll * step);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = __shfl_sync(kFull, *tmem_slot, 0);
  const int role = __shfl_sync(kFull, warp, 0);  // warp-uniform to the compiler as well
  load_words(0);
  {
    const int n = tid & 127, dim = read_column(D, q, n);  // R in the no-swizzle K-major layout:
#pragma unroll
    for (int k8 = tid >> 7; k8 < D / 8; k8 += NT / 128) {  // 16 bytes of k = 8 k8 .. + 7, column n
      const uint32_t s0 = (__popc(8 * k8 & dim) & 1) ? 0x80008000u : 0u;
      const uint32_t s1 = (__popc((8 * k8 + 4) & dim) & 1) ? 0x80008000u : 0u;
#pragma unroll
      for (int part = 0; part < (LO ? 2 : 1); ++part) {
        const uint4 v = *reinterpret_cast<const uint4*>(smem + SM::kOffA + part * 8 * D + k8 * 64 + (dim & 3) * 16);
        if (in_bounds(part * SM::kPart + k8 * 2048 + n * 16 + 16 <= SM::kOffA, a.status))
          st_chunk(sB + part * SM::kPart + k8 * 2048 + n * 16, v.x ^ s0, v.y ^ s0, v.z ^ s1, v.w ^ s1);
      }
    }
  }
  __syncthreads();  // the sums have been read: the operand tile takes their place

  const int row0 = 32 * (warp & 3) + 16 * ((warp >> 2) & 1);  // tensor-memory lanes row0 ..
  const uint32_t t_rows = tmem + ((uint32_t)row0 << 16);
  const bool my_side = side_of(row0 >> 6);                    // warp-uniform
  T* const my_out = static_cast<T*>(out_of(row0 >> 6)) + (size_t)h * D;
  const int my_dim = read_column(D, q, 2 * (lane & 3));       // first of 16, in the first half
  const bool wide = (((uintptr_t)my_out) & 31) == 0;
  // Byte of chunk c of a row of the staged table: 8 lanes read chunks 8 t + i of two rows for t
  // = 0..3 at once, so the low bits of c are turned by t and the row's parity.
  [[maybe_unused]] const uint32_t sT = smem_u32(smem + SM::kOffTable);
  [[maybe_unused]] auto table_at = [](int r, int c) {
    return r * 512 + (((c & 24) | ((c & 7) ^ ((c >> 3) | (r & 1) << 2))) << 4);
  };
  // x = n / sqrt(d) . acc / (ALPHA kRotScale)
  const float unit_scale = rsqrtf((float)D) / (alpha_of<BITS>() * kRotScale);
  bool fail = false, pending = false, ok = true;
  int k = 0, st = 0;
  for (int tile = first; tile < n_tiles; tile += step, ++k) {
    const int st1 = st == 2 ? 0 : st + 1;
    fill_tile(st);
    put_row(st1);
    fence_proxy_async();  // the tile's generic-proxy writes, before the tensor core reads them
    tc::fence_before();
    if (__syncthreads_or(!ok)) {  // the tile's only barrier without a rotary table
      fail = true;
      break;
    }
    if (role == 0) {
      tc::fence_after();
      const uint64_t ad = tc::sdesc(sA, 2048, 128), bd = tc::sdesc(sB, 2048, 128);
      if (tc::elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {  // descriptors count 16 bytes
          tc::mma_ss(tmem, ad + kk * 256, bd + kk * 256, kId, kk > 0);
          if constexpr (LO) tc::mma_ss(tmem, ad + kk * 256, bd + SM::kPart / 16 + kk * 256, kId, 1);
        }
        tc::commit(done);
      }
      __syncwarp();
    }
    pending = true;
    if constexpr (ROPE) {  // the table's rows of this tile, while the product runs
#pragma unroll
      for (int x = tid; x < 64 * 32; x += NT) {
        const int r = x >> 5, c = x & 31;  // 16-byte chunk c (two pairs) of row r
        const TileRow t = rows[st * kTile + r];
        if (t.blk != nullptr && in_bounds(t.pos < a.rope_max_pos, a.status))
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sT + table_at(r, c)),
                       "l"(a.rope + ((size_t)t.pos * (D / 2) + 64 * q + 2 * c) * 2)
                       : "memory");
      }
    }
    if (tile + step < n_tiles) load_words(st1);
    fetch_page();
    fetch_token(tile + 3ll * step);

    // ---- the product's rows: scale, rotary embedding, round, out --------------------------
    ok = __all_sync(kFull, mbar_wait(done, k & 1));  // warp-uniform: collective loads
    if constexpr (ROPE) {
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncthreads();
    }
    if (!ok) continue;  // reported at the next barrier (or after the loop)
    pending = false;
    tc::fence_after();
#pragma unroll
    for (int x = 0; x < kHalves; ++x) {
      const int hf = D == 128 ? x : warp >> 3;
      uint32_t v[32];
      [[maybe_unused]] uint32_t u[32];  // the other half: the rotary partners
      tc::ld16x64(t_rows + 64 * hf, v);
      if constexpr (ROPE) {
        if (!my_side) tc::ld16x64(t_rows + 64 * (hf ^ 1), u);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {  // rows row0 + lane / 4 + 8 e
        const int row = row0 + (lane >> 2) + 8 * e;
        const TileRow r = rows[st * kTile + row];
        if (r.blk == nullptr || !in_bounds(token_of(tile, row) < a.n_tokens, a.status)) continue;
        const float c = nrm[st * kTile + row] * unit_scale;
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float2 y = make_float2(__uint_as_float(v[4 * i + 2 * e]), __uint_as_float(v[4 * i + 2 * e + 1]));
          if constexpr (ROPE) {
            if (!my_side) {
              // (cos, sin) of the pairs my_dim + 2 i, + 1: a cos + b sin, or b cos - a sin
              const float4 t =
                  *reinterpret_cast<const float4*>(smem + SM::kOffTable + table_at(row, 8 * (lane & 3) + i));
              const float s0 = hf ? -t.y : t.y, s1 = hf ? -t.w : t.w;
              y = make_float2(fmaf(__uint_as_float(u[4 * i + 2 * e]), s0, y.x * t.x),
                              fmaf(__uint_as_float(u[4 * i + 2 * e + 1]), s1, y.y * t.z));
            }
          }
          o[i] = pack2<T>(f2_mul(y, make_float2(c, c)));
        }
        st_sector(my_out + (size_t)token_of(tile, row) * a.n_kv_heads * D + my_dim + hf * (D / 2), o, wide);
      }
    }
    tc::fence_before();  // the accumulator has been read: the next product may overwrite it
    st = st1;
  }
  if (__syncthreads_or(!ok) || fail) {
    // a bounded wait gave up: wait (bounded) for what is in flight, then release
    if (tid == 0) set_status(a.status, ISOQ_ST_TIMEOUT);
    if (pending) mbar_wait(done, (k - 1) & 1);
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after();
    tc::dealloc(tmem, kTileCols);
  }
}

template <int D, int BITS, typename T, bool LO, bool ROPE>
cudaError_t launch_tc(const DequantizeArgs& a, cudaStream_t stream, int n_sm) {
  using SM = ReadSmem<D, LO, ROPE>;
  static unsigned long long attr_set = 0;  // the shared-memory opt-in, per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !((attr_set >> dev) & 1ull)) {
    e = cudaFuncSetAttribute(dequantize_tc_kernel<D, BITS, T, LO, ROPE>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, SM::kBytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_set |= 1ull << dev;
  }
  const int per_tile = ROPE || (a.K && a.V) ? 64 : 128;
  const int n_tiles = (int)(((long long)a.n_tokens + per_tile - 1) / per_tile);
  const long long units = (long long)a.n_kv_heads * (D / 128);
  long long per_unit = (long long)n_sm * read_ctas<D, LO>(ROPE) / units;
  if (per_unit < 1) per_unit = 1;
  if (per_unit > n_tiles) per_unit = n_tiles;
  dequantize_tc_kernel<D, BITS, T, LO, ROPE><<<(unsigned)(units * per_unit), 2 * D, SM::kBytes, stream>>>(
      a, (int)units, n_tiles);
  return cudaGetLastError();
}

template <int D, int BITS>
cudaError_t launch_tc_t(const DequantizeArgs& a, cudaStream_t stream, int n_sm) {
  if (a.dtype == ISOQ_BF16)
    return a.rope ? launch_tc<D, BITS, __nv_bfloat16, false, true>(a, stream, n_sm)
                  : launch_tc<D, BITS, __nv_bfloat16, false, false>(a, stream, n_sm);
  if constexpr (D == 128) {
    if (a.rope) return launch_tc<D, BITS, __half, true, true>(a, stream, n_sm);
  }
  return launch_tc<D, BITS, __half, true, false>(a, stream, n_sm);
}

}  // namespace

// From 2^20 elements on (8192 vectors of 128, 4096 of 256): below, making R and the chain of
// one tile cost more than the warp kernel's shuffles.  Measured, 8 KV heads, d = 128 / 256, us a
// call (this kernel | the warp kernel), bf16: 256 tokens 5.1 | 3.7 / 6.4 | 6.0, 512 tokens
// 5.1 | 5.0 / 6.6 | 10.4, 4096 tokens 9.8 | 17.5 / 22.0 | 32.9; fp16: 512 tokens 5.7 | 5.1 /
// 7.5 | 10.4, 1024 tokens 5.8 | 8.0 / 10.5 | 18.8.  fp16 with the rotary embedding at d =
// 256 stays with the warp kernel: both parts of R leave no room for the staged table, and
// reading it in place took 330 us for 32768 tokens against 280.
bool use_dequantize_tc(const DequantizeArgs& a) {
  const long long vectors = (long long)a.n_tokens * a.n_kv_heads * ((a.K != nullptr) + (a.V != nullptr));
  if (a.dtype == ISOQ_F32 || (a.dtype == ISOQ_F16 && a.d == 256 && a.rope)) return false;
  return vectors * a.d >= (1ll << 20);
}

cudaError_t launch_dequantize_tc(const DequantizeArgs& a, cudaStream_t stream, int n_sm) {
  if (a.d == 256) return launch_tc_t<256, 3>(a, stream, n_sm);
  switch (a.bits) {
    case 2: return launch_tc_t<128, 2>(a, stream, n_sm);
    case 3: return launch_tc_t<128, 3>(a, stream, n_sm);
    case 4: return launch_tc_t<128, 4>(a, stream, n_sm);
  }
  return cudaErrorInvalidValue;
}

}  // namespace isoq
