// Matrix products grouped by expert with ragged sizes, on operands that need no dequantization: 16-bit
// floats (w16.hip) and 8-bit integers (i8.hip).
//
// The groups come as expert_offsets [E + 1] (moe_align's prefix sums): expert e owns the rows
// [offsets[e], offsets[e + 1]).  Three products share one kernel:
//   FWD: C[r, n]     = sum_k A[a(r), k] * W[e, n, k]          e the expert of row r
//   DX:  dA[r, k]    = sum_n dC[r, n] * W[e, n, k]
//   DW:  dW[e, n, k] = sum_{r of e} dC[r, n] * A[a(r), k]
// A workgroup computes a BM x BN tile of the output.  The contraction runs in steps of RB bytes an
// operand row (RB / 2 16-bit or RB integer elements); a step's two operand tiles reach LDS by direct
// global->LDS 16-byte loads through a ring of stages, one barrier per step.  An operand whose
// contraction axis is contiguous in memory ("rows") is kept as [row][RB bytes]; one whose other axis is
// contiguous (W in DX, both in DW) as [contraction row][tile columns], and its fragments are read with
// the transposing LDS load (ds_read_b64_tr_b16: a 16-lane group reads a 4 x 16 block and lane j gets
// column j).  16-byte chunks are XOR-swizzled so that neither kind of fragment read has bank conflicts (the results'
// way through LDS has: a third of the LDS cycles of bf16 weight gradients with 25 rows a group, whose results outweigh
// their contraction; 2-5 % of the others').
//
// What bounds it.  Many rows: the barrier of a step, one workgroup of 8 waves a CU, and clocks that fall with the matrix
// units' load (a dense library product of fp16 reaches 1.53 PFLOP/s on this card, of int8 2.15 POP/s): fp16 8 experts
// of 4096 x 14336 over 8192 rows 930-980 us (0.98-1.03 PFLOP/s, units busy 51 % of the cycles; about 2.5 rounds of tiles
// where the rows fill 2.0), int8 4096 x 28672 x 4096 402-412 us (2.3-2.4 POP/s, 52 %).  Few rows: the weights' bytes,
// many small workgroups a CU: 64 rows over 128 experts of 1536 x 2048, int8 28 us, bf16 57 us (5.7-5.9 TB/s).
//
// Fragments of v_mfma_f32_16x16x32 (16-bit) and v_mfma_i32_16x16x64_i8: lane l supplies 16 bytes, row
// l % 16, contraction bytes [16 (l / 16), +16) of a 64-byte group.  The weight fragment is the first
// operand, so a lane's four results are four neighbouring columns of one output row and are stored
// together.
#pragma once
#include <type_traits>

#include "launch.h"
#include "moe_common.h"

namespace moe {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int16_t i16x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

// Element kinds of the ragged products.
struct ElemBF16 {
  using Acc = f32x4;
  static constexpr int kBytes = 2;
  static __device__ __forceinline__ Acc mfma(const u32x4& a, const u32x4& b, const Acc& c) {
    return mfma16x16x32(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c);
  }
};
struct ElemF16 {
  using Acc = f32x4;
  static constexpr int kBytes = 2;
  static __device__ __forceinline__ Acc mfma(const u32x4& a, const u32x4& b, const Acc& c) {
    return mfma16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c);
  }
};
struct ElemI8 {
  using Acc = i32x4;
  static constexpr int kBytes = 1;
  static __device__ __forceinline__ Acc mfma(const u32x4& a, const u32x4& b, const Acc& c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
  }
};

enum RaggedMode { kFwd = 0, kDx = 1, kDw = 2 };

// What lanes past an operand's end load instead: zeros, so that they add nothing to the product.
static __device__ const u32x4 kZeroChunk = {0u, 0u, 0u, 0u};

// 16-byte chunk permutation of an operand kept as rows of RB bytes.  A 16-byte LDS read serves 16 lanes a
// cycle, not 16 neighbours but lanes 0-3, 12-15 and 20-27 together, and the rest likewise: of a fragment
// read, rows 0-3 and 12-15 at one chunk column with rows 4-11 at the next.  Both permutations put those 16
// chunks into 16 different places of the 256-byte bank line (measured: plain (row / 4) % 4 for 64-byte rows
// doubled the LDS cycles).
template <int RB>
__device__ __forceinline__ int row_swizzle(int row) {
  return RB == 64 ? ((row >> 3) & 1) | ((((row >> 2) ^ (row >> 3)) & 1) << 1) : (row >> 1) & 7;
}
// 32-byte window permutation of an operand kept as contraction rows: a transposing read covers 4 rows of
// each 16-lane group, groups 8 rows apart; the eight rows of half a wave fall in eight different windows.
__device__ __forceinline__ int col_swizzle(int crow) { return (crow & 3) | ((crow >> 1) & 4); }

// Direct global->LDS loads to a wave-uniform LDS byte address (lane l writes [16l, 16l+16), or [4l, 4l+4) from
// it); the second takes a uniform base and a 32-bit offset a lane, the third the same for bytes that no other workgroup
// reads (nontemporal).  The compiler adds no wait states inside assembly, and two are the program's to keep: one
// after a scalar write of m0, and five after a vector instruction's write of the scalar base (v_readfirstlane, or
// v_readlane of a spilled register; without them the load has taken an address of old and new halves).  A scalar
// copy of the base waits for such a write by itself, and is the one state that m0 needs.
__device__ __forceinline__ void g2lds16_at(const void* g, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(g), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ void g2lds16_at(const void* base, uint32_t off, uint32_t lds) {
  const void* copy;
  asm volatile("s_mov_b64 %0, %2\n\tglobal_load_lds_dwordx4 %1, %0" : "=&s"(copy) : "v"(off), "s"(base), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ void g2lds16_once_at(const void* base, uint32_t off, uint32_t lds) {
  const void* copy;
  asm volatile("s_mov_b64 %0, %2\n\tglobal_load_lds_dwordx4 %1, %0 nt" : "=&s"(copy) : "v"(off), "s"(base), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ void g2lds4_at(const void* g, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" : : "v"(g), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p);
}

// A row tile of the ragged groups: expert, first row, rows (at most the tile's height), height class.
struct RowTile {
  int e, row0, rows, cls;
};

__device__ __forceinline__ int group_end(const int32_t* off, int i, int R) { return min(max(off[i], 0), R); }

// Row tiles of one group, in one height H0 or two, H0 = 2 H1 (H1 zero: not there): whole tiles of H0, and the rest in
// the smaller height where that holds it, so that at most H1 - 1 padding rows (with one height H0 - 1) are multiplied.
struct TileCount {
  int n0, n1;
};
template <int H0, int H1>
__device__ __forceinline__ TileCount count_tiles(int rows) {
  const int rest = rows % H0;
  TileCount c{rows / H0, 0};
  if (H1 == 0 || rest > H1) c.n0 += rest > 0;
  else c.n1 = rest > 0;
  return c;
}

// Work order.  Workgroup b runs on XCD b % 8, each XCD with its own L2.  The output tiles of all experts,
// expert after expert, form one list per height, the highest first (the short ones then fill the end of the
// launch), and the XCDs share each list in contiguous eighths.  An expert's tiles (nt row tiles x nbn column
// blocks) are listed in bands of 8 row tiles, down a band's rows first: the 32 tiles that an XCD's CUs work on
// together form a block about as wide as high, so that its L2 takes in few rows of either operand.
constexpr int kBand = 8;
__device__ __forceinline__ void band_place(long long i, int nt, int nbn, int& tile, int& nb) {
  const long long band = (long long)kBand * nbn;
  const int g = (int)(i / band);
  const int r = (int)(i - g * band);
  const int high = min(kBand, nt - g * kBand);
  nb = r / high;
  tile = g * kBand + (r - nb * high);
}

// Takes this workgroup's XCD's share of a list of `total` tiles from its number j on the XCD: true and the place
// in the list, or false with the share taken off j.
__device__ __forceinline__ bool list_place(long long total, long long& j, long long& at) {
  const long long xcd = linear_block() & 7;
  const long long from = (xcd * total) >> 3, to = ((xcd + 1) * total) >> 3;
  at = from + j;
  if (at < to) return true;
  j -= to - from;
  return false;
}

// Inclusive sum of v over the lanes up to this one.
__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(v, d);
    if (lane >= d) v += u;
  }
  return v;
}

// The last round of the highest tiles, cut in halves.  An XCD's 32 CUs take its share of the list 32 tiles at a time (one
// workgroup a CU); where tiles are left over and would cost a round of their own, they are dealt as two tiles of the next
// height each, if that ends sooner beside the lower tiles (counted in lower tiles' time) and the grid has the workgroups
// for it.  True, with the place of the whole tile and its half, if workgroup j takes such a half; otherwise j is moved on
// to what the lists still hold.  bf16 1280 x 14336 x 4096 190 -> 154 us, 4352 x 8192 x 4096 314 -> 297 us; fp16 8 experts
// of 4096 x 14336 whose 528 tiles stand over two rounds of 256 1070 -> 985 us; where nothing is cut the same within 1 %.
constexpr int kXcdCus = 32;
constexpr int kHalvedHeight = 256;  // tiles of one workgroup a CU
__device__ __forceinline__ bool list_halved(int incl0, int n1, int nbn, long long& j, long long& at, int& half) {
  const long long total0 = (long long)__builtin_amdgcn_readlane(incl0, 63) * nbn, xcd = linear_block() & 7;
  const long long total1 = (long long)__builtin_amdgcn_readlane(wave_scan(n1, threadIdx.x & 63), 63) * nbn;
  const long long from = (xcd * total0) >> 3, count = (((xcd + 1) * total0) >> 3) - from;
  const long long lower = (((xcd + 1) * total1) >> 3) - ((xcd * total1) >> 3);
  const long long rest = count % kXcdCus, beside = 2 * (kXcdCus - rest);
  if (rest == 0 || j < count - rest) return false;
  if (((long long)gridDim.x * gridDim.y) >> 3 < count + rest + lower) return false;
  const long long whole = 2 + (lower > beside ? (lower - beside + kXcdCus - 1) / kXcdCus : 0);
  if ((2 * rest + lower + kXcdCus - 1) / kXcdCus >= whole) return false;
  const long long i = j - (count - rest);
  if (i < 2 * rest) {
    at = from + (count - rest) + (i >> 1);
    half = (int)(i & 1);
    return true;
  }
  j -= rest;  // 2 rest workgroups for rest tiles
  return false;
}

// Finds the workgroup's row tile and column block from the offsets: every wave takes PER consecutive experts a
// lane (all their offsets in one round trip), counts their tiles, scans the counts over its lanes, and the lane
// that holds the wanted tile finds its expert.  Offsets are clamped to [0, R], so no list of offsets leads out
// of the rows.
template <int H0, int H1, int PER>
__device__ __forceinline__ bool find_row_tile_per(const int32_t* __restrict__ off, int E, int R, int nbn, RowTile& t, int& nb) {
  const int lane = threadIdx.x & 63;
  int end[PER + 1];  // offsets of this lane's experts; past the last expert the groups are empty
#pragma unroll
  for (int i = 0; i <= PER; ++i) {
    const int e = min(lane * PER + i, E);
    end[i] = off ? group_end(off, e, R) : (e > 0 ? R : 0);  // without offsets one group holds all rows
  }
  TileCount n{0, 0};
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const TileCount c = count_tiles<H0, H1>(max(end[i + 1] - end[i], 0));
    n.n0 += c.n0;
    n.n1 += c.n1;
  }
  long long j = linear_block() >> 3, item;
  int incl = wave_scan(n.n0, lane), mine = n.n0, cls = 0, half = 0;
  bool halved = false;
  if constexpr (H1 > 0 && H0 >= kHalvedHeight) halved = list_halved(incl, n.n1, nbn, j, item, half);
  if (!halved && !list_place((long long)__builtin_amdgcn_readlane(incl, 63) * nbn, j, item)) {
    if (H1 == 0) return false;
    incl = wave_scan(n.n1, lane), mine = n.n1, cls = 1;
    if (!list_place((long long)__builtin_amdgcn_readlane(incl, 63) * nbn, j, item)) return false;
  }
  const int place = (int)(item / nbn);  // names the expert: its tiles x nbn items follow each other
  const int src = __builtin_ctzll(__ballot(incl > place));  // place < total: some lane's sum is past it
  // every lane walks its own experts; lane src's answer counts
  int before = incl - mine, at_i = 0, at_before = before, at_nt = 0, r0 = 0, r1 = 0, full0 = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const TileCount c = count_tiles<H0, H1>(max(end[i + 1] - end[i], 0));
    const int nt = cls == 0 ? c.n0 : c.n1;
    if (i == 0 || before <= place) at_i = i, at_before = before, at_nt = nt, r0 = end[i], r1 = end[i + 1], full0 = c.n0;
    before += nt;
  }
  at_i = __builtin_amdgcn_readlane(at_i, src);
  at_before = __builtin_amdgcn_readlane(at_before, src);
  at_nt = __builtin_amdgcn_readlane(at_nt, src);
  r0 = __builtin_amdgcn_readlane(r0, src);
  r1 = __builtin_amdgcn_readlane(r1, src);
  int tile;
  band_place(item - (long long)at_before * nbn, at_nt, nbn, tile, nb);
  int first = tile * H0, high = H0;
  if (H1 > 0 && cls > 0) {
    first = __builtin_amdgcn_readlane(full0, src) * H0;
    high = H1;
  }
  if (H1 > 0 && halved) {  // the upper or lower rows of a tile of the highest list
    first += half * H1;
    high = H1;
    cls = 1;
  }
  t = RowTile{src * PER + at_i, r0 + first, min(high, r1 - r0 - first), cls};
  return true;
}

template <int H0, int H1>
__device__ __forceinline__ bool find_row_tile(const int32_t* __restrict__ off, int E, int R, int nbn, RowTile& t, int& nb) {
  if (E <= 64) return find_row_tile_per<H0, H1, 1>(off, E, R, nbn, t, nb);
  if (E <= 128) return find_row_tile_per<H0, H1, 2>(off, E, R, nbn, t, nb);
  if (E <= 256) return find_row_tile_per<H0, H1, 4>(off, E, R, nbn, t, nb);
  if (E <= 512) return find_row_tile_per<H0, H1, 8>(off, E, R, nbn, t, nb);
  return find_row_tile_per<H0, H1, MOE_MAX_EXPERTS / 64>(off, E, R, nbn, t, nb);
}

__device__ __forceinline__ void store4(void* C, int out, size_t at, const float (&v)[4]) {
  if (out == MOE_OUT_F32) {
    *reinterpret_cast<f32x4*>(static_cast<float*>(C) + at) = f32x4{v[0], v[1], v[2], v[3]};
  } else {
    u16x4 b;
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = out == MOE_OUT_F16 ? f32_to_f16_bits(v[i]) : f32_to_bf16_bits(v[i]);
    *reinterpret_cast<u16x4*>(static_cast<uint16_t*>(C) + at) = b;
  }
}
__device__ __forceinline__ void store1(void* C, int out, size_t at, float v) {
  if (out == MOE_OUT_F32) static_cast<float*>(C)[at] = v;
  else static_cast<uint16_t*>(C)[at] = out == MOE_OUT_F16 ? f32_to_f16_bits(v) : f32_to_bf16_bits(v);
}

// Rows whose gathered indexes DW keeps in LDS at a time (a pass drains the ring of stages).
constexpr int kDwIds = 1024;

// Shape of one tile height's work: BM x BN by WM x WN waves, steps of RB bytes, NA stages of the A operand's tile
// and NB >= NA of the B operand's.  ONCE: for groups that are one tile high on the average, so that the B operand is read once.
template <int BM_, int BN_, int WM_, int WN_, int RB_, int NA_, int NB_ = NA_, bool ONCE_ = false>
struct TileShape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, RB = RB_, NA = NA_, NB = NB_;
  static constexpr bool ONCE = ONCE_;
  static constexpr int kLds = (NA * BM + NB * BN) * RB;
};
struct NoTile {
  static constexpr int BM = 0, BN = 0, WM = 0, WN = 0, RB = 0, NA = 0, NB = 0, kLds = 0;
  static constexpr bool ONCE = false;
};

// One output tile: rows t (DW: weight rows from m0) by column block nb.
// LATE: the bytes of the scales where they are loaded after the contraction, into the first stages (int8 tiles whose
// stages fill the LDS), else 0.
template <class T, int MODE, int EPI, class S, int LATE>
__device__ __forceinline__ void ragged_tile(const RaggedArgs& p, const RowTile& t, int nb, int m0, uint8_t* smem, int32_t* sRow,
                                            float* sScaleA, float* sScaleW) {
  constexpr int BM = S::BM, BN = S::BN, WM = S::WM, WN = S::WN, RB = S::RB, NA = S::NA, NB = S::NB;
  constexpr int NW = WM * WN;
  constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
  constexpr bool A_T = MODE == kDw, B_T = MODE != kFwd;  // operand kept as contraction rows
  constexpr bool I8 = T::kBytes == 1;
  constexpr int CR = RB / T::kBytes;  // contraction elements per step
  constexpr int SA = BM * RB, SB = BN * RB;
  constexpr int LA = SA / 1024, LB = SB / 1024;                        // wave-wide loads of a step
  constexpr int JA = (LA + NW - 1) / NW, JB = (LB + NW - 1) / NW;      // of one wave, at most
  constexpr int LMIN = LA / NW + LB / NW;                              // and at least
  // loads behind those of the next step when it is about to be read (see run)
  constexpr int BEHIND = (NA - 2) * LMIN + (NB > NA ? LB / NW : 0);
  static_assert(EPI != MOE_EPI_SILU_MUL || (MODE == kFwd && NI % 2 == 0), "SiLU*mul pairs gate and up blocks");
  static_assert((!I8 || BN % 64 == 0) && (!B_T || BN >= 128) && (!A_T || BM >= 128), "scales are loaded by 64 columns, windows permuted by 8");
  static_assert(!I8 || MODE == kFwd, "transposing reads are of 16-bit elements");
  static_assert(BM <= NW * 64 && (RB == 64 || RB == 128), "rows");
  // (issue_a, issue_b: a wave without a last load would not move its uniform base on)
  static_assert((LA % NW == 0 || JA == 1) && (LB % NW == 0 || JB == 1), "every wave has all its loads, or at most one");
  static_assert(SA % 1024 == 0 && SB % 1024 == 0 && LMIN >= 1 && BEHIND < 64 && NA >= 2 && NB - NA <= 1 && NB >= NA && NW % 2 == 0, "loads");

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int l16 = lane & 15, q = lane >> 4;
  const int N = p.N, K = p.K;
  // output columns and contraction length
  const int ND = MODE == kFwd ? (EPI == MOE_EPI_SILU_MUL ? N / 2 : N) : K;
  constexpr int BC = EPI == MOE_EPI_SILU_MUL ? BN / 2 : BN;  // output columns of a tile
  int my_row = 0;  // the activation row of tile row tid
  if constexpr (MODE != kDw) {
    if (tid < BM) {  // padding rows repeat the tile's first row
      const int r = t.row0 + (tid < t.rows ? tid : 0);
      my_row = MODE == kFwd && p.a_row_of ? p.a_row_of[r] / p.a_row_div : r;
      sRow[tid] = my_row;
    }
    __syncthreads();
  }
  const size_t w_e = (size_t)t.e * N * K;  // first element of the expert's weights
  const uint8_t* A = static_cast<const uint8_t*>(p.A);
  const uint8_t* W = static_cast<const uint8_t*>(p.W);
  const uint8_t* zero = reinterpret_cast<const uint8_t*>(&kZeroChunk);
  const uint32_t lds0 = lds_address(smem);

  // weight row of tile column nt (a SiLU*mul wave's columns: its gate rows, then their up rows); columns past
  // the edge read row 0, which only reaches results that are not stored
  auto weight_row = [&](int nt) -> int {
    if (EPI == MOE_EPI_SILU_MUL) {
      constexpr int WC = BN / WN;
      const int in = nt % WC, h = nb * BC + (nt / WC) * (WC / 2) + in % (WC / 2);
      return h < ND ? (in < WC / 2 ? h : ND + h) : 0;
    }
    const int n = nb * BN + nt;
    return n < N ? n : 0;
  };
  // the tile's scales, for the epilogue
  auto load_scales = [&]() {
    if (wave < (BM + 63) / 64) g2lds4_at(p.As + my_row, lds_address(sScaleA) + wave * 256);
    for (int i = wave; i < BN / 64; i += NW)
      g2lds4_at(p.Ws + (size_t)t.e * N + weight_row(i * 64 + lane), lds_address(sScaleW) + i * 256);
  };
  if constexpr (I8 && LATE == 0) load_scales();  // older than every load of a stage

  // Sources of this wave's loads; load j of an operand is its wave-wide load wave + NW * j of a step.
  // Rows kind: lane's chunk at row (wave + NW j) * 1024 / RB + lane / (RB / 16), contraction byte pos in the step
  // (the permutation does not depend on j).  Contraction-rows kind: chunk of contraction row
  // (wave + NW j) * 1024 / width + lane / (width / 16); columns past the edge read the last ones, which only
  // reach results that are not stored.  Activations may lie anywhere (64-bit addresses); dC and one expert's
  // weights are addressed from a uniform base that advances from step to step (32-bit offsets).
  const int rows_row = (lane * 16) / RB;
  const int pos = 16 * ((((lane * 16) % RB) >> 4) ^ row_swizzle<RB>(wave * (1024 / RB) + rows_row));
  auto cols_row = [&](int j, int width) { return (wave + NW * j) * (1024 / width) + lane * 16 / width; };
  auto cols_off = [&](int j, int width, int col0, int cols) -> uint32_t {
    const int crow = cols_row(j, width);
    const int col = col0 + 8 * (((lane * 16 % width) >> 4) ^ (2 * col_swizzle(crow)));
    return ((uint32_t)crow * cols + min(col, cols - 8)) * 2;
  };
  const bool gather = MODE == kDw && p.a_row_of;
  const uint8_t* pa[JA];  // FWD
  uint32_t oa[JA], ob[JB];
  const uint8_t *base_a = nullptr, *base_b;
#pragma unroll
  for (int j = 0; j < JA; ++j) {
    const int row = min((wave + NW * j) * (1024 / RB) + rows_row, BM - 1);
    if (MODE == kFwd) pa[j] = A + (size_t)sRow[row] * K * T::kBytes + pos;
    else if (MODE == kDx) oa[j] = (uint32_t)(sRow[row] - t.row0) * N * 2 + pos;
    else oa[j] = cols_off(j, BM * 2, m0, N);
  }
  if (MODE == kDx) base_a = A + (size_t)t.row0 * N * 2;
  if (MODE == kDw) base_a = W + (size_t)t.row0 * N * 2;
#pragma unroll
  for (int j = 0; j < JB; ++j) {
    if (MODE == kFwd) {
      const int nt = min((wave + NW * j) * (1024 / RB) + rows_row, BN - 1);
      ob[j] = (uint32_t)weight_row(nt) * K * T::kBytes + pos;
    } else {
      ob[j] = cols_off(j, BN * 2, nb * BN, K);
    }
  }
  if (MODE == kDw) {
    base_b = A + (gather ? 0 : (size_t)t.row0 * K * 2);
    if (gather) {  // only the column remains; the row comes with its index
#pragma unroll
      for (int j = 0; j < JB; ++j) ob[j] -= (uint32_t)cols_row(j, BN * 2) * K * 2;
    }
  } else {
    base_b = W + w_e * T::kBytes;
  }
  const size_t step_a = MODE == kDw ? (size_t)CR * N * 2 : RB, step_b = MODE == kFwd ? RB : (size_t)CR * K * 2;

  if constexpr ((!I8 || LATE > 0) && MODE != kDw) __syncthreads();  // every wave has its rows: the stages may be filled

  // contraction elements of this pass (DW: rows of the expert, as many at a time as sRow holds) and its full steps
  int kd = MODE == kFwd ? K : N;
  int full = kd / CR;
  // Issue load j of step s's A or B tile into a stage; an operand's steps in turn.  FULL: the step is known to lie
  // within the contraction; past it zeros are loaded.
  auto issue_a = [&](int s, int stage, int j, auto whole) {
    constexpr bool FULL = decltype(whole)::value;
    const int left = FULL ? 0 : kd - s * CR;  // elements of this step
    const int i = wave + NW * j;
    if (LA % NW != 0 && i >= LA) return;
    const uint32_t to = lds0 + stage * SA + i * 1024;
    if (!FULL && s >= full) {
      const uint8_t* from = MODE == kFwd ? pa[j] : base_a + oa[j];
      if (A_T ? cols_row(j, BM * 2) >= left : pos >= left * T::kBytes) from = zero;
      g2lds16_at(from, to);
    } else if (MODE == kFwd) {
      g2lds16_at(pa[j], to);
    } else {
      g2lds16_at(base_a, oa[j], to);
    }
    if (MODE == kFwd) pa[j] += RB;
    else if (j == JA - 1) base_a += step_a;
  };
  auto issue_b = [&](int s, int stage, int j, auto whole) {
    constexpr bool FULL = decltype(whole)::value;
    const int left = FULL ? 0 : kd - s * CR;
    const int i = wave + NW * j;
    if (LB % NW != 0 && i >= LB) return;
    const uint32_t to = lds0 + NA * SA + stage * SB + i * 1024;
    const bool tail = !FULL && s >= full;
    if (MODE == kDw && gather) {
      const uint8_t* from = A + (size_t)sRow[min(s * CR + cols_row(j, BN * 2), kd - 1)] * K * 2 + ob[j];
      if (tail && cols_row(j, BN * 2) >= left) from = zero;
      g2lds16_at(from, to);
    } else if (tail) {
      const uint8_t* from = base_b + ob[j];
      if (B_T ? cols_row(j, BN * 2) >= left : pos >= left * T::kBytes) from = zero;
      g2lds16_at(from, to);
    } else if (S::ONCE) {
      g2lds16_once_at(base_b, ob[j], to);
    } else {
      g2lds16_at(base_b, ob[j], to);
    }
    if (j == JB - 1) base_b += step_b;
  };

  // This lane's fragments.  Rows kind: 16 bytes of row row0 + l16.  Contraction-rows kind: contraction rows
  // 8 q + 4 h + l16 / 4 of the group, whose window permutation depends on the lane alone.
  const int frag_r = l16 * RB, frag_x = row_swizzle<RB>(l16);
  auto frag_rows = [&](const uint8_t* tile, int row0, int kk) -> u32x4 {
    return *reinterpret_cast<const u32x4*>(tile + row0 * RB + (frag_r + 16 * ((kk * 4 + q) ^ frag_x)));
  };
  const int frag_g = (l16 >> 2) | ((q & 1) << 2), frag_c = 8 * q + (l16 >> 2);
  auto frag_cols = [&](const uint8_t* tile, int width, int col0, int kk) -> u32x4 {
    u32x2 half[2];
    const uint8_t* at = tile + (kk * 32 * width) + (frag_c * width + (((col0 >> 4) ^ frag_g) << 5) + 8 * (l16 & 3));
#pragma unroll
    for (int h = 0; h < 2; ++h)
      half[h] = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) i16x4*)(at + 4 * h * width)));
    return u32x4{half[0][0], half[0][1], half[1][0], half[1][1]};
  };

  typename T::Acc acc[MI][NI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi)
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = typename T::Acc{0, 0, 0, 0};

  // Fragments of one 64-byte group of a stage: the tile columns, and one half of the wave's row blocks.
  constexpr int KK = RB / 64;  // 64-byte groups of a step
  constexpr int HALVES = MI % 2 == 0 ? 2 : 1, MH = MI / HALVES;
  constexpr int PH = KK * HALVES;  // phases of a step
  u32x4 fa[2][MH], fb[2][NI];
  // Read r of a phase's fragments: its NI column blocks first where it starts a group, then its MH row blocks.
  auto read_one = [&](int stage_a, int stage_b, int kk, int half, int abuf, int bbuf, int r) {
    if (half == 0 && r < NI) {
      const uint8_t* tb = smem + NA * SA + stage_b * SB;
      const int c = wn * (BN / WN) + r * 16;
      fb[bbuf][r] = B_T ? frag_cols(tb, BN * 2, c, kk) : frag_rows(tb, c, kk);
    } else {
      const uint8_t* ta = smem + stage_a * SA;
      const int i = half == 0 ? r - NI : r;
      const int c = wm * (BM / WM) + (half * MH + i) * 16;
      fa[abuf][i] = A_T ? frag_cols(ta, BM * 2, c, kk) : frag_rows(ta, c, kk);
    }
  };

  // Step s lives in stages s % NA and s % NB.  A step is PH phases (64-byte group, half of the row blocks); the
  // reads of the next phase's fragments are spread between the matrix instructions of a phase.  Before the last
  // phase of a step every wave has read all of its stages: there the wave waits for its own loads of the next step
  // (BEHIND later ones may still be in flight), the barrier publishes everyone's, and the stages just read are
  // refilled with steps s + NA and s + NB, these loads too between the matrix instructions: issued together they
  // stood in front of the next reads (int8, 4096 x 28672 x 4096: spreading them took 7 % off).
  auto run = [&](int steps) {
#pragma unroll
    for (int s = 0; s < NB; ++s) {
      if (s >= steps) continue;
      if (s < NA) {
#pragma unroll
        for (int j = 0; j < JA; ++j) issue_a(s, s, j, std::false_type{});
      }
#pragma unroll
      for (int j = 0; j < JB; ++j) issue_b(s, s, j, std::false_type{});
    }
    // step s is about to be read; near the end the loads behind it are fewer
    auto arrive = [&](int s) {
      const int behind = steps - 1 - s;
      if (behind >= NB - 2) wait_vmcnt<BEHIND>();
      else if (NA == NB && NA > 3 && behind == NA - 3) wait_vmcnt<(NA > 3 ? NA - 3 : 0) * LMIN>();
      else wait_vmcnt<0>();
      __syncthreads();
    };
    if (steps >= NB) wait_vmcnt<BEHIND + LMIN>();
    else wait_vmcnt<0>();
    __syncthreads();
#pragma unroll
    for (int r = 0; r < NI + MH; ++r) read_one(0, 0, 0, 0, 0, 0, r);
    int ca = 0, cb = 0;  // stages of the present step
    // MID: step s + NB lies within the contraction, so nothing has to be asked
    auto step = [&](int s, auto parity, auto mid) {
      constexpr int P = decltype(parity)::value;  // buffers of the step's first phase
      constexpr bool MID = decltype(mid)::value;
      const int na = ca + 1 == NA ? 0 : ca + 1, nbs = cb + 1 == NB ? 0 : cb + 1;  // stages of the next step
#pragma unroll
      for (int ph = 0; ph < PH; ++ph) {
        const int abuf = (P * PH + ph) & 1, bbuf = (P * KK + ph / HALVES) & 1;
        const bool last = ph + 1 == PH;
        const int nh = (ph + 1) % HALVES, nkk = last ? 0 : (ph + 1) / HALVES;  // the next phase
        const int reads = nh == 0 ? NI + MH : MH, loads = last && MID ? JA + JB : 0;
        const bool more = !last || MID || s + 1 < steps;
        if (last && more) {
          if constexpr (MID) {
            wait_vmcnt<BEHIND>();
            __syncthreads();
          } else {
            arrive(s + 1);
#pragma unroll
            for (int j = 0; j < JA; ++j)
              if (s + NA < steps) issue_a(s + NA, ca, j, std::false_type{});
#pragma unroll
            for (int j = 0; j < JB; ++j)
              if (s + NB < steps) issue_b(s + NB, cb, j, std::false_type{});
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        constexpr int M = MH * NI;
#pragma unroll
        for (int m = 0; m < M; ++m) {
          const int i = (ph % HALVES) * MH + m / NI, ni = m % NI;
          acc[i][ni] = T::mfma(fb[bbuf][ni], fa[abuf][m / NI], acc[i][ni]);
          // one after each instruction, so that the reads are back before the phase (or the barrier) ends
          const int n = reads + loads, k0 = n > M ? m * n / M : m, k1 = n > M ? (m + 1) * n / M : (m < n ? m + 1 : m);
#pragma unroll
          for (int k = k0; k < k1; ++k) {
            __builtin_amdgcn_sched_barrier(0);
            if (k >= reads + JA) issue_b(s + NB, cb, k - reads - JA, std::true_type{});
            else if (k >= reads) issue_a(s + NA, ca, k - reads, std::true_type{});
            else if (more) read_one(last ? na : ca, last ? nbs : cb, nkk, nh, abuf ^ 1, bbuf ^ 1, k);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      ca = na;
      cb = nbs;
    };
    constexpr std::integral_constant<int, 0> even{};
    constexpr std::integral_constant<int, 1> odd{};
    int s = 0;
    for (; s + 1 + NB < full; s += 2) {
      step(s, even, std::true_type{});
      step(s + 1, odd, std::true_type{});
    }
    for (; s + 1 < steps; s += 2) {
      step(s, even, std::false_type{});
      step(s + 1, odd, std::false_type{});
    }
    if (s < steps) step(s, even, std::false_type{});
  };
  if constexpr (MODE == kDw) {
    for (int pass = 0; pass < t.rows; pass += kDwIds) {
      kd = min(t.rows - pass, kDwIds);
      full = kd / CR;
      __syncthreads();  // the last pass's indexes and stages are no longer read
      if (gather) {
        for (int i = tid; i < kd; i += NW * 64) sRow[i] = p.a_row_of[t.row0 + pass + i] / p.a_row_div;
        __syncthreads();
      }
      run((kd + CR - 1) / CR);
    }
  } else {
    run((kd + CR - 1) / CR);
  }

  if constexpr (I8 && LATE > 0) {
    __syncthreads();  // the stages are no longer read
    load_scales();
    wait_vmcnt<0>();
    __syncthreads();
  }
  // Epilogue: lane (q, l16) holds columns 4q .. 4q+3 of each 16 x 16 block, of row l16.
  constexpr int NO = EPI == MOE_EPI_SILU_MUL ? NI / 2 : NI;
  auto results = [&](int mi, int ni, float sa, float (&v)[4]) {
    f32x4 ws = {1.f, 1.f, 1.f, 1.f}, us = ws;
    if constexpr (I8) {  // the integer sums are exact; one scale a row and a channel
      ws = *reinterpret_cast<const f32x4*>(&sScaleW[wn * (BN / WN) + ni * 16 + 4 * q]);
      if constexpr (EPI == MOE_EPI_SILU_MUL)
        us = *reinterpret_cast<const f32x4*>(&sScaleW[wn * (BN / WN) + (ni + NO) * 16 + 4 * q]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = (float)acc[mi][ni][i];
      if constexpr (I8) v[i] *= sa * ws[i];
      if constexpr (EPI == MOE_EPI_SILU_MUL) {
        float u = (float)acc[mi][ni + NO][i];
        if constexpr (I8) u *= sa * us[i];
        v[i] = silu_f32(v[i]) * u;
      }
    }
  };
  const int rows = MODE == kDw ? min(N - m0, BM) : t.rows;
  const size_t first = MODE == kDw ? w_e + (size_t)m0 * K : (size_t)t.row0 * ND;  // the tile's first row in C
  // Results pass through LDS (the stages are free) and are stored as whole rows, 16 bytes a lane; stored from the
  // registers they are 32- or 64-byte pieces of 16 rows.  The stores do not stay in the L2 (nontemporal), which the
  // operands need: 16-bit weight gradients of 256 experts of 1024 x 2048 over 800 tokens take 385 us stored from the
  // registers, 285 us staged and 231 us staged past the L2; int8 products of 256 experts of 2048 x 512 with 32-bit
  // results 73, 72 and 67 us; int8 SiLU*mul 4096 x 8192 x 4096 122, 118 and 116 us.  Rows that do not begin on 64 bytes
  // stay, as the L2 has to put together the lines that two tiles share (16-bit weight gradients of 14 experts of 2424 x
  // 4528: 70 us, past the L2 113 us).
  // 16-bit results go in one piece, 32-bit ones a wave row (BM / WM rows) at a time.
  constexpr int kTop = LATE;  // the scales stay
  constexpr bool kStaged = BM >= (EPI == MOE_EPI_SILU_MUL ? 128 : 32);  // lower ones (SiLU*mul halves the rows) gain nothing
  auto staged = [&](auto bytes) {
    constexpr int ES = decltype(bytes)::value, PASSES = ES == 4 ? WM : 1, PR = BM / PASSES;
    constexpr int NCH = BC * ES / 16, CE = 16 / ES;  // 16-byte chunks of a row, permuted by the row's number
    uint8_t* buf = smem + kTop;
    const int cols = min(BC, ND - nb * BC);
#pragma unroll
    for (int ps = 0; ps < PASSES; ++ps) {
      __syncthreads();
      if (PASSES == 1 || wm == ps) {
#pragma unroll
        for (int mi = 0; mi < MI; ++mi) {
          const int row = wm * (BM / WM) + mi * 16 + l16;
          const float sa = I8 ? sScaleA[row] : 1.f;
#pragma unroll
          for (int ni = 0; ni < NO; ++ni) {
            float v[4];
            results(mi, ni, sa, v);
            const int col = wn * (BC / WN) + ni * 16 + 4 * q, chunk = col / CE;
            uint8_t* at = buf + (row - ps * PR) * (BC * ES) + ((chunk ^ (row & (NCH - 1) & 15)) * 16);
            if constexpr (ES == 4) {
              *reinterpret_cast<f32x4*>(at) = f32x4{v[0], v[1], v[2], v[3]};
            } else {
              u16x4 b;
#pragma unroll
              for (int i = 0; i < 4; ++i) b[i] = p.out == MOE_OUT_F16 ? f32_to_f16_bits(v[i]) : f32_to_bf16_bits(v[i]);
              *reinterpret_cast<u16x4*>(at + (q & 1) * 8) = b;
            }
          }
        }
      }
      __syncthreads();
      uint8_t* C = static_cast<uint8_t*>(p.C) + (first + nb * BC) * ES;
      auto copy_out = [&](auto way) {
#pragma unroll 4
        for (int i = tid; i < PR * NCH; i += NW * 64) {
          const int r = i / NCH, row = ps * PR + r, chunk = i % NCH;
          const u32x4 w = *reinterpret_cast<const u32x4*>(buf + r * (BC * ES) + ((chunk ^ (row & (NCH - 1) & 15)) * 16));
          if (row >= rows || chunk * CE >= cols) continue;
          u32x4* to = reinterpret_cast<u32x4*>(C + ((size_t)row * ND + chunk * CE) * ES);
          if constexpr (decltype(way)::value) __builtin_nontemporal_store(w, to);
          else *to = w;
        }
      };
      // (a loop of its own for each: a choice at every store would lose the hint)
      if ((size_t)ND * ES % 64 == 0) copy_out(std::true_type{});
      else copy_out(std::false_type{});
    }
  };
  if constexpr (kStaged) {
    if constexpr (kTop + BM * BC * 2 <= S::kLds) {
      if (p.out != MOE_OUT_F32 && (ND & 7) == 0) return staged(std::integral_constant<int, 2>{});
    }
    if constexpr (kTop + BM / WM * BC * 4 <= S::kLds) {
      if (p.out == MOE_OUT_F32 && (ND & 3) == 0) return staged(std::integral_constant<int, 4>{});
    }
  }
  const bool whole = (ND & 3) == 0;  // rows are stored four columns at a time
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    const int row = wm * (BM / WM) + mi * 16 + l16;
    if (row >= rows) continue;
    const size_t at = first + (size_t)row * ND;
    const float sa = I8 ? sScaleA[row] : 1.f;
#pragma unroll
    for (int ni = 0; ni < NO; ++ni) {
      const int col = nb * BC + wn * (BC / WN) + ni * 16 + 4 * q;
      if (col >= ND) continue;
      float v[4];
      results(mi, ni, sa, v);
      if (whole) {
        store4(p.C, p.out, at + col, v);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (col + i < ND) store1(p.C, p.out, at + col + i, v[i]);
      }
    }
  }
}

template <class T, int MODE, int EPI, class S0, class S1>
__global__ __launch_bounds__(S0::WM * S0::WN * 64) void ragged_gemm_kernel(RaggedArgs p) {
  constexpr int BM = S0::BM, BN = S0::BN;
  constexpr int kLds = S0::kLds > S1::kLds ? S0::kLds : S1::kLds;
  constexpr bool I8 = T::kBytes == 1;
  static_assert(S1::BM == 0 || (S1::BN == BN && S1::WM * S1::WN == S0::WM * S0::WN), "one grid and workgroup size");
  __shared__ __attribute__((aligned(16))) uint8_t smem[kLds];
  // the row indexes lie in what the last stage later takes, so that the stages may fill the LDS; int8 tiles keep
  // room for the scales where there is any
  constexpr int kScales = ((BM < 64 ? 64 : BM) + BN) * 4;  // of the highest tile, which the lower ones keep to
  constexpr int kLate = I8 && kLds + BM * 4 + kScales > 160 * 1024 ? kScales : 0;
  constexpr bool kShareRow = (!I8 || kLate > 0) && MODE != kDw;
  __shared__ int32_t sRowOwn[MODE == kDw ? kDwIds : (kShareRow ? 1 : BM)];
  int32_t* sRow = kShareRow ? reinterpret_cast<int32_t*>(smem + kLds - BM * 4) : sRowOwn;
  constexpr bool kOwnScales = I8 && kLate == 0;
  __shared__ __attribute__((aligned(16))) float sScaleOwn[kOwnScales ? kScales / 4 : 1];
  float* sScaleA = I8 && kLate > 0 ? reinterpret_cast<float*>(smem) : sScaleOwn;
  float* sScaleW = sScaleA + (BM < 64 ? 64 : BM);
  const int N = p.N, K = p.K;
  const int ND = MODE == kFwd ? (EPI == MOE_EPI_SILU_MUL ? N / 2 : N) : K;  // output columns
  constexpr int BC = EPI == MOE_EPI_SILU_MUL ? BN / 2 : BN;
  const int nbn = (ND + BC - 1) / BC;
  if constexpr (MODE == kDw) {
    // every expert's tiles are shared evenly by the XCDs (an expert with many rows keeps all of them
    // busy), each share a piece of the expert's list; fewer than 8 tiles an expert are dealt one by one
    const int nbm = (N + BM - 1) / BM, per_e = nbm * nbn;
    const long long b = linear_block();
    int e, i, mb, nb;
    if (per_e >= 8) {
      const int xcd = (int)(b & 7), slots = (per_e + 7) / 8;
      e = (int)((b >> 3) / slots);
      i = (int)(((long long)xcd * per_e) >> 3) + (int)((b >> 3) % slots);
      if (i >= (int)(((long long)(xcd + 1) * per_e) >> 3)) return;
    } else {
      e = (int)(b / per_e);
      i = (int)(b % per_e);
    }
    // (with a split, e names a part of an expert's rows; each part's sums are an output of their own)
    if (e >= p.E * p.split) return;
    band_place(i, nbm, nbn, mb, nb);
    int r0 = group_end(p.offsets, e / p.split, p.R), rows = max(group_end(p.offsets, e / p.split + 1, p.R) - r0, 0);
    if (p.split > 1) {
      const int part = ((rows + p.split - 1) / p.split + 31) & ~31, from = min((e % p.split) * part, rows);
      rows = min(part, rows - from);
      r0 += from;
    }
    const RowTile t{e, r0, rows, 0};
    ragged_tile<T, MODE, EPI, S0, kLate>(p, t, nb, mb * BM, smem, sRow, sScaleA, sScaleW);
  } else {
    RowTile t;
    int nb;
    if (!find_row_tile<BM, S1::BM>(p.offsets, p.E, p.R, nbn, t, nb)) return;
    if (S1::BM == 0 || t.cls == 0) {
      ragged_tile<T, MODE, EPI, S0, kLate>(p, t, nb, 0, smem, sRow, sScaleA, sScaleW);
    } else if constexpr (S1::BM > 0) {
      ragged_tile<T, MODE, EPI, S1, kLate>(p, t, nb, 0, smem, sRow, sScaleA, sScaleW);
    }
  }
}

// Whether tiles of bm rows by bc of nd columns give every CU a workgroup (estimated: the host does not know the
// groups' sizes).
static inline bool fills(const RaggedArgs& a, int bm, int nd, int bc) {
  const long long groups = a.E < a.R ? a.E : a.R, tiles = a.R / bm > groups ? a.R / bm : groups;
  return tiles * ((nd + bc - 1) / bc) >= 192;
}

// Contraction bytes from which a last round cut in halves pays for its empty workgroups (2 us).
constexpr int kHalvesBytes = 4096;

// Launch of one configuration.
template <class T, int MODE, int EPI, class S0, class S1 = NoTile>
static hipError_t launch_ragged_cfg(const RaggedArgs& a, hipStream_t s) {
  constexpr int BM = S0::BM, BN = S0::BN;
  const int nd = MODE == kFwd ? (EPI == MOE_EPI_SILU_MUL ? a.N / 2 : a.N) : a.K;
  const int bc = EPI == MOE_EPI_SILU_MUL ? BN / 2 : BN;
  const long long nbn = (nd + bc - 1) / bc;
  dim3 grid;
  if (MODE == kDw) {
    const long long per_e = (long long)((a.N + BM - 1) / BM) * nbn;
    grid = grid2d((per_e >= 8 ? (per_e + 7) / 8 * 8 : per_e) * a.E * a.split);
  } else {
    // most row tiles that any groups of R rows give, and up to one more a list and XCD by the shares' rounding
    const long long m = a.offsets ? (a.E < a.R ? a.E : a.R) : 1;
    const long long tiles = a.R / BM + m;
    // and, where a tile's time is worth it, as many as a last round cut in halves takes
    const bool halves = S1::BM > 0 && BM >= kHalvedHeight && tiles * nbn <= 8 * 8 * kXcdCus && (MODE == kFwd ? a.K : a.N) * T::kBytes >= kHalvesBytes;
    grid = grid2d(8 * ((tiles * nbn + 7) / 8 + (halves ? 3 + kXcdCus : (S1::BM > 0 ? 3 : 0))));
  }
  ragged_gemm_kernel<T, MODE, EPI, S0, S1><<<grid, S0::WM * S0::WN * 64, 0, s>>>(a);
  return hipGetLastError();
}

// Tile choice of the forward product, by the mean rows of a group (groups without rows count, as the host knows
// no better).  Measured with weights from HBM, TB/s of weights or PFLOP/s, 64 experts of 1024 x 2048 unless said:
//   mean   1: 16 x 64 tiles with 2 stages (8 workgroups a CU) against 16 x 128 with 4: int8, 53 of 128 experts of
//             1536 x 2048, 5.2 against 4.6 TB/s; fp16 5.1 against 4.9;
//             the weights loaded past the L2 where their rows are whole 128-byte lines (K 2048: int8 33 -> 28 us, fp16
//             63 -> 57 us; K 2064, whose lines two steps share: int8 40 -> 57 us, fp16 91 -> 122 us);
//   mean  25: 32 x 128 against 64 x 128: int8 4.6 against 4.3, fp16 5.5 against 5.5 (256 experts);
//   mean  50: 64 x 128 against 32 x 128: int8 4.4 against 3.5, fp16 3.8 against 3.3;
//   mean 100: 64 x 128 against 256 x 256: fp16 0.29 against 0.29, int8 0.60 against 0.59;
//   mean 200: 256 x 256 against 64 x 128: fp16 0.53 against 0.47, int8 0.88 against 0.87;
//   mean 400: fp16 0.79 against 0.60, int8 1.33 against 1.10.
// A tile that would leave CUs idle gives way to a smaller one: one group of 77 rows, 1536 columns: 6.4 us with 16-row
// tiles, 12.3 us with 64.  Groups of more than 16 rows on 16-row tiles are several tiles high and few: their weights stay
// in the L2 for the group's next tile, and four stages hide what two do with eight workgroups a CU.  Two stages past the
// L2, two stages, four stages, us: int8 200 x 1024 x 2048 13.0, 8.9, 6.0, 400 x 1536 x 2048 14.2, 9.5, 8.3, 8 groups of
// 50 rows, 1024 x 2048, 13.2, 13.6, 9.2; bf16 4 groups of 50, 1024 x 2048, 22.5, 22.9, 11.0, 8 of 25, 2048 x 512, 8.4, 8.7, 6.9.
template <class T, int EPI>
static hipError_t launch_ragged_fwd(const RaggedArgs& a, hipStream_t s) {
  const long long mean = ((long long)a.R + a.E - 1) / a.E;
  const int cols = EPI == MOE_EPI_SILU_MUL ? 2 : 1;  // weight rows per output column
  if (mean > 128 && fills(a, 256, a.N, 256))
    return launch_ragged_cfg<T, kFwd, EPI, TileShape<256, 256, 2, 4, 128, 2, 3>, TileShape<128, 256, 2, 4, 128, 3>>(a, s);
  if (mean > 32 && fills(a, 64, a.N / cols, 128 / cols))
    return launch_ragged_cfg<T, kFwd, EPI, TileShape<64, 128, 1, 4, 128, 2>>(a, s);
  if (mean > 16 && fills(a, 32, a.N / cols, 128 / cols))
    return launch_ragged_cfg<T, kFwd, EPI, TileShape<32, 128, 1, 4, 128, 2>>(a, s);
  if (mean <= 16 && fills(a, 16, a.N / cols, 64 / cols)) {
    if ((long long)a.K * T::kBytes % 128 == 0) return launch_ragged_cfg<T, kFwd, EPI, TileShape<16, 64, 1, 2, 128, 2, 2, true>>(a, s);
    return launch_ragged_cfg<T, kFwd, EPI, TileShape<16, 64, 1, 2, 128, 2>>(a, s);
  }
  return launch_ragged_cfg<T, kFwd, EPI, TileShape<16, 64, 1, 2, 128, 4>>(a, s);
}

}  // namespace moe
