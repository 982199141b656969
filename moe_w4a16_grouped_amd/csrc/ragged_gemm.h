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
// global->LDS 16-byte loads through a ring of NS stages, one barrier per step.  An operand whose
// contraction axis is contiguous in memory ("rows") is kept as [row][RB bytes]; one whose other axis is
// contiguous (W in DX, both in DW) as [contraction row][tile columns], and its fragments are read with
// the transposing LDS load (ds_read_b64_tr_b16: a 16-lane group reads a 4 x 16 block and lane j gets
// column j).  16-byte chunks are XOR-swizzled so that neither kind of read has bank conflicts.
//
// Fragments of v_mfma_f32_16x16x32 (16-bit) and v_mfma_i32_16x16x64_i8: lane l supplies 16 bytes, row
// l % 16, contraction bytes [16 (l / 16), +16) of a 64-byte group.  The weight fragment is the first
// operand, so a lane's four results are four neighbouring columns of one output row and are stored
// together.
#pragma once
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

// 16-byte chunk permutation of an operand kept as rows of RB bytes: the 16 rows of a fragment read at one
// chunk column fall in 16 different chunks of a 256-byte bank line.
template <int RB>
__device__ __forceinline__ int row_swizzle(int row) {
  return RB == 64 ? (row >> 2) & 3 : (row >> 1) & 7;
}
// 32-byte window permutation of an operand kept as contraction rows: a transposing read covers 4 rows of
// each 16-lane group, groups 8 rows apart; the eight rows of half a wave fall in eight different windows.
__device__ __forceinline__ int col_swizzle(int crow) { return (crow & 3) | ((crow >> 1) & 4); }

// A row tile of the ragged groups: expert, first row, rows (at most BM).
struct RowTile {
  int e, row0, rows;
};

__device__ __forceinline__ int group_end(const int32_t* off, int i, int R) { return min(max(off[i], 0), R); }

// Finds the workgroup's row tile and column block from the offsets: every wave counts the tiles of
// E / 64 experts a lane, scans the counts over its lanes and walks the experts of the lane that holds the
// wanted tile.  Offsets are clamped to [0, R], so no list of offsets leads out of the rows.
template <int BM>
__device__ __forceinline__ bool find_row_tile(const int32_t* __restrict__ off, int E, int R, int nbn, RowTile& t, int& nb) {
  int tile;
  if (!off) {  // one group of all rows
    const int n = (R + BM - 1) / BM;
    if (!mm_work(linear_block(), nbn, n, tile, nb)) return false;
    t = RowTile{0, tile * BM, min(BM, R - tile * BM)};
    return true;
  }
  const int lane = threadIdx.x & 63;
  const int per = (E + 63) / 64;
  const int e0 = min(lane * per, E), e1 = min(e0 + per, E);
  int at = group_end(off, e0, R), n = 0;
  for (int e = e0; e < e1; ++e) {
    const int end = group_end(off, e + 1, R);
    n += (max(end - at, 0) + BM - 1) / BM;
    at = end;
  }
  int incl = n;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(incl, d);
    if (lane >= d) incl += v;
  }
  const int total = __builtin_amdgcn_readlane(incl, 63);
  if (!mm_work(linear_block(), nbn, total, tile, nb)) return false;
  const uint64_t past = __ballot(incl > tile);
  const int src = __builtin_ctzll(past);  // tile < total: some lane's sum is past it
  int left = tile - (__builtin_amdgcn_readlane(incl, src) - __builtin_amdgcn_readlane(n, src));
  int e = src * per;
  at = group_end(off, e, R);
  for (;; ++e) {
    const int end = group_end(off, e + 1, R);
    const int nt = (max(end - at, 0) + BM - 1) / BM;
    if (left < nt || e == E - 1) {
      const int r0 = at + left * BM;
      t = RowTile{e, r0, min(BM, end - r0)};
      return true;
    }
    left -= nt;
    at = end;
  }
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
template <int BM>
constexpr int dw_ids() { return BM >= 256 ? 4096 : 1024; }

template <class T, int MODE, int EPI, int BM, int BN, int WM, int WN, int RB, int NS>
__global__ __launch_bounds__(WM * WN * 64) void ragged_gemm_kernel(RaggedArgs p) {
  constexpr int NW = WM * WN;
  constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
  constexpr bool A_T = MODE == kDw, B_T = MODE != kFwd;  // operand kept as contraction rows
  constexpr int CR = RB / T::kBytes;                     // contraction elements per step
  constexpr int SA = BM * RB, SB = BN * RB, STAGE = SA + SB;
  constexpr int LA = SA / 1024, LT = STAGE / 1024;       // wave-wide loads of a step: the A tile's, all
  constexpr int LW = (LT + NW - 1) / NW, LMIN = LT / NW;
  static_assert(EPI != MOE_EPI_SILU_MUL || (MODE == kFwd && NI % 2 == 0), "SiLU*mul pairs gate and up blocks");
  static_assert(T::kBytes == 2 || MODE == kFwd, "transposing reads are of 16-bit elements");
  static_assert(SA % 1024 == 0 && SB % 1024 == 0 && LMIN >= 1 && (NS - 2) * LMIN < 64, "loads");
  __shared__ __attribute__((aligned(16))) uint8_t smem[NS * STAGE];
  __shared__ int32_t sRow[MODE == kDw ? dw_ids<BM>() : BM];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int l16 = lane & 15, q = lane >> 4;
  const int N = p.N, K = p.K;
  // output columns and contraction length
  const int ND = MODE == kFwd ? (EPI == MOE_EPI_SILU_MUL ? N / 2 : N) : K;
  constexpr int BC = EPI == MOE_EPI_SILU_MUL ? BN / 2 : BN;  // output columns of a tile
  const int nbn = (ND + BC - 1) / BC;

  RowTile t;
  int nb, m0 = 0;  // column block; DW: first weight row of the tile
  if constexpr (MODE == kDw) {
    // every expert's tiles are shared evenly by the XCDs (an expert with many rows keeps all of them
    // busy); fewer than 8 tiles an expert are dealt one by one
    const int nbm = (N + BM - 1) / BM, per_e = nbm * nbn;
    const long long b = linear_block();
    int e, i;
    if (per_e >= 8) {
      const int xcd = (int)(b & 7), slots = (per_e + 7) / 8;
      e = (int)((b >> 3) / slots);
      i = (int)(((long long)xcd * per_e) >> 3) + (int)((b >> 3) % slots);
      if (i >= (int)(((long long)(xcd + 1) * per_e) >> 3)) return;
    } else {
      e = (int)(b / per_e);
      i = (int)(b % per_e);
    }
    if (e >= p.E) return;
    m0 = (i / nbn) * BM;
    nb = i % nbn;
    const int r0 = group_end(p.offsets, e, p.R);
    t = RowTile{e, r0, max(group_end(p.offsets, e + 1, p.R) - r0, 0)};
  } else {
    if (!find_row_tile<BM>(p.offsets, p.E, p.R, nbn, t, nb)) return;
    for (int i = tid; i < BM; i += NW * 64) {  // padding rows repeat the tile's first row
      const int r = t.row0 + (i < t.rows ? i : 0);
      sRow[i] = MODE == kFwd && p.a_row_of ? p.a_row_of[r] / p.a_row_div : r;
    }
    __syncthreads();
  }
  const size_t w_e = (size_t)t.e * N * K;  // first element of the expert's weights
  const uint8_t* A = static_cast<const uint8_t*>(p.A);
  const uint8_t* W = static_cast<const uint8_t*>(p.W);
  const uint8_t* zero = reinterpret_cast<const uint8_t*>(&kZeroChunk);

  // Sources of this lane's loads (load j is the wave-wide load wave + NW * j of a step's LT).  Rows kind:
  // src is the chunk at contraction byte 0 and pos its byte in the step.  Contraction-rows kind: src is
  // the chunk of contraction row 0 (NULL when its columns lie past the edge) and pos its row in the step.
  const uint8_t* src[LW];
  int pos[LW];
#pragma unroll
  for (int j = 0; j < LW; ++j) {
    const int i = wave + NW * j;
    const bool is_a = i < LA;
    const int byte = (is_a ? i : i - LA) * 1024 + lane * 16;
    src[j] = nullptr;
    pos[j] = 0;
    if (is_a ? !A_T : !B_T) {
      const int row = byte / RB;
      pos[j] = 16 * (((byte % RB) >> 4) ^ row_swizzle<RB>(row));
      if (is_a) {
        const size_t width = (size_t)(MODE == kDx ? N : K) * T::kBytes;
        src[j] = A + (size_t)sRow[row] * width + pos[j];
      } else if (i < LT) {
        int n;
        if (EPI == MOE_EPI_SILU_MUL) {  // a wave's columns: its gate rows, then their up rows
          constexpr int WC = BN / WN;
          const int in = row % WC, h = nb * BC + (row / WC) * (WC / 2) + in % (WC / 2);
          n = h < ND ? (in < WC / 2 ? h : ND + h) : 0;
        } else {
          n = nb * BN + row;
          if (n >= N) n = 0;
        }
        src[j] = W + (w_e + (size_t)n * K) * T::kBytes + pos[j];
      }
    } else {
      const int width = (is_a ? BM : BN) * 2;
      const int crow = byte / width;
      const int col = (is_a ? m0 : nb * BN) + 8 * (((byte % width) >> 4) ^ (2 * col_swizzle(crow)));
      const int cols = is_a ? N : K;
      pos[j] = crow;
      // DX: rows of W; DW: rows of dC (A operand) and of A (B operand), whose row is added at the load
      const uint8_t* base = MODE == kDx ? W + w_e * 2 : (is_a ? W : A);
      if (col < cols) src[j] = base + (size_t)col * 2;
    }
  }

  // contraction of this pass: rows of the expert (DW), else the whole axis
  const int KD = MODE == kFwd ? K : N;
  int kd = MODE == kDw ? 0 : KD;  // elements in the present pass (DW sets it per pass)
  int pass0 = 0;                  // DW: first row of the pass within the expert
  auto issue = [&](int s, int stage) {
    uint8_t* st = smem + stage * STAGE;
#pragma unroll
    for (int j = 0; j < LW; ++j) {
      const int i = wave + NW * j;
      if (LT % NW != 0 && i >= LT) break;
      const uint8_t* from;
      const bool is_a = i < LA;
      if (is_a ? !A_T : !B_T) {
        from = src[j] + (size_t)s * RB;
        if ((s + 1) * RB > KD * T::kBytes && s * RB + pos[j] >= KD * T::kBytes) from = zero;
      } else {
        const int c = s * CR + pos[j];
        from = zero;
        if (src[j] && c < kd) {
          if (MODE == kDx) from = src[j] + (size_t)c * K * 2;
          else if (is_a) from = src[j] + (size_t)(t.row0 + pass0 + c) * N * 2;
          else from = src[j] + (size_t)(p.a_row_of ? sRow[c] : t.row0 + pass0 + c) * K * 2;
        }
      }
      g2lds16(from, st + i * 1024);
    }
  };

  // this lane's fragment offsets in a stage
  auto frag_rows = [&](const uint8_t* tile, int row0, int kk) -> u32x4 {
    return *reinterpret_cast<const u32x4*>(tile + (row0 + l16) * RB + 16 * ((kk * 4 + q) ^ row_swizzle<RB>(l16)));
  };
  auto frag_cols = [&](const uint8_t* tile, int width, int col0, int kk) -> u32x4 {
    u32x2 half[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int crow = kk * 32 + 8 * q + 4 * h + (l16 >> 2);
      const int byte = crow * width + (((col0 >> 4) ^ col_swizzle(crow)) << 5) + 8 * (l16 & 3);
      half[h] = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) i16x4*)(tile + byte)));
    }
    return u32x4{half[0][0], half[0][1], half[1][0], half[1][1]};
  };

  typename T::Acc acc[MI][NI];
#pragma unroll
  for (int mi = 0; mi < MI; ++mi)
#pragma unroll
    for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = typename T::Acc{0, 0, 0, 0};

  auto compute = [&](int stage) {
    const uint8_t* ta = smem + stage * STAGE;
    const uint8_t* tb = ta + SA;
#pragma unroll
    for (int kk = 0; kk < RB / 64; ++kk) {
      u32x4 a[MI], b[NI];
#pragma unroll
      for (int ni = 0; ni < NI; ++ni) {
        const int c = wn * (BN / WN) + ni * 16;
        b[ni] = B_T ? frag_cols(tb, BN * 2, c, kk) : frag_rows(tb, c, kk);
      }
#pragma unroll
      for (int mi = 0; mi < MI; ++mi) {
        const int r = wm * (BM / WM) + mi * 16;
        a[mi] = A_T ? frag_cols(ta, BM * 2, r, kk) : frag_rows(ta, r, kk);
      }
#pragma unroll
      for (int mi = 0; mi < MI; ++mi)
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) acc[mi][ni] = T::mfma(b[ni], a[mi], acc[mi][ni]);
    }
  };

  // Step s lives in stage s % NS.  A stage is read after this wave's loads for it have landed (those of
  // the steps behind it may still be in flight) and after the barrier that publishes everyone's; the
  // same barrier says that the stage of step s - 1, which the next loads overwrite, is no longer read.
  auto run = [&](int steps) {
#pragma unroll
    for (int s = 0; s < NS - 1; ++s)
      if (s < steps) issue(s, s);
    for (int s = 0; s < steps; ++s) {
      const int behind = min(NS - 2, steps - 1 - s);
      if (behind == NS - 2) wait_vmcnt<(NS - 2) * LMIN>();
      else if (NS > 3 && behind == NS - 3) wait_vmcnt<(NS > 3 ? NS - 3 : 0) * LMIN>();
      else wait_vmcnt<0>();
      __syncthreads();
      if (s + NS - 1 < steps) issue(s + NS - 1, (s + NS - 1) % NS);
      compute(s % NS);
    }
  };
  if constexpr (MODE == kDw) {
    for (pass0 = 0; pass0 < t.rows; pass0 += dw_ids<BM>()) {
      kd = min(t.rows - pass0, dw_ids<BM>());
      if (p.a_row_of) {
        __syncthreads();  // the last pass's indexes and stages are no longer read
        for (int i = tid; i < kd; i += NW * 64) sRow[i] = p.a_row_of[t.row0 + pass0 + i] / p.a_row_div;
      }
      __syncthreads();
      run((kd + CR - 1) / CR);
    }
  } else {
    run((KD + CR - 1) / CR);
  }

  // Epilogue: lane (q, l16) holds columns 4q .. 4q+3 of each 16 x 16 block, of row l16.
  const bool whole = (ND & 3) == 0;  // rows are stored four columns at a time
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    const int row = wm * (BM / WM) + mi * 16 + l16;
    size_t at;
    if constexpr (MODE == kDw) {
      if (m0 + row >= N) continue;
      at = w_e + (size_t)(m0 + row) * K;
    } else {
      if (row >= t.rows) continue;
      at = (size_t)(t.row0 + row) * ND;
    }
    float sa = 1.f;
    if constexpr (T::kBytes == 1) sa = p.As[sRow[row]];
    constexpr int NO = EPI == MOE_EPI_SILU_MUL ? NI / 2 : NI;
#pragma unroll
    for (int ni = 0; ni < NO; ++ni) {
      const int col = nb * BC + wn * (BC / WN) + ni * 16 + 4 * q;
      if (col >= ND) continue;
      float v[4], u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = (float)acc[mi][ni][i];
        if constexpr (EPI == MOE_EPI_SILU_MUL) u[i] = (float)acc[mi][ni + NO][i];
        if constexpr (T::kBytes == 1) {  // the integer sums are exact; one scale a row and a channel
          const float* ws = p.Ws + (size_t)t.e * N + min(col + i, ND - 1);
          v[i] *= sa * ws[0];
          if constexpr (EPI == MOE_EPI_SILU_MUL) u[i] *= sa * ws[ND];
        }
        if constexpr (EPI == MOE_EPI_SILU_MUL) v[i] = silu_f32(v[i]) * u[i];
      }
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

// Launch of one configuration.
template <class T, int MODE, int EPI, int BM, int BN, int WM, int WN, int RB, int NS>
static hipError_t launch_ragged_cfg(const RaggedArgs& a, hipStream_t s) {
  const int nd = MODE == kFwd ? (EPI == MOE_EPI_SILU_MUL ? a.N / 2 : a.N) : a.K;
  const int bc = EPI == MOE_EPI_SILU_MUL ? BN / 2 : BN;
  const int nbn = (nd + bc - 1) / bc;
  dim3 grid;
  if (MODE == kDw) {
    const long long per_e = (long long)((a.N + BM - 1) / BM) * nbn;
    grid = grid2d(per_e >= 8 ? (per_e + 7) / 8 * 8 * a.E : per_e * a.E);
  } else {
    const int tiles = a.offsets ? a.R / BM + (a.E < a.R ? a.E : a.R) : (a.R + BM - 1) / BM;
    grid = mm_grid(nbn, tiles);
  }
  ragged_gemm_kernel<T, MODE, EPI, BM, BN, WM, WN, RB, NS><<<grid, WM * WN * 64, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace moe
