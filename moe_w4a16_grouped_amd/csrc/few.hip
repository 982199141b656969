// The whole expert layer for at most 16 tokens in two launches: routing, gate_up with SiLU*mul in the first, down and the
// weighted sum in the second, on bf16 weights, or on int8 weights with one scale a channel and activations that stay in 16
// bits.  The ATOM page ("AMD ATOM推理引擎：如何用分页KV缓存和分段编译实现大模型推理性能翻倍"), section "8.1 MoE
// 路径：路由、专家并行与 MORI 通信", gives the layer's steps.
//
// So few tokens are bound by the chosen experts' weights, each read once, and by what stands before and behind that
// stream.  Hence: no step between the two products has a launch of its own; the weights go straight from memory to the
// registers in which the matrix instruction takes them, two chunks of loads ahead of their use, across the borders of the
// pieces that a workgroup is given; every workgroup routes by itself, so that nothing is handed between workgroups within
// a launch.
//
// The matrix instruction's 16 rows are rows of weights, its 16 columns tokens:
//   gate_up: 8 gate rows and the up rows of the same 8 columns of h, against all tokens; the waves of a workgroup take a
//            share of the contraction each and meet in LDS.
//   down:    8 rows (columns of y), each as two halves of the contraction, against at most 8 tokens of the expert, as
//            two halves too; the halves that belong together are added at the end.  So 8 columns of y make a workgroup
//            (256 of them at H 2048) and still whole instructions.  A workgroup sees every chosen expert, so the weighted
//            sum over a token's experts is its own, in the order of the slots.
// h stays in two bf16 parts (value, and what its rounding left), for about 16 significant bits: the traffic of h is small
// beside the weights', and y is then rounded once.  Sums are fp32.
#include <algorithm>

#include "../../include/moe_w4a16.h"
#include "launch.h"
#include "moe_common.h"
#include "topk.h"

namespace moe {

constexpr int kFewTokens = 16, kFewSlots = 256;  // T and T * k at most
constexpr int kFewWaves = 8;

// Eight int8 codes (two dwords) as bf16, exactly.
__device__ __forceinline__ bf16x8 i8x8_to_bf16(uint32_t a, uint32_t b) {
  bf16x8 r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    r[j] = (__bf16)(float)(int8_t)(a >> (8 * j));
    r[4 + j] = (__bf16)(float)(int8_t)(b >> (8 * j));
  }
  return r;
}

// A lane's 16 bytes of a weight row: PARTS operands of the matrix instruction, 8 elements each; STEP elements of the
// contraction in all four quarters of the wave.
struct FewW16 {
  static constexpr int PARTS = 1, STEP = 32, BYTES = 2;
  static constexpr bool SCALED = false;
  __device__ static __forceinline__ bf16x8 part(const u32x4& w, int) { return __builtin_bit_cast(bf16x8, w); }
};
struct FewW8 {
  static constexpr int PARTS = 2, STEP = 64, BYTES = 1;
  static constexpr bool SCALED = true;
  __device__ static __forceinline__ bf16x8 part(const u32x4& w, int i) { return i8x8_to_bf16(w[2 * i], w[2 * i + 1]); }
};

// An expert and at most 8 of its rows (flat slots t * k + s), as the second launch takes them.
struct FewEntry {
  int32_t expert, rows;
  int16_t row[8];  // past `rows` the last one again
  int32_t pad[2];
};
static_assert(sizeof(FewEntry) == 32, "two 16-byte loads");

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true));
  auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(a[0], a[1]);
  auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(b[0], b[1]);
}

// The k largest logits of a token by one wave, one after the other (equal ones by lower id): lane s gets slot s's id and
// weight.  u: the lane's keys, 0 where there is no expert (and, from here on, where it has been taken).
template <int NT, int NJ, int MOST>
__device__ __forceinline__ void few_route(uint32_t (&u)[MOST][NJ], int k, int (&id)[MOST], float (&weight)[MOST]) {
  const int lane = threadIdx.x & 63;
  float logit[NT];
#pragma unroll
  for (int a = 0; a < NT; ++a) id[a] = 0, logit[a] = 0.f;
  for (int s = 0; s < k; ++s) {
#pragma unroll
    for (int a = 0; a < NT; ++a) {
      uint32_t m = u[a][0];
#pragma unroll
      for (int j = 1; j < NJ; ++j) m = max(m, u[a][j]);
      m = __builtin_amdgcn_readfirstlane(wave_max_u32(m));
      int best = 0;
#pragma unroll
      for (int j = NJ - 1; j >= 0; --j) {
        const uint64_t b = __ballot(u[a][j] == m);
        if (b) best = 64 * j + (int)__builtin_ctzll(b);
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        if (lane + 64 * j == best) u[a][j] = 0u;
      if (lane == s) id[a] = best, logit[a] = from_ordered_bits(m);
    }
  }
#pragma unroll
  for (int a = 0; a < NT; ++a) {
    const float top = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(logit[a])));
    const float p = expf(logit[a] - top);
    float sum = 0.f;
    for (int s = 0; s < k; ++s) sum += __int_as_float(__builtin_amdgcn_readlane(__float_as_int(p), s));
    weight[a] = p / sum;
  }
}

// LDS of the first launch; the tokens stand behind it, 16 bytes apart in the banks.
struct FewLds {
  f32x4 part[2][kFewWaves][64];
  u32x4 zero;
  uint32_t mask[MOE_MAX_EXPERTS / 32];
  int32_t ids[kFewSlots];
  int32_t list[kFewSlots];                    // the chosen experts, ascending
  int16_t slot[kFewSlots][kFewTokens];        // a chosen expert's slot of each token, or -1
  int32_t more;
};

template <class W, int NJ>
__global__ __launch_bounds__(64 * kFewWaves) void few_gate_up_kernel(FewArgs p) {
  extern __shared__ u32x4 few_lds[];
  FewLds& s = *reinterpret_cast<FewLds*>(few_lds);
  char* xs = reinterpret_cast<char*>(few_lds) + (sizeof(FewLds) + 15) / 16 * 16;
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int T = p.T, H = p.H, I = p.I, E = p.E, k = p.k, R = T * k;
  const bool writer = blockIdx.x == gridDim.x - 1;
  const int xstride = 2 * H + 16;

  // the logits of this wave's tokens, then the tokens
  constexpr int NT = kFewTokens / kFewWaves;
  uint32_t u[NT][NJ];
#pragma unroll
  for (int a = 0; a < NT; ++a) {
    const int t = wave + a * kFewWaves;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int e = lane + 64 * j;
      u[a][j] = t < T && e < E ? max(ordered_bits(p.logits[(size_t)t * E + e]), 1u) : 0u;
    }
  }
  constexpr int kAhead = 4;
  const int xn = H / 8, xtotal = T * xn;
  u32x4 xr[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int c = tid + i * 64 * kFewWaves;
    if (c < xtotal) xr[i] = reinterpret_cast<const u32x4*>(p.x)[c];
  }
  if (tid < MOE_MAX_EXPERTS / 32) s.mask[tid] = 0u;
  if (tid == 0) s.zero = u32x4{0u, 0u, 0u, 0u}, s.more = 0;
  for (int i = tid; i < kFewSlots * kFewTokens / 8; i += 64 * kFewWaves)
    reinterpret_cast<u32x4*>(s.slot)[i] = u32x4{~0u, ~0u, ~0u, ~0u};
  if (wave < T) {
    int id[NT] = {};
    float weight[NT] = {};
    if (T <= kFewWaves) few_route<1>(u, k, id, weight);
    else few_route<NT>(u, k, id, weight);
#pragma unroll
    for (int a = 0; a < NT; ++a) {
      const int t = wave + a * kFewWaves;
      if (t < T && lane < k) {
        s.ids[t * k + lane] = id[a];
        if (writer) {
          p.ids[t * k + lane] = id[a];
          p.weight[t * k + lane] = weight[a];
        }
      }
    }
  }
  auto put = [&](int c, const u32x4& v) {
    const int t = c / xn;
    *reinterpret_cast<u32x4*>(xs + t * xstride + (c - t * xn) * 16) = v;
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int c = tid + i * 64 * kFewWaves;
    if (c < xtotal) put(c, xr[i]);
  }
  for (int c = tid + kAhead * 64 * kFewWaves; c < xtotal; c += 64 * kFewWaves) put(c, reinterpret_cast<const u32x4*>(p.x)[c]);
  __syncthreads();
  if (tid < R) atomicOr(&s.mask[s.ids[tid] >> 5], 1u << (s.ids[tid] & 31));
  __syncthreads();
  int n = 0;  // chosen experts
  {
    const int e = tid < R ? s.ids[tid] : 0;
    int rank = 0;
    for (int w = 0; w < (E + 31) / 32; ++w) {
      const uint32_t m = s.mask[w];
      n += __popc(m);
      rank += __popc(w < (e >> 5) ? m : (w == (e >> 5) ? m & ((1u << (e & 31)) - 1u) : 0u));
    }
    if (tid < R) {
      s.list[rank] = e;
      s.slot[rank][tid / k] = (int16_t)tid;
    }
  }
  n = __builtin_amdgcn_readfirstlane(n);
  __syncthreads();

  if (writer) {  // the entries: an expert's first 8 rows at its rank, a second 8 behind the experts
    FewEntry* table = reinterpret_cast<FewEntry*>(p.table) + 1;
    if (tid < n) {
      FewEntry* at = table + tid;
      int have = 0;
      for (int t = 0; t < T; ++t) {
        const int f = s.slot[tid][t];
        if (f < 0) continue;
        if (have == 8) {
          at->expert = s.list[tid];
          at->rows = 8;
          at = table + n + atomicAdd(&s.more, 1);
          have = 0;
        }
        for (int j = have; j < 8; ++j) at->row[j] = (int16_t)f;
        ++have;
      }
      at->expert = s.list[tid];
      at->rows = have;
    }
    __syncthreads();
    if (tid == 0) p.table[0] = n + s.more;
  }

  // this wave's share of the contraction, in chunks of C steps
  constexpr int C = 4, RING = 2, LANE = W::STEP / 4;
  const int steps = (H + W::STEP - 1) / W::STEP, share = (steps + kFewWaves - 1) / kFewWaves;
  const int chunks = (share + C - 1) / C, blocks = I / 8, tasks = n * blocks;
  const int k0 = wave * share * W::STEP + q * LANE;
  const int wrow = l16 < 8 ? l16 : I + l16 - 8;
  const char* xrow = xs + min(l16, T - 1) * xstride;
  struct Cursor {
    int task, chunk;
  };
  auto advance = [&](Cursor& c) {
    if (++c.chunk == chunks) c.chunk = 0, c.task += gridDim.x;
  };
  u32x4 ring[RING][C];
  float sg[RING], su[RING];  // scales of the column that this thread finishes
  auto valid = [&](int chunk, int i) { return chunk * C + i < share && k0 + (chunk * C + i) * W::STEP < H; };
  auto load = [&](const Cursor& c, int b) {
    if (c.task >= tasks) return;
    const int rank = c.task / blocks, block = c.task - rank * blocks;
    const int e = __builtin_amdgcn_readfirstlane(s.list[rank]);
    const char* row = static_cast<const char*>(p.w13) + ((size_t)e * (2 * I) + block * 8 + wrow) * (size_t)H * W::BYTES;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int at = min(k0 + (c.chunk * C + i) * W::STEP, H - LANE);
      ring[b][i] = *reinterpret_cast<const u32x4*>(row + (size_t)at * W::BYTES);
    }
    if (W::SCALED && tid < 8 * kFewTokens) {
      const float* sc = p.w13_s + (size_t)e * (2 * I) + block * 8 + (tid & 7);
      sg[b] = sc[0];
      su[b] = sc[I];
    }
  };
  Cursor use = {(int)blockIdx.x, 0}, ahead = use;
#pragma unroll
  for (int b = 0; b < RING; ++b) {
    load(ahead, b);
    advance(ahead);
  }
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  int turn = 0;
  while (use.task < tasks) {
#pragma unroll
    for (int b = 0; b < RING; ++b) {
      if (use.task < tasks) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
          const bool in = valid(use.chunk, i);
          u32x4 w = ring[b][i];
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = in ? w[j] : 0u;
          const char* xk = in ? xrow + (k0 + (use.chunk * C + i) * W::STEP) * 2 : reinterpret_cast<const char*>(&s.zero);
#pragma unroll
          for (int h = 0; h < W::PARTS; ++h) {
            const bf16x8 xv = *reinterpret_cast<const bf16x8*>(in ? xk + 16 * h : xk);
            acc = mfma16x16x32(W::part(w, h), xv, acc);
          }
        }
        const float scale_g = sg[b], scale_u = su[b];
        load(ahead, b);
        advance(ahead);
        if (use.chunk == chunks - 1) {
          s.part[turn][wave][lane] = acc;
          acc = f32x4{0.f, 0.f, 0.f, 0.f};
          __syncthreads();  // one a task: this half of part is written again only past the next task's barrier
          if (tid < 8 * kFewTokens) {
            const int c = tid & 7, t = tid >> 3;
            const int rank = use.task / blocks, block = use.task - rank * blocks;
            const int f = s.slot[rank][t];
            float g = 0.f, up = 0.f;
            const int from = (c >> 2) * 16 + t;
#pragma unroll
            for (int w = 0; w < kFewWaves; ++w) {
              g += reinterpret_cast<const float*>(&s.part[turn][w][from])[c & 3];
              up += reinterpret_cast<const float*>(&s.part[turn][w][from + 32])[c & 3];
            }
            if (W::SCALED) g *= scale_g, up *= scale_u;
            if (f >= 0) {
              const float h = silu_f32(g) * up;
              const uint32_t hi = f32_to_bf16_bits(h);
              const float left = h - bf16_bits_to_f32(hi);
              uint16_t* dst = p.h + ((size_t)f * blocks + block) * 16 + c;
              dst[0] = (uint16_t)hi;
              dst[8] = fabsf(left) < __builtin_inff() ? f32_to_bf16_bits(left) : (uint16_t)0;
            }
          }
          turn ^= 1;
        }
        advance(use);
      }
    }
  }
}

template <class W>
__global__ __launch_bounds__(64 * kFewWaves) void few_down_kernel(FewArgs p) {
  __shared__ FewEntry table[kFewSlots];
  __shared__ __attribute__((aligned(16))) float out[kFewSlots][8];
  __shared__ float weight[kFewSlots];
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int T = p.T, H = p.H, I = p.I, k = p.k, R = T * k;
  const int col0 = blockIdx.x * 8;
  const int n = p.table[0];
  if (tid < 2 * R) reinterpret_cast<u32x4*>(table)[tid] = reinterpret_cast<const u32x4*>(p.table)[2 + tid];
  if (tid < R) weight[tid] = p.weight[tid];
  __syncthreads();

  // units: an entry and a piece of the contraction; a piece is two halves of `share` steps
  constexpr int C = W::PARTS == 1 ? 4 : 2, RING = 2, LANE = W::STEP / 4;
  const int pieces = p.pieces, units = n * pieces;
  const int steps = (I + W::STEP - 1) / W::STEP, share = (steps + 2 * pieces - 1) / (2 * pieces), chunks = (share + C - 1) / C;
  const int half = l16 >> 3, m = l16 & 7;
  struct Cursor {
    int unit, chunk;
  };
  auto advance = [&](Cursor& c) {
    if (++c.chunk == chunks) c.chunk = 0, c.unit += kFewWaves;
  };
  u32x4 ring[RING][C], hv[RING][C][2 * W::PARTS];
  float sc[RING][4];
  auto start = [&](const Cursor& c, int piece) { return ((piece * 2 + half) * share + c.chunk * C) * W::STEP + q * LANE; };
  auto load = [&](const Cursor& c, int b) {
    if (c.unit >= units) return;
    const int entry = c.unit / pieces, piece = c.unit - entry * pieces;
    const int e = __builtin_amdgcn_readfirstlane(table[entry].expert);
    const char* row = static_cast<const char*>(p.w2) + ((size_t)e * H + col0 + m) * (size_t)I * W::BYTES;
    const uint16_t* hrow = p.h + (size_t)table[entry].row[m] * I * 2;
    const int k0 = start(c, piece);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int at = min(k0 + i * W::STEP, I - LANE);
      ring[b][i] = *reinterpret_cast<const u32x4*>(row + (size_t)at * W::BYTES);
#pragma unroll
      for (int h = 0; h < 2 * W::PARTS; ++h) hv[b][i][h] = *reinterpret_cast<const u32x4*>(hrow + at * 2 + 8 * h);
    }
    if (W::SCALED) {
#pragma unroll
      for (int r = 0; r < 4; ++r) sc[b][r] = p.w2_s[(size_t)e * H + col0 + 4 * (q & 1) + r];
    }
  };
  Cursor use = {wave, 0}, ahead = use;
#pragma unroll
  for (int b = 0; b < RING; ++b) {
    load(ahead, b);
    advance(ahead);
  }
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  while (use.unit < units) {
#pragma unroll
    for (int b = 0; b < RING; ++b) {
      if (use.unit < units) {
        const int entry = use.unit / pieces, piece = use.unit - entry * pieces;
        const int k0 = start(use, piece);
#pragma unroll
        for (int i = 0; i < C; ++i) {
          const bool in = use.chunk * C + i < share && k0 + i * W::STEP < I;
          u32x4 w = ring[b][i];
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = in ? w[j] : 0u;
#pragma unroll
          for (int h = 0; h < W::PARTS; ++h) {
            const bf16x8 a = W::part(w, h);
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              u32x4 x = hv[b][i][2 * h + v];
#pragma unroll
              for (int j = 0; j < 4; ++j) x[j] = in ? x[j] : 0u;
              acc = mfma16x16x32(a, __builtin_bit_cast(bf16x8, x), acc);
            }
          }
        }
        float scale[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) scale[r] = W::SCALED ? sc[b][r] : 1.f;
        load(ahead, b);
        advance(ahead);
        if (use.chunk == chunks - 1) {
          f32x4 o;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            o[r] = acc[r] + __shfl(acc[r], lane + 40);  // rows 8 + of columns 8 +: the other half
            if (W::SCALED) o[r] *= scale[r];
          }
          if (q < 2 && l16 < 8 && l16 < table[entry].rows)
            *reinterpret_cast<f32x4*>(&out[piece * R + table[entry].row[l16]][4 * q]) = o;
          acc = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        advance(use);
      }
    }
  }
  __syncthreads();
  if (tid < 8 * T) {
    const int t = tid >> 3, c = tid & 7;
    float y = 0.f;
    for (int s = 0; s < k; ++s) {
      const int f = t * k + s;
      float o = out[f][c];
      for (int i = 1; i < pieces; ++i) o += out[i * R + f][c];
      y = fmaf(weight[f], o, y);
    }
    p.y[(size_t)t * H + col0 + c] = f32_to_bf16_bits(y);
  }
}

// Pieces of the contraction that a second launch's units are cut into, so that the eight waves of a workgroup have one each
// even where a single token chose fewer experts.  pieces * T * k <= kFewSlots.
static int few_pieces(int k) { return k >= kFewWaves ? 1 : (kFewWaves + k - 1) / k; }

template <class W, int NJ>
static hipError_t launch_few_of(const FewArgs& p, hipStream_t s) {
  const int lds = (int)((sizeof(FewLds) + 15) / 16 * 16) + p.T * (2 * p.H + 16);
  const int most = std::max(1, std::min(3, (160 << 10) / lds));  // workgroups a CU
  const int tasks = std::min(p.E, p.T * p.k) * (p.I / 8);
  const int grid = std::min(tasks, 256 * most);
  if (lds > (64 << 10)) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(few_gate_up_kernel<W, NJ>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  few_gate_up_kernel<W, NJ><<<grid, 64 * kFewWaves, lds, s>>>(p);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  few_down_kernel<W><<<p.H / 8, 64 * kFewWaves, 0, s>>>(p);
  return hipGetLastError();
}

template <class W>
static hipError_t launch_few_w(const FewArgs& p, hipStream_t s) {
  if (p.E <= 128) return launch_few_of<W, 2>(p, s);
  if (p.E <= 256) return launch_few_of<W, 4>(p, s);
  if (p.E <= 512) return launch_few_of<W, 8>(p, s);
  return launch_few_of<W, 16>(p, s);
}

hipError_t launch_ffn_few(FewArgs p, bool i8, hipStream_t stream) {
  p.pieces = few_pieces(p.k);
  return i8 ? launch_few_w<FewW8>(p, stream) : launch_few_w<FewW16>(p, stream);
}

}  // namespace moe
