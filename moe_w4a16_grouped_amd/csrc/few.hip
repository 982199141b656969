// The whole expert layer for at most 16 tokens in two launches: routing, gate_up with SiLU*mul in the first, down and the
// weighted sum in the second, on bf16 weights, or on int8 weights with one scale a channel and activations that stay in 16
// bits.  The ATOM page ("AMD ATOM推理引擎：如何用分页KV缓存和分段编译实现大模型推理性能翻倍"), section "8.1 MoE
// 路径：路由、专家并行与 MORI 通信", gives the layer's steps.
//
// So few tokens are bound by the chosen experts' weights, each read once, and by what stands before and behind that
// stream.  Hence: no step between the two products has a launch of its own; the weights go straight from memory to the
// registers in which the matrix instruction takes them, two or three chunks of loads ahead of their use, across the borders of
// the pieces that a workgroup is given; every workgroup routes by itself, so that nothing is handed between workgroups
// within a launch.
//
// The matrix instruction's 16 rows are rows of weights, its 16 columns tokens:
//   gate_up: 8 gate rows and the up rows of the same 8 columns of h, against all tokens.  The waves of a workgroup take a
//            share of the contraction each and meet in LDS; where rows are short a wave takes such a task alone.
//   down:    8 rows (columns of y), each as two halves of the contraction, against at most 8 tokens of the expert, as
//            two halves too (or 4 rows as four quarters); what belongs together is added at the end.  So up to 4, 8 or 16
//            columns of y make a workgroup, as many as deal H evenly to the CUs.  A workgroup sees every chosen expert, so
//            the weighted sum over a token's experts is its own, in the order of the slots.  Only where H is small, and the
//            contraction long, do workgroups share columns: a third launch then adds their parts.
// h stays in two bf16 parts (value, and what its rounding left), for about 16 significant bits: what the matrix instruction takes
// beside bf16 weights, in the bytes of an fp32.  Of 16384 y of 8 tokens 40 come out as the second nearest bf16 (8 in an fp32 form), which
// adds 4e-7 of itself to y's distance from 64 bits, 1.687e-3; a third part would cost half as many matrix instructions, and half of h's
// LDS, again.  y is rounded once.  Sums are fp32.
//
// Measured, both launches and the weights' rate (a large copy reads and writes at 5.2 TB/s here, a sum reads at 4.0):
//   16 tokens, 8 experts of 4096 x 14336, bf16      474-493 us, 5.7 TB/s     (324 gate_up, 164 down)
//   8 tokens, 128 experts top-8, 2048 x 768, bf16    89 us, 5.5 TB/s         (58, 30)
//   16 tokens, 256 experts top-8, 2048 x 512, int8   72 us, 4.4 TB/s         (47, 23)
//   one token, 128 experts top-8, 2048 x 768         20 us bf16, 15 us int8  (12, 7.4 and 9.3, 6.6)
//   11 tokens, 60 experts top-6, 1040 x 336, int8    21 us                   (13, 8.7)
// The last two are latency: 3 us until a workgroup knows the experts (6 for 16 tokens), about 2 us a round trip to memory, and
// the border between the launches.
#include <algorithm>
#include <type_traits>

#include "launch.h"
#include "moe_common.h"
#include "moe_w4a16.h"
#include "topk.h"

namespace moe {

constexpr int kFewTokens = 16, kFewSlots = 256;  // T and T * k at most
constexpr int kFewWaves = 8;

// Eight int8 codes (two dwords) as bf16, exactly.
__device__ __forceinline__ bf16x8 i8x8_to_bf16(uint32_t a, uint32_t b) {
  bf16x8 r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    r[j] = (__bf16)(float)(int)__builtin_amdgcn_sbfe((int)a, 8 * j, 8);
    r[4 + j] = (__bf16)(float)(int)__builtin_amdgcn_sbfe((int)b, 8 * j, 8);
  }
  return r;
}

// A lane's 16 bytes of a weight row: PARTS operands of the matrix instruction, 8 elements each; LANE elements in all.
struct FewW16 {
  static constexpr int PARTS = 1, LANE = 8, BYTES = 2;
  static constexpr bool SCALED = false;
  __device__ static __forceinline__ bf16x8 part(const u32x4& w, int) { return __builtin_bit_cast(bf16x8, w); }
};
struct FewW8 {
  static constexpr int PARTS = 2, LANE = 16, BYTES = 1;
  static constexpr bool SCALED = true;
  __device__ static __forceinline__ bf16x8 part(const u32x4& w, int i) { return i8x8_to_bf16(w[2 * i], w[2 * i + 1]); }
};

// 16 bytes at an offset of a buffer; past its end (kFewPast in all of them) zeros, for which no bytes move.
constexpr uint32_t kFewPast = 0xFFFFFFF0u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t few_buffer(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00027000);
}
__device__ __forceinline__ u32x4 few_load(__amdgpu_buffer_rsrc_t r, uint32_t offset) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)offset, 0, 0));
}
__device__ __forceinline__ u32x4 few_keep(const u32x4& v, bool in) {
  return u32x4{in ? v[0] : 0u, in ? v[1] : 0u, in ? v[2] : 0u, in ? v[3] : 0u};
}

// An expert and at most 8 of its rows (flat slots t * k + s), as the second launch takes them.
struct FewEntry {
  int32_t expert, rows;
  int16_t row[8];
  int32_t pad[2];
};
static_assert(sizeof(FewEntry) == 32, "two 16-byte loads");

// The largest value of a wave, on the scalar side (row shifts, then the rows' last lanes broadcast: lane 63 has seen all).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_max_u32(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = dpp_max_u32<0x111, 0xF>(v);
  v = dpp_max_u32<0x112, 0xF>(v);
  v = dpp_max_u32<0x114, 0xF>(v);
  v = dpp_max_u32<0x118, 0xF>(v);
  v = dpp_max_u32<0x142, 0xA>(v);
  v = dpp_max_u32<0x143, 0xC>(v);
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// The k largest logits of NT tokens by one wave, one after the other (equal ones by lower id): lane s gets slot s's id and
// key.  u: the lane's keys, experts lane * NJ + j, 0 where there is none (and, from here on, where it has been taken).  The
// lowest lane that holds the largest key holds the lowest id of it, so one ballot finds the slot's expert.  Many waves of a
// compute unit do this at once, so instructions count as well as the chain: a radix select with compaction and ranking, as
// larger batches use it, is about twice as long.  chosen: lane w's bits of experts 32w .. 32w + 31, of all NT tokens.
template <int NT, int NJ, int MOST>
__device__ __forceinline__ void few_route(uint32_t (&u)[MOST][NJ], int k, int (&id)[MOST], uint32_t (&key)[MOST], uint32_t& chosen) {
  const int lane = threadIdx.x & 63;
  for (int s = 0; s < k; ++s) {
#pragma unroll
    for (int a = 0; a < NT; ++a) {
      uint32_t top = u[a][0];
#pragma unroll
      for (int j = 1; j < NJ; ++j) top = max(top, u[a][j]);
      const uint32_t m = wave_max_u32(top);
      const int owner = (int)__builtin_ctzll(__ballot(top == m));
      int at = NJ - 1;
#pragma unroll
      for (int j = NJ - 2; j >= 0; --j) at = u[a][j] == m ? j : at;
      const int best = __builtin_amdgcn_readlane(at, owner);
#pragma unroll
      for (int j = 0; j < NJ; ++j) u[a][j] = lane == owner && best == j ? 0u : u[a][j];
      const int e = owner * NJ + best;
      if (MOST > 1 || NT > 1) chosen |= lane == e >> 5 ? 1u << (e & 31) : 0u;
      id[a] = lane == s ? e : id[a];
      key[a] = lane == s ? m : key[a];
    }
  }
}

// Slot weights from the slots' logits (lane s: slot s), added in the order of the slots as moe_route_topk adds them.
__device__ __forceinline__ float few_weight(float logit, int k) {
  const float top = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(logit)));
  const float p = expf(logit - top);
  float sum = 0.f;
  for (int s = 0; s < k; ++s) sum += __int_as_float(__builtin_amdgcn_readlane(__float_as_int(p), s));
  return p / sum;
}

// h as two bf16: itself, and (upper half) what that leaves; nothing beside an infinity.
__device__ __forceinline__ uint32_t few_parts(float h) {
  const uint32_t hi = f32_to_bf16_bits(h);
  const float left = h - bf16_bits_to_f32(hi);
  return hi | (fabsf(left) < __builtin_inff() ? (uint32_t)f32_to_bf16_bits(left) << 16 : 0u);
}

// LDS of the first launch; the tokens stand behind it, 16 bytes apart in the banks.
struct FewLds {
  f32x4 part[2][kFewWaves][64];
  u32x4 zero[2];
  uint32_t mask[kFewWaves][MOE_MAX_EXPERTS / 32];  // the experts that a wave's tokens chose
  int32_t ids[kFewSlots];
  uint32_t keys[kFewSlots];
  int32_t list[kFewSlots];                    // the chosen experts, ascending
  int16_t slot[kFewSlots][kFewTokens];        // a chosen expert's slot of each token, or -1
  int32_t more[kFewSlots / 64];               // further entries of the experts of 64 ranks
};

// ONE: a single token.  ALONE: a task is a wave's own, the whole contraction of it, rather than a workgroup's.
template <class W, int NJ, bool ONE, bool ALONE>
__global__ __launch_bounds__(64 * kFewWaves) void few_gate_up_kernel(FewArgs p) {
  extern __shared__ u32x4 few_lds[];
  FewLds& s = *reinterpret_cast<FewLds*>(few_lds);
  char* xs = reinterpret_cast<char*>(few_lds) + (sizeof(FewLds) + 15) / 16 * 16;
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int T = ONE ? 1 : p.T, H = p.H, I = p.I, E = p.E, k = p.k, R = T * k;
  const bool writer = blockIdx.x == gridDim.x - 1;
  const int xstride = 2 * H + 16;

  // the logits of this wave's tokens, then the tokens
  constexpr int NT = ONE ? 1 : kFewTokens / kFewWaves;
  uint32_t u[NT][NJ];
#pragma unroll
  for (int a = 0; a < NT; ++a) {
    const int t = wave + a * kFewWaves;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int e = lane * NJ + j;
      u[a][j] = t < T && e < E ? max(ordered_bits(p.logits[(size_t)t * E + e]), 1u) : 0u;
    }
  }
  // a token's row by one wave, or by 2, 4 or 8 where there are fewer tokens: 8 chunks a lane at a time, of two rows 4 each
  constexpr int kAhead = 8;
  const int spread = T == 1 ? 3 : (T == 2 ? 2 : (T <= 4 ? 1 : 0)), xn = H / 8;
  const int xt = wave >> spread, xc = (wave & ((1 << spread) - 1)) * 64 + lane, xstep = 64 << spread;
  const bool two = !ONE && T > kFewWaves;
  const u32x4* x = reinterpret_cast<const u32x4*>(p.x);
  u32x4 xr[kAhead];
  auto fetch = [&](int from) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int t = xt + (two ? i / 4 * kFewWaves : 0), c = xc + (from + (two ? i % 4 : i)) * xstep;
      if (t < T && c < xn) xr[i] = x[t * xn + c];
    }
  };
  auto put = [&](int from) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int t = xt + (two ? i / 4 * kFewWaves : 0), c = xc + (from + (two ? i % 4 : i)) * xstep;
      if (t < T && c < xn) *reinterpret_cast<u32x4*>(xs + t * xstride + c * 16) = xr[i];
    }
  };
  fetch(0);
  if (tid == 0) s.zero[0] = s.zero[1] = u32x4{0u, 0u, 0u, 0u};
  for (int i = tid; i < R * (kFewTokens / 8); i += 64 * kFewWaves) reinterpret_cast<u32x4*>(s.slot)[i] = u32x4{~0u, ~0u, ~0u, ~0u};
  int id[NT] = {};
  uint32_t key[NT] = {}, chosen = 0u;
  if (wave < T) {
    if (!ONE && wave + kFewWaves < T) few_route<NT>(u, k, id, key, chosen);
    else few_route<1>(u, k, id, key, chosen);
#pragma unroll
    for (int a = 0; a < NT; ++a) {
      const int f = (wave + a * kFewWaves) * k + lane;
      if (wave + a * kFewWaves < T && lane < k) s.ids[f] = id[a], s.keys[f] = key[a];
    }
  }
  if (!ONE && lane < MOE_MAX_EXPERTS / 32) s.mask[wave][lane] = chosen;
  put(0);
  for (int from = two ? kAhead / 2 : kAhead; from * xstep < xn; from += two ? kAhead / 2 : kAhead) {
    fetch(from);
    put(from);
  }
  __syncthreads();
  int n = k;  // chosen experts
  if (!ONE) {  // each wave adds up the experts before every word of the mask, and a slot's thread finds its expert's rank
    uint32_t m = 0u;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) m |= s.mask[w][lane & (MOE_MAX_EXPERTS / 32 - 1)];
    if (lane >= MOE_MAX_EXPERTS / 32) m = 0u;
    int before = __popc(m);
#pragma unroll
    for (int d = 1; d < MOE_MAX_EXPERTS / 32; d <<= 1) {
      const int v = __shfl_up(before, d);
      if (lane >= d) before += v;
    }
    n = __builtin_amdgcn_readlane(before, MOE_MAX_EXPERTS / 32 - 1);
    before -= __popc(m);
    const int e = s.ids[min(tid, R - 1)];
    const int rank = __shfl(before, e >> 5) + __popc(__shfl((int)m, e >> 5) & ((1u << (e & 31)) - 1u));
    if (tid < R) {
      s.list[rank] = e;
      s.slot[rank][tid / k] = (int16_t)tid;
    }
    __syncthreads();
  }
  const int32_t* list = ONE ? s.ids : s.list;

  if (writer) {  // the routing, and the entries: an expert's first rows at its rank, further ones behind all experts, in their order
    for (int t = wave; t < T; t += kFewWaves) {
      const int f = t * k + min(lane, k - 1);
      const float w = few_weight(from_ordered_bits(s.keys[f]), k);
      if (lane < k) {
        p.ids[f] = s.ids[f];
        p.weight[f] = w;
      }
    }
    FewEntry* table = reinterpret_cast<FewEntry*>(p.table) + 1;
    int behind = n, entries = n;  // where this expert's further entries start, and the end of all
    if constexpr (!ONE) {
      int further = 0;  // at most 3: 16 rows by fours
      if (tid < n) {
        int rows = 0;
        const u32x4* slots = reinterpret_cast<const u32x4*>(s.slot[tid]);
#pragma unroll
        for (int i = 0; i < kFewTokens / 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) rows += __popc(~slots[i][j] & 0x80008000u);
        further = (rows - 1) / p.entry_rows;
      }
      const uint64_t ones = __ballot(further & 1), twos = __ballot(further & 2), below = (1ull << lane) - 1ull;
      behind += __popcll(ones & below) + 2 * __popcll(twos & below);
      if (lane == 0 && wave < kFewSlots / 64) s.more[wave] = __popcll(ones) + 2 * __popcll(twos);
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kFewSlots / 64; ++w) {
        behind += w < wave ? s.more[w] : 0;
        entries += s.more[w];
      }
    }
    if (tid < n) {
      FewEntry* at = table + tid;
      int have = 0;
      for (int t = 0; t < T; ++t) {
        const int f = ONE ? tid : s.slot[tid][t];
        if (f < 0) continue;
        if (have == p.entry_rows) {
          at->expert = list[tid];
          at->rows = have;
          at = table + behind++;
          have = 0;
        }
        at->row[have++] = (int16_t)f;
      }
      at->expert = list[tid];
      at->rows = have;
    }
    if (tid == 0) p.table[0] = entries;
  }

  // this wave's share of the contraction, in chunks of C steps
  constexpr int C = 4, RING = 2, STEP = 4 * W::LANE;
  const int steps = (H + STEP - 1) / STEP, share = ALONE ? steps : (steps + kFewWaves - 1) / kFewWaves;
  const int chunks = (share + C - 1) / C, blocks = I / 8;
  const int first = ALONE ? 0 : wave * share * STEP;             // of the contraction
  const int whole = max(0, min(share, (H - first) / STEP)) / C;  // chunks that lie within the share and the row
  const int some = min(share, (H - first + STEP - 1) / STEP);    // steps of which any lane's part does; others are not loaded (4
                                                                 // tokens, 68 experts top-9, int8 2112 x 2416: 74 us with them, 64)
  const uint32_t row_bytes = (uint32_t)H * W::BYTES;
  const uint32_t lane_offset = (uint32_t)(l16 < 8 ? l16 : I + l16 - 8) * row_bytes + (first + q * W::LANE) * W::BYTES;
  const char* xrow = xs + min(l16, T - 1) * xstride + (first + q * W::LANE) * 2;
  struct Cursor {
    int rank, block, chunk;
  };
  const int workers = ALONE ? gridDim.x * kFewWaves : gridDim.x, worker = ALONE ? blockIdx.x * kFewWaves + wave : blockIdx.x;
  const int rank_step = workers / blocks, block_step = workers - rank_step * blocks;
  auto advance = [&](Cursor& c) {
    if (++c.chunk < chunks) return;
    c.chunk = 0;
    c.rank += rank_step;
    c.block += block_step;
    if (c.block >= blocks) c.block -= blocks, ++c.rank;
  };
  u32x4 ring[RING][C];
  using Scales = std::conditional_t<ALONE, f32x4, float>;
  Scales sg[RING], su[RING];  // of the column that this thread finishes, or its four
  const uint32_t expert_bytes = (uint32_t)(2 * I) * row_bytes;
  auto load = [&](const Cursor& c, int b) {
    if (c.rank >= n) return;
    const int e = __builtin_amdgcn_readfirstlane(list[c.rank]);
    const auto buffer = few_buffer(static_cast<const char*>(p.w13) + (size_t)e * expert_bytes, expert_bytes);
    const uint32_t offset = lane_offset + (uint32_t)c.block * 8 * row_bytes + c.chunk * (C * STEP * W::BYTES);
#pragma unroll
    for (int i = 0; i < C; ++i) ring[b][i] = few_load(buffer, c.chunk * C + i < some ? offset + i * (STEP * W::BYTES) : kFewPast);
    if constexpr (W::SCALED && ALONE) if (c.chunk == chunks - 1) {
      const auto scales = few_buffer(p.w13_s + (size_t)e * (2 * I), (uint32_t)I * 8);
      sg[b] = __builtin_bit_cast(Scales, few_load(scales, (c.block * 8 + 4 * (q & 1)) * 4));
      su[b] = __builtin_bit_cast(Scales, few_load(scales, (I + c.block * 8 + 4 * (q & 1)) * 4));
    }
    if constexpr (W::SCALED && !ALONE) if (c.chunk == chunks - 1 && tid < 8 * kFewTokens) {
      const float* sc = p.w13_s + (size_t)e * (2 * I) + c.block * 8 + (tid & 7);
      sg[b] = sc[0];
      su[b] = sc[I];
    }
  };
  Cursor use = {worker / blocks, worker % blocks, 0}, ahead = use;
#pragma unroll
  for (int b = 0; b < RING; ++b) {
    load(ahead, b);
    advance(ahead);
  }
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  int turn = 0;
  for (;;) {
#pragma unroll
    for (int b = 0; b < RING; ++b) {
      if (use.rank >= n) return;
      const char* xk = xrow + use.chunk * (C * STEP * 2);
      if (use.chunk < whole) {
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
          for (int h = 0; h < W::PARTS; ++h)
            acc = mfma16x16x32(W::part(ring[b][i], h), *reinterpret_cast<const bf16x8*>(xk + i * (STEP * 2) + 16 * h), acc);
      } else {  // weights and tokens past the share or the row count as zeros
#pragma unroll
        for (int i = 0; i < C; ++i) {
          const int step = use.chunk * C + i;
          const bool in = step < share && first + step * STEP + q * W::LANE < H;
          const u32x4 w = few_keep(ring[b][i], in);
          const char* xi = in ? xk + i * (STEP * 2) : reinterpret_cast<const char*>(s.zero);
#pragma unroll
          for (int h = 0; h < W::PARTS; ++h)
            acc = mfma16x16x32(W::part(w, h), *reinterpret_cast<const bf16x8*>(xi + 16 * h), acc);
        }
      }
      const Scales scale_g = sg[b], scale_u = su[b];
      load(ahead, b);
      advance(ahead);
      if constexpr (ALONE) if (use.chunk == chunks - 1) {
        // gate rows are in the lower half of the wave, the up rows of the same columns and tokens 32 lanes on
        float h[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const auto gu = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[r]), __float_as_uint(acc[r]), false, false);
          float g = __uint_as_float(gu[0]), up = __uint_as_float(gu[1]);
          if (W::SCALED) g *= scale_g[r], up *= scale_u[r];
          h[r] = silu_f32(g) * up;
        }
        const int f = ONE ? (l16 == 0 ? use.rank : -1) : s.slot[use.rank][l16];
        if (lane < 32 && f >= 0) {
          u32x2 hi, lo;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t a = few_parts(h[2 * r]), b = few_parts(h[2 * r + 1]);
            hi[r] = (a & 0xFFFFu) | (b << 16);
            lo[r] = (a >> 16) | (b & 0xFFFF0000u);
          }
          u32x2* dst = reinterpret_cast<u32x2*>(p.h + ((size_t)f * blocks + use.block) * 16 + 4 * q);
          dst[0] = hi;
          dst[2] = lo;
        }
        acc = f32x4{0.f, 0.f, 0.f, 0.f};
      }
      if constexpr (!ALONE) if (use.chunk == chunks - 1) {
        s.part[turn][wave][lane] = acc;
        acc = f32x4{0.f, 0.f, 0.f, 0.f};
        __syncthreads();  // one a task: this half of part is written again only past the next task's barrier
        if (tid < 8 * kFewTokens) {
          const int c = tid & 7, t = tid >> 3;
          const int f = ONE ? (t == 0 ? use.rank : -1) : s.slot[use.rank][t];
          float g = 0.f, up = 0.f;
          const int from = (c >> 2) * 16 + t;
#pragma unroll
          for (int w = 0; w < kFewWaves; ++w) {
            g += reinterpret_cast<const float*>(&s.part[turn][w][from])[c & 3];
            up += reinterpret_cast<const float*>(&s.part[turn][w][from + 32])[c & 3];
          }
          if (W::SCALED) g *= scale_g, up *= scale_u;
          if (f >= 0) {
            const uint32_t parts = few_parts(silu_f32(g) * up);
            uint16_t* dst = p.h + ((size_t)f * blocks + use.block) * 16 + c;
            dst[0] = (uint16_t)parts;
            dst[8] = (uint16_t)(parts >> 16);
          }
        }
        turn ^= 1;
      }
      advance(use);
    }
  }
}

// The second launch: up to COLS (4, 8 or 16) columns of y a workgroup, whose group (blockIdx.y) takes every groups-th NW units.  A
// unit is an entry and every pieces-th super-chunk of SUPER elements of the contraction; a wave takes it from a place of
// its own on (workgroups in step would ask the same few memory channels).
// The instruction's 16 rows are 8 columns as two halves of the contraction, or 4 as four quarters (more workgroups where H
// is small); the 8 or 16 lanes of a row of weights read 128 or 256 bytes in a row of it, and what they take apart of the
// contraction is added at the end.  The entry's rows of h come as whole lines, one load a row and 256 elements, and reach
// the lanes that need them through the wave's own LDS: as operands straight from memory they would be fetched 4 to 16
// times over, which the L1s do not give beside the weights.
template <class W, int COLS, int SUPER, int TOK, int RING, int NW>
__global__ __launch_bounds__(64 * NW) void few_down_kernel(FewArgs p) {
  constexpr int kHRow = SUPER * 4 + 16, HB = SUPER / 256;  // a row of h in LDS, and its 1 KB loads
  constexpr int MR = COLS == 4 ? 4 : 8, CT = COLS / MR, SPLIT = 16 / MR;  // columns of an instruction, instructions, parts
  constexpr int LINE = 4 * SPLIT;                                        // lanes of a row of weights
  static_assert(TOK <= MR, "a column of the instruction for each row and part");
  extern __shared__ u32x4 few_lds[];
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int T = p.T, H = p.H, I = p.I, k = p.k, R = T * k, shift = p.pieces_shift;
  char* stage = reinterpret_cast<char*>(few_lds) + wave * (TOK * kHRow);
  FewEntry* table = reinterpret_cast<FewEntry*>(reinterpret_cast<char*>(few_lds) + NW * TOK * kHRow);
  float* weight = reinterpret_cast<float*>(table + R);
  f32x4* out = reinterpret_cast<f32x4*>(weight + (R + 3) / 4 * 4);  // [pieces][R][COLS / 4]
  const int groups = p.groups, group = blockIdx.y, col0 = blockIdx.x * p.cols, cols = min(p.cols, H - col0);
  const int n = __builtin_amdgcn_readfirstlane(p.table[0]);
  if (tid < 2 * R) reinterpret_cast<u32x4*>(table)[tid] = reinterpret_cast<const u32x4*>(p.table)[2 + tid];
  if (tid < R) weight[tid] = p.weight[tid];
  if (groups > 1)  // what other groups add counts as zero here
    for (int i = tid; i < (R << shift) * (COLS / 4); i += 64 * NW) out[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  __syncthreads();

  constexpr int C = SUPER / LINE / W::LANE;  // steps of a super-chunk
  const int pieces = 1 << shift, units = n << shift;
  const int supers = (I + SUPER - 1) / SUPER;
  const bool ragged = I % SUPER != 0;
  const int m = l16 & (MR - 1), in_line = q * SPLIT + l16 / MR;
  const uint32_t row_bytes = (uint32_t)I * W::BYTES;
  const uint32_t expert_bytes = (uint32_t)H * row_bytes;
  uint32_t lane_offset[CT];  // rows that are another workgroup's are past the end: no bytes move for them
#pragma unroll
  for (int ct = 0; ct < CT; ++ct)
    lane_offset[ct] = ct * MR + m < cols ? (uint32_t)(col0 + ct * MR + m) * row_bytes + in_line * 16 : expert_bytes;
  const char* hfrag = stage + min(m, TOK - 1) * kHRow + in_line * (W::PARTS * 32);
  struct Cursor {
    int i, unit, super, left;
  };
  const int turn = (blockIdx.x >> 3) % (supers >> shift), worker = wave + NW * group, workers = NW * groups;
  auto begin = [&](int i, int unit) {
    const int piece = unit & (pieces - 1);
    return Cursor{i, unit, piece + (turn << shift), (supers - piece + pieces - 1) >> shift};
  };
  auto advance = [&](Cursor& c) {
    if (--c.left == 0) {
      c = begin(c.i + 1, c.unit + workers);
      return;
    }
    c.super += pieces;
    if (c.super >= supers) c.super = c.unit & (pieces - 1);
  };
  u32x4 ring[RING][CT][C], hv[RING][TOK][HB];
  f32x4 sc[RING][CT];
  // lane i holds what the wave's i-th unit needs (there are at most 64), so that no unit waits for LDS
  const FewEntry& own = table[min((worker + workers * lane) >> shift, n - 1)];
  const int own_expert = own.expert, own_rows = own.rows;
  uint32_t own_row[(TOK + 1) / 2];
#pragma unroll
  for (int j = 0; j < (TOK + 1) / 2; ++j) own_row[j] = reinterpret_cast<const uint32_t*>(own.row)[j];
  auto row_of = [&](int i, int j) { return (__builtin_amdgcn_readlane(own_row[j >> 1], i) >> (16 * (j & 1))) & 0xFFFFu; };
  auto load = [&](const Cursor& c, int b) {
    if (c.unit >= units) return;
    const int e = __builtin_amdgcn_readlane(own_expert, c.i), rows = __builtin_amdgcn_readlane(own_rows, c.i);
    const auto buffer = few_buffer(static_cast<const char*>(p.w2) + (size_t)e * expert_bytes, expert_bytes);
    const uint32_t offset = c.super * (SUPER * W::BYTES);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int i = 0; i < C; ++i) ring[b][ct][i] = few_load(buffer, lane_offset[ct] + offset + i * (LINE * 16));
#pragma unroll
    for (int j = 0; j < TOK; ++j)
      if (j < rows) {
        const auto hrow = few_buffer(p.h + (size_t)row_of(c.i, j) * I * 2, (uint32_t)I * 4);
#pragma unroll
        for (int v = 0; v < HB; ++v) hv[b][j][v] = few_load(hrow, lane * 16 + c.super * (SUPER * 4) + v * 1024);
      }
    if (W::SCALED && c.left == 1) {
      const auto scales = few_buffer(p.w2_s + (size_t)e * H, (uint32_t)H * 4);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
        sc[b][ct] = __builtin_bit_cast(f32x4, few_load(scales, (col0 + ct * MR + (MR == 8 ? 4 * (q & 1) : 0)) * 4));
    }
  };
  Cursor use = begin(0, worker), ahead = use;
#pragma unroll
  for (int b = 0; b < RING; ++b) {
    load(ahead, b);
    advance(ahead);
  }
  f32x4 acc[CT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) acc[ct] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (;;) {
#pragma unroll
    for (int b = 0; b < RING; ++b) {
      if (use.unit >= units) goto summed;
      const int rows = __builtin_amdgcn_readlane(own_rows, use.i);
      const bool last = use.super == supers - 1 && ragged;  // weights past the row count as zeros; h past its end was read so
      if (last) {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
          for (int i = 0; i < C; ++i) ring[b][ct][i] = few_keep(ring[b][ct][i], use.super * SUPER + (i * LINE + in_line) * W::LANE < I);
      }
#pragma unroll
      for (int j = 0; j < TOK; ++j)
        if (j < rows) {
#pragma unroll
          for (int v = 0; v < HB; ++v) *reinterpret_cast<u32x4*>(stage + j * kHRow + v * 1024 + lane * 16) = hv[b][j][v];
        }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int h = 0; h < W::PARTS; ++h) {
          const char* at = hfrag + i * (LINE * W::PARTS * 32) + h * 32;
          const bf16x8 hi = *reinterpret_cast<const bf16x8*>(at), lo = *reinterpret_cast<const bf16x8*>(at + 16);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) {
            const bf16x8 a = W::part(ring[b][ct][i], h);
            acc[ct] = mfma16x16x32(a, hi, acc[ct]);
            acc[ct] = mfma16x16x32(a, lo, acc[ct]);
          }
        }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      f32x4 scale[CT];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) scale[ct] = W::SCALED ? sc[b][ct] : f32x4{1.f, 1.f, 1.f, 1.f};
      load(ahead, b);
      advance(ahead);
      if (use.left == 1) {
        const int f = (use.unit & (pieces - 1)) * R + table[use.unit >> shift].row[m];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          f32x4 o;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            // part n's results stand in rows and columns MR * n + : 20 or 40 lanes further each
            o[r] = acc[ct][r];
#pragma unroll
            for (int n = 1; n < SPLIT; ++n) o[r] += __shfl(acc[ct][r], (lane + n * (MR == 8 ? 40 : 20)) & 63);
            if (W::SCALED) o[r] *= scale[ct][r];
          }
          if (q < MR / 4 && l16 < rows) out[(f * CT + ct) * (MR / 4) + q] = o;
          acc[ct] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
      }
      advance(use);
    }
  }
summed:
  __syncthreads();
  const int t = tid / COLS, c = tid % COLS;
  const bool mine = tid < COLS * T && c < cols;
  float y = 0.f;
  if (mine) {
    const float* o8 = reinterpret_cast<const float*>(out) + c;
    for (int s = 0; s < k; s += 4) {  // four slots' values are asked for at a time; their sum is that of the slots in order
      float o[4], w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int f = t * k + min(s + j, k - 1);
        w[j] = weight[f];
        o[j] = o8[f * COLS];
        for (int i = 1; i < pieces; ++i) o[j] += o8[(i * R + f) * COLS];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (s + j < k && w[j] != 0.f) y = fmaf(w[j], o[j], y);  // a closed expert may hold anything
    }
  }
  if (!mine) return;
  const size_t at = (size_t)t * H + col0 + c;
  if (groups > 1) p.parts[(size_t)group * T * H + at] = y;
  else p.y[at] = f32_to_bf16_bits(y);
}

// y from the parts of the second launch's groups, in their order.
__global__ __launch_bounds__(256) void few_join_kernel(const float* __restrict__ parts, int groups, int n, uint16_t* __restrict__ y) {
  const int i = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  for (int g = 0; g < groups; g += 4) {
    f32x4 a[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = *reinterpret_cast<const f32x4*>(parts + (size_t)min(g + j, groups - 1) * n + i);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (g + j < groups) v += a[j];
  }
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = f32_to_bf16_bits(v[j]);
  *reinterpret_cast<u32x2*>(y + i) = u32x2{o[0] | o[1] << 16, o[2] | o[3] << 16};
}

// Columns of a workgroup of the second launch, at most `most`: H dealt evenly to 256 CUs, or to as many workgroups a CU as it
// takes.  The CUs share the memory's rate evenly, so that one with a workgroup more than the others ends far later (4 tokens, 68
// experts top-9, bf16, I 1024: 2048 columns, 256 workgroups of 8, 24.6 us; 2064, 258 of 8, 37.7, and 230 of 9 26.3; 1040, 130 of
// 8 or 260 of 4, 24.3, and 208 of 5 16.7; 8 tokens, 64 experts top-6, bf16 768 x 768 14.7 with 4 and 12.7 with 3).  Rows of the instruction that are left over move no bytes.
static int few_columns(int H, int most) {
  const int rounds = (H + 256 * most - 1) / (256 * most);
  return std::max(most / 2 + 1, (H + 256 * rounds - 1) / (256 * rounds));
}

// Entries that the second launch has to expect: of one token exactly its k, of more the distinct experts of even routing, or
// what the entries' rows make of all slots.
static double few_entries(const FewArgs& p) {
  if (p.T == 1) return p.k;
  double spared = 1.0;
  for (int t = 0; t < p.T; ++t) spared *= 1.0 - (double)p.k / p.E;
  return std::max(p.E * (1.0 - spared), (double)(p.T * p.k) / p.entry_rows);
}

template <class W, int NJ, bool ONE, bool ALONE>
static hipError_t launch_few_first(const FewArgs& p, hipStream_t s) {
  const int lds = (int)((sizeof(FewLds) + 15) / 16 * 16) + p.T * (2 * p.H + 16);
  // Workgroups a CU: of one token three, which then have a piece of the largest of its layers each; of more two, as every
  // workgroup routes all of them (11 tokens, 60 experts top-6, 1040 x 336 int8: 27.3 us with two, 29.6 with three).
  const int fit = std::max(1, std::min(ONE ? 3 : 2, (160 << 10) / lds));
  const int tasks = std::min(p.E, p.T * p.k) * (p.I / 8);
  const int grid = std::min(ALONE ? (tasks + kFewWaves - 1) / kFewWaves : tasks, 256 * fit);
  const auto kernel = few_gate_up_kernel<W, NJ, ONE, ALONE>;
  if (lds > (64 << 10)) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  kernel<<<grid, 64 * kFewWaves, lds, s>>>(p);
  return hipGetLastError();
}

template <class W, int NJ>
static hipError_t launch_few_of(const FewArgs& p, hipStream_t s) {
  // Short rows of weights: a wave a task, without the barrier and the meeting that a task of a workgroup ends with (12 tokens, 64
  // experts top-4, 256 x 7168: bf16 54 us against 127, int8 128 x 7168 29 against 135; int8 1536 x 1040 21.4 against 22.5,
  // bf16 1536 x 1040 36 against 33).  One token has too few tasks for that beyond H 512 (512 x 1536 int8: 7.2 us against 10.6,
  // 1024 x 512: 10.2 against 7.7).
  const bool alone = p.T == 1 ? p.H <= 512 : p.H * W::BYTES <= 1536;
  if (alone) return p.T == 1 ? launch_few_first<W, NJ, true, true>(p, s) : launch_few_first<W, NJ, false, true>(p, s);
  return p.T == 1 ? launch_few_first<W, NJ, true, false>(p, s) : launch_few_first<W, NJ, false, false>(p, s);
}

template <class W, int COLS, int SUPER, int TOK, int RING, int NW>
static hipError_t launch_few_second(FewArgs p, hipStream_t s) {
  const int R = p.T * p.k, supers = (p.I + SUPER - 1) / SUPER;
  const double entries = few_entries(p);
  // Groups of workgroups that share the units of the same columns where there are few columns and many units: a wave's super-chunk
  // takes about 0.9 us, the third launch that adds the groups' parts 4.5 (11 tokens, 118 experts top-8, int8 224 x 13712: 201 us
  // down in one group, 62 in eight; 10 tokens, 46 experts top-9, bf16 592 x 5280: 89 and 73).
  if (p.H <= kFewGroupsH && entries * supers > 16.0 * NW) p.groups = std::max(1, std::min(kFewGroups, 512 * COLS / p.H));
  p.cols = p.groups > 1 ? COLS : few_columns(p.H, COLS);
  const int columns = (p.H + p.cols - 1) / p.cols;
  // Pieces (a power of two) of the contraction that units are cut into, no more than there are super-chunks: one token's entries,
  // all alike, until every wave has a unit; of more tokens until there are about 32, so that the waves end together (9 tokens, 10
  // experts top-8, int8 1760 x 4672: 50 us uncut, 42 in quarters).  At most 64 units a wave, each a lane's, whatever
  // the routing: R bounds the entries.
  const double want = p.T == 1 ? NW * p.groups : 30;
  while (entries * (1 << p.pieces_shift) < want && (2 << p.pieces_shift) <= supers && (R << (p.pieces_shift + 1)) <= 64 * NW)
    ++p.pieces_shift;
  const int lds = NW * TOK * (SUPER * 4 + 16) + R * 32 + (R + 3) / 4 * 16 + (R << p.pieces_shift) * 4 * COLS;
  const auto kernel = few_down_kernel<W, COLS, SUPER, TOK, RING, NW>;
  if (lds > (64 << 10)) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  kernel<<<dim3(columns, p.groups), 64 * NW, lds, s>>>(p);
  if (p.groups > 1) {
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const int n = p.T * p.H;
    few_join_kernel<<<(n / 4 + 255) / 256, 256, 0, s>>>(p.parts, p.groups, n, p.y);
  }
  return hipGetLastError();
}

template <class W>
static hipError_t launch_few_w(FewArgs p, hipStream_t s) {
  // rows of an entry: more where the experts are crowded, so that their weights are read once
  const bool crowded = p.T * p.k > 2 * p.E;
  p.entry_rows = p.T == 1 ? 1 : (crowded ? 8 : 4);
  hipError_t e;
  if (p.E <= 128) e = launch_few_of<W, 2>(p, s);
  else if (p.E <= 256) e = launch_few_of<W, 4>(p, s);
  else if (p.E <= 512) e = launch_few_of<W, 8>(p, s);
  else e = launch_few_of<W, 16>(p, s);
  if (e != hipSuccess) return e;
  // 4 columns a workgroup where more would leave half the CUs idle and the contraction fills super-chunks of 512 (8 tokens, 64
  // experts top-6, 1024 x 512, bf16: 10.4 us against 13.5); 16 at most where 8 would be more than a workgroup a CU (16 tokens, 8
  // experts of 4096 x 14336: 163 us against 190; int8, 4 tokens, 256 experts, 7168 x 2048: 85 against 91)
  const bool narrow = p.H <= 1024 && p.I >= 512, wide = p.H > 2048;
  if (p.T == 1) {
    if (narrow) return launch_few_second<W, 4, 512, 1, 2, 8>(p, s);
    if (wide) return launch_few_second<W, 16, 256, 1, 2, 8>(p, s);
    return launch_few_second<W, 8, 256, 1, 3, 8>(p, s);
  }
  if (crowded) {
    if (wide) return launch_few_second<W, 16, 256, 8, 2, 8>(p, s);
    return launch_few_second<W, 8, 256, 8, 2, 8>(p, s);
  }
  if (narrow) return launch_few_second<W, 4, 512, 4, 2, 8>(p, s);
  // int8 units are half as long in bytes and convert their weights: twice the waves where a CU has one workgroup (16 tokens, 256
  // experts top-8, 2048 x 512: 24 us against 26; 4 tokens, 68 experts top-9, 2304 x 2048 31.7 against 39.4, but 5120 x 2048 64
  // against 61; bf16, 8 tokens, 128 experts, 2048 x 768: 32 us against 31, so not there)
  if constexpr (W::SCALED) {
    if (p.H <= 2048) return launch_few_second<W, 8, 256, 4, 2, 16>(p, s);
    if (p.H <= 4096) return launch_few_second<W, 16, 256, 4, 2, 16>(p, s);
  }
  if (wide) return launch_few_second<W, 16, 256, 4, 2, 8>(p, s);
  return launch_few_second<W, 8, 256, 4, 3, 8>(p, s);
}

hipError_t launch_ffn_few(const FewArgs& p, bool i8, hipStream_t stream) {
  return i8 ? launch_few_w<FewW8>(p, stream) : launch_few_w<FewW16>(p, stream);
}

}  // namespace moe
