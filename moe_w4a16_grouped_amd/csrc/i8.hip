// INT8 (W8A8) variant: 8-bit integer codes with one fp32 scale per activation row (token) and one per
// weight row (channel).  The ATOM page ("AMD ATOM推理引擎：如何用分页KV缓存和分段编译实现大模型推理性能翻倍"),
// section "6.1 Linear：按量化类型分派 GEMM", dispatches linears by their quantization type; section "8.2 量化
// 并非单一格式，而是一套执行契约" makes dynamic activation quantization part of a format's contract.
//
// value = code * scale, codes in [-127, 127].  A row is quantized as s = fp32(max |x| / 127), code = the
// integer nearest to the real quotient x / s, ties to even: exactly, so that the codes of a row do not
// depend on how a division rounds.  With n = rint(x * (1 / s)) the sign of fma(-(n + 1/2), s, x) says
// whether x / s lies above n + 1/2 (a fused multiply-add rounds once, so its sign is that of the exact
// difference); the same below.  Sums of products of codes are exact in int32 (K <= 2^17).
#include "ragged_gemm.h"

namespace moe {

__device__ __forceinline__ int i8_code(float x, float s, float inv) {
  float n = rintf(x * inv);
  const float up = fmaf(-(n + 0.5f), s, x), down = fmaf(-(n - 0.5f), s, x);
  const bool odd = ((int)n & 1) != 0;
  if (up > 0.f || (up == 0.f && odd)) n += 1.f;
  else if (down < 0.f || (down == 0.f && odd)) n -= 1.f;
  return (int)fminf(fmaxf(n, -127.f), 127.f);
}

// Eight consecutive elements of x as fp32.
template <int IN>
__device__ __forceinline__ void i8_load8(const void* x, size_t at, float (&v)[8]) {
  if (IN == MOE_IN_F32) {
    const f32x4* src = reinterpret_cast<const f32x4*>(static_cast<const float*>(x) + at);
    const f32x4 a = src[0], b = src[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) { v[j] = a[j]; v[4 + j] = b[j]; }
  } else {
    const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x) + at);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = IN == MOE_IN_F16 ? f16_bits_to_f32(w[j] & 0xFFFFu) : bf16_bits_to_f32(w[j] & 0xFFFFu);
      v[2 * j + 1] = IN == MOE_IN_F16 ? f16_bits_to_f32(w[j] >> 16) : bf16_bits_to_f32(w[j] >> 16);
    }
  }
}

// The largest magnitude as the bits of |x|, which order like the values with infinities and NaN above
// every finite one: a row that holds either gets the scale NaN and codes 0.
__device__ __forceinline__ uint32_t i8_amax8(const float (&v)[8], uint32_t m) {
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  return m;
}
__device__ __forceinline__ float i8_scale(uint32_t m) {
  return m >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : __uint_as_float(m) / 127.0f;
}
__device__ __forceinline__ u32x2 i8_codes8(const float (&v)[8], float s) {
  u32x2 w = {0u, 0u};
  if (!(s > 0.f)) return w;  // an all-zero row, or NaN
  // the quotients of a row of tiny values are taken 2^64 times as large (exactly): 1 / s must not overflow, nor a
  // difference be too small for fp32
  const float up = s < 0x1p-64f ? 0x1p64f : 1.0f;
  s *= up;
  const float inv = 1.0f / s;
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j >> 2] |= (uint32_t)(i8_code(v[j] * up, s, inv) & 0xFF) << (8 * (j & 3));
  return w;
}

// One workgroup per row, 8 elements a thread and chunk.  J chunks a thread stay in registers between the
// maximum and the codes; with J == 0 (longer rows) they are read again.  Small batches are bound by latency (77 x 2048: 3.3
// us), large ones by it too: 4096 x 4096 bf16 takes 17 us (3.0 TB/s of x and codes, where a copy reaches 4.9), as a
// workgroup waits for its one row before it writes and half of its four chunks a thread are empty there.
template <int IN, int J, int TH>
__global__ __launch_bounds__(TH) void i8_quant_kernel(const void* __restrict__ x, int rows, int K,
                                                      int8_t* __restrict__ q, float* __restrict__ s) {
  __shared__ uint32_t wmax[TH / 64];
  const long long row = linear_block();
  if (row >= rows) return;
  const int tid = threadIdx.x, nc = K / 8;
  const size_t base = (size_t)row * K;
  float v[J > 0 ? J : 1][8];
  uint32_t m = 0;
  if constexpr (J > 0) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = tid + j * TH;
      if (c < nc) {
        i8_load8<IN>(x, base + 8 * (size_t)c, v[j]);
        m = i8_amax8(v[j], m);
      }
    }
  } else {
    for (int c = tid; c < nc; c += TH) {
      i8_load8<IN>(x, base + 8 * (size_t)c, v[0]);
      m = i8_amax8(v[0], m);
    }
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
  if constexpr (TH > 64) {
    if ((tid & 63) == 0) wmax[tid >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < TH / 64; ++w) m = max(m, wmax[w]);
  }
  const float sc = i8_scale(m);
  if (tid == 0) s[row] = sc;
  if constexpr (J > 0) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = tid + j * TH;
      if (c < nc) *reinterpret_cast<u32x2*>(q + base + 8 * (size_t)c) = i8_codes8(v[j], sc);
    }
  } else {
    for (int c = tid; c < nc; c += TH) {
      i8_load8<IN>(x, base + 8 * (size_t)c, v[0]);
      *reinterpret_cast<u32x2*>(q + base + 8 * (size_t)c) = i8_codes8(v[0], sc);
    }
  }
}

template <int IN>
static hipError_t launch_quant(const void* x, int rows, int K, int8_t* q, float* s, hipStream_t st) {
  const dim3 grid = grid2d(rows);  // a launch dimension holds fewer than 2^32 threads
  if (K <= 512) i8_quant_kernel<IN, 1, 64><<<grid, 64, 0, st>>>(x, rows, K, q, s);
  else if (K <= 2048) i8_quant_kernel<IN, 1, 256><<<grid, 256, 0, st>>>(x, rows, K, q, s);
  else if (K <= 8192) i8_quant_kernel<IN, 4, 256><<<grid, 256, 0, st>>>(x, rows, K, q, s);
  else i8_quant_kernel<IN, 0, 256><<<grid, 256, 0, st>>>(x, rows, K, q, s);
  return hipGetLastError();
}

hipError_t launch_i8_quant(const void* x, int in_dtype, int rows, int K, int8_t* q, float* s, hipStream_t stream) {
  if (in_dtype == MOE_IN_F32) return launch_quant<MOE_IN_F32>(x, rows, K, q, s, stream);
  if (in_dtype == MOE_IN_F16) return launch_quant<MOE_IN_F16>(x, rows, K, q, s, stream);
  return launch_quant<MOE_IN_BF16>(x, rows, K, q, s, stream);
}

// ---------------------------------------------------------------------------------------------------
// A few rows (T <= 16, T * K <= kI8FewElems) in one launch: a workgroup takes all of them and 16 columns (SiLU*mul: 16
// gate rows of the weights and their up rows), quantizes the rows itself, into LDS, and its four waves take a quarter
// of the contraction each; their integer sums are exact in any order and meet in LDS.  x is asked for first and the
// weights and their scales right behind it, straight to registers, kI8FewAhead 64-byte groups at a time, so that one
// round trip covers them all.  Bound by latency, us on the device, this against the two launches: 1 x 2048 x 768 4.2
// against 7.4, 1 x 28672 x 4096 26 against 34, 4 x 2048 x 2048 6.5 against 8.9, 8 x 2048 x 768 6.6 against 7.4, 16 x
// 2048 x 512 7.2 against 7.1 (eager calls: 8 against 12).  Every workgroup repeats the quantization: with more than
// kI8FewCols columns more than four rows take the two launches (5 x 8192 x 1600: 12.1 against 9.5, 8 x 28672 x 1024: 20
// against 12.5).
constexpr int kI8FewRows = 16;
constexpr int kI8FewElems = 8192;
constexpr int kI8FewCols = 4096;
constexpr int kI8FewAhead = 8;

bool i8_few_always(int T, int K) { return T <= 4 && (long long)T * K <= kI8FewElems; }
bool i8_few_fits(int T, int K, int cols) {
  return i8_few_always(T, K) || (T <= kI8FewRows && (long long)T * K <= kI8FewElems && cols <= kI8FewCols);
}

// 256 threads a row for one row, 128 for two, 64 (a wave) for more
__device__ __forceinline__ int few_threads(int rows) { return rows == 1 ? 256 : (rows == 2 ? 128 : 64); }

// ROWS: rows of a thread, at most; CH: chunks of 8 elements that it holds of each.
template <int IN, int EPI, int ROWS, int CH>
__global__ __launch_bounds__(256) void linear_i8_few_kernel(const void* __restrict__ x, const int8_t* __restrict__ W,
                                                            const float* __restrict__ Ws, int T, int N, int K,
                                                            void* __restrict__ y, int out) {
  constexpr bool SILU = EPI == MOE_EPI_SILU_MUL;
  constexpr int NB = SILU ? 2 : 1;  // blocks of 16 weight rows
  // codes [rows][K rounded to 64, and 16 more], rows 16 bytes apart in the banks
  __shared__ __attribute__((aligned(16))) uint8_t codes[kI8FewElems + kI8FewRows * 80];
  __shared__ float sx[kI8FewRows];
  __shared__ uint32_t wmax[4];
  __shared__ int32_t part[3][NB * 4][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l16 = lane & 15, q = lane >> 4;
  const int ND = SILU ? N / 2 : N;
  const int col0 = blockIdx.x * 16;
  const int groups = (K + 63) / 64, share = (groups + 3) / 4;
  const int g0 = min(wave * share, groups), g1 = min(groups, g0 + share);
  const int stride = groups * 64 + 16;

  const int tpr = few_threads(T), nc = K / 8, c0 = tid % tpr, r0 = tid / tpr;
  float v[ROWS][CH][8];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int r = min(r0 + i * (256 / tpr), T - 1);
#pragma unroll
    for (int j = 0; j < CH; ++j)
      if (c0 + j * tpr < nc) i8_load8<IN>(x, (size_t)r * K + 8 * (size_t)(c0 + j * tpr), v[i][j]);
  }
  __builtin_amdgcn_sched_barrier(0);

  const int8_t* wrow[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int n = col0 + l16;  // past the edge row 0, which only reaches results that are not stored
    wrow[b] = W + (size_t)((n < ND ? n : 0) + b * ND) * K;
  }
  u32x4 w[kI8FewAhead][NB];
  auto load = [&](int g) {  // groups g .. g + kI8FewAhead - 1 of this wave's share; zeros past the row's end
#pragma unroll
    for (int i = 0; i < kI8FewAhead; ++i) {
      const int k = (g + i) * 64 + 16 * q;
#pragma unroll
      for (int b = 0; b < NB; ++b)
        w[i][b] = g + i < g1 && k < K ? *reinterpret_cast<const u32x4*>(wrow[b] + k) : u32x4{0u, 0u, 0u, 0u};
    }
  };
  load(g0);
  float ws[NB][4];  // the scales of wave 0's results
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = col0 + 4 * q + i;
      ws[b][i] = Ws[(n < ND ? n : 0) + b * ND];
    }
  __builtin_amdgcn_sched_barrier(0);

#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int r = r0 + i * (256 / tpr);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < CH; ++j)
      if (c0 + j * tpr < nc) m = i8_amax8(v[i][j], m);
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
    if (ROWS == 1 && tpr > 64) {  // one or two rows, whole waves a row
      if (lane == 0) wmax[wave] = m;
      __syncthreads();
      const int w0 = wave / (tpr / 64) * (tpr / 64);
      for (int k = 0; k < tpr / 64; ++k) m = max(m, wmax[w0 + k]);
    }
    const float sc = i8_scale(m);
    if (r < T) {
      if (c0 == 0) sx[r] = sc;
#pragma unroll
      for (int j = 0; j < CH; ++j)
        if (c0 + j * tpr < nc) *reinterpret_cast<u32x2*>(codes + r * stride + 8 * (c0 + j * tpr)) = i8_codes8(v[i][j], sc);
      // codes past the row's end meet weights of zero
    }
  }
  __syncthreads();

  i32x4 acc[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) acc[b] = i32x4{0, 0, 0, 0};
  const uint8_t* arow = codes + min(l16, T - 1) * stride + 16 * q;
  for (int g = g0; g < g1; g += kI8FewAhead) {
    if (g > g0) load(g);
#pragma unroll
    for (int i = 0; i < kI8FewAhead; ++i) {
      const u32x4 a = *reinterpret_cast<const u32x4*>(arow + min(g + i, groups - 1) * 64);
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[b] = ElemI8::mfma(w[i][b], a, acc[b]);
    }
  }
  if (wave > 0) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[wave - 1][b * 4 + i][lane] = acc[b][i];
  }
  __syncthreads();
  if (wave > 0 || l16 >= T) return;
  const float sa = sx[l16];
  auto sum = [&](int b, int i) {
    return (float)(acc[b][i] + part[0][b * 4 + i][lane] + part[1][b * 4 + i][lane] + part[2][b * 4 + i][lane]) * (sa * ws[b][i]);
  };
  const int col = col0 + 4 * q;
  const size_t at = (size_t)l16 * ND + col;
  float r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = SILU ? silu_f32(sum(0, i)) * sum(NB - 1, i) : sum(0, i);
  if ((ND & 3) == 0) {
    if (col < ND) store4(y, out, at, r);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + i < ND) store1(y, out, at + i, r[i]);
  }
}

template <int IN, int ROWS, int CH>
static hipError_t launch_few(const void* x, const int8_t* Wq, const float* Ws, int T, int N, int K, int epilogue, void* y,
                             int out, hipStream_t s) {
  const bool silu = epilogue == MOE_EPI_SILU_MUL;
  const int nd = silu ? N / 2 : N;
  const int grid = (nd + 15) / 16;
  if (silu) linear_i8_few_kernel<IN, MOE_EPI_SILU_MUL, ROWS, CH><<<grid, 256, 0, s>>>(x, Wq, Ws, T, N, K, y, out);
  else linear_i8_few_kernel<IN, MOE_EPI_NONE, ROWS, CH><<<grid, 256, 0, s>>>(x, Wq, Ws, T, N, K, y, out);
  return hipGetLastError();
}

// T * K <= kI8FewElems bounds the chunks of a row: K <= 8192, 4096 and 2730 for one, two and three rows (4, 4 and 6 of
// 256, 128 and 64 threads), 2048 for four (4), 1638 for five (4), 910 for nine (2).
template <int IN>
static hipError_t launch_few_of(const void* x, const int8_t* Wq, const float* Ws, int T, int N, int K, int epilogue,
                                void* y, int out, hipStream_t s) {
  if (T == 3) return launch_few<IN, 1, 6>(x, Wq, Ws, T, N, K, epilogue, y, out, s);
  if (T <= 4) return launch_few<IN, 1, 4>(x, Wq, Ws, T, N, K, epilogue, y, out, s);
  if (T <= 8) return launch_few<IN, 2, 4>(x, Wq, Ws, T, N, K, epilogue, y, out, s);
  return launch_few<IN, 4, 2>(x, Wq, Ws, T, N, K, epilogue, y, out, s);
}

hipError_t launch_linear_i8_few(const void* x, int in_dtype, const int8_t* Wq, const float* Ws, int T, int N, int K,
                                int epilogue, void* y, int out, hipStream_t stream) {
  if (in_dtype == MOE_IN_F32) return launch_few_of<MOE_IN_F32>(x, Wq, Ws, T, N, K, epilogue, y, out, stream);
  if (in_dtype == MOE_IN_F16) return launch_few_of<MOE_IN_F16>(x, Wq, Ws, T, N, K, epilogue, y, out, stream);
  return launch_few_of<MOE_IN_BF16>(x, Wq, Ws, T, N, K, epilogue, y, out, stream);
}

hipError_t launch_ragged_i8(const RaggedArgs& a, int epilogue, hipStream_t stream) {
  return epilogue == MOE_EPI_SILU_MUL ? launch_ragged_fwd<ElemI8, MOE_EPI_SILU_MUL>(a, stream)
                                      : launch_ragged_fwd<ElemI8, MOE_EPI_NONE>(a, stream);
}

}  // namespace moe
