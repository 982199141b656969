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
  const float inv = 1.0f / s;
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j >> 2] |= (uint32_t)(i8_code(v[j], s, inv) & 0xFF) << (8 * (j & 3));
  return w;
}

// One workgroup per row, 8 elements a thread and chunk.  J chunks a thread stay in registers between the
// maximum and the codes; with J == 0 (longer rows) they are read again.
template <int IN, int J, int TH>
__global__ __launch_bounds__(TH) void i8_quant_kernel(const void* __restrict__ x, int K, int8_t* __restrict__ q,
                                                      float* __restrict__ s) {
  __shared__ uint32_t wmax[TH / 64];
  const int row = blockIdx.x, tid = threadIdx.x, nc = K / 8;
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
  if (K <= 512) i8_quant_kernel<IN, 1, 64><<<rows, 64, 0, st>>>(x, K, q, s);
  else if (K <= 2048) i8_quant_kernel<IN, 1, 256><<<rows, 256, 0, st>>>(x, K, q, s);
  else if (K <= 8192) i8_quant_kernel<IN, 4, 256><<<rows, 256, 0, st>>>(x, K, q, s);
  else i8_quant_kernel<IN, 0, 256><<<rows, 256, 0, st>>>(x, K, q, s);
  return hipGetLastError();
}

hipError_t launch_i8_quant(const void* x, int in_dtype, int rows, int K, int8_t* q, float* s, hipStream_t stream) {
  if (in_dtype == MOE_IN_F32) return launch_quant<MOE_IN_F32>(x, rows, K, q, s, stream);
  if (in_dtype == MOE_IN_F16) return launch_quant<MOE_IN_F16>(x, rows, K, q, s, stream);
  return launch_quant<MOE_IN_BF16>(x, rows, K, q, s, stream);
}

hipError_t launch_ragged_i8(const RaggedArgs& a, int epilogue, hipStream_t stream) {
  return epilogue == MOE_EPI_SILU_MUL ? launch_ragged_fwd<ElemI8, MOE_EPI_SILU_MUL>(a, stream)
                                      : launch_ragged_fwd<ElemI8, MOE_EPI_NONE>(a, stream);
}

}  // namespace moe
