// Root-mean-square norm with the residual's addition, its 8-bit outputs, and its gradient: what stands in front of a block
// of experts.  The ATOM page ("AMD ATOM推理引擎：如何用分页KV缓存和分段编译实现大模型推理性能翻倍"), section "8.2 量化
// 并非单一格式，而是一套执行契约", makes dynamic activation quantization part of a format's contract; here the rows are
// quantized where they are formed, so that the products by expert read codes and the router 16 bits of one pass.
//
//   s = x + residual (fp32, rounded to the 16-bit type; s = x without a residual)
//   r = 1 / sqrt(mean(s^2) + eps),  y = s r w
//   codes of z = s w, top / max |z| to a row (int8, top 127) or to 128 columns (FP8 E4M3, top 448):
//     code = the integer, or E4M3 value, nearest to the real quotient top z / max |z|, ties to even
//     scale = max |z| r / top, rounded to fp32 once
// The codes do not depend on r, nor on the order in which anything is added: z is exact in 64 bits (at most 24 + 11
// significant bits), and of a quotient next to a border between two codes the exact products top z and border max |z|
// are compared.  Squares are added in 64 bits, which no 16-bit value overflows.  The 64-bit operations stand beside about
// 7 bytes of traffic an element and hide behind it.
#include "launch.h"
#include "moe_common.h"

#include "../../include/moe_w4a16.h"

namespace moe {

template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  const u32x2 b = __builtin_bit_cast(u32x2, v);
  const u32x2 m = {(uint32_t)__builtin_amdgcn_mov_dpp((int)b[0], CTRL, 0xF, 0xF, true),
                   (uint32_t)__builtin_amdgcn_mov_dpp((int)b[1], CTRL, 0xF, 0xF, true)};
  return __builtin_bit_cast(double, m);
}

// The two halves (rows of 16 lanes, or of 32) of v exchanged and combined: every lane then holds f of both.
template <bool HALF, class F>
__device__ __forceinline__ double swap_f64(double v, F f) {
  const u32x2 b = __builtin_bit_cast(u32x2, v);
  u32x2 lo, hi;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (HALF) {
      const auto p = __builtin_amdgcn_permlane32_swap(b[i], b[i], false, false);
      lo[i] = p[0];
      hi[i] = p[1];
    } else {
      const auto p = __builtin_amdgcn_permlane16_swap(b[i], b[i], false, false);
      lo[i] = p[0];
      hi[i] = p[1];
    }
  }
  return f(__builtin_bit_cast(double, lo), __builtin_bit_cast(double, hi));
}

// f over the 16 lanes of each row (quad swaps, half-row mirror, row mirror), then over the wave.
template <class F>
__device__ __forceinline__ double row16_f64(double v, F f) {
  v = f(v, dpp_f64<0xB1>(v));
  v = f(v, dpp_f64<0x4E>(v));
  v = f(v, dpp_f64<0x141>(v));
  return f(v, dpp_f64<0x140>(v));
}
template <class F>
__device__ __forceinline__ double wave_f64(double v, F f) {
  v = row16_f64(v, f);
  v = swap_f64<false>(v, f);
  return swap_f64<true>(v, f);
}
struct AddF64 {
  __device__ __forceinline__ double operator()(double a, double b) const { return a + b; }
};
struct MaxF64 {
  __device__ __forceinline__ double operator()(double a, double b) const { return fmax(a, b); }
};

// 1 / sqrt(v) and 1 / v from the hardware's estimates (about 2^-24) by Newton's iteration: 2^-46 or better.
__device__ __forceinline__ double rsqrt_f64(double v) {
  double r = __builtin_amdgcn_rsq(v);
  if (v > 0.0 && v < __builtin_inf()) r = r * (1.5 - 0.5 * v * r * r);  // 0 and infinity keep their limits
  return r;
}
__device__ __forceinline__ double recip_f64(double v) {
  const double r = __builtin_amdgcn_rcp(v);
  return r * (2.0 - v * r);
}

// The code of z where the largest magnitude is zmax, inv = 127 / zmax to 2^-45: a quotient that rounds to a border in
// fp32 may lie on either side of it; all others lie on fp32's side.
__device__ __forceinline__ int norm_code_i8(double z, double zmax, double inv) {
  const float v = (float)(z * inv);
  float n = rintf(v);
  if (__builtin_expect(fabsf(v - n) == 0.5f, 0)) {
    const double border = (double)v, d = 127.0 * z - border * zmax;  // both products exact
    if (d > 0.0) n = v + 0.5f;
    if (d < 0.0) n = v - 0.5f;
  }
  return (int)fminf(fmaxf(n, -127.f), 127.f);  // (a NaN, of a row that gets codes 0 anyway, becomes a number)
}

// fp32 whose E4M3 rounding (nearest, ties to even) is that of the real quotient 448 z / zmax, inv = 448 / zmax to 2^-45.
// Borders have five significant bits; below 2^-6 they are the odd multiples of 2^-10.
__device__ __forceinline__ float norm_quotient_f8(double z, double zmax, double inv) {
  float v = (float)(z * inv);
  const uint32_t b = __float_as_uint(v);
  if (__builtin_expect((b & 0xFFFFFu) == 0x80000u || (b & 0x7FFFFFFFu) < 0x3C800000u, 0)) {
    const float f = fabsf(v) * 1024.0f;
    const bool border = fabsf(v) < 0x1p-6f ? (f == rintf(f) && ((int)f & 1)) : true;
    const double d = 448.0 * z - (double)v * zmax;  // both products exact where v is a border
    if (border && d != 0.0) v = __uint_as_float((d > 0.0) == (v > 0.0f) ? b + 1 : b - 1);
  }
  return v;
}

template <bool WF32>
__device__ __forceinline__ void load_weight8(const void* w, int c, u32x4 (&raw)[WF32 ? 2 : 1]) {
  const u32x4* p = static_cast<const u32x4*>(w) + (size_t)c * (WF32 ? 2 : 1);
  raw[0] = p[0];
  if constexpr (WF32) raw[1] = p[1];
}
template <bool F16, bool WF32>
__device__ __forceinline__ void weight8(const u32x4 (&raw)[WF32 ? 2 : 1], float (&w)[8]) {
  if constexpr (WF32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = __uint_as_float(raw[0][i]);
      w[4 + i] = __uint_as_float(raw[1][i]);
    }
  } else {
    unpack8<F16>(raw[0], w);
  }
}

constexpr int kQuantNone = MOE_QUANT_NONE, kQuantI8 = MOE_QUANT_I8, kQuantF8 = MOE_QUANT_F8;

// s of chunk c (8 columns) of a row: x, or x + residual rounded to the type.
template <bool F16>
__device__ __forceinline__ u32x4 sum8(const NormArgs& p, size_t at) {
  u32x4 v = static_cast<const u32x4*>(p.x)[at];
  if (p.residual) {
    float a[8], b[8];
    unpack8<F16>(v, a);
    unpack8<F16>(static_cast<const u32x4*>(p.residual)[at], b);
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] += b[j];
    v = pack8<F16>(a);
  }
  return v;
}

// A chunk's part of the row's sums.
struct NormSums {
  double ss;    // sum of s^2
  double zmax;  // max |z| (int8)
  double bad;   // 0, or NaN where z holds an infinity or a NaN
};
template <bool F16, bool WF32, int QUANT>
__device__ __forceinline__ double norm_gather(const u32x4& sv, const u32x4 (&wv)[WF32 ? 2 : 1], NormSums& n) {
  float s[8], w[8];
  unpack8<F16>(sv, s);
  if (QUANT != kQuantNone) weight8<F16, WF32>(wv, w);
  double m = 0.0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    n.ss = fma((double)s[j], (double)s[j], n.ss);
    if (QUANT != kQuantNone) {
      const double z = (double)s[j] * (double)w[j];
      m = fmax(m, fabs(z));
      n.bad = fma(z, 0.0, n.bad);
    }
  }
  return m;
}

// A chunk's outputs.
template <bool F16, bool WF32, int QUANT>
__device__ __forceinline__ void norm_store(const NormArgs& p, const u32x4& sv, const u32x4 (&wv)[WF32 ? 2 : 1], float r,
                                           double zmax, double inv, size_t at) {
  float s[8], w[8];
  unpack8<F16>(sv, s);
  weight8<F16, WF32>(wv, w);
  if (p.y) {
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = s[j] * r * w[j];
    static_cast<u32x4*>(p.y)[at] = pack8<F16>(y);
  }
  if constexpr (QUANT == kQuantI8) {
    u32x2 c = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      c[j >> 2] |= (uint32_t)(norm_code_i8((double)s[j] * (double)w[j], zmax, inv) & 0xFF) << (8 * (j & 3));
    static_cast<u32x2*>(p.q)[at] = inv > 0.0 ? c : u32x2{0u, 0u};
  }
  if constexpr (QUANT == kQuantF8) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = norm_quotient_f8((double)s[j] * (double)w[j], zmax, inv);
    u32x2 c;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int b = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], 0, false);
      c[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2], v[4 * i + 3], b, true);
    }
    static_cast<u32x2*>(p.q)[at] = inv > 0.0 ? c : u32x2{0u, 0u};
  }
}

// The scale of codes whose largest magnitude is zmax, and what z is multiplied by: 0 (codes 0) where the scale is 0 or NaN.
__device__ __forceinline__ float norm_scale(double zmax, double r, double top, bool bad, double& inv) {
  const float scale = bad ? __uint_as_float(0x7FC00000u) : (float)(zmax * r * (1.0 / top));
  inv = scale > 0.0f ? top * recip_f64(zmax) : 0.0;
  return scale;
}

// TH threads a row (64: a wave, four rows a workgroup), NC chunks of 8 columns a thread, held between the sums and the
// outputs.
template <bool F16, bool WF32, int QUANT, int TH, int NC>
__global__ __launch_bounds__(TH < 256 ? 256 : TH) void rmsnorm_kernel(NormArgs p) {
  constexpr int kRows = TH < 256 ? 256 / TH : 1, kWaves = TH / 64;
  static_assert(TH >= 256 || TH == 64, "whole waves, or one, a row");
  __shared__ double part_ss[kWaves], part_z[kWaves];
  __shared__ int part_bad[kWaves];
  const int t = threadIdx.x % TH, wave = t >> 6, lane = t & 63;
  const long long row = linear_block() * kRows + threadIdx.x / TH;
  if (row >= p.T) return;  // of all threads of a row, and of a workgroup that meets at a barrier
  const int nc = p.H / 8;
  const size_t base = (size_t)row * nc;
  u32x4 sv[NC], wv[NC][WF32 ? 2 : 1];
  double blk[NC];
  NormSums n = {0.0, 0.0, 0.0};
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = t + j * TH;
    if (c < nc) {
      sv[j] = sum8<F16>(p, base + c);
      load_weight8<WF32>(p.w, c, wv[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = t + j * TH;
    blk[j] = 0.0;
    if (c < nc) {
      if (p.residual) static_cast<u32x4*>(p.s)[base + c] = sv[j];
      blk[j] = norm_gather<F16, WF32, QUANT>(sv[j], wv[j], n);
    }
    if (QUANT == kQuantI8) n.zmax = fmax(n.zmax, blk[j]);
  }
  n.ss = wave_f64(n.ss, AddF64{});
  if (QUANT == kQuantI8) n.zmax = wave_f64(n.zmax, MaxF64{});
  bool bad = QUANT != kQuantNone && __ballot(!(n.bad == 0.0)) != 0ull;
  if constexpr (TH > 64) {
    if (lane == 0) {
      part_ss[wave] = n.ss;
      if (QUANT == kQuantI8) part_z[wave] = n.zmax;
      if (QUANT != kQuantNone) part_bad[wave] = bad;
    }
    __syncthreads();
    n.ss = 0.0;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) {
      n.ss += part_ss[k];
      if (QUANT == kQuantI8) n.zmax = fmax(n.zmax, part_z[k]);
      if (QUANT != kQuantNone) bad |= part_bad[k] != 0;
    }
  }
  bad |= !(n.ss < __builtin_inf());
  const double rd = rsqrt_f64(fma(n.ss, p.inv_h, (double)p.eps));
  const float r = (float)rd;
  double inv = 0.0;
  if constexpr (QUANT == kQuantI8) {
    const float scale = norm_scale(n.zmax, rd, 127.0, bad, inv);
    if (t == 0) p.q_scale[row] = scale;
  }
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = t + j * TH;
    if (c < nc) {
      double zmax = n.zmax;
      if constexpr (QUANT == kQuantF8) {  // the 16 lanes of a block of 128 columns are within H together
        zmax = row16_f64(blk[j], MaxF64{});
        const float scale = norm_scale(zmax, rd, 448.0, bad, inv);
        if ((lane & 15) == 0) p.q_scale[(size_t)row * (nc / 16) + c / 16] = scale;
      }
      norm_store<F16, WF32, QUANT>(p, sv[j], wv[j], r, zmax, inv, base + c);
    }
  }
}

template <bool F16, bool WF32, int QUANT>
static hipError_t launch_norm_of(const NormArgs& p, hipStream_t s) {
  const dim3 grid = grid2d(p.T), grid4 = grid2d(((long long)p.T + 3) / 4);
  if (p.H <= 512) rmsnorm_kernel<F16, WF32, QUANT, 64, 1><<<grid4, 256, 0, s>>>(p);
  else if (p.H <= 2048) rmsnorm_kernel<F16, WF32, QUANT, 256, 1><<<grid, 256, 0, s>>>(p);
  else if (p.H <= 4096) rmsnorm_kernel<F16, WF32, QUANT, 256, 2><<<grid, 256, 0, s>>>(p);
  else if (p.H <= 8192) rmsnorm_kernel<F16, WF32, QUANT, 1024, 1><<<grid, 1024, 0, s>>>(p);
  else rmsnorm_kernel<F16, WF32, QUANT, 1024, 2><<<grid, 1024, 0, s>>>(p);
  return hipGetLastError();
}

template <bool F16, bool WF32>
static hipError_t launch_norm_quant(const NormArgs& p, int quant, hipStream_t s) {
  if (quant == kQuantI8) return launch_norm_of<F16, WF32, kQuantI8>(p, s);
  if (quant == kQuantF8) return launch_norm_of<F16, WF32, kQuantF8>(p, s);
  return launch_norm_of<F16, WF32, kQuantNone>(p, s);
}

hipError_t launch_rmsnorm(const NormArgs& p, bool f16, bool w_f32, int quant, hipStream_t stream) {
  if (f16) return w_f32 ? launch_norm_quant<true, true>(p, quant, stream) : launch_norm_quant<true, false>(p, quant, stream);
  return w_f32 ? launch_norm_quant<false, true>(p, quant, stream) : launch_norm_quant<false, false>(p, quant, stream);
}

// ---------------------------------------------------------------------------------------------------
// The gradient.  With xhat = s r and g = dy w:
//   dx = r g - xhat (r^2 mean(g s)) (+ ds),   dw = sum over the rows of dy xhat.
// r is formed again from s, which has to be read anyway.  A workgroup takes every nwg-th row, a thread the same columns of
// each, so that the weight's gradient stays in its registers; the next row is asked for before the current one's sums
// meet.  The workgroups' sums of rows go to the workspace and are added in the order of the workgroups.
template <bool F16, bool WF32, int TH, int NC>
__global__ __launch_bounds__(TH) void rmsnorm_grad_kernel(NormGradArgs p) {
  constexpr int kWaves = TH / 64;
  __shared__ double part[2][kWaves][2];
  const int t = threadIdx.x, wave = t >> 6, lane = t & 63;
  const int nc = p.H / 8, nwg = gridDim.x;
  u32x4 wv[NC][WF32 ? 2 : 1], sv[NC], gv[NC], av[NC];
  float dw[NC][8];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = t + j * TH;
    if (c < nc) load_weight8<WF32>(p.w, c, wv[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0.f;
  }
  auto load = [&](long long row) {
    const size_t base = (size_t)row * nc;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = t + j * TH;
      if (c < nc) {
        sv[j] = static_cast<const u32x4*>(p.s)[base + c];
        gv[j] = static_cast<const u32x4*>(p.dy)[base + c];
        if (p.ds) av[j] = static_cast<const u32x4*>(p.ds)[base + c];
      }
    }
  };
  int turn = 0;
  load(blockIdx.x);
  for (long long row = blockIdx.x; row < p.T; row += nwg, turn ^= 1) {
    double ss = 0.0, gs = 0.0;
    u32x4 s8[NC], g8[NC], a8[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      s8[j] = sv[j];
      g8[j] = gv[j];
      a8[j] = av[j];
    }
    if (row + nwg < p.T) load(row + nwg);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      if (t + j * TH < nc) {
        float s[8], d[8], w[8];
        unpack8<F16>(s8[j], s);
        unpack8<F16>(g8[j], d);
        weight8<F16, WF32>(wv[j], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss = fma((double)s[i], (double)s[i], ss);
          gs = fma((double)(d[i] * w[i]), (double)s[i], gs);
        }
      }
    }
    ss = wave_f64(ss, AddF64{});
    gs = wave_f64(gs, AddF64{});
    if constexpr (kWaves > 1) {
      if (lane == 0) {
        part[turn][wave][0] = ss;
        part[turn][wave][1] = gs;
      }
      __syncthreads();  // one a row: a wave writes this half of part again only past the next row's barrier
      ss = gs = 0.0;
#pragma unroll
      for (int k = 0; k < kWaves; ++k) {
        ss += part[turn][k][0];
        gs += part[turn][k][1];
      }
    }
    const double rd = rsqrt_f64(fma(ss, p.inv_h, (double)p.eps));
    const float r = (float)rd, k = (float)(rd * rd * (gs * p.inv_h));
    const size_t base = (size_t)row * nc;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = t + j * TH;
      if (c < nc) {
        float s[8], d[8], w[8], a[8], o[8];
        unpack8<F16>(s8[j], s);
        unpack8<F16>(g8[j], d);
        weight8<F16, WF32>(wv[j], w);
        if (p.ds) unpack8<F16>(a8[j], a);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xhat = s[i] * r;
          o[i] = fmaf(-xhat, k, r * (d[i] * w[i]));
          if (p.ds) o[i] += a[i];
          dw[j][i] = fmaf(d[i], xhat, dw[j][i]);
        }
        static_cast<u32x4*>(p.dx)[base + c] = pack8<F16>(o);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = t + j * TH;
    if (c < nc) {
      f32x4* dst = reinterpret_cast<f32x4*>(p.parts + (size_t)blockIdx.x * p.H) + 2 * (size_t)c;
      dst[0] = f32x4{dw[j][0], dw[j][1], dw[j][2], dw[j][3]};
      dst[1] = f32x4{dw[j][4], dw[j][5], dw[j][6], dw[j][7]};
    }
  }
}

// dw = the sum of n rows of parts [n, H]: 16 columns a workgroup, the rows dealt to 16 threads a column in turn, whose
// sums (64 bits) are added in order.
__global__ __launch_bounds__(256) void rmsnorm_dw_kernel(const float* __restrict__ parts, int n, int H, int out, void* __restrict__ dw) {
  __shared__ double sums[16][17];
  const int l = threadIdx.x & 15, g = threadIdx.x >> 4, c = blockIdx.x * 16 + l;
  double a = 0.0;
  if (c < H)
    for (int i = g; i < n; i += 16) a += (double)parts[(size_t)i * H + c];
  sums[g][l] = a;
  __syncthreads();
  if (g != 0 || c >= H) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) a += sums[i][l];
  const float v = (float)a;
  if (out == MOE_OUT_F32) static_cast<float*>(dw)[c] = v;
  else static_cast<uint16_t*>(dw)[c] = out == MOE_OUT_F16 ? f32_to_f16_bits(v) : f32_to_bf16_bits(v);
}

// Threads a row of the gradient's workgroups, and the workgroups: 4096 waves at most, which hold the card's memory busy.
static int grad_threads(int H) { return H <= 512 ? 64 : (H <= 2048 ? 256 : (H <= 8192 ? 512 : 1024)); }

int rmsnorm_grad_parts(int T, int H) {
  const int most = 262144 / grad_threads(H);
  return T < most ? T : most;
}

template <bool F16, bool WF32>
static hipError_t launch_norm_grad_of(const NormGradArgs& p, hipStream_t s) {
  const int n = rmsnorm_grad_parts(p.T, p.H);
  if (p.T == 0) {
  } else if (p.H <= 512) rmsnorm_grad_kernel<F16, WF32, 64, 1><<<n, 64, 0, s>>>(p);
  else if (p.H <= 2048) rmsnorm_grad_kernel<F16, WF32, 256, 1><<<n, 256, 0, s>>>(p);
  else if (p.H <= 4096) rmsnorm_grad_kernel<F16, WF32, 512, 1><<<n, 512, 0, s>>>(p);
  else if (p.H <= 8192) rmsnorm_grad_kernel<F16, WF32, 512, 2><<<n, 512, 0, s>>>(p);
  else rmsnorm_grad_kernel<F16, WF32, 1024, 2><<<n, 1024, 0, s>>>(p);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  rmsnorm_dw_kernel<<<(p.H + 15) / 16, 256, 0, s>>>(p.parts, n, p.H, p.dw_out, p.dw);
  return hipGetLastError();
}

hipError_t launch_rmsnorm_grad(const NormGradArgs& p, bool f16, bool w_f32, hipStream_t stream) {
  if (f16) return w_f32 ? launch_norm_grad_of<true, true>(p, stream) : launch_norm_grad_of<true, false>(p, stream);
  return w_f32 ? launch_norm_grad_of<false, true>(p, stream) : launch_norm_grad_of<false, false>(p, stream);
}

}  // namespace moe
