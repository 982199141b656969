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
// are compared.  Squares are added by fours in fp32 and the rest in 64 bits; rows whose squares or products leave
// the middle of fp32's range go through 64 bits once more, which no 16-bit value overflows.
//
// Bound by memory: a row is read once, held in registers between its sums and its outputs, and s, y, codes and scales are
// written from there.  8191 x 4096 with a residual to FP8 54 to 58 us, box by box (302 MB, 5.6 TB/s; 48 % of the issue slots are the vector
// unit's, and a large addition of two tensors runs at 6.3 TB/s); 801 x 2048 to int8 4.3 us, one row 2.2 us (from Python 9 to 10 and
// 11 to 13 us: the call's checks, outputs and launch).  The gradient of 8191 x 4096 with ds 48.5 + 4 us (268 MB, 5.5 TB/s).
#include <algorithm>

#include "launch.h"
#include "moe_common.h"
#include "moe_w4a16.h"

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
// f over values that repeat every N lanes (4, 8 or 16): what the waves of a workgroup left, one lane each.
template <int N, class F>
__device__ __forceinline__ double first_lanes_f64(double v, F f) {
  v = f(v, dpp_f64<0xB1>(v));
  v = f(v, dpp_f64<0x4E>(v));
  if (N > 4) v = f(v, dpp_f64<0x141>(v));
  return N > 8 ? f(v, dpp_f64<0x140>(v)) : v;
}
template <int N>
__device__ __forceinline__ uint32_t first_lanes_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));
  if (N > 4) v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));
  return N > 8 ? max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true)) : v;
}

// The largest value of each row of 16 lanes, and of the wave.
__device__ __forceinline__ uint32_t row16_max_u32(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true));
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = row16_max_u32(v);
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(b[0], b[1]);
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
__device__ __forceinline__ float norm_code_i8(double z, double zmax, double inv) {
  const float v = (float)(z * inv);
  float n = rintf(v);
  if (__builtin_expect(fabsf(v - n) == 0.5f, 0)) {
    const double border = (double)v, d = 127.0 * z - border * zmax;  // both products exact
    if (d > 0.0) n = v + 0.5f;
    if (d < 0.0) n = v - 0.5f;
  }
  return fminf(fmaxf(n, -127.f), 127.f);  // (a NaN, of a row that gets codes 0 anyway, becomes a number)
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

// Four squares added in fp32 (at most three roundings); all that these sums meet is added in 64 bits.
__device__ __forceinline__ float square4(const float* s) { return fmaf(s[3], s[3], fmaf(s[2], s[2], fmaf(s[1], s[1], s[0] * s[0]))); }

// A chunk's part of what a row's threads add up: the sum of s^2, and max |z|: with 16-bit weights as the bits of a float,
// which order like the values with infinities and NaN above all; with fp32 weights, whose products with s fp32 does not
// hold, as a double too.
template <bool F16, bool WF32, int QUANT>
__device__ __forceinline__ void norm_gather(const u32x4& sv, const u32x4 (&wv)[WF32 ? 2 : 1], double& ss, uint32_t& zbits, double& zmax) {
  float s[8], w[8];
  unpack8<F16>(sv, s);
  if (QUANT != kQuantNone) weight8<F16, WF32>(wv, w);
  float zabs = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (QUANT != kQuantNone) {
      zabs = __builtin_elementwise_maximum(zabs, fabsf(s[j] * w[j]));  // (a NaN stays)
      if (WF32) zmax = fmax(zmax, fabs((double)s[j] * (double)w[j]));
    }
  }
  zbits = __float_as_uint(zabs);
  ss += (double)square4(s) + (double)square4(s + 4);
}

// The same in 64 bits throughout, for rows whose squares or products leave the middle of fp32's range.  Returns whether z
// holds an infinity or a NaN.
template <bool F16, bool WF32, int QUANT>
__device__ __forceinline__ bool norm_gather_f64(const u32x4& sv, const u32x4 (&wv)[WF32 ? 2 : 1], double& ss, double& zmax) {
  float s[8], w[8];
  unpack8<F16>(sv, s);
  weight8<F16, WF32>(wv, w);
  double bad = 0.0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const double z = (double)s[j] * (double)w[j];
    ss = fma((double)s[j], (double)s[j], ss);
    if (QUANT != kQuantNone) zmax = fmax(zmax, fabs(z));
    bad = fma(z, 0.0, bad);
  }
  return QUANT != kQuantNone && !(bad == 0.0);
}

// Eight codes of z = s w where the largest magnitude is zmax; some false: codes 0.  fast: zmax lies in the middle of fp32's
// range, and zv holds z in fp32.  Then the codes are formed from two quotients a little below and above the true one (z, the
// reciprocal and the factor are off by less than 2^-21.7); where both give the same code, that is it, and only where some
// element's do not, within 2^-21 of a border, are the eight formed in 64 bits.
template <int QUANT>
__device__ __forceinline__ u32x2 norm_codes8(const float (&s)[8], const float (&w)[8], const float (&zv)[8], double zmax, bool some,
                                             bool fast) {
  constexpr float kTop = QUANT == kQuantI8 ? 127.f : 448.f;
  u32x2 c = {0u, 0u};
  bool close = !fast;
  if (fast) {
    const float f = kTop * __builtin_amdgcn_rcpf((float)zmax);
    const float below = f * (1.0f - 0x1p-21f), above = f * (1.0f + 0x1p-21f);
    uint32_t differ = 0u;
    if constexpr (QUANT == kQuantI8) {
      constexpr float kInt = 0x1.8p23f;  // a sum with it is an integer, rounded to nearest even, in the low bits
      uint32_t n[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        n[j] = __float_as_uint(fmaf(zv[j], below, kInt));
        differ |= n[j] ^ __float_as_uint(fmaf(zv[j], above, kInt));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __builtin_amdgcn_perm(n[4 * i + 1], n[4 * i], 0x0C0C0400u);
        const uint32_t hi = __builtin_amdgcn_perm(n[4 * i + 3], n[4 * i + 2], 0x04000C0Cu);
        c[i] = lo | hi;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float* z = zv + 4 * i;
        int a = __builtin_amdgcn_cvt_pk_fp8_f32(z[0] * below, z[1] * below, 0, false);
        a = __builtin_amdgcn_cvt_pk_fp8_f32(z[2] * below, z[3] * below, a, true);
        int b = __builtin_amdgcn_cvt_pk_fp8_f32(z[0] * above, z[1] * above, 0, false);
        b = __builtin_amdgcn_cvt_pk_fp8_f32(z[2] * above, z[3] * above, b, true);
        c[i] = (uint32_t)a;
        differ |= (uint32_t)(a ^ b);
      }
    }
    close = differ != 0u;
  }
  if (__builtin_expect(close, 0)) {
    const double inv = (double)kTop * recip_f64(zmax);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double z = (double)s[j] * (double)w[j];
      v[j] = QUANT == kQuantI8 ? norm_code_i8(z, zmax, inv) : norm_quotient_f8(z, zmax, inv);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (QUANT == kQuantI8) {
        c[i] = 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) c[i] |= ((uint32_t)(int)v[4 * i + j] & 0xFFu) << (8 * j);
      } else {
        const int b = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], 0, false);
        c[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2], v[4 * i + 3], b, true);
      }
    }
  }
  return some ? c : u32x2{0u, 0u};
}

// A chunk's outputs.  All stores of this kernel go past the L2, which they would only clear of rows to be read (to FP8 with a
// residual: 5000 x 4096 36.8 us against 39.7, 4096 x 2048 14.5 against 16.1, 8191 x 4096 58.1 against 59.9; 801 x 2048 to int8 4.5 both ways).
template <bool F16, bool WF32, int QUANT>
__device__ __forceinline__ void norm_store(const NormArgs& p, const u32x4& sv, const u32x4 (&wv)[WF32 ? 2 : 1], float r,
                                           double zmax, bool some, bool quick, size_t at) {
  float s[8], w[8];
  unpack8<F16>(sv, s);
  weight8<F16, WF32>(wv, w);
  if (p.y) {  // (s r) w: s w may leave the range of fp32 where y does not; the same whatever codes stand beside it
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = s[j] * r * w[j];
    store16<1>(pack8<F16>(y), static_cast<u32x4*>(p.y) + at);
  }
  if constexpr (QUANT != kQuantNone) {
    float z[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = s[j] * w[j];
    __builtin_nontemporal_store(norm_codes8<QUANT>(s, w, z, zmax, some, quick), static_cast<u32x2*>(p.q) + at);
  }
}

// TH threads a row (64: a wave, four rows a workgroup), NC chunks of 8 columns a thread, held between the sums and the
// outputs.
template <bool F16, bool WF32, int QUANT, int TH, int NC>
__global__ __launch_bounds__(TH < 256 ? 256 : TH) void rmsnorm_kernel(NormArgs p) {
  constexpr int kRows = TH < 256 ? 256 / TH : 1, kWaves = TH / 64;
  static_assert(TH >= 256 || TH == 64, "whole waves, or one, a row");
  __shared__ double part_ss[2][kWaves], part_z[2][kWaves];
  __shared__ uint32_t part_bits[2][kWaves];
  const int t = threadIdx.x % TH, wave = t >> 6, lane = t & 63;
  const long long row = linear_block() * kRows + threadIdx.x / TH;
  if (row >= p.T) return;  // of all threads of a row, and of a workgroup that meets at a barrier
  const int nc = p.H / 8;
  const size_t base = (size_t)row * nc;
  u32x4 sv[NC], wv[NC][WF32 ? 2 : 1];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = t + j * TH;
    if (c < nc) {
      sv[j] = sum8<F16>(p, base + c);
      load_weight8<WF32>(p.w, c, wv[j]);
    }
  }
  // the row's sums over its threads; bits: the largest of what the threads say, 0x7F800000 and above for infinities and NaN
  auto meet = [&](int turn, double& ss, double& zmax, uint32_t& bits) {
    ss = wave_f64(ss, AddF64{});
    if (QUANT == kQuantI8 && (WF32 || turn)) zmax = wave_f64(zmax, MaxF64{});
    if (QUANT != kQuantNone) bits = wave_max_u32(bits);
    if constexpr (TH > 64) {
      if (lane == 0) {
        part_ss[turn][wave] = ss;
        if (QUANT == kQuantI8 && (WF32 || turn)) part_z[turn][wave] = zmax;
        if (QUANT != kQuantNone) part_bits[turn][wave] = bits;
      }
      __syncthreads();
      const int k = lane & (kWaves - 1);
      ss = first_lanes_f64<kWaves>(part_ss[turn][k], AddF64{});
      if (QUANT == kQuantI8 && (WF32 || turn)) zmax = first_lanes_f64<kWaves>(part_z[turn][k], MaxF64{});
      if (QUANT != kQuantNone) bits = first_lanes_max<kWaves>(part_bits[turn][k]);
    }
  };
  double ss = 0.0;
  uint32_t bits = 0u;
  double zmax = 0.0, blk[NC];
  uint32_t blk_bits[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = t + j * TH;
    blk[j] = 0.0;
    blk_bits[j] = 0u;
    if (c < nc) {
      if (p.residual) store16<1>(sv[j], static_cast<u32x4*>(p.s) + base + c);
      norm_gather<F16, WF32, QUANT>(sv[j], wv[j], ss, blk_bits[j], blk[j]);
    }
    bits = max(bits, blk_bits[j]);
    if (WF32) zmax = fmax(zmax, blk[j]);
  }
  meet(0, ss, zmax, bits);
  // rows whose squares fp32 cannot add, or whose products or their quotients it cannot hold: once more in 64 bits (rows of
  // zeros too: they may be products that fp32 let vanish)
  const bool sums = ss < 1e36 && (ss > 1e-25 || p.eps > 1e-15f);
  bool fast = sums;
  if (QUANT != kQuantNone) fast = fast && bits >= 0x21800000u && bits < 0x7B800000u;  // 2^-60 and 2^120
  if (QUANT == kQuantI8 && !WF32) zmax = (double)__uint_as_float(bits);
  bool bad = false;
  if (!fast) {
    const double first = ss;
    ss = zmax = 0.0;
    bits = 0u;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      blk[j] = 0.0;
      if (t + j * TH < nc && norm_gather_f64<F16, WF32, QUANT>(sv[j], wv[j], ss, blk[j])) bits = 0x7F800000u;
      zmax = fmax(zmax, blk[j]);
    }
    meet(1, ss, zmax, bits);
    bad = bits >= 0x7F800000u || !(ss < __builtin_inf());
    if (sums) ss = first;  // what the row has without codes, for the same y
  }
  const double rd = rsqrt_f64(fma(ss, p.inv_h, (double)p.eps));
  const float r = (float)rd;
  // scales by r / top, rounded once; where one is 0 or NaN its codes are 0
  const double rtop = rd * (QUANT == kQuantI8 ? 1.0 / 127.0 : 1.0 / 448.0);
  auto scale_of = [&](double m) { return bad ? __uint_as_float(0x7FC00000u) : (float)(m * rtop); };
  float scale = 0.f;
  if constexpr (QUANT == kQuantI8) {
    scale = scale_of(zmax);
    if (t == 0) p.q_scale[row] = scale;
  }
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = t + j * TH;
    if (c < nc) {
      bool quick = fast;
      if constexpr (QUANT == kQuantF8) {  // the 16 lanes of a block of 128 columns are within H together
        if (!WF32 && fast) {
          zmax = (double)__uint_as_float(row16_max_u32(blk_bits[j]));
          if (zmax < 0x1p-60) {  // a block may be far smaller than its row, down to products that fp32 does not hold
            double unused = 0.0, m = 0.0;
            norm_gather_f64<F16, WF32, QUANT>(sv[j], wv[j], unused, m);
            zmax = row16_f64(m, MaxF64{});
          }
        } else {
          zmax = row16_f64(blk[j], MaxF64{});
        }
        scale = scale_of(zmax);
        if ((lane & 15) == 0) p.q_scale[(size_t)row * (nc / 16) + c / 16] = scale;
        quick = fast && zmax >= 0x1p-60;
      }
      norm_store<F16, WF32, QUANT>(p, sv[j], wv[j], r, zmax, scale > 0.f, quick, base + c);
    }
  }
}

template <bool F16, bool WF32, int QUANT>
static hipError_t launch_norm_of(const NormArgs& p, hipStream_t s) {
  // Threads a row so that few are idle and few barriers join them.  Up to 512 columns a wave holds a row; up to 1024 two waves'
  // worth, where there are rows enough for all CUs (4985 x 768 to int8 7.1 us, a workgroup a row 9.6; 4096 x 1024 to FP8 9.6 and
  // 11.1; of 16 to 64 rows 3.3 to 3.8 and 2.9 to 3.2).  Beyond that a workgroup a row: four chunks a wave are slower (801 x 2048
  // 5.4 us against 4.5, 4096 x 2048 9.4 against 7.7), and so are 512 threads up to 4096 columns (4096 x 2048 to FP8 17.7 against
  // 15.1) and 1024 up to 8192 (2000 x 8192 to FP8 29.2 against 24.7).
  const dim3 grid = grid2d(p.T), grid4 = grid2d(((long long)p.T + 3) / 4);
  if (p.H > 512 && p.H <= 1024 && p.T >= 2048) rmsnorm_kernel<F16, WF32, QUANT, 64, 2><<<grid4, 256, 0, s>>>(p);
  else if (p.H <= 512) rmsnorm_kernel<F16, WF32, QUANT, 64, 1><<<grid4, 256, 0, s>>>(p);
  else if (p.H <= 2048) rmsnorm_kernel<F16, WF32, QUANT, 256, 1><<<grid, 256, 0, s>>>(p);
  else if (p.H <= 4096) rmsnorm_kernel<F16, WF32, QUANT, 256, 2><<<grid, 256, 0, s>>>(p);
  else if (p.H <= 8192) rmsnorm_kernel<F16, WF32, QUANT, 512, 2><<<grid, 512, 0, s>>>(p);
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
// meet.  The workgroups' sums of rows go to the workspace and are added in the order of the workgroups.  Rows past 4096 columns are
// farther from their bytes: one workgroup of 1024 threads a CU, with threads that have no columns, and a barrier a row (2023 x 5192
// 24 us, its bytes 16; 2048 x 16384 90 us, 52; 4096 x 8192 57 us, 52).
// TH threads a row (64: a wave, four rows a workgroup, whose sums meet in LDS before they are written).
// A sum in fp32 takes at most kGradRows rows; then it is a part of its own, and the parts are added in 64 bits (100000 x 8192 1211 us,
// 1196 with one part a workgroup; twice the workgroups instead, of half the rows each, do not walk the rows side by side: 1253).
constexpr int kGradRows = 256;
template <bool F16, bool WF32, int TH, int NC>
__global__ __launch_bounds__(TH < 256 ? 256 : TH) void rmsnorm_grad_kernel(NormGradArgs p) {
  constexpr int kWaves = TH / 64, kRows = TH < 256 ? 256 / TH : 1;
  constexpr bool kAhead = NC == 1;  // with two chunks a thread a second row would not fit the registers of 1024 threads
  __shared__ double part[2][kWaves][2];
  const int t = threadIdx.x % TH, sub = threadIdx.x / TH, wave = t >> 6, lane = t & 63;
  const int nc = p.H / 8, step = gridDim.x * kRows;
  u32x4 wv[NC][WF32 ? 2 : 1], sv[NC], gv[NC], av[NC];
  float dw[NC][8];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = t + j * TH;
    if (c < nc) load_weight8<WF32>(p.w, c, wv[j]);
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
  long long row = (long long)blockIdx.x * kRows + sub;
  if (kAhead && row < p.T) load(row);
  for (int round = 0; round < p.rounds; ++round) {
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) dw[j][i] = 0.f;
    for (int left = kGradRows; left > 0 && row < p.T; --left, row += step, turn ^= 1) {
      double ss = 0.0, gs = 0.0;
      u32x4 s8[NC], g8[NC], a8[NC];
      if (!kAhead) load(row);
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        s8[j] = sv[j];
        g8[j] = gv[j];
        a8[j] = av[j];
      }
      if (kAhead && row + step < p.T) load(row + step);
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
          // past the L2 (8191 x 4096 48.5 us against 51.3, 8192 x 2048 28.6 both ways)
          store16<1>(pack8<F16>(o), static_cast<u32x4*>(p.dx) + base + c);
        }
      }
    }
    if constexpr (kRows > 1) {
      __shared__ f32x4 more[kRows - 1][TH * NC * 2];
      static_assert(NC == 1, "a thread's sums stand 16 bytes apart from its neighbour's");
      f32x4* mine = more[sub > 0 ? sub - 1 : 0];
      if (round > 0) __syncthreads();  // the last round's have been read
      if (sub > 0) {
        mine[t] = f32x4{dw[0][0], dw[0][1], dw[0][2], dw[0][3]};
        mine[TH + t] = f32x4{dw[0][4], dw[0][5], dw[0][6], dw[0][7]};
      }
      __syncthreads();
      if (sub == 0) {
#pragma unroll
        for (int r = 0; r < kRows - 1; ++r) {
          const f32x4* other = more[r];
#pragma unroll
          for (int i = 0; i < 8; ++i) dw[0][i] += other[(i >> 2) * TH + t][i & 3];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = t + j * TH;
      if (sub == 0 && c < nc) {
        f32x4* dst = reinterpret_cast<f32x4*>(p.parts + ((size_t)round * gridDim.x + blockIdx.x) * p.H) + 2 * (size_t)c;
        dst[0] = f32x4{dw[j][0], dw[j][1], dw[j][2], dw[j][3]};
        dst[1] = f32x4{dw[j][4], dw[j][5], dw[j][6], dw[j][7]};
      }
    }
  }
}

// dw = the sum of n rows of parts [n, H]: 32 columns a workgroup, the rows dealt to 128 groups of 8 threads, four columns a
// thread, whose sums (64 bits) are added in order.
__global__ __launch_bounds__(1024) void rmsnorm_dw_kernel(const float* __restrict__ parts, int n, int H, int out, void* __restrict__ dw) {
  __shared__ double sums[128][33];
  const int l = threadIdx.x & 7, g = threadIdx.x >> 3, c = blockIdx.x * 32 + 4 * l;
  double a[4] = {0.0, 0.0, 0.0, 0.0};
  if (c < H) {
#pragma unroll 4
    for (int i = g; i < n; i += 128) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(parts + (size_t)i * H + c);
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] += (double)v[j];
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) sums[g][4 * l + j] = a[j];
  __syncthreads();
  // 32 threads a column take four sums each, then one thread their sums
  const int col = threadIdx.x >> 5, k = threadIdx.x & 31;
  double v = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) v += sums[4 * k + i][col];
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  const int at = blockIdx.x * 32 + col;
  if (k != 0 || at >= H) return;
  const float r = (float)v;
  if (out == MOE_OUT_F32) static_cast<float*>(dw)[at] = r;
  else static_cast<uint16_t*>(dw)[at] = out == MOE_OUT_F16 ? f32_to_f16_bits(r) : f32_to_bf16_bits(r);
}

// Threads a row of the gradient's workgroups: one chunk of 8 columns each (8192 x 512: a wave a row 10.1 us, 256 threads 13.0; 8192 x
// 2048: 256 threads 27.5, 512 27.9, 1024 34.4; 8191 x 4096: 512 threads 50.6, 256 of two chunks 55.7, 1024 57.1; 4096 x 8192: 1024
// threads 51.1, 512 of two chunks 54.2).  Workgroups: as many as the card holds at once, so that few parts are left to add.
static int grad_threads(int H) { return H <= 512 ? 64 : (H <= 2048 ? 256 : (H <= 4096 ? 512 : 1024)); }

struct GradGrid {
  int workgroups, rounds;  // rounds: of kGradRows rows a workgroup's row
};
static GradGrid grad_grid(int T, int H) {
  const int th = grad_threads(H), rows = th < 256 ? 256 / th : 1, most = 1024 / std::max(1, th / 256);
  return {std::min((T + rows - 1) / rows, most), std::max(1, (T + kGradRows * rows * most - 1) / (kGradRows * rows * most))};
}
int rmsnorm_grad_parts(int T, int H) {
  const GradGrid g = grad_grid(T, H);
  return g.workgroups * g.rounds;
}

template <bool F16, bool WF32>
static hipError_t launch_norm_grad_of(NormGradArgs p, hipStream_t s) {
  const GradGrid g = grad_grid(p.T, p.H);
  const int n = g.workgroups;
  p.rounds = g.rounds;
  if (p.T == 0) {
  } else if (p.H <= 512) rmsnorm_grad_kernel<F16, WF32, 64, 1><<<n, 256, 0, s>>>(p);
  else if (p.H <= 2048) rmsnorm_grad_kernel<F16, WF32, 256, 1><<<n, 256, 0, s>>>(p);
  else if (p.H <= 4096) rmsnorm_grad_kernel<F16, WF32, 512, 1><<<n, 512, 0, s>>>(p);
  else if (p.H <= 8192) rmsnorm_grad_kernel<F16, WF32, 1024, 1><<<n, 1024, 0, s>>>(p);
  else rmsnorm_grad_kernel<F16, WF32, 1024, 2><<<n, 1024, 0, s>>>(p);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  rmsnorm_dw_kernel<<<(p.H + 31) / 32, 1024, 0, s>>>(p.parts, n * g.rounds, p.H, p.dw_out, p.dw);
  return hipGetLastError();
}

hipError_t launch_rmsnorm_grad(const NormGradArgs& p, bool f16, bool w_f32, hipStream_t stream) {
  if (f16) return w_f32 ? launch_norm_grad_of<true, true>(p, stream) : launch_norm_grad_of<true, false>(p, stream);
  return w_f32 ? launch_norm_grad_of<false, true>(p, stream) : launch_norm_grad_of<false, false>(p, stream);
}

}  // namespace moe
