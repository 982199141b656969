// Grouped products with 16-bit expert weights (bf16, fp16) and their gradients, and SiLU*mul of a stored
// gate_up result with its gradient: the training forms of the expert FFN, and its serving form where the
// weights are not quantized.  The products are ragged_gemm.h's kernel; the layer's order of work follows
// the ATOM page ("AMD ATOM推理引擎：如何用分页KV缓存和分段编译实现大模型推理性能翻倍"), section "8.1 MoE 路径：
// 路由、专家并行与 MORI 通信".
#include "ragged_gemm.h"

namespace moe {

// Tile choice of the gradients, by the mean rows of a group.  Measured (fp16, weights from HBM): row gradients of 256
// experts of 1024 x 2048 with 25 rows 195 us with 64 x 256 tiles, 206 us with 32 x 256, 226 us with 32 x 128; 64
// experts, mean 200: 97 us with 128 x 256 (two workgroups a CU) against 99 us with 256 x 256 and 109 with 64 x 256;
// mean 400: 143 against 159 and 181; mean 1024 (8 experts of 4096 x 14336): 1085 against 1010.  Below about 16 rows a
// group no one shape is best; 64 x 256 against 16 x 128, bf16, mean 7: 64 experts 52.8 against 52.9 us, 256 experts 186
// against 190, groups of 0 to 60 rows 47 against 52, but 128 experts of 1536 x 2048 156 against 139 and 14 of 2424 x 4528
// 76 against 57 (32 x 128 tiles, in the same order: 56, 190, 48, 147 and 55 us).
template <class T>
static hipError_t launch_dx(const RaggedArgs& a, hipStream_t s) {
  const long long mean = ((long long)a.R + a.E - 1) / a.E;
  if (mean > 512 && fills(a, 256, a.K, 256)) return launch_ragged_cfg<T, kDx, MOE_EPI_NONE, TileShape<256, 256, 2, 4, 64, 4>>(a, s);
  if (mean > 64 && fills(a, 128, a.K, 256))
    return launch_ragged_cfg<T, kDx, MOE_EPI_NONE, TileShape<128, 256, 1, 4, 64, 3>, TileShape<64, 256, 1, 4, 64, 3>>(a, s);
  if (fills(a, 64, a.K, 256)) return launch_ragged_cfg<T, kDx, MOE_EPI_NONE, TileShape<64, 256, 1, 4, 64, 2>>(a, s);
  return launch_ragged_cfg<T, kDx, MOE_EPI_NONE, TileShape<16, 128, 1, 4, 128, 4>>(a, s);
}

// Weight gradients (bf16) of 64 experts of 1024 x 2048, mean 100: 73 us with 256 x 128 tiles (two workgroups a CU), 73
// with 128 x 128, 81 with 256 x 256; mean 375: 130, 133, 139; 256 experts, mean 25: 231, 230, 258; mean 1024 (8 experts
// of 4096 x 14336, fp16, 32-bit results): 1239 against 1090 us with 256 x 256.  A few rows a group are all results:
// 256 x 128 against 128 x 128, mean 4: 256 experts 179 against 183 us, 128 of 1536 x 2048 137 against 140, 14 of 2424 x
// 4528 80 against 72; with 32-bit results 324 against 318, 245 against 249, 127 against 126.
//
// A few output tiles with many rows leave most CUs idle: the rows are then cut into parts, whose sums (fp32, in the
// workspace) a second launch adds in order.  One group of 8192 rows, 1024 x 2048 weights (128 tiles): 101
// -> 46 us; 128 x 256 weights: 73 -> 17 us; 4096 rows, 512 x 512 weights: 39 -> 16 us.
int dw_split(int R, int E, int N, int K) {
  const long long tiles = (long long)E * ((N + 127) / 128) * ((K + 127) / 128), mean = (long long)R / E;
  const long long most = 512 / tiles < mean / 256 ? 512 / tiles : mean / 256;  // two workgroups a CU, 256 rows a part
  return most < 2 ? 1 : (most > 8 ? 8 : (int)most);
}

__global__ __launch_bounds__(256) void add_parts_kernel(const f32x4* __restrict__ parts, long long per, int split, int out,
                                                        void* __restrict__ dW) {
  const long long i = linear_block() * 256 + threadIdx.x;  // four elements of expert blockIdx.z
  if (i >= per) return;
  const long long e = blockIdx.z;
  f32x4 sum = parts[e * split * per + i];
  for (int k = 1; k < split; ++k) sum += parts[(e * split + k) * per + i];
  const float v[4] = {sum[0], sum[1], sum[2], sum[3]};
  store4(dW, out, (size_t)(e * per + i) * 4, v);
}

template <class T>
static hipError_t launch_dw(const RaggedArgs& a, hipStream_t s) {
  const long long mean = ((long long)a.R + a.E - 1) / a.E;
  const long long tiles = (long long)a.E * ((a.N + 255) / 256) * ((a.K + 127) / 128);
  if (a.split > 1) {
    RaggedArgs b = a;
    b.C = a.parts;
    b.out = MOE_OUT_F32;
    hipError_t e = launch_ragged_cfg<T, kDw, MOE_EPI_NONE, TileShape<128, 128, 2, 2, 64, 3>>(b, s);
    if (e != hipSuccess) return e;
    const long long per = (long long)a.N * a.K / 4;  // N and K are multiples of 8
    dim3 grid = grid2d((per + 255) / 256);
    grid.z = a.E;
    add_parts_kernel<<<grid, 256, 0, s>>>(reinterpret_cast<const f32x4*>(a.parts), per, a.split, a.out, a.C);
    return hipGetLastError();
  }
  if (tiles < 512) return launch_ragged_cfg<T, kDw, MOE_EPI_NONE, TileShape<128, 128, 2, 2, 64, 3>>(a, s);
  if (mean <= 512) return launch_ragged_cfg<T, kDw, MOE_EPI_NONE, TileShape<256, 128, 2, 2, 64, 3>>(a, s);
  return launch_ragged_cfg<T, kDw, MOE_EPI_NONE, TileShape<256, 256, 2, 4, 64, 4>>(a, s);
}

template <class T>
static hipError_t launch_w16(const RaggedArgs& a, int mode, int epilogue, hipStream_t s) {
  if (mode == kDw) return launch_dw<T>(a, s);
  if (mode == kDx) return launch_dx<T>(a, s);
  if (epilogue == MOE_EPI_SILU_MUL) return launch_ragged_fwd<T, MOE_EPI_SILU_MUL>(a, s);
  return launch_ragged_fwd<T, MOE_EPI_NONE>(a, s);
}

hipError_t launch_ragged_w16(const RaggedArgs& a, int mode, bool f16, int epilogue, hipStream_t stream) {
  return f16 ? launch_w16<ElemF16>(a, mode, epilogue, stream) : launch_w16<ElemBF16>(a, mode, epilogue, stream);
}

// ---------------------------------------------------------------------------------------------------
// SiLU*mul of a stored gate_up result and its gradient.  With s = 1 / (1 + exp(-g)):
//   h = g s u,   du = dh g s,   dg = dh u s (1 + g (1 - s)).
// Pure traffic: a thread takes 8 columns (one 16-byte load of each operand), arithmetic in fp32, one
// rounding per output.  (s is 0 where exp(-g) passes fp32, g < -88.)  The gradient multiplies dh, u and
// a = s (1 + g (1 - s)), -0.1 < a < 1.1, as (larger of dh and u * a / 2) * smaller * 2: neither dh u, which may pass fp32
// where the product does not (and made NaN of it at s = 0), nor a small factor times a stands for itself on the way.
// PAST 1: results are stored past the L2
// (nontemporal), 512 x 14336 forward 9.0 -> 7.5 us, 8191 x 14336 121 -> 117 us, but 512 x 776 3.0 -> 3.4 us, so not a few
// megabytes, which the next launch finds in the L2s.  PAST 2: operands that the 256 MB memory-side cache cannot hold are
// loaded so too: 8191 x 14336 forward 117 -> 113 us (6.2 TB/s), gradient 202 -> 183 us (6.4 TB/s), but 8191 x 768, whose
// operands lie in that cache, 6.8 -> 8.3 us.
__device__ __forceinline__ float sigmoid_f32(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

constexpr long long kNearBytes = 8ll << 20;

template <bool F16, bool GRAD, int PAST>
__global__ __launch_bounds__(256) void silu_mul_kernel(const u32x4* G, const u32x4* dh, long long n, int chunks,
                                                       u32x4* out) {
  const long long at = linear_block() * 256 + threadIdx.x;
  if (at >= n) return;
  const long long row = at / chunks;
  const int c = (int)(at - row * chunks);
  float g[8], u[8], v[8];
  unpack8<F16>(load16<PAST>(G + row * 2 * chunks + c), g);
  unpack8<F16>(load16<PAST>(G + row * 2 * chunks + chunks + c), u);
  if constexpr (!GRAD) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = g[i] * sigmoid_f32(g[i]) * u[i];
    store16<PAST>(pack8<F16>(v), out + at);
  } else {
    float d[8], w[8];
    unpack8<F16>(load16<PAST>(dh + at), d);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = sigmoid_f32(g[i]);
      const float half = 0.5f * s * (1.0f + g[i] * (1.0f - s));
      const bool more = fabsf(d[i]) > fabsf(u[i]);
      v[i] = (more ? d[i] : u[i]) * half * (more ? u[i] : d[i]) * 2.0f;
      w[i] = d[i] * (g[i] * s);
    }
    store16<PAST>(pack8<F16>(v), out + row * 2 * chunks + c);
    store16<PAST>(pack8<F16>(w), out + row * 2 * chunks + chunks + c);
  }
}

template <bool F16, bool GRAD>
static hipError_t launch_silu_of(const u32x4* G, const u32x4* dh, long long n, int chunks, u32x4* out, hipStream_t s) {
  const dim3 grid = grid2d((n + 255) / 256);
  if (n * (GRAD ? 48 : 32) > kFarBytes) silu_mul_kernel<F16, GRAD, 2><<<grid, 256, 0, s>>>(G, dh, n, chunks, out);
  else if (n * (GRAD ? 32 : 16) > kNearBytes) silu_mul_kernel<F16, GRAD, 1><<<grid, 256, 0, s>>>(G, dh, n, chunks, out);
  else silu_mul_kernel<F16, GRAD, 0><<<grid, 256, 0, s>>>(G, dh, n, chunks, out);
  return hipGetLastError();
}

template <bool GRAD>
static hipError_t launch_silu(const uint16_t* G, const uint16_t* dh, bool f16, long long R, int I, uint16_t* out,
                              hipStream_t s) {
  const int chunks = I / 8;
  const long long n = R * chunks;
  const u32x4 *g = reinterpret_cast<const u32x4*>(G), *d = reinterpret_cast<const u32x4*>(dh);
  u32x4* o = reinterpret_cast<u32x4*>(out);
  return f16 ? launch_silu_of<true, GRAD>(g, d, n, chunks, o, s) : launch_silu_of<false, GRAD>(g, d, n, chunks, o, s);
}

hipError_t launch_silu_mul(const uint16_t* G, bool f16, long long R, int I, uint16_t* h, hipStream_t stream) {
  return launch_silu<false>(G, nullptr, f16, R, I, h, stream);
}
hipError_t launch_silu_mul_grad(const uint16_t* G, const uint16_t* dh, bool f16, long long R, int I, uint16_t* dG,
                                hipStream_t stream) {
  return launch_silu<true>(G, dh, f16, R, I, dG, stream);
}

}  // namespace moe
