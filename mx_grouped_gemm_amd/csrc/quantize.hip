// Row quantisation, optionally of SwiGLU (gfx950): the A operand of the grouped GEMM from plain rows, and
// SwiGLU's gradient.
//
//   act none:    y = x                          x [rows, K]
//   act SwiGLU:  y = g / (1 + exp(-g)) * u      x [rows, 2 K]: g the first K columns of a row, u the last K
// then per block of a row (128, 32 or 16 elements) a scale and codes, see quantize_store.
//
// Bound by HBM: 8 elements per lane, kPer vectors in flight per thread. y is never rounded to a
// narrower type before its quantisation.
#include "ops_launch.h"
#include "quant.h"

namespace bsg {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 2;               // vectors per thread
static_assert(kMaxElems / 8 / kPer + kThreads <= kMaxThreads && kMaxElems / 2 / 8 + kThreads <= kMaxThreads,
              "grids of the quantiser and of SwiGLU's gradient");

// exp(-c) for c <= 100 as 2^t 2^r: t, the rounded product -c log2(e), by the instruction for 2^x, r what its
// rounding left (2^r = 1 + r ln 2 to fp32; without r the error grows by |c| 2^-24, and 1.7 times as many codes
// of SwiGLU differed from exact ones). p becomes 2^t alone: infinite where c is far below 0.
__device__ __forceinline__ float exp_minus(float c, float& p) {
  constexpr float kHi = -1.44269502f, kLo = -1.92596303e-8f, kLn2 = 0.693147181f;     // kHi + kLo = -log2(e)
  const float t = c * kHi, r = __builtin_fmaf(c, kLo, __builtin_fmaf(c, kHi, -t));
  p = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(p, r * kLn2, p);
}

// g / (1 + exp(-g)) within about one unit of the last place: the quotient by the instruction for 1 / x,
// corrected once by its remainder and what the rounding of 1 + exp(-g) lost. Results below 1.1e-36 in
// magnitude (finite g < -87.3) are 0. The exponential is that of min(g, 100), past which it is lost behind 1
// (-g log2(e) itself would leave the range for the largest g). NaN stays NaN, and an infinity of either sign
// becomes it (g - g below; above, the remainder's inf - inf), so that the block shows it. expf and a full division made
// the kernel of 8192 x 2048 bf16 to e4m3 26 us, bound by the VALU; this takes 18 us, 4.7 TB/s.
__device__ __forceinline__ float silu(float g) {
  float p;
  const float e = exp_minus(__builtin_elementwise_minimum(g, 100.0f), p), d = 1.0f + e, lost = e - (d - 1.0f);
  const float q = __builtin_amdgcn_rcpf(d), y = g * q;
  return p >= 0x1p126f ? g - g : __builtin_fmaf(__builtin_fmaf(-y, lost, __builtin_fmaf(-y, d, g)), q, y);
}

template <typename T, int ACT, int Q>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(const void* __restrict__ x, long long vecs, int row_vecs,
                                                                 uint8_t* __restrict__ q, void* __restrict__ scales) {
  const long long base = (long long)blockIdx.x * (kThreads * kPer);
  // the block's first row and the place in it: one 64-bit division a block, 32-bit ones a thread
  const long long row0 = ACT ? base / row_vecs : 0;
  const uint32_t in0 = ACT ? (uint32_t)(base - row0 * row_vecs) : 0;
  Vec8<T> g[kPer], u[kPer];
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    const uint32_t at = i * kThreads + threadIdx.x;
    const long long v = base + at;
    g[i] = zero_vec<T>();
    u[i] = zero_vec<T>();
    if (v >= vecs) continue;
    if (ACT) {
      const uint32_t r = (in0 + at) / (uint32_t)row_vecs, c = (in0 + at) - r * row_vecs;
      const long long src = (row0 + r) * 2 * row_vecs + c;
      g[i] = load_vec<T>(x, src);
      u[i] = load_vec<T>(x, src + row_vecs);
    } else {
      g[i] = load_vec<T>(x, v);
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    const long long v = base + i * kThreads + threadIdx.x;
    if (v >= vecs) continue;
    float y[8];
    unpack<T>(g[i], y);
    if (ACT) {
      float f[8];
      unpack<T>(u[i], f);
#pragma unroll
      for (int k = 0; k < 8; k++) y[k] = silu(y[k]) * f[k];
    }
    quantize_store<Q>(y, v, q, scales);
  }
}

// Gradient of silu(g) u, with s = 1 / (1 + exp(-g)) and 1 - s = s exp(-g):
//   dg = dy u s (1 + g (1 - s)),   du = dy g s
// both 0 for g below -87 (where s leaves fp32). dx may be x: a thread reads its vectors of both halves before
// it writes them. Bound by HBM: 8192 x 2048 bf16 27 us, 6.2 TB/s, with one vector per thread and non-temporal
// accesses (31 us cached; two vectors per thread 29 and 32 us).
template <typename T>
__global__ __launch_bounds__(kThreads) void swiglu_backward_kernel(const void* __restrict__ dy, const void* x,
                                                                   long long vecs, int row_vecs, void* dx) {
  const long long base = (long long)blockIdx.x * kThreads, v = base + threadIdx.x;
  const long long row0 = base / row_vecs;      // as in the kernel above: one 64-bit division a block
  const uint32_t in = (uint32_t)(base - row0 * row_vecs) + threadIdx.x, r = in / (uint32_t)row_vecs;
  if (v >= vecs) return;
  const long long gate = (row0 + r) * 2 * row_vecs + (in - r * row_vecs), up = gate + row_vecs;
  const Vec8<T> gv = load_vec<T, true>(x, gate), uv = load_vec<T, true>(x, up), dv = load_vec<T, true>(dy, v);
  float g[8], u[8], d[8];
  unpack<T>(gv, g);
  unpack<T>(uv, u);
  unpack<T>(dv, d);
#pragma unroll
  for (int k = 0; k < 8; k++) {
    float p;
    const float m = __builtin_elementwise_maximum(g[k], -87.0f), c = __builtin_elementwise_minimum(m, 100.0f);
    const float e = exp_minus(c, p), q = __builtin_amdgcn_rcpf(1.0f + e), s = g[k] < -87.0f ? 0.f : q;
    g[k] = (d[k] * u[k]) * (s * __builtin_fmaf(c, e * q, 1.0f));
    u[k] = d[k] * (m * s);
  }
  store_vec<T, kWholeLines<T>>(dx, gate, pack<T>(g));
  store_vec<T, kWholeLines<T>>(dx, up, pack<T>(u));
}

template <typename T>
hipError_t launch_backward(const void* dy, const void* x, int rows, int K, void* dx, hipStream_t s) {
  const long long vecs = (long long)rows * (K / 8), blocks = (vecs + kThreads - 1) / kThreads;
  hipLaunchKernelGGL(swiglu_backward_kernel<T>, dim3((unsigned)blocks), dim3(kThreads), 0, s, dy, x, vecs, K / 8, dx);
  return hipGetLastError();
}

template <typename T, int ACT>
hipError_t launch(const void* x, int rows, int K, int quant, uint8_t* q, void* scales, hipStream_t s) {
  const int row_vecs = K / 8;
  const long long vecs = (long long)rows * row_vecs;
  const long long blocks = (vecs + kThreads * kPer - 1) / (kThreads * kPer);
  const dim3 grid((unsigned)blocks), block(kThreads);
  switch (quant) {
    case kE4M3Block: hipLaunchKernelGGL((quantize_rows_kernel<T, ACT, kE4M3Block>), grid, block, 0, s, x, vecs, row_vecs, q, scales); break;
    case kE4M3MX: hipLaunchKernelGGL((quantize_rows_kernel<T, ACT, kE4M3MX>), grid, block, 0, s, x, vecs, row_vecs, q, scales); break;
    case kE2M1MX: hipLaunchKernelGGL((quantize_rows_kernel<T, ACT, kE2M1MX>), grid, block, 0, s, x, vecs, row_vecs, q, scales); break;
    case kE2M1NV: hipLaunchKernelGGL((quantize_rows_kernel<T, ACT, kE2M1NV>), grid, block, 0, s, x, vecs, row_vecs, q, scales); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize(const void* x, int dtype, int act, int rows, int K, int quant, uint8_t* q, void* scales,
                           hipStream_t s) {
  if (rows == 0) return hipSuccess;
  switch (dtype * 2 + act) {
    case 2: return launch<F32, 0>(x, rows, K, quant, q, scales, s);
    case 3: return launch<F32, 1>(x, rows, K, quant, q, scales, s);
    case 4: return launch<BF16, 0>(x, rows, K, quant, q, scales, s);
    case 5: return launch<BF16, 1>(x, rows, K, quant, q, scales, s);
    case 6: return launch<F16, 0>(x, rows, K, quant, q, scales, s);
    case 7: return launch<F16, 1>(x, rows, K, quant, q, scales, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_swiglu_backward(const void* dy, const void* x, int dtype, int rows, int K, void* dx, hipStream_t s) {
  switch (dtype) {
    case kOutF32: return launch_backward<F32>(dy, x, rows, K, dx, s);
    case kOutBF16: return launch_backward<BF16>(dy, x, rows, K, dx, s);
    case kOutF16: return launch_backward<F16>(dy, x, rows, K, dx, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace bsg
