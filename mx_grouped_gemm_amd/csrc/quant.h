// Device helpers of the row-wise kernels around the GEMM: 8 consecutive elements per lane, loaded
// as 16-byte vectors (fp32: two), and the block quantisation of such lanes.
//
// A quantisation block of G elements is G / 8 neighbouring lanes (2, 4 or 16: inside one DPP row of
// 16 lanes), so its maximum is found by lane exchanges inside the VALU, without LDS.
#pragma once

#include "common.h"

namespace bsg {

// Row types, by the BSG_OUT_* codes of the C ABI.
struct F32 {};
struct BF16 {};
struct F16 {};
template <typename T> struct Row;
template <> struct Row<F32> { static constexpr int kBytes = 4; };
template <> struct Row<BF16> { static constexpr int kBytes = 2; };
template <> struct Row<F16> { static constexpr int kBytes = 2; };

// The bytes of 8 elements as they lie in memory.
template <typename T> struct Vec8 { v4i d[Row<T>::kBytes / 2]; };

// A wave's vectors are whole 128-byte lines to one instruction for the 2-byte types, halves of lines to each of
// fp32's two. Where rows are written in order, non-temporal stores pay for whole lines only (fp32: the norm's
// gradient of 16384 x 4096 196 us with them, 188 without; SwiGLU's 122 and 116).
template <typename T> constexpr bool kWholeLines = Row<T>::kBytes == 2;

// Vector v (8 elements each) of `p`.
template <typename T, bool kStream = false>
__device__ __forceinline__ Vec8<T> load_vec(const void* p, long long v) {
  Vec8<T> r;
  constexpr int n = Row<T>::kBytes / 2;
#pragma unroll
  for (int i = 0; i < n; i++) {
    const v4i* q = (const v4i*)p + v * n + i;
    r.d[i] = kStream ? __builtin_nontemporal_load(q) : *q;
  }
  return r;
}

template <typename T, bool kStream = false>
__device__ __forceinline__ void store_vec(void* p, long long v, const Vec8<T>& r) {
  constexpr int n = Row<T>::kBytes / 2;
#pragma unroll
  for (int i = 0; i < n; i++) {
    v4i* q = (v4i*)p + v * n + i;
    if (kStream) __builtin_nontemporal_store(r.d[i], q);
    else *q = r.d[i];
  }
}

template <typename T>
__device__ __forceinline__ Vec8<T> zero_vec() {
  Vec8<T> r;
#pragma unroll
  for (int i = 0; i < Row<T>::kBytes / 2; i++) r.d[i] = (v4i){0, 0, 0, 0};
  return r;
}

template <typename T>
__device__ __forceinline__ void unpack(const Vec8<T>& r, float (&f)[8]) {
  if constexpr (Row<T>::kBytes == 4) {
#pragma unroll
    for (int k = 0; k < 8; k++) f[k] = __uint_as_float((uint32_t)r.d[k / 4][k % 4]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const uint32_t w = (uint32_t)r.d[0][k];
      if constexpr (__is_same(T, BF16)) {
        f[2 * k] = __uint_as_float(w << 16);
        f[2 * k + 1] = __uint_as_float(w & 0xffff0000u);
      } else {
        f[2 * k] = (float)__builtin_bit_cast(_Float16, (uint16_t)w);
        f[2 * k + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w >> 16));
      }
    }
  }
}

// Round to nearest even into the row type.
template <typename T>
__device__ __forceinline__ Vec8<T> pack(const float (&f)[8]) {
  Vec8<T> r;
  if constexpr (Row<T>::kBytes == 4) {
#pragma unroll
    for (int k = 0; k < 8; k++) r.d[k / 4][k % 4] = (int)__float_as_uint(f[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; k++)
      r.d[0][k] = (int)(__is_same(T, BF16) ? bf16x2_bits(f[2 * k], f[2 * k + 1]) : f16x2_bits(f[2 * k], f[2 * k + 1]));
  }
  return r;
}

// Lane exchanges inside a DPP row of 16 lanes: with a neighbour (quad_perm), with the other half of
// a quad, mirrored inside 8 lanes, mirrored inside 16 lanes.
constexpr int kDppSwap1 = 0xB1, kDppSwap2 = 0x4E, kDppMirror8 = 0x141, kDppMirror16 = 0x140;
template <int kCtrl>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), kCtrl, 0xf, 0xf, true));
}

// The larger, NaN if either is (one instruction takes three operands).
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// Maximum over the LANES neighbouring lanes (2, 4 or 16) that share a quantisation block.
template <int LANES>
__device__ __forceinline__ float group_max(float v) {
  static_assert(LANES == 2 || LANES == 4 || LANES == 16, "a block is 2, 4 or 16 lanes");
  v = larger(v, dpp<kDppSwap1>(v));
  if constexpr (LANES >= 4) v = larger(v, dpp<kDppSwap2>(v));
  if constexpr (LANES >= 16) {
    v = larger(v, dpp<kDppMirror8>(v));
    v = larger(v, dpp<kDppMirror16>(v));
  }
  return v;
}

// Sum over each 16, 32 or 64 neighbouring lanes (all of them get it): the same pairs in the same order on
// every call.
__device__ __forceinline__ float lane_sum(float v, int lanes) {
  v += dpp<kDppSwap1>(v);
  v += dpp<kDppSwap2>(v);
  v += dpp<kDppMirror8>(v);
  v += dpp<kDppMirror16>(v);
  if (lanes > 16) v += __shfl_xor(v, 16);
  if (lanes > 32) v += __shfl_xor(v, 32);
  return v;
}
__device__ __forceinline__ float wave_sum(float v) { return lane_sum(v, kWave); }

// Quantised forms: element type and scale kind.
enum QuantKind { kE4M3Block = 0, kE4M3MX = 1, kE2M1MX = 2, kE2M1NV = 3 };
template <int Q> struct Quant {
  static constexpr bool kE2M1 = Q == kE2M1MX || Q == kE2M1NV;
  static constexpr int kBlock = Q == kE4M3Block ? 128 : Q == kE2M1NV ? 16 : 32;
  static constexpr int kLanes = kBlock / 8;
};

// Nearest e4m3fn (ties to even) of values within +-448, two per call, by the conversion instruction.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// Nearest e2m1 of values within +-6, eight codes in a dword, element 0 in the low nibble. The
// instruction divides by its scale operand first: 1 leaves the value as it is.
__device__ __forceinline__ uint32_t e2m1x8(const float (&y)[8]) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[0], y[1], 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[2], y[3], 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[4], y[5], 1.0f, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[6], y[7], 1.0f, 3);
  return w;
}

// y / s as fp32 division rounds it, for finite y and a divisor shared by many y: r is the correctly
// rounded 1 / s, and each of two corrections by the exact remainder takes the quotient nearer; after
// the first it is off by less than its last place, so the second rounds it correctly (Markstein's
// theorem). 6 instructions in place of about 11. The remainders and r must not underflow or overflow:
// s between 2^-100 and 2^100 (a quotient so small that its remainder is lost rounds to code 0 either way).
__device__ __forceinline__ float divide(float y, float s, float r) {
  float q = y * r;
  q = __builtin_fmaf(__builtin_fmaf(-q, s, y), r, q);
  return __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-q, s, y), r, q), y);     // s > 0; the sum of a -0 is +0
}

// Clamp to +-most.
__device__ __forceinline__ float clamp(float v, float most) { return __builtin_amdgcn_fmed3f(v, -most, most); }

// Quantises the lane's 8 values y (vector v of a matrix whose rows are whole blocks: codes and
// scales of a row-major matrix are then indexed by v alone) and stores the codes; the block's
// first lane stores its scale. All lanes of a block take part, or none.
//   e4m3, fp32 scale of 128: s = amax / 448 (1 if amax is 0, 2^-149 if it rounds to 0), codes of clamp(y / s),
//               both fp32 divisions
//   e8m0 of 32: code = floor(log2 amax) - emax + 127 in [0, 254] (127 if amax is 0); y 2^(127 - code)
//               is exact before the element's rounding and saturation
//   nvfp4: s = e4m3 of min(amax / 6, 448) (1 if amax is 0, the least subnormal if it rounds to 0),
//          codes of clamp(y / s)
// An amax that is infinite or NaN (of any NaN in the block) gives a scale that is: the clamps and the e2m1
// codes hide such values, the scale does not.
template <int Q>
__device__ __forceinline__ void quantize_store(const float (&y)[8], long long v, uint8_t* codes, void* scales) {
  constexpr int kLanes = Quant<Q>::kLanes;
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < 8; k++) amax = larger(amax, fabsf(y[k]));
  amax = group_max<kLanes>(amax);
  const bool first = (v & (kLanes - 1)) == 0;
  const long long block = v / kLanes;
  float z[8];
  if constexpr (Q == kE4M3Block) {
    float s = amax == 0.f ? 1.0f : amax / 448.0f;
    if (s >= 0x1p-100f && s <= 0x1p100f) {
      // |y / s| is at most 448 (1 + 2^-23), which rounds to 448: a clamp would change no code
      const float r = 1.0f / s;
#pragma unroll
      for (int k = 0; k < 8; k++) z[k] = divide(y[k], s, r);
    } else {
      // a subnormal s has few bits, so that |y / s| may reach 671, past the largest code: without the clamp such
      // quotients convert to NaN. The quotient of two infinities is NaN and stays it.
      if (s == 0.f) s = 0x1p-149f;
#pragma unroll
      for (int k = 0; k < 8; k++) z[k] = larger(-448.0f, __builtin_elementwise_minimum(y[k] / s, 448.0f));
    }
    if (first) ((float*)scales)[block] = s;
  } else if constexpr (Q == kE2M1NV) {
    uint32_t c = amax == 0.f ? 0x38u : e4m3x4(fminf(amax / 6.0f, 448.0f), 0.f, 0.f, 0.f) & 0xff;
    c = c == 0 ? 1u : amax < __builtin_inff() ? c : 0x7fu;      // 0x7f is NaN
    const float s = __builtin_amdgcn_cvt_f32_fp8((int)c, 0), r = 1.0f / s;
#pragma unroll
    for (int k = 0; k < 8; k++) z[k] = clamp(divide(clamp(y[k], 0x1p100f), s, r), 6.0f);
    if (first) ((uint8_t*)scales)[block] = (uint8_t)c;
  } else {
    constexpr int emax = Q == kE4M3MX ? 8 : 2;
    constexpr float most = Q == kE4M3MX ? 448.0f : 6.0f;
    int c = max((int)(__float_as_uint(amax) >> 23) - emax, 0);
    if (amax == 0.f) c = 127;
    if (!(amax < __builtin_inff())) c = 255;                           // NaN
    const float inv = __uint_as_float((uint32_t)(254 - c) << 23);      // 2^(127 - c): finite c are at most 252
#pragma unroll
    for (int k = 0; k < 8; k++) z[k] = clamp(y[k] * inv, most);
    if (first) ((uint8_t*)scales)[block] = (uint8_t)c;
  }
  if constexpr (Quant<Q>::kE2M1) {
    ((uint32_t*)codes)[v] = e2m1x8(z);
  } else {
    uint2 w;
    w.x = e4m3x4(z[0], z[1], z[2], z[3]);
    w.y = e4m3x4(z[4], z[5], z[6], z[7]);
    ((uint2*)codes)[v] = w;
  }
}

}  // namespace bsg
