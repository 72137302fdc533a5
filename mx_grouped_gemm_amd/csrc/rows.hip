// Token rows to the rows of their picks and back (gfx950): the grouped layout's row moves, their
// weighted sum and its gradient.
//
//   permute_rows      out[dest[t, j]] = x[t];   padding rows of the groups are zero
//   combine_rows      out[t] = sum over j of w[t, j] y[dest[t, j]]   (w absent: 1, the gradient of permute_rows)
//   combine_backward  dy[dest[t, j]] = w[t, j] dout[t],  dw[t, j] = <dout[t], y[dest[t, j]]>;  padding rows zero
//
// dest is -1 (or any value outside [0, M)) for a pick without a row: it is skipped, never read or
// written; its dw is 0. Sums in fp32 in the order of j. All three are token-major: a token's row is
// read once for all of its picks, and every grouped row once. Bound by HBM.
#include <type_traits>

#include "ops_launch.h"
#include "quant.h"

namespace bsg {
namespace {

constexpr int kThreads = 256;

// Picks are handled G at a time, G the largest divisor of top_k up to 8 (a kernel for each): all G are
// there, so their rows (and weights) come in one scalar load. The first G come before any loop, so that
// this load and the token row's are on their way together: with all of them inside the loop, which waits
// for the row first, the rows of 16384 x 8 picks, K 7168 bf16, took 418 us against 374.
constexpr int kMostPicks = 8;

// Zeroes every parts-th padding row of expert e's group, from row `part` on: rows
// expert_offsets[e] + counts[e] .. expert_offsets[e + 1], clamped into [0, M).
__device__ __forceinline__ void zero_padding(const int32_t* __restrict__ counts,
                                             const int32_t* __restrict__ expert_offsets, int e, int part, int parts,
                                             int M, int row_bytes, void* out) {
  const long long off = max(expert_offsets[e], 0);
  const long long lo = min(off + max(counts[e], 0), (long long)M), hi = min((long long)expert_offsets[e + 1], (long long)M);
  for (long long r = lo + part; r < hi; r += parts) {
    if ((row_bytes & 15) == 0 && ((uintptr_t)out & 15) == 0) {
      v4i* p = (v4i*)((uint8_t*)out + r * row_bytes);
      for (int k = threadIdx.x; k < row_bytes / 16; k += kThreads) p[k] = (v4i){0, 0, 0, 0};
    } else {
      int* p = (int*)((uint8_t*)out + r * row_bytes);
      for (int k = threadIdx.x; k < row_bytes / 4; k += kThreads) p[k] = 0;
    }
  }
}

// A wave's work in the row moves: 64 vectors of one token's row (the last ones of a row may be fewer),
// so that the token, its picks and their weights are uniform and come through the scalar unit.
struct Piece {
  long long t;
  int c;          // the lane's vector of the row; at or past row_vecs: none
};
__device__ __forceinline__ Piece wave_piece(uint32_t block, int per_row) {
  const uint32_t w = __builtin_amdgcn_readfirstlane(block * (kThreads / kWave) + (threadIdx.x >> 6));
  const uint32_t t = w / (uint32_t)per_row;
  return {(long long)t, (int)((w - t * per_row) * kWave + (threadIdx.x & 63))};
}

// V: 16-byte or 4-byte vectors. The first `pads` workgroups zero padding, pads / E of them for each
// expert (first: each has up to 127 rows to write, which would be the launch's tail), the rest move rows.
template <typename V, int G>
__global__ __launch_bounds__(kThreads) void permute_rows_kernel(
    const V* __restrict__ x, const int32_t* __restrict__ dest, int tokens, int top_k, int row_vecs, int per_row,
    const int32_t* __restrict__ counts, const int32_t* __restrict__ expert_offsets, int parts, int pads, int M,
    V* __restrict__ out) {
  const int b = blockIdx.x;
  if (b < pads) {
    zero_padding(counts, expert_offsets, b / parts, b % parts, parts, M, row_vecs * (int)sizeof(V), out);
    return;
  }
  const Piece p = wave_piece(b - pads, per_row);
  if (p.t >= tokens || p.c >= row_vecs) return;
  const V v = x[p.t * row_vecs + p.c];
  const int32_t* d = dest + p.t * top_k;
  auto place = [&](const int (&r)[G]) {
#pragma unroll
    for (int j = 0; j < G; j++)
      if (r[j] >= 0 && r[j] < M) __builtin_nontemporal_store(v, out + (long long)r[j] * row_vecs + p.c);
  };
  int r[G];
#pragma unroll
  for (int j = 0; j < G; j++) r[j] = d[j];
  place(r);
  for (int j0 = G; j0 < top_k; j0 += G) {
#pragma unroll
    for (int j = 0; j < G; j++) r[j] = d[j0 + j];
    place(r);
  }
}

// One vector of 8 elements of a token row per thread; the rows of G picks are all loaded before the
// first is added.
template <typename T, bool kWeighted, int G>
__global__ __launch_bounds__(kThreads) void combine_rows_kernel(const void* __restrict__ y,
                                                                const int32_t* __restrict__ dest,
                                                                const float* __restrict__ weights, int tokens, int top_k,
                                                                int row_vecs, int per_row, int M, void* __restrict__ out) {
  const Piece p = wave_piece(blockIdx.x, per_row);
  if (p.t >= tokens || p.c >= row_vecs) return;
  float acc[8];
#pragma unroll
  for (int k = 0; k < 8; k++) acc[k] = 0.f;
  for (int j0 = 0; j0 < top_k; j0 += G) {
    Vec8<T> v[G];
    int r[G];
    float w[G];
#pragma unroll
    for (int j = 0; j < G; j++) {
      r[j] = dest[p.t * top_k + j0 + j];
      w[j] = kWeighted ? weights[p.t * top_k + j0 + j] : 1.f;
    }
#pragma unroll
    for (int j = 0; j < G; j++) {
      const bool live = r[j] >= 0 && r[j] < M;
      v[j] = zero_vec<T>();
      if (live) v[j] = load_vec<T, true>(y, (long long)r[j] * row_vecs + p.c);
      if (!live) w[j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < G; j++) {
      float f[8];
      unpack<T>(v[j], f);
#pragma unroll
      for (int k = 0; k < 8; k++) acc[k] += kWeighted ? w[j] * f[k] : f[k];
    }
  }
  store_vec<T, true>(out, p.t * row_vecs + p.c, pack<T>(acc));
}

// The first `pads` workgroups zero padding, the rest take a token each (W = 4), or one a wave (W = 1, rows of up
// to 64 vectors: 16384 x 8 picks bf16, K 128 17 us against 33, K 256 25 and 37, K 512 50 and 49, K 1024 111 and
// 98), G picks at a time.
template <typename T, int G, int W>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(
    const void* __restrict__ dout, const void* __restrict__ y, const int32_t* __restrict__ dest,
    const float* __restrict__ weights, int tokens, int top_k, int row_vecs, const int32_t* __restrict__ counts,
    const int32_t* __restrict__ expert_offsets, int parts, int pads, int M, void* __restrict__ dy,
    float* __restrict__ dweights) {
  __shared__ float part[W][G];
  const int b = blockIdx.x;
  if (b < pads) {
    zero_padding(counts, expert_offsets, b / parts, b % parts, parts, M, row_vecs * 8 * Row<T>::kBytes, dy);
    return;
  }
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), tid = W == 1 ? threadIdx.x & 63 : threadIdx.x;
  const long long t = W == 1 ? (long long)(b - pads) * (kThreads / kWave) + wave : b - pads;
  if (t >= tokens) return;
  for (int j0 = 0; j0 < top_k; j0 += G) {
    int r[G];
    float w[G], dot[G];
#pragma unroll
    for (int j = 0; j < G; j++) {
      r[j] = dest[t * top_k + j0 + j];
      w[j] = weights[t * top_k + j0 + j];
      dot[j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < G; j++) {
      if (r[j] >= M) r[j] = -1;
      if (r[j] < 0) w[j] = 0.f;
    }
    for (int c = tid; c < row_vecs; c += W * kWave) {
      const Vec8<T> dv = load_vec<T>(dout, t * row_vecs + c);
      Vec8<T> v[G];
#pragma unroll
      for (int j = 0; j < G; j++)
        v[j] = r[j] >= 0 ? load_vec<T, true>(y, (long long)r[j] * row_vecs + c) : zero_vec<T>();
      float d[8];
      unpack<T>(dv, d);
#pragma unroll
      for (int j = 0; j < G; j++) {
        if (r[j] < 0) continue;
        float f[8], o[8];
        unpack<T>(v[j], f);
#pragma unroll
        for (int k = 0; k < 8; k++) {
          dot[j] += d[k] * f[k];
          o[k] = w[j] * d[k];
        }
        store_vec<T, true>(dy, (long long)r[j] * row_vecs + c, pack<T>(o));
      }
    }
#pragma unroll
    for (int j = 0; j < G; j++) dot[j] = wave_sum(dot[j]);
    if constexpr (W == 1) {
      if (tid == 0) {
#pragma unroll
        for (int j = 0; j < G; j++) dweights[t * top_k + j0 + j] = dot[j];
      }
      continue;
    }
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int j = 0; j < G; j++) part[wave][j] = dot[j];
    }
    __syncthreads();
    if ((int)threadIdx.x < G) {
      float s = 0.f;
#pragma unroll
      for (int q = 0; q < W; q++) s += part[q][threadIdx.x];
      dweights[t * top_k + j0 + threadIdx.x] = s;
    }
    __syncthreads();
  }
}

// Workgroups per expert for the padding rows: about 256 in all.
int padding_parts(int E) { return E >= 256 ? 1 : 256 / E; }

static_assert(kMaxMoveWaves * kWave + (kMaxExperts + 1) * kThreads <= kMaxThreads &&
                  (kMaxGradTokens + kMaxExperts) * kThreads <= kMaxThreads,
              "grids with at most kMaxExperts workgroups for padding rows");

// Waves of a row, and workgroups of the row moves.
int pieces(int row_vecs) { return (row_vecs + kWave - 1) / kWave; }
long long move_blocks_of(int tokens, int row_vecs) {
  return ((long long)tokens * pieces(row_vecs) + kThreads / kWave - 1) / (kThreads / kWave);
}

int picks_together(int top_k) {
  for (int g = kMostPicks; g > 1; g--)
    if (top_k % g == 0) return g;
  return 1;
}

// f with picks_together(top_k) as a constant.
template <typename F>
hipError_t with_picks(int top_k, F f) {
  switch (picks_together(top_k)) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 3: return f(std::integral_constant<int, 3>());
    case 4: return f(std::integral_constant<int, 4>());
    case 5: return f(std::integral_constant<int, 5>());
    case 6: return f(std::integral_constant<int, 6>());
    case 7: return f(std::integral_constant<int, 7>());
    default: return f(std::integral_constant<int, 8>());
  }
}

template <typename V>
hipError_t launch_permute(const void* x, int row_vecs, const int32_t* dest, int tokens, int top_k, const int32_t* counts,
                          const int32_t* expert_offsets, int E, int M, void* out, hipStream_t s) {
  const long long move = move_blocks_of(tokens, row_vecs);
  const int parts = padding_parts(E);
  return with_picks(top_k, [&](auto g) {
    hipLaunchKernelGGL((permute_rows_kernel<V, decltype(g)::value>), dim3((unsigned)(move + E * parts)), dim3(kThreads), 0,
                       s, (const V*)x, dest, tokens, top_k, row_vecs, pieces(row_vecs), counts, expert_offsets, parts,
                       E * parts, M, (V*)out);
    return hipGetLastError();
  });
}

template <typename T, bool kWeighted>
hipError_t launch_combine(const void* y, const int32_t* dest, const float* weights, int tokens, int top_k, int K, int M,
                          void* out, hipStream_t s) {
  const int V = K / 8;
  const long long blocks = move_blocks_of(tokens, V);
  return with_picks(top_k, [&](auto g) {
    hipLaunchKernelGGL((combine_rows_kernel<T, kWeighted, decltype(g)::value>), dim3((unsigned)blocks), dim3(kThreads), 0, s,
                       y, dest, weights, tokens, top_k, V, pieces(V), M, out);
    return hipGetLastError();
  });
}

template <typename T>
hipError_t launch_combine_bwd(const void* dout, const void* y, const int32_t* dest, const float* weights, int tokens,
                              int top_k, int K, const int32_t* counts, const int32_t* expert_offsets, int E, int M,
                              void* dy, float* dweights, hipStream_t s) {
  const int parts = padding_parts(E);
  const bool narrow = K / 8 <= kWave;      // a vector per lane
  const long long blocks = (narrow ? (tokens + 3LL) / 4 : (long long)tokens) + (long long)E * parts;
  return with_picks(top_k, [&](auto g) {
    constexpr int G = decltype(g)::value;
    hipLaunchKernelGGL((narrow ? combine_backward_kernel<T, G, 1> : combine_backward_kernel<T, G, kThreads / kWave>),
                       dim3((unsigned)blocks), dim3(kThreads), 0, s, dout, y, dest, weights, tokens, top_k, K / 8, counts,
                       expert_offsets, parts, E * parts, M, dy, dweights);
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_permute_rows(const void* x, int row_bytes, const int32_t* dest, int tokens, int top_k,
                               const int32_t* counts, const int32_t* expert_offsets, int E, int M, void* out,
                               hipStream_t s) {
  // 16-byte vectors where rows and buffers are whole ones (scale rows need not be), else 4-byte
  const bool wide = row_bytes % 16 == 0 && (((uintptr_t)x | (uintptr_t)out) & 15) == 0;
  return wide ? launch_permute<v4i>(x, row_bytes / 16, dest, tokens, top_k, counts, expert_offsets, E, M, out, s)
              : launch_permute<int>(x, row_bytes / 4, dest, tokens, top_k, counts, expert_offsets, E, M, out, s);
}

hipError_t launch_combine_rows(const void* y, int dtype, const int32_t* dest, const float* weights, int tokens, int top_k,
                               int K, int M, void* out, hipStream_t s) {
  if (tokens == 0) return hipSuccess;
  switch (dtype) {
    case kOutF32: return weights ? launch_combine<F32, true>(y, dest, weights, tokens, top_k, K, M, out, s)
                            : launch_combine<F32, false>(y, dest, weights, tokens, top_k, K, M, out, s);
    case kOutBF16: return weights ? launch_combine<BF16, true>(y, dest, weights, tokens, top_k, K, M, out, s)
                            : launch_combine<BF16, false>(y, dest, weights, tokens, top_k, K, M, out, s);
    case kOutF16: return weights ? launch_combine<F16, true>(y, dest, weights, tokens, top_k, K, M, out, s)
                            : launch_combine<F16, false>(y, dest, weights, tokens, top_k, K, M, out, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_combine_backward(const void* dout, const void* y, int dtype, const int32_t* dest, const float* weights,
                                   int tokens, int top_k, int K, const int32_t* counts, const int32_t* expert_offsets,
                                   int E, int M, void* dy, float* dweights, hipStream_t s) {
  switch (dtype) {
    case kOutF32: return launch_combine_bwd<F32>(dout, y, dest, weights, tokens, top_k, K, counts, expert_offsets, E, M, dy, dweights, s);
    case kOutBF16: return launch_combine_bwd<BF16>(dout, y, dest, weights, tokens, top_k, K, counts, expert_offsets, E, M, dy, dweights, s);
    case kOutF16: return launch_combine_bwd<F16>(dout, y, dest, weights, tokens, top_k, K, counts, expert_offsets, E, M, dy, dweights, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace bsg
