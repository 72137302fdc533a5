// Internal launchers (C++ linkage) of the operators around the GEMM, called by ops_api.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "launch.h"

namespace bsg {

// Size limits that the entry points check, so that every grid's threads fit the 32 bits they are counted in: each
// launcher has a static_assert of what it makes of them.
constexpr long long kMaxThreads = 0xffffffffLL;
constexpr long long kMaxElems = 1LL << 35;     // rows x K of the quantiser, twice those of SwiGLU's gradient
constexpr long long kMaxMoveWaves = 1LL << 25; // of the row moves: tokens x 64 vectors of a row
constexpr long long kMaxGradTokens = 1LL << 23;       // of the weighted sum's gradient
constexpr int kMaxExperts = 4096;
constexpr long long kMaxFewRowsCols = 1LL << 21;      // of the few-row product: tiles x 32 columns

// Row types (`dtype`) are the BSG_OUT_* codes: 1 f32, 2 bf16, 3 f16. Quantised forms (`quant`) are the
// QuantKind codes of quant.h.

// Rows (act 0: [rows, K]; 1: silu(first K) * (last K) of [rows, 2 K]) to codes and scales.
hipError_t launch_quantize(const void* x, int dtype, int act, int rows, int K, int quant, uint8_t* q, void* scales,
                           hipStream_t stream);

// Gradient of silu(first K) * (last K) of x [rows, 2 K].
hipError_t launch_swiglu_backward(const void* dy, const void* x, int dtype, int rows, int K, void* dx, hipStream_t stream);

// h = x + residual (if given), rstd, and the quantised h * rstd * weight.
hipError_t launch_rms_norm_quantize(const void* x, const void* residual, const void* weight, int dtype, int rows, int K,
                                    float eps, int quant, void* residual_out, float* rstd, uint8_t* q, void* scales,
                                    int num_cus, hipStream_t stream);

// Its gradient. partials: float[rms_norm_backward_groups * K].
int rms_norm_backward_groups(int rows, int num_cus);
hipError_t launch_rms_norm_backward(const void* dy, const void* h, const void* weight, const float* rstd,
                                    const void* dresidual, int dtype, int rows, int K, void* dx, float* dweight,
                                    float* partials, int num_cus, hipStream_t stream);

// Stable sort of picks by expert: counts, group offsets, tile map, row of every pick.
size_t route_sort_workspace_bytes(int n, int E);
hipError_t launch_route_sort(const int32_t* ids, int n, int E, int num_tiles, int padded, int M, int32_t* counts,
                             int32_t* expert_offsets, int32_t* tile_offsets, int32_t* expert_ids, int32_t* dest,
                             int32_t* workspace, hipStream_t stream);

// Rows of `row_bytes` to the rows of their picks; padding rows of the groups become zero.
hipError_t launch_permute_rows(const void* x, int row_bytes, const int32_t* dest, int tokens, int top_k,
                               const int32_t* counts, const int32_t* expert_offsets, int E, int M, void* out,
                               hipStream_t stream);

// out[t] = sum over picks of weight * y[dest]; weights may be null (1).
hipError_t launch_combine_rows(const void* y, int dtype, const int32_t* dest, const float* weights, int tokens, int top_k,
                               int K, int M, void* out, hipStream_t stream);

// dy[dest] = weight * dout, dweights = <dout, y[dest]>; padding rows of dy become zero.
hipError_t launch_combine_backward(const void* dout, const void* y, int dtype, const int32_t* dest, const float* weights,
                                   int tokens, int top_k, int K, const int32_t* counts, const int32_t* expert_offsets,
                                   int E, int M, void* dy, float* dweights, hipStream_t stream);

// MX product for M-tiles of few rows.
hipError_t launch_mx_few_rows(const GemmArgs& a, int fmt_a, int fmt_b, int out, hipStream_t stream);

}  // namespace bsg
