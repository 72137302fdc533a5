// C ABI of the operators around the grouped GEMM: argument validation and dispatch. Declarations and
// contracts: include/bsgemm.h. Every check is made on the host before anything is enqueued, in the
// order formats, sizes, NULL, alignment, device, with a workspace's size after its alignment.
#include "../../include/bsgemm.h"

#include <hip/hip_runtime.h>

#include "device.h"
#include "ops_launch.h"

using bsg::aligned;
using bsg::check_device;

namespace {

bool row_type(uint32_t t) { return t == BSG_OUT_F32 || t == BSG_OUT_BF16 || t == BSG_OUT_F16; }

// QuantKind of a q_fmt word, or -1.
int quant_kind(uint32_t q_fmt) {
  switch (q_fmt) {
    case BSG_QUANT(BSG_ELEM_E4M3, BSG_SCALE_BLOCKWISE): return 0;
    case BSG_QUANT(BSG_ELEM_E4M3, BSG_SCALE_MX): return 1;
    case BSG_QUANT(BSG_ELEM_E2M1, BSG_SCALE_MX): return 2;
    case BSG_QUANT(BSG_ELEM_E2M1, BSG_SCALE_NV): return 3;
    default: return -1;
  }
}

// Alignment of a quantised output's scales: whole floats (blockwise), bytes otherwise.
uintptr_t scale_align(int quant) { return quant == 0 ? 4 : 1; }

constexpr int32_t kMaxNormK = 32768;         // a row is held in one workgroup's registers
constexpr int32_t kMaxNormRows = (1 << 22) - 1;   // a workgroup of up to 1024 threads each
constexpr int32_t kMaxPicks = 1 << 24;       // of a sort: 4096 chunks, 8192 above 2048 experts
constexpr int32_t kMaxRowsK = 1 << 22;       // K of the few-row product: its 256-row buffers stay under 2 GiB

int status(hipError_t e) { return e == hipSuccess ? BSG_OK : BSG_ERR_LAUNCH; }

bool picks_ok(int32_t tokens, int32_t top_k) {
  return tokens >= 0 && top_k >= 1 && (long long)tokens * top_k <= INT32_MAX;
}

// Waves of the row moves, 64 vectors of a row each.
bool waves_ok(int32_t tokens, int32_t row_vecs) { return (long long)tokens * ((row_vecs + 63LL) / 64) <= bsg::kMaxMoveWaves; }

}  // namespace

extern "C" int bsgemm_quantize(const void* x, uint32_t x_dtype, uint32_t act, int32_t rows, int32_t K, uint32_t q_fmt,
                               void* q, void* scales, void* stream) {
  const int quant = quant_kind(q_fmt);
  if (!row_type(x_dtype) || quant < 0 || (act != BSG_ACT_NONE && act != BSG_ACT_SWIGLU)) return BSG_ERR_FMT;
  if (rows < 0 || K <= 0 || K % 128 || K > (1 << 30) || (long long)rows * K > bsg::kMaxElems) return BSG_ERR_SHAPE;
  if (rows > 0 && (!x || !q || !scales)) return BSG_ERR_NULL;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scales, scale_align(quant))) return BSG_ERR_ALIGN;
  if (rows == 0) return BSG_OK;
  if (int st = check_device()) return st;
  return status(bsg::launch_quantize(x, (int)x_dtype, act == BSG_ACT_SWIGLU ? 1 : 0, rows, K, quant,
                                     static_cast<uint8_t*>(q), scales, static_cast<hipStream_t>(stream)));
}

extern "C" int bsgemm_swiglu_backward(const void* dy, const void* x, uint32_t dtype, int32_t rows, int32_t K, void* dx,
                                      void* stream) {
  if (!row_type(dtype)) return BSG_ERR_FMT;
  if (rows < 0 || K <= 0 || K % 8 || K > (1 << 30) || (long long)rows * K > bsg::kMaxElems / 2) return BSG_ERR_SHAPE;
  if (rows > 0 && (!dy || !x || !dx)) return BSG_ERR_NULL;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(dx, 16)) return BSG_ERR_ALIGN;
  if (rows == 0) return BSG_OK;
  if (int st = check_device()) return st;
  return status(bsg::launch_swiglu_backward(dy, x, (int)dtype, rows, K, dx, static_cast<hipStream_t>(stream)));
}

extern "C" int bsgemm_rms_norm_quantize(const void* x, const void* residual, const void* weight, uint32_t dtype,
                                        int32_t rows, int32_t K, float eps, uint32_t q_fmt, void* residual_out,
                                        float* rstd, void* q, void* scales, void* stream) {
  const int quant = quant_kind(q_fmt);
  if (!row_type(dtype) || quant < 0) return BSG_ERR_FMT;
  if (rows < 0 || rows > kMaxNormRows || K <= 0 || K % 128 || K > kMaxNormK || !(eps >= 0.f)) return BSG_ERR_SHAPE;
  if (rows > 0 && (!x || !weight || !q || !scales || (!residual) != (!residual_out))) return BSG_ERR_NULL;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(residual_out, 16) ||
      !aligned(rstd, 4) || !aligned(q, 16) || !aligned(scales, scale_align(quant)))
    return BSG_ERR_ALIGN;
  if (rows == 0) return BSG_OK;
  int num_cus = 0;
  if (int st = check_device(&num_cus)) return st;
  return status(bsg::launch_rms_norm_quantize(x, residual, weight, (int)dtype, rows, K, eps, quant, residual_out, rstd,
                                              static_cast<uint8_t*>(q), scales, num_cus,
                                              static_cast<hipStream_t>(stream)));
}

extern "C" int bsgemm_rms_norm_backward_workspace_size(int32_t rows, int32_t K, size_t* bytes) {
  if (rows < 0 || K <= 0 || K % 128 || K > kMaxNormK) return BSG_ERR_SHAPE;
  if (!bytes) return BSG_ERR_NULL;
  int num_cus = 0;
  if (int st = check_device(&num_cus)) return st;
  *bytes = (size_t)bsg::rms_norm_backward_groups(rows, num_cus) * K * sizeof(float);
  return BSG_OK;
}

extern "C" int bsgemm_rms_norm_backward(const void* dy, const void* h, const void* weight, const float* rstd,
                                        const void* dresidual, uint32_t dtype, int32_t rows, int32_t K, void* dx,
                                        float* dweight, void* workspace, size_t workspace_bytes, void* stream) {
  if (!row_type(dtype)) return BSG_ERR_FMT;
  if (rows < 0 || K <= 0 || K % 128 || K > kMaxNormK) return BSG_ERR_SHAPE;
  if (!dweight || (rows > 0 && (!dy || !h || !weight || !rstd || !dx || !workspace))) return BSG_ERR_NULL;
  if (!aligned(dy, 16) || !aligned(h, 16) || !aligned(weight, 16) || !aligned(rstd, 4) || !aligned(dresidual, 16) ||
      !aligned(dx, 16) || !aligned(dweight, 4) || !aligned(workspace, 16))
    return BSG_ERR_ALIGN;
  int num_cus = 0;
  if (int st = check_device(&num_cus)) return st;
  if (workspace_bytes < (size_t)bsg::rms_norm_backward_groups(rows, num_cus) * K * sizeof(float)) return BSG_ERR_SHAPE;
  return status(bsg::launch_rms_norm_backward(dy, h, weight, rstd, dresidual, (int)dtype, rows, K, dx, dweight,
                                              static_cast<float*>(workspace), num_cus,
                                              static_cast<hipStream_t>(stream)));
}

extern "C" int bsgemm_route_sort_workspace_size(int32_t num_picks, int32_t num_experts, size_t* bytes) {
  if (num_picks < 0 || num_picks > kMaxPicks || num_experts < 1 || num_experts > bsg::kMaxExperts) return BSG_ERR_SHAPE;
  if (!bytes) return BSG_ERR_NULL;
  *bytes = bsg::route_sort_workspace_bytes(num_picks, num_experts);
  return BSG_OK;
}

extern "C" int bsgemm_route_sort(const int32_t* topk_ids, int32_t num_picks, int32_t num_experts, int32_t num_tiles,
                                 int32_t padded, int32_t M, int32_t* counts, int32_t* expert_offsets,
                                 int32_t* tile_offsets, int32_t* expert_ids, int32_t* dest, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  if (num_picks < 0 || num_picks > kMaxPicks || num_experts < 1 || num_experts > bsg::kMaxExperts || num_tiles < 0 ||
      num_tiles == INT32_MAX || M < 0)
    return BSG_ERR_SHAPE;
  const size_t need = bsg::route_sort_workspace_bytes(num_picks, num_experts);
  if (!counts || !expert_offsets || !tile_offsets || (num_tiles > 0 && !expert_ids) ||
      (num_picks > 0 && (!topk_ids || !dest)) || (need > 0 && !workspace))
    return BSG_ERR_NULL;
  if (!aligned(topk_ids, 4) || !aligned(counts, 4) || !aligned(expert_offsets, 4) || !aligned(tile_offsets, 4) ||
      !aligned(expert_ids, 4) || !aligned(dest, 4) || !aligned(workspace, 4))
    return BSG_ERR_ALIGN;
  if (workspace_bytes < need) return BSG_ERR_SHAPE;
  if (int st = check_device()) return st;
  return status(bsg::launch_route_sort(topk_ids, num_picks, num_experts, num_tiles, padded ? 1 : 0, M, counts,
                                       expert_offsets, tile_offsets, expert_ids, dest,
                                       static_cast<int32_t*>(workspace), static_cast<hipStream_t>(stream)));
}

extern "C" int bsgemm_permute_rows(const void* x, int32_t row_bytes, const int32_t* dest, int32_t tokens,
                                   int32_t top_k, const int32_t* counts, const int32_t* expert_offsets,
                                   int32_t num_experts, int32_t M, void* out, void* stream) {
  if (!picks_ok(tokens, top_k) || row_bytes <= 0 || row_bytes % 4 || num_experts < 1 || num_experts > bsg::kMaxExperts || M < 0 ||
      !waves_ok(tokens, row_bytes / 4))
    return BSG_ERR_SHAPE;
  if (!counts || !expert_offsets || (tokens > 0 && (!x || !dest)) || (M > 0 && !out)) return BSG_ERR_NULL;
  if (!aligned(x, 4) || !aligned(dest, 4) || !aligned(counts, 4) || !aligned(expert_offsets, 4) || !aligned(out, 4))
    return BSG_ERR_ALIGN;
  if (M == 0) return BSG_OK;
  if (int st = check_device()) return st;
  return status(bsg::launch_permute_rows(x, row_bytes, dest, tokens, top_k, counts, expert_offsets, num_experts, M, out,
                                         static_cast<hipStream_t>(stream)));
}

extern "C" int bsgemm_combine_rows(const void* y, uint32_t dtype, const int32_t* dest, const float* weights,
                                   int32_t tokens, int32_t top_k, int32_t K, int32_t M, void* out, void* stream) {
  if (!row_type(dtype)) return BSG_ERR_FMT;
  if (!picks_ok(tokens, top_k) || K <= 0 || K % 8 || M < 0 || !waves_ok(tokens, K / 8)) return BSG_ERR_SHAPE;
  if (tokens > 0 && (!dest || !out || (M > 0 && !y))) return BSG_ERR_NULL;
  if (!aligned(y, 16) || !aligned(dest, 4) || !aligned(weights, 4) || !aligned(out, 16)) return BSG_ERR_ALIGN;
  if (tokens == 0) return BSG_OK;
  if (int st = check_device()) return st;
  return status(bsg::launch_combine_rows(y, (int)dtype, dest, weights, tokens, top_k, K, M, out,
                                         static_cast<hipStream_t>(stream)));
}

extern "C" int bsgemm_combine_backward(const void* dout, const void* y, uint32_t dtype, const int32_t* dest,
                                       const float* weights, int32_t tokens, int32_t top_k, int32_t K,
                                       const int32_t* counts, const int32_t* expert_offsets, int32_t num_experts,
                                       int32_t M, void* dy, float* dweights, void* stream) {
  if (!row_type(dtype)) return BSG_ERR_FMT;
  if (!picks_ok(tokens, top_k) || K <= 0 || K % 8 || K > (INT32_MAX / 4) || num_experts < 1 || num_experts > bsg::kMaxExperts ||
      M < 0 || tokens > bsg::kMaxGradTokens)
    return BSG_ERR_SHAPE;
  if (!counts || !expert_offsets || (tokens > 0 && (!dout || !dest || !weights || !dweights)) ||
      (M > 0 && (!y || !dy)))
    return BSG_ERR_NULL;
  if (!aligned(dout, 16) || !aligned(y, 16) || !aligned(dest, 4) || !aligned(weights, 4) || !aligned(counts, 4) ||
      !aligned(expert_offsets, 4) || !aligned(dy, 16) || !aligned(dweights, 4))
    return BSG_ERR_ALIGN;
  if (int st = check_device()) return st;
  return status(bsg::launch_combine_backward(dout, y, (int)dtype, dest, weights, tokens, top_k, K, counts,
                                             expert_offsets, num_experts, M, dy, dweights,
                                             static_cast<hipStream_t>(stream)));
}

extern "C" int bsgemm_grouped_few_rows(const void* A, const void* a_scales, const void* B, const void* b_scales,
                                       const int32_t* expert_ids, const int32_t* tile_offsets, int32_t num_tiles,
                                       void* C, int32_t M, int32_t N, int32_t K, int32_t num_experts, uint32_t fmt,
                                       void* stream) {
  const uint32_t fa = fmt & 0xF, fb = (fmt >> 4) & 0xF, sk = (fmt >> 8) & 0xF, out = (fmt >> 12) & 0xF;
  if ((fmt >> 16) || !row_type(out) || sk != BSG_SCALE_MX || (fa != BSG_ELEM_E4M3 && fa != BSG_ELEM_E2M1) ||
      (fb != BSG_ELEM_E4M3 && fb != BSG_ELEM_E2M1) || (fa == BSG_ELEM_E4M3 && fb == BSG_ELEM_E4M3))
    return BSG_ERR_FMT;
  if (M < 0 || N <= 0 || K <= 0 || N % 128 || K % 128 || K > kMaxRowsK || num_experts < 1 || num_tiles < 0)
    return BSG_ERR_SHAPE;
  const bool dense = !expert_ids && !tile_offsets;
  const int32_t tiles = dense ? (int32_t)(((long long)M + 127) / 128) : num_tiles;
  if ((long long)tiles * (N / 32) > bsg::kMaxFewRowsCols) return BSG_ERR_SHAPE;
  // an empty tensor's pointer is NULL: a call with nothing to do takes it
  const bool none = M == 0 || tiles == 0;
  if ((!dense && ((num_tiles > 0 && !expert_ids) || !tile_offsets)) || (!none && (!A || !a_scales || !B || !b_scales || !C)))
    return BSG_ERR_NULL;
  if (!aligned(A, 16) || !aligned(B, 16) || !aligned(C, 16) || !aligned(a_scales, 4) || !aligned(b_scales, 4) ||
      !aligned(expert_ids, 4) || !aligned(tile_offsets, 4))
    return BSG_ERR_ALIGN;
  if (none) return BSG_OK;
  bsg::GemmArgs args{};
  if (int st = check_device(&args.num_cus)) return st;
  args.A = A;
  args.a_scales = a_scales;
  args.B = B;
  args.b_scales = b_scales;
  args.expert_ids = dense ? nullptr : expert_ids;
  args.tile_offsets = dense ? nullptr : tile_offsets;
  args.C = C;
  args.M = M;
  args.N = N;
  args.K = K;
  args.num_experts = dense ? 1 : num_experts;
  args.num_tiles = tiles;
  return status(bsg::launch_mx_few_rows(args, (int)fa, (int)fb, (int)out, static_cast<hipStream_t>(stream)));
}
