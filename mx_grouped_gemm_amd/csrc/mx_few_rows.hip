// MX product for M-tiles of few rows (gfx950): C[rows of tile t] = A[rows] * B[e]^T with e4m3 / e2m1
// elements (one of the two operands e2m1) and one e8m0 scale per 32 K-elements, the operation of
// mx_scaled.hip scheduled for the handful of rows that an expert gets in a decode batch.
//
// In pairs with an e4m3 operand the instruction cuts the product of each K-element, toward zero, at 2^-13 of the
// power of two of the largest among 8 consecutive ones: at most 7 x 2^-13 = 8.5e-4 of sum |a b| (K = 128: 8.4e-6
// for normal values, 2.3e-4 for elements and scales of wide ranges). Products of two e2m1 values span
// 2^7 and lose nothing there: their sums are off by fp32 additions only. mx_scaled.hip carries the same.
// e4m3 x e4m3 is not built: bsgemm_grouped takes it.
//
// There the work is the stream of B (N K / 2 bytes and N K / 32 scales an expert for e2m1), read
// once, so B goes straight from memory to registers: a lane (r16, q) of a wave that owns a fragment
// of 16 columns loads the operand of column r16 for one v_mfma_scale_f32_16x16x128_f8f6f4 step (128
// K-elements) as it lies in memory (e2m1: 16 bytes, the four lanes of a column 64 consecutive ones),
// and reloads the same registers for the next chunk as soon as the instruction has taken them. Two
// steps of e2m1 are the two halves of 128-byte lines: their loads follow each other and are cached
// (with the non-temporal policy the second half is fetched again: 185 against 150 us).
//
// Two schedules, chosen by the number of workgroups that a call gives (see launch):
//  * wide: a workgroup is W = 8, 4 or 2 waves of 32 columns each, over all of K. A chunk (512 K) of the
//    tile's rows is staged in LDS once for all of them, one chunk ahead; so are the scales of 1024 K
//    (from memory in place, a wave's 16 scattered rows of 8 bytes cost the address unit as much as
//    1 KiB of B: 183 -> 142 us with cached pairs, 110 us with staged scales and 8 waves).
//    128 x 8 picks over 32 experts, N 4096, K 7168: 103 us, 5.1 TB/s; a stream of B alone in this lane
//    layout reads 6.1 TB/s.
//  * split: a workgroup is 16 columns, its 8 waves take every 8th chunk of K and add their partial sums
//    in LDS in a fixed order; A comes straight from the caches, 32 rows at a time. For a few tiles of
//    few rows, where latency counts: one token, N 4096, K 7168: 5.7 us in a graph of such calls.
#include "common.h"
#include "ops_launch.h"

namespace bsg {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kSteps = 4;                    // of 128 K-elements in a chunk
constexpr int kTileRows = 128;
constexpr uint32_t kOutside = 0x80000000u;   // past the end of every buffer here: such a load gives 0

// element formats (codes of the C ABI: 1 e4m3, 2 e2m1): code of the f8f6f4 instruction, bytes of a
// row in a step, 16-byte vectors per lane and step. Lane q holds bytes 16 q .. of an e2m1 row, and
// bytes 16 q .. and 64 + 16 q .. of an e4m3 row.
template <int F> struct Elem;
template <> struct Elem<1> { static constexpr int kCode = 0, kStepBytes = 128, kVecs = 2; };
template <> struct Elem<2> { static constexpr int kCode = 4, kStepBytes = 64, kVecs = 1; };

template <int F> struct Step { v4u d[Elem<F>::kVecs]; };

// The lane's operand of the step whose first byte in the lane's row is `off` (the lane's own 16 q included).
template <int F>
__device__ __forceinline__ Step<F> load_step(__amdgpu_buffer_rsrc_t data, uint32_t off) {
  Step<F> r;
#pragma unroll
  for (int h = 0; h < Elem<F>::kVecs; h++) r.d[h] = __builtin_amdgcn_raw_buffer_load_b128(data, off + 64 * h, 0, 0);
  return r;
}

template <int F>
__device__ __forceinline__ v8i operand(const Step<F>& s) {
  const v4u lo = s.d[0], hi = s.d[Elem<F>::kVecs - 1];
  if constexpr (Elem<F>::kVecs == 1) return (v8i){(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], 0, 0, 0, 0};
  return (v8i){(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// B rows as the first operand: lane (r16, q) gets row r16 of A and columns 4 q .. 4 q + 3. The scales
// are in byte 0 of sb and sa.
template <int FA, int FB>
__device__ __forceinline__ v4f multiply(const Step<FB>& b, uint32_t sb, const Step<FA>& a, uint32_t sa, v4f acc) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand<FB>(b), operand<FA>(a), acc, Elem<FB>::kCode,
                                                          Elem<FA>::kCode, 0, (int)sb, 0, (int)sa);
}

// Byte of step s of chunk `ch` in a row of `steps` steps, or kOutside behind its last step.
template <int F>
__device__ __forceinline__ uint32_t step_at(int ch, int s, int steps, uint32_t row) {
  const int at = ch * kSteps + s;
  return at < steps ? row + (uint32_t)at * Elem<F>::kStepBytes : kOutside;
}

// Keeps the compiler from moving memory operations across: the counts of wait_vmcnt below rely on a
// chunk's copies being issued before the loads of B that follow them here.
__device__ __forceinline__ void fence() { asm volatile("" ::: "memory"); }

// ---- wide -------------------------------------------------------------------------------------
constexpr int kWideFrags = 2, kWaveCols = kWideFrags * 16;
constexpr int kWideSteps = 4;                // steps of a chunk: what is staged of A at a time
constexpr int kGroup = 8;                    // steps whose scales are staged at a time: 32 bytes a row
constexpr int kGroupChunks = kGroup / kWideSteps;

// LDS of a workgroup. Two stages of A: a chunk of the tile's rows in 16-byte slots, slot c of row r at
// place c ^ (r % 16) of its row, which spreads one slot of a fragment's 16 rows over all banks. Two
// stages of scales: a group of the tile's rows, then of every wave's columns, 32 bytes each.
template <int FA, int W> struct WideLds {
  static constexpr int kRowBytes = kWideSteps * Elem<FA>::kStepBytes, kSlots = kRowBytes / 16;
  static constexpr int kStage = kTileRows * kRowBytes;
  static constexpr int kScaleRow = 4 * kGroup, kScales = 2 * kStage, kScaleStage = (kTileRows + W * kWaveCols) * kScaleRow;
  static constexpr int kBytes = kScales + 2 * kScaleStage;
  static_assert(kBytes <= 160 * 1024, "LDS");
  static_assert(kSlots % 16 == 0, "slots are exchanged within 16");
  static __device__ __forceinline__ int place(int r, int c) { return c ^ (r & 15); }
};

// Copies chunk `ch` of 16 NF rows, shared by the waves: 1 KiB an instruction.
template <int FA, int W, int NF>
__device__ __forceinline__ void wide_copy_a(uint8_t* lds, __amdgpu_buffer_rsrc_t a, int ch, int steps, int wave, int lane) {
  using L = WideLds<FA, W>;
  constexpr int kRowsEach = 1024 / L::kRowBytes, kCopies = 16 * NF / kRowsEach;
  const uint32_t row_bytes = (uint32_t)steps * Elem<FA>::kStepBytes;
#pragma unroll
  for (int k = 0; k < (kCopies + W - 1) / W; k++) {
    const int copy = k * W + wave;
    if (copy >= kCopies) break;
    const int r = copy * kRowsEach + lane / L::kSlots, c = L::place(r, lane % L::kSlots);
    const int s = ch * kWideSteps + c / (Elem<FA>::kStepBytes / 16);
    buf2lds16(a, s < steps ? r * row_bytes + (uint32_t)ch * L::kRowBytes + c * 16 : kOutside, 0, as_lds(lds + copy * 1024));
  }
}

// Copies the scales of group g: of A, 32 rows an instruction, and of every wave's own columns.
// A group that ends behind K takes bytes of the next row along (or zeros behind the last): no step uses them.
template <int W, int NF, int kScaleRow>
__device__ __forceinline__ void wide_copy_scales(uint8_t* lds, __amdgpu_buffer_rsrc_t sa, __amdgpu_buffer_rsrc_t sb, int g,
                                                 int steps, int wave, int lane) {
  const uint32_t in = (uint32_t)g * kScaleRow + (lane & 1) * 16;
  const uint32_t out = g * kGroup < steps ? 0 : kOutside;
#pragma unroll
  for (int k = 0; k < (NF + 2 * W - 1) / (2 * W); k++) {
    const int rows32 = k * W + wave;
    if (rows32 * 32 < 16 * NF)
      buf2lds16(sa, (uint32_t)(rows32 * 32 + lane / 2) * steps * 4 + in + out, 0, as_lds(lds + rows32 * 1024));
  }
#pragma unroll
  for (int c = 0; c < kWaveCols / 32; c++)
    buf2lds16(sb, (uint32_t)(wave * kWaveCols + c * 32 + lane / 2) * steps * 4 + in + out, 0,
              as_lds(lds + kTileRows * kScaleRow + (wave * (kWaveCols / 32) + c) * 1024));
}

// 16 NF rows (those of the buffers a and sa; further ones read as zeros) times the workgroup's columns.
template <int FA, int FB, int OUT, int W, int NF>
__device__ __forceinline__ void wide_tile(uint8_t* lds, __amdgpu_buffer_rsrc_t a, __amdgpu_buffer_rsrc_t sa,
                                          __amdgpu_buffer_rsrc_t b, __amdgpu_buffer_rsrc_t sb, int steps, int live,
                                          void* C, size_t c_off, int N, int cols) {
  using L = WideLds<FA, W>;
  const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t b_bytes = (uint32_t)steps * Elem<FB>::kStepBytes;
  uint32_t b_row[kWideFrags];
#pragma unroll
  for (int c = 0; c < kWideFrags; c++) b_row[c] = (wave * kWaveCols + c * 16 + r16) * b_bytes + 16 * q;
  v4f acc[NF][kWideFrags];
#pragma unroll
  for (int f = 0; f < NF; f++)
#pragma unroll
    for (int c = 0; c < kWideFrags; c++) acc[f][c] = (v4f){0.f, 0.f, 0.f, 0.f};

  Step<FB> bs[kWideSteps][kWideFrags];
  auto load_b = [&](int s, int ch) {
#pragma unroll
    for (int c = 0; c < kWideFrags; c++) {
      const int at = ch * kWideSteps + s;
      bs[s][c] = load_step<FB>(b, at < steps ? b_row[c] + (uint32_t)at * Elem<FB>::kStepBytes : kOutside);
    }
  };
  // issue order, here as in the loop: scales, A's chunk, B's
  wide_copy_scales<W, NF, L::kScaleRow>(lds + L::kScales, sa, sb, 0, steps, wave, lane);
  wide_copy_a<FA, W, NF>(lds, a, 0, steps, wave, lane);
#pragma unroll
  for (int s = 0; s < kWideSteps; s++) {
    fence();
    load_b(s, 0);
  }
  // loads of B issued after a chunk's copies: what may still be outstanding when the chunk is needed
  constexpr int kBehind = kWideSteps * kWideFrags * Elem<FB>::kVecs;
  const int chunks = (steps + kWideSteps - 1) / kWideSteps;
  for (int ch = 0; ch < chunks; ch++) {
    fence();
    wait_vmcnt<kBehind>();                   // this wave's copies of the chunk have landed
    barrier();                               // ... every wave's, and the other stages are free
    const uint8_t* st = lds + (ch & 1) * L::kStage;
    const int g = ch / kGroupChunks;
    const uint8_t* sc = lds + L::kScales + (g & 1) * L::kScaleStage + ch % kGroupChunks * kWideSteps * 4;
    if (ch % kGroupChunks == 0)
      wide_copy_scales<W, NF, L::kScaleRow>(lds + L::kScales + (~g & 1) * L::kScaleStage, sa, sb, g + 1, steps, wave, lane);
    wide_copy_a<FA, W, NF>(lds + (~ch & 1) * L::kStage, a, ch + 1, steps, wave, lane);
    fence();
#pragma unroll
    for (int s = 0; s < kWideSteps; s++) {
      if (ch * kWideSteps + s < steps) {
        uint32_t b_scale[kWideFrags];
#pragma unroll
        for (int c = 0; c < kWideFrags; c++)
          b_scale[c] = *(const uint32_t*)(sc + (kTileRows + wave * kWaveCols + c * 16 + r16) * L::kScaleRow + 4 * s) >> (8 * q);
#pragma unroll
        for (int f = 0; f < NF; f++) {
          const int r = f * 16 + r16;
          Step<FA> as;
#pragma unroll
          for (int h = 0; h < Elem<FA>::kVecs; h++)
            as.d[h] = *(const v4u*)(st + r * L::kRowBytes + 16 * L::place(r, s * (Elem<FA>::kStepBytes / 16) + 4 * h + q));
          const uint32_t a_scale = *(const uint32_t*)(sc + r * L::kScaleRow + 4 * s) >> (8 * q);
#pragma unroll
          for (int c = 0; c < kWideFrags; c++) acc[f][c] = multiply<FA, FB>(bs[s][c], b_scale[c], as, a_scale, acc[f][c]);
        }
      }
      // an e2m1 step is half a 128-byte line: both halves are reloaded together
      if (Elem<FB>::kVecs == 2) {
        load_b(s, ch + 1);
      } else if (s & 1) {
        load_b(s - 1, ch + 1);
        load_b(s, ch + 1);
      }
      fence();
    }
  }
  wait_vmcnt<0>();                           // the copies behind the last chunk have landed
#pragma unroll
  for (int f = 0; f < NF; f++) {
    if (f * 16 + r16 >= live) continue;
#pragma unroll
    for (int c = 0; c < kWideFrags; c++)
      if (wave * kWaveCols + c * 16 < cols)
        store4<OUT>(C, c_off + (size_t)(f * 16 + r16) * N + wave * kWaveCols + c * 16 + 4 * q, acc[f][c][0], acc[f][c][1],
                    acc[f][c][2], acc[f][c][3]);
  }
}

// Row buffers of a pass over rows [row, row + live).
struct ARows { __amdgpu_buffer_rsrc_t data, scales; };
template <int FA>
__device__ __forceinline__ ARows a_rows(const GemmArgs& g, size_t row, int live, int steps) {
  const size_t bytes = (size_t)steps * Elem<FA>::kStepBytes;
  return {make_rsrc((const uint8_t*)g.A + row * bytes, live * bytes),
          make_rsrc((const uint8_t*)g.a_scales + row * steps * 4, (uint64_t)live * steps * 4)};
}

template <int FA, int FB, int OUT, int W>
__global__ __launch_bounds__(W* kWave) void mx_few_rows_wide_kernel(GemmArgs g, int n_blocks) {
  constexpr int kWideCols = W * kWaveCols;
  __shared__ __attribute__((aligned(16))) uint8_t lds[WideLds<FA, W>::kBytes];
  const int t = blockIdx.x / n_blocks, n0 = (blockIdx.x % n_blocks) * kWideCols;
  const TileRows tr = tile_rows(g.expert_ids, g.tile_offsets, t, g.M, kTileRows, g.num_experts);
  if (tr.rows <= 0) return;
  const int e = __builtin_amdgcn_readfirstlane(tr.expert);
  const int row0 = __builtin_amdgcn_readfirstlane(tr.row0), rows = __builtin_amdgcn_readfirstlane(tr.rows);
  const int steps = g.K / 128;
  const size_t col = (size_t)e * g.N + n0, b_bytes = (size_t)steps * Elem<FB>::kStepBytes;
  const int cols = min(kWideCols, g.N - n0);       // further columns read as zeros and are not stored
  const auto b = make_rsrc((const uint8_t*)g.B + col * b_bytes, cols * b_bytes);
  const auto sb = make_rsrc((const uint8_t*)g.b_scales + col * steps * 4, (uint64_t)cols * steps * 4);
  const ARows a = a_rows<FA>(g, (size_t)row0, rows, steps);
  const size_t c_off = (size_t)row0 * g.N + n0;
  switch ((rows + 15) / 16) {
    case 1: wide_tile<FA, FB, OUT, W, 1>(lds, a.data, a.scales, b, sb, steps, rows, g.C, c_off, g.N, cols); break;
    case 2: wide_tile<FA, FB, OUT, W, 2>(lds, a.data, a.scales, b, sb, steps, rows, g.C, c_off, g.N, cols); break;
    case 3: wide_tile<FA, FB, OUT, W, 3>(lds, a.data, a.scales, b, sb, steps, rows, g.C, c_off, g.N, cols); break;
    case 4: wide_tile<FA, FB, OUT, W, 4>(lds, a.data, a.scales, b, sb, steps, rows, g.C, c_off, g.N, cols); break;
    case 5:
    case 6: wide_tile<FA, FB, OUT, W, 6>(lds, a.data, a.scales, b, sb, steps, rows, g.C, c_off, g.N, cols); break;
    default: wide_tile<FA, FB, OUT, W, 8>(lds, a.data, a.scales, b, sb, steps, rows, g.C, c_off, g.N, cols); break;
  }
}

// ---- split ------------------------------------------------------------------------------------
constexpr int kSplitWaves = 8, kSplitCols = 16, kSplitRows = 32;
constexpr int kPitch = kSplitCols + 4;       // floats per row of a wave's partial sums in LDS

// A wave's share of NF fragments of 16 x 16: chunks wave, wave + waves, ... of K; the sums go to red.
template <int FA, int FB, int NF>
__device__ __forceinline__ void split_pass(float* red, const ARows& a, __amdgpu_buffer_rsrc_t b, __amdgpu_buffer_rsrc_t sb,
                                           int steps, int wave) {
  const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
  const uint32_t a_bytes = (uint32_t)steps * Elem<FA>::kStepBytes;
  const uint32_t b_row = r16 * (uint32_t)steps * Elem<FB>::kStepBytes + 16 * q, s_row = r16 * (uint32_t)steps * 4;
  v4f acc[NF];
  Step<FB> bs[kSteps];
  Step<FA> as[kSteps][NF];
  v4u b_scale, a_scale[NF];
  const int chunks = (steps + kSteps - 1) / kSteps;
  auto load_scales = [&](int ch) {
    const uint32_t at = ch < chunks ? (uint32_t)ch * 16 : kOutside;
    b_scale = __builtin_amdgcn_raw_buffer_load_b128(sb, s_row + at, 0, 0);
#pragma unroll
    for (int f = 0; f < NF; f++)
      a_scale[f] = __builtin_amdgcn_raw_buffer_load_b128(a.scales, f * 64 * (uint32_t)steps + s_row + at, 0, 0);
  };
  auto load = [&](int ch, int s) {
    bs[s] = load_step<FB>(b, step_at<FB>(ch, s, steps, b_row));
#pragma unroll
    for (int f = 0; f < NF; f++)
      as[s][f] = load_step<FA>(a.data, step_at<FA>(ch, s, steps, (f * 16 + r16) * a_bytes + 16 * q));
  };
#pragma unroll
  for (int f = 0; f < NF; f++) acc[f] = (v4f){0.f, 0.f, 0.f, 0.f};
  load_scales(wave);
#pragma unroll
  for (int s = 0; s < kSteps; s++) load(wave, s);
  for (int ch = wave; ch < chunks; ch += kSplitWaves) {
    uint32_t sbv[kSteps], sav[kSteps][NF];
#pragma unroll
    for (int s = 0; s < kSteps; s++) {
      sbv[s] = b_scale[s] >> (8 * q);
#pragma unroll
      for (int f = 0; f < NF; f++) sav[s][f] = a_scale[f][s] >> (8 * q);
    }
    load_scales(ch + kSplitWaves);
#pragma unroll
    for (int s = 0; s < kSteps; s++) {
      if (ch * kSteps + s < steps) {
#pragma unroll
        for (int f = 0; f < NF; f++) acc[f] = multiply<FA, FB>(bs[s], sbv[s], as[s][f], sav[s][f], acc[f]);
      }
      load(ch + kSplitWaves, s);
    }
  }
#pragma unroll
  for (int f = 0; f < NF; f++) *(v4f*)(red + (f * 16 + r16) * kPitch + 4 * q) = acc[f];
}

template <int FA, int FB, int OUT>
__global__ __launch_bounds__(kSplitWaves* kWave) void mx_few_rows_split_kernel(GemmArgs g, int n_blocks) {
  __shared__ __attribute__((aligned(16))) float red[kSplitWaves][kSplitRows * kPitch];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = blockIdx.x / n_blocks, n0 = (blockIdx.x % n_blocks) * kSplitCols;
  const TileRows tr = tile_rows(g.expert_ids, g.tile_offsets, t, g.M, kTileRows, g.num_experts);
  if (tr.rows <= 0) return;
  const int e = __builtin_amdgcn_readfirstlane(tr.expert);
  const int row0 = __builtin_amdgcn_readfirstlane(tr.row0), rows = __builtin_amdgcn_readfirstlane(tr.rows);
  const int steps = g.K / 128;
  const size_t col = (size_t)e * g.N + n0, b_bytes = (size_t)steps * Elem<FB>::kStepBytes;
  const auto b = make_rsrc((const uint8_t*)g.B + col * b_bytes, kSplitCols * b_bytes);
  const auto sb = make_rsrc((const uint8_t*)g.b_scales + col * steps * 4, (uint64_t)kSplitCols * steps * 4);
  for (int m0 = 0; m0 < rows; m0 += kSplitRows) {
    const int live = min(kSplitRows, rows - m0);
    const size_t row = (size_t)(row0 + m0);
    const ARows a = a_rows<FA>(g, row, live, steps);
    if (m0) __syncthreads();                 // the pass before has been added up
    if (live <= 16) split_pass<FA, FB, 1>(red[wave], a, b, sb, steps, wave);
    else split_pass<FA, FB, 2>(red[wave], a, b, sb, steps, wave);
    __syncthreads();
    for (int i = threadIdx.x; i < live * (kSplitCols / 4); i += kSplitWaves * kWave) {
      const int r = i / (kSplitCols / 4), c = i % (kSplitCols / 4) * 4;
      v4f s = *(const v4f*)(red[0] + r * kPitch + c);
#pragma unroll
      for (int w = 1; w < kSplitWaves; w++) s += *(const v4f*)(red[w] + r * kPitch + c);
      store4<OUT>(g.C, (row + r) * g.N + n0 + c, s[0], s[1], s[2], s[3]);
    }
  }
}

static_assert(2 * kMaxFewRowsCols * kSplitWaves * kWave <= kMaxThreads, "the split schedule's grid, the larger one");

template <int FA, int FB, int OUT, int W>
hipError_t launch_wide(const GemmArgs& a, int n_blocks, hipStream_t s) {
  hipLaunchKernelGGL((mx_few_rows_wide_kernel<FA, FB, OUT, W>), dim3((unsigned)(a.num_tiles * n_blocks)), dim3(W * kWave), 0, s,
                     a, n_blocks);
  return hipGetLastError();
}

// The narrowest of 2, 4 and 8 waves that give at most one workgroup per compute unit (8 if none does):
// wider ones stage A for more columns, narrower ones occupy more units; but the split schedule below
// half a workgroup of 2 waves per unit. Measured (us, in a graph of calls on different weights; e2m1 x
// e2m1, K 7168 and N 4096 but where said; 2, 4, 8 waves, split):
//   1 x 1                           11.8   15.9   29.2    5.7
//   1 x 64                          18.8   20.2   32.6   15.2
//   2 x 40, N 2048, K 4096          10.1   12.0   19.8    9.4
//   2 x 64                          21.1   23.0   36.2   27.2
//   3 x 8                           16.7   20.9   37.0   15.3
//   8 x 16, N 2048, K 4096          10.3   13.1   21.0   15.3
//   4 x 8                           17.8   21.6   37.7   19.8
//   6 x 16                          25.8   23.3   39.1   31.6
//   1 x 8, N 28672                  24.6   23.9   39.3   31.3
//   8 x 32                          28.0   26.7   41.3   54.4
//   9 x 8, K 4096                   25.6   24.7   23.0   27.6
//   12 x 20                         48.4   46.5   43.4   66.7
//   32 x 32                        104.1  101.2   99.9  207.7
//   32 x 100                       166.2  134.9  125.5  680.8
template <int FA, int FB, int OUT>
hipError_t launch(const GemmArgs& a, hipStream_t s) {
  auto n_blocks = [&](int waves) { return (a.N + waves * kWaveCols - 1) / (waves * kWaveCols); };
  const long long tiles = a.num_tiles < a.M ? a.num_tiles : a.M;      // a tile that is used has a row
  auto blocks = [&](int waves) { return tiles * n_blocks(waves); };
  if (blocks(4) > a.num_cus) return launch_wide<FA, FB, OUT, 8>(a, n_blocks(8), s);
  if (blocks(2) > a.num_cus) return launch_wide<FA, FB, OUT, 4>(a, n_blocks(4), s);
  if (2 * blocks(2) >= a.num_cus) return launch_wide<FA, FB, OUT, 2>(a, n_blocks(2), s);
  const int split = a.N / kSplitCols;
  hipLaunchKernelGGL((mx_few_rows_split_kernel<FA, FB, OUT>), dim3((unsigned)(a.num_tiles * split)),
                     dim3(kSplitWaves * kWave), 0, s, a, split);
  return hipGetLastError();
}

template <int FA, int FB>
hipError_t launch_out(const GemmArgs& a, int out, hipStream_t s) {
  switch (out) {
    case kOutF32: return launch<FA, FB, kOutF32>(a, s);
    case kOutBF16: return launch<FA, FB, kOutBF16>(a, s);
    case kOutF16: return launch<FA, FB, kOutF16>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_mx_few_rows(const GemmArgs& a, int fmt_a, int fmt_b, int out, hipStream_t s) {
  switch (fmt_a * 4 + fmt_b) {
    case 6: return launch_out<1, 2>(a, out, s);
    case 9: return launch_out<2, 1>(a, out, s);
    case 10: return launch_out<2, 2>(a, out, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace bsg
