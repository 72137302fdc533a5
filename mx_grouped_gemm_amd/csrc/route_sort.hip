// Stable sort of top-k picks by expert (gfx950): per-expert counts, group offsets, the M-tile map
// and the row of every pick, in one to three launches.
//
//   counts[e]         picks i with ids[i] = e (ids outside [0, E) are dropped)
//   expert_offsets    exclusive sums of the groups' rows (padded: whole 128-row tiles)
//   tile_offsets, expert_ids   as the tile map of counts
//   dest[i]           expert_offsets[e] + number of picks i' < i with ids[i'] = e; -1 where dropped or >= M
//
// The picks are cut into chunks, one per workgroup; a chunk's waves take consecutive segments of
// it. In a wave 64 picks are matched against each other by ballots over the bits of
// their ids, which gives each pick its place among equals without atomics, so the order is the
// picks' own on every call. With one chunk everything happens in one launch (a decode batch); with
// more, a first launch writes every chunk's histogram, and each workgroup of the last sums the
// chunks before its own. Where that is much (see kMostCounts), a launch in between turns the histograms into
// these sums, so that the work grows with the picks, not with their square. What bounds it is the latency of
// these steps, not their bytes.
#include "ops_launch.h"
#include "quant.h"

namespace bsg {
namespace {

constexpr int kSteps = 8;                    // most 64-pick steps of a wave
constexpr int kSegment = kSteps * kWave;     // most consecutive picks per wave
constexpr int kTile = 128;

// Waves per workgroup: the LDS holds a counter per wave and expert, so above 2048 experts there is
// room for 4 waves' only.
int waves_for(int E) { return E <= 2048 ? 8 : 4; }
int chunks_of(int n, int E) {
  const int chunk = waves_for(E) * kSegment;
  return n <= chunk ? 1 : (n + chunk - 1) / chunk;
}
// Most counts (chunks x experts) that every workgroup of the last launch sums itself. Measured (us a call in a
// graph; itself, with the launch in between):
//     4096 counts, 256 experts   18.3   19.7        16384 counts, 256 experts   26.4   20.1
//     8192 counts,   8 experts   31.0   34.7        32768 counts,  32 experts   61.3   39.3
//     8192 counts,  32 experts   19.1   18.2       262144 counts, 256 experts    304   47.4
//     8192 counts, 512 experts   22.4   20.8      2097152 counts, 4096 experts  5475   83.9
constexpr int kMostCounts = 8192;

// place[waves][E], row_start[E + 1], tile_start[E + 1], total[E], before[E]
constexpr size_t lds_bytes(int waves, int E) { return ((size_t)waves * E + 2 * (E + 1) + 2 * E) * sizeof(int); }
static_assert(lds_bytes(8, 2048) + 64 <= 160 * 1024 && lds_bytes(4, 4096) + 64 <= 160 * 1024, "LDS");

// Lanes of the wave whose id equals this lane's; id is below 2^bits, dead lanes match nothing.
__device__ __forceinline__ uint64_t match(int id, bool live, int bits) {
  uint64_t m = __ballot(live);
  for (int b = 0; b < bits; b++) {
    const bool one = (id >> b) & 1;
    const uint64_t v = __ballot(one);
    m &= one ? v : ~v;
  }
  return live ? m : 0;
}

__device__ __forceinline__ uint64_t below(int lane) { return (1ull << lane) - 1; }

// The wave's picks begin .. begin + 64 steps - 1 (below n), all loaded at once: ids outside [0, E) and
// missing picks become -1.
__device__ __forceinline__ void load_picks(const int32_t* __restrict__ ids, int n, int begin, int steps, int E,
                                           int (&id)[kSteps]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int k = 0; k < kSteps; k++) {
    const int i = begin + k * kWave + lane;
    id[k] = k < steps && i < n ? ids[i] : -1;
  }
#pragma unroll
  for (int k = 0; k < kSteps; k++)
    if (id[k] < 0 || id[k] >= E) id[k] = -1;
}

// Adds the wave's picks to hist[E], one addition for each distinct id of a step.
__device__ __forceinline__ void histogram(const int (&id)[kSteps], int steps, int bits, int* hist) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int k = 0; k < kSteps; k++) {
    if (k >= steps) break;
    const bool live = id[k] >= 0;
    const uint64_t m = match(id[k], live, bits);
    if (live && (m & below(lane)) == 0) atomicAdd(&hist[id[k]], __popcll(m));
  }
}

template <int kWaves>
__global__ __launch_bounds__(kWaves* kWave) void route_chunk_counts_kernel(const int32_t* __restrict__ ids, int n, int E,
                                                                      int bits, int32_t* __restrict__ chunk_counts) {
  constexpr int kThreads = kWaves * kWave;
  extern __shared__ int hist[];
  int id[kSteps];
  load_picks(ids, n, (blockIdx.x * kWaves + (threadIdx.x >> 6)) * kSegment, kSteps, E, id);
  for (int e = threadIdx.x; e < E; e += kThreads) hist[e] = 0;
  __syncthreads();
  histogram(id, kSteps, bits, hist);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kThreads) chunk_counts[(long long)blockIdx.x * E + e] = hist[e];
}

// Each chunk's row of chunk_counts becomes the picks of every expert in the chunks before it, and the row behind
// them the totals: 64 experts per workgroup, a 16th of the chunks per wave, 16 loads on their way at once.
__global__ __launch_bounds__(1024) void route_chunk_starts_kernel(int32_t* chunk_counts, int chunks, int E) {
  __shared__ int part[16][kWave];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e = blockIdx.x * kWave + lane;
  const int per = (chunks + 15) / 16, first = wave * per, last = min(first + per, chunks);
  auto load = [&](int c0, int (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 16; i++) v[i] = e < E && c0 + i < last ? chunk_counts[(long long)(c0 + i) * E + e] : 0;
  };
  int sum = 0, v[16];
  for (int c0 = first; c0 < last; c0 += 16) {
    load(c0, v);
#pragma unroll
    for (int i = 0; i < 16; i++) sum += v[i];
  }
  part[wave][lane] = sum;
  __syncthreads();
  int next = 0;
  for (int w = 0; w < wave; w++) next += part[w][lane];
  for (int c0 = first; c0 < last; c0 += 16) {
    load(c0, v);
#pragma unroll
    for (int i = 0; i < 16; i++) {
      if (e < E && c0 + i < last) chunk_counts[(long long)(c0 + i) * E + e] = next;
      next += v[i];
    }
  }
  if (wave == 15 && e < E) chunk_counts[(long long)chunks * E + e] = next;
}

// segment: consecutive picks per wave, a multiple of 64 (with one chunk, what spreads it over all waves).
// starts: chunk_counts are the sums of route_chunk_starts_kernel.
template <int kWaves>
__global__ __launch_bounds__(kWaves* kWave) void route_sort_kernel(
    const int32_t* __restrict__ ids, int n, int segment, int E, int bits, int T, int padded, int M, int starts,
    const int32_t* __restrict__ chunk_counts, int32_t* __restrict__ counts, int32_t* __restrict__ expert_offsets,
    int32_t* __restrict__ tile_offsets, int32_t* __restrict__ expert_ids, int32_t* __restrict__ dest) {
  constexpr int kThreads = kWaves * kWave;
  extern __shared__ int lds[];
  __shared__ int wave_rows[kWaves], wave_tiles[kWaves];
  int* place = lds;
  int* row_start = lds + kWaves * E;
  int* tile_start = row_start + E + 1;
  int* total_of = tile_start + E + 1;              // picks of each expert, and those of earlier chunks
  int* before_of = total_of + E;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int chunk = blockIdx.x, chunks = gridDim.x;
  const int begin = (chunk * kWaves + wave) * segment, steps = segment / kWave;
  int id[kSteps];
  load_picks(ids, n, begin, steps, E, id);
  for (int i = tid; i < kWaves * E; i += kThreads) place[i] = 0;
  if (starts) {
    for (int e = tid; e < E; e += kThreads) {
      total_of[e] = chunk_counts[(long long)chunks * E + e];
      before_of[e] = chunk_counts[(long long)chunk * E + e];
    }
  } else {
    for (int i = tid; i < 2 * E; i += kThreads) total_of[i] = 0;
  }
  __syncthreads();
  int* mine = place + wave * E;                    // next row of this wave's picks of an expert
  histogram(id, steps, bits, mine);
  if (chunks > 1 && !starts) {
    const int all = chunks * E, earlier = chunk * E;      // all: at most kMostCounts
    for (int i = tid; i < all; i += kThreads) {
      const int v = chunk_counts[i], e = i % E;
      if (v) {
        atomicAdd(&total_of[e], v);
        if (i < earlier) atomicAdd(&before_of[e], v);
      }
    }
  }
  __syncthreads();

  // per expert: total, rows before this chunk, and the waves' first places; experts in rounds of
  // kThreads, each round's groups laid out by a scan over the workgroup
  int row_base = 0, tile_base = 0;
  for (int e0 = 0; e0 < E; e0 += kThreads) {
    const int e = e0 + tid;
    int total = 0, before = 0;
    if (e < E) {
      total = total_of[e];
      before = before_of[e];
      if (chunks == 1)
        for (int w = 0; w < kWaves; w++) total += place[w * E + e];
    }
    const int tiles = (total + kTile - 1) / kTile;
    const int rows = padded ? tiles * kTile : total;
    int r = rows, t = tiles;                       // inclusive sums over the wave
    for (int d = 1; d < 64; d <<= 1) {
      const int ur = __shfl_up(r, d), ut = __shfl_up(t, d);
      if (lane >= d) {
        r += ur;
        t += ut;
      }
    }
    if (lane == 63) {
      wave_rows[wave] = r;
      wave_tiles[wave] = t;
    }
    __syncthreads();
    int row0 = row_base + r - rows, tile0 = tile_base + t - tiles;
    for (int w = 0; w < kWaves; w++) {
      if (w < wave) {
        row0 += wave_rows[w];
        tile0 += wave_tiles[w];
      }
      row_base += wave_rows[w];
      tile_base += wave_tiles[w];
    }
    if (e < E) {
      row_start[e] = row0;
      tile_start[e] = tile0;
      if (chunk == 0) {
        counts[e] = total;
        expert_offsets[e] = row0;
      }
      int next = row0 + before;
      for (int w = 0; w < kWaves; w++) {
        const int v = place[w * E + e];
        place[w * E + e] = next;
        next += v;
      }
    }
    __syncthreads();                               // wave_rows / wave_tiles are free again
  }
  if (tid == 0) {
    row_start[E] = row_base;
    tile_start[E] = tile_base;
    if (chunk == 0) expert_offsets[E] = row_base;
  }
  __syncthreads();

  // rows of the picks, 64 at a time in order: place[e] moves on by the number of equal picks
#pragma unroll
  for (int k = 0; k < kSteps; k++) {
    if (k >= steps) break;
    const int i = begin + k * kWave + lane;
    const bool live = id[k] >= 0;
    const uint64_t m = match(id[k], live, bits);
    int row = -1;
    if (live) row = mine[id[k]] + __popcll(m & below(lane));
    __builtin_amdgcn_wave_barrier();               // every lane has read before a leader writes
    if (live && (m & below(lane)) == 0) mine[id[k]] = row + __popcll(m);
    __builtin_amdgcn_wave_barrier();
    if (i < n) dest[i] = row < M ? row : -1;
  }

  // tile map, shared by the workgroups: the tile's expert is the last that starts at or before it
  for (long long t = chunk * kThreads + tid; t <= T; t += chunks * kThreads) {      // T may be near 2^31
    int e = -1, start = row_base;
    if (t < tile_base) {
      int a = 0, b = E;                            // tile_start[a] <= t < tile_start[b]
      while (b - a > 1) {
        const int mid = (a + b) >> 1;
        if (tile_start[mid] <= t) a = mid; else b = mid;
      }
      e = a;
      start = row_start[e] + ((int)t - tile_start[e]) * kTile;
    }
    tile_offsets[t] = padded ? (int32_t)(t * kTile) : start;
    if (t < T) expert_ids[t] = e;
  }
}

template <int kWaves>
hipError_t launch(const int32_t* ids, int n, int E, int T, int padded, int M, int32_t* counts, int32_t* expert_offsets,
                  int32_t* tile_offsets, int32_t* expert_ids, int32_t* dest, int32_t* workspace, hipStream_t s) {
  int bits = 0;
  while ((1 << bits) < E) bits++;
  const int chunks = chunks_of(n, E);
  const bool starts = chunks > 1 && (long long)chunks * E > kMostCounts;
  const int segment = chunks > 1 ? kSegment : max(1, (n + kWaves * kWave - 1) / (kWaves * kWave)) * kWave;
  const dim3 grid(chunks), block(kWaves * kWave);
  if (chunks > 1) {
    hipLaunchKernelGGL(route_chunk_counts_kernel<kWaves>, grid, block, E * sizeof(int), s, ids, n, E, bits, workspace);
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (starts) {
    hipLaunchKernelGGL(route_chunk_starts_kernel, dim3((E + kWave - 1) / kWave), dim3(1024), 0, s, workspace, chunks, E);
    if (hipError_t e = hipGetLastError()) return e;
  }
  hipLaunchKernelGGL(route_sort_kernel<kWaves>, grid, block, lds_bytes(kWaves, E), s, ids, n, segment, E, bits, T, padded,
                     M, starts ? 1 : 0, workspace, counts, expert_offsets, tile_offsets, expert_ids, dest);
  return hipGetLastError();
}

}  // namespace

size_t route_sort_workspace_bytes(int n, int E) {
  const int chunks = chunks_of(n, E);
  return chunks > 1 ? ((size_t)chunks + 1) * E * sizeof(int32_t) : 0;      // the histograms and their totals
}

hipError_t launch_route_sort(const int32_t* ids, int n, int E, int T, int padded, int M, int32_t* counts,
                             int32_t* expert_offsets, int32_t* tile_offsets, int32_t* expert_ids, int32_t* dest,
                             int32_t* workspace, hipStream_t s) {
  return waves_for(E) == 8
             ? launch<8>(ids, n, E, T, padded, M, counts, expert_offsets, tile_offsets, expert_ids, dest, workspace, s)
             : launch<4>(ids, n, E, T, padded, M, counts, expert_offsets, tile_offsets, expert_ids, dest, workspace, s);
}

}  // namespace bsg
