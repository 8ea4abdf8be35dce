// Grouping of (token, slot) pairs by expert for callers outside the layer: the
// stable counting sort of permute.hip for ids that may lie outside [0, E).
//
// "Kolibri Pre-Training from Scratch" §6.1 sends token t to the experts I_t; the
// German guide "Kolibri 1 im Detail" (section on routing): tokens are brought to
// their experts with no per-expert capacity.  Pair p = t K + k of expert e gets
// the place  offsets[e] + #{p' < p : expert e};  pairs without an expert (on
// another GPU, dropped) are a last bucket with no counts and no places.
//
// All integer work: the order does not depend on the launch.  Lanes of one bucket
// are found with nine ballots over the bits of its number, the rank among them is a
// popcount, and the lowest such lane advances the bucket's running place.
//
// Up to kSmall pairs take one launch: a block to 1024 pairs, one a thread, and every
// block counts all pairs, before its own, its own by wave, and behind.  More take
// two launches, kBlockWaves chunks of consecutive pairs a block, one a wave:
//  1. every block counts its pairs -> block_counts[b][bucket];
//  2. every block reads the whole table (at most kMaxBlocks rows), which gives
//     each bucket's total and its pairs in earlier blocks, scans the totals in
//     expert order, counts its own chunks, and walks them in order.
// Latencies bound it, one call after the other in a graph, loads nearly level: six
// pairs 3.7 us, 6185 5.0 (8.5 in one block, which has four waves a SIMD walk through
// them), 24000 8.6 (9.9 in two launches), 32768 9.9 (10.1 in one), 98304 11.1 (1.2 MB).
// The counts are LDS atomics by bucket, so pairs of one bucket wait for each other:
// 6185 pairs of which half have no expert here 6.8, all with one expert 9.2; 24576 with
// one expert 25 (every block counts them all), 98304 17, 393216 24 (level 15.6).  Every
// token with the same six or five experts costs 0.1 to 0.7 us.  Sixteen waves a block keep
// the table short and the walks shorter: with four (the layer's form, which also makes
// the GEMMs' tile table) 98304 pairs take 14.4 us.
#include <algorithm>

#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kBlockWaves = 16;
constexpr int kThreads = kBlockWaves * kWave;
constexpr int64_t kSmall = 24576;  // pairs of the one-launch form
constexpr int kAllAtOnce = 8;      // its loads of ids in flight
constexpr int64_t kMaxBlocks = 64;
constexpr int kAtOnce = 4;         // loads of ids in flight
constexpr int64_t kChunk = kAtOnce * kWave;  // pairs a wave, at least
constexpr int kBuckets = 385;      // E <= 384, and the pairs without an expert

__device__ __forceinline__ uint32_t bucket_of(int32_t id, int E) {
  return min((uint32_t)id, (uint32_t)E);
}

// Places of up to 64 consecutive pairs: pos holds the wave's running place in
// every bucket.
__device__ __forceinline__ void place_wave(uint32_t e, bool ok, int E, int64_t pair, uint32_t* pos,
                                           int32_t* __restrict__ sorted_src,
                                           int32_t* __restrict__ src_pos) {
  uint64_t same = ballot(ok);
#pragma unroll
  for (int b = 0; b < 9; ++b) {
    const bool bit = (e >> b) & 1u;
    const uint64_t set = ballot(bit);
    same &= bit ? set : ~set;
  }
  const uint64_t lower = same & lanemask_lt();
  if (ok) {
    const uint32_t at = pos[e] + (uint32_t)__popcll(lower);
    sorted_src[at] = e < (uint32_t)E ? (int32_t)pair : -1;
    src_pos[pair] = e < (uint32_t)E ? (int32_t)at : -1;
  }
  __builtin_amdgcn_wave_barrier();
  if (ok && lower == 0ull) pos[e] += (uint32_t)__popcll(same);
  __builtin_amdgcn_wave_barrier();
}

// Totals of the buckets (in tot, by all threads) -> the start of the bucket of
// thread tid, in bucket order.
__device__ __forceinline__ uint32_t bucket_start(const uint32_t* tot, int B, uint32_t* wave_sum) {
  const int tid = threadIdx.x, w = tid >> 6;
  const uint32_t c = tid < B ? tot[tid] : 0u;
  const uint32_t incl = wave_inclusive_sum_dpp_u32(c);
  if (lane_id() == kWave - 1) wave_sum[w] = incl;
  __syncthreads();
  uint32_t before = 0;
  for (int q = 0; q < w; ++q) before += wave_sum[q];
  return before + incl - c;
}

// Exclusive sums over the waves of each bucket's counts, from `start` on.
__device__ __forceinline__ void spread(uint32_t (*pos)[kBuckets], int e, uint32_t start) {
  uint32_t c[kBlockWaves];
#pragma unroll
  for (int q = 0; q < kBlockWaves; ++q) c[q] = pos[q][e];
#pragma unroll
  for (int q = 0; q < kBlockWaves; ++q) {
    pos[q][e] = start;
    start += c[q];
  }
}

__global__ __launch_bounds__(kThreads) void group_small_kernel(
    const int32_t* __restrict__ ids, int pairs, int E, int32_t* __restrict__ counts,
    int32_t* __restrict__ offsets, int32_t* __restrict__ sorted_src,
    int32_t* __restrict__ src_pos) {
  __shared__ uint32_t pos[kBlockWaves][kBuckets];
  __shared__ uint32_t before[kBuckets], after[kBuckets], tot[kBuckets], wave_sum[kBlockWaves];
  const int tid = threadIdx.x, w = tid >> 6, B = E + 1;
  const int own = blockIdx.x * kThreads;  // the block's pairs, one a thread
  uint32_t e[kAllAtOnce], mine = 0;
  auto load = [&](int i0) {
#pragma unroll
    for (int j = 0; j < kAllAtOnce; ++j) {
      const int i = i0 + j * kThreads + tid;
      e[j] = i < pairs ? bucket_of(ids[i], E) : 0u;
    }
  };
  load(0);
  for (int i = tid; i < kBlockWaves * kBuckets; i += kThreads) (&pos[0][0])[i] = 0u;
  if (tid < B) before[tid] = after[tid] = 0u;
  __syncthreads();
  for (int i0 = 0; i0 < pairs; i0 += kAllAtOnce * kThreads) {
    if (i0 > 0) load(i0);
#pragma unroll
    for (int j = 0; j < kAllAtOnce; ++j) {
      const int at = i0 + j * kThreads;
      uint32_t* to = at < own ? before : at > own ? after : pos[w];
      if (at == own) mine = e[j];
      if (at + tid < pairs) atomicAdd(&to[e[j]], 1u);
    }
  }
  __syncthreads();
  if (tid < B) {
    uint32_t sum = before[tid] + after[tid];
#pragma unroll
    for (int q = 0; q < kBlockWaves; ++q) sum += pos[q][tid];
    tot[tid] = sum;
  }
  __syncthreads();
  const uint32_t start = bucket_start(tot, B, wave_sum);
  if (tid < B) {
    if (own == 0) {
      if (tid < E) counts[tid] = (int32_t)tot[tid];
      offsets[tid] = (int32_t)start;
    }
    spread(pos, tid, start + before[tid]);
  }
  __syncthreads();
  place_wave(mine, own + tid < pairs, E, own + tid, pos[w], sorted_src, src_pos);
}

__global__ __launch_bounds__(kThreads) void group_count_kernel(
    const int32_t* __restrict__ ids, int64_t pairs, int E, int64_t cw,
    uint32_t* __restrict__ block_counts) {
  __shared__ uint32_t cnt[kBuckets];
  const int tid = threadIdx.x, B = E + 1;
  if (tid < B) cnt[tid] = 0u;
  __syncthreads();
  const int64_t i0 = (int64_t)blockIdx.x * kBlockWaves * cw;
  const int64_t i1 = min(pairs, i0 + kBlockWaves * cw);
  for (int64_t i = i0 + tid; i < i1; i += kAtOnce * kThreads) {
    int32_t id[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) id[j] = i + j * kThreads < i1 ? ids[i + j * kThreads] : 0;
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
      if (i + j * kThreads < i1) atomicAdd(&cnt[bucket_of(id[j], E)], 1u);
  }
  __syncthreads();
  if (tid < B) block_counts[(size_t)blockIdx.x * B + tid] = cnt[tid];
}

__global__ __launch_bounds__(kThreads) void group_place_kernel(
    const int32_t* __restrict__ ids, int64_t pairs, int E, int64_t cw, int n_blocks,
    const uint32_t* __restrict__ block_counts, int32_t* __restrict__ counts,
    int32_t* __restrict__ offsets, int32_t* __restrict__ sorted_src,
    int32_t* __restrict__ src_pos) {
  __shared__ uint32_t pos[kBlockWaves][kBuckets];
  __shared__ uint32_t half_tot[512], half_pre[512], tot[kBuckets], wave_sum[kBlockWaves];
  const int tid = threadIdx.x, w = tid >> 6, lane = lane_id(), B = E + 1, b = blockIdx.x;
  // the wave's first pairs
  const int64_t i0 = ((int64_t)b * kBlockWaves + w) * cw, i1 = min(pairs, i0 + cw);
  uint32_t x[kAtOnce];
  auto load = [&](int64_t i) {
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int64_t at = i + j * kWave + lane;
      x[j] = at < i1 ? bucket_of(ids[at], E) : 0u;
    }
  };
  load(i0);
  // the table: two threads a bucket, each half of the rows, all loads in flight
  const int e = tid & 511;
  uint32_t sum = 0, pre = 0;
  if (e < B) {
    constexpr int kHalf = (int)(kMaxBlocks / 2);
    const int r0 = (tid >> 9) * kHalf;
    for (int r1 = r0; r1 < min(n_blocks, r0 + kHalf); r1 += 16) {
      uint32_t v[16];
#pragma unroll
      for (int j = 0; j < 16; ++j)
        v[j] = r1 + j < n_blocks ? block_counts[(size_t)(r1 + j) * B + e] : 0u;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        sum += v[j];
        pre += r1 + j < b ? v[j] : 0u;
      }
    }
  }
  for (int i = tid; i < kBlockWaves * kBuckets; i += kThreads) (&pos[0][0])[i] = 0u;
  if (tid >= 512) {
    half_tot[e] = sum;
    half_pre[e] = pre;
  }
  __syncthreads();
  for (int64_t i = i0; i < i1; i += kChunk) {
    if (i > i0) load(i);
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
      if (i + j * kWave + lane < i1) atomicAdd(&pos[w][x[j]], 1u);
  }
  if (tid < B) {
    sum += half_tot[tid];
    pre += half_pre[tid];
    tot[tid] = sum;
  }
  __syncthreads();
  const uint32_t start = bucket_start(tot, B, wave_sum);
  if (tid < B) {
    if (b == 0) {
      if (tid < E) counts[tid] = (int32_t)sum;
      offsets[tid] = (int32_t)start;
    }
    spread(pos, tid, start + pre);
  }
  __syncthreads();
  for (int64_t i = i0; i < i1; i += kChunk) {
    if (cw > kChunk) load(i);
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int64_t at = i + j * kWave;
      if (at < i1) place_wave(x[j], at + lane < i1, E, at + lane, pos[w], sorted_src, src_pos);
    }
  }
}

int64_t chunk_of(int64_t pairs) {
  const int64_t per = (pairs + kBlockWaves * kMaxBlocks - 1) / (kBlockWaves * kMaxBlocks);
  return std::max(kChunk, (per + kWave - 1) / kWave * kWave);
}
int64_t blocks_of(int64_t pairs) {
  const int64_t bp = chunk_of(pairs) * kBlockWaves;
  return (pairs + bp - 1) / bp;
}

}  // namespace

size_t group_work_words(int64_t pairs, int E) {
  return pairs <= kSmall ? 0 : (size_t)blocks_of(pairs) * (size_t)(E + 1);
}

hipError_t launch_group(const int32_t* ids, int64_t pairs, int E, int32_t* counts,
                        int32_t* offsets, int32_t* sorted_src, int32_t* src_pos,
                        uint32_t* block_counts, hipStream_t stream) {
  if (pairs <= kSmall) {
    const int64_t blocks = std::max<int64_t>(1, (pairs + kThreads - 1) / kThreads);
    hipLaunchKernelGGL(group_small_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, stream, ids,
                       (int)pairs, E, counts, offsets, sorted_src, src_pos);
    return hipGetLastError();
  }
  const int64_t cw = chunk_of(pairs), n = blocks_of(pairs);
  const dim3 grid((unsigned)n), block(kThreads);
  hipLaunchKernelGGL(group_count_kernel, grid, block, 0, stream, ids, pairs, E, cw, block_counts);
  hipLaunchKernelGGL(group_place_kernel, grid, block, 0, stream, ids, pairs, E, cw, (int)n,
                     block_counts, counts, offsets, sorted_src, src_pos);
  return hipGetLastError();
}

}  // namespace moe
