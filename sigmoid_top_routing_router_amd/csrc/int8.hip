// Products in 8-bit integers with a scale for each row (token) and each output
// channel, dense or grouped by expert, and the row quantiser.
//
// A row x becomes s = amax|x| (1 / 127), the reciprocal and the product rounded to
// fp32, and the integers q = rne(x / s) in [-127, 127]; weights the same way, a row
// of W being an output channel.  Then
//   y_tc = s_t s_c sum_k q_tk q_ck,
// the sum exact in 32-bit integers (|sum| <= 2^14 k < 2^31 for k <= 65536; the
// code -128 of a caller's own included), converted to fp32 (one rounding of
// 2^-24 above 2^24), times both scales, and y rounded to bf16 once.  With a
// second weight: silu(y) * y', formed in fp32 ("Kolibri 1 im Detail", routing
// section, SwiGLU paragraph).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "common.h"
#include "fp8_codes.h"
#include "gemm_args.h"
#include "kernels.h"
#include "lane_swaps.h"

namespace moe {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));
typedef float f32x4_t __attribute__((ext_vector_type(4), aligned(4)));

constexpr float kInt8Max = 127.0f;

// Four integers.  The quotient v / s rounded to fp32 as q = v y, q + (v - s q) y
// with y = 1 / s (three operations in the place of a division's; the residual is
// exact but for 9 of the 2^14 pairs of significands of v and of the largest value,
// where it has 25 bits, and the sum is the rounded quotient for each of them, found
// by trying all in exact arithmetic): half of the largest value is a tie
// but for the rounding of s, and the product alone then misses the quotient's
// integer.  divide: s is so small that the residual would lose bits below the
// smallest subnormal.
__device__ __forceinline__ uint32_t int8x4(const float (&v)[4], float s, float y, bool divide) {
  uint32_t c = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float q = v[i] * y;
    const float z = divide ? v[i] / s : fmaf(fmaf(-s, q, v[i]), y, q);
    const float r = fminf(fmaxf(rintf(z), -kInt8Max), kInt8Max);
    c |= ((uint32_t)(int)r & 0xFFu) << (8 * i);
  }
  return c;
}

// LANES lanes take a row of up to WORDS 16-byte words each, which stay in registers
// between the maximum and the integers; WORDS 0: rows longer than that, read twice.
// A row with an infinity or NaN has the scale NaN and integers 0.
template <int LANES, int WORDS>
__global__ __launch_bounds__(256) void quant_int8_kernel(const u32x4_t* __restrict__ X, int64_t n,
                                                         int words, u32x2_t* __restrict__ Q,
                                                         float* __restrict__ S) {
  const int lane = threadIdx.x % LANES;
  const int64_t row = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  if (row >= n) return;
  const u32x4_t* x = X + row * words;
  constexpr int kHeld = WORDS > 0 ? WORDS : 1;
  u32x4_t v[kHeld];
  uint32_t m = 0;
  auto top = [&](u32x4_t w) { m = max(m, abs_max8(make_uint4(w[0], w[1], w[2], w[3]))); };
  if constexpr (WORDS > 0) {
#pragma unroll
    for (int j = 0; j < WORDS; ++j)
      v[j] = j * LANES + lane < words ? x[j * LANES + lane] : u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < WORDS; ++j) top(v[j]);
  } else {
    for (int c = lane; c < words; c += LANES) top(x[c]);
  }
  m = wave_max_u32(m);
  if constexpr (LANES > kWave) {
    static_assert(LANES == 256, "the block's four waves");
    __shared__ uint32_t part[4];
    if (lane % kWave == 0) part[lane / kWave] = m;
    __syncthreads();
    m = max(max(part[0], part[1]), max(part[2], part[3]));
  }
  const float amax = __uint_as_float(m);
  const bool finite = m < 0x7F800000u, zero = m == 0u;
  const float s = amax * (1.0f / kInt8Max), inv = 1.0f / s;
  const bool divide = amax < 0x1p-60f;
  auto store = [&](u32x4_t w, int c) {
    u32x2_t q = {0u, 0u};
    if (finite && !zero) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float f[4] = {__uint_as_float(w[2 * i] << 16),
                            __uint_as_float(w[2 * i] & 0xFFFF0000u),
                            __uint_as_float(w[2 * i + 1] << 16),
                            __uint_as_float(w[2 * i + 1] & 0xFFFF0000u)};
        q[i] = int8x4(f, s, inv, divide);
      }
    }
    Q[row * words + c] = q;
  };
  if constexpr (WORDS > 0) {
#pragma unroll
    for (int j = 0; j < WORDS; ++j)
      if (j * LANES + lane < words) store(v[j], j * LANES + lane);
  } else {
    for (int c = lane; c < words; c += LANES) store(x[c], c);
  }
  if (lane == 0) S[row] = finite ? s : __uint_as_float(0x7FC00000u);
}

// ---------------------------------------------------------------- product
// The 256-column tile: MB * 64 rows (MB 32-row blocks for each of two wave
// rows), eight waves of up to 32 MB x 64 outputs in MB x 2 accumulators of
// v_mfma_i32_32x32x32_i8.
constexpr int kCols = 256;
constexpr int kStage = 128;                  // bytes of k in a stage: a whole line of a row
constexpr int kQuarter = 64 * kStage;        // 64 weight rows of a stage
constexpr int kXcds = 8, kCus = 256;
constexpr int kListed = 64;                  // tiles that a block works on, at most
constexpr uint32_t kNoRow = 0xFFFFFFFFu - 256u * 1024u;  // past any buffer: the load gives zeros
// ... with a place in the row added too (which alone is less than any buffer's bytes)
static_assert(kInt8MaxGathered <= kNoRow && (uint64_t)256 * kInt8MaxDepth <= kNoRow &&
                  (uint64_t)kNoRow + kInt8MaxDepth <= 0xFFFFFFFFu,
              "kNoRow lies past a gathered a and past a tile's rows and weights");

template <int MB>
struct TileShape {
  static constexpr int rows = 64 * MB;
  static constexpr int a_bytes = rows * kStage;
  static constexpr int b_at = 2 * a_bytes;
  static constexpr int quarters = 12;  // of B's ring: three stages
  static constexpr int lds = b_at + quarters * kQuarter;
  static_assert(lds <= 160 * 1024, "a CU's LDS");
};

// Rows of one tile.
struct Tile {
  int expert, rows;
  int64_t row0;
};

// A segment of c rows in tiles of at most bm rows, near each other in size and
// multiples of 32 but for the last.
__device__ __forceinline__ uint32_t seg_tiles(uint32_t c, uint32_t bm) { return (c + bm - 1) / bm; }
__device__ __forceinline__ uint32_t seg_rows(uint32_t c, uint32_t n) {
  return ((c + n - 1) / n + 31) / 32 * 32;
}

// The segments of the experts, 64 of them a group, one a lane.  Bounds are
// clamped to [0, rows], so that offsets that do not ascend lead nowhere else.
struct Segments {
  static constexpr int kGroups = 6;  // E <= 384
  uint32_t lo[kGroups], n[kGroups], incl[kGroups], total;
  __device__ __forceinline__ void read(const Int8Args& a, uint32_t bm) {
    const int lane = lane_id();
    total = 0;
    int32_t first[kGroups], end[kGroups];  // all loads in flight at once
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int e = min(64 * g + lane, a.E - 1);
      first[g] = a.offsets[e];
      end[g] = a.offsets[e + 1];
    }
    const int rows = (int)a.rows;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int l = min(max(first[g], 0), rows), h = min(max(end[g], l), rows);
      lo[g] = (uint32_t)l;
      n[g] = 64 * g + lane < a.E ? (uint32_t)(h - l) : 0u;
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      incl[g] = wave_inclusive_sum_dpp_u32(seg_tiles(n[g], bm)) + total;
      total = readlane_u32(incl[g], 63);
    }
  }
  // Tile mt < total.
  __device__ __forceinline__ Tile tile(uint32_t mt, uint32_t bm, bool even) const {
    Tile t{0, 0, 0};
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const uint64_t past = ballot(incl[g] > mt);
      if (t.rows == 0 && past != 0) {
        const int l = __ffsll((unsigned long long)past) - 1;
        const uint32_t c = readlane_u32(n[g], l), k = seg_tiles(c, bm);
        const uint32_t i = mt - (readlane_u32(incl[g], l) - k);
        const uint32_t step = even ? seg_rows(c, k) : bm;
        t.expert = 64 * g + l;
        t.row0 = (int64_t)readlane_u32(lo[g], l) + i * step;
        t.rows = (int)min(step, c - min(c, i * step));
      }
    }
    return t;
  }
};

__device__ __forceinline__ float silu_mul(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}
__device__ __forceinline__ void block_barrier() {
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The tiles of a block, one a lane: blocks are dealt to the XCDs in turn, each XCD
// takes a contiguous run of the work and its blocks take that run's tiles in turn,
// so that the blocks at work together share operands in the XCD's L2.
struct List {
  uint32_t row0, rest;  // rest: expert, rows, column tile
  int count;
  // fn(item, column tile) -> Tile
  template <class F>
  __device__ __forceinline__ void fill(uint32_t work, F&& fn) {
    const uint32_t share = (work + kXcds - 1) / kXcds, per = gridDim.x / kXcds;
    const uint32_t begin = blockIdx.x % kXcds * share, end = min(begin + share, work);
    const int lane = lane_id();
    count = 0;
    row0 = rest = 0;
    for (uint32_t item = begin + blockIdx.x / kXcds; item < end && count < kListed; item += per) {
      uint32_t nt = 0;
      const Tile t = fn(item, nt);
      if (t.rows > 0) {
        row0 = lane == count ? (uint32_t)t.row0 : row0;
        rest = lane == count ? (uint32_t)t.expert << 22 | (uint32_t)t.rows << 12 | nt : rest;
        ++count;
      }
    }
    count = __builtin_amdgcn_readfirstlane(count);
  }
  __device__ __forceinline__ Tile tile(int i, int& nt) const {
    const uint32_t r = readlane_u32(rest, i);
    nt = (int)(r & 0xFFFu);
    return Tile{(int)(r >> 22), (int)(r >> 12 & 0x3FFu), (int64_t)readlane_u32(row0, i)};
  }
};

// A buffer whose place is the same in all lanes, kept in scalar registers.
struct Buffer {
  uint32_t lo, hi, bytes;
  __device__ __forceinline__ void set(const void* base, uint32_t n) {
    lo = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)base);
    hi = __builtin_amdgcn_readfirstlane((uint32_t)((uintptr_t)base >> 32));
    bytes = __builtin_amdgcn_readfirstlane(n);
  }
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc() const {
    const uint64_t at = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane(hi) << 32 |
                        (uint32_t)__builtin_amdgcn_readfirstlane(lo);
    return make_rsrc((const void*)at, (uint32_t)__builtin_amdgcn_readfirstlane(bytes));
  }
};

// A block's tiles one after the other, found once: a block to each tile spent 1.9 us
// on finding it, 4.4 until its first products and 5.1 behind its last ones, next to 25
// us of products.  98304 rows of 384 experts, 2560 deep, 2 x 512 columns, tiles of 192
// rows: 355 us that way, 344 this way; 2048 rows of 128 experts, 512 deep, 2560
// columns: 41 and 32.
//
// The next tile's first stages are asked for in front of a tile's stores, but as
// compiled they are not under way through them: the wait for the rows' scales takes
// the strictest count of the paths that meet there, so the first store waits for
// nearly all of these loads; the pairs of the results' rows, fetched behind the last
// product, are waited for before the first of them; and MB 4 keeps 10 or 11 registers
// in scratch, the weights' offsets among them, whose reloads between these loads wait
// for the ones before.  About 9 tiles a block pay that in the product above.
//
// What bounds it: dense, the power of the matrix instructions (8192 x 8192 x 8192:
// 405 to 422 us, 2.6 to 2.7 POP/s, in use 71% of the time at 1.7 GHz); few rows an
// expert, the weights' way from HBM (64 tokens of six among 384 experts: 0.64 GB in 97
// to 101 us, 6.4 to 6.6 TB/s); many rows of many experts, both in part, and what the
// change of tiles above costs, which is in all of these figures.  The 98304 rows above,
// 22 to 1243 an expert: 339 us in tiles of 256 (355 to 395 in a long row, as the clock
// falls), the same loads without products 304, from L2 with products 265, products
// alone 210; 256 rows an expert: 298, 266, 233 and 186.  Tiles in descending size,
// dealt so that all blocks end together, were no faster.
//
// The results go past the caches (98304 rows, 512 deep, 2560 columns: 287 us without,
// 281 so, of 206 that its bytes would take at a copy's rate: a tile is four stages of
// products, and a block changes tiles about 23 times).  ONCE: so do the weights.
template <int MB, bool UP, bool ONCE>
__device__ __forceinline__ void int8_tiles(const Int8Args& a, const List& list, char* lds) {
  typedef TileShape<MB> S;
  constexpr int OC = UP ? kCols / 2 : kCols;  // output columns of a tile
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wg = wave >> 2, wp = wave & 3;
  const int nk = (a.k + kStage - 1) / kStage;

  // Wave (wg, wp): the first or second half of the tile's 32-row blocks, and
  // weight rows 64 wp .. + 63, or with UP 32 wp of w and of w_up.
  const int b_row[2] = {UP ? 32 * wp : 64 * wp, UP ? kCols / 2 + 32 * wp : 64 * wp + 32};
  const int fr = lane & 31;
  const int b_quarter[2] = {b_row[0] >> 6, b_row[1] >> 6};
  const int b_base[2] = {((b_row[0] & 63) + fr) * kStage, ((b_row[1] & 63) + fr) * kStage};
  // the first 32-row block of the wave's half, and how many it has
  auto first_of = [&](const Tile& t) { return wg ? ((t.rows + 31) / 32 + 1) / 2 : 0; };
  auto live_of = [&](const Tile& t, int n) {
    const int blocks = (t.rows + 31) / 32, half = (blocks + 1) / 2;
    return __builtin_amdgcn_readfirstlane((UP ? 32 * wp : 64 * wp) < n ? (wg ? blocks - half : half)
                                                                       : 0);
  };

  // Loads: a wave brings MB times 8 rows of A and 4 times 8 rows of B a stage,
  // 128 bytes a row; load i covers rows 8 (8 i + wave) .. + 7 of the tile.
  // Lane l fills slot l & 7 of row l >> 3 with the row's chunk (l & 7) ^ ((row >> 1)
  // & 7).  Rows past the tile and chunks past k read zeros.
  const int sub = lane >> 3;
  const int chunk = (lane & 7) ^ ((4 * wave + (sub >> 1)) & 7);
  const bool k_in = (nk - 1) * kStage + chunk * 16 < a.k;  // this lane's chunk of the last stage
  uint32_t a_off[MB], a_pair[MB], r_pair[MB], b_off;
  Buffer ra, rw, ru;
  Tile tile;
  int col0, cols;
  // The pairs of the rows of A that the wave loads (a_pair) and of those whose
  // results it holds (r_pair), all loads at once; a row past the tile gives its last
  // one's.
  auto pairs_of = [&](const Tile& t, auto row, uint32_t(&pair)[MB]) {
#pragma unroll
    for (int j = 0; j < MB; ++j) {
      const int r = min(row(j), t.rows - 1);
      pair[j] = a.sorted_src ? (uint32_t)a.sorted_src[t.row0 + r] : (uint32_t)r;
    }
  };
  auto a_pairs = [&](int i) {
    int nt;
    pairs_of(list.tile(i, nt), [&](int j) { return 8 * (8 * j + wave) + sub; }, a_pair);
  };
  auto r_pairs = [&](int i) {
    int nt;
    const Tile t = list.tile(i, nt);
    pairs_of(t, [&](int m) { return 32 * (first_of(t) + m) + fr; }, r_pair);
  };
  // the row of A of a pair, or of the tile's row
  auto a_row = [&](uint32_t pair) {
    return a.sorted_src ? min(max((int)pair, 0) / (uint32_t)a.K, (uint32_t)a.a_rows - 1u) : pair;
  };
  auto open = [&](int i) {
    int nt;
    tile = list.tile(i, nt);
    col0 = nt * OC;
    cols = min(OC, a.cols - col0);
#pragma unroll
    for (int j = 0; j < MB; ++j)
      a_off[j] = 8 * (8 * j + wave) + sub < tile.rows
                     ? a_row(a_pair[j]) * (uint32_t)a.k + (uint32_t)chunk * 16u
                     : kNoRow;
    b_off = (uint32_t)(8 * wave + sub) * (uint32_t)a.k + (uint32_t)chunk * 16u;
    const int64_t w_row = (int64_t)tile.expert * a.cols + col0;
    const uint32_t w_bytes = (uint32_t)cols * (uint32_t)a.k;
    if (a.sorted_src) ra.set(a.a, (uint32_t)(a.a_rows * a.k));
    else ra.set(a.a + tile.row0 * a.k, (uint32_t)tile.rows * (uint32_t)a.k);
    rw.set(a.w + w_row * a.k, w_bytes);
    ru.set((UP ? a.w_up : a.w) + w_row * a.k, w_bytes);
  };
  auto load_a = [&](int kt, int slot, int i) {
    dma16(ra.rsrc(), kt == nk - 1 && !k_in ? kNoRow : a_off[i], (uint32_t)kt * kStage,
          (lds_void_t*)(lds + slot * S::a_bytes + (8 * i + wave) * 1024));
  };
  // quarter i of stage kt at place q of the ring: rows 64 i .. + 63 of the tile's
  // weight, with UP 64 (i % 2) .. + 63 of w or w_up; rows past the tile's columns
  // lie past the buffer
  auto load_b = [&](int kt, int q, int i) {
    const uint32_t off = b_off + (uint32_t)(UP ? i & 1 : i) * 64u * (uint32_t)a.k;
    dma16<ONCE ? kCpolNT : 0>(
        UP && i >= 2 ? ru.rsrc() : rw.rsrc(), kt == nk - 1 && !k_in ? kNoRow : off,
        (uint32_t)kt * kStage, (lds_void_t*)(lds + S::b_at + q * kQuarter + wave * 1024));
  };
  auto place = [&](int q) { return q >= S::quarters ? q - S::quarters : q; };
  // a tile's first stages: A's two slots, B's three stages
  auto load_first = [&] {
    // stage by stage, as the waits count them
    auto in_order = [] {
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < MB; ++i) load_a(0, 0, i);
#pragma unroll
    for (int i = 0; i < 4; ++i) load_b(0, i, i);
    in_order();
    if (nk > 1) {
#pragma unroll
      for (int i = 0; i < MB; ++i) load_a(1, 1, i);
#pragma unroll
      for (int i = 0; i < 4; ++i) load_b(1, 4 + i, i);
    }
    in_order();
    if (nk > 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) load_b(2, 8 + i, i);
    }
    in_order();
  };

  const int slot0 = ((lane >> 5) ^ ((lane >> 1) & 7)) * 16;  // of step s: ^ 32 s

  a_pairs(0);
  r_pairs(0);
  open(0);
  load_first();
  for (int it = 0; it < list.count; ++it) {
    const Tile now = tile;
    const int now_col0 = col0, now_cols = cols;
    const int first = first_of(now), live = live_of(now, now_cols);
    const int a_base = (32 * first + fr) * kStage;
    // the rows' scales, and the next tile's pairs
    float sr[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m)
      sr[m] = a.a_scales[a.sorted_src ? (int64_t)a_row(r_pair[m]) : now.row0 + r_pair[m]];
    if (it + 1 < list.count) a_pairs(it + 1);

    i32x16_t acc[MB][2];
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[m][f][r] = 0;

    // Stage kt is four steps of 32 bytes of k; the fragments of the next step are
    // read while a step's products run.  The barrier in front of the last step
    // frees A's slot and B's quarters of the stage: A two stages on goes there at
    // once (two loads, the rest in the next stage's first step), B three stages on
    // in that stage's second and third step.  The waits count the loads that may
    // be in flight, all of them younger than those waited for; others between
    // them (scales, the last tile's stores) make a wait longer, never shorter.
    typedef std::true_type T;
    typedef std::false_type F;
    auto run = [&](auto live_tag) {
      constexpr int LIVE = decltype(live_tag)::value;
      constexpr int NF = LIVE > 0 ? LIVE : 1;
      i32x4_t fa[2][NF], fb[2][2];
      auto read = [&](int set, int slot, int q0, int step) {
#pragma unroll
        for (int f = 0; f < 2; ++f)
          fb[set][f] = *reinterpret_cast<const i32x4_t*>(
              lds + S::b_at + place(q0 + b_quarter[f]) * kQuarter + ((b_base[f] + slot0) ^ (32 * step)));
#pragma unroll
        for (int m = 0; m < NF; ++m)
          fa[set][m] = *reinterpret_cast<const i32x4_t*>(
              lds + slot * S::a_bytes + 32 * m * kStage + ((a_base + slot0) ^ (32 * step)));
      };
      if (nk > 2) wait_vmcnt<MB + 8>();
      else if (nk > 1) wait_vmcnt<MB + 4>();
      else wait_vmcnt<0>();
      block_barrier();
      int slot = 0, q0 = 0;  // of stage kt
      if (LIVE > 0) read(0, 0, 0, 0);
      // ld_a1: the rest of A(kt + 1); ld_b: B(kt + 2); ld_a2: A(kt + 2);
      // next: there is a stage kt + 1; ahead: loads of B(kt + 2) may be in flight at the barrier.
      auto stage = [&](int kt, auto ld_a1, auto ld_b, auto ld_a2, auto next, auto ahead) {
        const int q1 = place(q0 + 4);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int cur = s & 1;
          if (s == 3 && next) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            if (ahead) wait_vmcnt<4>();
            else wait_vmcnt<0>();
            block_barrier();
          }
          if (s == 0 && ld_a1) {
#pragma unroll
            for (int i = 2; i < MB; ++i) load_a(kt + 1, slot ^ 1, i);
          }
          if ((s == 1 || s == 2) && ld_b) {
            load_b(kt + 2, place(q1 + 2 * s + 2), 2 * s - 2);
            load_b(kt + 2, place(q1 + 2 * s + 3), 2 * s - 1);
          }
          if (s == 3 && ld_a2) {
#pragma unroll
            for (int i = 0; i < (MB < 2 ? MB : 2); ++i) load_a(kt + 2, slot, i);
          }
          if (LIVE > 0) {
            if (s < 3) read(cur ^ 1, slot, q0, s + 1);
            else if (next) read(cur ^ 1, slot ^ 1, q1, 0);
          }
          __builtin_amdgcn_sched_barrier(0);
          if (LIVE > 0) {
#pragma unroll
            for (int m = 0; m < NF; ++m)
#pragma unroll
              for (int f = 0; f < 2; ++f)
                acc[m][f] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[cur][f], fa[cur][m],
                                                                  acc[m][f], 0, 0, 0);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        slot ^= 1;
        q0 = q1;
      };
      stage(0, F{}, F{}, nk > 2, nk > 1, nk > 2);
      for (int kt = 1; kt + 2 < nk; ++kt) stage(kt, T{}, T{}, T{}, T{}, T{});
      if (nk >= 3) stage(nk - 2, T{}, F{}, F{}, T{}, F{});
      if (nk >= 2) stage(nk - 1, F{}, F{}, F{}, F{}, F{});
    };
    switch (live) {
      case 0: run(std::integral_constant<int, 0>{}); break;
      case 1: run(std::integral_constant<int, 1>{}); break;
      case 2: run(std::integral_constant<int, MB < 2 ? MB : 2>{}); break;
      case 3: run(std::integral_constant<int, MB < 3 ? MB : 3>{}); break;
      default: run(std::integral_constant<int, MB>{}); break;
    }
    // what follows is formed from the lane's number anew: kept from tile to tile it
    // would not fit the registers next to the products
    int me = lane;
    asm volatile("" : "+v"(me));
    // the channels' scales, ahead of the next tile's loads: they come back first
    f32x4_t sc[2][4];
    if (live > 0) {
      const int64_t w_row = (int64_t)now.expert * a.cols + now_col0;
      const __amdgpu_buffer_rsrc_t rs = make_rsrc(a.w_scales + w_row, (uint32_t)now_cols * 4u);
      const __amdgpu_buffer_rsrc_t rt =
          make_rsrc((UP ? a.w_up_scales : a.w_scales) + w_row, (uint32_t)now_cols * 4u);
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          sc[f][q] = __builtin_bit_cast(
              f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                           UP && f ? rt : rs,
                           (int)((uint32_t)((UP ? 32 * wp : b_row[f]) + 8 * q + 4 * (me >> 5)) * 4u), 0, 0));
    }
    if (it + 1 < list.count) {
      r_pairs(it + 1);
      // all waves have read their last fragments before LDS is filled again
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      block_barrier();
      open(it + 1);
      load_first();
    }

    // The products have the weights first, so a lane holds output row (l & 31) of a
    // block and columns 8 (r / 4) + 4 (l / 32) + r % 4.  Columns of two register
    // groups are joined with the other half's to eight (16 bytes), then rows trade
    // places between lanes: eight lanes hold 64 columns of a row, a whole line
    // (with UP four lanes 32 columns).
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      if (m >= live) break;
      uint32_t v[2][2][4];  // [f][column groups 2 u and 2 u + 1]
#pragma unroll
      for (int f = 0; f < (UP ? 1 : 2); ++f)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float y[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int q = 2 * u + g, r = 4 * q + 2 * j + e;
                y[e] = (float)acc[m][f][r] * (sr[m] * sc[f][q][2 * j + e]);
                if (UP) y[e] = silu_mul(y[e], (float)acc[m][1][r] * (sr[m] * sc[1][q][2 * j + e]));
              }
              v[f][u][2 * g + j] = pack_bf16(y[0], y[1]);
            }
#pragma unroll
          for (int j = 0; j < 2; ++j) swap_halves(v[f][u][j], v[f][u][2 + j]);
        }
#pragma unroll
      for (int f = 0; f < (UP ? 1 : 2); ++f)
#pragma unroll
        for (int j = 0; j < 4; ++j) swap_rows16(v[f][0][j], v[f][1][j]);
      auto store = [&](const uint32_t (&w)[4], int r, int c) {
        const int at = 32 * (first + m) + r;
        if (at < now.rows && c < now_cols)
          __builtin_nontemporal_store(
              u32x4_t{w[0], w[1], w[2], w[3]},
              reinterpret_cast<u32x4_t*>(a.out + (now.row0 + at) * a.cols + now_col0 + c));
      };
      if constexpr (UP) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
          store(v[0][u], 16 * u + (me & 15),
                32 * wp + 16 * ((me >> 4) & 1) + 8 * (me >> 5));
      } else {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
          for (int j = 0; j < 4; ++j) swap_rows8(v[0][u][j], v[1][u][j]);
#pragma unroll
          for (int f = 0; f < 2; ++f)
            store(v[f][u], 16 * u + 8 * f + line_row(me), 64 * wp + line_col(me));
        }
      }
    }
  }
}

// Dense: the tiles of four row tiles follow each other on a column tile.
constexpr uint32_t kRowGroup = 4;

template <int MB, bool UP>
__global__ __launch_bounds__(512, 2) void int8_dense_kernel(Int8Args a, uint32_t m_tiles,
                                                            uint32_t col_tiles) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  List list;
  list.fill(m_tiles * col_tiles, [&](uint32_t item, uint32_t& nt) {
    const uint32_t group = item / (kRowGroup * col_tiles), in = item % (kRowGroup * col_tiles);
    const uint32_t deep = min(kRowGroup, m_tiles - group * kRowGroup);
    nt = in / deep;
    Tile t;
    t.expert = 0;
    t.row0 = (int64_t)(group * kRowGroup + in % deep) * TileShape<MB>::rows;
    t.rows = (int)min((int64_t)TileShape<MB>::rows, a.rows - t.row0);
    return t;
  });
  if (list.count > 0) int8_tiles<MB, UP, false>(a, list, lds);
}

template <int MB, bool UP, bool ONCE>
__global__ __launch_bounds__(512, 2) void int8_grouped_kernel(Int8Args a, uint32_t col_tiles) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  constexpr uint32_t bm = TileShape<MB>::rows;
  List list;
  {
    Segments s;
    s.read(a, bm);
    list.fill(s.total * col_tiles, [&](uint32_t item, uint32_t& nt) {
      nt = item % col_tiles;
      return s.tile(item / col_tiles, bm, true);
    });
  }
  if (list.count > 0) int8_tiles<MB, UP, ONCE>(a, list, lds);
}

// Few rows: a block takes 16 RG rows and 16 CB columns (of each weight), its four
// waves share out k, 128 bytes (a line of every row) in turn, straight from memory
// into the matrix instructions' registers (v_mfma_i32_16x16x64_i8), kDepth lines of
// each row in flight a wave; the waves' sums meet in LDS (integers: in any order
// the same).  What the expert gives, weights and scales, is on its way before the
// rows' pairs are known.  Latencies bound it: one token's six experts of 2 x 512
// columns, 2560 deep, 16 MB, 6.4 us; with the weights behind the pairs 6.9.
template <int RG, int CB, bool UP, bool GROUPED>
__global__ __launch_bounds__(256, 2) void int8_few_kernel(Int8Args a, int col_tiles) {
  constexpr int NB = UP ? 2 * CB : CB, kOut = RG * NB;
  constexpr int kDepth = RG + NB >= 8 ? 2 : RG + NB >= 5 ? 3 : 16 / (RG + NB);
  constexpr int kBm = 16 * RG, kOc = 16 * CB;
  __shared__ __attribute__((aligned(16))) i32x4_t sums[4][kOut][64];
  Tile tile;
  const int nt = (int)(blockIdx.x % (unsigned)col_tiles);
  const uint32_t mt = blockIdx.x / (unsigned)col_tiles;
  if constexpr (GROUPED) {
    Segments s;
    s.read(a, kBm);
    if (mt >= s.total) return;
    tile = s.tile(mt, kBm, false);
    if (tile.rows <= 0) return;
  } else {
    tile.expert = 0;
    tile.row0 = (int64_t)mt * kBm;
    tile.rows = (int)min((int64_t)kBm, a.rows - tile.row0);
  }
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 15, piece = 16 * (lane >> 4);
  const int col0 = nt * kOc, cols = min(kOc, a.cols - col0);
  const int64_t w_row = (int64_t)tile.expert * a.cols + col0;
  const uint32_t w_bytes = (uint32_t)cols * (uint32_t)a.k;
  const __amdgpu_buffer_rsrc_t ra =
      a.sorted_src ? make_rsrc(a.a, (uint32_t)(a.a_rows * a.k))
                   : make_rsrc(a.a + tile.row0 * a.k, (uint32_t)tile.rows * (uint32_t)a.k);
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.w + w_row * a.k, w_bytes);
  const __amdgpu_buffer_rsrc_t ru = make_rsrc((UP ? a.w_up : a.w) + w_row * a.k, w_bytes);
  uint32_t pair[RG], a_off[RG], b_off[CB];
#pragma unroll
  for (int r = 0; r < RG; ++r) {
    const int i = min(16 * r + row, tile.rows - 1);
    pair[r] = a.sorted_src ? (uint32_t)a.sorted_src[tile.row0 + i] : 0u;
  }
#pragma unroll
  for (int c = 0; c < CB; ++c)
    b_off[c] = 16 * c + row < cols ? (uint32_t)(16 * c + row) * (uint32_t)a.k : kNoRow;

  i32x4_t fa[kDepth][2][RG], fb[kDepth][2][NB], acc[RG][NB];
  // line i of this wave
  auto load_b = [&](int buf, int i) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = (4 * i + wave) * 128 + 64 * h + piece;
      const bool in = at < a.k;
#pragma unroll
      for (int c = 0; c < NB; ++c) {
        const uint32_t off = b_off[c % CB];
        fb[buf][h][c] = __builtin_bit_cast(
            i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                         c < CB ? rw : ru, (int)(in && off != kNoRow ? off + (uint32_t)at : kNoRow),
                         0, 0));
      }
    }
  };
  auto load_a = [&](int buf, int i) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = (4 * i + wave) * 128 + 64 * h + piece;
      const bool in = at < a.k;
#pragma unroll
      for (int r = 0; r < RG; ++r)
        fa[buf][h][r] = __builtin_bit_cast(
            i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                         ra, (int)(in && a_off[r] != kNoRow ? a_off[r] + (uint32_t)at : kNoRow), 0,
                         0));
    }
  };
#pragma unroll
  for (int r = 0; r < RG; ++r)
#pragma unroll
    for (int c = 0; c < NB; ++c) acc[r][c] = i32x4_t{0, 0, 0, 0};
  const int lines = (a.k + 127) / 128, mine = (lines - wave + 3) / 4;  // of this wave
  // all that is known by the expert first, then what waits for the rows' pairs
#pragma unroll
  for (int d = 0; d < kDepth; ++d) load_b(d, d);
  // output block (r, c) of the columns: wave (r CB + c) % 4; lane l has row l & 15
  // and columns 4 (l / 16) ..
  constexpr int kMine = (RG * CB + 3) / 4;
  float sr[kMine];
  f32x4_t sc[kMine], su[kMine];
  auto block_of = [&](int j, int& r, int& i, int& col) {
    const int o = wave + 4 * j;
    r = o / CB;
    i = 16 * r + row;
    col = 16 * (o % CB) + 4 * (lane >> 4);
    return o < RG * CB && i < tile.rows && col < cols;
  };
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    int r, i, col;
    sc[j] = su[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    if (!block_of(j, r, i, col)) continue;
    sc[j] = *reinterpret_cast<const f32x4_t*>(a.w_scales + w_row + col);
    if (UP) su[j] = *reinterpret_cast<const f32x4_t*>(a.w_up_scales + w_row + col);
  }
  uint32_t a_row[RG];
#pragma unroll
  for (int r = 0; r < RG; ++r) {
    a_row[r] = a.sorted_src ? min(max((int)pair[r], 0) / (uint32_t)a.K, (uint32_t)a.a_rows - 1u)
                            : 16u * r + row;
    a_off[r] = 16 * r + row < tile.rows ? a_row[r] * (uint32_t)a.k : kNoRow;
  }
#pragma unroll
  for (int d = 0; d < kDepth; ++d) load_a(d, d);
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    int r, i, col;
    sr[j] = 0.0f;
    if (!block_of(j, r, i, col)) continue;
    uint32_t from = 0;
#pragma unroll
    for (int q = 0; q < RG; ++q) from = q == r ? a_row[q] : from;
    sr[j] = a.a_scales[a.sorted_src ? (int64_t)from : tile.row0 + from];
  }
  for (int i = 0; i < mine; i += kDepth) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < NB; ++c)
#pragma unroll
          for (int r = 0; r < RG; ++r)
            acc[r][c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[d][h][c], fa[d][h][r], acc[r][c],
                                                              0, 0, 0);
      // past the wave's last line: zeros, without a memory access
      load_b(d, i + kDepth + d);
      load_a(d, i + kDepth + d);
    }
  }
#pragma unroll
  for (int r = 0; r < RG; ++r)
#pragma unroll
    for (int c = 0; c < NB; ++c) sums[wave][r * NB + c][lane] = acc[r][c];
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    int r, i, col;
    if (!block_of(j, r, i, col)) continue;
    const int c = (wave + 4 * j) % CB;
    auto total = [&](int b) {
      i32x4_t t = sums[0][b][lane];
#pragma unroll
      for (int w = 1; w < 4; ++w) t += sums[w][b][lane];
      return t;
    };
    const i32x4_t g = total(r * NB + c);
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = (float)g[e] * (sr[j] * sc[j][e]);
    if constexpr (UP) {
      const i32x4_t u = total(r * NB + CB + c);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = silu_mul(y[e], (float)u[e] * (sr[j] * su[j][e]));
    }
    *reinterpret_cast<u32x2_t*>(a.out + (tile.row0 + i) * a.cols + col0 + col) =
        u32x2_t{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
  }
}

}  // namespace

hipError_t launch_quant_int8(const uint16_t* X, int64_t n, int cols, int8_t* Q, float* S,
                             hipStream_t stream) {
  const int words = cols / 8;
  const int lanes = words <= 6 * 64 ? 64 : 256;
  const int64_t most = int64_t(1) << 23;  // rows a launch: fewer than 2^32 threads
  for (int64_t r0 = 0; r0 < n; r0 += most) {
    const int64_t m = std::min(most, n - r0);
    const dim3 grid((unsigned)((m * lanes + 255) / 256)), block(256);
    const u32x4_t* x = reinterpret_cast<const u32x4_t*>(X + r0 * cols);
    u32x2_t* q = reinterpret_cast<u32x2_t*>(Q + r0 * cols);
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, block, 0, stream, x, m, words, q, S + r0);
    };
    if (words <= 2 * 64) go(quant_int8_kernel<64, 2>);
    else if (words <= 6 * 64) go(quant_int8_kernel<64, 6>);
    else if (words <= 4 * 256) go(quant_int8_kernel<256, 4>);
    else if (words <= 8 * 256) go(quant_int8_kernel<256, 8>);
    else go(quant_int8_kernel<256, 0>);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

namespace {
template <int MB>
hipError_t allow_lds() {
  const void* kernels[] = {
      (const void*)int8_grouped_kernel<MB, true, false>,
      (const void*)int8_grouped_kernel<MB, false, false>,
      (const void*)int8_grouped_kernel<MB, true, true>,
      (const void*)int8_grouped_kernel<MB, false, true>,
      (const void*)int8_dense_kernel<MB, true>, (const void*)int8_dense_kernel<MB, false>};
  static std::atomic<uint32_t> done[6];
  for (int i = 0; i < 6; ++i) {
    const hipError_t e = set_lds_limit_once(kernels[i], TileShape<MB>::lds, done[i]);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
// The LDS of every tile kernel, on a device's first call: another size's call, which
// may be a captured one, finds its kernel ready.
hipError_t allow_lds_once() {
  static std::atomic<uint32_t> all{0};
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint32_t bit = dev >= 0 && dev < 32 ? 1u << dev : 0u;
  if (bit && (all.load(std::memory_order_acquire) & bit)) return hipSuccess;
  if ((e = allow_lds<1>()) != hipSuccess || (e = allow_lds<2>()) != hipSuccess ||
      (e = allow_lds<3>()) != hipSuccess || (e = allow_lds<4>()) != hipSuccess)
    return e;
  all.fetch_or(bit, std::memory_order_release);
  return hipSuccess;
}
template <class Kernel, class... Args>
hipError_t launch_tiles(Kernel kernel, int lds, int64_t blocks, hipStream_t stream, Args... args) {
  if (blocks >= (int64_t(1) << 23)) return hipErrorInvalidConfiguration;  // 2^32 threads
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(512), lds, stream, args...);
  return hipGetLastError();
}
// Blocks for that many tiles: one a CU, unless their lists overflow.
int64_t tile_blocks(int64_t tiles) {
  const int64_t need = std::max(std::min<int64_t>(tiles, kCus), (tiles + kListed - 1) / kListed);
  return (need + kXcds - 1) / kXcds * kXcds;
}

// Tiles of bm rows, at most: experts without rows have none.
int64_t most_tiles(const Int8Args& a, int64_t bm) {
  return a.offsets ? a.rows / bm + std::min<int64_t>(a.E, a.rows) : (a.rows + bm - 1) / bm;
}

template <int RG, int CB>
hipError_t launch_few(const Int8Args& a, hipStream_t stream) {
  const int col_tiles = (a.cols + 16 * CB - 1) / (16 * CB);
  const int64_t blocks = most_tiles(a, 16 * RG) * col_tiles;
  if (blocks >= (int64_t(1) << 24)) return hipErrorInvalidConfiguration;  // 2^32 threads
  const dim3 grid((unsigned)blocks), block(256);
  if (a.offsets && a.w_up)
    hipLaunchKernelGGL((int8_few_kernel<RG, CB, true, true>), grid, block, 0, stream, a, col_tiles);
  else if (a.offsets)
    hipLaunchKernelGGL((int8_few_kernel<RG, CB, false, true>), grid, block, 0, stream, a, col_tiles);
  else if (a.w_up)
    hipLaunchKernelGGL((int8_few_kernel<RG, CB, true, false>), grid, block, 0, stream, a, col_tiles);
  else
    hipLaunchKernelGGL((int8_few_kernel<RG, CB, false, false>), grid, block, 0, stream, a, col_tiles);
  return hipGetLastError();
}
}  // namespace

namespace {
int column_tiles(const Int8Args& a) {
  const int oc = a.w_up ? kCols / 2 : kCols;
  return (a.cols + oc - 1) / oc;
}
template <int MB>
hipError_t launch_grouped(const Int8Args& a, hipStream_t stream) {
  const int col_tiles = column_tiles(a);
  const int64_t blocks = tile_blocks(most_tiles(a, TileShape<MB>::rows) * col_tiles);
  auto go = [&](auto kernel) {
    return launch_tiles(kernel, TileShape<MB>::lds, blocks, stream, a, (uint32_t)col_tiles);
  };
  // Most experts have one tile, and their weights do not fit the memory-side cache:
  // each is read once (2560 x 2 x 512, 384 experts, a row each 112 us, 101 so; 64 rows
  // each 224, 211; 128 rows in tiles of 192 would take 260 for 257).
  const int64_t experts = std::min<int64_t>(a.E, a.rows);
  const int64_t weights = experts * a.cols * (int64_t)a.k * (a.w_up ? 2 : 1);
  const bool once = a.rows <= experts * (TileShape<MB>::rows / 2) && weights > (int64_t(256) << 20);
  if (once) return a.w_up ? go(int8_grouped_kernel<MB, true, true>)
                          : go(int8_grouped_kernel<MB, false, true>);
  return a.w_up ? go(int8_grouped_kernel<MB, true, false>)
                : go(int8_grouped_kernel<MB, false, false>);
}
template <int MB>
hipError_t launch_dense(const Int8Args& a, hipStream_t stream) {
  const int col_tiles = column_tiles(a);
  const int64_t m_tiles = most_tiles(a, TileShape<MB>::rows);
  const int64_t blocks = tile_blocks(m_tiles * col_tiles);
  auto go = [&](auto kernel) {
    return launch_tiles(kernel, TileShape<MB>::lds, blocks, stream, a, (uint32_t)m_tiles,
                        (uint32_t)col_tiles);
  };
  return a.w_up ? go(int8_dense_kernel<MB, true>) : go(int8_dense_kernel<MB, false>);
}

// Tiles of bm rows that are expected: every expert with rows has its share of
// them, and half a tile more where that share is over half a tile.
double expected_tiles(const Int8Args& a, int bm) {
  if (!a.offsets) return (double)((a.rows + bm - 1) / bm);
  const double experts = (double)std::min<int64_t>(a.E, a.rows), share = (double)a.rows / experts;
  return experts * std::max(1.0, share / bm + 0.5);
}
// A launch's cost, to rank the forms: a fit to the microseconds of shapes from 1 to
// 16384 rows, 512 to 8192 deep, dense and with 16 to 384 experts.  The shortest launches
// are within a fifth of it, those of 30 us take up to half as much again (4096 rows of
// 2560 x 2560 22 for 30; 2048 of 128 experts 21 for 31), long ones twice, as neither memory's share nor the falling clock is in it (98304
// rows of 2560, 2 x 512 columns: 243 for 339; of 512, 2560 columns: 144 for 282; 64 rows
// an expert: 110 for 214; 8192 x 8192 x 8192: 289 for 417), so that between MB 3 and 4 it
// ranks by less than it is off.  Rows are all N K, pairs without an expert here too.
// Tiles: 0.22 (MB + 1) a stage and 1 a tile, 256 at a time; experts' weights that no
// more than a tile or two share slow a stage by 0.18 where there is more than one round.
double tile_cost(const Int8Args& a, int mb) {
  const double rounds = std::ceil(expected_tiles(a, 64 * mb) * column_tiles(a) / kCus);
  const double stage = 0.22 * (mb + 1) + (a.offsets && rounds > 1 ? 0.18 : 0.0);
  return 3.5 + rounds * (1.0 + (a.k + kStage - 1) / kStage * stage);
}
// Few rows: what the blocks read at 8 TB/s, 1.2 for every further 256 blocks (twice
// that where each looks for its expert), but no block faster than its own operands
// at 40 KB a microsecond.
double few_cost(const Int8Args& a, int rg, int cb) {
  const int nb = a.w_up ? 2 * cb : cb;
  const double tiles = expected_tiles(a, 16 * rg);
  const double rows = std::min((double)a.rows / tiles, 16.0 * rg);
  const double blocks = tiles * ((a.cols + 16 * cb - 1) / (16 * cb));
  const double bytes = (rows + 16.0 * nb) * a.k;  // of a block
  const double more = (a.offsets ? 2.4 : 1.2) * std::max(0.0, blocks / kCus - 1.0);
  return (a.offsets ? 5.0 : 4.2) + std::max(blocks * bytes / 8e6 + more, bytes / 40e3);
}
}  // namespace

// The cheapest form by the fits above.  2560 x 2560 weights, us: 1 row 4.8 (few,
// 1 x 1; tiles of MB 1 11.7), 64 rows 8.5 (few, 2 x 2; 11.7), 512 rows 12.7 (MB 1;
// MB 4 27, few-row blocks of 64 x 64 25), 4096 rows 29 (MB 3; MB 1 42); 8192 x 8192 x
// 8192 405 to 422 (MB 4; MB 2 449).
hipError_t launch_int8_matmul(const Int8Args& a, hipStream_t stream) {
  typedef hipError_t (*Launch)(const Int8Args&, hipStream_t);
  struct Form {
    double cost;
    Launch launch;
  };
  const Form forms[] = {
      {tile_cost(a, 1), a.offsets ? launch_grouped<1> : launch_dense<1>},
      {tile_cost(a, 2), a.offsets ? launch_grouped<2> : launch_dense<2>},
      {tile_cost(a, 3), a.offsets ? launch_grouped<3> : launch_dense<3>},
      {tile_cost(a, 4), a.offsets ? launch_grouped<4> : launch_dense<4>},
      {few_cost(a, 1, 1), launch_few<1, 1>},
      {few_cost(a, 1, 2), launch_few<1, 2>},
      {few_cost(a, 2, 1), launch_few<2, 1>},
      {few_cost(a, 2, 2), launch_few<2, 2>},
      {few_cost(a, 4, 2), launch_few<4, 2>},
  };
  const hipError_t e = allow_lds_once();
  if (e != hipSuccess) return e;
  const Form* best = forms;
  for (const Form& f : forms)
    if (f.cost < best->cost) best = &f;
  return best->launch(a, stream);
}

}  // namespace moe
