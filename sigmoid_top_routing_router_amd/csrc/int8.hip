// Products in 8-bit integers with a scale for each row (token) and each output
// channel, dense or grouped by expert, and the row quantiser.
//
// A row x becomes s = amax|x| / 127 and the integers q = rne(x / s) in [-127,
// 127]; weights the same way, a row of W being an output channel.  Then
//   y_tc = s_t s_c sum_k q_tk q_ck,
// the sum exact in 32-bit integers (|sum| <= 2^14 k < 2^31 for k <= 65536; the
// code -128 of a caller's own included), converted to fp32 (one rounding of
// 2^-24 above 2^24), times both scales, and y rounded to bf16 once.  With a
// second weight: silu(y) * y', formed in fp32 ("Kolibri 1 im Detail", routing
// section, SwiGLU paragraph).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.h"
#include "fp8_codes.h"
#include "gemm_args.h"
#include "kernels.h"

namespace moe {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

constexpr float kInt8Max = 127.0f;

// Four integers.  The quotient v / s rounded to fp32 as q = v y, q + (v - s q) y
// with y = 1 / s (three operations in the place of a division's; the residual is
// exact): half of the largest value is a tie but for the rounding of s, and the
// product alone then misses the quotient's integer.  divide: s is so small that
// the residual would not be exact.
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

// A wave takes a row.  A row with an infinity or NaN has the scale NaN and
// integers 0.
__global__ __launch_bounds__(256) void quant_int8_kernel(const u32x4_t* __restrict__ X, int64_t n,
                                                         int words, u32x2_t* __restrict__ Q,
                                                         float* __restrict__ S) {
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= n) return;
  const int lane = lane_id();
  const u32x4_t* x = X + row * words;
  uint32_t m = 0;
  for (int c = lane; c < words; c += kWave) {
    const u32x4_t v = x[c];
    m = max(m, abs_max8(make_uint4(v[0], v[1], v[2], v[3])));
  }
  m = wave_max_u32(m);
  const float amax = __uint_as_float(m);
  const bool finite = m < 0x7F800000u, zero = m == 0u;
  const float s = amax / kInt8Max, inv = 1.0f / s;
  const bool divide = amax < 0x1p-60f;
  for (int c = lane; c < words; c += kWave) {
    const u32x4_t v = x[c];
    u32x2_t q = {0u, 0u};
    if (finite && !zero) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float f[4] = {__uint_as_float(v[2 * i] << 16),
                            __uint_as_float(v[2 * i] & 0xFFFF0000u),
                            __uint_as_float(v[2 * i + 1] << 16),
                            __uint_as_float(v[2 * i + 1] & 0xFFFF0000u)};
        q[i] = int8x4(f, s, inv, divide);
      }
    }
    Q[row * words + c] = q;
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
constexpr int kLds = 160 * 1024;
constexpr int kXcds = 8;
constexpr uint32_t kNoRow = 0xFFFFFFFFu - 256u * 1024u;  // past any buffer: the load gives zeros

template <int MB>
struct TileShape {
  static constexpr int rows = 64 * MB;
  static constexpr int a_bytes = rows * kStage;
  static constexpr int b_at = 2 * a_bytes;
  static constexpr int quarters = (kLds - b_at) / kQuarter;  // of B's ring: 12 or 10
  static_assert(quarters >= 8, "two stages of B at least");
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
  __device__ __forceinline__ void read(const Int8Args& a, uint32_t bm, bool) {
    const int lane = lane_id();
    total = 0;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int e = 64 * g + lane;
      lo[g] = n[g] = 0;
      if (e < a.E) {
        const int64_t l = min(max((int64_t)a.offsets[e], (int64_t)0), a.rows);
        const int64_t h = min(max((int64_t)a.offsets[e + 1], l), a.rows);
        lo[g] = (uint32_t)l;
        n[g] = (uint32_t)(h - l);
      }
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

// Blocks are dealt to the XCDs in turn; each takes a contiguous run of the work.
__device__ __forceinline__ bool xcd_item(int64_t block, int64_t work, int64_t& item) {
  const int64_t share = (work + kXcds - 1) / kXcds, local = block / kXcds;
  item = block % kXcds * share + local;
  return local < share && item < work;
}

// The row of A behind output row r.
__device__ __forceinline__ int64_t a_row_of(const Int8Args& a, int64_t r) {
  if (!a.sorted_src) return r;
  const int64_t t = (int64_t)a.sorted_src[r] / a.K;
  return min(max(t, (int64_t)0), a.a_rows - 1);
}

__device__ __forceinline__ float silu_mul(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2_t v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ void block_barrier() {
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <int MB, bool UP>
__device__ __forceinline__ void int8_tile(const Int8Args& a, const Tile& tile, int nt,
                                          char* lds) {
  typedef TileShape<MB> S;
  constexpr int OC = UP ? kCols / 2 : kCols;  // output columns of a tile
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wg = wave >> 2, wp = wave & 3;
  const int rows = tile.rows, col0 = nt * OC, cols = min(OC, a.cols - col0);

  // Loads: a wave brings MB times 8 rows of A and 4 times 8 rows of B a stage,
  // 128 bytes a row; load i covers rows 8 (8 i + wave) .. + 7 of the tile.
  // Lane l fills slot l & 7 of row l >> 3 with the row's chunk (l & 7) ^ ((row >> 1)
  // & 7).  Rows past the tile and chunks past k read zeros.
  const int sub = lane >> 3;
  const int chunk = (lane & 7) ^ ((4 * wave + (sub >> 1)) & 7);
  uint32_t a_off[MB], b_off[4];
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int r = 8 * (8 * i + wave) + sub;
    a_off[i] = kNoRow;
    if (r < rows)
      a_off[i] = (uint32_t)(a.sorted_src ? a_row_of(a, tile.row0 + r) : r) * (uint32_t)a.k +
                 (uint32_t)chunk * 16u;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = (8 * (8 * i + wave) + sub) & (OC - 1);
    b_off[i] = r < cols ? (uint32_t)r * (uint32_t)a.k + (uint32_t)chunk * 16u : kNoRow;
  }
  const int64_t w_row = (int64_t)tile.expert * a.cols + col0;
  const __amdgpu_buffer_rsrc_t ra =
      a.sorted_src ? make_rsrc(a.a, (uint32_t)(a.a_rows * a.k))
                   : make_rsrc(a.a + tile.row0 * a.k, (uint32_t)rows * (uint32_t)a.k);
  const uint32_t w_bytes = (uint32_t)cols * (uint32_t)a.k;
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.w + w_row * a.k, w_bytes);
  const __amdgpu_buffer_rsrc_t ru = make_rsrc((UP ? a.w_up : a.w) + w_row * a.k, w_bytes);
  const int nk = (a.k + kStage - 1) / kStage;
  const bool k_in = (nk - 1) * kStage + chunk * 16 < a.k;  // this lane's chunk of the last stage

  auto load_a = [&](int kt, int slot, int i) {
    dma16(ra, kt == nk - 1 && !k_in ? kNoRow : a_off[i], (uint32_t)kt * kStage,
          (lds_void_t*)(lds + slot * S::a_bytes + (8 * i + wave) * 1024));
  };
  // quarter i of stage kt at place q of the ring
  auto load_b = [&](int kt, int q, int i) {
    dma16(UP && i >= 2 ? ru : rw, b_off[i], (uint32_t)kt * kStage,
          (lds_void_t*)(lds + S::b_at + q * kQuarter + wave * 1024));
  };
  auto place = [&](int q) { return q >= S::quarters ? q - S::quarters : q; };

  // Wave (wg, wp): the first or second half of the tile's 32-row blocks, and
  // weight rows 64 wp .. + 63, or with UP 32 wp of w and of w_up.
  const int blocks = (rows + 31) / 32, half = (blocks + 1) / 2;
  const int first = wg ? half : 0;
  const int live = __builtin_amdgcn_readfirstlane(wg ? blocks - half : half);
  int b_row[2];
  b_row[0] = UP ? 32 * wp : 64 * wp;
  b_row[1] = UP ? kCols / 2 + 32 * wp : 64 * wp + 32;
  const bool any = __builtin_amdgcn_readfirstlane(
      live > 0 && (UP ? 32 * wp : 64 * wp) < cols ? 1 : 0) != 0;
  const int fr = lane & 31;
  const int a_base = (32 * first + fr) * kStage;
  const int b_quarter[2] = {b_row[0] >> 6, b_row[1] >> 6};
  const int b_base[2] = {((b_row[0] & 63) + fr) * kStage, ((b_row[1] & 63) + fr) * kStage};
  int slot_of[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) slot_of[s] = ((2 * s + (lane >> 5)) ^ ((lane >> 1) & 7)) * 16;

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
  // once (two loads, the rest in the next stage's first step).  B's ring holds
  // three stages (MB 4), so that all of B three stages on follows in the second
  // and third step; with MB 5 two and a half: there the second half of B two
  // stages on, then the first half three stages on.
  constexpr bool kDeep = S::quarters >= 12;
  constexpr int kAhead = kDeep ? 4 : 2;  // quarters three stages on, in flight at the barrier
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
            lds + S::b_at + place(q0 + b_quarter[f]) * kQuarter + b_base[f] + slot_of[step]);
#pragma unroll
      for (int m = 0; m < NF; ++m)
        fa[set][m] = *reinterpret_cast<const i32x4_t*>(lds + slot * S::a_bytes + a_base +
                                                       32 * m * kStage + slot_of[step]);
    };
#pragma unroll
    for (int i = 0; i < MB; ++i) load_a(0, 0, i);
#pragma unroll
    for (int i = 0; i < 4; ++i) load_b(0, i, i);
    if (nk > 1) {
#pragma unroll
      for (int i = 0; i < MB; ++i) load_a(1, 1, i);
#pragma unroll
      for (int i = 0; i < 4; ++i) load_b(1, 4 + i, i);
    }
    if (nk > 2) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) load_b(2, 8 + i, i);
    }
    if (nk > 2) wait_vmcnt<MB + 4 + kAhead>();
    else if (nk > 1) wait_vmcnt<MB + 4>();
    else wait_vmcnt<0>();
    block_barrier();
    int slot = 0, q0 = 0;  // of stage kt
    if (LIVE > 0) read(0, 0, 0, 0);
    // ld_a1: the rest of A(kt + 1) and, with MB 5, of B(kt + 1); ld_b: B(kt + 2);
    // ld_a2: A(kt + 2); next: there is a stage kt + 1; ahead: loads of B(kt + 2)
    // may be in flight at the barrier.
    auto stage = [&](int kt, auto ld_a1, auto ld_b, auto ld_a2, auto next, auto ahead) {
      const int q1 = place(q0 + 4);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int cur = s & 1;
        if (s == 3 && next) {
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
          if (ahead) wait_vmcnt<kAhead>();
          else wait_vmcnt<0>();
          block_barrier();
        }
        if (s == 0 && ld_a1) {
#pragma unroll
          for (int i = 2; i < MB; ++i) load_a(kt + 1, slot ^ 1, i);
        }
        if (s == 1) {
          if (kDeep) {
            if (ld_b) {
              load_b(kt + 2, place(q1 + 4), 0);
              load_b(kt + 2, place(q1 + 5), 1);
            }
          } else if (ld_a1) {
            load_b(kt + 1, place(q1 + 2), 2);
            load_b(kt + 1, place(q1 + 3), 3);
          }
        }
        if (s == 2 && ld_b) {
          if (kDeep) {
            load_b(kt + 2, place(q1 + 6), 2);
            load_b(kt + 2, place(q1 + 7), 3);
          } else {
            load_b(kt + 2, place(q1 + 4), 0);
            load_b(kt + 2, place(q1 + 5), 1);
          }
        }
        if (s == 3 && ld_a2) {
          load_a(kt + 2, slot, 0);
          load_a(kt + 2, slot, 1);
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
              acc[m][f] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[cur][f], fa[cur][m], acc[m][f],
                                                                0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      slot ^= 1;
      q0 = q1;
    };
    // stage 0: A(1), B(1) and the first of B(2) came with the prologue, with MB 5
    // but for nothing; its barrier leaves those of B(2) in flight
    stage(0, F{}, F{}, nk > 2, nk > 1, nk > 2);
    for (int kt = 1; kt + 2 < nk; ++kt) stage(kt, T{}, T{}, T{}, T{}, T{});
    if (nk >= 3) stage(nk - 2, T{}, F{}, F{}, T{}, F{});
    if (nk >= 2) stage(nk - 1, F{}, F{}, F{}, F{}, F{});
  };
  switch (any ? live : 0) {
    case 0: run(std::integral_constant<int, 0>{}); break;
    case 1: run(std::integral_constant<int, 1>{}); break;
    case 2: run(std::integral_constant<int, 2>{}); break;
    case 3: run(std::integral_constant<int, 3>{}); break;
    case 4: run(std::integral_constant<int, 4>{}); break;
    default: run(std::integral_constant<int, MB>{}); break;
  }

  // ---- epilogue.  The products have the weights first, so a lane holds output
  // row (l & 31) of a block and columns 8 (r / 4) + 4 (l / 32) + r % 4.
  const int ocol = 4 * (lane >> 5);
  const __amdgpu_buffer_rsrc_t rsw = make_rsrc(a.w_scales + w_row, (uint32_t)cols * 4u);
  const __amdgpu_buffer_rsrc_t rsu =
      make_rsrc((UP ? a.w_up_scales : a.w_scales) + w_row, (uint32_t)cols * 4u);
  typedef float f32x4_t __attribute__((ext_vector_type(4)));
  f32x4_t sc[2][4];
  float sr[MB];
  if (any) {
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        sc[f][q] = __builtin_bit_cast(
            f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                         UP && f ? rsu : rsw,
                         (int)((uint32_t)((UP ? 32 * wp : b_row[f]) + 8 * q + ocol) * 4u), 0, 0));
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      const int r = 32 * (first + m) + fr;
      sr[m] = m < live && r < rows ? a.a_scales[a_row_of(a, tile.row0 + r)] : 0.0f;
    }
  }
  __syncthreads();  // the last fragments have been read
  if constexpr (UP) {
    constexpr int kRow = OC * 2 + 8;
    static_assert(S::rows * kRow <= kLds, "staged tile");
    if (any) {
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        if (m >= live) break;
        char* to = lds + (32 * (first + m) + fr) * kRow + (32 * wp + ocol) * 2;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float h[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            h[j] = silu_mul((float)acc[m][0][4 * q + j] * (sr[m] * sc[0][q][j]),
                            (float)acc[m][1][4 * q + j] * (sr[m] * sc[1][q][j]));
          *reinterpret_cast<u32x2_t*>(to + 16 * q) =
              u32x2_t{pack_bf16(h[0], h[1]), pack_bf16(h[2], h[3])};
        }
      }
    }
    __syncthreads();
    // 16 lanes a row
    const int ch = tid & 15;
    if (8 * ch < cols) {
      for (int r = tid >> 4; r < rows; r += 32) {
        const char* from = lds + r * kRow + ch * 16;
        const u32x2_t lo = *reinterpret_cast<const u32x2_t*>(from);
        const u32x2_t hi = *reinterpret_cast<const u32x2_t*>(from + 8);
        *reinterpret_cast<u32x4_t*>(a.out + (tile.row0 + r) * a.cols + col0 + 8 * ch) =
            u32x4_t{lo[0], lo[1], hi[0], hi[1]};
      }
    }
  } else if (any) {
    // the wave's 64 columns of a block, one whole line of every row: through LDS
    // of its own
    constexpr int kRow = 128 + 8;
    char* mine = lds + wave * (32 * kRow + 128);
    const int ch = lane & 7, col = col0 + 64 * wp + 8 * ch;
    const bool col_ok = 64 * wp + 8 * ch < cols;
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      if (m >= live) break;
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float y[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) y[j] = (float)acc[m][f][4 * q + j] * (sr[m] * sc[f][q][j]);
          *reinterpret_cast<u32x2_t*>(mine + fr * kRow + (32 * f + 8 * q + ocol) * 2) =
              u32x2_t{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + sub, at = 32 * (first + m) + r;
        const char* from = mine + r * kRow + ch * 16;
        const u32x2_t lo = *reinterpret_cast<const u32x2_t*>(from);
        const u32x2_t hi = *reinterpret_cast<const u32x2_t*>(from + 8);
        if (col_ok && at < rows)
          *reinterpret_cast<u32x4_t*>(a.out + (tile.row0 + at) * a.cols + col) =
              u32x4_t{lo[0], lo[1], hi[0], hi[1]};
      }
    }
  }
}

// Dense: the tiles of four row tiles follow each other on a column tile, so that
// the blocks of an XCD at work together share both operands.
constexpr int kRowGroup = 4;

template <bool UP>
__global__ __launch_bounds__(512, 2) void int8_dense_kernel(Int8Args a, int64_t m_tiles,
                                                            int col_tiles) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  int64_t item;
  if (!xcd_item(blockIdx.x, m_tiles * col_tiles, item)) return;
  const int64_t group = item / (kRowGroup * col_tiles), in = item % (kRowGroup * col_tiles);
  const int deep = (int)min((int64_t)kRowGroup, m_tiles - group * kRowGroup);
  Tile t;
  t.expert = 0;
  t.row0 = (group * kRowGroup + in % deep) * TileShape<4>::rows;
  t.rows = (int)min((int64_t)TileShape<4>::rows, a.rows - t.row0);
  int8_tile<4, UP>(a, t, (int)(in / deep), lds);
}

template <bool UP>
__global__ __launch_bounds__(512, 2) void int8_grouped_kernel(Int8Args a, int col_tiles) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  constexpr uint32_t bm = TileShape<5>::rows;
  Segments s;
  s.read(a, bm, true);
  int64_t item;
  if (!xcd_item(blockIdx.x, (int64_t)s.total * col_tiles, item)) return;
  const Tile t = s.tile((uint32_t)(item / col_tiles), bm, true);
  if (t.rows <= 0) return;
  int8_tile<5, UP>(a, t, (int)(item % col_tiles), lds);
}

}  // namespace

hipError_t launch_quant_int8(const uint16_t* X, int64_t n, int cols, int8_t* Q, float* S,
                             hipStream_t stream) {
  const int64_t most = int64_t(1) << 24;  // rows a launch: fewer than 2^32 threads
  for (int64_t r0 = 0; r0 < n; r0 += most) {
    const int64_t m = std::min(most, n - r0);
    hipLaunchKernelGGL(quant_int8_kernel, dim3((unsigned)((m + 3) / 4)), dim3(256), 0, stream,
                       reinterpret_cast<const u32x4_t*>(X + r0 * cols), m, cols / 8,
                       reinterpret_cast<u32x2_t*>(Q + r0 * cols), S + r0);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

namespace {
// Both launches' kernels use all of a CU's LDS.
template <class Kernel, class... Args>
hipError_t launch_tiles(Kernel kernel, std::atomic<uint32_t>& configured, int64_t blocks,
                        hipStream_t stream, Args... args) {
  const hipError_t e = set_lds_limit_once((const void*)kernel, kLds, configured);
  if (e != hipSuccess) return e;
  if (blocks >= (int64_t(1) << 23)) return hipErrorInvalidConfiguration;  // 2^32 threads
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(512), kLds, stream, args...);
  return hipGetLastError();
}
int64_t xcd_blocks(int64_t work) { return (work + kXcds - 1) / kXcds * kXcds; }
}  // namespace

hipError_t launch_int8_matmul(const Int8Args& a, hipStream_t stream) {
  static std::atomic<uint32_t> configured[4];
  const int oc = a.w_up ? kCols / 2 : kCols;
  const int col_tiles = (a.cols + oc - 1) / oc;
  if (a.offsets) {
    const int64_t bm = TileShape<5>::rows;
    const int64_t m_tiles = a.rows / bm + std::min<int64_t>(a.E, a.rows);
    const int64_t blocks = xcd_blocks(m_tiles * col_tiles);
    if (a.w_up)
      return launch_tiles(int8_grouped_kernel<true>, configured[0], blocks, stream, a, col_tiles);
    return launch_tiles(int8_grouped_kernel<false>, configured[1], blocks, stream, a, col_tiles);
  }
  const int64_t bm = TileShape<4>::rows, m_tiles = (a.rows + bm - 1) / bm;
  const int64_t blocks = xcd_blocks(m_tiles * col_tiles);
  if (a.w_up)
    return launch_tiles(int8_dense_kernel<true>, configured[2], blocks, stream, a, m_tiles,
                        col_tiles);
  return launch_tiles(int8_dense_kernel<false>, configured[3], blocks, stream, a, m_tiles,
                      col_tiles);
}

}  // namespace moe
