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

#include "common.h"
#include "fp8_codes.h"
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
// Rows of one tile: expert, first row, rows; false past the last tile.  Every
// lane of a wave calls it; the segments are clamped to [0, rows), so offsets
// that do not ascend give no access out of range.
struct Tile {
  int expert, rows;
  int64_t row0;
};
__device__ __forceinline__ bool find_tile(const Int8Args& a, int64_t mt, int bm, Tile& out) {
  if (!a.offsets) {
    out.expert = 0;
    out.row0 = mt * bm;
    out.rows = (int)min((int64_t)bm, a.rows - out.row0);
    return out.rows > 0;
  }
  const int lane = lane_id();
  int64_t before = 0;  // tiles of the experts before this group of 64
  for (int e0 = 0; e0 < a.E; e0 += kWave) {
    const int e = e0 + lane;
    int64_t lo = 0, hi = 0;
    if (e < a.E) {
      lo = min(max((int64_t)a.offsets[e], (int64_t)0), a.rows);
      hi = min(max((int64_t)a.offsets[e + 1], lo), a.rows);
    }
    const uint32_t tiles = (uint32_t)((hi - lo + bm - 1) / bm);
    const uint32_t incl = wave_inclusive_sum_u32(tiles);
    const uint32_t total = readlane_u32(incl, kWave - 1);
    if (mt < before + total) {
      const uint64_t past = ballot((int64_t)incl + before > mt);
      const int l = __ffsll((unsigned long long)past) - 1;
      const int64_t first = before + readlane_u32(incl, l) - readlane_u32(tiles, l);
      const int64_t lo_l = readlane_u32((uint32_t)lo, l), hi_l = readlane_u32((uint32_t)hi, l);
      out.expert = e0 + l;
      out.row0 = lo_l + (mt - first) * bm;
      out.rows = (int)min((int64_t)bm, hi_l - out.row0);
      return true;
    }
    before += total;
  }
  return false;
}

// The row of A behind output row r, and of its scale.
__device__ __forceinline__ int64_t a_row_of(const Int8Args& a, int64_t r) {
  if (!a.sorted_src) return r;
  const int64_t t = (int64_t)a.sorted_src[r] / a.K;
  return min(max(t, (int64_t)0), a.a_rows - 1);
}

__device__ __forceinline__ float silu_mul(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

// 64 rows x 64 columns a block, 32 x 32 a wave, operands straight from memory.
template <bool UP>
__global__ __launch_bounds__(256) void int8_plain_kernel(Int8Args a, int col_tiles) {
  Tile tile;
  if (!find_tile(a, (int64_t)blockIdx.x / col_tiles, 64, tile)) return;
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  const int rr = 32 * (wave & 1) + (lane & 31);
  const int cc = (int)(blockIdx.x % col_tiles) * 64 + 32 * (wave >> 1);
  const bool row_ok = rr < tile.rows;
  const int64_t ar = row_ok ? a_row_of(a, tile.row0 + rr) : 0;
  const int wc = cc + (lane & 31);
  const bool col_ok = wc < a.cols;
  const int8_t* pa = a.a + ar * a.k;
  const int64_t wr = (int64_t)tile.expert * a.cols + (col_ok ? wc : 0);
  const int8_t* pw = a.w + wr * a.k;
  const int8_t* pu = UP ? a.w_up + wr * a.k : nullptr;
  i32x16_t acc = {}, accu = {};
  for (int k0 = 0; k0 < a.k; k0 += 32) {
    const int k = k0 + 16 * (lane >> 5);
    const bool in = k < a.k;
    const i32x4_t z = {0, 0, 0, 0};
    const i32x4_t fa = in && row_ok ? *reinterpret_cast<const i32x4_t*>(pa + k) : z;
    const i32x4_t fw = in && col_ok ? *reinterpret_cast<const i32x4_t*>(pw + k) : z;
    acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw, fa, acc, 0, 0, 0);
    if (UP) {
      const i32x4_t fu = in && col_ok ? *reinterpret_cast<const i32x4_t*>(pu + k) : z;
      accu = __builtin_amdgcn_mfma_i32_32x32x32_i8(fu, fa, accu, 0, 0, 0);
    }
  }
  if (!row_ok) return;
  const float sa = a.a_scales[ar];
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int col = cc + 8 * (r / 4) + 4 * (lane >> 5) + r % 4;
    if (col >= a.cols) continue;
    const int64_t sc = (int64_t)tile.expert * a.cols + col;
    float y = (float)acc[r] * (sa * a.w_scales[sc]);
    if (UP) y = silu_mul(y, (float)accu[r] * (sa * a.w_up_scales[sc]));
    a.out[(tile.row0 + rr) * a.cols + col] = __builtin_bit_cast(uint16_t, (__bf16)y);
  }
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

hipError_t launch_int8_matmul(const Int8Args& a, hipStream_t stream) {
  const int64_t col_tiles = (a.cols + 63) / 64;
  const int64_t m_tiles = a.offsets ? a.rows / 64 + a.E : (a.rows + 63) / 64;
  const int64_t blocks = m_tiles * col_tiles;
  if (blocks >= (int64_t(1) << 24)) return hipErrorInvalidConfiguration;
  if (a.w_up)
    hipLaunchKernelGGL(int8_plain_kernel<true>, dim3((unsigned)blocks), dim3(256), 0, stream, a,
                       (int)col_tiles);
  else
    hipLaunchKernelGGL(int8_plain_kernel<false>, dim3((unsigned)blocks), dim3(256), 0, stream, a,
                       (int)col_tiles);
  return hipGetLastError();
}

}  // namespace moe
