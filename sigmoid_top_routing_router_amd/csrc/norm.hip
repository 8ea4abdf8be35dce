// Root-mean-square norm of the residual stream, with its addition, the
// sandwich form and an E4M3 output, and its backward pass.
//
// "Kolibri 1 im Detail" (block description): every sublayer is normalised
// before and after, then added to the residual stream.  One pass over a row:
//   u = x                              or x * rsqrt(mean(x^2) + eps) * w_post
//   r = residual + u
//   y = r * rsqrt(mean(r^2) + eps) * w
// y leaves in bf16 and / or, per 1 x 128 group, as s = amax / 448 and the
// E4M3 code of y / s; the codes are formed from the fp32 y (one rounding, not
// two).  Backward, with a = rsqrt(mean(r^2) + eps), n = r a, h = dy w:
//   dr = dres + a (h - n mean(h n)),  dw = sum_t dy n,  dresidual = dr,
// and through the sandwich norm of x (b = rsqrt(mean(x^2) + eps), m = x b,
// k = dr w_post): dx = b (k - m mean(k m)), dw_post = sum_t dr m.  The two
// reciprocal roots are formed again from r and x, which are read anyway, so
// the forward pass keeps nothing for it.
//
// All statistics, sums and the row itself are fp32; a row is read once and
// kept in registers, eight columns a thread, so that all of a row's loads are
// in flight at once: rows of up to 512 columns belong to one wave (WAVE; four
// rows to a block of 256, no barrier), wider ones to a block of as many waves
// as they need.  A thread's columns are consecutive (VEC = 8: 16-byte loads of
// bf16) when the width is a multiple of 8 and every pointer 16-byte aligned,
// else a row's threads apart (VEC = 1).
#include "common.h"
#include "kernels.h"

namespace moe {

namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2_t v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ uint16_t one_bf16(float a) {
  return __builtin_bit_cast(uint16_t, (__bf16)a);
}

// VEC consecutive values of a bf16 or fp32 row at column c.
template <int VEC>
__device__ __forceinline__ void load_bf16(const uint16_t* p, float* v) {
  if constexpr (VEC == 8) {
    const u32x4_t t = *reinterpret_cast<const u32x4_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(t[i] << 16);
      v[2 * i + 1] = __uint_as_float(t[i] & 0xFFFF0000u);
    }
  } else {
    v[0] = bf16_bits_to_f32(*p);
  }
}
template <int VEC>
__device__ __forceinline__ void load_f32(const float* p, float* v) {
  if constexpr (VEC == 8) {
    const f32x4_t a = *reinterpret_cast<const f32x4_t*>(p);
    const f32x4_t b = *reinterpret_cast<const f32x4_t*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  } else {
    v[0] = *p;
  }
}
template <int VEC, bool F32>
__device__ __forceinline__ void load_any(const void* base, int64_t at, float* v) {
  if constexpr (F32) load_f32<VEC>(reinterpret_cast<const float*>(base) + at, v);
  else load_bf16<VEC>(reinterpret_cast<const uint16_t*>(base) + at, v);
}
template <int VEC>
__device__ __forceinline__ void store_bf16(uint16_t* p, const float* v) {
  if constexpr (VEC == 8) {
    const u32x4_t t = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                       pack_bf16(v[6], v[7])};
    *reinterpret_cast<u32x4_t*>(p) = t;
  } else {
    *p = one_bf16(v[0]);
  }
}
template <int VEC>
__device__ __forceinline__ void store_f32(float* p, const float* v) {
  if constexpr (VEC == 8) {
    const f32x4_t a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
    *reinterpret_cast<f32x4_t*>(p) = a;
    *reinterpret_cast<f32x4_t*>(p + 4) = b;
  } else {
    *p = v[0];
  }
}

// Sum over the wave: DPP inside each 16-lane row, then the four rows.
__device__ __forceinline__ float wave_sum_f32(float v) {
  v += __uint_as_float(dpp_u32<kDppQuadSwap1>(__float_as_uint(v)));
  v += __uint_as_float(dpp_u32<kDppQuadSwap2>(__float_as_uint(v)));
  v += __uint_as_float(dpp_u32<kDppRowHalfMirror>(__float_as_uint(v)));
  v += __uint_as_float(dpp_u32<kDppRowMirror>(__float_as_uint(v)));
  const uint32_t u = __float_as_uint(v);
  return (__uint_as_float(readlane_u32(u, 0)) + __uint_as_float(readlane_u32(u, 16))) +
         (__uint_as_float(readlane_u32(u, 32)) + __uint_as_float(readlane_u32(u, 48)));
}

// Sums of NS values over a row's wave, or the block's.  `part` holds NS floats
// per wave of the block; it is not written again before the next barrier.
template <bool WAVE, int NS>
__device__ __forceinline__ void row_sums(float (&v)[NS], float* part) {
#pragma unroll
  for (int i = 0; i < NS; ++i) v[i] = wave_sum_f32(v[i]);
  if constexpr (!WAVE) {
    const int wave = threadIdx.x >> 6, W = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < NS; ++i) part[wave * NS + i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] = 0.0f;
    for (int w = 0; w < W; ++w) {
#pragma unroll
      for (int i = 0; i < NS; ++i) v[i] += part[w * NS + i];
    }
  }
}

constexpr int kWaveD = 512;  // widest row of one wave
// Blocks along x of norm_kernel's grid: a grid's threads along x stay below
// 2^32.
constexpr int64_t kGridX = 1 << 20;

constexpr float kE4M3Max = 448.0f;

struct NormArgs {
  const uint16_t* x;
  const void* residual;
  const void* post_w;
  const void* w;
  int64_t n;
  int d;
  float eps;
  bool stream_f32, weight_f32;
  uint16_t* y;
  void* r_out;
  uint8_t* codes;
  float* scales;
};

// Bound by its passes over memory: 65536 x 2560, fp32 stream, sandwich, bf16
// and E4M3 outputs, 2.18 GB in 427 us, 5.1 TB/s.  16384 x 2560, bf16 with an
// fp32 stream: 87 us; with one wave a row (forty columns a lane) 104 us, and
// 64 such rows 3.2 us against 5.8.  512 columns: a wave and a block of one
// wave took the same.
template <bool WAVE, int VEC, bool POST, bool SF32, bool WF32>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void norm_kernel(NormArgs a) {
  constexpr int NV = 8 / VEC;
  __shared__ float part[2][16];
  const int threads = WAVE ? 64 : blockDim.x;  // of a row
  const int t = WAVE ? threadIdx.x & 63 : threadIdx.x;
  const int64_t block = (int64_t)blockIdx.y * kGridX + blockIdx.x;
  const int64_t row = WAVE ? block * 4 + (threadIdx.x >> 6) : block;
  if (row >= a.n) return;  // a whole wave (WAVE: no barrier below)
  const int d = a.d;
  const int64_t base = row * d;
  const float inv_d = 1.0f / (float)d;
  // columns past the row load column 0 and count as 0: a load under a branch
  // would be waited for inside it
  auto inside = [&](int j) { return (j * threads + t) * VEC < d; };
  auto column = [&](int j) { return inside(j) ? (j * threads + t) * VEC : 0; };
  float v[NV][VEC], q[NV][VEC], w[NV][VEC], pw[NV][VEC];
  if (a.residual) {
#pragma unroll
    for (int j = 0; j < NV; ++j) load_any<VEC, SF32>(a.residual, base + column(j), q[j]);
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = column(j);
    load_bf16<VEC>(a.x + base + c, v[j]);
    if constexpr (POST) load_any<VEC, WF32>(a.post_w, c, pw[j]);
    load_any<VEC, WF32>(a.w, c, w[j]);
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      v[j][i] = inside(j) ? v[j][i] : 0.0f;
      w[j][i] = inside(j) ? w[j][i] : 0.0f;
      if constexpr (POST) pw[j][i] = inside(j) ? pw[j][i] : 0.0f;
    }
  if constexpr (POST) {
    float ss[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) ss[0] += v[j][i] * v[j][i];
    row_sums<WAVE>(ss, part[0]);
    const float b = rsqrtf(ss[0] * inv_d + a.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[j][i] = v[j][i] * b * pw[j][i];
  }
  if (a.residual) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[j][i] += inside(j) ? q[j][i] : 0.0f;
  }
  if (a.r_out) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * threads + t) * VEC;
      if (c < d) {
        if constexpr (SF32) store_f32<VEC>(reinterpret_cast<float*>(a.r_out) + base + c, v[j]);
        else store_bf16<VEC>(reinterpret_cast<uint16_t*>(a.r_out) + base + c, v[j]);
      }
    }
  }
  float ss[1] = {0.0f};
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i) ss[0] += v[j][i] * v[j][i];
  row_sums<WAVE>(ss, part[1]);
  const float s = rsqrtf(ss[0] * inv_d + a.eps);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * threads + t) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[j][i] = v[j][i] * s * w[j][i];
    if (c < d && a.y) store_bf16<VEC>(a.y + base + c, v[j]);
    if constexpr (VEC == 8) {
      // 16 neighbouring lanes hold one 1 x 128 group (d % 128 == 0 here), all
      // of them inside the row or none
      if (a.codes) {
        // as integers the magnitudes keep their order and a NaN comes last, so
        // that a group with a NaN gets a NaN scale and not the others' codes
        uint32_t mb = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) mb = max(mb, __float_as_uint(v[j][i]) & 0x7FFFFFFFu);
        const float m = __uint_as_float(row16_max_u32(mb));
        const float sc = m / kE4M3Max;
        u32x2_t q = {0u, 0u};
        if (m != 0.0f) {
          float z[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            z[i] = fminf(fmaxf(v[j][i] / sc, -kE4M3Max), kE4M3Max);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            int pk = __builtin_amdgcn_cvt_pk_fp8_f32(z[4 * k], z[4 * k + 1], 0, false);
            pk = __builtin_amdgcn_cvt_pk_fp8_f32(z[4 * k + 2], z[4 * k + 3], pk, true);
            q[k] = (uint32_t)pk;
          }
        }
        if (c < d) {
          *reinterpret_cast<u32x2_t*>(a.codes + base + c) = q;
          if ((threadIdx.x & 15) == 0) a.scales[(base + c) >> 7] = (m != 0.0f) ? sc : 0.0f;
        }
      }
    }
  }
}

struct NormGradArgs {
  const uint16_t* dy;
  const void* r;
  const uint16_t* x;
  const void* dres;
  const void* w;
  const void* post_w;
  int64_t n;
  int d;
  float eps;
  bool stream_f32, weight_f32;
  uint16_t* dx;
  void* dr_out;
  float* part_w;     // [blocks][d] partial sums of dw, then (POST) of dw_post
};

// Grid-stride over the rows; a thread keeps the sums of its own eight columns
// over the block's rows, and every block leaves one partial row of them (its
// rows' groups added in order through LDS), so the result does not depend on
// the order in which blocks run.  A row belongs to one wave (WAVE, four rows
// to a block of 256) or to the whole block, as many waves as its columns need;
// everything it reads is asked for before the first sum: the passes over memory
// bound it (16384 x 2560, fp32 stream, sandwich: 755 MB in 139 us, 5.4 TB/s; a
// wave per row, forty columns a lane and two waves a SIMD, took 250 us).
template <bool WAVE, int VEC, bool POST, bool SF32, bool WF32>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void norm_grad_kernel(NormGradArgs a) {
  constexpr int NV = 8 / VEC;
  constexpr int RPB = WAVE ? 4 : 1;
  __shared__ float part[2][2][2 * 16];
  const int threads = WAVE ? 64 : blockDim.x;  // of a row
  const int t = WAVE ? threadIdx.x & 63 : threadIdx.x;
  const int sub = WAVE ? threadIdx.x >> 6 : 0;
  const int d = a.d;
  const float inv_d = 1.0f / (float)d;
  // as in norm_kernel
  auto inside = [&](int j) { return (j * threads + t) * VEC < d; };
  auto column = [&](int j) { return inside(j) ? (j * threads + t) * VEC : 0; };
  float dw[NV][VEC], dp[NV][VEC], w[NV][VEC], pw[NV][VEC];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) dw[j][i] = dp[j][i] = 0.0f;
    load_any<VEC, WF32>(a.w, column(j), w[j]);
    if constexpr (POST) load_any<VEC, WF32>(a.post_w, column(j), pw[j]);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      w[j][i] = inside(j) ? w[j][i] : 0.0f;
      if constexpr (POST) pw[j][i] = inside(j) ? pw[j][i] : 0.0f;
    }
  }
  int flip = 0;
  // a block of one row at a time has one loop count, for the barriers
  for (int64_t row = (int64_t)blockIdx.x * RPB + sub; row < a.n;
       row += (int64_t)gridDim.x * RPB, flip ^= 1) {
    const int64_t base = row * d;
    float r[NV][VEC], g[NV][VEC], q[NV][VEC], xs[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = column(j);
      load_any<VEC, SF32>(a.r, base + c, r[j]);
      load_bf16<VEC>(a.dy + base + c, g[j]);
      if constexpr (POST) load_bf16<VEC>(a.x + base + c, xs[j]);
    }
    if (a.dres) {
#pragma unroll
      for (int j = 0; j < NV; ++j) load_any<VEC, SF32>(a.dres, base + column(j), q[j]);
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) q[j][i] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        r[j][i] = inside(j) ? r[j][i] : 0.0f;
        g[j][i] = inside(j) ? g[j][i] : 0.0f;
        q[j][i] = inside(j) ? q[j][i] : 0.0f;
        if constexpr (POST) xs[j][i] = inside(j) ? xs[j][i] : 0.0f;
      }
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        s[0] += r[j][i] * r[j][i];
        s[1] += g[j][i] * w[j][i] * r[j][i];
      }
    row_sums<WAVE>(s, part[flip][0]);
    const float ra = rsqrtf(s[0] * inv_d + a.eps);
    // the mean first: n and mean(h n) have the sizes of 1 and h at any scale of
    // r, a^3 leaves fp32 below 1e-13 and above 1e12
    const float mean1 = ra * s[1] * inv_d;  // mean(h n)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * threads + t) * VEC;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float n = r[j][i] * ra;
        dw[j][i] += g[j][i] * n;
        r[j][i] = q[j][i] + ra * (g[j][i] * w[j][i] - n * mean1);  // dr from here on
      }
      if (c < d) {
        if (a.dr_out) {
          if constexpr (SF32) store_f32<VEC>(reinterpret_cast<float*>(a.dr_out) + base + c, r[j]);
          else store_bf16<VEC>(reinterpret_cast<uint16_t*>(a.dr_out) + base + c, r[j]);
        }
        if (!POST && a.dx) store_bf16<VEC>(a.dx + base + c, r[j]);
      }
    }
    if constexpr (POST) {
      float p[2] = {0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          p[0] += xs[j][i] * xs[j][i];
          p[1] += r[j][i] * pw[j][i] * xs[j][i];
        }
      row_sums<WAVE>(p, part[flip][1]);
      const float rb = rsqrtf(p[0] * inv_d + a.eps);
      const float mean2 = rb * p[1] * inv_d;  // mean(k m)
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * threads + t) * VEC;
        float o[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float m = xs[j][i] * rb;
          dp[j][i] += r[j][i] * m;
          o[i] = rb * (r[j][i] * pw[j][i] - m * mean2);
        }
        if (c < d && a.dx) store_bf16<VEC>(a.dx + base + c, o);
      }
    }
  }
  // the block's partial row
  float* out = a.part_w + (int64_t)blockIdx.x * (POST ? 2 : 1) * d;
  if constexpr (!WAVE) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * threads + t) * VEC;
      if (c < d) {
        store_f32<VEC>(out + c, dw[j]);
        if (POST) store_f32<VEC>(out + d + c, dp[j]);
      }
    }
  } else {
    // the four waves' sums in order
    __shared__ float red[RPB][512];
#pragma unroll
    for (int q = 0; q < (POST ? 2 : 1); ++q) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          red[sub][(j * 64 + t) * VEC + i] = q ? dp[j][i] : dw[j][i];
      __syncthreads();
      for (int c = threadIdx.x; c < d; c += 256)
        out[q * d + c] = (red[0][c] + red[1][c]) + (red[2][c] + red[3][c]);
    }
  }
}

// Sums the partial rows [rows][cols] in a fixed order: a block takes 32
// columns, 32 groups of rows, then the groups in order.
__global__ __launch_bounds__(1024) void sum_rows_kernel(const float* __restrict__ part, int rows,
                                                        int cols, int d, float* __restrict__ out0,
                                                        float* __restrict__ out1) {
  __shared__ float red[32][33];
  const int cx = threadIdx.x & 31, gy = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cx;
  float s = 0.0f;
  if (c < cols)
#pragma unroll 8
    for (int r = gy; r < rows; r += 32) s += part[(int64_t)r * cols + c];
  red[gy][cx] = s;
  __syncthreads();
  if (gy == 0 && c < cols) {
    float v = 0.0f;
#pragma unroll
    for (int g = 0; g < 32; ++g) v += red[g][cx];
    if (c < d) { if (out0) out0[c] = v; }
    else if (out1) out1[c - d] = v;
  }
}

bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

int row_threads(int d) { return (d + 511) / 512 * 64; }

// The kernels are built for every form (row of a wave or a block, vector width,
// sandwich or not, types of the stream and of the weights): a type chosen at
// run time inside them puts a branch around every load, which the compiler
// then waits for one by one (1025 x 1001, sandwich, backward: 18.8 us, 15.2
// without those branches, 9 without the ones on the row's end too).
#define MOE_NORM_TYPES(kernel, wave, vec, post)                                             \
  do {                                                                                      \
    if (a.stream_f32 && a.weight_f32)                                                       \
      hipLaunchKernelGGL((kernel<wave, vec, post, true, true>), grid, dim3(threads), 0,     \
                         stream, a);                                                        \
    else if (a.stream_f32)                                                                  \
      hipLaunchKernelGGL((kernel<wave, vec, post, true, false>), grid, dim3(threads), 0,    \
                         stream, a);                                                        \
    else if (a.weight_f32)                                                                  \
      hipLaunchKernelGGL((kernel<wave, vec, post, false, true>), grid, dim3(threads), 0,    \
                         stream, a);                                                        \
    else                                                                                    \
      hipLaunchKernelGGL((kernel<wave, vec, post, false, false>), grid, dim3(threads), 0,   \
                         stream, a);                                                        \
  } while (0)
#define MOE_NORM_FORM(kernel, wave, vec)                          \
  do {                                                            \
    if (a.post_w) MOE_NORM_TYPES(kernel, wave, vec, true);        \
    else MOE_NORM_TYPES(kernel, wave, vec, false);                \
  } while (0)
#define MOE_NORM_LAUNCH(kernel)                                   \
  do {                                                            \
    if (wave && vec) MOE_NORM_FORM(kernel, true, 8);              \
    else if (vec) MOE_NORM_FORM(kernel, false, 8);                \
    else if (wave) MOE_NORM_FORM(kernel, true, 1);                \
    else MOE_NORM_FORM(kernel, false, 1);                         \
  } while (0)

}  // namespace

hipError_t launch_rms_norm(const uint16_t* x, const void* residual, const void* post_w,
                           const void* w, int64_t n, int d, float eps, bool stream_f32,
                           bool weight_f32, uint16_t* y, void* r_out, uint8_t* codes,
                           float* scales, hipStream_t stream) {
  if (n <= 0) return hipSuccess;
  if (d < 1 || d > kNormMaxD) return hipErrorInvalidValue;
  const NormArgs a{x, residual, post_w, w, n, d, eps, stream_f32, weight_f32, y, r_out, codes, scales};
  const bool vec = d % 8 == 0 && al16(x) && al16(residual) && al16(post_w) && al16(w) && al16(y) &&
                   al16(r_out) && al16(codes);
  // a 1 x 128 group is 16 lanes of 8 columns
  if (codes && (!vec || d % 128)) return hipErrorInvalidValue;
  const bool wave = d <= kWaveD;
  const int64_t blocks = wave ? (n + 3) / 4 : n;
  const dim3 grid((unsigned)(blocks < kGridX ? blocks : kGridX),
                  (unsigned)((blocks + kGridX - 1) / kGridX));
  const int threads = wave ? 256 : row_threads(d);
  MOE_NORM_LAUNCH(norm_kernel);
  return hipGetLastError();
}

// Blocks, and so partial rows.  Rows of a block: some twelve waves a CU in a
// whole number of blocks (16384 x 2560, sandwich, five waves a row: 138 us with
// 512 blocks, 161 with 1024, 176 with 256), two rows each or more (256 x 2560:
// 7 us, with four rows 10, with eight 16).  Rows of a wave: up to four blocks a
// CU (65536 x 256: 27 us with 1024 blocks, 38 with 512, 28 with 2048).  Measured
// at these two widths only; the others follow from the waves a CU holds.
int rms_norm_grad_blocks(int64_t n, int d) {
  const bool wave = d <= kWaveD;
  const int waves = (d + 511) / 512;
  const int64_t most = 256 * (wave ? 4 : waves < 12 ? 12 / waves : 1);
  const int64_t per = wave ? 4 : 2;
  const int64_t need = (n + per - 1) / per;
  return (int)(need < 1 ? 1 : need < most ? need : most);
}

hipError_t launch_rms_norm_grad(const uint16_t* dy, const void* r, const uint16_t* x,
                                const void* dres, const void* w, const void* post_w, int64_t n,
                                int d, float eps, bool stream_f32, bool weight_f32, uint16_t* dx,
                                void* dr_out, float* dw, float* dw_post, float* part,
                                hipStream_t stream) {
  if (n < 0 || d < 1 || d > kNormMaxD) return hipErrorInvalidValue;
  const int blocks = rms_norm_grad_blocks(n, d);
  const NormGradArgs a{dy, r, x, dres, w, post_w, n, d, eps, stream_f32, weight_f32, dx, dr_out, part};
  const bool vec = d % 8 == 0 && al16(dy) && al16(r) && al16(x) && al16(dres) && al16(w) &&
                   al16(post_w) && al16(dx) && al16(dr_out);
  const bool wave = d <= kWaveD;
  const int threads = wave ? 256 : row_threads(d);
  const dim3 grid((unsigned)blocks);
  MOE_NORM_LAUNCH(norm_grad_kernel);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (!dw && !dw_post) return hipSuccess;
  const int cols = post_w ? 2 * d : d;
  hipLaunchKernelGGL(sum_rows_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(1024), 0, stream,
                     part, blocks, cols, d, dw, dw_post);
  return hipGetLastError();
}

}  // namespace moe
