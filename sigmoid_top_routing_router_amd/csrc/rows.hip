// Rows of tokens on their way to the experts and back, and the gradients.
//
// "Kolibri Pre-Training from Scratch" §6.1: y_t = f_shared(x_t) + sum_k s_tk
// f_e(x_t), e = I_tk.  With pos(t, k) the place of pair (t, k) in the order
// grouped by expert (permute.hip; none for a pair whose expert is elsewhere),
// base the shared expert's output and R the experts' output rows:
//   permute            rows[pos(t, k)] = x_t
//   permute_backward   dx_t = sum_k drows[pos(t, k)]
//   unpermute          y_t = base_t + sum_k s_tk R[pos(t, k)]
//   unpermute_backward dR[pos(t, k)] = s_tk dy_t,  ds_tk = <dy_t, R[pos(t, k)]>
// ("Kolibri 1 im Detail", routing section: tokens are brought to their experts
// with no per-expert capacity.)  Every kernel walks the tokens, so a token's
// row is read or written once and each grouped row once; a pair's place is
// checked against the number of pairs, so that no access leaves the rows.
// Sums over k run in fp32 in the order of k and are rounded once.
//
// Rows kept in 8 bits are E4M3 codes with one fp32 scale per 1 x 128 group (the
// rule of fp8_quant.hip): unpermute can leave them for the rows that it reads,
// permute and unpermute_backward read them in the place of bf16 rows.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "fp8_codes.h"
#include "kernels.h"
#include "lane_swaps.h"

namespace moe {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// What a thread moves of a row: 16 bytes, at any element (gfx950 takes them from any
// address), or one element of rows shorter than that.  The last piece of a row that
// is not whole pieces ends with the row and repeats elements of the one before it:
// copies and sums write the same values there twice, dot products leave them out.
// (Element by element, 1237 tokens of 777 fp32, five each: the gradients 18.8 us;
// this way 8.7.)
template <bool F32, bool VEC>
struct Piece;
typedef u32x4_t u32x4b_t __attribute__((aligned(2)));  // of bf16 elements
typedef u32x4_t u32x4f_t __attribute__((aligned(4)));  // of fp32 elements
template <>
struct Piece<false, true> {
  typedef u32x4_t raw;
  typedef u32x4b_t mem;
  static constexpr bool F32 = false;
  static constexpr int V = 8;
  static __device__ __forceinline__ void open(raw v, float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(v[i] << 16);
      f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ raw close(const float (&f)[V]) {
    return raw{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
               pack_bf16(f[6], f[7])};
  }
};
template <>
struct Piece<true, true> {
  typedef u32x4_t raw;
  typedef u32x4f_t mem;
  static constexpr bool F32 = true;
  static constexpr int V = 4;
  static __device__ __forceinline__ void open(raw v, float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
  }
  static __device__ __forceinline__ raw close(const float (&f)[V]) {
    return raw{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
               __float_as_uint(f[3])};
  }
};
template <>
struct Piece<false, false> {
  typedef uint16_t raw;
  typedef uint16_t mem;
  static constexpr bool F32 = false;
  static constexpr int V = 1;
  static __device__ __forceinline__ void open(raw v, float (&f)[V]) { f[0] = bf16_to_f32(v); }
  static __device__ __forceinline__ raw close(const float (&f)[V]) {
    return __builtin_bit_cast(uint16_t, (__bf16)f[0]);
  }
};
template <>
struct Piece<true, false> {
  typedef uint32_t raw;
  typedef uint32_t mem;
  static constexpr bool F32 = true;
  static constexpr int V = 1;
  static __device__ __forceinline__ void open(raw v, float (&f)[V]) { f[0] = __uint_as_float(v); }
  static __device__ __forceinline__ raw close(const float (&f)[V]) { return __float_as_uint(f[0]); }
};

// Eight E4M3 codes times their group's scale, in fp32.
__device__ __forceinline__ void open_codes(u32x2_t c, float s, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], false);
    const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], true);
    f[4 * i] = lo[0] * s;
    f[4 * i + 1] = lo[1] * s;
    f[4 * i + 2] = hi[0] * s;
    f[4 * i + 3] = hi[1] * s;
  }
}

// quant8 of fp8_codes.h, with the quotients v / s as q = v y, q + (v - s q) y, y =
// 1 / s: three operations for the division's ten.  The residual is exact but for 35 of
// the 2^14 pairs of significands of v and of the group's maximum, where it has 25 bits;
// the sum is the rounded quotient for each of them (all tried in exact arithmetic).
// divide: s is infinite, or so small that the residual would lose bits below the
// smallest subnormal.  16384 tokens of 2560, six each, with codes: 187 us with divisions, 155 so.
__device__ __forceinline__ uint2 quant8_by(uint4 v, float s, float y, bool divide) {
  if (divide) return quant8(v, s);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  auto quotient = [&](uint32_t bits) {
    const float x = __uint_as_float(bits), q = x * y;
    return fminf(fmaxf(fmaf(fmaf(-s, q, x), y, q), -kE4M3Max), kE4M3Max);
  };
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = fp8x2(quotient(w[i] << 16), quotient(w[i] & 0xFFFF0000u));
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// Rows of d elements in ppr pieces.
struct Shape {
  uint32_t d, ppr, n_rows;
  // first element of piece c of a row
  template <int V>
  __device__ __forceinline__ int64_t at(int64_t row, uint32_t c) const {
    return row * d + min(c * V, d - V);
  }
  // elements that the piece repeats
  template <int V>
  __device__ __forceinline__ uint32_t repeated(uint32_t c) const {
    return c * V - min(c * V, d - V);
  }
};
// Of the tokens' rows, which the call before often left in the memory-side cache
// and the K pairs' blocks share; NT: of the grouped rows, read once (16384 tokens of
// 2560 bf16, six each: permute 98 us with the former so, 115 with non-temporal loads;
// the sum of grouped rows 99 with the latter so, 106 without).
template <class P, bool NT>
__device__ __forceinline__ typename P::raw load_piece(const void* p, int64_t at) {
  typedef typename std::conditional<P::F32, uint32_t, uint16_t>::type elem;
  const typename P::mem* from =
      reinterpret_cast<const typename P::mem*>(reinterpret_cast<const elem*>(p) + at);
  if constexpr (NT) return __builtin_nontemporal_load(from);
  else return *from;
}
template <class P, bool NT>
__device__ __forceinline__ void store_piece(typename P::raw v, void* p, int64_t at) {
  typedef typename std::conditional<P::F32, uint32_t, uint16_t>::type elem;
  typename P::mem* to = reinterpret_cast<typename P::mem*>(reinterpret_cast<elem*>(p) + at);
  if constexpr (NT) __builtin_nontemporal_store(v, to);
  else *to = v;
}

// Token and piece of a thread in a launch over all pieces of all rows.
__device__ __forceinline__ bool piece_of(int64_t N, uint32_t ppr, int64_t& t, uint32_t& c) {
  const int64_t first = (int64_t)blockIdx.x * 256, t0 = first / ppr;
  const uint32_t r = (uint32_t)(first - t0 * ppr) + threadIdx.x;
  t = t0 + r / ppr;
  c = r % ppr;
  return t < N;
}

// KEPT: x are codes, with scales xs.
template <bool F32, bool VEC, bool KEPT, int K>
__global__ __launch_bounds__(256) void permute_kernel(
    const void* __restrict__ x, const float* __restrict__ xs, const int32_t* __restrict__ src_pos,
    int64_t N, Shape shape, void* __restrict__ rows) {
  typedef Piece<F32, VEC> P;
  int64_t t;
  uint32_t c;
  if (!piece_of(N, shape.ppr, t, c)) return;
  uint32_t p[K];
#pragma unroll
  for (int k = 0; k < K; ++k) p[k] = (uint32_t)src_pos[t * K + k];
  typename P::raw v;
  if constexpr (KEPT) {
    const int64_t at = t * shape.ppr + c;
    float f[8];
    open_codes(reinterpret_cast<const u32x2_t*>(x)[at], xs[at >> 4], f);
    v = P::close(f);
  } else {
    v = load_piece<P, false>(x, shape.at<P::V>(t, c));
  }
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (p[k] < shape.n_rows) store_piece<P, true>(v, rows, shape.at<P::V>(p[k], c));
}

// y = base + sum_k w R (w NULL: 1, base NULL: 0).  KEEP: the rows' codes too;
// 16 lanes hold a group of a row.
template <bool F32, bool VEC, bool KEEP, int K>
__global__ __launch_bounds__(256) void unpermute_kernel(
    const void* __restrict__ rows, const int32_t* __restrict__ src_pos,
    const float* __restrict__ w, const void* __restrict__ base, int64_t N, Shape shape,
    void* __restrict__ y, u32x2_t* __restrict__ codes, float* __restrict__ scales) {
  typedef Piece<F32, VEC> P;
  int64_t t;
  uint32_t c;
  if (!piece_of(N, shape.ppr, t, c)) return;
  uint32_t p[K];
  float s[K];
  typename P::raw v[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    p[k] = (uint32_t)src_pos[t * K + k];
    s[k] = w ? w[t * K + k] : 1.0f;
  }
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (p[k] < shape.n_rows) v[k] = load_piece<P, true>(rows, shape.at<P::V>(p[k], c));
  float acc[P::V];
  if (base) {
    P::open(load_piece<P, false>(base, shape.at<P::V>(t, c)), acc);
  } else {
#pragma unroll
    for (int j = 0; j < P::V; ++j) acc[j] = 0.0f;
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (p[k] >= shape.n_rows) continue;
    float f[P::V];
    P::open(v[k], f);
#pragma unroll
    for (int j = 0; j < P::V; ++j) acc[j] = fmaf(s[k], f[j], acc[j]);
    if constexpr (KEEP) {
      const uint4 u = make_uint4(v[k][0], v[k][1], v[k][2], v[k][3]);
      const float top = __uint_as_float(row16_max_u32(abs_max8(u)));
      const float scale = top / kE4M3Max;
      const bool divide = !(top >= 0x1p-60f && top < __builtin_inff());
      const uint2 q =
          top != 0.0f ? quant8_by(u, scale, 1.0f / scale, divide) : make_uint2(0, 0);
      const int64_t at = (int64_t)p[k] * shape.ppr + c;
      __builtin_nontemporal_store(u32x2_t{q.x, q.y}, codes + at);
      if ((threadIdx.x & 15) == 0) scales[at >> 4] = top != 0.0f ? scale : 0.0f;
    }
  }
  store_piece<P, false>(P::close(acc), y, shape.at<P::V>(t, c));
}

// LANES lanes take a token: its dy row once, the K rows beside it.  KEPT: the rows
// are codes.
template <bool F32, bool VEC, bool KEPT, int K, int LANES>
__global__ __launch_bounds__(256) void unpermute_grad_kernel(
    const void* __restrict__ dy, const void* __restrict__ rows, const float* __restrict__ scales,
    const int32_t* __restrict__ src_pos, const float* __restrict__ w, int64_t N, Shape shape,
    void* __restrict__ drows, float* __restrict__ dw) {
  typedef Piece<F32, VEC> P;
  const uint32_t lane = threadIdx.x % LANES;
  const int64_t t = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  if (t >= N) return;
  uint32_t p[K];
  float s[K], dot[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    p[k] = (uint32_t)src_pos[t * K + k];
    s[k] = w ? w[t * K + k] : 1.0f;
    dot[k] = 0.0f;
  }
  for (uint32_t c = lane; c < shape.ppr; c += LANES) {
    const typename P::raw gv = load_piece<P, false>(dy, shape.at<P::V>(t, c));
    typename P::raw v[K];
    u32x2_t q[K];
    float qs[K];
    if (dw) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (p[k] >= shape.n_rows) continue;
        if constexpr (KEPT) {
          const int64_t at = (int64_t)p[k] * shape.ppr + c;
          q[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(rows) + at);
          qs[k] = scales[at >> 4];
        } else {
          v[k] = load_piece<P, true>(rows, shape.at<P::V>(p[k], c));
        }
      }
    }
    float g[P::V];
    P::open(gv, g);
    const uint32_t skip = shape.repeated<P::V>(c);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (p[k] >= shape.n_rows) continue;
      if (drows) {
        float o[P::V];
#pragma unroll
        for (int j = 0; j < P::V; ++j) o[j] = s[k] * g[j];
        store_piece<P, true>(P::close(o), drows, shape.at<P::V>(p[k], c));
      }
      if (dw) {
        float f[P::V];
        if constexpr (KEPT) open_codes(q[k], qs[k], f);
        else P::open(v[k], f);
#pragma unroll
        for (int j = 0; j < P::V; ++j)
          if (KEPT || (uint32_t)j >= skip) dot[k] = fmaf(g[j], f[j], dot[k]);
      }
    }
  }
  if (!dw) return;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int o = (LANES < kWave ? LANES : kWave) / 2; o > 0; o >>= 1)
      dot[k] += __shfl_xor(dot[k], o);
  if constexpr (LANES > kWave) {
    static_assert(LANES == 256, "the block's four waves");
    __shared__ float part[4][K];
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (lane % kWave == 0) part[lane / kWave][k] = dot[k];
    __syncthreads();
    if (lane < K)
      dw[t * K + lane] = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (lane == 0) dw[t * K + k] = dot[k];
  }
}

// fn(K) with K as a constant.
template <class F>
hipError_t with_k(int K, F&& fn) {
  switch (K) {
#define MOE_K_CASE(n) case n: fn(std::integral_constant<int, n>{}); break;
    MOE_K_CASE(1) MOE_K_CASE(2) MOE_K_CASE(3) MOE_K_CASE(4)
    MOE_K_CASE(5) MOE_K_CASE(6) MOE_K_CASE(7) MOE_K_CASE(8)
#undef MOE_K_CASE
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}
// Pieces of a row; vec: of 16 bytes.
Shape shape_of(int64_t N, int d, int K, bool f32, bool& vec) {
  const int V = f32 ? 4 : 8;
  vec = d >= V;
  return Shape{(uint32_t)d, (uint32_t)(vec ? (d + V - 1) / V : d), (uint32_t)(N * K)};
}
template <class T>
T* at(T* p, int64_t bytes) {
  typedef typename std::conditional<std::is_const<T>::value, const char, char>::type byte;
  return p ? reinterpret_cast<T*>(reinterpret_cast<byte*>(p) + bytes) : nullptr;
}
// Calls fn(t0, n) for runs of tokens whose launch stays below 2^31 threads.
template <class F>
hipError_t token_runs(int64_t N, int64_t threads_per_token, F&& fn) {
  const int64_t most = std::max<int64_t>(1, ((int64_t(1) << 31) - 256) / threads_per_token);
  for (int64_t t0 = 0; t0 < N; t0 += most) {
    const hipError_t e = fn(t0, std::min(most, N - t0));
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
unsigned blocks_of(int64_t threads) { return (unsigned)((threads + 255) / 256); }

}  // namespace

hipError_t launch_permute_rows(const void* x, const float* x_scales, const int32_t* src_pos,
                               int64_t N, int d, int K, bool f32, void* rows, hipStream_t stream) {
  const bool kept = x_scales != nullptr;
  bool vec;
  const Shape shape = shape_of(N, d, K, f32, vec);
  const int es = f32 ? 4 : 2;
  return token_runs(N, shape.ppr, [&](int64_t t0, int64_t n) {
    const void* xt = at(x, t0 * d * (kept ? 1 : es));
    const float* st = x_scales ? x_scales + t0 * (d / 128) : nullptr;
    const dim3 grid(blocks_of(n * shape.ppr)), block(256);
    return with_k(K, [&](auto k) {
      constexpr int kk = decltype(k)::value;
      auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, block, 0, stream, xt, st, src_pos + t0 * K, n,
                           shape, rows);
      };
      if (kept) go(permute_kernel<false, true, true, kk>);
      else if (f32 && vec) go(permute_kernel<true, true, false, kk>);
      else if (f32) go(permute_kernel<true, false, false, kk>);
      else if (vec) go(permute_kernel<false, true, false, kk>);
      else go(permute_kernel<false, false, false, kk>);
    });
  });
}

hipError_t launch_unpermute_rows(const void* rows, const int32_t* src_pos, const float* w,
                                 const void* base, int64_t N, int d, int K, bool f32, void* y,
                                 uint8_t* codes, float* scales, hipStream_t stream) {
  bool vec;
  const Shape shape = shape_of(N, d, K, f32, vec);
  const int es = f32 ? 4 : 2;
  return token_runs(N, shape.ppr, [&](int64_t t0, int64_t n) {
    const dim3 grid(blocks_of(n * shape.ppr)), block(256);
    return with_k(K, [&](auto k) {
      constexpr int kk = decltype(k)::value;
      auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, block, 0, stream, rows, src_pos + t0 * K,
                           w ? w + t0 * K : nullptr, at(base, t0 * d * es), n, shape,
                           at(y, t0 * d * es), reinterpret_cast<u32x2_t*>(codes), scales);
      };
      if (codes) go(unpermute_kernel<false, true, true, kk>);
      else if (f32 && vec) go(unpermute_kernel<true, true, false, kk>);
      else if (f32) go(unpermute_kernel<true, false, false, kk>);
      else if (vec) go(unpermute_kernel<false, true, false, kk>);
      else go(unpermute_kernel<false, false, false, kk>);
    });
  });
}

hipError_t launch_unpermute_grad(const void* dy, const void* rows, const float* row_scales,
                                 const int32_t* src_pos, const float* w, int64_t N, int d, int K,
                                 bool f32, void* drows, float* dw, hipStream_t stream) {
  const bool kept = row_scales != nullptr;
  bool vec;
  const Shape shape = shape_of(N, d, K, f32, vec);
  const int es = f32 ? 4 : 2;
  const int lanes = shape.ppr > 128 ? 256 : shape.ppr > 32 ? 64 : shape.ppr > 16 ? 32 : 16;
  return token_runs(N, lanes, [&](int64_t t0, int64_t n) {
    const dim3 grid(blocks_of(n * lanes)), block(256);
    return with_k(K, [&](auto k) {
      constexpr int kk = decltype(k)::value;
      auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, block, 0, stream, at(dy, t0 * d * es), rows, row_scales,
                           src_pos + t0 * K, w ? w + t0 * K : nullptr, n, shape,
                           drows, dw ? dw + t0 * K : nullptr);
      };
      auto pick = [&](auto l) {
        constexpr int W = decltype(l)::value;
        if (kept) go(unpermute_grad_kernel<false, true, true, kk, W>);
        else if (f32 && vec) go(unpermute_grad_kernel<true, true, false, kk, W>);
        else if (f32) go(unpermute_grad_kernel<true, false, false, kk, W>);
        else if (vec) go(unpermute_grad_kernel<false, true, false, kk, W>);
        else go(unpermute_grad_kernel<false, false, false, kk, W>);
      };
      if (lanes == 256) pick(std::integral_constant<int, 256>{});
      else if (lanes == 64) pick(std::integral_constant<int, 64>{});
      else if (lanes == 32) pick(std::integral_constant<int, 32>{});
      else pick(std::integral_constant<int, 16>{});
    });
  });
}

}  // namespace moe
