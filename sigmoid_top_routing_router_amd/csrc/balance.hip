// Balance loss of the router over the segments of a batch, the loads it is
// formed from, and its gradient with respect to the logits.
//
// "Kolibri Pre-Training from Scratch" §7 and §8 name auxiliary balance losses
// as the alternative to the quantile bias and the load-error injection.  With
// the loads c_ge of segment g, f_ge = E c_ge / sum_e c_ge and the mean score
// P_ge = mean_{t in g} p_te:
//   L = coef / G sum_g sum_e f_ge P_ge,
// p = sigma(z), sigma(z) / sum_e sigma(z) or softmax(z).  f is a constant for
// the gradient; with w = coef dL / (G T_g) and D = sum_e sigma(z):
//   sigma:       dz = w f s (1 - s)
//   normalised:  dz = w (s (1 - s) / D) (f - sum_e f p)
//   softmax:     dz = w p (f - sum_e f p)
//
// Rows are read 16 lanes each, four to a wave: a lane holds four columns out
// of every 64, so a row's reductions stay inside a DPP row and a wave reads
// four contiguous rows.  Both passes are bound by memory: 65536 x
// 384 logits in 16 segments, 100 MB read in 25 us (4.0 TB/s, what a plain
// reduction reaches); the gradient added to one that is there, 302 MB in 67 us
// (4.5 TB/s, a copy's rate).
//
// Forward: block b owns the rows [b R, (b + 1) R), walks the segments that
// meet them and leaves one partial row of score sums and loads for each, in
// slot b + g.  Along the batch (b, g) only ever grows, so slots are distinct
// and there are fewer than blocks + G of them; no atomics on floating point,
// no clearing.  The combine launch sums every segment's slots in block order
// (one block per segment and 64 experts), and its last block adds the
// segments' terms, in order, in fp64.
#include "common.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kMaxE = 384;
constexpr int kNC = kMaxE / 64;  // most 4-column pieces of a lane

enum Score { kSigmoid = 0, kSigmoidNorm = 1, kSoftmax = 2 };

__device__ __forceinline__ float row16_sum_f32(float v) {
  v += __uint_as_float(dpp_u32<kDppQuadSwap1>(__float_as_uint(v)));
  v += __uint_as_float(dpp_u32<kDppQuadSwap2>(__float_as_uint(v)));
  v += __uint_as_float(dpp_u32<kDppRowHalfMirror>(__float_as_uint(v)));
  return v + __uint_as_float(dpp_u32<kDppRowMirror>(__float_as_uint(v)));
}

// Segment bounds as given, kept inside the batch: whatever the arrays hold,
// no row outside [0, N) is touched.
struct Segs {
  const int32_t* begin;
  const int32_t* end;
  int32_t N;
  int G;
  __device__ __forceinline__ int32_t lo(int g) const {
    return begin ? min(max(begin[g], 0), N) : 0;
  }
  __device__ __forceinline__ int32_t hi(int g) const {
    return begin ? min(max(end[g], 0), N) : N;
  }
};

// The column of a lane's value (j, i).  QUADS: E is a multiple of 4; a lane has
// four consecutive columns, and its loads are 16 bytes wide where the array is
// aligned (vec).  Else neighbouring lanes have neighbouring columns (65536 x
// 383, gradient: 87 us in quads).
template <bool QUADS>
__device__ __forceinline__ int column(int j, int i, int l16) {
  return 64 * j + (QUADS ? 4 * l16 + i : 16 * i + l16);
}

// The NC x 4 columns of row t that this lane holds; columns past E give fill.
template <int NC, bool QUADS>
__device__ __forceinline__ void load_row(const float* __restrict__ Z, int64_t t, int E, int l16,
                                         bool vec, float fill, float (&v)[NC][4]) {
  const float* p = Z + t * E;
  if constexpr (QUADS) {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = column<QUADS>(j, 0, l16);
      if (vec) {
        const float4 q = c < E ? *reinterpret_cast<const float4*>(p + c)
                               : make_float4(fill, fill, fill, fill);
        v[j][0] = q.x; v[j][1] = q.y; v[j][2] = q.z; v[j][3] = q.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = c < E ? p[c + i] : fill;
      }
    }
  } else {
    // columns past E load column 0: a load under a branch of its own would be
    // waited for inside it
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = column<QUADS>(j, i, l16);
        v[j][i] = p[c < E ? c : 0];
      }
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = column<QUADS>(j, i, l16) < E ? v[j][i] : fill;
  }
}

// The scores p of row t; a column past E gets 0.
// slope: dp/dz without the sum over the row (see the formulas above).
template <int SCORE, int NC, bool QUADS>
__device__ __forceinline__ void scores(const float* __restrict__ Z, int64_t t, int E, int l16,
                                       bool vec, float (&v)[NC][4], float (&slope)[NC][4]) {
  load_row<NC, QUADS>(Z, t, E, l16, vec, -INFINITY, v);
  if constexpr (SCORE == kSoftmax) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) m = fmaxf(m, v[j][i]);
    m = row16_max_f32(m);
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[j][i] = __expf(v[j][i] - m);
        s += v[j][i];
      }
    const float inv = 1.0f / row16_sum_f32(s);
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) slope[j][i] = v[j][i] = v[j][i] * inv;
  } else {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // e = exp(-|z|) keeps sigma and sigma (1 - sigma) = e / (1 + e)^2
        // exact to a few ulp for either sign
        const float z = v[j][i];
        const float e = __expf(-fabsf(z));
        const float q = __builtin_amdgcn_rcpf(1.0f + e);
        v[j][i] = z >= 0.0f ? q : e * q;
        slope[j][i] = e * q * q;
        s += v[j][i];
      }
    if constexpr (SCORE == kSigmoidNorm) {
      s = row16_sum_f32(s);
      // A sum below 1/2: every logit is below zero (far below, every sigma would
      // be 0).  The row is read again and its scores are taken exp(-m) times as
      // large, m being its largest logit: sigma exp(-m) = exp(z - m) / (1 + e).
      if (s < 0.5f) {
        load_row<NC, QUADS>(Z, t, E, l16, vec, -INFINITY, v);
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) m = fmaxf(m, v[j][i]);
        m = row16_max_f32(m);
        s = 0.0f;
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float q = __builtin_amdgcn_rcpf(1.0f + __expf(v[j][i]));
            v[j][i] = __expf(v[j][i] - m) * q;
            slope[j][i] = v[j][i] * q;
            s += v[j][i];
          }
        s = row16_sum_f32(s);
      }
      const float inv = 1.0f / s;
#pragma unroll
      for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[j][i] *= inv;
          slope[j][i] *= inv;
        }
    }
  }
}

constexpr int kFwdWaves = 4;

template <int SCORE, int NC, bool QUADS>
__global__ __launch_bounds__(64 * kFwdWaves) void balance_partial_kernel(
    const float* __restrict__ Z, const int32_t* __restrict__ ids, Segs sg, int E, int K, int R,
    bool vec, float* __restrict__ sums, uint32_t* __restrict__ loads, uint32_t* ticket) {
  __shared__ uint32_t cnt[kMaxE];
  __shared__ float red[kFwdWaves][kMaxE];
  if (blockIdx.x == 0 && threadIdx.x == 0) *ticket = 0u;
  const int lane = lane_id(), w = threadIdx.x >> 6, l16 = lane & 15, sub = lane >> 4;
  const int32_t b0 = (int32_t)blockIdx.x * R;
  const int32_t b1 = min(sg.N, b0 + R);
  // the first segment that ends behind the block's first row
  int g = 0;
  {
    int a = 0, z = sg.G;
    while (a < z) {
      const int m = (a + z) >> 1;
      if (sg.hi(m) > b0) z = m; else a = m + 1;
    }
    g = a;
  }
  for (; g < sg.G; ++g) {
    const int32_t lo = max(sg.lo(g), b0), hi = min(sg.hi(g), b1);
    if (sg.lo(g) >= b1) break;
    if (lo >= hi) continue;
    for (int e = threadIdx.x; e < E; e += 64 * kFwdWaves) cnt[e] = 0u;
    __syncthreads();
    if (ids) {
      const int64_t p1 = (int64_t)hi * K;
      for (int64_t i = (int64_t)lo * K + threadIdx.x; i < p1; i += 64 * kFwdWaves) {
        const uint32_t e = (uint32_t)ids[i];
        if (e < (uint32_t)E) atomicAdd(&cnt[e], 1u);  // ids outside [0,E) are not counted
      }
    }
    float acc[NC][4];
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
    for (int32_t t0 = lo; t0 < hi; t0 += 4 * kFwdWaves) {
      const int32_t t = t0 + 4 * w + sub;
      if (t < hi) {  // whole DPP rows
        float v[NC][4], slope[NC][4];
        scores<SCORE, NC, QUADS>(Z, t, E, l16, vec, v, slope);
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[j][i] += v[j][i];
      }
    }
    // the four rows of the wave, then the waves in order
#pragma unroll
    for (int j = 0; j < NC; ++j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[j][i] += __shfl_xor(acc[j][i], 16);
        acc[j][i] += __shfl_xor(acc[j][i], 32);
        const int c = column<QUADS>(j, i, l16);
        if (sub == 0 && c < E) red[w][c] = acc[j][i];
      }
    }
    __syncthreads();
    const int64_t slot = ((int64_t)blockIdx.x + g) * E;
    for (int e = threadIdx.x; e < E; e += 64 * kFwdWaves) {
      float s = red[0][e];
#pragma unroll
      for (int q = 1; q < kFwdWaves; ++q) s += red[q][e];
      sums[slot + e] = s;
      loads[slot + e] = cnt[e];
    }
    __syncthreads();
  }
}

constexpr int kCombWaves = 8;

// Block (x: 64 experts, y: segment).  terms[g][x] = {sum_e c P, sum_e c}.
__global__ __launch_bounds__(64 * kCombWaves) void balance_combine_kernel(
    const float* __restrict__ sums, const uint32_t* __restrict__ loads, Segs sg, int E, int R,
    const int32_t* __restrict__ counts_in, bool have_ids, double coef, double* terms,
    uint32_t* ticket, int32_t* __restrict__ counts_out, float* __restrict__ mean_out,
    float* __restrict__ loss) {
  __shared__ double s_sum[kCombWaves][64];
  __shared__ uint32_t s_cnt[kCombWaves][64];
  __shared__ uint32_t s_last;
  const int lane = lane_id(), w = threadIdx.x >> 6;
  const int e = blockIdx.x * 64 + lane;
  const int tiles = (int)gridDim.x;
  for (int g = blockIdx.y; g < sg.G; g += gridDim.y) {
    const int32_t lo = sg.lo(g), hi = sg.hi(g);
    double s = 0.0;
    uint32_t c = 0u;
    if (lo < hi && e < E) {
      const int b0 = lo / R, b1 = (hi - 1) / R;
#pragma unroll 8
      for (int b = b0 + w; b <= b1; b += kCombWaves) {
        const int64_t at = ((int64_t)b + g) * E + e;
        s += (double)sums[at];
        c += loads[at];
      }
    }
    s_sum[w][lane] = s;
    s_cnt[w][lane] = c;
    __syncthreads();
    if (w == 0) {
      s = 0.0;
      c = 0u;
#pragma unroll
      for (int q = 0; q < kCombWaves; ++q) {
        s += s_sum[q][lane];
        c += s_cnt[q][lane];
      }
      const double mean = lo < hi ? s / (double)(hi - lo) : 0.0;
      double used = 0.0;
      if (e < E) {
        if (mean_out) mean_out[(int64_t)g * E + e] = (float)mean;
        if (counts_out && have_ids) counts_out[(int64_t)g * E + e] = (int32_t)c;
        used = counts_in ? (double)counts_in[(int64_t)g * E + e] : (double)c;
      }
      double dot = used * mean;
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) {
        dot += __shfl_xor(dot, o);
        used += __shfl_xor(used, o);
      }
      if (lane == 0) {
        terms[((int64_t)g * tiles + blockIdx.x) * 2] = dot;
        terms[((int64_t)g * tiles + blockIdx.x) * 2 + 1] = used;
      }
    }
    __syncthreads();
  }
  // the last block to arrive adds the segments; which one it is changes
  // nothing in the sum's order
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(ticket, 1u) == gridDim.x * gridDim.y - 1u ? 1u : 0u;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  double sum = 0.0;
  for (int g = threadIdx.x; g < sg.G; g += 64 * kCombWaves) {
    double dot = 0.0, tot = 0.0;
    for (int x = 0; x < tiles; ++x) {
      dot += terms[((int64_t)g * tiles + x) * 2];
      tot += terms[((int64_t)g * tiles + x) * 2 + 1];
    }
    if (tot > 0.0) sum += dot / tot;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
  if (lane == 0) s_sum[0][w] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double v = 0.0;
    for (int q = 0; q < kCombWaves; ++q) v += s_sum[0][q];
    loss[0] = (float)(v * coef * (double)E / (double)sg.G);
  }
}

// Each wave takes four consecutive rows at a time, 16 lanes a row; f of the
// row's segment stays in registers until a row of another segment comes.
template <int SCORE, int NC, bool QUADS>
__global__ __launch_bounds__(256) void balance_grad_kernel(
    const float* __restrict__ Z, const int32_t* __restrict__ counts, Segs sg, int E, int RW,
    bool vec, float coef, const float* __restrict__ grad_loss, const float* G, float* out) {
  const int lane = lane_id(), l16 = lane & 15, sub = lane >> 4;
  const int32_t wave = (int32_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t r0 = (int64_t)wave * RW;
  if (r0 >= sg.N) return;
  const int32_t r1 = (int32_t)min((int64_t)sg.N, r0 + RW);
  const float scale = coef * (grad_loss ? grad_loss[0] : 1.0f) / (float)sg.G;
  int gcur = -1;
  float f[NC][4];
  float wrow = 0.0f;
  int32_t seg_lo = 0, seg_hi = 0;  // rows of segment gcur, or the gap around the row
  for (int32_t t = (int32_t)r0 + sub; t < r1; t += 4) {
    if (!(t >= seg_lo && t < seg_hi)) {
      // the last segment that begins at or before t holds t, or none does
      int a = 0, z = sg.G;
      while (a < z) {
        const int m = (a + z) >> 1;
        if (sg.lo(m) <= t) a = m + 1; else z = m;
      }
      const int g = a - 1;
      seg_lo = g >= 0 ? sg.lo(g) : 0;
      seg_hi = g >= 0 ? sg.hi(g) : 0;
      gcur = g >= 0 && t >= seg_lo && t < seg_hi ? g : -1;
      if (gcur >= 0) {
        float tot = 0.0f;
        double total = 0.0;
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = column<QUADS>(j, i, l16);
            const int32_t n = c < E ? counts[(int64_t)gcur * E + c] : 0;
            f[j][i] = (float)n;
            total += (double)n;
          }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) total += __shfl_xor(total, o);
        tot = total > 0.0 ? (float)((double)E / total) : 0.0f;
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) f[j][i] *= tot;
        wrow = scale / (float)(seg_hi - seg_lo);
      }
    }
    float o[NC][4];
    const bool inside = gcur >= 0;
    if (inside) {
      float v[NC][4], slope[NC][4];
      scores<SCORE, NC, QUADS>(Z, t, E, l16, vec, v, slope);
      float dot = 0.0f;
      if constexpr (SCORE != kSigmoid) {
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) dot += f[j][i] * v[j][i];
        dot = row16_sum_f32(dot);
      }
#pragma unroll
      for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][i] = wrow * (slope[j][i] * (f[j][i] - dot));
    } else {
      if (G == out) continue;  // added in place: nothing to add
#pragma unroll
      for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][i] = 0.0f;
    }
    if (G) {
      float q[NC][4];
      load_row<NC, QUADS>(G, t, E, l16, vec, 0.0f, q);
#pragma unroll
      for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][i] += q[j][i];
    }
    float* p = out + (int64_t)t * E;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      if (QUADS && vec) {
        const int c = column<QUADS>(j, 0, l16);
        if (c < E)
          *reinterpret_cast<float4*>(p + c) = make_float4(o[j][0], o[j][1], o[j][2], o[j][3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = column<QUADS>(j, i, l16);
          if (c < E) p[c] = o[j][i];
        }
      }
    }
  }
}

bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace

// Rows of one block of the partial pass: 16 at a time (four waves of four),
// at most 1024 blocks, so that the partial rows stay small beside the logits
// (65536 x 384: 3.1 MB, 9 us in the combine launch, beside 100 MB).
int balance_block_rows(int64_t N) {
  const int64_t per = (N + 1023) / 1024;
  return (int)((per + 15) / 16 * 16);
}
int64_t balance_slots(int64_t N, int G) {
  const int R = balance_block_rows(N);
  return (N + R - 1) / R + G;
}

template <int SCORE>
static void start_partial(int nc, dim3 grid, hipStream_t stream, const float* Z,
                          const int32_t* ids, const Segs& sg, int E, int K, int R, bool vec,
                          const BalanceWork& w) {
#define MOE_NC(n)                                                                              \
  case n:                                                                                      \
    if (E % 4 == 0)                                                                            \
      hipLaunchKernelGGL((balance_partial_kernel<SCORE, n, true>), grid, dim3(64 * kFwdWaves), \
                         0, stream, Z, ids, sg, E, K, R, vec, w.sums, w.loads, w.ticket);      \
    else                                                                                       \
      hipLaunchKernelGGL((balance_partial_kernel<SCORE, n, false>), grid,                      \
                         dim3(64 * kFwdWaves), 0, stream, Z, ids, sg, E, K, R, vec, w.sums,    \
                         w.loads, w.ticket);                                                   \
    break;
  switch (nc) { MOE_NC(1) MOE_NC(2) MOE_NC(3) MOE_NC(4) MOE_NC(5) MOE_NC(6) }
#undef MOE_NC
}

hipError_t launch_balance_loss(const float* Z, const int32_t* ids, const int32_t* counts_in,
                               const int32_t* begin, const int32_t* end, int64_t N, int E, int K,
                               int G, int score, float coef, const BalanceWork& w, float* loss,
                               int32_t* counts_out, float* mean_out, hipStream_t stream) {
  const int R = balance_block_rows(N);
  const Segs sg{begin, end, (int32_t)N, G};
  const bool vec = E % 4 == 0 && al16(Z);
  const dim3 grid((unsigned)((N + R - 1) / R));
  const int nc = (E + 63) / 64;
  if (score == kSigmoid) start_partial<kSigmoid>(nc, grid, stream, Z, ids, sg, E, K, R, vec, w);
  else if (score == kSigmoidNorm)
    start_partial<kSigmoidNorm>(nc, grid, stream, Z, ids, sg, E, K, R, vec, w);
  else start_partial<kSoftmax>(nc, grid, stream, Z, ids, sg, E, K, R, vec, w);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const dim3 cgrid((unsigned)nc, (unsigned)(G < 1024 ? G : 1024));
  hipLaunchKernelGGL(balance_combine_kernel, cgrid, dim3(64 * kCombWaves), 0, stream, w.sums,
                     w.loads, sg, E, R, counts_in, ids != nullptr, (double)coef, w.terms, w.ticket,
                     counts_out, mean_out, loss);
  return hipGetLastError();
}

template <int SCORE>
static void start_grad(int nc, dim3 grid, hipStream_t stream, const float* Z,
                       const int32_t* counts, const Segs& sg, int E, int RW, bool vec, float coef,
                       const float* gl, const float* G, float* out) {
#define MOE_NC(n)                                                                              \
  case n:                                                                                      \
    if (E % 4 == 0)                                                                            \
      hipLaunchKernelGGL((balance_grad_kernel<SCORE, n, true>), grid, dim3(256), 0, stream, Z, \
                         counts, sg, E, RW, vec, coef, gl, G, out);                            \
    else                                                                                       \
      hipLaunchKernelGGL((balance_grad_kernel<SCORE, n, false>), grid, dim3(256), 0, stream,   \
                         Z, counts, sg, E, RW, vec, coef, gl, G, out);                         \
    break;
  switch (nc) { MOE_NC(1) MOE_NC(2) MOE_NC(3) MOE_NC(4) MOE_NC(5) MOE_NC(6) }
#undef MOE_NC
}

hipError_t launch_balance_grad(const float* Z, const int32_t* counts, const int32_t* begin,
                               const int32_t* end, int64_t N, int E, int G, int score, float coef,
                               const float* grad_loss, const float* grad_in, float* grad_out,
                               hipStream_t stream) {
  const Segs sg{begin, end, (int32_t)N, G};
  const bool vec = E % 4 == 0 && al16(Z) && al16(grad_in) && al16(grad_out);
  // at most 8192 waves, four rows at a time each
  const int64_t per = (N + 8191) / 8192;
  const int RW = (int)((per + 3) / 4 * 4);
  const int64_t waves = (N + RW - 1) / RW;
  const dim3 grid((unsigned)((waves + 3) / 4));
  const int nc = (E + 63) / 64;
  if (score == kSigmoid)
    start_grad<kSigmoid>(nc, grid, stream, Z, counts, sg, E, RW, vec, coef, grad_loss, grad_in, grad_out);
  else if (score == kSigmoidNorm)
    start_grad<kSigmoidNorm>(nc, grid, stream, Z, counts, sg, E, RW, vec, coef, grad_loss, grad_in, grad_out);
  else
    start_grad<kSoftmax>(nc, grid, stream, Z, counts, sg, E, RW, vec, coef, grad_loss, grad_in, grad_out);
  return hipGetLastError();
}

}  // namespace moe
