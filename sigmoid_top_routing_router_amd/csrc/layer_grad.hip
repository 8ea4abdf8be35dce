// Backward pass of the MoE layer: the matrix products whose operands are not
// both k-contiguous, and the small kernels around them.
//
// "Kolibri 1 im Detail" (routing section, SwiGLU paragraph) and "Kolibri
// Pre-Training from Scratch" §6.1, differentiated: for a pair p = (t, e) with
// s = sigma(z_te), G = x W_g^T, U = x W_u^T, H = silu(G) U (formed again) and
// Q = dy W_d,
//   dS = Q . H,  dU = s Q silu(G),  dG = s Q U sigma(G)(1 + G(1 - sigma(G))),
//   dx_t = sum_k (dG W_g + dU W_u) + [shared expert, s = 1] + dZ W_r,
//   dW_g = dG^T x,  dW_u = dU^T x,  dW_d = dy^T (s H),  dW_r = dZ^T x,
//   dZ = grad_logits + [e chosen for t] dS s (1 - s).
// G and U come from the forward pass's tile engine, whose epilogue forms dG,
// dU, s H and Q . H (grouped_gemm.hip).  Here:
//  * rows_kernel: Q (fp32) and dx, C[row, n] = sum_k A[row, k] B[k, n]: the
//    rows are k-contiguous, the weights are read as they are stored, n
//    contiguous;
//  * weights_kernel: every weight gradient, C[m, n] = sum_row A[row, m]
//    B[row, n] over the rows of an expert's segment: both operands n
//    contiguous.
// Both multiply 256 x 256 tiles in stages of 64 k with
// v_mfma_f32_32x32x16_bf16, eight waves of 128 x 64, two waves to a SIMD.
// A stage (32 KB of each operand) is in LDS twice; the next one's LDS-DMA
// loads are issued as soon as every wave has left the stage before, so they
// have a whole stage of MFMAs to land.  The loads are written in assembly
// (they have no register result): as builtins, the compiler waits for all of
// them in front of the first transposing LDS read, which it takes for a
// possible reader of what they write, and a stage then never overlaps the
// next one's loads.  An operand whose k runs across rows
// is kept as [k][256] in LDS and read with the transposing LDS read
// (ds_read_b64_tr_b16: 16 lanes fetch 4 k x 16 columns and each gets one
// column's four k), so no transposed copy of a weight or an activation is
// ever made.  Its 16-byte chunk c of row k sits at c ^ 4 (k & 3): the four k
// of one read are then on four different groups of banks.
#include "common.h"
#include "gemm_args.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int TM = 256, TN = 256, TK = 64;
constexpr int kOpBytes = 32 * 1024;            // one operand of one stage
constexpr int kSlotBytes = 2 * kOpBytes;
constexpr int kIdsOff = 2 * kSlotBytes;        // gathered row offsets (weights_kernel)
constexpr int kIdsMax = 8192;
constexpr int kLdsBytes = 160 * 1024;
static_assert(kIdsOff + kIdsMax * 4 <= kLdsBytes, "LDS layout");
constexpr int kXcds = 8;
// An offset past the end of any operand: the load returns zeros.  Operands
// are smaller than this (checked by the entry point).
constexpr uint32_t kNoAddr = kGradMaxOperandBytes;

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ void stage_barrier() {
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2_t v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

typedef int i32x4_t __attribute__((ext_vector_type(4)));
// Raw buffer descriptor in scalar registers (stride 0; reads past `bytes`
// return zeros).
__device__ __forceinline__ i32x4_t buffer_at(const void* base, uint32_t bytes) {
  const uint64_t a = (uint64_t)base;
  return i32x4_t{__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
                 __builtin_amdgcn_readfirstlane((int)((uint32_t)(a >> 32) & 0xFFFFu)),
                 __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}
// LDS-DMA: 16 bytes per lane from buffer + off to LDS at l + 16 * lane.
// Counted on vmcnt; the waits are this file's own (wait_vmcnt).  m0 (the LDS
// address) is set and used inside; nothing else in these kernels uses it.
__device__ __forceinline__ void dma(i32x4_t r, uint32_t off, const char* l) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass does not know these operands
  const int at = __builtin_amdgcn_readfirstlane((int)(uint32_t)(lds_void_t*)l);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(at), "v"(off), "s"(r) : "memory");
#endif
}

// Work item of a block: blocks are dealt to the XCDs in turn, each XCD takes
// a contiguous run of items.
__device__ __forceinline__ int64_t xcd_item(int64_t block, int64_t share) {
  return (block % kXcds) * share + block / kXcds;
}

// Eight k of one column from a [k][256] stage: two transposing reads.
__device__ __forceinline__ bf16x8_t read_tr(const char* p) {
  const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)p);
  const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p + 4 * 512));
  typedef short s16x8_t __attribute__((ext_vector_type(8)));
  const s16x8_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  return __builtin_bit_cast(bf16x8_t, v);
}

// What a wave reads of a stage.  A operand: [256 rows][64 k], chunk c of row r
// at c ^ ((r >> 1) & 7) (ATR false), or [64 k][256] (ATR true); B: [64 k][256].
template <bool ATR>
struct Frags {
  int a_base, a_x[4], b_x[2];
  __device__ __forceinline__ Frags(int lane, int wg, int wp) {
    const int i = lane & 15, kq = i >> 2, half = (lane >> 4) & 1;
    const int krow = (8 * (lane >> 5) + kq) * 512;
    const int sub = (2 * half + ((i & 3) >> 1)) * 16 + (i & 1) * 8;
    if (ATR) {
      a_base = krow;
#pragma unroll
      for (int m = 0; m < 4; ++m) a_x[m] = (16 * wg + 4 * (m ^ kq)) * 16 + sub;
    } else {
      a_base = (wg * 128 + (lane & 31)) * 128;
#pragma unroll
      for (int m = 0; m < 4; ++m)  // by k-step: chunk 2 ks + (lane >> 5)
        a_x[m] = ((2 * m + (lane >> 5)) ^ ((lane >> 1) & 7)) * 16;
    }
#pragma unroll
    for (int f = 0; f < 2; ++f) b_x[f] = krow + ((8 * wp + 4 * f) ^ (4 * kq)) * 16 + sub;
  }
  __device__ __forceinline__ bf16x8_t a(const char* s, int ks, int m) const {
    if (ATR) return read_tr(s + a_base + a_x[m] + ks * (16 * 512));
    return *reinterpret_cast<const bf16x8_t*>(s + a_base + m * (32 * 128) + a_x[ks]);
  }
  __device__ __forceinline__ bf16x8_t b(const char* s, int ks, int f) const {
    return read_tr(s + b_x[f] + ks * (16 * 512));
  }
};

template <bool ATR, int LIVE>
__device__ __forceinline__ void multiply_stage(const char* slot, const Frags<ATR>& fr,
                                               floatx16_t (&acc)[4][2]) {
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    bf16x8_t A[4], B[2];
#pragma unroll
    for (int f = 0; f < 2; ++f) B[f] = fr.b(slot + kOpBytes, ks, f);
#pragma unroll
    for (int m = 0; m < LIVE; ++m) A[m] = fr.a(slot, ks, m);
#pragma unroll
    for (int m = 0; m < LIVE; ++m)
#pragma unroll
      for (int f = 0; f < 2; ++f)
        acc[m][f] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(B[f], A[m], acc[m][f], 0, 0, 0);
  }
}

// The accumulators hold the tile transposed (the B fragment is the first
// operand): lane l has tile row (l & 31) of a block and columns 8 (r / 4) +
// 4 (l / 32) + r % 4.  bf16 results pass through the idle LDS and leave as
// 16-byte pieces of whole rows; row_ptr(r) is the output of tile row r, or
// null.
constexpr int kOutStride = TN * 2 + 8;
static_assert(TM * kOutStride <= kLdsBytes, "staged tile");
template <class RowPtr>
__device__ __forceinline__ void store_bf16_tile(floatx16_t (&acc)[4][2], int lane, int wg, int wp,
                                                int tid, char* lds, int cols, RowPtr row_ptr) {
  __syncthreads();
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    char* row = lds + (wg * 128 + m * 32 + (lane & 31)) * kOutStride + (wp * 64 + 4 * (lane >> 5)) * 2;
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<uint2*>(row + (32 * f + 8 * q) * 2) =
            make_uint2(pack_bf16(acc[m][f][4 * q], acc[m][f][4 * q + 1]),
                       pack_bf16(acc[m][f][4 * q + 2], acc[m][f][4 * q + 3]));
  }
  __syncthreads();
  const int ch = tid & 31;
  if (ch * 8 >= cols) return;
  for (int r = tid >> 5; r < TM; r += 16) {
    uint16_t* p = row_ptr(r);
    if (!p) break;  // rows run out in order
    const char* src = lds + r * kOutStride + ch * 16;
    const uint2 lo = *reinterpret_cast<const uint2*>(src);
    const uint2 hi = *reinterpret_cast<const uint2*>(src + 8);
    *reinterpret_cast<uint4*>(p + ch * 8) = make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
}

__device__ __forceinline__ void clear_acc(floatx16_t (&acc)[4][2]) {
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[m][f][r] = 0.0f;
}

// ---------------------------------------------------------------- rows
// PAIR: rows of the tile table, else tokens.  F32: the fp32 result (Q), whose
// pairs gather their rows of A; else bf16 (parts of dx).
template <bool PAIR, bool F32>
__device__ __forceinline__ void rows_tile(const RowsProblem& p, int64_t item, char* lds) {
  constexpr bool GATHER = PAIR && F32;
  const int64_t mt = item / p.n_tiles_n;
  const int nt = (int)(item % p.n_tiles_n);
  int expert = 0, rows;
  int64_t row0;
  if constexpr (PAIR) {
    const int4 ent = reinterpret_cast<const int4*>(p.tiles)[mt];
    expert = ent.x;
    row0 = ent.y;
    rows = ent.z;
  } else {
    row0 = mt * TM;
    rows = (int)min((int64_t)TM, p.rows_dense - row0);
  }
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wg = wave >> 2, wp = wave & 3;
  const int n0 = nt * TN;

  // LDS-DMA: load i of a wave covers A rows 8 (8 i + wave) .. + 7 (lane ->
  // row + (l >> 3), slot l & 7) and B k-rows 2 (8 i + wave) .. + 1 (lane ->
  // row + (l >> 5), slot l & 31).
  const int a_chunk = (lane & 7) ^ ((4 * wave + (lane >> 4)) & 7);
  const int b_k = 2 * wave + (lane >> 5);
  const int b_chunk = (lane & 31) ^ (4 * (b_k & 3));
  const bool b_col = n0 + 8 * b_chunk < p.ncols;
  uint32_t a_row[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * (8 * i + wave) + (lane >> 3);
    a_row[i] = r >= rows ? 0xFFFFFFFFu
               : GATHER ? (uint32_t)p.gather[row0 + r] / (uint32_t)p.gather_div : (uint32_t)r;
  }
  floatx16_t acc[4][2];
  clear_acc(acc);
  const Frags<false> fr(lane, wg, wp);
  int live_m = (rows - wg * 128 + 31) / 32;
  live_m = __builtin_amdgcn_readfirstlane(live_m < 0 ? 0 : live_m > 4 ? 4 : live_m);
  const bool live = __builtin_amdgcn_readfirstlane(live_m > 0 && n0 + wp * 64 < p.ncols);

  int parity = 0;  // LDS slot of the next stage; runs on over the segments
  for (int sgi = 0; sgi < p.n_seg; ++sgi) {
    const RowsSegment& sg = p.seg[sgi];
    // a gathered A spans the whole buffer, a direct one this tile's rows
    const i32x4_t ra = buffer_at(GATHER ? sg.A : sg.A + row0 * sg.lda,
                                 (uint32_t)((GATHER ? p.a_rows : rows) * sg.lda * 2));
    const i32x4_t rb = buffer_at(sg.B + (int64_t)expert * sg.b_expert_stride,
                                 (uint32_t)sg.kdim * (uint32_t)p.ncols * 2u);
    const int nk = (sg.kdim + TK - 1) / TK;
    uint32_t a_off[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      a_off[i] = a_row[i] != 0xFFFFFFFFu
                     ? a_row[i] * (uint32_t)(sg.lda * 2) + (uint32_t)a_chunk * 16u : kNoAddr;
    const uint32_t b_base = (uint32_t)(n0 + 8 * b_chunk) * 2u;
    const uint32_t b_pitch = (uint32_t)p.ncols * 2u;
    auto issue = [&](int ks, int slot) {
      char* s = lds + slot * kSlotBytes;
      const int k0 = ks * TK;
      const bool ka = k0 + 8 * a_chunk < sg.kdim;  // kdim % 8 == 0: whole chunks
#pragma unroll
      for (int i = 0; i < 4; ++i)
        dma(ra, ka ? a_off[i] + (uint32_t)k0 * 2u : kNoAddr, s + (8 * i + wave) * 1024);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = k0 + 16 * i + b_k;
        dma(rb, b_col && k < sg.kdim ? b_base + (uint32_t)k * b_pitch : kNoAddr,
            s + kOpBytes + (8 * i + wave) * 1024);
      }
    };
    // the slot is free: the barrier that opened the stage before this one (the
    // last segment's last) is behind every wave's reads of it
    issue(0, parity);
    for (int ks = 0; ks < nk; ++ks) {
      wait_vmcnt<0>();
      stage_barrier();
      const int cur = parity;
      parity ^= 1;
      if (ks + 1 < nk) issue(ks + 1, parity);
      const char* slot = lds + cur * kSlotBytes;
      if (live) {
        if (live_m > 2) multiply_stage<false, 4>(slot, fr, acc);
        else multiply_stage<false, 2>(slot, fr, acc);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
  }

  if constexpr (F32) {
    float* out = reinterpret_cast<float*>(p.out);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int r = wg * 128 + m * 32 + (lane & 31);
      if (!live || r >= rows) continue;
      float* o = out + (row0 + r) * p.ldo + n0;
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = wp * 64 + 32 * f + 8 * q + 4 * (lane >> 5);
          if (n0 + c < p.ncols)
            *reinterpret_cast<float4*>(o + c) =
                make_float4(acc[m][f][4 * q], acc[m][f][4 * q + 1], acc[m][f][4 * q + 2],
                            acc[m][f][4 * q + 3]);
        }
    }
    return;
  }
  uint16_t* out = reinterpret_cast<uint16_t*>(p.out) + row0 * p.ldo + n0;
  store_bf16_tile(acc, lane, wg, wp, tid, lds, p.ncols - n0,
                  [&](int r) { return r < rows ? out + r * p.ldo : nullptr; });
}

// The work item of block b of a problem's share of the grid.
template <bool PAIR, bool F32>
__device__ __forceinline__ void rows_block(const RowsProblem& p, int64_t b, char* lds) {
  const int64_t m_tiles = PAIR ? (int64_t)*p.n_tiles : (p.rows_dense + TM - 1) / TM;
  const int64_t work = m_tiles * p.n_tiles_n;
  const int64_t share = (work + kXcds - 1) / kXcds;
  if (b / kXcds >= share) return;
  const int64_t item = xcd_item(b, share);
  if (item < work) rows_tile<PAIR, F32>(p, item, lds);
}

// The tokens' blocks first (fewer items), then the pairs'.
template <bool F32>
__global__ __launch_bounds__(512, 2) void rows_kernel(RowsProblem token, RowsProblem pair,
                                                      int64_t token_blocks) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int64_t b = blockIdx.x;
  if (b < token_blocks) rows_block<false, F32>(token, b, lds);
  else rows_block<true, F32>(pair, b - token_blocks, lds);
}

// ---------------------------------------------------------------- weights
enum Gathered { kNeither, kA, kB };
template <Gathered GATHER>
__device__ __forceinline__ void weights_tile(const WeightsProblem& p, int expert, int tile,
                                             char* lds) {
  const int m0 = (tile / p.tiles_n) * TM;
  const int n0 = (tile % p.tiles_n) * TN;
  int64_t first, rows;
  if (p.offsets) {
    first = p.offsets[expert];
    rows = (int64_t)p.offsets[expert + 1] - first;
  } else {
    first = 0;
    rows = p.rows_dense;
  }
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wg = wave >> 2, wp = wave & 3;
  const int kr = 2 * wave + (lane >> 5);  // k-row of load i: 16 i + kr
  const int chunk = (lane & 31) ^ (4 * (kr & 3));
  const bool a_in = m0 + 8 * chunk < p.a_cols, b_in = n0 + 8 * chunk < p.b_cols;
  const uint32_t a_col = (uint32_t)(m0 + 8 * chunk) * 2u, b_col = (uint32_t)(n0 + 8 * chunk) * 2u;
  uint32_t* ids = reinterpret_cast<uint32_t*>(lds + kIdsOff);
  const uint32_t a_pitch = (uint32_t)p.lda * 2u, b_pitch = (uint32_t)p.ldb * 2u;
  const uint32_t g_pitch = GATHER == kA ? a_pitch : b_pitch;

  floatx16_t acc[4][2];
  clear_acc(acc);
  const Frags<true> fr(lane, wg, wp);
  const bool live =
      __builtin_amdgcn_readfirstlane(m0 + wg * 128 < p.a_cols && n0 + wp * 64 < p.b_cols);
  for (int64_t c0 = 0; c0 < rows; c0 += kIdsMax) {
    const int cr = (int)min((int64_t)kIdsMax, rows - c0);
    const int nk = (cr + TK - 1) / TK;
    if (c0 > 0) stage_barrier();  // the chunk before is read to its end
    if constexpr (GATHER != kNeither) {
      for (int r = tid; r < nk * TK; r += 512)
        ids[r] = r < cr ? (uint32_t)(p.src[first + c0 + r] / p.src_div) * g_pitch : kNoAddr;
      __syncthreads();
    }
    // direct operands: this chunk's rows; gathered ones: the whole buffer
    const int64_t base = first + c0;
    const i32x4_t ra = buffer_at(GATHER == kA ? p.A : p.A + base * p.lda,
                                 (uint32_t)((GATHER == kA ? p.src_rows : cr) * p.lda * 2));
    const i32x4_t rb = buffer_at(GATHER == kB ? p.B : p.B + base * p.ldb,
                                 (uint32_t)((GATHER == kB ? p.src_rows : cr) * p.ldb * 2));
    auto issue = [&](int ks, int slot) {
      char* s = lds + slot * kSlotBytes;
      uint32_t at[4];
      if constexpr (GATHER != kNeither) {
#pragma unroll
        for (int i = 0; i < 4; ++i) at[i] = ids[ks * TK + 16 * i + kr];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = ks * TK + 16 * i + kr;
        const bool in = r < cr;
        const uint32_t ga = GATHER == kA ? at[i] : (uint32_t)r * a_pitch;
        const uint32_t gb = GATHER == kB ? at[i] : (uint32_t)r * b_pitch;
        dma(ra, in && a_in ? ga + a_col : kNoAddr, s + (8 * i + wave) * 1024);
        dma(rb, in && b_in ? gb + b_col : kNoAddr, s + kOpBytes + (8 * i + wave) * 1024);
      }
    };
    issue(0, 0);
    for (int ks = 0; ks < nk; ++ks) {
      wait_vmcnt<0>();
      stage_barrier();
      if (ks + 1 < nk) issue(ks + 1, (ks + 1) & 1);
      if (live) multiply_stage<true, 4>(lds + (ks & 1) * kSlotBytes, fr, acc);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
  }
  const int64_t eo = (int64_t)expert * p.out_stride;
  store_bf16_tile(acc, lane, wg, wp, tid, lds, p.b_cols - n0, [&](int r) -> uint16_t* {
    const int m = m0 + r;
    if (m >= p.a_cols || (!p.out1 && m >= p.split)) return nullptr;
    return (m < p.split ? p.out0 + eo + (int64_t)m * p.b_cols
                        : p.out1 + eo + (int64_t)(m - p.split) * p.b_cols) + n0;
  });
}

// Items: the dense problems' tiles first (their sums run over all tokens),
// then per expert the tiles of its gate/up and of its down gradient, which
// share the expert's rows.
__global__ __launch_bounds__(512, 2) void weights_kernel(WeightsLaunch w) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  int64_t b = blockIdx.x;
  for (int i = 0; i < w.n_dense; ++i) {
    const int t = w.dense[i].tiles_m * w.dense[i].tiles_n;
    if (b < t) {
      weights_tile<kNeither>(w.dense[i], 0, (int)b, lds);
      return;
    }
    b -= t;
  }
  const int t0 = w.expert[0].tiles_m * w.expert[0].tiles_n;
  const int t1 = w.expert[1].tiles_m * w.expert[1].tiles_n;
  const int64_t work = (int64_t)w.E * (t0 + t1);
  const int64_t share = (work + kXcds - 1) / kXcds;
  if (b / kXcds >= share) return;
  const int64_t item = xcd_item(b, share);
  if (item >= work) return;
  const int e = (int)(item / (t0 + t1));
  const int r = (int)(item % (t0 + t1));
  if (r < t0) weights_tile<kB>(w.expert[0], e, r, lds);
  else weights_tile<kA>(w.expert[1], e, r - t0, lds);
}

// ---------------------------------------------------------------- small kernels
// One thread per pair: the id kept inside [0, E), and the pair's weight
// sigma(z), 0 for an id outside the range (such a pair has no gradient).
__global__ __launch_bounds__(256) void pairs_kernel(const int32_t* __restrict__ ids,
                                                    const float* __restrict__ Z, int64_t pairs,
                                                    int E, int K, int32_t* __restrict__ ids_out,
                                                    float* __restrict__ S) {
  const int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (p >= pairs) return;
  const uint32_t e = (uint32_t)ids[p];
  const bool in = e < (uint32_t)E;
  ids_out[p] = in ? (int32_t)e : 0;
  S[p] = in ? sigmoid_weight(Z[p / K * E + e]) : 0.0f;
}

// m-tiles of bm rows from the segment offsets: one block; thread e counts its
// expert's tiles, a scan places them.
__global__ __launch_bounds__(512) void row_tiles_kernel(const int32_t* __restrict__ offsets, int E,
                                                        int32_t* __restrict__ tiles,
                                                        int32_t* __restrict__ n_tiles) {
  __shared__ uint32_t wsum[8];
  const int e = threadIdx.x, w = e >> 6;
  const int32_t off = e < E ? offsets[e] : 0;
  const int32_t cnt = e < E ? offsets[e + 1] - off : 0;
  const uint32_t nt = (uint32_t)(cnt + TM - 1) / TM;
  const uint32_t inc = wave_inclusive_sum_u32(nt);
  if (lane_id() == 63) wsum[w] = inc;
  __syncthreads();
  uint32_t base = 0;
  for (int i = 0; i < w; ++i) base += wsum[i];
  uint32_t t = base + inc - nt;
  for (int32_t r = 0; r < cnt; r += TM)
    reinterpret_cast<int4*>(tiles)[t++] = make_int4(e, off + r, min(TM, cnt - r), r);
  if (e == 511) *n_tiles = (int32_t)(base + inc);
}

// A wave per token: dZ = grad_in + the chosen experts' dS s (1 - s), in fp32
// and, padded to ldb columns with zeros, in bf16 as an operand of the router
// products.  s (1 - s) = e / (1 + e)^2 with e = exp(-|z|).  The partial score
// gradients of a pair's column tiles are added in order; a token's pairs too.
__global__ __launch_bounds__(256) void logits_grad_kernel(
    const float* __restrict__ Z, const int32_t* __restrict__ ids_raw,
    const int32_t* __restrict__ src_pos, const float* __restrict__ dscore_part, int parts,
    int64_t N, int E, int K, const float* grad_in, float* grad_out, uint16_t* __restrict__ dzb,
    int ldb) {
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= N) return;
  const int lane = lane_id();
  // lane k < K: pair (t, k)
  int32_t id = -1;
  float dz = 0.0f;
  if (lane < K) {
    id = ids_raw[t * K + lane];
    if ((uint32_t)id < (uint32_t)E) {
      const float* dp = dscore_part + (int64_t)src_pos[t * K + lane] * parts;
      float ds = 0.0f;
      for (int i = 0; i < parts; ++i) ds += dp[i];
      const float e = expf(-fabsf(Z[t * E + id]));
      const float q = 1.0f + e;
      dz = ds * (e / (q * q));
    } else {
      id = -1;
    }
  }
  for (int c = lane; c < ldb; c += 64) {
    float v = 0.0f;
    if (c < E) {
      v = grad_in ? grad_in[t * E + c] : 0.0f;
      for (int k = 0; k < K; ++k) {
        const float add = __uint_as_float(readlane_u32(__float_as_uint(dz), k));
        if ((int32_t)readlane_u32((uint32_t)id, k) == c) v += add;
      }
      grad_out[t * E + c] = v;
    }
    if (dzb) dzb[t * ldb + c] = __builtin_bit_cast(uint16_t, (__bf16)v);
  }
}

// dx[t] = base[t] + sum_k Y[src_pos[t, k]] in fp32, slot order, 8 columns a
// thread (base NULL: zero).
template <int K>
__global__ __launch_bounds__(256) void sum_pairs_kernel(const uint16_t* __restrict__ base,
                                                        const uint16_t* __restrict__ Y,
                                                        const int32_t* __restrict__ src_pos,
                                                        int64_t N, int d,
                                                        uint16_t* __restrict__ out) {
  typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
  const int cpr = d / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= N * cpr) return;
  const int64_t t = i / cpr;
  const int c = (int)(i % cpr) * 8;
  u32x4_t v[K + 1];
#pragma unroll
  for (int k = 0; k < K; ++k)
    v[k] = __builtin_nontemporal_load(
        reinterpret_cast<const u32x4_t*>(Y + (int64_t)src_pos[t * K + k] * d + c));
  v[K] = base ? *reinterpret_cast<const u32x4_t*>(base + t * d + c) : u32x4_t{0u, 0u, 0u, 0u};
  float s[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    s[2 * j] = __uint_as_float(v[K][j] << 16);
    s[2 * j + 1] = __uint_as_float(v[K][j] & 0xFFFF0000u);
  }
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s[2 * j] += __uint_as_float(v[k][j] << 16);
      s[2 * j + 1] += __uint_as_float(v[k][j] & 0xFFFF0000u);
    }
  const u32x4_t o = {pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3]), pack_bf16(s[4], s[5]),
                     pack_bf16(s[6], s[7])};
  *reinterpret_cast<u32x4_t*>(out + t * d + c) = o;
}

}  // namespace

// ---------------------------------------------------------------- launchers
hipError_t launch_pairs(const int32_t* ids, const float* Z, int64_t pairs, int E, int K,
                        int32_t* ids_out, float* S, hipStream_t stream) {
  hipLaunchKernelGGL(pairs_kernel, dim3((unsigned)((pairs + 255) / 256)), dim3(256), 0, stream, ids,
                     Z, pairs, E, K, ids_out, S);
  return hipGetLastError();
}

hipError_t launch_row_tiles(const int32_t* offsets, int E, int32_t* tiles, int32_t* n_tiles,
                            hipStream_t stream) {
  hipLaunchKernelGGL(row_tiles_kernel, dim3(1), dim3(512), 0, stream, offsets, E, tiles, n_tiles);
  return hipGetLastError();
}

int grad_tile_rows() { return TM; }

static int64_t rows_blocks(const RowsProblem& p) {
  const int64_t m_tiles = p.tiles ? p.max_tiles : (p.rows_dense + TM - 1) / TM;
  return (m_tiles * p.n_tiles_n + kXcds - 1) / kXcds * kXcds;
}

template <bool F32>
static hipError_t start_rows(const RowsProblem& t, const RowsProblem& r, int64_t token_blocks,
                             int64_t blocks, hipStream_t stream) {
  static std::atomic<uint32_t> configured{0};
  const hipError_t e = set_lds_limit_once((const void*)rows_kernel<F32>, kLdsBytes, configured);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(rows_kernel<F32>, dim3((unsigned)blocks), dim3(512), kLdsBytes, stream, t, r,
                     token_blocks);
  return hipGetLastError();
}

hipError_t launch_rows(const RowsProblem* token, const RowsProblem& pair, bool out_f32,
                       hipStream_t stream) {
  RowsProblem t{}, r = pair;
  if (token) t = *token;
  t.n_tiles_n = (t.ncols + TN - 1) / TN;
  r.n_tiles_n = (r.ncols + TN - 1) / TN;
  const int64_t tb = token ? rows_blocks(t) : 0;
  const int64_t blocks = tb + rows_blocks(r);
  if (blocks > 0x7FFFFFF0LL) return hipErrorInvalidConfiguration;
  return out_f32 ? start_rows<true>(t, r, tb, blocks, stream)
                 : start_rows<false>(t, r, tb, blocks, stream);
}

hipError_t launch_weights(WeightsLaunch w, hipStream_t stream) {
  static std::atomic<uint32_t> configured{0};
  hipError_t e = set_lds_limit_once((const void*)weights_kernel, kLdsBytes, configured);
  if (e != hipSuccess) return e;
  int64_t blocks = 0;
  for (int i = 0; i < w.n_dense; ++i) {
    w.dense[i].tiles_m = (w.dense[i].a_cols + TM - 1) / TM;
    w.dense[i].tiles_n = (w.dense[i].b_cols + TN - 1) / TN;
    blocks += (int64_t)w.dense[i].tiles_m * w.dense[i].tiles_n;
  }
  int64_t per = 0;
  for (int i = 0; i < 2; ++i) {
    w.expert[i].tiles_m = (w.expert[i].a_cols + TM - 1) / TM;
    w.expert[i].tiles_n = (w.expert[i].b_cols + TN - 1) / TN;
    per += (int64_t)w.expert[i].tiles_m * w.expert[i].tiles_n;
  }
  blocks += (w.E * per + kXcds - 1) / kXcds * kXcds;
  if (blocks > 0x7FFFFFF0LL) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(weights_kernel, dim3((unsigned)blocks), dim3(512), kLdsBytes, stream, w);
  return hipGetLastError();
}

hipError_t launch_logits_grad(const float* Z, const int32_t* ids, const int32_t* src_pos,
                              const float* dscore_part, int parts, int64_t N, int E, int K,
                              const float* grad_in, float* grad_out, uint16_t* dzb, int ldb,
                              hipStream_t stream) {
  hipLaunchKernelGGL(logits_grad_kernel, dim3((unsigned)((N + 3) / 4)), dim3(256), 0, stream, Z,
                     ids, src_pos, dscore_part, parts, N, E, K, grad_in, grad_out, dzb, ldb);
  return hipGetLastError();
}

hipError_t launch_sum_pairs(const uint16_t* base, const uint16_t* Y, const int32_t* src_pos,
                            int64_t N, int K, int d, uint16_t* out, hipStream_t stream) {
  const dim3 grid((unsigned)((N * (d / 8) + 255) / 256));
#define MOE_K(n)                                                                              \
  case n:                                                                                     \
    hipLaunchKernelGGL(sum_pairs_kernel<n>, grid, dim3(256), 0, stream, base, Y, src_pos, N,  \
                       d, out);                                                               \
    break;
  switch (K) { MOE_K(1) MOE_K(2) MOE_K(3) MOE_K(4) MOE_K(5) MOE_K(6) MOE_K(7) MOE_K(8)
    default: return hipErrorInvalidValue;
  }
#undef MOE_K
  return hipGetLastError();
}

}  // namespace moe
