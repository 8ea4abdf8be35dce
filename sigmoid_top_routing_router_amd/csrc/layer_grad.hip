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
//  * rows_tile: Q and the parts of dx (fp32), C[row, n] = sum_k A[row, k]
//    B[k, n]: the rows are k-contiguous, the weights are read as they are
//    stored, n contiguous;
//  * weights_tiles: every weight gradient, C[m, n] = sum_row A[row, m]
//    B[row, n] over the rows of an expert's segment: both operands n
//    contiguous.
// Q is a launch of its own (rows_kernel); the parts of dx and the weights'
// gradients share one (gradients_kernel: 333 tokens of 320, 20 experts of 160,
// 11 us, in two launches 11 + 10).
// Both multiply 128 x 256 tiles with v_mfma_f32_32x32x16_bf16, four waves of
// 128 x 64, two blocks to a CU, so that one block's start, loads and stores
// pass behind the other's MFMAs.  rows_tile has long sums: A in stages of 64
// k (whole 128-byte lines of its rows) kept twice, B in halves of 32 k kept
// three times.  weights_tiles has short ones (an expert's rows, some 256) and
// large results: stages of 32 k kept three times, and a block takes two tiles
// under each other as one stream of stages, so that a tile's first loads and
// the last tile's stores pass behind MFMAs (one, three or four tiles at a time
// were not faster).
//
// The loads are written in assembly (they have no register result): as
// builtins, the compiler waits for all of them in front of the first
// transposing LDS read, which it takes for a possible reader of what they
// write, and a stage then never overlaps the next one's loads (the dx parts
// below with bf16 results: 1.68 ms so, 0.87 in assembly).  An operand whose k
// runs across rows is kept as [k][256] in LDS and read with the transposing
// LDS read (ds_read_b64_tr_b16: 16 lanes fetch 4 k x 16 columns and each gets
// one column's four k), so no transposed copy of a weight or an activation is
// ever made.  Its 16-byte chunk c of row k sits at c ^ 4 (k & 3): the four k
// of one read are then on four different groups of banks (no bank conflicts
// counted).
//
// Measured at 16384 tokens of 2560, 384 experts of 512, six a token, a shared
// expert of 512 (256 rows an expert, 6 GB of routed weights and gradients):
//   Q          301 GFLOP   0.39 ms   770 TFLOP/s, 2.3 GB read + written
//   dx parts   633 GFLOP   0.88 ms   720 TFLOP/s, 3.8 GB, 4.3 TB/s
//   weights    934 GFLOP   1.47 ms   635 TFLOP/s, 5.5 GB, 3.7 TB/s
// All are bound by the CU's path to the caches, which loads into LDS and
// results share: dx loads 7.3 GB into LDS and stores 1.2 (9.7 TB/s; loads
// alone reach some 12), the weights' gradients load 10.7 GB and store 3.0 (9.3
// TB/s).  Of the latter, MFMAs and LDS reads alone take 0.60 ms, without stores
// 0.77, loads and stores without MFMAs 1.3.  Two blocks of 128 x 256 a CU came
// together with a sixth of the address work, non-temporal stores and this order
// of items, in the place of one block of 256 x 256: weights 1.48 ms after 1.67, Q
// 0.40 after 0.43 (bf16 parts: dx 0.80 after 0.84).  What the tile's shape alone
// gives was not measured; 256 x 256 would load two thirds as much into LDS.
#include <type_traits>

#include "common.h"
#include "gemm_args.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int TM = 128, TN = 256;              // rows and columns of a tile
// rows_tile
constexpr int TK = 64;
constexpr int kRaBytes = TM * TK * 2;          // A of one stage, two slots
constexpr int kRbOff = 2 * kRaBytes;
constexpr int kRbBytes = TK / 2 * TN * 2;      // B of half a stage, three slots
constexpr int kRowsLds = kRbOff + 3 * kRbBytes;
static_assert(2 * kRowsLds <= 160 * 1024, "two blocks share a CU");
// weights_tiles
constexpr int WK = 32;
constexpr int kWaBytes = WK * TM * 2;          // A of one stage, then B
constexpr int kWSlot = kWaBytes + WK * TN * 2;
constexpr int kWSlots = 3;
constexpr int kIdsOff = kWSlots * kWSlot;      // gathered rows of eight stages
constexpr int kIdsSlot = 64 * 4;               // a wave loads 64, the first 32 are used
constexpr int kIdsSlots = 8;
constexpr int kWeightsLds = kIdsOff + kIdsSlots * kIdsSlot;
constexpr int kWGroup = 2;                     // tiles of a block
static_assert(2 * kWeightsLds <= 160 * 1024, "two blocks share a CU");
constexpr int kXcds = 8;
constexpr int64_t kMaxGradBlocks = (1 << 24) - 8;  // a grid's threads stay below 2^32

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// The wave's LDS reads have come back before it lets the others on: what they
// read may be overwritten then.
__device__ __forceinline__ void stage_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
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
__device__ __forceinline__ i32x4_t buffer_at(uint64_t a, uint32_t bytes) {
  return i32x4_t{__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
                 __builtin_amdgcn_readfirstlane((int)((uint32_t)(a >> 32) & 0xFFFFu)),
                 __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}
__device__ __forceinline__ i32x4_t buffer_at(const void* base, uint32_t bytes) {
  return buffer_at((uint64_t)base, bytes);
}
// An offset past the end of any operand: the load returns zeros.  Operands
// are smaller than this (checked by the entry point).
constexpr uint32_t kNoAddr = kGradMaxOperandBytes;
// LDS addresses are byte offsets of the block's LDS (these kernels have no
// static LDS, so the dynamic array starts at 0).
// LDS-DMA: 16 (dma4: 4) bytes per lane from a buffer to LDS at `at` + 16 (4) *
// lane.  Counted on vmcnt; the waits are this file's own (wait_vmcnt).  m0 (the
// LDS address) is set and used inside; nothing else in these kernels uses it.
// The first load of a block waits for m0 (one wait state) and for the scalar
// registers that v_readfirstlane may have written right in front of it (five):
// the compiler counts these for its own instructions only.
#define MOE_DMA_OPEN "s_mov_b32 m0, %0\n\ts_nop 3\n\t"
#define MOE_DMA16_NEXT(v, r) "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tbuffer_load_dwordx4 " v ", " r
__device__ __forceinline__ void dma4(i32x4_t r, uint32_t off, int at) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass does not know these operands
  asm volatile(MOE_DMA_OPEN "buffer_load_dword %1, %2, 0 offen lds"
               :: "s"(__builtin_amdgcn_readfirstlane(at)), "v"(off), "s"(r) : "memory");
#endif
}
// Four loads, each 1 KB after the other in LDS, at off + soff of the buffer.
__device__ __forceinline__ void dma_4(i32x4_t r, const uint32_t (&v)[4], uint32_t soff, int at) {
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile(MOE_DMA_OPEN "buffer_load_dwordx4 %1, %5, %6 offen lds\n\t"
               MOE_DMA16_NEXT("%2", "%5, %6 offen lds\n\t")
               MOE_DMA16_NEXT("%3", "%5, %6 offen lds\n\t")
               MOE_DMA16_NEXT("%4", "%5, %6 offen lds")
               :: "s"(__builtin_amdgcn_readfirstlane(at)), "v"(v[0]), "v"(v[1]), "v"(v[2]),
                  "v"(v[3]), "s"(r), "s"(__builtin_amdgcn_readfirstlane((int)soff))
               : "memory", "scc");
#endif
}
// Two loads of one buffer.
__device__ __forceinline__ void dma_2(i32x4_t r, const uint32_t (&v)[2], int at) {
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile(MOE_DMA_OPEN "buffer_load_dwordx4 %1, %3, 0 offen lds\n\t"
               MOE_DMA16_NEXT("%2", "%3, 0 offen lds")
               :: "s"(__builtin_amdgcn_readfirstlane(at)), "v"(v[0]), "v"(v[1]), "s"(r)
               : "memory", "scc");
#endif
}
template <class T>
__device__ __forceinline__ T lds_read(int at) {
  return *(const __attribute__((address_space(3))) T*)(uint32_t)at;
}

// Work item of a block: blocks are dealt to the XCDs in turn, each XCD takes
// a contiguous run of items.
__device__ __forceinline__ int64_t xcd_item(int64_t block, int64_t share) {
  return (block % kXcds) * share + block / kXcds;
}

// Eight k of one column from a stage of PITCH bytes a k-row: two transposing
// reads.
template <int PITCH>
__device__ __forceinline__ bf16x8_t read_tr(int at) {
  const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(uint32_t)at);
  const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(uint32_t)(at + 4 * PITCH));
  typedef short s16x8_t __attribute__((ext_vector_type(8)));
  const s16x8_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  return __builtin_bit_cast(bf16x8_t, v);
}

// What a lane reads of a [k][PITCH / 2] operand for the 32 columns of block
// blk: block_off(blk) + PITCH k of the k-step's first row.
template <int PITCH>
struct KRows {
  int kq, row, sub;
  __device__ __forceinline__ explicit KRows(int lane) {
    const int i = lane & 15;
    kq = i >> 2;
    row = (8 * (lane >> 5) + kq) * PITCH;
    sub = (2 * ((lane >> 4) & 1) + ((i & 3) >> 1)) * 16 + (i & 1) * 8;
  }
  __device__ __forceinline__ int block_off(int blk) const {
    return row + ((4 * blk) ^ (4 * kq)) * 16 + sub;
  }
};

template <int LIVE>
struct Fragments {  // of one k-step
  bf16x8_t A[LIVE], B[2];
};
// FIRST: the tile's first products.
template <bool FIRST, int LIVE>
__device__ __forceinline__ void multiply(const Fragments<LIVE>& f, floatx16_t (&acc)[4][2]) {
#pragma unroll
  for (int m = 0; m < LIVE; ++m)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      acc[m][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
          f.B[i], f.A[m], FIRST ? floatx16_t{} : acc[m][i], 0, 0, 0);
}

// The accumulators hold the wave's 128 x 64 outputs transposed (the B fragment
// is the first operand): lane l has row (l & 31) of a block and columns
// 8 (r / 4) + 4 (l / 32) + r % 4 of its register r.
//
// The upper 32 lanes' a change places with the lower lanes' b; the odd rows'
// (of 16 lanes) a with the even rows' b; within every 16 lanes, the upper
// eight's a with the lower eight's b.
__device__ __forceinline__ void swap_halves(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void swap_rows16(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void swap_rows8(uint32_t& a, uint32_t& b) {
  constexpr int kRor8 = 0x128;  // row_ror:8; the bank masks write one half of the 16
  const uint32_t a0 = a;
  a = (uint32_t)__builtin_amdgcn_update_dpp((int)a, (int)b, kRor8, 0xF, 0xC, false);
  b = (uint32_t)__builtin_amdgcn_update_dpp((int)b, (int)a0, kRor8, 0xF, 0x3, false);
}

// bf16 results, sixteen stores of 8 rows x 128 bytes: a lane's four columns of
// two register groups are joined with the other half's to eight (16 bytes),
// then rows trade places between lanes until eight lanes hold the 64 columns
// of one row, a whole cache line (32 rows x 32 bytes a store took twice the
// time).  Always sixteen: rows and columns past the result fall outside the
// buffer.  Lane l stores row line_row(l), columns line_col(l) .. + 7 of every
// group of eight rows; `at` is that place's byte offset, pitch a row's bytes.
__device__ __forceinline__ int line_row(int lane) { return lane & 7; }
__device__ __forceinline__ int line_col(int lane) {
  return 32 * ((lane >> 3) & 1) + 16 * ((lane >> 4) & 1) + 8 * (lane >> 5);
}
constexpr uint32_t kNoStore = 0x80000000u;  // past any result (below 2 GiB)
template <int CPOL>
__device__ __forceinline__ void store_lines(const floatx16_t (&acc)[4][2],
                                            __amdgpu_buffer_rsrc_t out, uint32_t at,
                                            uint32_t pitch) {
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    uint32_t v[2][2][4];  // [f][register groups 2 u and 2 u + 1]
#pragma unroll
    for (int f = 0; f < 2; ++f) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          v[f][u][j] = pack_bf16(acc[m][f][8 * u + 2 * j], acc[m][f][8 * u + 2 * j + 1]);
          v[f][u][2 + j] = pack_bf16(acc[m][f][8 * u + 4 + 2 * j], acc[m][f][8 * u + 5 + 2 * j]);
          swap_halves(v[f][u][j], v[f][u][2 + j]);
        }
#pragma unroll
      for (int j = 0; j < 4; ++j) swap_rows16(v[f][0][j], v[f][1][j]);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int j = 0; j < 4; ++j) swap_rows8(v[0][u][j], v[1][u][j]);
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const i32x4_t w = {(int)v[f][u][0], (int)v[f][u][1], (int)v[f][u][2], (int)v[f][u][3]};
        __builtin_amdgcn_raw_buffer_store_b128(
            w, out, (int)(at + (uint32_t)(32 * m + 16 * u + 8 * f) * pitch), 0, CPOL);
      }
    }
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

// Blocks of a share of the grid that deals `work` items to the XCDs.
__host__ __device__ __forceinline__ int64_t xcd_blocks(int64_t work) {
  return (work + kXcds - 1) / kXcds * kXcds;
}

// ---------------------------------------------------------------- rows
// PAIR: rows of the tile table, else tokens.  The results are fp32: Q, and the
// parts of dx, which are summed before they are rounded.
//
// The segments' stages are one stream.  Half-stage h (32 k) opens with a wait
// for the wave's own loads of it and the barrier that shows them to all waves
// and frees what half-stage h - 1 read; then it loads B of half-stage h + 2
// and, when h is the first half of stage j, A of stage j + 1.  Rows past the
// tile repeat its last row and columns past the result column 0 (what they
// give is not stored); k past a segment reads zeros of both.
template <bool PAIR, bool GATHER>
__device__ __forceinline__ void rows_tile(const RowsProblem& p, int64_t mt, int nt) {
  const int n0 = nt * TN;
  int expert = 0, rows;
  int64_t row0;
  if constexpr (PAIR) {
    const int4 ent = reinterpret_cast<const int4*>(p.tiles)[mt];
    expert = ent.x;
    row0 = ent.y;
    rows = ent.z & 0xFF;
  } else {
    row0 = mt * TM;
    rows = (int)min((int64_t)TM, p.rows_dense - row0);
  }
  const int tid = threadIdx.x, lane = tid & 63;
  const int wp = __builtin_amdgcn_readfirstlane(tid >> 6);  // columns 64 wp ..

  // LDS-DMA: load i of a wave covers A rows 32 wp + 8 i .. + 7 (lane -> row +
  // (l >> 3), slot l & 7, which holds chunk (l & 7) ^ ((row >> 1) & 7)) and B
  // k-rows 8 wp + 2 i + x (lane -> x = l >> 5, slot l & 31).
  uint32_t a_row[4];  // row index, or byte offset when gathered
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = min(32 * wp + 8 * i + (lane >> 3), rows - 1);
    a_row[i] = GATHER ? p.gather[row0 + r] : (uint32_t)r;
  }
  const uint32_t b_pitch = (uint32_t)p.ncols * 2u;
  uint32_t b_lane[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = 8 * wp + 2 * i + (lane >> 5);
    const int c = n0 + 8 * ((lane & 31) ^ (4 * (k & 3)));
    b_lane[i] = (uint32_t)k * b_pitch + (uint32_t)(c < p.ncols ? c : 0) * 2u;
  }
  // the next stage to load
  i32x4_t ra = {};
  uint64_t b_at = 0;     // address of the stage in B
  uint32_t a_lane[4] = {};
  int seg = -1, left = 0;  // left: k of the segment from this stage on
  uint32_t a_k = 0;        // byte offset of the stage in A's rows
  const int chunk0 = (lane & 7) ^ (lane >> 4);  // of loads 0 and 2; 1 and 3: ^ 4
  auto next_stage = [&] {
    left -= TK;
    a_k += TK * 2;
    b_at += (uint64_t)TK * b_pitch;
    if (left <= 0 && seg + 1 < p.n_seg) {
      ++seg;
      const RowsSegment& sg = p.seg[seg];
      // a gathered A spans the whole buffer, a direct one this tile's rows
      ra = buffer_at(GATHER ? sg.A : sg.A + row0 * sg.lda,
                     (uint32_t)((GATHER ? p.a_rows : rows) * sg.lda * 2));
      b_at = (uint64_t)(sg.B + (int64_t)expert * sg.b_expert_stride);
      left = sg.kdim;
      a_k = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        a_lane[i] = a_row[i] * (GATHER ? 1u : (uint32_t)(sg.lda * 2)) +
                    (uint32_t)(chunk0 ^ (4 * (i & 1))) * 16u;
    }
    if (left < TK) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        a_lane[i] = 8 * (chunk0 ^ (4 * (i & 1))) < left ? a_lane[i] + a_k : kNoAddr;
      a_k = 0;
    }
  };
  int total = 0;
  for (int i = 0; i < p.n_seg; ++i) total += (p.seg[i].kdim + TK - 1) / TK;
  int a_slot = 0, b_slot = 0;  // of the next loads
  auto load_a = [&] {
    dma_4(ra, a_lane, a_k, a_slot + wp * 4096);
    a_slot ^= kRaBytes;
  };
  auto load_b = [&](int half) {
    const int n = min(max(left - half * (TK / 2), 0), TK / 2);  // past the last stage: none
    const i32x4_t rb = buffer_at(b_at + (uint64_t)(half * (TK / 2)) * b_pitch, (uint32_t)n * b_pitch);
    dma_4(rb, b_lane, 0u, kRbOff + b_slot + wp * 4096);
    b_slot = b_slot == 2 * kRbBytes ? 0 : b_slot + kRbBytes;
  };

  floatx16_t acc[4][2];
  clear_acc(acc);
  const KRows<512> kb(lane);
  const int b_off[2] = {kRbOff + kb.block_off(2 * wp), kRbOff + kb.block_off(2 * wp + 1)};
  const int a_base = (lane & 31) * 128, a_swz = (lane >> 1) & 7, a_hi = lane >> 5;
  auto run = [&](auto live_tag) {
    constexpr int LIVE = decltype(live_tag)::value;  // row blocks with valid rows
    constexpr int NF = LIVE > 0 ? LIVE : 1;
    int a_read = 0, b_read = 0;
    auto half = [&](auto half_tag) {
      constexpr int HALF = decltype(half_tag)::value;
      if (HALF == 0) wait_vmcnt<4>();
      else wait_vmcnt<8>();
      stage_barrier();
      Fragments<NF> f[2];
      if constexpr (LIVE > 0) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int i = 0; i < 2; ++i) f[k].B[i] = read_tr<512>(b_read + b_off[i] + k * (16 * 512));
          const int at = a_read + a_base + ((2 * (2 * HALF + k) + a_hi) ^ a_swz) * 16;
#pragma unroll
          for (int m = 0; m < NF; ++m) f[k].A[m] = lds_read<bf16x8_t>(at + m * (32 * 128));
        }
      }
      if (HALF == 0) {
        next_stage();
        load_a();
      }
      load_b(HALF);
      if constexpr (LIVE > 0) {
        multiply<false>(f[0], acc);
        multiply<false>(f[1], acc);
      }
      b_read = b_read == 2 * kRbBytes ? 0 : b_read + kRbBytes;
    };
    for (int j = 0; j < total; ++j) {
      half(std::integral_constant<int, 0>{});
      half(std::integral_constant<int, 1>{});
      a_read ^= kRaBytes;
    }
  };
  next_stage();
  load_a();
  load_b(0);
  load_b(1);
  const bool live = __builtin_amdgcn_readfirstlane(n0 + wp * 64 < p.ncols);
  const int live_m = (rows + 31) / 32;
  if (!live) run(std::integral_constant<int, 0>{});
  else if (live_m == 1) run(std::integral_constant<int, 1>{});
  else if (live_m == 2) run(std::integral_constant<int, 2>{});
  else if (live_m == 3) run(std::integral_constant<int, 3>{});
  else run(std::integral_constant<int, 4>{});
  wait_vmcnt<0>();  // nothing may still write the LDS when another block has it
  if (!live) return;

  // Thirty-two stores of 8 rows x 128 bytes, as store_lines makes them: the
  // four register groups of a block trade rows until eight lanes hold one
  // row's 32 columns.  Q is read by the next launch; the parts of dx pass the
  // caches (non-temporal).
  const uint32_t pitch = (uint32_t)p.ldo * 4u;
  const __amdgpu_buffer_rsrc_t out = make_rsrc(p.out + row0 * p.ldo, (uint32_t)rows * pitch);
  const int col = n0 + wp * 64 + 16 * ((lane >> 3) & 1) + 8 * ((lane >> 4) & 1) + 4 * (lane >> 5);
#pragma unroll
  for (int f = 0; f < 2; ++f) {
    const int c = col + 32 * f;
    const uint32_t at = c < p.ncols ? (uint32_t)(lane & 7) * pitch + (uint32_t)c * 4u : kNoStore;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      uint32_t v[4][4];  // rows 0, 16, 8, 24 .. + 7 of the block after the trades
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q][j] = __float_as_uint(acc[m][f][4 * q + j]);
        swap_rows16(v[0][j], v[1][j]);
        swap_rows16(v[2][j], v[3][j]);
        swap_rows8(v[0][j], v[2][j]);
        swap_rows8(v[1][j], v[3][j]);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const i32x4_t w = {(int)v[q][0], (int)v[q][1], (int)v[q][2], (int)v[q][3]};
        const int row = 32 * m + 16 * (q & 1) + 8 * (q >> 1);
        __builtin_amdgcn_raw_buffer_store_b128(w, out, (int)(at + (uint32_t)row * pitch), 0,
                                               GATHER ? 0 : kCpolNT);
      }
    }
  }
}

// The work item of block b of a problem's share of the grid.  Items run over
// the row tiles of an expert (of the tokens) four at a time: the four of a
// column tile follow each other, so that they read the same B within the time
// that the L2 keeps it, then the next column tile, which reads the same A.
constexpr int kRowGroup = 4;
template <bool PAIR, bool GATHER>
__device__ __forceinline__ void rows_block(const RowsProblem& p, int64_t b) {
  const int64_t m_tiles = PAIR ? (int64_t)*p.n_tiles : (p.rows_dense + TM - 1) / TM;
  const int64_t work = m_tiles * p.n_tiles_n;
  const int64_t share = (work + kXcds - 1) / kXcds;
  if (b / kXcds >= share) return;
  const int64_t item = xcd_item(b, share);
  if (item >= work) return;
  const int64_t mt = item / p.n_tiles_n;
  int64_t index = mt, count = m_tiles;  // of the tile among its expert's
  if constexpr (PAIR) {
    const int4 ent = reinterpret_cast<const int4*>(p.tiles)[mt];
    index = ent.z >> 8;
    count = ent.w;
  }
  const int in_group = (int)(index % kRowGroup);
  const int group = (int)min((int64_t)kRowGroup, count - (index - in_group));
  const int l = in_group * p.n_tiles_n + (int)(item % p.n_tiles_n);
  rows_tile<PAIR, GATHER>(p, mt - in_group + l % group, l / group);
}

// Q of the shared expert (token, its token_blocks blocks first) and of the
// pairs.
__global__ __launch_bounds__(256, 2) void rows_kernel(RowsProblem token, RowsProblem pair,
                                                      int64_t token_blocks) {
  const int64_t b = blockIdx.x;
  if (b < token_blocks) rows_block<false, false>(token, b);
  else rows_block<true, true>(pair, b - token_blocks);
}

// ---------------------------------------------------------------- weights
// Tiles mt0 .. mt0 + T - 1 of column tile nt.  Stage s of the stream is k-block
// s % nk of tile s / nk, two k-steps of 16.  At the top of stage s every wave
// waits for its loads of stage s, then passes the barrier that shows them to
// all waves, and issues one batch: the gathered rows of stage s + 4 (4-byte
// LDS-DMA, the same bytes from every wave) and the six operand loads of stage
// s + 2, whose rows came with batch s - 2; past the last stage they go on
// loading the last tile's rows, so that every batch has as many.  The wait lets
// batch s - 1 stay in flight, and in a tile's first two stages the sixteen
// stores of the tile before: behind batch s - 2 in the order that vmcnt counts.
//
// Row r of a stage in LDS holds k-row pi(r) of the block of 32, the same for A
// and B (their products are summed over k, so its order is free): r = 8 w + 2 i
// + x holds 8 w + 4 x + i, which lets a lane fetch its four gathered rows at
// once.  Rows past the segment are zero in the operand that is not gathered;
// the gathered one repeats the segment's last row there.  Columns past an
// operand load column 0 instead; what they give is never stored.
enum Gathered { kNeither, kA, kB };
template <Gathered GATHER>
__device__ __forceinline__ void weights_tiles(const WeightsProblem& p, int expert, int mt0, int T,
                                              int nt) {
  const int n0 = nt * TN;
  int64_t first, rows;
  if constexpr (GATHER != kNeither) {
    first = p.offsets[expert];
    rows = (int64_t)p.offsets[expert + 1] - first;
  } else {
    first = 0;
    rows = p.rows_dense;
  }
  const int tid = threadIdx.x, lane = tid & 63;
  const int wp = __builtin_amdgcn_readfirstlane(tid >> 6);  // 0..3: columns 64 wp ..
  const bool live = __builtin_amdgcn_readfirstlane(n0 + wp * 64 < p.b_cols);

  floatx16_t acc[4][2];
  // The results are not read again here: non-temporal, they leave the caches
  // to the operands.
  const __amdgpu_buffer_rsrc_t ro = make_rsrc(p.out + (int64_t)expert * p.out_stride,
                                              (uint32_t)p.a_cols * (uint32_t)p.b_cols * 2u);
  const uint32_t o_pitch = (uint32_t)p.b_cols * 2u;
  const int o_col = n0 + wp * 64 + line_col(lane);
  const uint32_t o_lane =
      o_col < p.b_cols ? (uint32_t)line_row(lane) * o_pitch + (uint32_t)o_col * 2u : kNoStore;
  auto store = [&](int mt) {
    store_lines<kCpolNT>(acc, ro, o_lane + (uint32_t)(mt * TM) * o_pitch, o_pitch);
  };
  if (rows == 0) {  // an expert without rows: zeros
    clear_acc(acc);
    for (int t = 0; t < T; ++t) store(mt0 + t);
    return;
  }

  // LDS-DMA: load i of a wave fills A rows 8 wp + 4 i + q of the stage (lane ->
  // q = l >> 4, slot l & 15), i < 2, and B rows 8 wp + 2 i + x (lane -> x = l
  // >> 5, slot l & 31), i < 4.
  const int nk = (int)((rows + WK - 1) / WK);
  const uint32_t a_pitch = (uint32_t)p.lda * 2u, b_pitch = (uint32_t)p.ldb * 2u;
  const int q = lane >> 4, x = lane >> 5;
  const int a_chunk = (lane & 15) ^ (4 * q);                   // row & 3 = q
  const int b_slot = lane & 31;
  int b_chunk[4];                                              // row & 3 = 2 (i & 1) + x
#pragma unroll
  for (int i = 0; i < 4; ++i) b_chunk[i] = b_slot ^ (4 * (2 * (i & 1) + x));
  uint32_t b_lane[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = n0 + 8 * b_chunk[i] < p.b_cols ? n0 + 8 * b_chunk[i] : 0;
    b_lane[i] = (uint32_t)c * 2u + (GATHER == kB ? 0u : (uint32_t)(8 * wp + 4 * x + i) * b_pitch);
  }
  const int a_id = 8 * wp + 4 * (q & 1) + (q >> 1), b_id = 8 * wp + 4 * x;  // first gathered row
  const char* a_base = reinterpret_cast<const char*>(p.A) + (GATHER == kA ? 0 : first * (int64_t)a_pitch);
  const char* b_base = reinterpret_cast<const char*>(p.B) + (GATHER == kB ? 0 : first * (int64_t)b_pitch);
  const uint32_t g_bytes = (uint32_t)(p.tok_rows * (int64_t)(GATHER == kA ? a_pitch : b_pitch));
  const i32x4_t r_ids = buffer_at(p.tok + first, 0x7FFFFFFFu);
  const int last_row = (int)rows - 1;

  // the next batch's position: gathered rows, then operands
  int ik = 0, dk = 0, dt = 0, islot = 0, dslot = 0, dids = 0;
  uint32_t a_lane[2];
  auto set_tile = [&] {
    const int c = (mt0 + dt) * TM + 8 * a_chunk;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      a_lane[i] = (uint32_t)(c < p.a_cols ? c : 0) * 2u +
                  (GATHER == kA ? 0u : (uint32_t)(a_id + 2 * i) * a_pitch);
  };
  auto next_ids = [&] {
    if constexpr (GATHER != kNeither) {
      dma4(r_ids, (uint32_t)min(ik * WK + lane, last_row) * 4u, kIdsOff + islot * kIdsSlot);
      islot = (islot + 1) & (kIdsSlots - 1);
      ik = ik + 1 == nk ? 0 : ik + 1;
    }
  };
  auto next_data = [&] {
    const int64_t row = (int64_t)dk * WK;
    const uint32_t left = (uint32_t)min((int64_t)WK, rows - row);
    uint32_t a[2] = {a_lane[0], a_lane[1]}, b[4] = {b_lane[0], b_lane[1], b_lane[2], b_lane[3]};
    const int id = kIdsOff + dids * kIdsSlot;
    if constexpr (GATHER == kA) {
#pragma unroll
      for (int i = 0; i < 2; ++i) a[i] += lds_read<uint32_t>(id + (a_id + 2 * i) * 4);
    } else if constexpr (GATHER == kB) {
      typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
      const u32x4_t r = lds_read<u32x4_t>(id + b_id * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] += r[i];
    }
    const i32x4_t ra = GATHER == kA ? buffer_at(a_base, g_bytes)
                                    : buffer_at(a_base + row * (int64_t)a_pitch, left * a_pitch);
    const i32x4_t rb = GATHER == kB ? buffer_at(b_base, g_bytes)
                                    : buffer_at(b_base + row * (int64_t)b_pitch, left * b_pitch);
    const int at = dslot * kWSlot;
    dma_2(ra, a, at + wp * 2048);
    dma_4(rb, b, 0u, at + kWaBytes + wp * 4096);
    dslot = dslot == kWSlots - 1 ? 0 : dslot + 1;
    dids = (dids + 1) & (kIdsSlots - 1);
    if (++dk == nk) {
      dk = 0;
      if (dt + 1 < T) {
        ++dt;
        set_tile();
      }
    }
  };
  set_tile();
  if constexpr (GATHER != kNeither) {
    next_ids();
    next_ids();
    wait_vmcnt<0>();
    stage_barrier();
  }
  // batches -2 and -1
  for (int s = 0; s < 2; ++s) {
    next_ids();
    next_data();
  }
  constexpr int kBatch = GATHER != kNeither ? 7 : 6;

  const KRows<256> ka(lane);
  const KRows<512> kb(lane);
  int a_off[4], b_off[2];
#pragma unroll
  for (int m = 0; m < 4; ++m) a_off[m] = ka.block_off(m);
#pragma unroll
  for (int f = 0; f < 2; ++f) b_off[f] = kWaBytes + kb.block_off(2 * wp + f);
  auto run = [&](auto live_tag) {
    constexpr bool LIVE = decltype(live_tag)::value;
    int slot = 0;
    auto read = [&](Fragments<4>& f, int k) {  // k-step k of the stage in slot
#pragma unroll
      for (int i = 0; i < 2; ++i) f.B[i] = read_tr<512>(slot + b_off[i] + k * (16 * 512));
#pragma unroll
      for (int m = 0; m < 4; ++m) f.A[m] = read_tr<256>(slot + a_off[m] + k * (16 * 256));
    };
    auto stage = [&](auto first_tag, bool behind_stores) {
      if (behind_stores) wait_vmcnt<kBatch + 16>();
      else wait_vmcnt<kBatch>();
      stage_barrier();  // and every wave has left stage s - 1, whose slot is s + 2's
      Fragments<4> f0, f1;
      if constexpr (LIVE) {
        read(f0, 0);
        read(f1, 1);
      }
      next_ids();
      next_data();
      if constexpr (LIVE) {
        multiply<decltype(first_tag)::value>(f0, acc);
        multiply<false>(f1, acc);
      }
      slot = slot == (kWSlots - 1) * kWSlot ? 0 : slot + kWSlot;
    };
    for (int t = 0; t < T; ++t) {
      const bool stored = LIVE && t > 0;
      stage(std::true_type{}, stored);
      if (nk > 1) stage(std::false_type{}, stored);
      for (int k = 2; k < nk; ++k) stage(std::false_type{}, false);
      if constexpr (LIVE) store(mt0 + t);
    }
  };
  if (live) run(std::true_type{});
  else run(std::false_type{});
  wait_vmcnt<0>();  // nothing may still write the LDS when it is used again
}

// Items: the dense problems' tiles first (their sums run over all tokens),
// then expert by expert the gate and up tiles, then the down tiles: what the
// blocks of one XCD read at a time (one or two experts' rows of x and dG | dU,
// or of dy and s H) then stays in its L2.
__device__ __forceinline__ void weights_block(const WeightsLaunch& w, int64_t b) {
  for (int i = 0; i < w.n_dense; ++i) {
    const int t = w.dense[i].tiles_m * w.dense[i].tiles_n;
    if (b < t) {
      weights_tiles<kNeither>(w.dense[i], 0, (int)b / w.dense[i].tiles_n, 1,
                              (int)b % w.dense[i].tiles_n);
      return;
    }
    b -= t;
  }
  // gate and up have the same tiles
  const WeightsProblem &gu = w.expert[0], &dn = w.expert[2];
  const int gm = (gu.tiles_m + kWGroup - 1) / kWGroup, dm = (dn.tiles_m + kWGroup - 1) / kWGroup;
  const int per_gu = 2 * gm * gu.tiles_n, per_dn = dm * dn.tiles_n;
  const int64_t gu_blocks = xcd_blocks((int64_t)w.E * per_gu);
  const bool up_down = b >= gu_blocks;
  if (up_down) b -= gu_blocks;
  const int per = up_down ? per_dn : per_gu;
  const int64_t work = (int64_t)w.E * per;
  const int64_t share = (work + kXcds - 1) / kXcds;
  if (b / kXcds >= share) return;
  const int64_t item = xcd_item(b, share);
  if (item >= work) return;
  const int e = (int)(item / per);
  const int r = (int)(item % per);
  if (!up_down) {
    const int n = r / (2 * gm), g = r % (2 * gm);  // the tiles of one column tile of x together
    const int m = g % gm * kWGroup;
    weights_tiles<kB>(w.expert[g / gm], e, m, min(kWGroup, gu.tiles_m - m), n);
  } else {
    const int m = r / dn.tiles_n * kWGroup;
    weights_tiles<kA>(dn, e, m, min(kWGroup, dn.tiles_m - m), r % dn.tiles_n);
  }
}

// The parts of dx (the tokens' token_blocks blocks, then the pairs', row_blocks
// in all), then the weights' gradients: one launch, whose second part begins
// on the CUs that the first has left.
__global__ __launch_bounds__(256, 2) void gradients_kernel(RowsProblem token, RowsProblem pair,
                                                           int64_t token_blocks,
                                                           int64_t row_blocks, WeightsLaunch w) {
  const int64_t b = blockIdx.x;
  if (b < token_blocks) rows_block<false, false>(token, b);
  else if (b < row_blocks) rows_block<true, false>(pair, b - token_blocks);
  else weights_block(w, b - row_blocks);
}

// ---------------------------------------------------------------- small kernels
// One thread per pair: the id kept inside [0, E), and the pair's weight
// sigma(z), -1 for an id outside the range: such a pair is dropped.  It stays
// a row of expert 0's segment, all zeros whatever its token holds: x and dy
// are gathered from no address, and the epilogue of G and U puts zeros in
// their place.
__global__ __launch_bounds__(256) void pairs_kernel(const int32_t* __restrict__ ids,
                                                    const float* __restrict__ Z, int64_t pairs,
                                                    int E, int K, int32_t* __restrict__ ids_out,
                                                    float* __restrict__ S) {
  const int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (p >= pairs) return;
  const uint32_t e = (uint32_t)ids[p];
  const bool in = e < (uint32_t)E;
  ids_out[p] = in ? (int32_t)e : 0;
  S[p] = in ? sigmoid_weight(Z[p / K * E + e]) : -1.0f;
}

// Of the grouped pairs: the byte offset of every row's token in x (pitch bytes
// a token; the same in dy), kNoAddr for a dropped pair; block 0 also makes the
// row tiles of rows_tile from the segment offsets (thread e counts its
// expert's tiles, a scan places them).
__global__ __launch_bounds__(512) void grouped_rows_kernel(
    const int32_t* __restrict__ sorted_src, const float* __restrict__ S, int64_t pairs, int K,
    uint32_t pitch, const int32_t* __restrict__ offsets, int E, uint32_t* __restrict__ tok,
    int32_t* __restrict__ tiles, int32_t* __restrict__ n_tiles) {
  const int64_t i = (int64_t)blockIdx.x * 512 + threadIdx.x;
  if (i < pairs) {
    const int32_t p = sorted_src[i];
    tok[i] = S[p] < 0.0f ? kNoAddr : (uint32_t)(p / K) * pitch;
  }
  if (blockIdx.x != 0) return;
  __shared__ uint32_t wsum[8];
  const int e = threadIdx.x, w = e >> 6;
  const int32_t off = e < E ? offsets[e] : 0;
  const int32_t cnt = e < E ? offsets[e + 1] - off : 0;
  const uint32_t nt = (uint32_t)(cnt + TM - 1) / TM;
  const uint32_t inc = wave_inclusive_sum_u32(nt);
  if (lane_id() == 63) wsum[w] = inc;
  __syncthreads();
  uint32_t base = 0;
  for (int j = 0; j < w; ++j) base += wsum[j];
  uint32_t t = base + inc - nt;
  for (int32_t r = 0; r < cnt; r += TM)
    reinterpret_cast<int4*>(tiles)[t++] =
        make_int4(e, off + r, min(TM, cnt - r) | (r / TM) << 8, (int)nt);
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

// dx[t] = base[t] + sum_k Y[src_pos[t, k]], slot order, 4 columns a thread
// (base NULL: zero), rounded once.  One pass over the parts: 1.26 GB in 215 us
// (16384 x 2560, six parts and the tokens'), 5.8 TB/s.  With bf16 parts it and
// the parts' product took 230 us less of the layer's 3.9 ms, and dx was off by
// 0.0029 of its size instead of 0.0024.
template <int K>
__global__ __launch_bounds__(256) void sum_pairs_kernel(const float* __restrict__ base,
                                                        const float* __restrict__ Y,
                                                        const int32_t* __restrict__ src_pos,
                                                        int64_t N, int d,
                                                        uint16_t* __restrict__ out) {
  typedef float f32x4_t __attribute__((ext_vector_type(4)));
  const int cpr = d / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= N * cpr) return;
  const int64_t t = i / cpr;
  const int c = (int)(i % cpr) * 4;
  f32x4_t v[K + 1];
#pragma unroll
  for (int k = 0; k < K; ++k)
    v[k] = __builtin_nontemporal_load(
        reinterpret_cast<const f32x4_t*>(Y + (int64_t)src_pos[t * K + k] * d + c));
  v[K] = base ? __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(base + t * d + c))
              : f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) v[K][j] += v[k][j];
  *reinterpret_cast<uint2*>(out + t * d + c) =
      make_uint2(pack_bf16(v[K][0], v[K][1]), pack_bf16(v[K][2], v[K][3]));
}

}  // namespace

// ---------------------------------------------------------------- launchers
hipError_t launch_pairs(const int32_t* ids, const float* Z, int64_t pairs, int E, int K,
                        int32_t* ids_out, float* S, hipStream_t stream) {
  hipLaunchKernelGGL(pairs_kernel, dim3((unsigned)((pairs + 255) / 256)), dim3(256), 0, stream, ids,
                     Z, pairs, E, K, ids_out, S);
  return hipGetLastError();
}

hipError_t launch_grouped_rows(const int32_t* sorted_src, const float* S, int64_t pairs, int K,
                               uint32_t pitch, const int32_t* offsets, int E, uint32_t* tok,
                               int32_t* tiles, int32_t* n_tiles, hipStream_t stream) {
  hipLaunchKernelGGL(grouped_rows_kernel, dim3((unsigned)((pairs + 511) / 512)), dim3(512), 0,
                     stream, sorted_src, S, pairs, K, pitch, offsets, E, tok, tiles, n_tiles);
  return hipGetLastError();
}

int grad_tile_rows() { return TM; }

static int64_t rows_blocks(const RowsProblem& p) {
  const int64_t m_tiles = p.tiles ? p.max_tiles : (p.rows_dense + TM - 1) / TM;
  return xcd_blocks(m_tiles * p.n_tiles_n);
}

// Column tiles, and the blocks of the tokens' part and of both.
static void set_rows(RowsProblem& t, RowsProblem& r, bool token, int64_t& tb, int64_t& blocks) {
  t.n_tiles_n = (t.ncols + TN - 1) / TN;
  r.n_tiles_n = (r.ncols + TN - 1) / TN;
  tb = token ? rows_blocks(t) : 0;
  blocks = tb + rows_blocks(r);
}

hipError_t launch_rows(const RowsProblem* token, const RowsProblem& pair, hipStream_t stream) {
  static std::atomic<uint32_t> configured{0};
  const hipError_t e = set_lds_limit_once((const void*)rows_kernel, kRowsLds, configured);
  if (e != hipSuccess) return e;
  RowsProblem t = token ? *token : RowsProblem{}, r = pair;
  int64_t tb, blocks;
  set_rows(t, r, token != nullptr, tb, blocks);
  if (blocks > kMaxGradBlocks) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(rows_kernel, dim3((unsigned)blocks), dim3(256), kRowsLds, stream, t, r, tb);
  return hipGetLastError();
}

hipError_t launch_gradients(const RowsProblem* token, const RowsProblem& pair, WeightsLaunch w,
                            hipStream_t stream) {
  constexpr int kLds = kRowsLds > kWeightsLds ? kRowsLds : kWeightsLds;
  static std::atomic<uint32_t> configured{0};
  const hipError_t e = set_lds_limit_once((const void*)gradients_kernel, kLds, configured);
  if (e != hipSuccess) return e;
  RowsProblem t = token ? *token : RowsProblem{}, r = pair;
  int64_t tb, rb;
  set_rows(t, r, token != nullptr, tb, rb);
  int64_t blocks = rb;
  auto set_tiles = [](WeightsProblem& q) {
    q.tiles_m = (q.a_cols + TM - 1) / TM;
    q.tiles_n = (q.b_cols + TN - 1) / TN;
  };
  for (int i = 0; i < w.n_dense; ++i) {
    set_tiles(w.dense[i]);
    blocks += (int64_t)w.dense[i].tiles_m * w.dense[i].tiles_n;
  }
  for (WeightsProblem& q : w.expert) set_tiles(q);
  auto items = [](const WeightsProblem& q) { return (q.tiles_m + kWGroup - 1) / kWGroup * q.tiles_n; };
  blocks += xcd_blocks((int64_t)w.E * 2 * items(w.expert[0])) + xcd_blocks((int64_t)w.E * items(w.expert[2]));
  if (blocks > kMaxGradBlocks) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(gradients_kernel, dim3((unsigned)blocks), dim3(256), kLds, stream, t, r, tb,
                     rb, w);
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

hipError_t launch_sum_pairs(const float* base, const float* Y, const int32_t* src_pos,
                            int64_t N, int K, int d, uint16_t* out, hipStream_t stream) {
  const dim3 grid((unsigned)((N * (d / 4) + 255) / 256));
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
