// bf16 MFMA GEMM core for gfx950 with the MLP's fused epilogues.
//
// C[m,n] = sum_k A[m,k] B[k,n], bf16 operands, float32 accumulation on the
// bf16 MFMA instructions.  Every product of the tensor-parallel MLP's forward
// and backward is one launch with an operand layout and an epilogue (KC: K
// contiguous; MC: the other dimension contiguous; X^T, dZ^T and, when the
// planner chooses, A_i^T and B_i^T are transposed copies):
//
//   forward   P_i = X A_i          A: KC  B: MC (A_i) or KC (A_i^T)  epilogue GeLU -> G_i (and P_i)
//             Z_i = G_i B_i        A: KC  B: MC (B_i) or KC (B_i^T)  epilogue float32
//   backward  P_i = X A_i          as in the forward, epilogue bf16 (recompute)
//             dG_i = dZ B_i^T      A: KC  B: KC          epilogue dGeLU -> dP_i, G_i^T
//             dB_i = G_i^T dZ      A: KC  B: KC (dZ^T)   epilogue float32 (split-K)
//             dA_i = X^T dP_i      A: KC (X^T)  B: MC    epilogue float32 (split-K)
//             dX_i = dP_i A_i^T    A: KC  B: KC          epilogue float32
//
// (The split of A by columns and B by rows that makes rank i's work exactly
// these products: "大模型训练" notes §3.1; GeLU between the two GEMMs: QLM page
// §2.1.2.2 part 3; fusing the activation into the producing kernel so the
// float32 pre-activation never round-trips through memory: asorrir.com survey,
// part 三, 算子融合.)
//
// One kernel, gemm_x16_kernel, in three tile shapes (256 x 256, 256 x 128, 128 x
// 128): four waves, one per SIMD, each accumulating its sub-tile as 16 x 16
// blocks on v_mfma_f32_16x16x32_bf16, with loads and LDS reads placed between
// its MFMAs (its comment has the schedule).  Design points:
//  * A K-contiguous operand sits in LDS as 128-row slots of [rows][64 k]
//    (128-byte rows), so an MFMA operand fragment is one ds_read_b128 per lane
//    (8 consecutive k of one row); an N-contiguous one as [64 k][128 n] slots,
//    read with two ds_read_b64_tr_b16 per fragment.
//  * Operands go from memory straight into LDS with buffer_load ... lds (16
//    bytes per lane, no staging registers, no LDS write instructions).  Buffer
//    descriptors return zeros for out-of-range chunks, which handles ragged
//    sizes without branches.
//  * 16-byte chunks are XOR-swizzled within LDS rows so that the lanes of one
//    read instruction fall on distinct banks; the DMA loads apply the inverse
//    permutation on the memory side, so each DMA still writes 1 KiB of
//    contiguous LDS.
//  * The MFMA takes the B fragment as its first operand, so each lane ends with
//    4 consecutive output columns of one row; the epilogue restages them
//    through LDS and stores whole 128-byte lines.
//  * Workgroups are renumbered so that consecutive output tiles (which share
//    operand panels) run on the same XCD and its L2, then grouped 4 tiles tall.

#pragma once

#include "common.h"
#include "epilogue.h"

namespace tpmlp {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint16_t u16x4_t __attribute__((ext_vector_type(4)));
typedef uint16_t u16x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void_t;
typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef short i16x8_t __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) i16x4_t lds_i16x4_t;

// Rows of tiles per group of the grouped order: an XCD's 32 co-resident tiles span
// 4 rows x 8 columns of tiles (measured 1% faster than 8 x 4 and 2 x 16).
constexpr int GROUP_M = 4;
constexpr int NUM_XCD = 8;
constexpr uint32_t OOB = 0x7FFFFFF0u;  // voffset past num_records: the load returns 0

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)OOB, 0x00020000);
}

// ds_read_b64_tr_b16 from LDS address `p`.  Issued through inline assembly:
// the builtin makes the compiler wait for every vector-memory load in flight
// (vmcnt(0)) before it, in case an LDS-DMA load targets the same bytes, which
// would stall the load pipeline of this kernel on every memory phase (30 such
// waits in the main loop of the N-contiguous kernels with this compiler).
// Callers read only bytes whose loads and writes have already been waited for
// and made visible by a barrier, and wait for the results themselves
// (lgkmcnt(0)) before using them.  The compiler takes the output register as
// written when the statement issues, so no result may be left unused (its
// register could be handed out again while the read is in flight): every one
// is a fragment that the MFMAs after that wait consume.
typedef __attribute__((address_space(3))) char lds_char_t;
__device__ __forceinline__ i16x4_t ds_read_tr(const char* p) {
  i16x4_t v;
  const uint32_t a = (uint32_t)(uintptr_t)(const lds_char_t*)p;
  asm volatile("ds_read_b64_tr_b16 %0, %1" : "=v"(v) : "v"(a));
  return v;
}
// The same through the builtin, for the epilogue: no LDS-DMA load is in flight
// there, so the compiler orders the read after the wave's own LDS stores and
// waits for its result by itself, without waiting for the global loads.
__device__ __forceinline__ i16x4_t ds_read_tr_lds(const char* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)(const lds_char_t*)p);
}

// ---------------------------------------------------------------------------
// Pieces of the 16 x 16 x 32 kernel (gemm_x16_kernel)
// ---------------------------------------------------------------------------

// N-contiguous slot of the 16 x 16 x 32 kernel: 64 k-rows of 128 n, 256-byte rows.
// The 16-byte chunk holding n .. n+7 of k-row k sits at (n / 8) ^ (4 (k % 4) + 2
// ((k / 8) % 2)).  A transposing fragment read takes, per 16-lane group, 4
// consecutive k-rows x 32 bytes, and the LDS serves two groups per cycle whose
// k-rows lie 8 apart: the first term puts a group's 4 rows on distinct banks
// (unswizzled, rows 256 bytes apart hit the same ones), the second moves the
// other group's to the remaining banks.
__device__ __forceinline__ int mc16_x(int k) { return 4 * (k & 3) + 2 * ((k >> 3) & 1); }
__device__ __forceinline__ int mc16_off(int k, int n) { return k * 256 + (((n >> 3) ^ mc16_x(k)) << 4) + (n & 7) * 2; }

// K-contiguous [128 rows][64 k] slot of the 16 x 16 x 32 kernel: the 16-byte chunk c
// of row r sits at position c ^ ((r / 2) % 8).  The XOR depends on r % 16 only, so
// the 16-row fragments of a slot differ by a constant 2048 bytes (one base register
// per lane serves all of them), and the 16 rows of a fragment read at one chunk
// land on distinct 16-byte bank groups (even rows on 8 positions in one half of
// the banks, odd rows on 8 in the other).
__device__ __forceinline__ int swz16(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int tile16_off(int r, int c) { return r * 128 + ((c ^ swz16(r)) << 4); }

// LDS-DMA loads of one 128-row K-contiguous quarter of a K step: 4 instructions per
// wave of 1 KiB, instruction i of wave w filling rows 8 (4i + w) .. +7 of the slot;
// lane q writes position q % 8 of row q / 8 and loads the chunk the swizzle places
// there, which depends on the lane and w % 2 only.  Each lane's byte offset from
// the quarter's (first row, first k of the step) is computed once per tile, with
// lanes whose row is outside the operand set to OOB, so the only per-step masking
// left is that of a K tail.
struct QuarterKC {
  uint32_t voff[4];  // instruction i
  int kc;            // first k of the lane's chunk inside the K step

  __device__ __forceinline__ void init(int64_t ld, int rows_left, int w, int lane) {
    kc = 8 * ((lane & 7) ^ swz16(8 * w + (lane >> 3)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * (4 * i + w) + (lane >> 3);
      voff[i] = r < rows_left ? (uint32_t)(((int64_t)r * ld + kc) * 2) : OOB;
    }
  }
  // EPI_GLU: the quarter's 64 pairs, rows 32 i .. +31 (instruction i) gate rows for even
  // i and the same pairs' up rows for odd i, which the descriptor's base moves on to.
  __device__ __forceinline__ void init_pairs(int64_t ld, int pairs_left, int w, int lane) {
    kc = 8 * ((lane & 7) ^ swz16(8 * w + (lane >> 3)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 32 * (i >> 1) + 8 * w + (lane >> 3);
      voff[i] = r < pairs_left ? (uint32_t)(((int64_t)r * ld + kc) * 2) : OOB;
    }
  }
  // rs: descriptor based at the quarter's (first row, first k of the step); k_left:
  // elements of K from the step's first k (64 or more: no tail).
  __device__ __forceinline__ void issue(__amdgpu_buffer_rsrc_t rs, char* slot, int k_left, int w, int i) const {
    const uint32_t off = kc < k_left ? voff[i] : OOB;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)(slot + (4 * i + w) * 1024), 16, off, 0, 0, 0);
  }
};

// The same for an N-contiguous quarter (64 k-rows x 128 n, mc16_off layout):
// instruction i of wave w fills k-rows 4 (4i + w) .. +3; lane q writes position
// q % 16 of k-row q / 16 and loads the chunk placed there, which depends on the
// lane and on w / 2 only.
struct QuarterMC {
  uint32_t voff[4];
  int lane_k;  // k-row of the lane's chunk in instruction 0

  __device__ __forceinline__ void init(int64_t ld, int n_left, int w, int lane) {
    lane_k = 4 * w + (lane >> 4);
    const int n = 8 * ((lane & 15) ^ mc16_x(lane_k));
#pragma unroll
    for (int i = 0; i < 4; ++i)
      voff[i] = n < n_left ? (uint32_t)(((int64_t)(lane_k + 16 * i) * ld + n) * 2) : OOB;
  }
  // EPI_GLU: columns 64 b .. +31 of the quarter are pairs 32 b .. +31's gate columns, 64 b
  // + 32 .. +63 their up columns, `n` elements further in the row.
  __device__ __forceinline__ void init_pairs(int64_t ld, int pairs_left, int n_up, int w, int lane) {
    lane_k = 4 * w + (lane >> 4);
    const int c = 8 * ((lane & 15) ^ mc16_x(lane_k)), pair = 32 * (c >> 6) + (c & 31), up = (c >> 5) & 1;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      voff[i] = pair < pairs_left ? (uint32_t)(((int64_t)(lane_k + 16 * i) * ld + pair + (up ? n_up : 0)) * 2) : OOB;
  }
  // rs: descriptor based at the quarter's (first k of the step, first n).
  __device__ __forceinline__ void issue(__amdgpu_buffer_rsrc_t rs, char* slot, int k_left, int w, int i) const {
    const uint32_t off = lane_k + 16 * i < k_left ? voff[i] : OOB;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)(slot + (4 * i + w) * 1024), 16, off, 0, 0, 0);
  }
};

// Byte offset of lane `lane`'s first transposing read of the 16 x 16 x 32 B
// fragment at columns n0 .. n0+15 of an N-contiguous half, sub-step 0: in 16-lane
// group g, source lane s reads k-row 8g + s / 4, columns n0 + 4 (s % 4) .. +3, and
// ds_read_b64_tr_b16 hands lane i of the group the 4 k-values of column n0 + i.
// The second read (k-rows + 4) is 1024 bytes further, sub-step 1 (k + 32) 8192.
__device__ __forceinline__ uint32_t mc16_lane_off(int n0, int lane) {
  const int g = lane >> 4, sl = lane & 15;
  return mc16_off(8 * g + (sl >> 2), n0 + 4 * (sl & 3));
}

// Logical tile of workgroup `bid`: XCD-aware renumbering, then grouped order.
__device__ __forceinline__ void tile_of(int bid, int nblocks, int tiles_m, int tiles_n, int& tm, int& tn,
                                        int& split) {
  const int q = nblocks / NUM_XCD, rem = nblocks % NUM_XCD;
  const int xcd = bid % NUM_XCD, idx = bid / NUM_XCD;
  const int logical = xcd * q + min(xcd, rem) + idx;
  const int tiles = tiles_m * tiles_n;
  split = logical / tiles;
  const int t = logical % tiles;
  const int per_group = GROUP_M * tiles_n;
  const int group = t / per_group;
  const int first_m = group * GROUP_M;
  const int gsize = min(tiles_m - first_m, GROUP_M);
  const int in_group = t % per_group;
  tm = first_m + in_group % gsize;
  tn = in_group / gsize;
}

// Epilogue.  With the B fragment as the MFMA's first operand, accumulator
// register r of fragment (i, j) holds C[32i + lane%32][32j + 8(r/4) + 4(lane/32) + r%4]
// of the wave's sub-tile.  Each wave stages 64 rows of its float32 sub-tile
// at a time in LDS (row stride 256 bytes, 16-byte chunks XOR-swizzled by the
// row), reads them back row-contiguous and finishes 8 (bf16 outputs) or 4
// (float32) consecutive columns per lane, so every store instruction writes
// whole 128-byte lines.
// `stage` is this wave's 16 KiB of LDS, free of operand data; row_w and col_w
// are the first output row and column of the wave's (32 FM) x 64 tile.
constexpr int ROW_B = 256;  // staged row stride in bytes (64 float32)

// The dGeLU epilogue keeps the bf16 G rows of a chunk in its staging bytes at a
// 128-byte pitch (rows 2i and 2i+1 share one 256-byte line, so a store of two
// rows covers all 64 banks), 16-byte chunks swizzled by the row.  A transposing
// read of a 16-lane group takes rows b + 8 q + r (q, r < 4; b a multiple of 32)
// at one column chunk: for each parity of r those are 8 rows, and the swizzle
// puts them on 8 distinct chunks (one bank half per parity); the two groups that
// share a 32-lane half read different 8-byte halves of their chunks, so every
// read and store is free of bank conflicts.
__device__ __forceinline__ int gt_swz(int r) { return ((r >> 3) + 4 * ((r >> 1) & 1)) & 7; }
constexpr int G_ROW_B = 128;  // staged G row pitch in bytes

// The epilogue proper, independent of the MFMA accumulator layout.  The wave's
// region is NC chunks of 64 x 64, laid out nh chunks tall: chunk c covers rows
// row_w + 64 (c % nh) and columns col_w + 64 (c / nh) onward.  stage_chunk(c, sc)
// writes the chunk's float32 values (times sc for FP8 products, scale_fn() the
// product of the operands' scales) into `stage` (row r in 0..63 at r * ROW_B,
// 16-byte chunk q in 0..15 at position q ^ (r & 15)), and the chunk is finished
// from there.
// FP8 (FP8 products): EPI_BF16 and EPI_DGELU also collect the amax of what they
// write into args.amax_out when set (of the GeLU of the written values with
// args.amax_gelu), and EPI_DGELU writes dP only (no G^T).
// Paired products (EPI_F32_PAIR, EPI_F32_ACC_PAIR): stage_chunk2(c) writes product
// 1's values of chunk c the same way into `stage2`, and each output element is
// (running sum + product 0) + product 1, in that order.
template <int EPI, int NC, bool FP8, class StageChunk, class ScaleFn, class StageChunk2>
__device__ __forceinline__ void store_staged(StageChunk&& stage_chunk, ScaleFn&& scale_fn, const GemmArgs& args,
                                             char* stage, int row_w, int col_w, int nh, int split, int lane,
                                             StageChunk2&& stage_chunk2, char* stage2) {
  constexpr bool PAIR = EPI == EPI_F32_PAIR || EPI == EPI_F32_ACC_PAIR;
  constexpr bool ACC = EPI == EPI_F32_ACC || EPI == EPI_F32_ACC_PAIR;
  // FP8: running extremes of the written values (AmaxTrack, epilogue.h; invalid
  // elements enter as 0), updated without branches.
  AmaxTrack am;
  // Each phase below issues all of its memory operations before it waits for
  // any, and the global loads an epilogue needs (the dGeLU pre-activations, the
  // EPI_F32_ACC running sum) are double-buffered: chunk c + 1's are in flight
  // while chunk c is finished, so only the first chunk's latency is exposed.
  // LDS reads are batched ahead of the stores that use them.  Both loads go
  // through a buffer descriptor on the chunk's (uniform) first row and column,
  // so rows and columns outside the output read as zero without a branch.
  u16x8_t pre[2][8];
  f32x4_t old[2][16];
  auto row0 = [&](int c) { return row_w + 64 * (c % nh); };
  constexpr int CHUNK_N = is_glu(EPI) ? 32 : 64;  // output columns of a chunk (EPI_GLU: 32 pairs)
  auto col0 = [&](int c) { return col_w + CHUNK_N * (c / nh); };
  auto load_old = [&](int c) {
    const int r0 = row0(c), c0 = col0(c);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(reinterpret_cast<const float*>(args.out) + (int64_t)r0 * args.ldo + c0);
#pragma unroll
    for (int it = 0; it < 16; ++it) {
      const int q = it * 64 + lane, r = q >> 4, cq = q & 15;
      const bool ok = r0 + r < args.M && c0 + 4 * cq < args.N;
      const uint32_t off = (uint32_t)(((int64_t)r * args.ldo + 4 * cq) * 4);
      old[c & 1][it] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, ok ? off : OOB, 0, 0));
    }
  };
  // EPI_DGLU: the gates in pre[0], the ups in pre[1], of one chunk (loaded while it is
  // staged; a second chunk's would not fit the registers).
  auto load_pairs = [&](int c) {
    const int r0 = row0(c), c0 = col0(c);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const __amdgpu_buffer_rsrc_t rs = make_rsrc(args.aux + (int64_t)r0 * args.ldo + (half ? args.N : 0) + c0);
#pragma unroll
      for (int it = 0; it < 8; ++it) {
        const int q = it * 64 + lane, r = q >> 3, cp = q & 7;
        const bool ok = r0 + r < args.M && c0 + 8 * cp < args.N;
        const uint32_t off = (uint32_t)(((int64_t)r * args.ldo + 8 * cp) * 2);
        pre[half][it] = __builtin_bit_cast(u16x8_t, __builtin_amdgcn_raw_buffer_load_b128(rs, ok ? off : OOB, 0, 0));
      }
    }
  };
  // EPI_DGLU32: all of them, eight float32 values of either in a lane's row.
  f32x4_t wide[2][is_dglu32(EPI) ? 16 : 1];
  auto load_wide_pairs = [&](int c) {
    const int r0 = row0(c), c0 = col0(c);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const __amdgpu_buffer_rsrc_t rs =
          make_rsrc(reinterpret_cast<const float*>(args.aux) + (int64_t)r0 * args.ldo + (half ? args.N : 0) + c0);
#pragma unroll
      for (int u = 0; u < (is_dglu32(EPI) ? 16 : 1); ++u) {
        const int q = (u >> 1) * 64 + lane, r = q >> 3, cp = q & 7;
        const bool ok = r0 + r < args.M && c0 + 8 * cp < args.N;
        const uint32_t off = (uint32_t)(((int64_t)r * args.ldo + 8 * cp + 4 * (u & 1)) * 4);
        wide[half][u] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, ok ? off : OOB, 0, 0));
      }
    }
  };
  auto load_pre = [&](int c) {
    const int r0 = row0(c), c0 = col0(c);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(args.aux + (int64_t)r0 * args.ldo + c0);
#pragma unroll
    for (int it = 0; it < 8; ++it) {
      const int q = it * 64 + lane, r = q >> 3, cp = q & 7;
      const bool ok = r0 + r < args.M && c0 + 8 * cp < args.N;  // N % 8 == 0: 8 columns in or out together
      const uint32_t off = (uint32_t)(((int64_t)r * args.ldo + 8 * cp) * 2);
      pre[c & 1][it] = __builtin_bit_cast(u16x8_t, __builtin_amdgcn_raw_buffer_load_b128(rs, ok ? off : OOB, 0, 0));
    }
  };
  // The loads stay where they are issued: a scheduling barrier after each batch
  // keeps the compiler from sinking them to their uses (one round trip each)
  // when registers run short.
  if (EPI == EPI_DGELU) load_pre(0);
  // (Paired launches hold two staged products: their running-sum loads are not
  // double-buffered, which leaves the registers that holds.)
  if (ACC && !PAIR) load_old(0);
  __builtin_amdgcn_sched_barrier(0);
  // FP8: the product of the operands' scales, which stage_chunk applies (taken
  // after the first loads are issued, so that the scales' load overlaps them).
  const float sc = FP8 ? scale_fn() : 1.0f;
#pragma unroll
  for (int ch = 0; ch < NC; ++ch) {
    const int h = ch % nh;  // used by the stores below through row_w + 64 * h
    const int col_c = col0(ch);
    if (ACC && PAIR) {
      load_old(ch);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (ACC && !PAIR && ch + 1 < NC) {
      load_old(ch + 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (is_dglu(EPI)) {
      if constexpr (is_dglu32(EPI)) load_wide_pairs(ch);
      else load_pairs(ch);
      __builtin_amdgcn_sched_barrier(0);
    }
    stage_chunk(ch, sc);
    if (PAIR) stage_chunk2(ch);
    if (EPI == EPI_DGELU && ch + 1 < NC) {
      load_pre(ch + 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (is_glu(EPI)) {
      // A staged row holds 32 gate values and the same pairs' 32 up values; a lane
      // finishes eight pairs of a row.
      const int64_t row = row_w + 64 * h;
      const __amdgpu_buffer_rsrc_t rh = make_rsrc(reinterpret_cast<uint16_t*>(args.out) + row * args.ldo + col_c);
      f32x4_t x[4][4];
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int q = it * 64 + lane, r = q >> 2, cp = q & 3;
#pragma unroll
        for (int v = 0; v < 4; ++v)
          x[it][v] = *reinterpret_cast<const f32x4_t*>(stage + r * ROW_B + (((8 * (v >> 1) + 2 * cp + (v & 1)) ^ (r & 15)) << 4));
      }
      __builtin_amdgcn_sched_barrier(0);  // the reads stay one batch
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int q = it * 64 + lane, r = q >> 2, cp = q & 3;
        const bool ok = row + r < args.M && col_c + 8 * cp < args.N;  // N % 8 == 0
        u16x8_t v;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = f32_to_bf16(act_f32<act_of_epi(EPI)>(x[it][e >> 2][e & 3]) * x[it][2 + (e >> 2)][e & 3]);
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), rh,
                                               ok ? (uint32_t)(((int64_t)r * args.ldo + 8 * cp) * 2) : OOB, 0, 0);
      }
      if (args.out2) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const __amdgpu_buffer_rsrc_t rp = make_rsrc(args.out2 + row * args.ldt + (half ? args.N : 0) + col_c);
#pragma unroll
          for (int it = 0; it < 4; ++it) {
            const int q = it * 64 + lane, r = q >> 2, cp = q & 3;
            const bool ok = row + r < args.M && col_c + 8 * cp < args.N;
            u16x8_t v;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = f32_to_bf16(x[it][2 * half + (e >> 2)][e & 3]);
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), rp,
                                                   ok ? (uint32_t)(((int64_t)r * args.ldt + 8 * cp) * 2) : OOB, 0, 0);
          }
        }
      }
    } else if (EPI == EPI_F32 || ACC || PAIR) {
      const bool keep = EPI == EPI_F32 && !FP8 && args.aux;        // the next launch reads it
      const bool final_out = args.k_split >= args.K && !keep;      // nor a split-K slice
      const __amdgpu_buffer_rsrc_t rs = make_rsrc(reinterpret_cast<float*>(args.out) +
                                                  (int64_t)split * args.split_stride +
                                                  (int64_t)(row_w + 64 * h) * args.ldo + col_c);
      // Two batches of 8 vectors: with both running-sum buffers live, 16 would
      // not fit beside the accumulators.
#pragma unroll
      for (int b8 = 0; b8 < 16; b8 += 8) {
        f32x4_t xs[8], ys[PAIR ? 8 : 1];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int q = (b8 + u) * 64 + lane, r = q >> 4, c = q & 15;
          xs[u] = *reinterpret_cast<const f32x4_t*>(stage + r * ROW_B + ((c ^ (r & 15)) << 4));
          if constexpr (PAIR) ys[u] = *reinterpret_cast<const f32x4_t*>(stage2 + r * ROW_B + ((c ^ (r & 15)) << 4));
        }
        __builtin_amdgcn_sched_barrier(0);  // the reads stay one batch
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int it = b8 + u, q = it * 64 + lane, r = q >> 4, c = q & 15;
          const bool ok = row_w + 64 * h + r < args.M && col_c + 4 * c < args.N;
          if (ACC) xs[u] += old[ch & 1][it];
          if constexpr (PAIR) xs[u] += ys[u];
          const uint32_t off = (uint32_t)(((int64_t)r * args.ldo + 4 * c) * 4);
          if (final_out)  // non-temporal: a final output is not read again by this launch
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, xs[u]), rs, ok ? off : OOB, 0, 2);
          else
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, xs[u]), rs, ok ? off : OOB, 0, 0);
        }
      }
    } else {
      const int64_t base = (int64_t)(row_w + 64 * h) * args.ldo + col_c;
      const __amdgpu_buffer_rsrc_t rs = make_rsrc(reinterpret_cast<uint16_t*>(args.out) + base);
      // EPI_DGLU32's pairs leave registers for half of the chunk's values at a time: rows 0 .. 31, whose
      // h (below) takes the bytes of rows 0 .. 15, then rows 32 .. 63.
      constexpr int BATCH = is_dglu32(EPI) ? 4 : 8;
#pragma unroll
      for (int b = 0; b < 8; b += BATCH) {
        f32x4_t x0s[BATCH], x1s[BATCH];
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
          const int q = (b + u) * 64 + lane, r = q >> 3, cp = q & 7;
          x0s[u] = *reinterpret_cast<const f32x4_t*>(stage + r * ROW_B + (((2 * cp) ^ (r & 15)) << 4));
          x1s[u] = *reinterpret_cast<const f32x4_t*>(stage + r * ROW_B + (((2 * cp + 1) ^ (r & 15)) << 4));
        }
        __builtin_amdgcn_sched_barrier(0);  // the reads stay one batch
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
          const int it = b + u, q = it * 64 + lane, r = q >> 3, cp = q & 7;
          const float x[8] = {x0s[u][0], x0s[u][1], x0s[u][2], x0s[u][3],
                              x1s[u][0], x1s[u][1], x1s[u][2], x1s[u][3]};
          const bool ok = row_w + 64 * h + r < args.M && col_c + 8 * cp < args.N;  // N % 8 == 0
          const uint32_t off = ok ? (uint32_t)(((int64_t)r * args.ldo + 8 * cp) * 2) : OOB;
          auto store = [&](const __amdgpu_buffer_rsrc_t& rd, const u16x8_t& v) {
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), rd, off, 0, 0);
          };
          u16x8_t v1, v2;
          if (EPI == EPI_GELU) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              v1[e] = epi_gelu(x[e]);
              v2[e] = f32_to_bf16(x[e]);
            }
            store(rs, v1);
            if (args.out2) store(make_rsrc(args.out2 + base), v2);
          } else if (EPI == EPI_BF16) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v1[e] = f32_to_bf16(x[e]);
            store(rs, v1);
            if (FP8) {
#pragma unroll
              for (int e = 0; e < 8; ++e) am.add(ok ? bf16_to_f32(v1[e]) : 0.0f);
            }
          } else if constexpr (is_dglu(EPI)) {
            u16x8_t v3;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float g, up, a, da;
              if constexpr (is_dglu32(EPI)) {
                g = wide[0][2 * it + (e >> 2)][e & 3];
                up = wide[1][2 * it + (e >> 2)][e & 3];
              } else {
                g = bf16_to_f32(pre[0][it][e]);
                up = bf16_to_f32(pre[1][it][e]);
              }
              act_grad_f32<act_of_epi(EPI)>(g, a, da);
              v1[e] = f32_to_bf16(x[e] * up * da);
              v3[e] = f32_to_bf16(x[e] * a);
              v2[e] = f32_to_bf16(a * up);
            }
            store(rs, v1);
            store(make_rsrc(reinterpret_cast<uint16_t*>(args.out) + base + args.N), v3);
            // G of this row over the chunk's float32 values, as for EPI_DGELU below
            *reinterpret_cast<u16x8_t*>(stage + r * G_ROW_B + ((cp ^ gt_swz(r)) << 4)) = v2;
          } else if (FP8) {  // EPI_DGELU of an FP8 product: dP and its amax
#pragma unroll
            for (int e = 0; e < 8; ++e) v1[e] = f32_to_bf16(dgelu_f32(x[e], pre[ch & 1][it][e]));
            store(rs, v1);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float v = ok ? bf16_to_f32(v1[e]) : 0.0f;
              am.v_max = fmaxf(am.v_max, v);
              am.v_min = fminf(am.v_min, v);
            }
          } else {  // EPI_DGELU
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const DGelu d = epi_dgelu(x[e], pre[ch & 1][it][e]);
              v1[e] = d.dp;
              v2[e] = d.g;
            }
            store(rs, v1);
            // Keep G of this row in LDS, over the chunk's float32 values (the
            // wave has read all of them above, and its LDS accesses complete in
            // order), at G_ROW_B pitch, 16-byte chunks swizzled by the row
            // (gt_swz).  Rows and columns outside the output hold values that no
            // transposed store below reads.
            *reinterpret_cast<u16x8_t*>(stage + r * G_ROW_B + ((cp ^ gt_swz(r)) << 4)) = v2;
          }
        }
      }
      if ((EPI == EPI_DGELU && !FP8) || is_dglu(EPI)) {
        // Transposed store of G in whole 128-byte lines.  ds_read_b64_tr_b16
        // takes, in each 16-lane group, 4 rows x 16 columns (source lane 4 r + q:
        // row r, columns 4 q .. +3) and hands lane i column i.  Source lane
        // 4 r + q reads the 4 columns 8 it + 4 (g % 2) .. +3 of G row
        // m0(q) + r, with m0(q) = 32 (g / 2) + 8 q, so lane 4 q + e receives
        // rows m0(q) .. +3 of column 8 it + 4 (g % 2) + e; a second read gives
        // rows +4 .. +7.  The 8 lanes (g / 2, q) of a column then hold its 64
        // rows: one store instruction writes 8 columns x 128 bytes of G^T.  All
        // eight steps are read first, then stored.
        const int g = lane >> 4, j = lane & 15, jq = j & 3, jr = j >> 2;
        const int half = (g & 1) ? 8 : 0;
        i16x4_t lo[8], hi[8];
#pragma unroll
        for (int it = 0; it < 8; ++it) {
          const int ka = 32 * (g >> 1) + 8 * jq + jr, kb = ka + 4;  // source role: q = jq, r = jr
          lo[it] = ds_read_tr_lds(stage + ka * G_ROW_B + ((it ^ gt_swz(ka)) << 4) + half);
          hi[it] = ds_read_tr_lds(stage + kb * G_ROW_B + ((it ^ gt_swz(kb)) << 4) + half);
        }
        const int m0 = row_w + 64 * h;
        const __amdgpu_buffer_rsrc_t rt = make_rsrc(args.out2 + (int64_t)col_c * args.ldt + m0);
#pragma unroll
        for (int it = 0; it < 8; ++it) {
          // destination role: lane 4 q + e with q = jr, e = jq
          const int fo = 8 * it + 4 * (g & 1) + jq, mo = 32 * (g >> 1) + 8 * jr;
          const bool ok = col_c + fo < args.N && m0 + mo < args.M;
          const uint32_t off = (uint32_t)(((int64_t)fo * args.ldt + mo) * 2);
          const u16x8_t v = {(uint16_t)lo[it][0], (uint16_t)lo[it][1], (uint16_t)lo[it][2], (uint16_t)lo[it][3],
                             (uint16_t)hi[it][0], (uint16_t)hi[it][1], (uint16_t)hi[it][2], (uint16_t)hi[it][3]};
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), rt, ok ? off : OOB, 0, 0);
        }
      }
    }
  }
  if (FP8 && (EPI == EPI_BF16 || EPI == EPI_DGELU) && args.amax_out)
    slot_max(args.amax_out, AMAX_SUB, am.result(EPI == EPI_BF16 && args.amax_gelu));
}

}  // namespace

// The kernel has external linkage (a kernel template in an anonymous namespace
// does not get its host launch stubs emitted for every instantiation).
namespace kern {

// BM x BN tile (256 x 256, 256 x 128 or 128 x 128) on v_mfma_f32_16x16x32_bf16.
// The LDS is a ring of ten 16 KiB slots, each one 128-row (or 128-column)
// quarter of a K step (64): A's BM / 128 quarters, then B's BN / 128.  Wave (wm,
// wn) computes a (BM / 2) x (BN / 2) sub-tile as FI x FJ blocks of 16 x 16 (FI =
// BM / 32, FJ = BN / 32: 256, 128 or 64 accumulator registers).  A K step is two
// sub-steps of 32 k; in each a wave issues FI FJ MFMAs of 16 cycles and, between
// them, the LDS reads of the next sub-step's fragments and one batch of loads for
// step k+D (D = 2 for 256-row tiles, whose steps take four slots; D = 4 for 128 x
// 128, whose steps take two):
//   sub-step 0 of step k: the A quarters of step k+D (into slots of step k-1,
//         which no wave reads any more)
//   then: wait until the next sub-step's fragments are in registers and step k+1
//         has landed (vmcnt: only loads issued after step k+1's may be in
//         flight); barrier
//   sub-step 1 of step k: the B quarters of step k+D (256-row tiles: into step
//         k's first slots, which no wave reads after the barrier), and the reads
//         of step k+1's sub-step 0.
// The next sub-step's B fragments go to the other half of a double buffer; an A
// fragment is reloaded as soon as its row of MFMAs has been issued (MFMAs run
// row by row), so A needs no second buffer.  The deeper prefetch of the small
// tile covers memory latency over its shorter K steps (a quarter of the MFMAs).
//
// The body, gemm_x16.h, is workgroup `bid` of `nblocks` of the product args_in with the
// workgroup's LDS in `smem`.  It is included, not called: as a function, here or in
// gemm_group.hip's kernels, it takes other registers.
constexpr int LDS_BYTES = 160 * 1024;

template <int LB, int EPI, int BM, int BN, int F8>
__global__ void __launch_bounds__(256)
gemm_x16_kernel(GemmArgs args_in) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ __attribute__((aligned(1024))) char smem[LDS_BYTES];
  const int bid = blockIdx.x, nblocks = gridDim.x;
#include "gemm_x16.h"
#else
  (void)args_in;
#endif
}

}  // namespace kern

}  // namespace tpmlp
