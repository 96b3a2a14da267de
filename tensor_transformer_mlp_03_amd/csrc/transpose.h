// The transposes' tile (reduce.hip), for kernels that transpose besides (gemm_group.hip).
#pragma once

#include "common.h"

namespace tpmlp {
namespace {

typedef uint32_t transpose_u32x4 __attribute__((ext_vector_type(4)));

// bf16 transpose, one 64 x 64 tile per wave.  Lane (rb, cb) = (lane / 8,
// lane % 8) loads the 8 x 8 block at rows 8*rb .. +7, columns 8*cb .. +7 of the
// tile (8 loads of 16 bytes: one instruction reads 8 rows x 128 bytes), turns
// it around in registers with v_perm_b32 and writes rows 8*cb .. +7 of the
// output tile, columns 8*rb .. +7 (one instruction writes 8 rows x 128 bytes).
// C is a multiple of 8 and, without PAD, R too, so a block is entirely inside or outside.
// The four waves of a workgroup take four consecutive row tiles of one column
// tile, and consecutive workgroups continue along the rows, so that the output
// rows (R * 2 bytes apart, often a power of two) are written in long runs
// rather than 64 rows at a time at one stride, which would load one memory
// channel.  One launch can transpose two matrices of the same shape (X and dZ
// before a backward): workgroups [0, blocks) take the first, [blocks, 2 blocks)
// the second.
struct TransposeArgs {
  const uint16_t* in[2];
  uint16_t* out[2];
  int64_t R, C;  // in is [R][C] (rows of ld_in elements), out is [C][R] (rows of ld_out)
  int64_t ld_in, ld_out;
  int row_groups;  // groups of four 64-row tiles
  int blocks;      // workgroups per matrix
};

// PAD: R need not be a multiple of 8; the output's rows are filled up to one with zeros.
template <bool PAD>
__device__ __forceinline__ void transpose_tile(const TransposeArgs& a, int block) {
#if defined(__HIP_DEVICE_COMPILE__)
  const int lane = threadIdx.x & 63;
  const int job = block >= a.blocks ? 1 : 0;  // uniform over the workgroup
  const int bid = block - job * a.blocks;
  const uint16_t* in = job ? a.in[1] : a.in[0];
  uint16_t* out = job ? a.out[1] : a.out[0];
  const int rg = bid % a.row_groups, ct = bid / a.row_groups;
  // The wave's 64 x 64 tile starts at (tr, tc); the buffer descriptor is built
  // from that wave-uniform origin (a per-lane base would not fit the scalar
  // descriptor and would serialize the loads).
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t tr = ((int64_t)rg * 4 + wave) * 64, tc = (int64_t)ct * 64;
  if (tr >= a.R) return;
  const int lr = 8 * (lane >> 3), lc = 8 * (lane & 7);
  const int64_t r0 = tr + lr, c0 = tc + lc;
  if (r0 >= a.R || c0 >= a.C) return;
  const __amdgpu_buffer_rsrc_t rs =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(in + tr * a.ld_in + tc), (short)0, 0x7FFFFFF0, 0x00020000);
  transpose_u32x4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t off = (uint32_t)(((lr + i) * a.ld_in + lc) * 2);
    if (PAD && r0 + i >= a.R) off = 0x7FFFFFF0u;  // past the descriptor: zeros
    v[i] = __builtin_bit_cast(transpose_u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
  }
  // Output row c0 + j takes element j of each of the 8 input rows: dword e
  // packs input rows 2e and 2e+1, i.e. the halves of v[2e] and v[2e+1] that
  // hold column j (low halves for even j, high halves for odd j).
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
    transpose_u32x4 o;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = __builtin_amdgcn_perm(v[2 * e + 1][j >> 1], v[2 * e][j >> 1], sel);
    *reinterpret_cast<transpose_u32x4*>(out + (c0 + j) * a.ld_out + r0) = o;
  }
#else
  (void)a;
#endif
}

}  // namespace

// The workgroups that transpose in[0] (and in[1], if there); 0 if the sizes are invalid.
inline int plan_transpose(TransposeArgs& a, const uint16_t* in0, uint16_t* out0, const uint16_t* in1, uint16_t* out1, int64_t R,
                          int64_t C, int64_t ld_in, int64_t ld_out) {
  if (ld_in < C || (ld_in & 7) || (C & 7) || ld_out < R || (ld_out & 7)) return 0;
  if (!in0 || !out0 || (in1 && !out1)) return 0;
  a.in[0] = in0;
  a.out[0] = out0;
  a.in[1] = in1;
  a.out[1] = out1;
  a.R = R;
  a.C = C;
  a.ld_in = ld_in;
  a.ld_out = ld_out;
  a.row_groups = (int)((R + 255) / 256);
  const int64_t blocks = (int64_t)a.row_groups * ((C + 63) / 64);
  const int jobs = in1 ? 2 : 1;
  if (blocks * jobs > INT32_MAX) return 0;
  a.blocks = (int)blocks;
  return (int)(blocks * jobs);
}

}  // namespace tpmlp
