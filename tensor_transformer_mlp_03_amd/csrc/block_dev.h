// Device helpers of the block operators: four-element loads and stores of float32
// and bf16 rows with element alignment, and sums over a wave or a workgroup.
#pragma once

#include "block.h"
#include "epilogue.h"

namespace tpmlp {

// Vectors that only need their element's alignment: rows may start at any element
// (odd row strides, column blocks, slices of a gradient bucket).  The compiler
// still moves them with one instruction; on aligned rows it costs nothing.
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint16_t u16x4_u __attribute__((ext_vector_type(4), aligned(2)));
typedef uint16_t u16x8_u __attribute__((ext_vector_type(8), aligned(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Storage types of a row.
struct F32 {
  typedef float elem;
  typedef f32x4_u vec;
};
struct BF16 {
  typedef uint16_t elem;
  typedef u16x4_u vec;
};

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(uint16_t v) { return bf16_to_f32(v); }
__device__ __forceinline__ f32x4 widen(f32x4_u v) { return f32x4{v[0], v[1], v[2], v[3]}; }
__device__ __forceinline__ f32x4 widen(u16x4_u v) {
  return f32x4{bf16_to_f32(v[0]), bf16_to_f32(v[1]), bf16_to_f32(v[2]), bf16_to_f32(v[3])};
}

__device__ __forceinline__ void put(float* p, f32x4 v) { *reinterpret_cast<f32x4_u*>(p) = f32x4_u{v[0], v[1], v[2], v[3]}; }
__device__ __forceinline__ void put(uint16_t* p, f32x4 v) {
  *reinterpret_cast<u16x4_u*>(p) = u16x4_u{f32_to_bf16(v[0]), f32_to_bf16(v[1]), f32_to_bf16(v[2]), f32_to_bf16(v[3])};
}
__device__ __forceinline__ void put1(float* p, float v) { *p = v; }
__device__ __forceinline__ void put1(uint16_t* p, float v) { *p = f32_to_bf16(v); }

// Elements i .. i+3 of a row of n >= 4 elements, zeros past its end.  Every lane
// reads four elements inside the row (the last four where i + 4 > n), so no lane
// branches around the load; a lane on the ragged end shifts what it read.
template <class T>
__device__ __forceinline__ f32x4 load4(const typename T::elem* row, int i, int n) {
  const int at = min(i, n - 4);
  f32x4 v = widen(*reinterpret_cast<const typename T::vec*>(row + at));
  if (i > at) {
    const int s = i - at;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    if (s == 1) o = f32x4{v[1], v[2], v[3], 0.0f};
    if (s == 2) o = f32x4{v[2], v[3], 0.0f, 0.0f};
    if (s == 3) o = f32x4{v[3], 0.0f, 0.0f, 0.0f};
    v = o;
  }
  return v;
}

// Stores elements i .. i+3 of a row of n elements, those inside it.
template <class T>
__device__ __forceinline__ void store4(typename T::elem* row, int i, int n, f32x4 v) {
  if (i + 4 <= n) {
    put(row + i, v);
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (i + e < n) put1(row + i + e, v[e]);
  }
}

// A row that a wave reads or writes four elements a lane.  FULL rows (n a multiple
// of 4, every row at a multiple of four elements) go through a buffer descriptor
// of the row's length: a chunk past the end reads zeros and writes nothing, without
// a branch or an address select, and the address is one 32-bit offset a lane.  The
// row's pointer has to be uniform over the wave.  Other rows take load4 and store4.
template <class T, bool FULL>
struct Row;

template <class T>
struct Row<T, false> {
  typedef typename T::elem elem;
  elem* p;
  int n;
  __device__ __forceinline__ Row(const void* base, int64_t at, int n_)
      : p(const_cast<elem*>(static_cast<const elem*>(base)) + at), n(n_) {}
  __device__ __forceinline__ f32x4 load(int i) const { return load4<T>(p, i, n); }
  __device__ __forceinline__ void store(int i, f32x4 v) const { store4<T>(p, i, n, v); }
};

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

#if defined(__HIP_DEVICE_COMPILE__)
template <class T>
struct Row<T, true> {
  __amdgpu_buffer_rsrc_t rs;
  __device__ __forceinline__ Row(const void* base, int64_t at, int n)
      : rs(__builtin_amdgcn_make_buffer_rsrc(
            const_cast<typename T::elem*>(static_cast<const typename T::elem*>(base)) + at, (short)0,
            (int)(n * sizeof(typename T::elem)), 0x00020000)) {}
  __device__ __forceinline__ f32x4 load(int i) const {
    if constexpr (sizeof(typename T::elem) == 4) {
      return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, i * 4, 0, 0));
    } else {
      const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rs, i * 2, 0, 0));
      return f32x4{__builtin_bit_cast(float, v[0] << 16), __builtin_bit_cast(float, v[0] & 0xFFFF0000u),
                   __builtin_bit_cast(float, v[1] << 16), __builtin_bit_cast(float, v[1] & 0xFFFF0000u)};
    }
  }
  __device__ __forceinline__ void store(int i, f32x4 v) const {
    if constexpr (sizeof(typename T::elem) == 4) {
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rs, i * 4, 0, 0);
    } else {
      const u32x2 o = {(uint32_t)f32_to_bf16(v[0]) | (uint32_t)f32_to_bf16(v[1]) << 16,
                       (uint32_t)f32_to_bf16(v[2]) | (uint32_t)f32_to_bf16(v[3]) << 16};
      __builtin_amdgcn_raw_buffer_store_b64(o, rs, i * 2, 0, 0);
    }
  }
};
#else
template <class T>
struct Row<T, true> : Row<T, false> {
  using Row<T, false>::Row;
};
#endif

// Parameter vectors are float32 or bf16 by a flag uniform over the launch.
template <bool FULL>
__device__ __forceinline__ f32x4 load_params(const void* p, int bf16, int64_t at, int i, int n) {
  return bf16 ? Row<BF16, FULL>(p, at, n).load(i) : Row<F32, FULL>(p, at, n).load(i);
}
__device__ __forceinline__ float load_param(const void* p, int bf16, int64_t i) {
  return bf16 ? bf16_to_f32(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// Sums N values over the W waves that share a row, each lane receiving all of
// them, in an order that depends on W alone.  `slot`: N * W floats of LDS that no
// other sum uses before every wave has passed one more barrier.
template <int W, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* slot, int wave) {
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = wave_sum(v[j]);
  if (W == 1) return;
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int j = 0; j < N; ++j) slot[j * W + wave] = v[j];
  __syncthreads();
#pragma unroll
  for (int j = 0; j < N; ++j) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) t += slot[j * W + w];
    v[j] = t;
  }
}

}  // namespace tpmlp
