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
// reads four elements inside the row (the last four, v, where i + 4 > n), so no lane
// branches around the load; a lane on the ragged end shifts what it read.
__device__ __forceinline__ f32x4 from4(f32x4 v, int i, int n) {
  if (i > n - 4) {
    const int s = i - (n - 4);
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
// row's pointer has to be uniform over the wave.  Other rows take from4 and store4.
// A row of length 0 reads zeros and touches no memory.  NT marks FULL rows' accesses
// as non-temporal, for launches that move more than BLOCK_NT_BYTES.
template <class T, bool FULL, bool NT = false>
struct Row;

template <class T, bool NT>
struct Row<T, false, NT> {
  typedef typename T::elem elem;
  typedef typename T::vec raw;  // four elements as loaded
  elem* p;
  int n;
  __device__ __forceinline__ Row(const void* base, int64_t at, int n_)
      : p(const_cast<elem*>(static_cast<const elem*>(base)) + at), n(n_) {}
  __device__ __forceinline__ raw load_raw(int i) const {
    if (n == 0) return raw{0, 0, 0, 0};  // uniform
    return *reinterpret_cast<const raw*>(p + min(i, n - 4));
  }
  // The conversion apart from the load, for a row that is fetched before it is used.
  static __device__ __forceinline__ f32x4 widen_raw(raw v, int i, int n) { return from4(widen(v), i, n); }
  __device__ __forceinline__ f32x4 load(int i) const { return widen_raw(load_raw(i), i, n); }
  __device__ __forceinline__ void store(int i, f32x4 v) const { store4<T>(p, i, n, v); }
};

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

#if defined(__HIP_DEVICE_COMPILE__)
template <class T, bool NT>
struct Row<T, true, NT> {
  static constexpr bool WIDE = sizeof(typename T::elem) == 4;
  static constexpr int AUX = NT ? 2 : 0;
  typedef uint32_t raw __attribute__((ext_vector_type(sizeof(typename T::elem))));
  __amdgpu_buffer_rsrc_t rs;
  __device__ __forceinline__ Row(const void* base, int64_t at, int n)
      : rs(__builtin_amdgcn_make_buffer_rsrc(
            const_cast<typename T::elem*>(static_cast<const typename T::elem*>(base)) + at, (short)0,
            (int)(n * sizeof(typename T::elem)), 0x00020000)) {}
  __device__ __forceinline__ raw load_raw(int i) const {
    if constexpr (WIDE)
      return __builtin_bit_cast(raw, __builtin_amdgcn_raw_buffer_load_b128(rs, i * 4, 0, AUX));
    else
      return __builtin_bit_cast(raw, __builtin_amdgcn_raw_buffer_load_b64(rs, i * 2, 0, AUX));
  }
  static __device__ __forceinline__ f32x4 widen_raw(raw v, int, int) {
    if constexpr (WIDE)
      return __builtin_bit_cast(f32x4, v);
    else
      return f32x4{__builtin_bit_cast(float, v[0] << 16), __builtin_bit_cast(float, v[0] & 0xFFFF0000u),
                   __builtin_bit_cast(float, v[1] << 16), __builtin_bit_cast(float, v[1] & 0xFFFF0000u)};
  }
  __device__ __forceinline__ f32x4 load(int i) const { return widen_raw(load_raw(i), i, 0); }
  __device__ __forceinline__ void store(int i, f32x4 v) const {
    if constexpr (WIDE) {
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rs, i * 4, 0, AUX);
    } else {
      const u32x2 o = {(uint32_t)f32_to_bf16(v[0]) | (uint32_t)f32_to_bf16(v[1]) << 16,
                       (uint32_t)f32_to_bf16(v[2]) | (uint32_t)f32_to_bf16(v[3]) << 16};
      __builtin_amdgcn_raw_buffer_store_b64(o, rs, i * 2, 0, AUX);
    }
  }
};
#else
template <class T, bool NT>
struct Row<T, true, NT> : Row<T, false, NT> {
  using Row<T, false, NT>::Row;
};
#endif

// NV chunks of a parameter vector that is float32 or bf16 by a flag uniform over the
// launch: loaded under the flag, converted later under the flag again, so that the
// loads of several vectors are in flight together.
template <int NV, bool FULL>
struct Params {
  typedef typename Row<F32, FULL>::raw raw32;
  typedef typename Row<BF16, FULL>::raw raw16;
  raw32 v[NV];  // bf16: the first half of each
  template <class At>
  __device__ __forceinline__ void fetch(const void* p, int bf16, int64_t at, At&& place, int n) {
    if (bf16) {
      const Row<BF16, FULL> m(p, at, n);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const raw16 t = m.load_raw(place(k));
        __builtin_memcpy(&v[k], &t, sizeof t);
      }
    } else {
      const Row<F32, FULL> m(p, at, n);
#pragma unroll
      for (int k = 0; k < NV; ++k) v[k] = m.load_raw(place(k));
    }
  }
  __device__ __forceinline__ f32x4 get(int k, int bf16, int i, int n) const {
    raw16 t;
    __builtin_memcpy(&t, &v[k], sizeof t);
    return bf16 ? Row<BF16, FULL>::widen_raw(t, i, n) : Row<F32, FULL>::widen_raw(v[k], i, n);
  }
};

// One chunk of such a vector.
template <bool FULL>
__device__ __forceinline__ f32x4 load_params(const void* p, int bf16, int64_t at, int i, int n) {
  return bf16 ? Row<BF16, FULL>(p, at, n).load(i) : Row<F32, FULL>(p, at, n).load(i);
}
__device__ __forceinline__ float load_param(const void* p, int bf16, int64_t i) {
  return bf16 ? bf16_to_f32(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

// Sum over the wave, on every lane, in the register file: within quads, the halves
// of a 16-lane row and its two halves by DPP moves, between rows by the swaps of
// gfx950.  No LDS access, whose latency six times over was most of a short row's time.
#if defined(__HIP_DEVICE_COMPILE__)
template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
  const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true);
  return v + __builtin_bit_cast(float, o);
}
__device__ __forceinline__ float wave_sum(float v) {
  v = add_dpp<0xB1>(v);   // quad_perm [1,0,3,2]
  v = add_dpp<0x4E>(v);   // quad_perm [2,3,0,1]
  v = add_dpp<0x141>(v);  // row_half_mirror: the other quad of eight lanes
  v = add_dpp<0x140>(v);  // row_mirror: the other eight lanes of the row
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  const auto rows = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  const uint32_t r0 = rows[0], r1 = rows[1];  // values: a bit cast of a vector's element would take its first
  v = __builtin_bit_cast(float, r0) + __builtin_bit_cast(float, r1);
  const uint32_t c = __builtin_bit_cast(uint32_t, v);
  const auto halves = __builtin_amdgcn_permlane32_swap(c, c, false, false);
  const uint32_t h0 = halves[0], h1 = halves[1];
  return __builtin_bit_cast(float, h0) + __builtin_bit_cast(float, h1);
}
#else
__device__ inline float wave_sum(float v) { return v; }
#endif

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// Sums N values over the W waves that share a row (W 1, 4, 8 or 16), every lane
// receiving all of them, in an order that depends on W alone.  Each wave's lanes read
// one of the N W wave sums each, add them within groups of W lanes and hand the sums
// to scalar registers, where they take no room of the rows'.  `slot`: N * W floats of
// LDS that no other sum uses before every wave has passed one more barrier.
template <int W, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* slot, int wave) {
#if defined(__HIP_DEVICE_COMPILE__)
  auto scalar = [](float x, int lane) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
  };
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = wave_sum(v[j]);
  if (W == 1) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = scalar(v[j], 0);
    return;
  }
  const int lane = threadIdx.x & 63;
  if (lane == 0)
#pragma unroll
    for (int j = 0; j < N; ++j) slot[j * W + wave] = v[j];
  __syncthreads();
  constexpr int PER = 64 / W;  // sums of one pass
#pragma unroll
  for (int j0 = 0; j0 < N; j0 += PER) {
    float x = slot[min(j0 * W + lane, N * W - 1)];
    x = add_dpp<0xB1>(x);
    x = add_dpp<0x4E>(x);
    if (W >= 8) x = add_dpp<0x141>(x);
    if (W >= 16) x = add_dpp<0x140>(x);
#pragma unroll
    for (int j = j0; j < N && j < j0 + PER; ++j) v[j] = scalar(x, (j - j0) * W);
  }
#endif
}

}  // namespace tpmlp
