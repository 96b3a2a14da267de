// The global norm of many gradients and their clipping:
//
//   norm = |scale| sqrt(sum g^2),  c = max_norm / norm if norm is finite and above max_norm, else 1,
//   out = g (scale c)
//
// The tensors are cut into chunks of CLIP_CHUNK elements, numbered through; a
// workgroup takes every gridDim-th chunk and finds its tensor in the table of the
// kernel's arguments.  Squares are summed in float64: a float32 gradient's square
// cannot overflow there, and the sum's rounding stays far below the float32 norm's.
// Every workgroup writes its own partial sum and the partials are added in their
// order, so the norm does not depend on timing.  A norm that is not finite leaves
// the gradients as they are (times scale): the caller sees it and skips the step.
//
// Bound by bandwidth: 420M float32 summed in 250 us (6.7 TB/s) and scaled into other
// buffers in 565 us (5.9 TB/s).  The summing pass marks its loads as non-temporal except
// for the last 256 MB, which the scaling pass begins with (857 us without the first,
// 861 without the second, 823 with both); 4096 to 16384 scaling workgroups are alike,
// 2048 are 2% slower.  60 small tensors: 4.1 + 4.6 us, latency.  Both hold within one launch
// of 128 tensors.  More tensors are several launches, each of which keeps its own last 256 MB
// and which scale in the order in which they summed, so that what the cache holds of the last
// is evicted by the first: 273M float32 in 260 tensors 552 us (5.9 TB/s of two reads and a
// write), 105M in 100 tensors 201 us (6.3).

#include "block_dev.h"

namespace tpmlp {
namespace {

constexpr int64_t SIZE_MASK = (int64_t(1) << 62) - 1;

__device__ __forceinline__ double block_sum(double v, double* slot) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
  __syncthreads();
  return (slot[0] + slot[1]) + (slot[2] + slot[3]);
}

// Tensor of a chunk: the last one whose first chunk is at or before it (tensors
// without elements have no chunk).  The table is in the kernel's arguments; two
// looks at neighbouring entries cost two loads' latency where a binary search costs
// seven.
__device__ __forceinline__ int tensor_of(const ClipArgs& a, uint32_t chunk) {
  int t = -1;
#pragma unroll
  for (int k = 0; k < CLIP_TENSORS / 8; ++k) t += a.eighth[k] <= chunk;
  t *= 8;
  int n = -1;
#pragma unroll
  for (int k = 0; k < 8; ++k) n += a.first[t + k] <= chunk;
  return t + n;
}

// Batches of four vectors a thread are loaded before the first is used.
template <class T, bool NT>
__device__ __forceinline__ typename T::vec load_vec(const typename T::elem* p) {
  const typename T::vec* v = reinterpret_cast<const typename T::vec*>(p);
  return NT ? __builtin_nontemporal_load(v) : *v;
}

template <class T, bool NT>
__device__ __forceinline__ double chunk_sumsq(const typename T::elem* g, int n) {
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  auto add = [&](f32x4 v) {
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = __builtin_fma((double)v[e], (double)v[e], s[e]);
  };
  int i = 4 * (int)threadIdx.x;
  for (; i + 3 * 1024 + 4 <= n; i += 4 * 1024) {
    typename T::vec v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = load_vec<T, NT>(g + i + k * 1024);
#pragma unroll
    for (int k = 0; k < 4; ++k) add(widen(v[k]));
  }
  for (; i + 4 <= n; i += 1024) add(widen(load_vec<T, false>(g + i)));
  for (; i < n && i >= (n & ~3); ++i) {
    const double v = widen(g[i]);
    s[0] = __builtin_fma(v, v, s[0]);
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

__global__ void __launch_bounds__(256) clip_sumsq_kernel(ClipArgs a) {
  __shared__ double slot[4];
  double sum = 0.0;
  for (uint32_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    const int t = tensor_of(a, c);
    const int64_t at = (int64_t)(c - a.first[t]) * CLIP_CHUNK, size = a.size[t] & SIZE_MASK;
    const int n = (int)min(CLIP_CHUNK, size - at);
    // What a second pass of one launch will still find in the Infinity Cache is read so as to stay there.
    const bool keep = c + CLIP_KEEP >= a.chunks;
    if (a.size[t] >> 62) {
      const uint16_t* g = static_cast<const uint16_t*>(a.in[t]) + at;
      sum += keep ? chunk_sumsq<BF16, false>(g, n) : chunk_sumsq<BF16, true>(g, n);
    } else {
      const float* g = static_cast<const float*>(a.in[t]) + at;
      sum += keep ? chunk_sumsq<F32, false>(g, n) : chunk_sumsq<F32, true>(g, n);
    }
  }
  sum = block_sum(sum, slot);
  if (threadIdx.x == 0) a.part[blockIdx.x] = sum;
}

struct ClipTotalArgs {
  const double* part;
  int n;
  double* total;
};

__device__ __forceinline__ double partials(const double* part, int n, double* slot) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += 256) s += part[i];
  return block_sum(s, slot);
}

__global__ void __launch_bounds__(256) clip_total_kernel(ClipTotalArgs a) {
  __shared__ double slot[4];
  const double s = partials(a.part, a.n, slot);
  if (threadIdx.x == 0) *a.total = s;
}

template <class T>
__device__ __forceinline__ void chunk_scale(const typename T::elem* g, typename T::elem* o, int n, float m) {
  int i = 4 * (int)threadIdx.x;
  for (; i + 3 * 1024 + 4 <= n; i += 4 * 1024) {
    typename T::vec v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = load_vec<T, true>(g + i + k * 1024);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const f32x4 x = widen(v[k]) * m;
      typename T::vec t;
      if constexpr (sizeof(typename T::elem) == 4) t = typename T::vec{x[0], x[1], x[2], x[3]};
      else t = typename T::vec{f32_to_bf16(x[0]), f32_to_bf16(x[1]), f32_to_bf16(x[2]), f32_to_bf16(x[3])};
      __builtin_nontemporal_store(t, reinterpret_cast<typename T::vec*>(o + i + k * 1024));
    }
  }
  for (; i + 4 <= n; i += 1024) put(o + i, widen(load_vec<T, false>(g + i)) * m);
  for (; i < n && i >= (n & ~3); ++i) put1(o + i, widen(g[i]) * m);
}

// Every workgroup adds the partials itself (at most CLIP_BLOCKS of them, from the
// L2), which saves the launch of a kernel that would.
__global__ void __launch_bounds__(256) clip_scale_kernel(ClipArgs a) {
  __shared__ double slot[4];
  const double total = partials(a.part, a.n_part, slot);
  const float norm = (float)(sqrt(total) * fabs((double)a.scale));
  const bool clip = norm > a.max_norm && norm <= 3.402823466e38f;
  const float m = clip ? (float)((double)a.scale * ((double)a.max_norm / (sqrt(total) * fabs((double)a.scale)))) : a.scale;
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.norm) *a.norm = norm;
  const uint32_t all = a.chunks;
  for (uint32_t k = blockIdx.x; k < all; k += gridDim.x) {
    const uint32_t c = all - 1 - k;  // last chunks first: of the last launch those are still in the Infinity Cache
    const int t = tensor_of(a, c);
    if (m == 1.0f && a.in[t] == a.out[t]) continue;  // in place and nothing to change
    const int64_t at = (int64_t)(c - a.first[t]) * CLIP_CHUNK, size = a.size[t] & SIZE_MASK;
    const int n = (int)min(CLIP_CHUNK, size - at);
    if (a.size[t] >> 62)
      chunk_scale<BF16>(static_cast<const uint16_t*>(a.in[t]) + at, static_cast<uint16_t*>(a.out[t]) + at, n, m);
    else
      chunk_scale<F32>(static_cast<const float*>(a.in[t]) + at, static_cast<float*>(a.out[t]) + at, n, m);
  }
}

}  // namespace

hipError_t launch_clip_sumsq(const ClipArgs& a, int blocks, hipStream_t s) {
  return launch_kernel(clip_sumsq_kernel, dim3((unsigned)blocks), dim3(256), s, a);
}
hipError_t launch_clip_total(const double* part, int n, double* total, hipStream_t s) {
  return launch_kernel(clip_total_kernel, dim3(1), dim3(256), s, ClipTotalArgs{part, n, total});
}
hipError_t launch_clip_scale(const ClipArgs& a, int blocks, hipStream_t s) {
  return launch_kernel(clip_scale_kernel, dim3((unsigned)blocks), dim3(256), s, a);
}

}  // namespace tpmlp
