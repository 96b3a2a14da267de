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
// without elements have no chunk).
__device__ __forceinline__ int tensor_of(const ClipArgs& a, uint32_t chunk) {
  int lo = 0, hi = a.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.first[mid] <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <class T>
__device__ __forceinline__ double chunk_sumsq(const typename T::elem* g, int n) {
  double s0 = 0.0, s1 = 0.0;
  int i = 4 * (int)threadIdx.x;
#pragma unroll 4
  for (; i + 4 <= n; i += 1024) {
    const f32x4 v = widen(*reinterpret_cast<const typename T::vec*>(g + i));
    s0 = __builtin_fma((double)v[0], (double)v[0], s0);
    s1 = __builtin_fma((double)v[1], (double)v[1], s1);
    s0 = __builtin_fma((double)v[2], (double)v[2], s0);
    s1 = __builtin_fma((double)v[3], (double)v[3], s1);
  }
  for (; i < n && i >= (n & ~3); ++i) {
    const double v = widen(g[i]);
    s0 = __builtin_fma(v, v, s0);
  }
  return s0 + s1;
}

__global__ void __launch_bounds__(256) clip_sumsq_kernel(ClipArgs a) {
  __shared__ double slot[4];
  double sum = 0.0;
  for (uint32_t c = blockIdx.x; c < a.first[a.n]; c += gridDim.x) {
    const int t = tensor_of(a, c);
    const int64_t at = (int64_t)(c - a.first[t]) * CLIP_CHUNK, size = a.size[t] & SIZE_MASK;
    const int n = (int)min(CLIP_CHUNK, size - at);
    sum += (a.size[t] >> 62) ? chunk_sumsq<BF16>(static_cast<const uint16_t*>(a.in[t]) + at, n)
                             : chunk_sumsq<F32>(static_cast<const float*>(a.in[t]) + at, n);
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
#pragma unroll 4
  for (; i + 4 <= n; i += 1024) put(o + i, widen(*reinterpret_cast<const typename T::vec*>(g + i)) * m);
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
  for (uint32_t c = blockIdx.x; c < a.first[a.n]; c += gridDim.x) {
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
