// Dropout of a block's output with its bias, added to the residual stream, and its gradients:
//
//   out = r + m (.) (y + b) / (1 - p),    dy = m (.) dout / (1 - p),    db = sum over rows of dy
//
// m[i, j] is 1 where the 16-bit random number of the element is at least 65536 p, rounded,
// and the scale is that of the rounded p.  (Dropout behind the row-parallel product, before
// the residual's addition: QLM page §2.1.2.2 and §2.1.3.)  The mask is never stored: the
// number is a function of a seed, a step, a site and the element's row and column, so a
// backward makes it again, and ranks that hold row slices of one tensor agree on it.
//
// Numbers: Philox 4x32 with ten rounds (J. Salmon, M. Moraes, R. Dror, D. Shaw, Parallel
// random numbers: as easy as 1, 2, 3, SC 2011), key = the seed's halves, counter = (column /
// 8, row, site, step).  Its four words are the numbers of eight columns, low half first:
// 16 bits an element, which round p to 1 / 65536, instead of 32 halve the arithmetic.
//
// Bound by bandwidth: 2048 x 20480 with a float32 y and a bf16 stream 59.5 us, 5.6 TB/s; with
// one round of Philox instead of ten 59 (its multiplications run below the loads).  dy and
// db of 4096 x 1024 9.9 us, 25 MB in two launches.

#include "block_dev.h"
#include "gated.h"

#include <algorithm>

namespace tpmlp {
namespace {

// The eight numbers of columns 8 g .. 8 g + 7 of a row, two a word.
__device__ __forceinline__ u32x4 philox(uint32_t g, uint32_t row, uint32_t site, uint32_t step, uint64_t seed) {
  uint32_t c0 = g, c1 = row, c2 = site, c3 = step;
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u, p1 = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)p1;
    c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)p0;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{c0, c1, c2, c3};
}

__device__ __forceinline__ uint32_t number(u32x4 w, int e) { return e & 1 ? w[e >> 1] >> 16 : w[e >> 1] & 0xFFFFu; }

// Eight elements of a row from column c on: FULL rows by aligned vectors, others by vectors at any
// element, but for the row's last few.
template <class T, bool FULL, bool NT>
__device__ __forceinline__ void load8(const void* base, int64_t at, int c, int n, float (&v)[8]) {
  const typename T::elem* p = static_cast<const typename T::elem*>(base) + at + c;
  if constexpr (FULL) {
    if constexpr (sizeof(typename T::elem) == 4) {
      const f32x4* q = reinterpret_cast<const f32x4*>(p);
      const f32x4 a = NT ? __builtin_nontemporal_load(q) : q[0], b = NT ? __builtin_nontemporal_load(q + 1) : q[1];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = e < 4 ? a[e & 3] : b[e & 3];
    } else {
      const u32x4* q = reinterpret_cast<const u32x4*>(p);
      const u32x4 a = NT ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] = __builtin_bit_cast(float, e & 1 ? a[e >> 1] & 0xFFFF0000u : a[e >> 1] << 16);
    }
  } else if (c + 8 <= n) {  // at any element
    const typename T::vec* q = reinterpret_cast<const typename T::vec*>(p);
    const f32x4 a = widen(q[0]), b = widen(q[1]);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < 4 ? a[e & 3] : b[e & 3];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c + e < n ? widen(p[e]) : 0.0f;
  }
}

// NT32: float32 non-temporal, whose stores write every other 16 bytes: a lane's rows in turn
// (drop_bias_kernel) gain by it, dy of 2048 x 20480 64 -> 48.6 us, neighbouring items
// lose, 48 -> 54.
template <class T, bool FULL, bool NT, bool NT32>
__device__ __forceinline__ void store8(void* base, int64_t at, int c, int n, const float (&v)[8]) {
  typename T::elem* p = static_cast<typename T::elem*>(base) + at + c;
  if constexpr (FULL) {
    if constexpr (sizeof(typename T::elem) == 4) {
      f32x4* q = reinterpret_cast<f32x4*>(p);
      const f32x4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
      if (NT32) {
        __builtin_nontemporal_store(a, q);
        __builtin_nontemporal_store(b, q + 1);
      } else {
        q[0] = a;
        q[1] = b;
      }
    } else {
      u32x4 a;
#pragma unroll
      for (int e = 0; e < 4; ++e) a[e] = (uint32_t)f32_to_bf16(v[2 * e]) | (uint32_t)f32_to_bf16(v[2 * e + 1]) << 16;
      u32x4* q = reinterpret_cast<u32x4*>(p);
      if (NT) __builtin_nontemporal_store(a, q);
      else *q = a;
    }
  } else if (c + 8 <= n) {
    put(p, f32x4{v[0], v[1], v[2], v[3]});
    put(p + 4, f32x4{v[4], v[5], v[6], v[7]});
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < n) put1(p + e, v[e]);
  }
}

constexpr int DROP_ITEMS = 2;  // groups of eight columns a lane

// One group of eight columns of a row a lane and item; first_row + row is the row that the
// numbers go by.
template <class YT, class RT, bool FULL, bool NT>
__global__ void __launch_bounds__(256) drop_kernel(DropArgs a) {
  const uint64_t seed = a.state[0];
  const uint32_t step = (uint32_t)a.state[1];
  const uint32_t items = (uint32_t)(a.M * a.groups);
  const uint32_t first = blockIdx.x * (256u * DROP_ITEMS) + threadIdx.x;
  float y[DROP_ITEMS][8], r[DROP_ITEMS][8];
  uint32_t row[DROP_ITEMS];
  int c[DROP_ITEMS];
#pragma unroll
  for (int u = 0; u < DROP_ITEMS; ++u) {
    const uint32_t i = min(first + 256u * u, items - 1);
    row[u] = i / (uint32_t)a.groups;
    c[u] = 8 * (int)(i - row[u] * (uint32_t)a.groups);
    load8<YT, FULL, NT>(a.y, row[u] * a.ld_y, c[u], a.H, y[u]);
    if (a.r) load8<RT, FULL, NT>(a.r, row[u] * a.ld_r, c[u], a.H, r[u]);
  }
#pragma unroll
  for (int u = 0; u < DROP_ITEMS; ++u) {
    if (first + 256u * u >= items) break;
    const u32x4 w = philox((uint32_t)c[u] / 8, (uint32_t)(a.first_row + row[u]), a.site, step, seed);
    if (a.bias) {
      float b[8];
      if (a.bias_bf16) load8<BF16, FULL, false>(a.bias, 0, c[u], a.H, b);
      else load8<F32, FULL, false>(a.bias, 0, c[u], a.H, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[u][e] += b[e];
    }
    float o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float kept = number(w, e) >= a.drop ? y[u][e] * a.scale : 0.0f;
      o[e] = a.r ? r[u][e] + kept : kept;
    }
    store8<RT, FULL, NT, false>(a.out, row[u] * a.ld_out, c[u], a.H, o);
  }
}

// The backward with the bias's gradient: four waves share a stripe of 64 groups of columns
// (fewer, and several rows a wave, where a row has fewer) over chunk_rows rows, DROP_ROWS of
// a lane's rows loaded at a time; the sums of their unrounded dy meet in LDS.  The gradient is
// read without the non-temporal mark: 2048 x 20480 in bf16 43.5 us with it, 29.7 without.
constexpr int DROP_ROWS = 4;

template <class GT, class YT, bool FULL, bool NT>
__global__ void __launch_bounds__(256) drop_bias_kernel(DropArgs a) {
  __shared__ float sums[256][9];
  const uint64_t seed = a.state[0];
  const uint32_t step = (uint32_t)a.state[1];
  int width = 64;  // lanes of a row: uniform
  while (width / 2 >= a.groups) width /= 2;
  const int g = blockIdx.x * 64 + (threadIdx.x & (width - 1)), c = 8 * g;
  const int64_t end = min(a.M, (int64_t)(blockIdx.y + 1) * a.chunk_rows);
  const int step_rows = 256 / width;
  float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  if (g < a.groups) {
    for (int64_t row = blockIdx.y * a.chunk_rows + threadIdx.x / width; row < end; row += DROP_ROWS * step_rows) {
      float v[DROP_ROWS][8];
#pragma unroll
      for (int u = 0; u < DROP_ROWS; ++u) load8<GT, FULL, false>(a.y, min(row + u * step_rows, end - 1) * a.ld_y, c, a.H, v[u]);
#pragma unroll
      for (int u = 0; u < DROP_ROWS; ++u) {
        const int64_t r = row + u * step_rows;
        if (r >= end) break;
        const u32x4 w = philox((uint32_t)g, (uint32_t)(a.first_row + r), a.site, step, seed);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[u][e] = number(w, e) >= a.drop ? v[u][e] * a.scale : 0.0f;
          s[e] += v[u][e];
        }
        store8<YT, FULL, NT, NT>(a.out, r * a.ld_out, c, a.H, v[u]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) sums[threadIdx.x][e] = s[e];
  __syncthreads();
  for (int i = threadIdx.x; i < width * 8; i += 256) {
    const int lane = i >> 3, e = i & 7, col = 8 * (blockIdx.x * 64 + lane) + e;
    float t = 0.0f;
    for (int k = 0; k < step_rows; ++k) t += sums[k * width + lane][e];
    if (col < a.H) a.part[blockIdx.y * (int64_t)a.H + col] = t;
  }
}

// db[j] = sum over chunks of part[chunk][j]: 16 columns a workgroup, 16 runs of chunks each,
// eight loads at a time.
__global__ void __launch_bounds__(256) drop_sum_kernel(DropSumArgs a) {
  __shared__ float sums[16][17];
  const int c = threadIdx.x & 15, k = threadIdx.x >> 4, col = blockIdx.x * 16 + c;
  float s = 0.0f;
  if (col < a.H)
    for (int64_t i = k; i < a.chunks; i += 128) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = a.part[min(i + 16 * u, a.chunks - 1) * a.H + col];
#pragma unroll
      for (int u = 0; u < 8; ++u) s += i + 16 * u < a.chunks ? v[u] : 0.0f;
    }
  sums[k][c] = s;
  __syncthreads();
  if (k == 0 && col < a.H) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += sums[i][c];
    a.db[col] = t;
  }
}

template <class Y, class O>
hipError_t drop_form(const DropArgs& a, bool full, hipStream_t s) {
  const uint32_t blocks = (uint32_t)((a.M * a.groups + 256 * DROP_ITEMS - 1) / (256 * DROP_ITEMS));
  if (!full) return launch_kernel(drop_kernel<Y, O, false, false>, dim3(blocks), dim3(256), s, a);
  return launch_kernel(a.nt ? drop_kernel<Y, O, true, true> : drop_kernel<Y, O, true, false>, dim3(blocks), dim3(256), s, a);
}

template <class G, class Y>
hipError_t bias_form(const DropArgs& a, const DropPlan& p, bool full, hipStream_t s) {
  const dim3 grid((unsigned)((a.groups + 63) / 64), (unsigned)p.chunks);
  if (!full) return launch_kernel(drop_bias_kernel<G, Y, false, false>, grid, dim3(256), s, a);
  return launch_kernel(a.nt ? drop_bias_kernel<G, Y, true, true> : drop_bias_kernel<G, Y, true, false>, grid, dim3(256), s, a);
}

#define BY_TYPES(form, yt, ot, ...)                                                                       \
  (yt == TPMLP_BF16 ? (ot == TPMLP_BF16 ? form<BF16, BF16>(__VA_ARGS__) : form<BF16, F32>(__VA_ARGS__)) \
                    : (ot == TPMLP_BF16 ? form<F32, BF16>(__VA_ARGS__) : form<F32, F32>(__VA_ARGS__)))

const char* advance(const void* p, int64_t elems, int type) {
  return p ? static_cast<const char*>(p) + elems * (type == TPMLP_BF16 ? 2 : 4) : nullptr;
}

}  // namespace

DropPlan plan_drop(int64_t M, int64_t H) {
  // About 512 workgroups, of at least 16 rows each; a chunk's sums cost H floats both ways.
  const int64_t stripes = (H + 511) / 512;
  const int64_t want = std::max<int64_t>(1, 512 / stripes);
  DropPlan p;
  p.chunk_rows = std::max<int64_t>(16, (M + want - 1) / want);
  p.chunks = std::max<int64_t>(1, (M + p.chunk_rows - 1) / p.chunk_rows);
  p.ws_bytes = size_t(p.chunks) * H * sizeof(float);
  return p;
}

hipError_t launch_drop(DropArgs a, int y_type, int out_type, bool full, hipStream_t s) {
  // Items of one launch are counted in 31 bits.
  const int64_t most = std::max<int64_t>(1, (int64_t(1) << 31) / a.groups - 1);
  const int64_t M = a.M;
  for (int64_t row = 0; row < M; row += most) {
    DropArgs b = a;
    b.M = std::min(most, M - row);
    b.first_row = a.first_row + row;
    b.y = advance(a.y, row * a.ld_y, y_type);
    b.r = advance(a.r, row * a.ld_r, out_type);
    b.out = const_cast<char*>(advance(a.out, row * a.ld_out, out_type));
    const hipError_t e = BY_TYPES(drop_form, y_type, out_type, b, full, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_drop_bias(const DropArgs& a, const DropPlan& p, float* db, int y_type, int out_type, bool full, hipStream_t s) {
  const hipError_t e = BY_TYPES(bias_form, y_type, out_type, a, p, full, s);
  if (e != hipSuccess) return e;
  const DropSumArgs f{a.part, db, p.chunks, a.H};
  return launch_kernel(drop_sum_kernel, dim3((unsigned)((a.H + 15) / 16)), dim3(256), s, f);
}

}  // namespace tpmlp
