// Tokens sorted by expert and brought back.
//
// Token t chooses K experts; its choice k is pair p = t K + k.  Sorting is stable
// (pairs of one expert keep their order), every expert's segment of the sorted
// buffers starts at a multiple of `align` rows (the MLP's token counts are
// multiples of 8), and rows that no pair fills are padding:
//
//   row_of[p]: the sorted row of pair p, -1 if dropped;  src_of[row]: the pair, -1 for padding
//   dispatch     Xs[row_of[p]] = X[p / K], zeros on padding
//   combine      Y[t] = sum_k w[t,k] Zs[row_of[t,k]]  (dispatch's gradient is this with w = 1)
//   its gradient dZs[row_of[p]] = w_p dY[p / K], zeros on padding;  dw_p = <dY[p / K], Zs[row_of[p]]>
//
// All three walk the tokens, not the sorted rows: a token's row is read (or
// written) once and its K sorted rows are whole-row accesses wherever they lie.
// A pair that was dropped is never loaded, so what a padding row holds (a NaN of
// the expert's product) reaches no output.

#include "block_dev.h"

namespace tpmlp {
namespace {

// ---------------------------------------------------------------------------
// Sort
// ---------------------------------------------------------------------------
constexpr int SORT_THREADS = 1024, SORT_WAVES = SORT_THREADS / 64;

// The pair's expert, or -1 where its id names none.
__device__ __forceinline__ int expert_of(const RouteSortArgs& a, int64_t p) {
  if (a.ids64) {
    const int64_t e = static_cast<const int64_t*>(a.ids)[p];
    return e >= 0 && e < a.E ? (int)e : -1;
  }
  const int32_t e = static_cast<const int32_t*>(a.ids)[p];
  return e >= 0 && e < a.E ? e : -1;
}

// Pairs of each expert in one workgroup's part.
__global__ void __launch_bounds__(SORT_THREADS) route_hist_kernel(RouteSortArgs a) {
  __shared__ int count[TPMLP_ROUTE_MAX_EXPERTS];
  for (int e = threadIdx.x; e < a.E; e += SORT_THREADS) count[e] = 0;
  __syncthreads();
  const int64_t p0 = (int64_t)blockIdx.x * a.per_block, p1 = min(p0 + a.per_block, a.pairs);
  for (int64_t p = p0 + threadIdx.x; p < p1; p += SORT_THREADS) {
    const int e = expert_of(a, p);
    if (e >= 0) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += SORT_THREADS) a.hist[(int64_t)blockIdx.x * a.E + e] = count[e];
}

// Lanes of the wave whose value equals this lane's (bits: enough for every value).
__device__ __forceinline__ uint64_t same_lanes(int v, int bits) {
  uint64_t m = ~uint64_t(0);
  for (int b = 0; b < bits; ++b) {
    const bool set = (v >> b) & 1;
    const uint64_t with = __ballot(set);
    m &= set ? with : ~with;
  }
  return m;
}

// Places one workgroup's pairs.  Each of its waves takes a contiguous run of them:
// first every wave counts its run, then the counts are turned into the row where
// the wave's first pair of each expert goes (the segment's start, plus the pairs of
// earlier workgroups, plus those of earlier waves), and the waves walk their runs
// 64 pairs at a time, a pair's place among equal experts of the 64 given by the
// lanes before it.  With one workgroup (ONE) there is no histogram to read.
template <bool ONE>
__global__ void __launch_bounds__(SORT_THREADS) route_place_kernel(RouteSortArgs a) {
  __shared__ int lds[(SORT_WAVES + 2) * TPMLP_ROUTE_MAX_EXPERTS + 1 + SORT_WAVES];
  const int E = a.E, tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  int* next = lds;                        // [waves][E]
  int* start = next + SORT_WAVES * E;     // [E + 1] first row of each segment
  int* total = start + E + 1;             // [E] pairs of each expert
  int* scan = total + E;                  // [waves] sums of the scan over experts
  for (int e = tid; e < SORT_WAVES * E; e += SORT_THREADS) next[e] = 0;
  __syncthreads();
  const int64_t p0 = (int64_t)blockIdx.x * a.per_block, p1 = min(p0 + a.per_block, a.pairs);
  const int64_t run = ((p1 - p0 + SORT_WAVES - 1) / SORT_WAVES + 63) / 64 * 64;
  const int64_t w0 = min(p0 + wave * run, p1), w1 = min(w0 + run, p1);
  for (int64_t p = w0 + lane; p < w1; p += 64) {
    const int e = expert_of(a, p);
    if (e >= 0) atomicAdd(&next[wave * E + e], 1);
  }
  __syncthreads();
  // Pairs of expert e in all workgroups and in those before this one.  E is at
  // most the workgroup's size, so a thread has one expert.
  const int e = tid;
  int all = 0, before = 0, mine = 0;
  if (e < E) {
    if (ONE) {
      for (int w = 0; w < SORT_WAVES; ++w) all += next[w * E + e];
    } else {
      for (int b = 0; b < a.blocks; ++b) {
        const int n = a.hist[(int64_t)b * E + e];
        all += n;
        before += b < (int)blockIdx.x ? n : 0;
      }
    }
    mine = a.capacity ? min(all, a.capacity) : all;
  }
  // Exclusive scan of the segment lengths over the experts.
  const int len = e < E ? (a.capacity ? a.capacity : (mine + a.align - 1) / a.align * a.align) : 0;
  int inc = len;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int up = __shfl_up(inc, off, 64);
    if (lane >= off) inc += up;
  }
  if (lane == 63) scan[wave] = inc;
  __syncthreads();
  int base = inc - len;
  for (int w = 0; w < wave; ++w) base += scan[w];
  if (e < E) {
    start[e] = base;
    if (e == E - 1) start[E] = base + len;
    total[e] = mine;
    int at = before;  // rank of the wave's first pair among the expert's
    for (int w = 0; w < SORT_WAVES; ++w) {
      const int n = next[w * E + e];
      next[w * E + e] = at;
      at += n;
    }
    if (blockIdx.x == 0) {
      a.counts[e] = mine;
      a.offsets[e] = base;
      if (e == E - 1) a.offsets[E] = base + len;
    }
  }
  __syncthreads();
  const int bits = 32 - __clz(E);  // of 0 .. E, E standing for a dropped pair
  for (int64_t p = w0 + lane; p - lane < w1; p += 64) {  // all lanes stay for the ballots
    const bool in = p < w1;
    const int id = in ? expert_of(a, p) : -1;
    const int key = id < 0 ? E : id;
    const uint64_t same = same_lanes(key, bits);
    if (!in) continue;
    int row = -1;
    if (id >= 0) {
      volatile int* at = next + wave * E + id;  // other lanes of the wave write it too
      const int first = *at, rank = first + __popcll(same & ((uint64_t(1) << lane) - 1));
      __builtin_amdgcn_wave_barrier();
      // The last lane of each expert moves its counter; a wave's LDS accesses are in order.
      if ((same >> lane) == 1) *at = first + __popcll(same);
      if (!a.capacity || rank < a.capacity) row = start[id] + rank;
      if (row >= a.rows) row = -1;
      if (row >= 0) a.src_of[row] = (int32_t)p;
    }
    a.row_of[p] = row;
  }
  // Padding: rows past a segment's pairs and past the last segment.
  const int64_t stride = (int64_t)gridDim.x * SORT_THREADS;
  for (int64_t r = (int64_t)blockIdx.x * SORT_THREADS + tid; r < a.rows; r += stride) {
    int lo = 0, hi = E;  // the last segment that starts at or before r (start[0] = 0)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= r) lo = mid;
      else hi = mid;
    }
    if (r >= start[E] || r - start[lo] >= total[lo]) a.src_of[r] = -1;
  }
}

// ---------------------------------------------------------------------------
// Dispatch, combine and their gradients
// ---------------------------------------------------------------------------
constexpr int DISPATCH_CHUNKS = 4;  // 512-element chunks of a row that a wave moves
constexpr int DISPATCH_COLS = 512 * DISPATCH_CHUNKS;

// Where the eight elements at i of a row of n >= 8 are read and written: a lane on
// the ragged end takes the row's last eight, which overlap its neighbour's with
// equal values.
__device__ __forceinline__ int at8(int i, int n) { return min(i, n - 8); }

// Zeros columns [c0, c1) of a row.
__device__ __forceinline__ void zero_cols(uint16_t* row, int c0, int c1, int n, int lane) {
  for (int i = c0 + 8 * lane; i < c1; i += 512) *reinterpret_cast<u16x8_u*>(row + at8(i, n)) = u16x8_u{0, 0, 0, 0, 0, 0, 0, 0};
}

__global__ void __launch_bounds__(256) route_dispatch_kernel(RouteDispatchArgs a) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int seg = (int)blockIdx.y, c0 = seg * DISPATCH_COLS, c1 = min(c0 + DISPATCH_COLS, a.H);
  if ((int)blockIdx.x >= a.token_blocks) {  // padding: 64 rows a wave
    const int64_t r0 = ((int64_t)((int)blockIdx.x - a.token_blocks) * 4 + wave) * 64;
    if (r0 >= a.rows) return;
    uint64_t pad = __ballot(r0 + lane < a.rows && a.src_of[r0 + lane] < 0);
    while (pad) {
      const int b = __ffsll((unsigned long long)pad) - 1;
      pad &= pad - 1;
      zero_cols(a.xs + (r0 + b) * a.ld_xs, c0, c1, a.H, lane);
    }
    return;
  }
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t >= a.T) return;
  const uint16_t* x = a.x + t * a.ld_x;
  u16x8_u v[DISPATCH_CHUNKS];
#pragma unroll
  for (int c = 0; c < DISPATCH_CHUNKS; ++c) v[c] = *reinterpret_cast<const u16x8_u*>(x + at8(c0 + c * 512 + 8 * lane, a.H));
  for (int k = 0; k < a.K; ++k) {
    const int row = a.row_of[t * a.K + k];
    if ((uint32_t)row >= (uint64_t)a.rows) continue;  // dropped
    uint16_t* o = a.xs + row * a.ld_xs;
#pragma unroll
    for (int c = 0; c < DISPATCH_CHUNKS; ++c) {
      const int i = c0 + c * 512 + 8 * lane;
      if (i < a.H) *reinterpret_cast<u16x8_u*>(o + at8(i, a.H)) = v[c];
    }
  }
}

constexpr int COMBINE_CHUNKS = 4;  // 256-element chunks of a row that a wave sums
constexpr int COMBINE_COLS = 256 * COMBINE_CHUNKS;

template <class ZT, class YT>
__global__ void __launch_bounds__(256) route_combine_kernel(RouteCombineArgs a) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t >= a.T) return;
  const int c0 = (int)blockIdx.y * COMBINE_COLS;
  f32x4 sum[COMBINE_CHUNKS];
#pragma unroll
  for (int c = 0; c < COMBINE_CHUNKS; ++c) sum[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int k = 0; k < a.K; ++k) {
    const int row = a.row_of[t * a.K + k];
    if ((uint32_t)row >= (uint64_t)a.rows) continue;
    const float w = a.w ? a.w[t * a.K + k] : 1.0f;
    const auto* z = static_cast<const typename ZT::elem*>(a.zs) + row * a.ld_zs;
#pragma unroll
    for (int c = 0; c < COMBINE_CHUNKS; ++c) {
      const f32x4 v = load4<ZT>(z, c0 + c * 256 + 4 * lane, a.H);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[c][e] = __builtin_fmaf(v[e], w, sum[c][e]);
    }
  }
  auto* y = static_cast<typename YT::elem*>(a.y) + t * a.ld_y;
#pragma unroll
  for (int c = 0; c < COMBINE_CHUNKS; ++c) store4<YT>(y, c0 + c * 256 + 4 * lane, a.H, sum[c]);
}

constexpr int BWD_PAIRS = 8;  // choices of one token handled together

template <class DT, class ZT>
__global__ void __launch_bounds__(256) route_combine_bwd_kernel(RouteCombineBwdArgs a) {
  __shared__ float dots[BWD_PAIRS][4];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  if ((int)blockIdx.x >= a.token_blocks) {  // padding rows of dZs: 64 a wave
    const int64_t r0 = ((int64_t)((int)blockIdx.x - a.token_blocks) * 4 + wave) * 64;
    if (r0 >= a.rows) return;
    uint64_t pad = __ballot(r0 + lane < a.rows && a.src_of[r0 + lane] < 0);
    while (pad) {
      const int b = __ffsll((unsigned long long)pad) - 1;
      pad &= pad - 1;
      zero_cols(a.dzs + (r0 + b) * a.ld_dzs, 0, a.H, a.H, lane);
    }
    return;
  }
  const int64_t t = blockIdx.x;
  const auto* dy = static_cast<const typename DT::elem*>(a.dy) + t * a.ld_dy;
  for (int k0 = 0; k0 < a.K; k0 += BWD_PAIRS) {
    const int n = min(BWD_PAIRS, a.K - k0);
    int row[BWD_PAIRS];
    float w[BWD_PAIRS], dot[BWD_PAIRS];
#pragma unroll
    for (int j = 0; j < BWD_PAIRS; ++j) {
      const int r = j < n ? a.row_of[t * a.K + k0 + j] : -1;
      row[j] = (uint32_t)r < (uint64_t)a.rows ? r : -1;
      w[j] = j < n && a.w ? a.w[t * a.K + k0 + j] : 1.0f;
      dot[j] = 0.0f;
    }
    for (int i = 4 * (int)threadIdx.x; i < a.H; i += 1024) {
      const f32x4 d = load4<DT>(dy, i, a.H);
#pragma unroll
      for (int j = 0; j < BWD_PAIRS; ++j) {
        if (row[j] < 0) continue;  // uniform over the workgroup
        if (a.dw) {
          const f32x4 z = load4<ZT>(static_cast<const typename ZT::elem*>(a.zs) + row[j] * a.ld_zs, i, a.H);
#pragma unroll
          for (int e = 0; e < 4; ++e) dot[j] = __builtin_fmaf(d[e], z[e], dot[j]);
        }
        if (a.dzs) store4<BF16>(a.dzs + row[j] * a.ld_dzs, i, a.H, d * w[j]);
      }
    }
    if (!a.dw) continue;
    __syncthreads();  // the sums of the eight choices before are read
#pragma unroll
    for (int j = 0; j < BWD_PAIRS; ++j) {
      const float s = wave_sum(dot[j]);
      if (lane == 0) dots[j][wave] = s;
    }
    __syncthreads();
    if ((int)threadIdx.x < n) {
      const float* s = dots[threadIdx.x];
      a.dw[t * a.K + k0 + threadIdx.x] = (s[0] + s[1]) + (s[2] + s[3]);
    }
  }
}

int blocks_of(int64_t n, int64_t per) { return (int)((n + per - 1) / per); }

}  // namespace

int64_t route_sort_blocks(int64_t pairs, int64_t* per_block) {
  // One workgroup sorts up to 4096 pairs by itself; larger sorts give each 2048.
  const int64_t per = pairs <= 4096 ? 4096 : 2048;
  *per_block = per;
  return pairs <= per ? 1 : (pairs + per - 1) / per;
}

hipError_t launch_route_sort(const RouteSortArgs& a, hipStream_t s) {
  if (a.E < 1 || a.E > TPMLP_ROUTE_MAX_EXPERTS || a.blocks < 1) return hipErrorInvalidValue;
  if (a.blocks == 1) return launch_kernel(route_place_kernel<true>, dim3(1), dim3(SORT_THREADS), s, a);
  hipError_t e = launch_kernel(route_hist_kernel, dim3((unsigned)a.blocks), dim3(SORT_THREADS), s, a);
  if (e != hipSuccess) return e;
  return launch_kernel(route_place_kernel<false>, dim3((unsigned)a.blocks), dim3(SORT_THREADS), s, a);
}

hipError_t launch_route_dispatch(RouteDispatchArgs a, hipStream_t s) {
  if (a.H < 8) return hipErrorInvalidValue;
  a.segments = blocks_of(a.H, DISPATCH_COLS);
  a.token_blocks = blocks_of(a.T, 4);
  const int64_t blocks = a.token_blocks + (a.rows + 255) / 256;
  if (blocks < 1 || blocks > INT32_MAX) return blocks < 1 ? hipSuccess : hipErrorInvalidValue;
  return launch_kernel(route_dispatch_kernel, dim3((unsigned)blocks, (unsigned)a.segments), dim3(256), s, a);
}

hipError_t launch_route_combine(RouteCombineArgs a, int z_type, int y_type, hipStream_t s) {
  if (a.H < 4 || a.T < 1) return hipErrorInvalidValue;
  a.segments = blocks_of(a.H, COMBINE_COLS);
  const dim3 grid((unsigned)blocks_of(a.T, 4), (unsigned)a.segments), block(256);
  if (z_type == TPMLP_BF16)
    return y_type == TPMLP_BF16 ? launch_kernel(route_combine_kernel<BF16, BF16>, grid, block, s, a)
                                : launch_kernel(route_combine_kernel<BF16, F32>, grid, block, s, a);
  return y_type == TPMLP_BF16 ? launch_kernel(route_combine_kernel<F32, BF16>, grid, block, s, a)
                              : launch_kernel(route_combine_kernel<F32, F32>, grid, block, s, a);
}

hipError_t launch_route_combine_bwd(RouteCombineBwdArgs a, int dy_type, int z_type, hipStream_t s) {
  if (a.H < 8) return hipErrorInvalidValue;
  a.token_blocks = (int)a.T;
  const int64_t blocks = a.T + (a.dzs ? (a.rows + 255) / 256 : 0);
  if (blocks < 1 || blocks > INT32_MAX) return blocks < 1 ? hipSuccess : hipErrorInvalidValue;
  const dim3 grid((unsigned)blocks), block(256);
  if (dy_type == TPMLP_BF16)
    return z_type == TPMLP_BF16 ? launch_kernel(route_combine_bwd_kernel<BF16, BF16>, grid, block, s, a)
                                : launch_kernel(route_combine_bwd_kernel<BF16, F32>, grid, block, s, a);
  return z_type == TPMLP_BF16 ? launch_kernel(route_combine_bwd_kernel<F32, BF16>, grid, block, s, a)
                              : launch_kernel(route_combine_bwd_kernel<F32, F32>, grid, block, s, a);
}

}  // namespace tpmlp
