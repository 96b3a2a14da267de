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
//
// The moves are bound by bandwidth: 32768 x 3584 to four experts each 234 us, 5.05 TB/s,
// four fifths of it scattered row writes; the gradient of 2048 x 4096 to eight each, of which
// a capacity keeps 12160 of 16384 pairs, 88 us for 401 MB (4.6 TB/s), and its way back
// (combine without weights) 43.5 us for 233 MB (5.4 TB/s).  The sort is bound by latency: 16
// pairs 3.7 us, 131072 pairs 5.0 + 7.6 us.

#include "block_dev.h"

#include <algorithm>

namespace tpmlp {
namespace {

// ---------------------------------------------------------------------------
// Sort
// ---------------------------------------------------------------------------
constexpr int SORT_THREADS = 1024, SORT_WAVES = SORT_THREADS / 64, SORT_MOST_BLOCKS = 256;

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
// Workgroups past a.blocks place nothing: they share the marking of padding rows, of
// which a capacity can give many times the pairs, and so make the segments themselves,
// with ONE from a count of all pairs.
template <bool ONE>
__global__ void __launch_bounds__(SORT_THREADS) route_place_kernel(RouteSortArgs a) {
  __shared__ int lds[(SORT_WAVES + 4) * TPMLP_ROUTE_MAX_EXPERTS + 1 + SORT_WAVES];
  const int E = a.E, tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  int* next = lds;                        // [waves][E]
  int* start = next + SORT_WAVES * E;     // [E + 1] first row of each segment
  int* total = start + E + 1;             // [E] pairs of each expert
  int* scan = total + E;                  // [waves] sums of the scan over experts
  int* sums = scan + SORT_WAVES;          // [2][E] pairs in all and in earlier workgroups
  for (int e = tid; e < SORT_WAVES * E; e += SORT_THREADS) next[e] = 0;
  __syncthreads();
  const int64_t p0 = ONE ? 0 : min((int64_t)blockIdx.x * a.per_block, a.pairs), p1 = min(p0 + a.per_block, a.pairs);
  const int64_t run = ((p1 - p0 + SORT_WAVES - 1) / SORT_WAVES + 63) / 64 * 64;
  const int64_t w0 = min(p0 + wave * run, p1), w1 = min(w0 + run, p1);
  for (int64_t p = w0 + lane; p < w1; p += 64) {
    const int e = expert_of(a, p);
    if (e >= 0) atomicAdd(&next[wave * E + e], 1);
  }
  __syncthreads();
  // Pairs of each expert in all workgroups and in those before this one: the threads
  // stand E wide on a row of the histogram and as many rows deep as they go.
  if (!ONE) {
    for (int i = tid; i < 2 * E; i += SORT_THREADS) sums[i] = 0;
    __syncthreads();
    const int lines = SORT_THREADS / E;  // E is at most half the workgroup's size
    const int he = tid % E, line = tid / E;
    if (line < lines) {
      int all = 0, before = 0;
#pragma unroll 8
      for (int b = line; b < a.blocks; b += lines) {
        const int n = a.hist[(int64_t)b * E + he];
        all += n;
        before += b < (int)blockIdx.x ? n : 0;
      }
      atomicAdd(&sums[he], all);
      atomicAdd(&sums[E + he], before);
    }
    __syncthreads();
  }
  const int e = tid;  // a thread has one expert at most
  int before = 0, mine = 0;
  if (e < E) {
    int all = 0;
    if (ONE) {
      for (int w = 0; w < SORT_WAVES; ++w) all += next[w * E + e];
    } else {
      all = sums[e];
      before = sums[E + e];
    }
    mine = a.capacity ? min(all, a.capacity) : all;
  }
  // Exclusive scan of the segment lengths over the experts.
  const int len = e < E ? (a.capacity ? a.capacity : (int)(((uint32_t)mine + a.align - 1) / a.align * a.align)) : 0;
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
  const int64_t place_to = (int)blockIdx.x < a.blocks ? w1 : w0;
  for (int64_t p = w0 + lane; p - lane < place_to; p += 64) {  // all lanes stay for the ballots
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
    if (a.capacity) lo = (int)((uint32_t)r / (uint32_t)a.capacity);  // rows are E * capacity
    else while (hi - lo > 1) {
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
// The rows of up to 64 choices, one a lane: row_of of the token's choices k0 onward,
// -1 where there is none, none inside the sorted buffer, or no such choice.
__device__ __forceinline__ int choice_rows(const int32_t* row_of, int64_t t, int K, int k0, int64_t rows, int lane) {
  const int k = k0 + lane;
  const int r = k < K ? row_of[t * K + k] : -1;
  return (uint32_t)r < (uint64_t)rows ? r : -1;
}
__device__ __forceinline__ int lane_value(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// bf16 rows that are only moved, eight elements a lane; n a multiple of eight and rows
// at multiples of eight elements (FULL), through a descriptor as Row has it; other
// rows with n >= 8 read and write the row's last eight elements on the ragged end,
// which overlap the neighbour's with equal values.
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));

template <bool FULL, bool NT>
struct Row8;
template <bool NT>
struct Row8<false, NT> {
  uint16_t* p;
  int n;
  __device__ __forceinline__ Row8(const uint16_t* base, int64_t at, int n_) : p(const_cast<uint16_t*>(base) + at), n(n_) {}
  __device__ __forceinline__ u16x8 load(int i) const { return *reinterpret_cast<const u16x8_u*>(p + min(i, n - 8)); }
  __device__ __forceinline__ void store(int i, u16x8 v) const {
    if (i < n) *reinterpret_cast<u16x8_u*>(p + min(i, n - 8)) = v;
  }
};
#if defined(__HIP_DEVICE_COMPILE__)
template <bool NT>
struct Row8<true, NT> {
  __amdgpu_buffer_rsrc_t rs;
  __device__ __forceinline__ Row8(const uint16_t* base, int64_t at, int n)
      : rs(__builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(base) + at, (short)0, n * 2, 0x00020000)) {}
  __device__ __forceinline__ u16x8 load(int i) const {
    return __builtin_bit_cast(u16x8, __builtin_amdgcn_raw_buffer_load_b128(rs, i * 2, 0, NT ? 2 : 0));
  }
  __device__ __forceinline__ void store(int i, u16x8 v) const {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rs, i * 2, 0, NT ? 2 : 0);
  }
};
#else
template <bool NT>
struct Row8<true, NT> : Row8<false, NT> {
  using Row8<false, NT>::Row8;
};
#endif

constexpr int DISPATCH_CHUNKS = 4;  // 512-element chunks of a row that a wave moves
constexpr int DISPATCH_COLS = 512 * DISPATCH_CHUNKS;

// Zeros columns [c0, c1) of the padding rows among pad_rows (at most 64) from r0 on.
template <bool FULL, bool NT>
__device__ __forceinline__ void zero_padding(uint16_t* out, int64_t ld, const int32_t* src_of, int64_t rows, int64_t r0,
                                             int pad_rows, int c0, int c1, int n, int lane) {
  uint64_t pad = __ballot(lane < pad_rows && r0 + lane < rows && src_of[min(r0 + lane, rows - 1)] < 0);
  while (pad) {
    const int b = __ffsll((unsigned long long)pad) - 1;
    pad &= pad - 1;
    const Row8<FULL, NT> o(out, (r0 + b) * ld, n);
    for (int i = c0 + 8 * lane; i < c1; i += 512) o.store(i, u16x8{0, 0, 0, 0, 0, 0, 0, 0});
  }
}

template <bool FULL, bool NT>
__global__ void __launch_bounds__(256) route_dispatch_kernel(RouteDispatchArgs a) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  // A row's segments are neighbouring workgroups, so that whole rows are written at
  // about one time; the padding comes first, where it runs beside the tokens.
  const int block = (int)(blockIdx.x / a.segments), c0 = (int)(blockIdx.x % a.segments) * DISPATCH_COLS;
  if (block < a.pad_blocks) {
    const int64_t r0 = ((int64_t)block * 4 + wave) * a.pad_rows;
    if (r0 < a.rows)
      zero_padding<FULL, NT>(a.xs, a.ld_xs, a.src_of, a.rows, r0, a.pad_rows, c0, min(c0 + DISPATCH_COLS, a.H), a.H, lane);
    return;
  }
  const int64_t t = (int64_t)(block - a.pad_blocks) * 4 + wave;
  if (t >= a.T) return;
  const int rows = choice_rows(a.row_of, t, a.K, 0, a.rows, lane);
  const Row8<FULL, NT> x(a.x, t * a.ld_x, a.H);
  u16x8 v[DISPATCH_CHUNKS];
#pragma unroll
  for (int c = 0; c < DISPATCH_CHUNKS; ++c) v[c] = x.load(c0 + c * 512 + 8 * lane);
  for (int k = 0; k < a.K; ++k) {
    const int row = lane_value(rows, k);
    if (row < 0) continue;  // dropped
    const Row8<FULL, NT> o(a.xs, row * a.ld_xs, a.H);
#pragma unroll
    for (int c = 0; c < DISPATCH_CHUNKS; ++c) o.store(c0 + c * 512 + 8 * lane, v[c]);
  }
}

// Short rows (at most 256 elements): a row is `lanes` lanes of eight elements (a power
// of two), and the wave writes 64 / lanes of the token's rows at once.
__global__ void __launch_bounds__(256) route_dispatch_short_kernel(RouteDispatchArgs a) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  if ((int)blockIdx.x < a.pad_blocks) {
    const int64_t r0 = ((int64_t)blockIdx.x * 4 + wave) * a.pad_rows;
    if (r0 < a.rows) zero_padding<false, false>(a.xs, a.ld_xs, a.src_of, a.rows, r0, a.pad_rows, 0, a.H, a.H, lane);
    return;
  }
  const int64_t t = (int64_t)((int)blockIdx.x - a.pad_blocks) * 4 + wave;
  if (t >= a.T) return;
  const int rows = choice_rows(a.row_of, t, a.K, 0, a.rows, lane);
  const int i = 8 * (lane & (a.lanes - 1)), group = lane / a.lanes, groups = 64 / a.lanes, at = min(i, a.H - 8);
  const u16x8_u v = *reinterpret_cast<const u16x8_u*>(a.x + t * a.ld_x + at);
  for (int k0 = 0; k0 < a.K; k0 += groups) {
    const int row = __shfl(rows, min(k0 + group, 63), 64);
    if (k0 + group < a.K && row >= 0 && i < a.H) *reinterpret_cast<u16x8_u*>(a.xs + row * a.ld_xs + at) = v;
  }
}

// A wave sums CHUNKS 256-element chunks of a token's rows, four choices' loads in
// flight together.  A choice that takes no part is a row of length zero with weight
// zero: it reads no memory and adds nothing.
constexpr int COMBINE_CHOICES = 4;

template <class ZT, class YT, int CHUNKS, bool FULL, bool NT>
__global__ void __launch_bounds__(256) route_combine_kernel(RouteCombineArgs a) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t >= a.T) return;
  auto at = [&](int c) { return ((int)blockIdx.y * CHUNKS + c) * 256 + 4 * lane; };
  const int rows = choice_rows(a.row_of, t, a.K, 0, a.rows, lane);
  const float ws = rows >= 0 && a.w ? a.w[t * a.K + lane] : 1.0f;
  f32x4 sum[CHUNKS];
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) sum[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int k0 = 0; k0 < a.K; k0 += COMBINE_CHOICES) {
    typedef Row<ZT, FULL, NT> RZ;
    typename RZ::raw z[COMBINE_CHOICES][CHUNKS];
    float w[COMBINE_CHOICES];
#pragma unroll
    for (int j = 0; j < COMBINE_CHOICES; ++j) {
      const int k = min(k0 + j, 63), row = k0 + j < a.K ? lane_value(rows, k) : -1;
      w[j] = row >= 0 ? lane_value(ws, k) : 0.0f;
      const RZ r(a.zs, row >= 0 ? row * a.ld_zs : 0, row >= 0 ? a.H : 0);
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) z[j][c] = r.load_raw(at(c));
    }
#pragma unroll
    for (int j = 0; j < COMBINE_CHOICES; ++j)
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c) {
        const f32x4 v = RZ::widen_raw(z[j][c], at(c), a.H);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[c][e] = __builtin_fmaf(v[e], w[j], sum[c][e]);
      }
  }
  const Row<YT, FULL, NT> y(a.y, t * a.ld_y, a.H);
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c) y.store(at(c), sum[c]);
}

// W waves a token (one where a row is no longer than a wave's four passes), NP choices
// together; a choice that takes no part is a row of length zero.
template <class DT, class ZT, int W, int NP, bool FULL, bool NT>
__global__ void __launch_bounds__(256) route_combine_bwd_kernel(RouteCombineBwdArgs a) {
  __shared__ float dots[NP][4];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  if ((int)blockIdx.x < a.pad_blocks) {  // first, where it runs beside the tokens
    const int64_t r0 = ((int64_t)blockIdx.x * 4 + wave) * a.pad_rows;
    if (r0 < a.rows) zero_padding<false, NT>(a.dzs, a.ld_dzs, a.src_of, a.rows, r0, a.pad_rows, 0, a.H, a.H, lane);
    return;
  }
  const int64_t t = W == 1 ? (int64_t)((int)blockIdx.x - a.pad_blocks) * 4 + wave : (int64_t)((int)blockIdx.x - a.pad_blocks);
  if (t >= a.T) return;  // W == 1 only, where no barrier follows
  const int rows = choice_rows(a.row_of, t, a.K, 0, a.rows, lane);
  const float ws = rows >= 0 && a.w ? a.w[t * a.K + lane] : 1.0f;
  const Row<DT, FULL, NT> dy(a.dy, t * a.ld_dy, a.H);
  for (int k0 = 0; k0 < a.K; k0 += NP) {
    float w[NP], dot[NP];
    int row[NP];
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int k = min(k0 + j, 63);
      row[j] = k0 + j < a.K ? lane_value(rows, k) : -1;
      w[j] = lane_value(ws, k);
      dot[j] = 0.0f;
    }
    for (int i = 4 * (W == 1 ? lane : (int)threadIdx.x); i < a.H; i += 256 * W) {
      typedef Row<ZT, FULL, NT> RZ;
      typename RZ::raw z[NP];
      const auto d0 = dy.load_raw(i);
      if (a.dw)
#pragma unroll
        for (int j = 0; j < NP; ++j) z[j] = RZ(a.zs, row[j] >= 0 ? row[j] * a.ld_zs : 0, row[j] >= 0 ? a.H : 0).load_raw(i);
      const f32x4 d = Row<DT, FULL, NT>::widen_raw(d0, i, a.H);
      if (a.dzs)
#pragma unroll
        for (int j = 0; j < NP; ++j)
          if (row[j] >= 0) Row<BF16, FULL, NT>(a.dzs, row[j] * a.ld_dzs, a.H).store(i, d * w[j]);
      if (a.dw)
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          const f32x4 v = RZ::widen_raw(z[j], i, a.H);
#pragma unroll
          for (int e = 0; e < 4; ++e) dot[j] = __builtin_fmaf(d[e], v[e], dot[j]);
        }
    }
    if (!a.dw) continue;
    if (W == 1) {
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        // A dropped pair's dot is with zeros, and an infinity of dY times them is no 0.
        const float s = row[j] >= 0 ? wave_sum(dot[j]) : 0.0f;
        if (lane == j && k0 + j < a.K) a.dw[t * a.K + k0 + j] = s;
      }
      continue;
    }
    __syncthreads();  // the sums of the choices before are read
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const float s = row[j] >= 0 ? wave_sum(dot[j]) : 0.0f;
      if (lane == 0) dots[j][wave] = s;
    }
    __syncthreads();
    const int j = (int)threadIdx.x;
    if (j < NP && k0 + j < a.K) {
      const float* s = dots[j];
      a.dw[t * a.K + k0 + j] = (s[0] + s[1]) + (s[2] + s[3]);
    }
  }
}

int blocks_of(int64_t n, int64_t per) { return (int)((n + per - 1) / per); }

}  // namespace

int64_t route_sort_blocks(int64_t pairs, int64_t* per_block) {
  // One workgroup sorts up to 4096 pairs by itself; larger sorts give each 2048, and
  // more where that would be over 256 of them: each reads all the others' histograms.
  const int64_t per = pairs <= 4096 ? 4096 : pairs <= SORT_MOST_BLOCKS * 2048 ? 2048 : (pairs + SORT_MOST_BLOCKS - 1) / SORT_MOST_BLOCKS;
  *per_block = per;
  return pairs <= per ? 1 : (pairs + per - 1) / per;
}

hipError_t launch_route_sort(const RouteSortArgs& a, hipStream_t s) {
  if (a.E < 1 || a.E > TPMLP_ROUTE_MAX_EXPERTS || a.blocks < 1) return hipErrorInvalidValue;
  // A workgroup for each 1024 rows.  With as many as place pairs (one up to 4096 pairs) 4096
  // pairs to 256 experts took 104 us for 131072 rows and 12.4 for 5888, now 8.9 and 9.3.
  const int64_t pad = std::min<int64_t>((a.rows + SORT_THREADS - 1) / SORT_THREADS, SORT_MOST_BLOCKS);
  const dim3 place((unsigned)std::max<int64_t>(a.blocks, pad));
  if (a.blocks == 1) return launch_kernel(route_place_kernel<true>, place, dim3(SORT_THREADS), s, a);
  hipError_t e = launch_kernel(route_hist_kernel, dim3((unsigned)a.blocks), dim3(SORT_THREADS), s, a);
  if (e != hipSuccess) return e;
  return launch_kernel(route_place_kernel<false>, place, dim3(SORT_THREADS), s, a);
}

namespace {
// Rows that one wave looks through for padding: few where there are few, so that the
// zeroing of several rows is not one wave's work.
int pad_rows_for(int64_t rows) { return rows <= 16384 ? 4 : 64; }
}  // namespace

hipError_t launch_route_dispatch(RouteDispatchArgs a, bool full, bool nt, hipStream_t s) {
  if (a.H < 8 || a.K < 1 || a.K > 64) return hipErrorInvalidValue;
  a.segments = blocks_of(a.H, DISPATCH_COLS);
  a.pad_rows = pad_rows_for(a.rows);
  a.pad_blocks = blocks_of(a.rows, 4 * a.pad_rows);
  const int64_t blocks = ((int64_t)a.pad_blocks + blocks_of(a.T, 4)) * a.segments;
  if (blocks < 1) return hipSuccess;
  if (!block_grid_ok(blocks, 256)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks), block(256);
  if (a.H <= 256) {  // 32768 tokens of 64 with 8 choices: 37 us by whole waves
    for (a.lanes = 1; 8 * a.lanes < a.H;) a.lanes *= 2;
    return launch_kernel(route_dispatch_short_kernel, grid, block, s, a);
  }
  if (!full) return launch_kernel(route_dispatch_kernel<false, false>, grid, block, s, a);
  return nt ? launch_kernel(route_dispatch_kernel<true, true>, grid, block, s, a)
            : launch_kernel(route_dispatch_kernel<true, false>, grid, block, s, a);
}

namespace {

template <class ZT, class YT>
hipError_t launch_combine(const RouteCombineArgs& a, bool full, bool nt, hipStream_t s) {
  // Few tokens: a chunk to a wave, so that more waves share the latency.  Launches bound by
  // memory: four, 2048 x 4096 of eight choices 52 us (56.9 with two, 59.2 with one); smaller
  // ones are better with two (16384 x 200 11.8 against 12.8 us).
  const int chunks = full && nt ? 4 : a.T <= 2048 ? 1 : 2;
  const dim3 grid((unsigned)blocks_of(a.T, 4), (unsigned)blocks_of(a.H, 256 * chunks)), block(256);
  if (!full) return chunks == 1 ? launch_kernel(route_combine_kernel<ZT, YT, 1, false, false>, grid, block, s, a)
                                : launch_kernel(route_combine_kernel<ZT, YT, 2, false, false>, grid, block, s, a);
  if (chunks == 4) return launch_kernel(route_combine_kernel<ZT, YT, 4, true, true>, grid, block, s, a);
  return chunks == 1 ? launch_kernel(route_combine_kernel<ZT, YT, 1, true, false>, grid, block, s, a)
                     : launch_kernel(route_combine_kernel<ZT, YT, 2, true, false>, grid, block, s, a);
}

template <class DT, class ZT, int W>
hipError_t launch_combine_bwd(RouteCombineBwdArgs a, bool full, bool nt, hipStream_t s) {
  a.pad_rows = pad_rows_for(a.rows);
  a.pad_blocks = a.dzs ? blocks_of(a.rows, 4 * a.pad_rows) : 0;
  const int64_t blocks = a.pad_blocks + (W == 1 ? blocks_of(a.T, 4) : a.T);
  if (blocks < 1) return hipSuccess;
  if (!block_grid_ok(blocks, 256)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks), block(256);
#define BWD_FORM(NP)                                                                                            \
  return !full ? launch_kernel(route_combine_bwd_kernel<DT, ZT, W, NP, false, false>, grid, block, s, a)        \
         : nt  ? launch_kernel(route_combine_bwd_kernel<DT, ZT, W, NP, true, true>, grid, block, s, a)          \
               : launch_kernel(route_combine_bwd_kernel<DT, ZT, W, NP, true, false>, grid, block, s, a)
  if (a.K <= 2) BWD_FORM(2);
  if (a.K <= 4) BWD_FORM(4);
  BWD_FORM(8);
#undef BWD_FORM
}

template <class DT, class ZT>
hipError_t launch_combine_bwd(const RouteCombineBwdArgs& a, bool full, bool nt, hipStream_t s) {
  return a.H <= 1024 ? launch_combine_bwd<DT, ZT, 1>(a, full, nt, s) : launch_combine_bwd<DT, ZT, 4>(a, full, nt, s);
}

}  // namespace

hipError_t launch_route_combine(const RouteCombineArgs& a, int z_type, int y_type, bool full, bool nt, hipStream_t s) {
  if (a.H < 4 || a.T < 1 || a.K < 1 || a.K > 64) return hipErrorInvalidValue;
  if (z_type == TPMLP_BF16)
    return y_type == TPMLP_BF16 ? launch_combine<BF16, BF16>(a, full, nt, s) : launch_combine<BF16, F32>(a, full, nt, s);
  return y_type == TPMLP_BF16 ? launch_combine<F32, BF16>(a, full, nt, s) : launch_combine<F32, F32>(a, full, nt, s);
}

hipError_t launch_route_combine_bwd(const RouteCombineBwdArgs& a, int dy_type, int z_type, bool full, bool nt, hipStream_t s) {
  if (a.H < 8 || a.K < 1 || a.K > 64) return hipErrorInvalidValue;
  if (dy_type == TPMLP_BF16)
    return z_type == TPMLP_BF16 ? launch_combine_bwd<BF16, BF16>(a, full, nt, s) : launch_combine_bwd<BF16, F32>(a, full, nt, s);
  return z_type == TPMLP_BF16 ? launch_combine_bwd<F32, BF16>(a, full, nt, s) : launch_combine_bwd<F32, F32>(a, full, nt, s);
}

}  // namespace tpmlp
