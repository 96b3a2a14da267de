// Argument checks of the C entry points, all before any HIP call.
#pragma once

#include <algorithm>
#include <cstdint>
#include <string>
#include <utility>
#include <vector>

#include "block.h"
#include "host.h"

namespace tpmlp {

constexpr int64_t MAX_TOKENS = int64_t(1) << 23;  // as the MLP's M
constexpr int64_t MAX_LD = int64_t(1) << 31;

// Runs an entry point's body; an exception (the host is out of memory while it
// writes an error's text) becomes a status.
template <class F>
inline tpmlp_status guarded(F&& body) {
  try {
    g_last_error.clear();
    return body();
  } catch (...) {
    return TPMLP_ERR_HIP;
  }
}

#define TRY(x)                          \
  do {                                  \
    if (tpmlp_status st_ = (x)) return st_; \
  } while (0)

// A strided matrix that a call reads or writes (p NULL: absent).
struct Mat {
  const void* p;
  int64_t rows, cols, ld;
  int elem;  // bytes
  const char* name;
};

inline int size_of(int type) { return type == TPMLP_BF16 ? 2 : 4; }
inline bool type_ok(int t) { return t == TPMLP_F32 || t == TPMLP_BF16; }

inline bool empty(const Mat& m) { return !m.p || m.rows < 1 || m.cols < 1; }

inline bool overlap(const Mat& a, const Mat& b) {
  if (empty(a) || empty(b)) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  const uint64_t pa = uint64_t(a.ld) * a.elem, pb = uint64_t(b.ld) * b.elem;
  const uint64_t wa = uint64_t(a.cols) * a.elem, wb = uint64_t(b.cols) * b.elem;
  if (a0 >= b0 + (b.rows - 1) * pb + wb || b0 >= a0 + (a.rows - 1) * pa + wa) return false;
  if (pa != pb) return true;
  // Equal pitches: column blocks of one buffer are disjoint if their columns are.
  const uint64_t off = b0 >= a0 ? (b0 - a0) % pa : (pa - (a0 - b0) % pa) % pa;
  return off < wa || off + wb > pa;
}

// Pointer and stride of a matrix that has to be there unless it has no elements.
inline tpmlp_status check_mat(const Mat& m) {
  if (m.ld < m.cols || m.ld > MAX_LD) return fail(TPMLP_ERR_SHAPE, std::string("ld of ") + m.name + " is below its row length or above 2^31");
  if (m.rows > 0 && m.cols > 0 && !m.p) return fail(TPMLP_ERR_NULL, std::string(m.name) + " is NULL");
  if (reinterpret_cast<uintptr_t>(m.p) % m.elem) return fail(TPMLP_ERR_ALIGN, std::string(m.name) + " is not aligned to its elements");
  return TPMLP_OK;
}

// Each output must be disjoint from every other matrix.  `same`: (output, input)
// indices that may also be one matrix.
template <size_t NO, size_t NI>
inline tpmlp_status check_overlaps(const Mat (&outs)[NO], const Mat (&ins)[NI], int same_out = -1, int same_in = -1) {
  for (size_t i = 0; i < NO; ++i) {
    for (size_t j = i + 1; j < NO; ++j)
      if (overlap(outs[i], outs[j])) return fail(TPMLP_ERR_ALIAS, std::string(outs[i].name) + " overlaps " + outs[j].name);
    for (size_t j = 0; j < NI; ++j) {
      if ((int)i == same_out && (int)j == same_in && outs[i].p == ins[j].p && outs[i].ld == ins[j].ld) continue;
      if (overlap(outs[i], ins[j])) return fail(TPMLP_ERR_ALIAS, std::string(outs[i].name) + " overlaps " + ins[j].name);
    }
  }
  return TPMLP_OK;
}

inline hipStream_t stream_of(void* s) { return static_cast<hipStream_t>(s); }

inline tpmlp_status launched(hipError_t e, const char* what) { return e == hipSuccess ? TPMLP_OK : hip_fail(e, what); }

inline int64_t ld_or(int64_t ld, int64_t cols) { return ld ? ld : cols; }

// Whether every row of the matrix starts at a multiple of `n` elements.
inline bool starts_at(const Mat& m, int n) {
  return empty(m) || (reinterpret_cast<uintptr_t>(m.p) % (n * m.elem) == 0 && (m.rows < 2 || m.ld % n == 0));
}
inline bool quads(const Mat& m) { return starts_at(m, 4); }
template <size_t NO, size_t NI>
inline bool all_quads(int64_t H, const Mat (&outs)[NO], const Mat (&ins)[NI]) {
  return H % 4 == 0 && std::all_of(outs, outs + NO, quads) && std::all_of(ins, ins + NI, quads);
}

// Whether a launch over these matrices moves more than BLOCK_NT_BYTES.
template <size_t NO, size_t NI>
inline bool past_caches(const Mat (&outs)[NO], const Mat (&ins)[NI]) {
  int64_t bytes = 0;
  for (const Mat& m : outs) bytes += empty(m) ? 0 : m.rows * m.cols * m.elem;
  for (const Mat& m : ins) bytes += empty(m) ? 0 : m.rows * m.cols * m.elem;
  return bytes > BLOCK_NT_BYTES;
}

// Dense buffers of the calls whose tensors are contiguous and 16-byte aligned.
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

struct Range {
  const void* p;
  size_t bytes;
  const char* name;
};

inline bool overlap(const Range& a, const Range& b) {
  if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// Each output must be disjoint from every other range.
inline tpmlp_status check_alias(const std::vector<Range>& outs, const std::vector<Range>& ins) {
  for (size_t i = 0; i < outs.size(); ++i) {
    for (size_t j = i + 1; j < outs.size(); ++j)
      if (overlap(outs[i], outs[j]))
        return fail(TPMLP_ERR_ALIAS, std::string(outs[i].name) + " overlaps " + outs[j].name);
    for (const Range& r : ins)
      if (overlap(outs[i], r)) return fail(TPMLP_ERR_ALIAS, std::string(outs[i].name) + " overlaps " + r.name);
  }
  return TPMLP_OK;
}

inline tpmlp_status check_ptrs(std::initializer_list<std::pair<const void*, const char*>> ptrs) {
  for (auto& p : ptrs)
    if (!p.first) return fail(TPMLP_ERR_NULL, std::string(p.second) + " is NULL");
  for (auto& p : ptrs)
    if (!aligned16(p.first)) return fail(TPMLP_ERR_ALIGN, std::string(p.second) + " is not 16-byte aligned");
  return TPMLP_OK;
}

}  // namespace tpmlp
