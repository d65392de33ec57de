// Host-side argument checks shared by the operators of include/block_ops.h.
#pragma once

#include <cstdint>

#include "../../../include/block_ops.h"

namespace block_ops {

constexpr int64_t kMaxExtent = (int64_t)1 << 46;  // elements: byte offsets stay in int64
constexpr int64_t kMaxRows = 0x7FFFFFFFLL;        // B * L: 32-bit row indices

inline bool is_flag(int v) { return v == 0 || v == 1; }

// Byte range [lo, hi) that a buffer's elements lie in.
struct Span {
  uintptr_t lo = 0, hi = 0;
};
inline bool overlaps(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }

inline Span bytes_at(const void* p, uint64_t n) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Span{lo, lo + n};
}

// One past the last element of `extents` steps along non-negative strides, each cell `width`
// wide; -1 if it is too large.
template <int N>
inline int64_t extent_of(const int64_t (&extents)[N], const int64_t (&strides)[N], int64_t width) {
  __int128 end = width;
  for (int i = 0; i < N; ++i) end += (__int128)(extents[i] - 1) * strides[i];
  return end > kMaxExtent ? -1 : (int64_t)end;
}

// The worst of several findings: an invalid argument is reported before a misalignment.
struct Findings {
  fn_status status = FN_OK;
  void add(fn_status s) {
    if (s == FN_ERR_INVALID_ARG || status == FN_OK) status = (status == FN_ERR_INVALID_ARG) ? status : s;
  }
  void require(bool ok, fn_status s) {
    if (!ok) add(s);
  }
};

inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// A row-addressed input of 2-byte elements: strides and alignment.
inline void check_operand(const fn_operand& o, bool frame_axis, Findings& f) {
  f.require(o.stride_b >= 0 && o.stride_f >= 0 && o.stride_l >= 0, FN_ERR_INVALID_ARG);
  f.require(frame_axis || o.stride_f == 0, FN_ERR_INVALID_ARG);
  f.require(aligned16(o.ptr) && o.stride_b % 8 == 0 && o.stride_f % 8 == 0 && o.stride_l % 8 == 0,
            FN_ERR_MISALIGNED);
}

// Output rows of `width` elements: strides that keep the rows apart, and alignment to
// `unit` elements (16 bytes).
inline void check_output(const void* p, int64_t sb, int64_t sl, int64_t B, int64_t L, int64_t width,
                         int64_t unit, Findings& f) {
  f.require(sb >= 0 && sl >= 0, FN_ERR_INVALID_ARG);
  f.require(L <= 1 || sl >= width, FN_ERR_INVALID_ARG);
  f.require(B <= 1 || (__int128)sb >= (__int128)(L - 1) * sl + width, FN_ERR_INVALID_ARG);
  f.require(aligned16(p) && sb % unit == 0 && sl % unit == 0, FN_ERR_MISALIGNED);
}

// The byte range of a row-addressed operand's (B, L, width) elements; false if too large.
inline bool operand_span(const fn_operand& o, int64_t B, int64_t F, int64_t L, int64_t width, int size,
                         Span* out) {
  const int64_t n[3] = {B, F, L}, s[3] = {o.stride_b, o.stride_f, o.stride_l};
  const int64_t e = extent_of(n, s, width);
  if (e < 0) return false;
  *out = bytes_at(o.ptr, (uint64_t)e * size);
  return true;
}

// Whether output rows are the operand's own rows, element for element.
inline bool same_rows(const fn_operand& o, const void* p, int64_t sb, int64_t sl, int64_t B, int64_t L) {
  return o.ptr == p && o.stride_f == 0 && (B == 1 || o.stride_b == sb) && (L == 1 || o.stride_l == sl);
}

// Keeps the runtime's status of this thread's last failed launch; FN_OK or FN_ERR_CUDA.
fn_status launch_status(int cuda_error);

// FN_ERR_CUDA (cudaErrorLaunchTimeout), once, after a kernel has set *gave_up; FN_OK otherwise.
fn_status wait_status(int* gave_up);

}  // namespace block_ops
