// operands.h -- host checks of the operands that a call reads and writes: rows
// of some bytes, a stride apart.
#pragma once

#include <cstddef>
#include <cstdint>

#include "hb.h"

namespace hb {

hb_status internal_fail(hb_status s, const char* msg);
hb_status internal_failf(hb_status s, const char* fmt, ...);

// `rows` rows of `bytes` bytes each, `stride` bytes apart; p NULL: not given.
struct Operand {
  const void* p;
  int64_t rows, bytes, stride;
  const char* name;
  uintptr_t begin() const { return reinterpret_cast<uintptr_t>(p); }
  uintptr_t end() const { return begin() + (uintptr_t)((rows - 1) * stride + bytes); }
  bool given() const { return p != nullptr && rows > 0 && bytes > 0; }
};

// The same bytes, row for row.
inline bool same_rows(const Operand& a, const Operand& b) {
  return a.p == b.p && a.bytes == b.bytes && (a.stride == b.stride || a.rows == 1);
}

// Whether two operands share a byte.  Rows of one stride that lie side by side
// in the columns of one array do not; of two strides, overlapping extents count
// as shared.
inline bool share_bytes(const Operand& a, const Operand& b) {
  if (!a.given() || !b.given()) return false;
  if (a.end() <= b.begin() || b.end() <= a.begin()) return false;
  if (a.stride != b.stride || a.stride <= 0) return true;
  const Operand &lo = a.begin() <= b.begin() ? a : b, &hi = a.begin() <= b.begin() ? b : a;
  const int64_t at = (int64_t)((hi.begin() - lo.begin()) % (uintptr_t)a.stride);
  return at < lo.bytes || at + hi.bytes > a.stride;
}

// An output may be one of the inputs, row for row where `in_place` allows it,
// and shares no byte with them otherwise.
inline hb_status check_apart(const Operand& out, const Operand& in, bool in_place) {
  if (!share_bytes(out, in) || (in_place && same_rows(out, in))) return HB_OK;
  return internal_failf(HB_ERR_INVALID_ARG, "%s and %s overlap", out.name, in.name);
}

// 16-byte vectors from the first row on.
inline hb_status check_rows(const Operand& o) {
  if (!o.p) return internal_failf(HB_ERR_INVALID_ARG, "%s is NULL", o.name);
  if (reinterpret_cast<uintptr_t>(o.p) & 15u)
    return internal_failf(HB_ERR_INVALID_ARG, "%s is not 16-byte aligned", o.name);
  if (o.rows <= 1) return HB_OK;
  if (o.stride < o.bytes)
    return internal_failf(HB_ERR_SHAPE, "%s: rows of %lld bytes are %lld bytes apart", o.name, (long long)o.bytes,
                          (long long)o.stride);
  if (o.stride % 16) return internal_failf(HB_ERR_INVALID_ARG, "%s: rows are not a multiple of 16 bytes apart", o.name);
  return HB_OK;
}

}  // namespace hb
