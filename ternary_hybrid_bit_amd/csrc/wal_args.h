// Argument checks shared by the entry points that take strided rows (host).
#pragma once

#include "wal_internal.h"

namespace wal {

// n rows of `width` bytes, `pitch` bytes apart.
struct Rows {
  uintptr_t at = 0;
  uint64_t n = 0, pitch = 0, width = 0;
  uint64_t end() const { return at + (n ? (n - 1) * pitch + width : 0); }
};

inline Rows rows(const void* p, uint64_t n, uint64_t ld, uint64_t width, uint64_t elem) {
  return Rows{reinterpret_cast<uintptr_t>(p), n, ld * elem, width * elem};
}
inline Rows flat(const void* p, uint64_t bytes) {
  return Rows{reinterpret_cast<uintptr_t>(p), bytes ? 1u : 0u, bytes, bytes};
}

// Whether two sets of rows share a byte.  Rows of one pitch may lie side by
// side (columns of one buffer); any other pair is judged by its whole span.
inline bool meet(const Rows& a, const Rows& b) {
  if (!a.n || !b.n || a.at >= b.end() || b.at >= a.end()) return false;
  if (a.pitch == b.pitch && a.pitch) {
    const uint64_t d = a.at <= b.at ? (b.at - a.at) % a.pitch : (a.pitch - (a.at - b.at) % a.pitch) % a.pitch;
    if (d >= a.width && d + b.width <= a.pitch) return false;
  }
  return true;
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool dtype_ok(int t) { return t == WAL_X_F32 || t == WAL_X_BF16; }
inline uint32_t elem_bytes(int dtype) { return dtype == WAL_X_BF16 ? 2 : 4; }

// Rows a kernel reads or writes 16 bytes at a time.
inline int check_rows(const void* p, uint32_t ld, uint64_t width, int dtype) {
  if (!p || ld < width) return WAL_ERR_ARG;
  if (!aligned(p, 16) || ((uint64_t)ld * elem_bytes(dtype)) % 16) return WAL_ERR_ALIGN;
  return WAL_OK;
}

}  // namespace wal
