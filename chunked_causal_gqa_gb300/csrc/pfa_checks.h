// pfa_checks.h -- argument checks that the entry points of the 8-bit and of the 4-bit
// cache's operators share.
#pragma once
#include "pfa_internal.h"

#include "../../include/pfa.h"

#include <cmath>

namespace pfa {

constexpr int64_t kMaxLen = ((int64_t)1 << 31) - 4096;  // positions and row counts

inline size_t elem(int dtype) { return dtype == PFA_F32 ? 4 : 2; }
inline bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) & (a - 1); }
inline size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

// n rows of `width` bytes, `pitch` bytes apart.
struct Rows {
  const void* p;
  int64_t n;
  size_t pitch, width;
  size_t span() const { return (size_t)(n - 1) * pitch + width; }
};

// Whether two sets of rows share a byte.  Columns of one buffer (the same
// pitch) are told apart by their column ranges; anything else by its span.
inline bool share(const Rows& a, const Rows& b) {
  if (!overlaps(a.p, a.span(), b.p, b.span())) return false;
  if (a.pitch != b.pitch) return true;
  const int64_t pitch = (int64_t)a.pitch;
  int64_t d = ((int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p))) % pitch;
  if (d < 0) d += pitch;  // b's first column in a's rows
  return d < (int64_t)a.width || d + (int64_t)b.width > pitch;
}

inline int check_span(int64_t B, int64_t T, int64_t start_pos, const int64_t* lengths) {
  if (B < 0 || T < 0 || B > kMaxLen || T > kMaxLen || B * T > kMaxLen) return PFA_ERR_SHAPE;
  if (lengths) return misaligned(lengths, 8) ? PFA_ERR_ALIGNMENT : PFA_OK;
  // without lengths: one sequence, its position known to the host
  if (B > 1 || start_pos < 0 || start_pos > kMaxLen || start_pos + T > kMaxLen)
    return PFA_ERR_SHAPE;
  return PFA_OK;
}

// Shapes of the attention entries.
inline int check_attention(int64_t B, int64_t T, int H, int Hkv, int D, float scale, int dtype) {
  if (dtype != PFA_F32 && dtype != PFA_BF16) return PFA_ERR_DTYPE;
  if (B < 0 || T < 0 || H <= 0 || Hkv <= 0 || H % Hkv != 0 || H / Hkv > 128) return PFA_ERR_SHAPE;
  if (D != 128 && D != 512) return PFA_ERR_SHAPE;
  if (!std::isfinite(scale)) return PFA_ERR_VALUE;
  return PFA_OK;
}

}  // namespace pfa
