// Argument checks that the C-ABI layers of the operators share: sizes, types and
// which buffers may meet.  Not installed.
#pragma once

#include "step_internal.h"

namespace rsx {
namespace {

constexpr size_t kMaxSize = 0x7fffffffu;  // dims, rows, tokens

size_t float_size(int t) {
  return t == RSX_FLOAT32 ? 4 : t == RSX_BFLOAT16 || t == RSX_FLOAT16 ? 2 : 0;
}
size_t token_size(int t) { return t == RSX_INT32 ? 4 : t == RSX_INT64 ? 8 : 0; }

// Ids first .. first + vocab - 1 are token ids; past the largest they would wrap.
bool ids_wrap(int64_t first, size_t vocab) { return vocab != 0 && first > INT64_MAX - static_cast<int64_t>(vocab - 1); }

// A buffer as rows of `width` bytes, `pitch` bytes apart.
struct Area {
  uintptr_t lo, hi;
  size_t width, pitch;
  size_t align;
};
Area rows_area(const void* p, size_t rows, size_t dim, size_t stride, size_t es) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  const size_t bytes = rows == 0 || dim == 0 ? 0 : ((rows - 1) * stride + dim) * es;
  return {lo, lo + bytes, dim * es, stride * es, es};
}
Area flat_area(const void* p, size_t n, size_t es) { return rows_area(p, n != 0 ? 1 : 0, n, n, es); }

bool meet(const Area& a, const Area& b) {
  if (a.lo == a.hi || b.lo == b.hi || a.hi <= b.lo || b.hi <= a.lo) return false;
  if (a.pitch == b.pitch && a.pitch != 0) {
    const uintptr_t off = b.lo >= a.lo ? (b.lo - a.lo) % a.pitch : (a.pitch - (a.lo - b.lo) % a.pitch) % a.pitch;
    if (off >= a.width && off + b.width <= a.pitch) return false;  // rows that interleave
  }
  return true;
}
bool same(const Area& a, const Area& b) {
  return a.lo == b.lo && a.hi == b.hi && a.pitch == b.pitch && a.align == b.align;
}

// The buffers of one call.  Outputs may meet nothing else, but for `twin`, an
// input that an output may be.
struct Areas {
  static constexpr int kMost = 12;
  Area in[kMost], out[kMost];
  int nin = 0, nout = 0;
  bool bad = false, large = false;

  void check(const Area& a, const void* p) {
    const bool some = a.hi != a.lo;
    bad = bad || (some && p == nullptr) || (reinterpret_cast<uintptr_t>(p) & (a.align - 1)) != 0 || a.hi < a.lo;
    large = large || a.hi - a.lo > kMaxSpan;
  }
  Area& read(const void* p, size_t rows, size_t dim, size_t stride, size_t es) {
    bad = bad || (stride < dim && stride != 0);
    large = large || stride > kMaxSpan / es || (rows > 1 && stride * es > kMaxSpan / rows);
    if (large) return in[0];
    in[nin] = rows_area(p, rows, dim, stride, es);
    check(in[nin], p);
    return in[nin++];
  }
  Area& write(const void* p, size_t rows, size_t dim, size_t stride, size_t es) {
    bad = bad || stride < dim;
    large = large || stride > kMaxSpan / es || (rows > 1 && stride * es > kMaxSpan / rows);
    if (large) return out[0];
    out[nout] = rows_area(p, rows, dim, stride, es);
    check(out[nout], p);
    return out[nout++];
  }
  void read_flat(const void* p, size_t n, size_t es) { read(p, n != 0 ? 1 : 0, n, n, es); }
  void write_flat(const void* p, size_t n, size_t es) { write(p, n != 0 ? 1 : 0, n, n, es); }
  void workspace(const void* p, size_t have, size_t need) {
    bad = bad || have < need || (need != 0 && (p == nullptr || (reinterpret_cast<uintptr_t>(p) & 255u) != 0));
    if (!bad && need != 0) write_flat(p, need, 1);
  }
  // twins: how many of the first inputs the first output may coincide with.
  rsx_status_t status(int twins = 0) const {
    if (bad) return RSX_ERR_INVALID_ARGUMENT;
    if (large) return RSX_ERR_UNSUPPORTED;
    for (int o = 0; o < nout; ++o) {
      for (int i = 0; i < nin; ++i)
        if (meet(out[o], in[i]) && !(o == 0 && i < twins && same(out[o], in[i]))) return RSX_ERR_ALIASING;
      for (int p = o + 1; p < nout; ++p)
        if (meet(out[o], out[p])) return RSX_ERR_ALIASING;
    }
    return RSX_SUCCESS;
  }
};

}  // namespace
}  // namespace rsx
