// Products that are stored as they are, copies of matrices as 16-bit parts, and
// products of few rows: shared launches of the product operators.
#pragma once

#include "product.h"
#include "product_internal.h"

namespace rsx {

enum Layouts { kNT, kNN, kTN };  // A row, B row; A row, B col; A col, B col

struct StoreArgs {
  void* out;
  uint64_t ld;
  int type;
  const float* add;  // fp32 [m][n] to add, or null
  const float* row;  // then a factor for each row, or null
  int accumulate;    // add what `out` holds
  void* out2;        // the second product's of a stack of two
  uint64_t ld2;
};

// Steps of a product of `segments` times k.
inline uint64_t steps_of(uint64_t k, uint64_t segments) { return segments * (k == 0 ? 1 : (k + kStep - 1) / kStep); }
inline Schedule store_schedule(uint64_t m, uint64_t n, uint64_t k, uint64_t segments, uint64_t batch = 1) {
  return schedule(m, n, batch, steps_of(k, segments), false, false);
}
inline uint64_t store_ws(uint64_t m, uint64_t n, uint64_t k, uint64_t segments, uint64_t batch = 1) {
  return store_schedule(m, n, k, segments, batch).bytes;
}
// half: the parts are fp16, else bf16.  ws: store_ws bytes.
hipError_t launch_store(bool half, Layouts l, ProductArgs p, const StoreArgs& e, void* ws, hipStream_t s);

// Rows of a copy start on cache lines.
inline uint64_t copy_ld(uint64_t cols) { return (cols + 63) & ~63ull; }
inline uint64_t copy_bytes(uint64_t rows, uint64_t cols, int count) { return count * ((rows * copy_ld(cols) * 2 + 255) & ~255ull); }

// Memory for a matrix's parts.
inline Parts take_parts(Arena& ws, uint64_t rows, uint64_t cols, int count) {
  Parts p = {{nullptr, nullptr, nullptr}, copy_ld(cols), count};
  for (int i = 0; i < count; ++i) p.part[i] = ws.take(rows * p.ld * 2);
  return p;
}
inline Operand operand(const Parts& p) { return {{p.part[0], p.part[1], p.part[2]}, p.ld}; }
// (of a single row, the stride says nothing and may be anything)
inline Operand operand(const Matrix& m) { return {{m.p, nullptr, nullptr}, m.rows <= 1 ? m.cols : m.ld}; }

// Matrices of one type to be kept as parts, zeros behind their columns: one launch.
struct Copies {
  static constexpr int kMost = 6;
  Matrix from[kMost];
  Parts to[kMost];
  uint64_t begin[kMost + 1];  // workgroups before each
  int n;
};
hipError_t launch_copies(Copies& c, int type, bool half, hipStream_t s);

// A matrix as an operand of `count` parts of bf16 (or fp16 with half): itself
// where that is possible, else a copy.
struct Prepared {
  Operand op;
  Parts copy;
  bool copied;
};
inline Prepared take_operand(Arena& ws, const Matrix& m, int type, int count, bool half, bool copies) {
  Prepared r;
  const bool same = count == 1 && type == (half ? RSX_FLOAT16 : RSX_BFLOAT16);
  r.copied = !same || (copies && !in_place(m));
  // counting, `copies` stands for every matrix: their addresses are not known
  if (!same || (copies && (ws.base == nullptr || r.copied))) r.copy = take_parts(ws, m.rows, m.cols, count);
  r.op = r.copied ? operand(r.copy) : operand(m);
  return r;
}
inline void fill_operand(Copies& c, const Prepared& r, const Matrix& m) {
  if (!r.copied || m.rows == 0 || m.cols == 0) return;
  c.from[c.n] = m;
  c.to[c.n++] = r.copy;
}

}  // namespace rsx
