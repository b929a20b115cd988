// Orthogonalised updates: X0 = G / (|G| + eps), |G| the Frobenius norm, then
// `steps` times A = X X^T, B = b A + c A A, X = a X + B X, with X the matrix or
// its transpose, whichever is wider than tall, so that A is the smaller square.
//
// Each step draws the singular values towards 1 by an odd polynomial; small ones
// grow by a factor of a in each step, 485 in five of the usual coefficients, and
// errors with them: with X, A and B in one 16-bit value each, the update of a
// matrix of low rank and little noise comes out 2% off.  So each is the sum of two
// fp16 values, 22 bits, and a product three products of parts: as near to the
// exact result as fp32 products throughout (rms 5e-5 and 5e-5 of that matrix),
// at the rate of 16-bit matrix instructions.  All three are bounded, and are kept
// times 2^12, the parts' exponents far from either end: values up to 16 fit.
//
// Of a bf16 update the last step multiplies the first parts alone, from a square
// of kSingle on: its roundings are not drawn out any more, and with them the matrix
// above is off by 1.75e-3 (rms) where bf16's own rounding leaves 1.66e-3.  One step
// earlier it would be 2.5e-3.  In a small square few roundings decide, as with any
// common factor: a single vector came out 4.9e-3 off.  For the same reason a small
// square in fp32 has three parts; there the time is the launches'.
//
// A and B are symmetric: only tiles on and below the diagonal are multiplied,
// and stored to both sides.
//
// 11008 x 4096 bf16, a step: A 558 us, B 211, X 911 (1210 TFLOP/s as multiplied); X0
// 115 once.  Of small matrices the time is that of the launches, each waiting for
// the one before: 22 of 4 of 256 x 1024 fp32, 175 us.
#include "product_store.h"

namespace rsx {
namespace {

constexpr float kScale = 4096.0f, kUnscale = 1.0f / 4096.0f;
constexpr uint64_t kSingle = 256, kTriple = 128;
constexpr uint32_t kNormGroups = 512;  // workgroups that sum a matrix's squares, at most

#define RSX_TRY(x)                        \
  do {                                    \
    const hipError_t st_ = (x);           \
    if (st_ != hipSuccess) return st_;    \
  } while (0)

// A stack of matrices as two parts.
struct Stack {
  Parts p;
  uint64_t each;  // elements from one to the next
  __device__ __forceinline__ Parts at(uint32_t i) const {
    Parts r = p;
#pragma unroll
    for (int k = 0; k < 3; ++k) r.part[k] = static_cast<f16_t*>(p.part[k]) + i * each;
    return r;
  }
};

// Sums of squares in fp64: no update's values leave its range.
template <class S>
__global__ __launch_bounds__(256) void square_sums(const S* x, uint64_t ld, uint64_t each, uint32_t rows, uint32_t cols, double* sums) {
  const uint32_t chunks = (cols + 7) / 8;
  const uint64_t all = static_cast<uint64_t>(rows) * chunks;
  const S* m = x + blockIdx.y * each;
  double s = 0.0;
  for (uint64_t t = blockIdx.x * 256ull + threadIdx.x; t < all; t += gridDim.x * 256ull) {
    const auto v = load_row<S, 8, false>(m + t / chunks * ld, static_cast<uint32_t>(t % chunks) * 8, cols);
#pragma unroll
    for (int e = 0; e < 8; ++e) s += static_cast<double>(static_cast<float>(v[e])) * static_cast<double>(static_cast<float>(v[e]));
  }
#pragma unroll
  for (int lanes = 1; lanes < 64; lanes *= 2) s += __shfl_xor(s, lanes);
  __shared__ double part[4];
  if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = s;
  __syncthreads();
  if (threadIdx.x == 0) sums[blockIdx.y * kNormGroups + blockIdx.x] = (part[0] + part[1]) + (part[2] + part[3]);
}

// X0 as parts, of G or (TALL) of its transpose: tiles of 64 x 64 through LDS.
// The rows of A and B are as long as X0 has rows, filled up to 8 with zeros here.
template <class S, bool TALL>
__global__ __launch_bounds__(256) void first_parts(const S* x, uint64_t ld, uint64_t each, uint32_t rows, uint32_t cols,
                                                   const double* sums, uint32_t groups, float eps, Stack to, Stack gram, Stack poly) {
  __shared__ float tile[64][65];
  __shared__ double part[4];
  const uint32_t t = threadIdx.x, m = blockIdx.z;
  double s = 0.0;
  for (uint32_t i = t; i < groups; i += 256) s += sums[m * kNormGroups + i];
#pragma unroll
  for (int lanes = 1; lanes < 64; lanes *= 2) s += __shfl_xor(s, lanes);
  if (t % 64 == 0) part[t / 64] = s;
  const S* g = x + m * each;
  const uint32_t n = TALL ? cols : rows, wide = TALL ? rows : cols;  // of X0
  const uint32_t r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;         // of X0
  for (uint32_t i = t / 64; i < 64; i += 4) {
    const uint32_t r = (TALL ? c0 : r0) + i, c = (TALL ? r0 : c0) + t % 64;  // of G
    const float v = r < rows && c < cols ? static_cast<float>(g[r * ld + c]) : 0.0f;
    if (TALL) tile[t % 64][i] = v;
    else tile[i][t % 64] = v;
  }
  __syncthreads();
  // in fp64 up to the last rounding: |G| and G may both be far from 1
  const double by = static_cast<double>(kScale) / (sqrt((part[0] + part[1]) + (part[2] + part[3])) + static_cast<double>(eps));
  const Parts p = to.at(m);
  for (uint32_t i = t / 16; i < 64; i += 16) {
    const uint32_t r = r0 + i, c = c0 + t % 16 * 4;
    if (r >= n) break;
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = static_cast<float>(static_cast<double>(tile[i][t % 16 * 4 + e]) * by);
    put_parts<f16_t, 4>(p, r, c, wide, v);
  }
  if (blockIdx.x == 0 && n % 8 != 0 && t < 64 && r0 + t < n) {
    const Parts ga = gram.at(m), po = poly.at(m);
    for (uint32_t c = n; c < ((n + 7) & ~7u); ++c)
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        if (i >= ga.count) break;
        static_cast<f16_t*>(ga.part[i])[(r0 + t) * ga.ld + c] = 0.0f;
        static_cast<f16_t*>(po.part[i])[(r0 + t) * po.ld + c] = 0.0f;
      }
  }
}

// A symmetric matrix of `size` rows gets v at (m, n ..), what is on and below the
// diagonal, and then the same values at (n, m ..), what is above.  The sums above
// the diagonal in its own tiles are left: their parts' products add up in another
// order, and a value is written once.
template <bool ABOVE>
__device__ __forceinline__ void put_half(const Parts& p, uint32_t row, uint32_t col, uint32_t size, f32x8 v) {
  typedef Vec<f16_t, 8>::type V;
  if (row >= size || (ABOVE ? col + 7 <= row || col >= size : col > row)) return;
  const uint64_t at = row * p.ld + col;
  const bool whole = ABOVE ? col > row && col + 7 < size : col + 7 <= row;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if (i >= p.count) break;
    const V h = __builtin_convertvector(v, V);
    f16_t* a = static_cast<f16_t*>(p.part[i]) + at;
    if (whole) {
      *reinterpret_cast<V*>(a) = h;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (ABOVE ? col + e > row && col + e < size : col + e <= row) a[e] = h[e];
    }
    const f32x8 back = __builtin_convertvector(h, f32x8);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = fabsf(back[e]) < INFINITY ? v[e] - back[e] : 0.0f;
  }
}

struct GramArgs {
  Stack to;
};
struct Gram {
  typedef GramArgs Args;
  template <class T, class TILE, int N>
  static __device__ __forceinline__ void run(const ProductArgs& p, const Where& w, const GramArgs& e,
                                             const f32x4 (&acc)[TILE::TN][N], uint32_t i0, RSX_LDS char* lds) {
    const Parts to = e.to.at(w.batch);
    staged<TILE, false, N>(
        w, acc, i0, lds,
        [&](uint32_t m, uint32_t n, f32x8 v) {
          v *= kUnscale;
          put_half<false>(to, m, n, p.m, v);
          return v;
        },
        [&](uint32_t m, uint32_t n, f32x8 v) { put_half<true>(to, n, m, p.m, v); });
  }
};

struct PolyArgs {
  Stack gram, to;
  float b, c;
};
struct Poly {
  typedef PolyArgs Args;
  template <class T, class TILE, int N>
  static __device__ __forceinline__ void run(const ProductArgs& p, const Where& w, const PolyArgs& e,
                                             const f32x4 (&acc)[TILE::TN][N], uint32_t i0, RSX_LDS char* lds) {
    const Parts gram = e.gram.at(w.batch), to = e.to.at(w.batch);
    staged<TILE, false, N>(
        w, acc, i0, lds,
        [&](uint32_t m, uint32_t n, f32x8 v) {
          if (m >= p.m || n > m) return v;
          const f32x8 g = get_parts<f16_t, 8>(gram, m, n);  // rows are filled to 8
          v = g * e.b + v * (e.c * kUnscale);
          put_half<false>(to, m, n, p.m, v);
          return v;
        },
        [&](uint32_t m, uint32_t n, f32x8 v) { put_half<true>(to, n, m, p.m, v); });
  }
};

struct ApplyArgs {
  Stack x, to;
  void* out;  // the last step's: null before
  uint64_t ld, each;
  int type, tall;
  float a;
};
struct Apply {
  typedef ApplyArgs Args;
  template <class T, class TILE, int N>
  static __device__ __forceinline__ void run(const ProductArgs& p, const Where& w, const ApplyArgs& e,
                                             const f32x4 (&acc)[TILE::TN][N], uint32_t i0, RSX_LDS char* lds) {
    const Parts x = e.x.at(w.batch), to = e.to.at(w.batch);
    const uint64_t first = w.batch * e.each;
    staged<TILE, false, N>(
        w, acc, i0, lds,
        [&](uint32_t m, uint32_t n, f32x8 v) {
          if (m >= p.m || n >= ((p.n + 7) & ~7u)) return v;
          v = get_parts<f16_t, 8>(x, m, n) * e.a + v * kUnscale;
          if (e.out == nullptr) {
            put_parts<f16_t, 8>(to, m, n, p.n, v);
          } else {
            v *= kUnscale;
            if (!e.tall && n < p.n) put_as<8>(e.type, e.out, first + m * e.ld, n, p.n, v);
          }
          return v;
        },
        [&](uint32_t m, uint32_t n, f32x8 v) {
          if (m < p.m && n < p.n) put_as<8>(e.type, e.out, first + n * e.ld, m, p.m, v);
        },
        e.out != nullptr && e.tall);
  }
};

struct Space {
  double* sums;
  Stack x, y, gram, poly;
  void* pieces;
};
// The schedules of a step's products of `parts` parts.
struct Spread {
  Schedule gram, poly, apply;
  uint64_t bytes() const {
    const uint64_t b = gram.bytes < poly.bytes ? poly.bytes : gram.bytes;
    return b < apply.bytes ? apply.bytes : b;
  }
};
Spread spread(uint64_t batch, uint64_t n, uint64_t wide, int parts) {
  const uint64_t segs = segments_of(parts, parts);
  return {schedule(n, n, batch, steps_of(wide, segs), true, true), schedule(n, n, batch, steps_of(n, segs), true, true),
          schedule(n, wide, batch, steps_of(n, segs), false, true)};
}
Stack take_stack(Arena& ws, uint64_t batch, uint64_t rows, uint64_t cols, int parts) {
  Stack s = {};
  s.p = take_parts(ws, batch * rows, cols, parts);
  s.each = rows * s.p.ld;
  return s;
}
int parts_of(uint64_t n, int type) { return type == RSX_FLOAT32 && n < kTriple ? 3 : 2; }
Space plan(Arena& ws, uint64_t batch, uint64_t n, uint64_t wide, int parts) {
  Space p;
  p.sums = static_cast<double*>(ws.take(batch * kNormGroups * sizeof(double)));
  p.x = take_stack(ws, batch, n, wide, parts);
  p.y = take_stack(ws, batch, n, wide, parts);
  p.gram = take_stack(ws, batch, n, n, parts);
  p.poly = take_stack(ws, batch, n, n, parts);
  const uint64_t one = spread(batch, n, wide, 1).bytes(), all = spread(batch, n, wide, parts).bytes();
  p.pieces = ws.take(one < all ? all : one);
  return p;
}

template <int LB, bool TRIANGLE, class EPILOGUE>
hipError_t multiply(ProductArgs p, const Stack& a, const Stack& b, int parts, const Schedule& c, void* pieces,
                    const typename EPILOGUE::Args& e, hipStream_t s) {
  add_segments(p, operand(a.p), parts, operand(b.p), parts);
  p.batch_a = a.each;
  p.batch_b = b.each;
  return c.tile == 2 ? launch_tiles<f16_t, Small, kRow, LB, false, TRIANGLE, EPILOGUE>(p, c, pieces, e, s)
                     : launch_product<f16_t, kRow, LB, false, TRIANGLE, EPILOGUE>(p, c, pieces, e, s);
}

template <class S>
hipError_t start(const NewtonSchulzArgs& a, const Space& w, uint64_t n, uint64_t wide, bool tall, hipStream_t s) {
  const uint64_t chunks = (a.rows * ((a.cols + 7) / 8) + 255) / 256;
  const uint32_t groups = static_cast<uint32_t>(chunks < kNormGroups ? chunks : kNormGroups);
  const S* x = static_cast<const S*>(a.x);
  const uint32_t rows = static_cast<uint32_t>(a.rows), cols = static_cast<uint32_t>(a.cols);
  RSX_TRY(launch(square_sums<S>, dim3(groups, static_cast<uint32_t>(a.batch)), 256, 0, s, x, a.x_ld, a.x_batch, rows, cols, w.sums));
  const dim3 grid(static_cast<uint32_t>((wide + 63) / 64), static_cast<uint32_t>((n + 63) / 64), static_cast<uint32_t>(a.batch));
  return tall ? launch(first_parts<S, true>, grid, 256, 0, s, x, a.x_ld, a.x_batch, rows, cols, w.sums, groups, a.eps, w.x, w.gram, w.poly)
              : launch(first_parts<S, false>, grid, 256, 0, s, x, a.x_ld, a.x_batch, rows, cols, w.sums, groups, a.eps, w.x, w.gram, w.poly);
}

}  // namespace

uint64_t newton_schulz_ws(uint64_t batch, uint64_t rows, uint64_t cols) {
  const uint64_t n = rows < cols ? rows : cols, wide = rows < cols ? cols : rows;
  uint64_t most = 0;  // of any type
  for (const int parts : {2, n < kTriple ? 3 : 2}) {
    Arena ws(nullptr);
    plan(ws, batch, n, wide, parts);
    most = most < ws.at ? ws.at : most;
  }
  return most;
}

hipError_t launch_newton_schulz(const NewtonSchulzArgs& a, hipStream_t s) {
  const bool tall = a.rows > a.cols;
  const uint64_t n = tall ? a.cols : a.rows, wide = tall ? a.rows : a.cols;
  Arena ws(a.ws);
  const int all = parts_of(n, a.type);
  const Space w = plan(ws, a.batch, n, wide, all);
  RSX_TRY(a.type == RSX_FLOAT32    ? start<float>(a, w, n, wide, tall, s)
          : a.type == RSX_BFLOAT16 ? start<bf16_t>(a, w, n, wide, tall, s) : start<f16_t>(a, w, n, wide, tall, s));
  Stack x = w.x, y = w.y;
  for (int step = 0; step < a.steps; ++step) {
    const bool last = step + 1 == a.steps;
    const int parts = last && step != 0 && n >= kSingle && a.type == RSX_BFLOAT16 ? 1 : all;  // a single step is the first one too
    const Spread c = spread(a.batch, n, wide, parts);
    ProductArgs p = {};
    p.batch = static_cast<uint32_t>(a.batch);
    p.m = p.n = static_cast<uint32_t>(n);
    p.k = static_cast<uint32_t>(wide);
    RSX_TRY((multiply<kRow, true, Gram>(p, x, x, parts, c.gram, w.pieces, {w.gram}, s)));
    p.k = static_cast<uint32_t>(n);
    RSX_TRY((multiply<kRow, true, Poly>(p, w.gram, w.gram, parts, c.poly, w.pieces, {w.gram, w.poly, a.b, a.c}, s)));
    p.n = static_cast<uint32_t>(wide);
    RSX_TRY((multiply<kCol, false, Apply>(p, w.poly, x, parts, c.apply, w.pieces, {x, y, last ? a.out : nullptr, a.out_ld, a.out_batch, a.type, tall, a.a}, s)));
    const Stack t = x;
    x = y;
    y = t;
  }
  return hipSuccess;
}

}  // namespace rsx
