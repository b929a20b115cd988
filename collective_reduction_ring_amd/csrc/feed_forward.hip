// The gated feed-forward block and its gradients.
//
//   g = x Wg^T, u = x Wu^T, s = act(g) * u, y = s Wd^T
//   ds = dy Wd, dg = ds * u * act'(g), du = ds * act(g)
//   dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x, dWd = dy^T s
//
// Both projections, the activation and the product are one launch: a tile of
// the double product has the same columns of g and of u in one lane's registers.
// So are ds and what it makes: its epilogue reads g and u, and leaves dg, du and
// s.  dx is one product whose k runs through both matrices.  No matrix is
// transposed in memory.
//
// What is rounded: s (and dg, du) to the matrices' type, as the next product's
// operand (s in two parts of it, where w_down is small); in fp32 they are kept
// whole, as three bf16 parts.  g and u stay fp32 for the gradient: rounded to bf16 as
// well, they leave the weights' gradients off by 3.5e-3 (rms) where one rounding of an
// operand and one of the result leave 2.4e-3; their way through memory costs 3% more
// time (8192 x 4096 x 11008).
//
// The time is the tile products'.  8192 x 4096 x 11008 bf16: both projections 1240 us
// (200 of them the writes of g, u and s), down 530 (1410 TFLOP/s), ds 860 (1.26 GB
// through its epilogue), dx 1050, a weight gradient 594 (1244 TFLOP/s).
#include "few_rows.h"
#include "product_store.h"

namespace rsx {
namespace {

template <int N>
struct Slope {
  typename Vec<float, N>::type value, slope;
};

// 1 / (1 + exp(-z)) and the rest to 1, each with all its digits, in some fifteen
// instructions: the exponential of -|z| by powers of two, with what the argument's
// rounding took put back, and the hardware's reciprocal (one step off at most).
// (8192 x 4096 x 11008: the launches with the two epilogues take 1259 and 756 us, with
// the library's exponential and divisions 1269 and 779; gelu, with the library's erfc
// and exponential, 1315 and 803.)
struct Logistic {
  float p, rest;
};
__device__ __forceinline__ Logistic logistic(float z) {
  // exp(-104) is below the smallest number; the maximum of a NaN is NaN (fmaxf's would be the number)
  const float a = __builtin_elementwise_maximum(-fabsf(z), -104.0f), t = a * 1.44269504f;
  const float lost = fmaf(a, 1.44269504f, -t) + a * 1.92596299e-8f;  // log2 e is the sum of the two
  const float e = __builtin_amdgcn_exp2f(t), x = fmaf(e, lost * 0.693147181f, e);
  const float large = __builtin_amdgcn_rcpf(1.0f + x), small = x * large;
  return z >= 0.0f ? Logistic{large, small} : Logistic{small, large};
}

// act(x) and act'(x), elementwise, in fp32.
template <bool SLOPE, int N>
__device__ __forceinline__ Slope<N> activation(int act, typename Vec<float, N>::type x) {
  Slope<N> r;
  switch (act) {
    case RSX_ACT_RELU:
#pragma unroll
      for (int e = 0; e < N; ++e) {
        r.value[e] = x[e] > 0.0f || x[e] != x[e] ? x[e] : 0.0f;
        if (SLOPE) r.slope[e] = x[e] > 0.0f ? 1.0f : x[e] != x[e] ? x[e] : 0.0f;
      }
      break;
    case RSX_ACT_GELU:  // x Phi(x); erfc keeps the digits of Phi far below 0
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float phi = 0.5f * erfcf(x[e] * -0.70710678118654752f);
        r.value[e] = x[e] * phi;
        if (SLOPE) r.slope[e] = phi + x[e] * (0.39894228040143268f * expf(-0.5f * x[e] * x[e]));
      }
      break;
    case RSX_ACT_GELU_TANH:  // (1 + tanh z) / 2 = 1 / (1 + exp(-2z))
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float q = x[e] * x[e];
        const Logistic z = logistic(1.5957691216057308f * x[e] * (1.0f + 0.044715f * q));
        r.value[e] = x[e] * z.p;
        if (SLOPE) {  // p (1 - p) z' x; far out the first two are 0 and x^3 may not be finite
          const float t = z.p * z.rest;
          r.slope[e] = t == 0.0f ? z.p : z.p + x[e] * t * (1.5957691216057308f * (1.0f + 3.0f * 0.044715f * q));
        }
      }
      break;
    default:  // RSX_ACT_SILU
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const Logistic z = logistic(x[e]);
        r.value[e] = x[e] * z.p;
        if (SLOPE) r.slope[e] = z.p + x[e] * (z.p * z.rest);
      }
  }
  return r;
}

struct GateArgs {
  Parts s;
  float* s32;  // the few-row form in fp32 keeps s as it is, rows of p.rows
  float* gate;  // null: not kept
  float* up;
  int act;
};

struct Gate {
  typedef GateArgs Args;
  template <class T, int N>
  static __device__ __forceinline__ void one(const GateArgs& e, uint64_t m, uint32_t c, uint32_t n, typename Vec<float, N>::type g,
                                             typename Vec<float, N>::type u) {
    if (e.gate) {
      put<float, N>(e.gate + m * n, c, n, g);
      put<float, N>(e.up + m * n, c, n, u);
    }
    auto s = activation<false, N>(e.act, g).value;
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] *= u[i];
    if constexpr (sizeof(T) == 4) put<float, N>(e.s32 + m * n, c, n, s);
    else put_parts<T, N>(e.s, m, c, n, s);
  }
  template <class T, class TILE, int N>
  static __device__ __forceinline__ void run(const ProductArgs& p, const Where& w, const GateArgs& e,
                                             const f32x4 (&acc)[TILE::TN][N], uint32_t i0, RSX_LDS char* lds) {
    staged<TILE, true, N>(w, acc, i0, lds, [&](uint32_t m, uint32_t c, f32x8 g, f32x8 u) {
      if (m < p.m) one<T, 8>(e, m, c, p.n, g, u);
    });
  }
  template <class T, int RG>
  static __device__ __forceinline__ void few(const FewArgs& p, const GateArgs& e, uint32_t row, uint32_t c, const f32x4 (&v)[2 * RG]) {
    if (row >= p.n) return;
#pragma unroll
    for (int r = 0; r < RG; ++r) one<T, 4>(e, row, c + 16 * r, p.rows, v[r], v[r + RG]);
  }
};

struct GateGradArgs {
  const float* gate;
  const float* up;
  Parts s, dg, du;  // count 0: not wanted
  int act;
};

struct GateGrad {
  typedef GateGradArgs Args;
  template <class T, class TILE, int N>
  static __device__ __forceinline__ void run(const ProductArgs& p, const Where& w, const GateGradArgs& e,
                                             const f32x4 (&acc)[TILE::TN][N], uint32_t i0, RSX_LDS char* lds) {
    staged<TILE, false, N>(w, acc, i0, lds, [&](uint32_t m, uint32_t c, f32x8 ds) {
      if (m >= p.m || c >= ((p.n + 7) & ~7u)) return;
      const uint64_t row = static_cast<uint64_t>(m) * p.n;
      const f32x8 g = get<float, 8>(e.gate + row, c, p.n), u = get<float, 8>(e.up + row, c, p.n);
      const Slope<8> a = activation<true, 8>(e.act, g);
      f32x8 s, dg, du;
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        s[x] = a.value[x] * u[x];
        dg[x] = ds[x] * u[x] * a.slope[x];
        du[x] = ds[x] * a.value[x];
      }
      put_parts<T, 8>(e.s, m, c, p.n, s);
      put_parts<T, 8>(e.dg, m, c, p.n, dg);
      put_parts<T, 8>(e.du, m, c, p.n, du);
    });
  }
};

struct FewStore {
  typedef StoreArgs Args;
  template <class T, int RG>
  static __device__ __forceinline__ void few(const FewArgs& p, const StoreArgs& e, uint32_t row, uint32_t c, const f32x4 (&v)[RG]) {
    if (row >= p.n) return;
#pragma unroll
    for (int r = 0; r < RG; ++r)
      if (c + 16 * r < p.rows) put_as<4>(e.type, e.out, row * e.ld, c + 16 * r, p.rows, v[r]);
  }
};

struct FewSumsArgs {
  float* to;  // [cut][row][column]
};
struct FewSums {
  typedef FewSumsArgs Args;
  template <class T, int RG>
  static __device__ __forceinline__ void few(const FewArgs& p, const FewSumsArgs& e, uint32_t row, uint32_t c, const f32x4 (&v)[RG]) {
    if (row >= p.n) return;
    float* to = e.to + (static_cast<uint64_t>(few_cut(p)) * p.n + row) * p.rows;
#pragma unroll
    for (int r = 0; r < RG; ++r)
      if (c + 16 * r < p.rows) put<float, 4>(to, c + 16 * r, p.rows, v[r]);
  }
};
__global__ __launch_bounds__(256) void few_add(const float* sums, uint32_t cuts, uint32_t rows, uint32_t dim, void* out, uint64_t ld, int type) {
  const uint64_t t = block_id() * 256 + threadIdx.x, all = static_cast<uint64_t>(rows) * dim;
  if (t >= all) return;
  float v = sums[t];
  for (uint32_t c = 1; c < cuts; ++c) v += sums[c * all + t];
  const uint32_t c = static_cast<uint32_t>(t % dim);
  put_as<1>(type, out, t / dim * ld, c, c + 1, typename Vec<float, 1>::type{v});
}
// Whether a call takes the few-row form.  16-bit matrices that the tiles read in
// place are faster there from 33 rows on (4096 x 11008 bf16: 83 us for 32 rows and
// 94 for 33 to 128 in tiles, 122 for 64 here); others would be copied first.
bool few_form(const FeedForwardArgs& a) { return a.rows <= (a.type == RSX_FLOAT32 || a.copies ? kFewRows : 32); }
// Bytes of s in the few-row form: fp32, or two parts.
uint64_t few_product_bytes(const FeedForwardArgs& a) { return (a.rows * copy_ld(a.hidden) * 4 + 255) & ~255ull; }

// Parts of s.  Rounded once to 16 bits, it leaves a bf16 result of any size off by
// 2.35e-3 (rms), in two parts by 1.66e-3, which is the result's own rounding.  The
// second part doubles the down product's operations, or the reads of s with few
// rows.  While w_down has fewer than kSmall elements that is 0.5 to 4 us up to 64 rows,
// 9 at most with 1024 and 16 with 8192 (128 x 512: 6.7, 19.9 and 22.8 us with 1, 1024
// and 8192 rows for 6.1, 15.6 and 18.0; 24 x 7104: 141 with 8192 for 111); with more it
// grows with them (256 x 11008: 336 for 220; 4096 x 11008: 64 for 55.7 with 8 rows, 2120
// for 1590 with 8192).  How many rows a call has plays no part: a row has the same
// digits in any.
constexpr uint64_t kSmall = 1 << 18;
int product_parts(const FeedForwardArgs& a) { return a.type == RSX_FLOAT32 ? 3 : a.dim * a.hidden < kSmall ? 2 : 1; }
// Parts of a matrix of `type` as an operand: fp32 is three bf16 values exactly.
int parts_of(int type) { return type == RSX_FLOAT32 ? 3 : 1; }

ProductArgs sizes(uint64_t m, uint64_t n, uint64_t k) {
  ProductArgs p = {};
  p.m = static_cast<uint32_t>(m);
  p.n = static_cast<uint32_t>(n);
  p.k = static_cast<uint32_t>(k);
  p.batch = 1;
  return p;
}

#define RSX_TRY(x)                        \
  do {                                    \
    const hipError_t st_ = (x);           \
    if (st_ != hipSuccess) return st_;    \
  } while (0)

// Into how many stretches of k the second product's workgroups are cut where its
// rows are too few for the CUs: 256 at least, and 1024 k a stretch.  (192 rows of
// 26577 bf16: 72 us uncut.)
uint32_t few_cuts(uint64_t dim, uint64_t hidden) {
  const uint64_t groups = (dim + 15) / 16, most = hidden / 1024, cuts = groups ? kCus / groups : 0;
  return static_cast<uint32_t>(cuts < 2 || most < 2 ? 1 : cuts < most ? cuts : most);
}

template <class T>
hipError_t few(const FeedForwardArgs& a, void* s, hipStream_t stream) {
  const uint64_t rest = a.rows * copy_ld(a.hidden);
  GateArgs e = {{{s, static_cast<char*>(s) + rest * 2, nullptr}, copy_ld(a.hidden), product_parts(a)}, static_cast<float*>(s), a.gate, a.up, a.act};
  FewArgs p = {a.x.p, a.w_gate.p, a.w_up.p, a.x.ld, a.w_gate.ld, a.w_up.ld, static_cast<uint32_t>(a.rows),
               static_cast<uint32_t>(a.hidden), static_cast<uint32_t>(a.dim)};
  if (a.hidden) RSX_TRY((launch_few<T, 1, true, Gate>(p, e, stream)));
  p = {s, a.w_down.p, nullptr, sizeof(T) == 4 ? a.hidden : copy_ld(a.hidden), a.w_down.ld, 0, static_cast<uint32_t>(a.rows),
       static_cast<uint32_t>(a.dim), static_cast<uint32_t>(a.hidden), 0, rest};
  const uint32_t cuts = few_cuts(a.dim, a.hidden);
  constexpr bool CAN = sizeof(T) == 2;
  const bool two = CAN && product_parts(a) == 2;
  if (cuts == 1) {
    const StoreArgs to = {a.out, a.out_ld, a.type, nullptr, nullptr, 0};
    return two ? launch_few<T, 1, false, FewStore, CAN>(p, to, stream) : launch_few<T, 1, false, FewStore>(p, to, stream);
  }
  float* sums = reinterpret_cast<float*>(static_cast<char*>(s) + few_product_bytes(a));
  p.cuts = cuts;
  RSX_TRY((two ? launch_few<T, 1, false, FewSums, CAN>(p, {sums}, stream) : launch_few<T, 1, false, FewSums>(p, {sums}, stream)));
  return launch(few_add, grid_of((a.rows * a.dim + 255) / 256), 256, 0, stream, sums, cuts, static_cast<uint32_t>(a.rows),
                static_cast<uint32_t>(a.dim), a.out, a.out_ld, a.type);
}

struct Forward {
  Prepared x, wg, wu, wd;
  Parts s;
  Schedule gate;
  void* split;
};
Forward plan(const FeedForwardArgs& a, Arena& ws) {
  Forward f = {};
  const int n = parts_of(a.type);
  const bool half = a.type == RSX_FLOAT16;
  f.x = take_operand(ws, a.x, a.type, n, half, a.copies);
  f.wg = take_operand(ws, a.w_gate, a.type, n, half, a.copies);
  f.wu = take_operand(ws, a.w_up, a.type, n, half, a.copies);
  f.wd = take_operand(ws, a.w_down, a.type, n, half, a.copies);
  const int ns = product_parts(a);
  f.s = take_parts(ws, a.rows, a.hidden, ns);
  const uint64_t segs = segments_of(n, n), split = store_ws(a.rows, a.dim, a.hidden, segments_of(ns, n));
  f.gate = schedule(a.rows, 2 * a.hidden, 1, steps_of(a.dim, segs), false, false);
  f.split = ws.take(split > f.gate.bytes ? split : f.gate.bytes);
  return f;
}

struct Backward {
  Prepared dout, x, wg, wu, wd;
  Parts s, dg, du;
  Schedule gate;
  void* split;
};
Backward plan(const FeedForwardGradArgs& a, Arena& ws) {
  Backward b = {};
  const int n = parts_of(a.type);
  const bool half = a.type == RSX_FLOAT16;
  b.dout = take_operand(ws, a.dout, a.type, n, half, a.copies);
  b.wd = take_operand(ws, a.w_down, a.type, n, half, a.copies);
  if (a.dw_gate) {
    b.x = take_operand(ws, a.x, a.type, n, half, a.copies);
    b.s = take_parts(ws, a.rows, a.hidden, n);
  }
  if (a.dx) {
    b.wg = take_operand(ws, a.w_gate, a.type, n, half, a.copies);
    b.wu = take_operand(ws, a.w_up, a.type, n, half, a.copies);
  }
  // one above the other, so that the two products with x are one launch
  b.dg = take_parts(ws, 2 * a.rows, a.hidden, n);
  b.du = b.dg;
  if (ws.base != nullptr)
    for (int i = 0; i < n; ++i) b.du.part[i] = static_cast<char*>(b.dg.part[i]) + a.rows * b.dg.ld * 2;
  const uint64_t segs = segments_of(n, n);
  b.gate = schedule(a.rows, a.hidden, 1, steps_of(a.dim, segs), false, false);
  uint64_t split = b.gate.bytes;
  if (a.dx) {
    const uint64_t x = store_ws(a.rows, a.dim, a.hidden, 2 * segs);
    split = split < x ? x : split;
  }
  if (a.dw_gate) {
    const uint64_t g = store_ws(a.hidden, a.dim, a.rows, segs, 2), d = store_ws(a.dim, a.hidden, a.rows, segs);
    split = split < g ? g : split;
    split = split < d ? d : split;
  }
  b.split = ws.take(split);
  return b;
}

}  // namespace

uint64_t feed_forward_ws(const FeedForwardArgs& a) {
  uint64_t few = 0;
  if (few_form(a)) {
    const uint32_t cuts = few_cuts(a.dim, a.hidden);
    few = few_product_bytes(a) + (cuts > 1 ? cuts * a.rows * a.dim * 4 : 0);
    if (!a.copies) return few;
  }
  // what is right for matrices that are copied is right for others too
  FeedForwardArgs b = a;
  b.copies = a.copies && few == 0;
  if (few_form(b)) return few;
  Arena ws(nullptr);
  plan(b, ws);
  return ws.at > few ? ws.at : few;
}

hipError_t launch_feed_forward(const FeedForwardArgs& a, hipStream_t s) {
  if (few_form(a))
    return a.type == RSX_FLOAT32 ? few<float>(a, a.ws, s) : a.type == RSX_BFLOAT16 ? few<bf16_t>(a, a.ws, s) : few<f16_t>(a, a.ws, s);
  const bool half = a.type == RSX_FLOAT16;
  const int n = parts_of(a.type);
  Arena ws(a.ws);
  const Forward f = plan(a, ws);
  Copies c = {};
  fill_operand(c, f.x, a.x);
  fill_operand(c, f.wg, a.w_gate);
  fill_operand(c, f.wu, a.w_up);
  fill_operand(c, f.wd, a.w_down);
  RSX_TRY(launch_copies(c, a.type, half, s));
  ProductArgs p = sizes(a.rows, a.hidden, a.dim);
  add_segments(p, f.x.op, n, f.wg.op, n, &f.wu.op);
  const GateArgs e = {f.s, nullptr, a.gate, a.up, a.act};
  RSX_TRY((half ? launch_product<f16_t, kRow, kRow, true, false, Gate>(p, f.gate, f.split, e, s)
                : launch_product<bf16_t, kRow, kRow, true, false, Gate>(p, f.gate, f.split, e, s)));
  p = sizes(a.rows, a.dim, a.hidden);
  add_segments(p, operand(f.s), product_parts(a), f.wd.op, n);
  return launch_store(half, kNT, p, {a.out, a.out_ld, a.type, nullptr, nullptr, 0}, f.split, s);
}

uint64_t feed_forward_grad_ws(const FeedForwardGradArgs& a) {
  Arena ws(nullptr);
  plan(a, ws);
  return ws.at;
}

hipError_t launch_feed_forward_grad(const FeedForwardGradArgs& a, hipStream_t s) {
  const bool half = a.type == RSX_FLOAT16;
  const int n = parts_of(a.type);
  Arena ws(a.ws);
  const Backward b = plan(a, ws);
  Copies c = {};
  fill_operand(c, b.dout, a.dout);
  fill_operand(c, b.wd, a.w_down);
  if (a.dw_gate) fill_operand(c, b.x, a.x);
  if (a.dx) {
    fill_operand(c, b.wg, a.w_gate);
    fill_operand(c, b.wu, a.w_up);
  }
  RSX_TRY(launch_copies(c, a.type, half, s));
  ProductArgs p = sizes(a.rows, a.hidden, a.dim);
  add_segments(p, b.dout.op, n, b.wd.op, n);
  const GateGradArgs e = {a.gate, a.up, b.s, b.dg, b.du, a.act};
  RSX_TRY((half ? launch_product<f16_t, kRow, kCol, false, false, GateGrad>(p, b.gate, b.split, e, s)
                : launch_product<bf16_t, kRow, kCol, false, false, GateGrad>(p, b.gate, b.split, e, s)));
  if (a.dx) {
    p = sizes(a.rows, a.dim, a.hidden);
    add_segments(p, operand(b.dg), n, b.wg.op, n);
    add_segments(p, operand(b.du), n, b.wu.op, n);
    RSX_TRY(launch_store(half, kNN, p, {a.dx, a.dx_ld, a.type, nullptr, nullptr, 0}, b.split, s));
  }
  if (!a.dw_gate) return hipSuccess;
  p = sizes(a.hidden, a.dim, a.rows);
  add_segments(p, operand(b.dg), n, b.x.op, n);
  p.batch = 2;
  p.batch_a = a.rows * b.dg.ld;
  RSX_TRY(launch_store(half, kTN, p, {a.dw_gate, a.dw_gate_ld, a.weight_type, nullptr, nullptr, a.accumulate, a.dw_up, a.dw_up_ld}, b.split, s));
  p = sizes(a.dim, a.hidden, a.rows);
  add_segments(p, b.dout.op, n, operand(b.s), n);
  return launch_store(half, kTN, p, {a.dw_down, a.dw_down_ld, a.weight_type, nullptr, nullptr, a.accumulate}, b.split, s);
}

}  // namespace rsx
