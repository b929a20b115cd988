// Layer norm forward and backward, and the 8-bit checkpoints of its input.
//
//   mean = sum x / D,  rstd = (sum (x - mean)^2 / D + eps)^(-1/2),
//   xhat = (x - mean) rstd,  y = xhat w + b;
//   g = dy w,  dx = rstd (g - mean(g) - xhat mean(g xhat)),
//   dw = sum over rows of dy xhat,  db = sum over rows of dy.
//
// Everything is held in fp32 and rounded once, at the store.  All kernels
// here are bound by HBM: a row is read once into registers, its sums are taken
// there (the variance from the differences, and for a large mean the mean's own
// error too, so no digits are lost to it), and the result is written from them.
// Measured: 32768 rows of 4096 bf16 forward 91 us (5.9 TB/s), backward 139 us
// (5.8 TB/s); rows that are no multiple of 16 bytes share cache lines and run at
// 4.3 to 5 TB/s.
#include "step_device.h"

namespace rsx {
namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------- forward
// A row of values from about 1e16 on may have finite differences whose squares
// overflow: their sum is then taken again over differences scaled by 2^-80, which
// all are numbers.  A sum that is none is taken again of values scaled by 2^-32.
// The tests are the same for every lane of the row; a row that has an infinity or
// a NaN stays without a number.
constexpr float kScaleDown = 0x1p-80f, kSumDown = 0x1p-32f;
__device__ __forceinline__ bool squares_overflow(float sq, float mean) {
  return sq == INFINITY && fabsf(mean) < INFINITY;
}
__device__ __forceinline__ bool is_number(float v) { return fabsf(v) < INFINITY; }
// The mean as one sum gives it; the product as it is rounded, everywhere:
// contracted into a difference it would be another mean there.
__device__ __forceinline__ float first_mean(float sum, float inv_dim) { return fresh(sum * inv_dim); }
// That mean is off by roundings of its own size: the 30 values 1e4 had a mean of
// 10000.001, and y 0.3 for 0.  Where it is larger than the spread, the mean of
// the differences from it, whose roundings are of the spread's size, is taken out
// of it and of them.  Smaller means are off by no more than the differences are
// (16384 rows of 4096 bf16: 46.9 us, with that sum in every row 49.0; rows that
// all need it: 16384 of 8000 bf16 100 us for 95, 8192 of 30000 248 for 225).
__device__ __forceinline__ bool mean_is_large(float first, float sq, float inv_dim, float factor) {
  const float m = first * factor;
  return m * m > sq * inv_dim;
}
// The difference from the first mean, scaled; `first` is scaled already.  Exact
// scalings by powers of two, so one rounding.
__device__ __forceinline__ float difference(float x, float factor, float first) { return fmaf(x, factor, -first); }
struct Centre {
  float mean, rstd;
  float scale, shift;  // xhat = difference * scale + shift
};
// off: the mean of the differences, sq: the sum of their squares.
__device__ __forceinline__ Centre centre(float first, float off, float sq, float inv_dim, float eps, float factor) {
  const float left = fmaf(-off, off, sq * inv_dim), var = left < 0.0f ? 0.0f : left;  // a NaN stays
  const float scale = 1.0f / sqrtf(var + eps * factor * factor);
  return {first + (factor == 1.0f ? off : off * (1.0f / kScaleDown)), scale * factor, scale, -off * scale};
}

// G lanes share R rows; each holds EPL elements of each, vectors of E at
// (j * G + lane) * E.  Up to G = 64 a row is in one wave: no barrier, and
// several groups in a workgroup.  A lane's rows share the weights' loads.
// Single rows of 16 elements a lane are the few ones: eight waves to a SIMD, all
// of a CU's at once (2048 rows of 4096 fp32: 11.7 us, with seven 14.2).
template <class T, class W, int G, int EPL, int R>
__global__ __launch_bounds__(G > 64 ? G : kThreads, R == 1 && EPL == 16 && G <= 256 ? 8 : 1) void norm_kernel(NormArgs a) {
  constexpr int E = 16 / sizeof(T);
  constexpr int V = EPL / E;
  constexpr int kGroups = G > 64 ? 1 : kThreads / G;
  typedef Vec<T, E> X;
  __shared__ float slots[2][R][16];
  const uint32_t dim = static_cast<uint32_t>(a.dim);
  const uint64_t row = (block_id() * kGroups + sub_row<G, kGroups * G>()) * R;
  if (row >= a.rows) return;  // all the lanes of a row
  const uint32_t lane = threadIdx.x % G;

  typename X::type raw[R][V];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    // Past the last row it once more, with nothing stored.
    const T* x = static_cast<const T*>(a.x) + min(row + k, a.rows - 1) * a.x_stride;
#pragma unroll
    for (int j = 0; j < V; ++j) raw[k][j] = load_in<T, E>(x, (j * G + lane) * E, dim);
  }

  const float inv_dim = 1.0f / static_cast<float>(dim);
  float sum[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    sum[k] = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      raw[k][j] = in_place<T, E>(raw[k][j], (j * G + lane) * E, dim);
      const typename X::wide f = widen<T, E>(raw[k][j]);
#pragma unroll
      for (int i = 0; i < E; ++i) sum[k] += f[i];
    }
  }
  int turn = 0;
  group_sum<G, R>(sum, slots[turn]);
  float first[R], sq[R], off[R], factor[R];
  bool lost = false;
#pragma unroll
  for (int k = 0; k < R; ++k) {
    first[k] = first_mean(sum[k], inv_dim);
    factor[k] = 1.0f;
    off[k] = 0.0f;
    lost = lost || !is_number(sum[k]);
  }
  // Behind a branch: kept over it in 32 bits, a row takes twice the registers
  // (16384 rows of 8000 bf16: 102 us, so 95).
  auto widen_anew = [&] {
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) raw[k][j] = fresh(raw[k][j]);
  };
  if (lost) {
    float part[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      part[k] = 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const typename X::wide f = widen<T, E>(raw[k][j]);
#pragma unroll
        for (int i = 0; i < E; ++i) part[k] = fmaf(f[i], kSumDown, part[k]);
      }
    }
    turn ^= 1;
    group_sum<G, R>(part, slots[turn]);
#pragma unroll
    for (int k = 0; k < R; ++k)
      if (!is_number(sum[k])) first[k] = first_mean(part[k], inv_dim) * (1.0f / kSumDown);
  }
  // Not of the longest rows, of which a CU has one workgroup anyway (8192 rows of
  // 30000 bf16: 236 us, so 226).
  if constexpr (EPL < 32 && sizeof(T) == 2) widen_anew();

  // The first time without the factors: they are 1.
  auto squares = [&](bool scaled) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      sq[k] = 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint32_t e = (j * G + lane) * E;
        typename X::wide f = widen<T, E>(raw[k][j]);
#pragma unroll
        for (int i = 0; i < E; ++i) f[i] = scaled ? difference(f[i], factor[k], first[k] * factor[k]) : f[i] - first[k];
        if (e + E <= dim) {
#pragma unroll
          for (int i = 0; i < E; ++i) sq[k] = fmaf(f[i], f[i], sq[k]);
        } else {
#pragma unroll
          for (int i = 0; i < E; ++i)
            if (e + i < dim) sq[k] = fmaf(f[i], f[i], sq[k]);
        }
      }
    }
    turn ^= 1;
    group_sum<G, R>(sq, slots[turn]);
  };
  squares(false);
  bool over = false;
#pragma unroll
  for (int k = 0; k < R; ++k)
    if (squares_overflow(sq[k], first[k])) {
      factor[k] = kScaleDown;
      over = true;
    }
  if (over) {
    widen_anew();
    squares(true);
  }
  // The same for all the lanes of a row, and for a workgroup where they exchange.
  bool any = false;
#pragma unroll
  for (int k = 0; k < R; ++k) any = any || mean_is_large(first[k], sq[k], inv_dim, factor[k]);
  if (any) {
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const typename X::wide f = widen<T, E>(raw[k][j]);
#pragma unroll
        for (int i = 0; i < E; ++i)
          if ((j * G + lane) * E + i < dim) off[k] += difference(f[i], factor[k], first[k] * factor[k]);
      }
    group_sum<G, R>(off, slots[turn ^ 1]);
#pragma unroll
    for (int k = 0; k < R; ++k)
      off[k] = mean_is_large(first[k], sq[k], inv_dim, factor[k]) ? off[k] * inv_dim : 0.0f;
  }
  widen_anew();
  Centre c[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    c[k] = centre(first[k], off[k], sq[k], inv_dim, a.eps, factor[k]);
    if (lane == 0 && row + k < a.rows) {
      if (a.mean != nullptr) a.mean[row + k] = c[k].mean;
      if (a.rstd != nullptr) a.rstd[row + k] = c[k].rstd;
    }
  }

  const W* w = static_cast<const W*>(a.weight);
  const W* b = static_cast<const W*>(a.bias);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t e = (j * G + lane) * E;
    typename X::wide weight = 1.0f, bias = 0.0f;
    if (w != nullptr) weight = widen<W, E>(load_pair<W, E>(w, e, dim));
    if (b != nullptr) bias = widen<W, E>(load_pair<W, E>(b, e, dim));
#pragma unroll
    for (int k = 0; k < R; ++k) {
      if (row + k >= a.rows) break;
      typename X::wide f = widen<T, E>(raw[k][j]);
      if (a.codes != nullptr) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < E; ++i) m = fmaxf(m, ck_magnitude(f[i]));
        const uint32_t byte = ck_scale_byte(ck_largest<32 / E>(m));
        const float inverse = ck_inverse(byte);
        typename Vec<int8_t, E>::type q;
#pragma unroll
        for (int i = 0; i < E; ++i) q[i] = ck_code(f[i], inverse);
        store_row<int8_t, E>(a.codes + (row + k) * a.dim, e, dim, q);
        if (e % kCkBlock == 0 && e < dim)
          a.scales[(row + k) * ck_blocks(a.dim) + e / kCkBlock] = static_cast<uint8_t>(byte);
      }
#pragma unroll
      for (int i = 0; i < E; ++i)
        f[i] = fmaf(difference(f[i], factor[k], first[k] * factor[k]), c[k].scale, c[k].shift) * weight[i] + bias[i];
      store_row<T, E>(static_cast<T*>(a.y) + (row + k) * a.y_stride, e, dim, narrow<T, E>(f));
    }
  }
}

// Rows too long for the registers, or too short for a vector: a workgroup reads
// its row three times, with a large mean four, after the first from the caches.
template <class T, class W>
__global__ __launch_bounds__(1024) void norm_long_kernel(NormArgs a) {
  constexpr int E = 16 / sizeof(T);
  constexpr uint32_t kStep = 1024 * E;
  typedef Vec<T, E> X;
  __shared__ float slots[2][1][16];
  const uint32_t dim = static_cast<uint32_t>(a.dim);
  const uint64_t row = block_id();
  if (row >= a.rows) return;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const float inv_dim = 1.0f / static_cast<float>(dim);

  float sum[1] = {0.0f};
  for (uint32_t e = threadIdx.x * E; e < dim; e += kStep) {
    const typename X::wide f = widen<T, E>(load_row<T, E, false>(x, e, dim));
#pragma unroll
    for (int i = 0; i < E; ++i) sum[0] += f[i];
  }
  int turn = 0;
  group_sum<1024, 1>(sum, slots[turn]);
  float first = first_mean(sum[0], inv_dim);
  if (!is_number(sum[0])) {
    float part[1] = {0.0f};
    for (uint32_t e = threadIdx.x * E; e < dim; e += kStep) {
      const typename X::wide f = widen<T, E>(load_row<T, E, false>(x, e, dim));
#pragma unroll
      for (int i = 0; i < E; ++i) part[0] = fmaf(f[i], kSumDown, part[0]);
    }
    turn ^= 1;
    group_sum<1024, 1>(part, slots[turn]);
    first = first_mean(part[0], inv_dim) * (1.0f / kSumDown);
  }

  float sq[1], off[1] = {0.0f}, factor = 1.0f;
  for (;;) {
    sq[0] = 0.0f;
    for (uint32_t e = threadIdx.x * E; e < dim; e += kStep) {
      const typename X::wide f = widen<T, E>(load_row<T, E, false>(x, e, dim));
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float d = difference(f[i], factor, first * factor);
        if (e + i < dim) sq[0] = fmaf(d, d, sq[0]);
      }
    }
    turn ^= 1;
    group_sum<1024, 1>(sq, slots[turn]);
    if (factor != 1.0f || !squares_overflow(sq[0], first)) break;
    factor = kScaleDown;
  }
  if (mean_is_large(first, sq[0], inv_dim, factor)) {  // the same for the workgroup
    for (uint32_t e = threadIdx.x * E; e < dim; e += kStep) {
      const typename X::wide f = widen<T, E>(load_row<T, E, false>(x, e, dim));
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (e + i < dim) off[0] += difference(f[i], factor, first * factor);
    }
    group_sum<1024, 1>(off, slots[turn ^ 1]);
    off[0] *= inv_dim;
  }
  const Centre c = centre(first, off[0], sq[0], inv_dim, a.eps, factor);
  if (threadIdx.x == 0) {
    if (a.mean != nullptr) a.mean[row] = c.mean;
    if (a.rstd != nullptr) a.rstd[row] = c.rstd;
  }
  const W* w = static_cast<const W*>(a.weight);
  const W* b = static_cast<const W*>(a.bias);
  T* y = static_cast<T*>(a.y) + row * a.y_stride;
  // Whole steps for every lane: the lanes of a checkpoint block stay together.
  for (uint32_t at = 0; at < dim; at += kStep) {
    const uint32_t e = at + threadIdx.x * E;
    typename X::wide f = widen<T, E>(load_row<T, E, false>(x, e, dim));
    if (a.codes != nullptr) {
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < E; ++i) m = fmaxf(m, ck_magnitude(f[i]));
      const uint32_t byte = ck_scale_byte(ck_largest<32 / E>(m));
      const float inverse = ck_inverse(byte);
      typename Vec<int8_t, E>::type q;
#pragma unroll
      for (int i = 0; i < E; ++i) q[i] = ck_code(f[i], inverse);
      store_row<int8_t, E>(a.codes + row * a.dim, e, dim, q);
      if (e % kCkBlock == 0 && e < dim) a.scales[row * ck_blocks(a.dim) + e / kCkBlock] = static_cast<uint8_t>(byte);
    }
#pragma unroll
    for (int i = 0; i < E; ++i) f[i] = fmaf(difference(f[i], factor, first * factor), c.scale, c.shift);
    if (w != nullptr) f *= widen<W, E>(load_row<W, E, false>(w, e, dim));
    if (b != nullptr) f += widen<W, E>(load_row<W, E, false>(b, e, dim));
    store_row<T, E>(y, e, dim, narrow<T, E>(f));
  }
}

// --------------------------------------------------------------- backward
// A row's input as the backward pass finds it: its own elements, or 8-bit
// codes and their scale.
template <class T, int E, bool CK>
struct Input {
  typename Vec<T, E>::type x;
};
template <class T, int E>
struct Input<T, E, true> {
  typename Vec<int8_t, E>::type q;
  uint32_t scale;
};
// IN: rows of at least E elements.
template <class T, int E, bool CK, bool IN = false>
__device__ __forceinline__ Input<T, E, CK> load_input(const NormGradArgs& a, uint64_t row, uint32_t e, uint32_t dim) {
  Input<T, E, CK> v;
  if constexpr (CK) {
    const int8_t* codes = a.codes + row * a.dim;
    v.q = IN ? load_in<int8_t, E>(codes, e, dim) : load_row<int8_t, E>(codes, e, dim);
    v.scale = a.scales[row * ck_blocks(a.dim) + min(e, dim - 1) / kCkBlock];
  } else {
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    v.x = IN ? load_in<T, E>(x, e, dim) : load_row<T, E>(x, e, dim);
  }
  return v;
}
template <class T, int E, bool CK>
__device__ __forceinline__ Input<T, E, CK> input_in_place(Input<T, E, CK> v, uint32_t e, uint32_t dim) {
  if constexpr (CK)
    v.q = in_place<int8_t, E>(v.q, e, dim);
  else
    v.x = in_place<T, E>(v.x, e, dim);
  return v;
}
template <class T, int E, bool CK>
__device__ __forceinline__ typename Vec<T, E>::wide input_value(const Input<T, E, CK>& v) {
  if constexpr (CK) {
    return __builtin_convertvector(v.q, typename Vec<T, E>::wide) * ck_step(v.scale);
  } else {
    return widen<T, E>(v.x);
  }
}

// Workgroups of the backward pass: each keeps the weight gradient of the rows
// it takes in registers and writes one partial row of it at the end.
constexpr uint32_t kGradGroups = 512;

// Each of the K / G groups of G lanes in a workgroup takes R rows at a time,
// and loads its next ones before it exchanges the sums of these.  dw and db
// are summed per workgroup over its rows in order, then over workgroups by
// norm_sum_kernel: a fixed order, whatever the timing.
//
// What bounds it is how much of the rows is on its way while a row's sums are
// exchanged, and that is a question of registers.  So a lane's rows share its
// dw, db and weights; rows and weights are held as they came, and what is made
// of them is made twice; a workgroup of 1024 keeps the weights in LDS, and of
// fp32 rows the input (8192 rows of 16384: 405 us with 68 bytes of a lane
// spilled, 302 us so).
template <class T, class W, int G, int EPL, int K, int R, bool CK>
__global__ __launch_bounds__(K) void norm_grad_kernel(NormGradArgs a, uint32_t pitch) {
  constexpr int E = 16 / sizeof(T);
  constexpr int V = EPL / E;
  constexpr int kGroups = K / G;
  constexpr bool kWeightsInLds = K == 1024;
  constexpr bool kInputInLds = K == 1024 && E == 4 && !CK;
  typedef Vec<T, E> X;
  __shared__ float slots[2][2 * R][16];
  __shared__ float join[kGroups > 1 ? K * EPL : 1];
  __shared__ typename Vec<W, E>::type lds_w[kWeightsInLds ? V : 1][kWeightsInLds ? K : 1];
  __shared__ Input<T, E, CK> lds_x[kInputInLds ? R * V : 1][kInputInLds ? K : 1];
  const uint32_t lane = threadIdx.x % G;
  const uint32_t sub = sub_row<G, K>();
  const uint32_t dim = static_cast<uint32_t>(a.dim);
  const uint64_t step = static_cast<uint64_t>(gridDim.x) * (kGroups * R);
  const T* dy = static_cast<const T*>(a.dy);
  T* dx = static_cast<T*>(a.dx);
  const float inv_dim = 1.0f / static_cast<float>(dim);
  uint64_t row = (static_cast<uint64_t>(blockIdx.x) * kGroups + sub) * R;

  typename Vec<W, E>::type held_w[kWeightsInLds ? 1 : V];
  typename X::wide dw[V], db[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    typename Vec<W, E>::type w = static_cast<W>(1.0f);
    if (a.weight != nullptr)
      w = load_pair<W, E>(static_cast<const W*>(a.weight), (j * G + lane) * E, dim);
    if constexpr (kWeightsInLds)
      lds_w[j][threadIdx.x] = w;  // read by this lane alone
    else
      held_w[j] = w;
    dw[j] = 0.0f;
    db[j] = 0.0f;
  }
  auto weight = [&](int j) {
    if constexpr (kWeightsInLds)
      return widen<W, E>(lds_w[j][fresh(threadIdx.x)]);
    else
      return widen<W, E>(fresh(held_w[j]));
  };

  typename X::type next_dy[R][V];
  Input<T, E, CK> next_x[R][V];
  float next_mean[R], next_rstd[R];
  auto load = [&](uint64_t first) {
    const uint32_t e = fresh(lane * E);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const uint64_t r = min(first + k, a.rows - 1);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        next_x[k][j] = load_input<T, E, CK, true>(a, r, e + j * (G * E), dim);
        next_dy[k][j] = load_in<T, E>(dy + r * a.dy_stride, e + j * (G * E), dim);
      }
      next_mean[k] = a.mean[r];
      next_rstd[k] = a.rstd[r];
    }
  };
  // With one row to a workgroup the loop's condition says as much.
  auto there = [&](int k) { return kGroups * R == 1 || row + k < a.rows; };
  load(row);
  uint32_t turn = 0;
  // The same turns for the whole workgroup: it shares the sums' barrier.
  for (uint64_t first = row - sub * R; first < a.rows; first += step, row += step, turn ^= 1u) {
    typename X::type this_dy[R][V];
    Input<T, E, CK> this_x[R][V];
    float mean[R], rstd[R], s[2 * R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      mean[k] = next_mean[k];
      rstd[k] = next_rstd[k];
      s[2 * k] = s[2 * k + 1] = 0.0f;
      if (!there(k)) mean[k] = rstd[k] = 0.0f;
    }
    const uint32_t e = fresh(lane * E);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const typename X::wide w = weight(j);
#pragma unroll
      for (int k = 0; k < R; ++k) {
        this_dy[k][j] = in_place<T, E>(next_dy[k][j], e + j * (G * E), dim);
        this_x[k][j] = input_in_place<T, E, CK>(next_x[k][j], e + j * (G * E), dim);
        if (!there(k)) {  // past the last row all is 0, and adds nothing
          this_dy[k][j] = static_cast<T>(0.0f);
          this_x[k][j] = {};
        }
        if constexpr (kInputInLds) lds_x[k * V + j][threadIdx.x] = this_x[k][j];
        const typename X::wide d = widen<T, E>(this_dy[k][j]), g = d * w;
        const typename X::wide xhat = (input_value<T, E, CK>(this_x[k][j]) - mean[k]) * rstd[k];
        db[j] += d;
#pragma unroll
        for (int i = 0; i < E; ++i) {
          dw[j][i] = fmaf(d[i], xhat[i], dw[j][i]);
          s[2 * k] += g[i];
          s[2 * k + 1] = fmaf(g[i], xhat[i], s[2 * k + 1]);
        }
      }
    }
    if (first + step < a.rows) load(row + step);
    group_sum<G, 2 * R>(s, slots[turn]);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const typename X::wide w = weight(j);
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const float c1 = s[2 * k] * inv_dim, c2 = s[2 * k + 1] * inv_dim;
        if constexpr (kInputInLds) this_x[k][j] = lds_x[k * V + j][fresh(threadIdx.x)];
        const typename X::wide g = widen<T, E>(fresh(this_dy[k][j])) * w;
        const typename X::wide xhat = (input_value<T, E, CK>(this_x[k][j]) - mean[k]) * rstd[k];
        typename X::wide f;
#pragma unroll
        for (int i = 0; i < E; ++i) f[i] = (g[i] - fmaf(xhat[i], c2, c1)) * rstd[k];
        store_row<T, E>(dx + (row + k) * a.dx_stride, e + j * (G * E), there(k) ? dim : 0u, narrow<T, E>(f));
      }
    }
  }

  // One partial row of dw and one of db for each workgroup.
  float* part = a.partial + static_cast<uint64_t>(blockIdx.x) * 2 * pitch;
#pragma unroll
  for (int k = 0; k < 2; ++k, part += pitch) {
    if constexpr (kGroups > 1) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const uint32_t e = (j * G + lane) * E + i;
          if (e < dim) join[sub * (G * EPL) + e] = k == 0 ? dw[j][i] : db[j][i];
        }
      __syncthreads();
      for (uint32_t e = threadIdx.x; e < dim; e += K) {
        float t = 0.0f;
#pragma unroll
        for (int r = 0; r < kGroups; ++r) t += join[r * (G * EPL) + e];
        part[e] = t;
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) store_row<float, E>(part, (j * G + lane) * E, dim, k == 0 ? dw[j] : db[j]);
    }
  }
}

// Rows too long for the registers: the row's own pass reads x and dy twice,
// and the weight gradient gets a pass by columns (norm_columns_kernel).
template <class T, class W, bool CK>
__global__ __launch_bounds__(1024) void norm_grad_long_kernel(NormGradArgs a) {
  constexpr int E = 16 / sizeof(T);
  constexpr uint32_t kStep = 1024 * E;
  typedef Vec<T, E> X;
  __shared__ float slots[1][2][16];
  const uint32_t dim = static_cast<uint32_t>(a.dim);
  const uint64_t row = block_id();
  if (row >= a.rows) return;
  const T* dy = static_cast<const T*>(a.dy) + row * a.dy_stride;
  const W* weight = static_cast<const W*>(a.weight);
  T* dx = static_cast<T*>(a.dx) + row * a.dx_stride;
  const float inv_dim = 1.0f / static_cast<float>(dim), mean = a.mean[row], rstd = a.rstd[row];
  float s[2] = {0.0f, 0.0f};
  for (uint32_t e = threadIdx.x * E; e < dim; e += kStep) {
    const typename X::wide xhat = (input_value<T, E, CK>(load_input<T, E, CK>(a, row, e, dim)) - mean) * rstd;
    typename X::wide g = widen<T, E>(load_row<T, E, false>(dy, e, dim));
    if (weight != nullptr) g *= widen<W, E>(load_row<W, E, false>(weight, e, dim));
#pragma unroll
    for (int i = 0; i < E; ++i) {
      s[0] += g[i];
      s[1] = fmaf(g[i], xhat[i], s[1]);
    }
  }
  group_sum<1024, 2>(s, slots[0]);
  const float c1 = s[0] * inv_dim, c2 = s[1] * inv_dim;
  for (uint32_t e = threadIdx.x * E; e < dim; e += kStep) {
    const typename X::wide xhat = (input_value<T, E, CK>(load_input<T, E, CK>(a, row, e, dim)) - mean) * rstd;
    typename X::wide g = widen<T, E>(load_row<T, E, false>(dy, e, dim));
    if (weight != nullptr) g *= widen<W, E>(load_row<W, E, false>(weight, e, dim));
#pragma unroll
    for (int i = 0; i < E; ++i) g[i] = (g[i] - fmaf(xhat[i], c2, c1)) * rstd;
    store_row<T, E>(dx, e, dim, narrow<T, E>(g));
  }
}

// Partial rows of dw and db by columns: workgroup (c, p) sums rows p, p + P,
// ... of its kThreads * E columns.  It reads dy before the row pass stores dx,
// which may take dy's place.
template <class T, bool CK>
__global__ __launch_bounds__(kThreads) void norm_columns_kernel(NormGradArgs a, uint32_t pitch, uint32_t parts,
                                                                uint32_t column_groups) {
  constexpr int E = 16 / sizeof(T);
  typedef Vec<T, E> X;
  const uint32_t dim = static_cast<uint32_t>(a.dim);
  const uint32_t block = static_cast<uint32_t>(block_id());  // below 2^30
  const uint32_t e = (block % column_groups * kThreads + threadIdx.x) * E;
  const uint32_t p = block / column_groups;
  if (p >= parts) return;
  typename X::wide dw = 0.0f, db = 0.0f;
  for (uint64_t row = p; row < a.rows; row += parts) {
    const typename X::wide d = widen<T, E>(load_row<T, E>(static_cast<const T*>(a.dy) + row * a.dy_stride, e, dim));
    const typename X::wide xhat =
        (input_value<T, E, CK>(load_input<T, E, CK>(a, row, e, dim)) - a.mean[row]) * a.rstd[row];
    db += d;
#pragma unroll
    for (int i = 0; i < E; ++i) dw[i] = fmaf(d[i], xhat[i], dw[i]);
  }
  float* part = a.partial + static_cast<uint64_t>(p) * 2 * pitch;
  store_row<float, E>(part, e, dim, dw);
  store_row<float, E>(part + pitch, e, dim, db);
}

// dw (the first half of the workgroups) and db from the partial rows: 32 columns
// a workgroup, in 32 parts of the rows; no rows at all give zeros.
template <class W>
__global__ __launch_bounds__(1024) void norm_sum_kernel(const float* partial, uint32_t pitch, uint32_t parts,
                                                        uint32_t dim, W* dweight, W* dbias) {
  __shared__ float join[32][33];
  const uint32_t block = static_cast<uint32_t>(block_id()), groups = (dim + 31) / 32, which = block < groups ? 0u : 1u;
  W* out = which == 0 ? dweight : dbias;
  if (out == nullptr) return;
  const uint32_t column = threadIdx.x % 32, slice = threadIdx.x / 32;
  const uint32_t e = (block - which * groups) * 32 + column;
  float t = 0.0f;
  if (e < dim) {
    const float* p = partial + static_cast<uint64_t>(which) * pitch + e;
#pragma unroll 16
    for (uint32_t r = slice; r < parts; r += 32) t += p[static_cast<uint64_t>(r) * 2 * pitch];
  }
  join[slice][column] = t;
  __syncthreads();
  if (threadIdx.x < 32 && e < dim) {
    float s = 0.0f;
#pragma unroll
    for (int r = 0; r < 32; ++r) s += join[r][column];
    out[e] = static_cast<W>(s);
  }
}

// ------------------------------------------------------------ checkpoints
// A thread has V vectors of 8 elements on their way.  Rows of up to 2048: `lanes`
// threads to a row (a power of two, at least 4: a block's lanes stay together),
// the vectors in V rows.  Longer ones are cut into pieces of 2048, a workgroup
// takes V pieces one after the other, from row to row; lanes is 256.
struct Place {
  uint64_t row;
  uint32_t e;
};
template <int V>
__device__ __forceinline__ void pack_places(Place (&p)[V], uint32_t lanes, uint32_t pieces) {
  const uint64_t block = block_id();
  if (pieces == 1) {
    const uint32_t rows = kThreads / lanes;
#pragma unroll
    for (int k = 0; k < V; ++k) p[k] = {(block * V + k) * rows + threadIdx.x / lanes, threadIdx.x % lanes * 8};
  } else {
    uint64_t row = block * V / pieces;
    uint32_t piece = static_cast<uint32_t>(block * V - row * pieces);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      p[k] = {row, piece * (kThreads * 8) + threadIdx.x * 8};
      const bool last = ++piece == pieces;
      row += last ? 1 : 0;
      piece = last ? 0 : piece;
    }
  }
}

template <class T, int V>
__global__ __launch_bounds__(kThreads) void pack_kernel(PackArgs a, uint32_t lanes, uint32_t pieces) {
  const uint32_t dim = static_cast<uint32_t>(a.dim);
  Place p[V];
  pack_places<V>(p, lanes, pieces);
  typename Vec<T, 8>::type raw[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const T* x = static_cast<const T*>(a.x) + min(p[k].row, a.rows - 1) * a.stride;
    raw[k] = dim >= 8 ? load_wide<T, 8, true>(x, p[k].e, dim) : load_row<T, 8>(x, p[k].e, dim);
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
    if (dim >= 8) raw[k] = wide_in_place<T, 8>(raw[k], p[k].e, dim);
    const typename Vec<T, 8>::wide f = widen<T, 8>(raw[k]);
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, ck_magnitude(f[i]));
    const uint32_t byte = ck_scale_byte(ck_largest<4>(m));
    const float inverse = ck_inverse(byte);
    typename Vec<int8_t, 8>::type q;
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = ck_code(f[i], inverse);
    if (p[k].row >= a.rows) return;
    store_row<int8_t, 8>(a.codes + p[k].row * a.dim, p[k].e, dim, q);
    if (p[k].e % kCkBlock == 0 && p[k].e < dim)
      a.scales[p[k].row * ck_blocks(a.dim) + p[k].e / kCkBlock] = static_cast<uint8_t>(byte);
  }
}

template <class T, int V>
__global__ __launch_bounds__(kThreads) void unpack_kernel(PackArgs a, uint32_t lanes, uint32_t pieces) {
  const uint32_t dim = static_cast<uint32_t>(a.dim);
  Place p[V];
  pack_places<V>(p, lanes, pieces);
  typename Vec<int8_t, 8>::type q[V];
  uint32_t byte[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const uint64_t row = min(p[k].row, a.rows - 1);
    const int8_t* codes = a.codes + row * a.dim;
    q[k] = dim >= 8 ? load_in<int8_t, 8>(codes, p[k].e, dim) : load_row<int8_t, 8>(codes, p[k].e, dim);
    byte[k] = a.scales[row * ck_blocks(a.dim) + min(p[k].e, dim - 1) / kCkBlock];
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
    if (dim >= 8) q[k] = in_place<int8_t, 8>(q[k], p[k].e, dim);
    if (p[k].row >= a.rows) return;
    const typename Vec<T, 8>::wide f = __builtin_convertvector(q[k], typename Vec<T, 8>::wide) * ck_step(byte[k]);
    store_row<T, 8>(static_cast<T*>(a.out) + p[k].row * a.stride, p[k].e, dim, narrow<T, 8>(f));
  }
}

template <class T, int V>
hipError_t checkpoint_go(const PackArgs& a, bool pack, hipStream_t s) {
  uint32_t lanes = 4;
  while (lanes < kThreads && lanes * 8 < a.dim) lanes *= 2;
  const uint32_t pieces = static_cast<uint32_t>((a.dim + kThreads * 8 - 1) / (kThreads * 8));
  const uint64_t rows = kThreads / lanes;  // of one vector of the workgroup; 1 where rows have pieces
  const uint64_t items = (a.rows + rows - 1) / rows * pieces;
  return launch(pack ? pack_kernel<T, V> : unpack_kernel<T, V>, grid_of((items + V - 1) / V), kThreads, 0, s, a, lanes,
                pieces);
}

template <class T>
hipError_t checkpoint(const PackArgs& a, bool pack, hipStream_t s) {
  // 32768 rows of 4096 bf16, both ways: 138 us, with one vector 157; one where
  // there is little to do.
  return a.rows * a.dim < (1u << 21) ? checkpoint_go<T, 1>(a, pack, s) : checkpoint_go<T, 4>(a, pack, s);
}

// --------------------------------------------------------------- launches
// Rows from which on two share a group and its weights' loads (32768 rows of
// 4096 bf16 with fp32 weights: 96 us, one by one 120); fewer leave CUs idle.
// Rows of more than 4096 are their own group's (16384 rows of 8000 bf16: 96 us,
// in pairs 111).
constexpr uint64_t kPairRows = 4096;

template <class T, class W, int G, int EPL, int R = 1>
hipError_t norm_go(const NormArgs& a, hipStream_t s) {
  if constexpr (R > 1)
    if (a.rows < kPairRows) return norm_go<T, W, G, EPL, 1>(a, s);
  constexpr uint32_t kRows = (G > 64 ? 1 : kThreads / G) * R;
  const uint64_t grid = (a.rows + kRows - 1) / kRows;
  return launch(norm_kernel<T, W, G, EPL, R>, grid_of(grid), G > 64 ? G : kThreads, 0, s, a);
}

template <class T, class W>
hipError_t norm(const NormArgs& a, hipStream_t s) {
  if (a.dim < 16 / sizeof(T)) return launch(norm_long_kernel<T, W>, grid_of(a.rows), 1024, 0, s, a);
  // Lanes as the row fills them with 8 to 24 elements each.  More elements and
  // fewer lanes leave too few waves, more lanes wait longer at the barriers
  // (16384 rows of 4096 bf16: 256 lanes 47 us, 64 lanes 71, 512 lanes 62).
  if (a.dim <= 128) return norm_go<T, W, 16, 8, 2>(a, s);
  if (a.dim <= 256) return norm_go<T, W, 32, 8, 2>(a, s);
  if (a.dim <= 512) return norm_go<T, W, 64, 8, 2>(a, s);
  if (a.dim <= 1024) return norm_go<T, W, 64, 16, 2>(a, s);
  if (a.dim <= 2048) return norm_go<T, W, 128, 16, 2>(a, s);
  if (a.dim <= 4096) return norm_go<T, W, 256, 16, 2>(a, s);
  if (a.dim <= 8192) return norm_go<T, W, 512, 16>(a, s);
  if (a.dim <= 12288) return norm_go<T, W, 512, 24>(a, s);
  if (a.dim <= 16384) return norm_go<T, W, 1024, 16>(a, s);
  if (a.dim <= 32768) return norm_go<T, W, 1024, 32>(a, s);
  return launch(norm_long_kernel<T, W>, grid_of(a.rows), 1024, 0, s, a);
}

uint32_t grad_pitch(uint64_t dim) { return static_cast<uint32_t>((dim + 15) / 16 * 16); }
uint32_t grad_parts(uint64_t rows) { return static_cast<uint32_t>(rows < kGradGroups ? rows : kGradGroups); }

template <class T, class W, int G, int EPL, int K, int R, bool CK>
hipError_t grad_go(const NormGradArgs& a, uint32_t pitch, uint32_t* parts, hipStream_t s) {
  constexpr uint64_t kRows = K / G * R;
  *parts = grad_parts((a.rows + kRows - 1) / kRows);
  return launch(norm_grad_kernel<T, W, G, EPL, K, R, CK>, dim3(*parts), K, 0, s, a, pitch);
}

// Rows too long for the registers, or too short for a vector.
template <class T, class W, bool CK>
hipError_t grad_long(const NormGradArgs& a, uint32_t pitch, uint32_t* parts, hipStream_t s) {
  *parts = grad_parts(a.rows);
  const uint32_t per = kThreads * (16 / sizeof(T));
  const uint32_t columns = static_cast<uint32_t>((a.dim + per - 1) / per);
  const hipError_t e = launch(norm_columns_kernel<T, CK>, grid_of(static_cast<uint64_t>(columns) * *parts), kThreads, 0, s, a,
                              pitch, *parts, columns);
  if (e != hipSuccess) return e;
  return launch(norm_grad_long_kernel<T, W, CK>, grid_of(a.rows), 1024, 0, s, a);
}

template <class T, class W, bool CK>
hipError_t norm_grad(const NormGradArgs& a, hipStream_t s) {
  const uint32_t pitch = grad_pitch(a.dim);
  uint32_t parts = 0;
  hipError_t e = hipSuccess;
  if (a.rows != 0) {
    // Few elements to a lane, so that its sums of dw and db leave registers to
    // the rows on their way (16384 rows of 4096 bf16 from a checkpoint: 8
    // elements 83 us, 16 elements 112).
    if (a.dim < 16 / sizeof(T) || a.dim > 16384) {
      e = grad_long<T, W, CK>(a, pitch, &parts, s);
    } else if (a.dim <= 128) {
      e = grad_go<T, W, 16, 8, 256, 2, CK>(a, pitch, &parts, s);
    } else if (a.dim <= 256) {
      e = grad_go<T, W, 32, 8, 256, 2, CK>(a, pitch, &parts, s);
    } else if (a.dim <= 512) {
      e = grad_go<T, W, 64, 8, 256, 2, CK>(a, pitch, &parts, s);
    } else if (a.dim <= 1024) {
      e = grad_go<T, W, 128, 8, 256, 2, CK>(a, pitch, &parts, s);
    } else if (a.dim <= 2048) {
      e = grad_go<T, W, 256, 8, 512, 1, CK>(a, pitch, &parts, s);
    } else if (a.dim <= 4096) {
      e = grad_go<T, W, 512, 8, 512, 1, CK>(a, pitch, &parts, s);
    } else if (a.dim <= 8192) {
      e = grad_go<T, W, 512, 16, 512, 1, CK>(a, pitch, &parts, s);
    } else {
      e = grad_go<T, W, 1024, 16, 1024, 1, CK>(a, pitch, &parts, s);
    }
  }
  if (e != hipSuccess || (a.dweight == nullptr && a.dbias == nullptr)) return e;
  return launch(norm_sum_kernel<W>, grid_of((a.dim + 31) / 32 * 2), 1024, 0, s, a.partial, pitch, parts,
                static_cast<uint32_t>(a.dim), static_cast<W*>(a.dweight), static_cast<W*>(a.dbias));
}

template <class T, class W>
hipError_t norm_grad_by_input(const NormGradArgs& a, hipStream_t s) {
  return a.x == nullptr ? norm_grad<T, W, true>(a, s) : norm_grad<T, W, false>(a, s);
}

}  // namespace

uint64_t layer_norm_grad_ws(uint64_t rows, uint64_t dim) {
  return static_cast<uint64_t>(grad_parts(rows)) * 2 * grad_pitch(dim) * sizeof(float);
}

hipError_t launch_layer_norm(const NormArgs& a, hipStream_t s) {
  if (a.type == RSX_FLOAT32) return norm<float, float>(a, s);
  if (a.type == RSX_BFLOAT16)
    return a.weight_type == RSX_FLOAT32 ? norm<bf16_t, float>(a, s) : norm<bf16_t, bf16_t>(a, s);
  return a.weight_type == RSX_FLOAT32 ? norm<f16_t, float>(a, s) : norm<f16_t, f16_t>(a, s);
}

hipError_t launch_layer_norm_grad(const NormGradArgs& a, hipStream_t s) {
  if (a.type == RSX_FLOAT32) return norm_grad_by_input<float, float>(a, s);
  if (a.type == RSX_BFLOAT16)
    return a.weight_type == RSX_FLOAT32 ? norm_grad_by_input<bf16_t, float>(a, s)
                                        : norm_grad_by_input<bf16_t, bf16_t>(a, s);
  return a.weight_type == RSX_FLOAT32 ? norm_grad_by_input<f16_t, float>(a, s) : norm_grad_by_input<f16_t, f16_t>(a, s);
}

hipError_t launch_checkpoint_pack(const PackArgs& a, hipStream_t s) {
  if (a.type == RSX_FLOAT32) return checkpoint<float>(a, true, s);
  return a.type == RSX_BFLOAT16 ? checkpoint<bf16_t>(a, true, s) : checkpoint<f16_t>(a, true, s);
}
hipError_t launch_checkpoint_unpack(const PackArgs& a, hipStream_t s) {
  if (a.type == RSX_FLOAT32) return checkpoint<float>(a, false, s);
  return a.type == RSX_BFLOAT16 ? checkpoint<bf16_t>(a, false, s) : checkpoint<f16_t>(a, false, s);
}

}  // namespace rsx
