// Layer norm forward and backward, and the 8-bit checkpoints of its input.
//
//   mean = sum x / D,  rstd = (sum (x - mean)^2 / D + eps)^(-1/2),
//   xhat = (x - mean) rstd,  y = xhat w + b;
//   g = dy w,  dx = rstd (g - mean(g) - xhat mean(g xhat)),
//   dw = sum over rows of dy xhat,  db = sum over rows of dy.
//
// Everything is held in fp32 and rounded once, at the store.  All kernels
// here are bound by HBM: a row is read once into registers, both its sums are
// taken there (the variance from the differences, so no digits are lost to a
// large mean), and the result is written from them.
#include "step_device.h"

namespace rsx {
namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------- forward
// A row of values from about 1e16 on may have finite differences whose squares
// overflow: their sum is then taken again over differences scaled by 2^-80.
// The test is the same for every lane of the row.
constexpr float kScaleDown = 0x1p-80f;
__device__ __forceinline__ bool squares_overflow(float sq, float mean, float factor) {
  return sq == INFINITY && fabsf(mean) < INFINITY && factor == 1.0f;
}

// G lanes share a row; each holds EPL of its elements, vectors of E at
// (j * G + lane) * E.  G = 64 puts a row in one wave: no barrier, and four
// rows in a workgroup.
template <class T, class W, int G, int EPL>
__global__ __launch_bounds__(G > kThreads ? G : kThreads) void norm_kernel(NormArgs a) {
  constexpr int E = 16 / sizeof(T);
  constexpr int V = EPL / E;
  constexpr int kRows = G >= kThreads ? 1 : kThreads / G;
  typedef Vec<T, E> X;
  __shared__ float slots[2][1][16];
  const uint32_t lane = threadIdx.x % G;
  const uint32_t dim = static_cast<uint32_t>(a.dim);
  const uint64_t row = block_id() * kRows + (kRows > 1 ? threadIdx.x / G : 0);
  if (row >= a.rows) return;  // whole waves, and the whole workgroup where it shares a row
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;

  typename X::type raw[V];
#pragma unroll
  for (int j = 0; j < V; ++j) raw[j] = load_row<T, E>(x, (j * G + lane) * E, dim);

  const float inv_dim = 1.0f / static_cast<float>(dim);
  float sum[1] = {0.0f};
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const typename X::wide f = widen<T, E>(raw[j]);
#pragma unroll
    for (int i = 0; i < E; ++i) sum[0] += f[i];
  }
  group_sum<G, 1>(sum, slots[0]);
  const float mean = sum[0] * inv_dim;

  float sq[1], factor = 1.0f;
  for (int turn = 1;; turn = 0) {
    sq[0] = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t e = (j * G + lane) * E;
      const typename X::wide f = (widen<T, E>(raw[j]) - mean) * factor;
      if (e + E <= dim) {
#pragma unroll
        for (int i = 0; i < E; ++i) sq[0] = fmaf(f[i], f[i], sq[0]);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
          if (e + i < dim) sq[0] = fmaf(f[i], f[i], sq[0]);
      }
    }
    group_sum<G, 1>(sq, slots[turn]);
    if (!squares_overflow(sq[0], mean, factor)) break;
    factor = kScaleDown;
  }
  const float rstd = factor / sqrtf(sq[0] * inv_dim + a.eps * factor * factor);
  if (lane == 0) {
    if (a.mean != nullptr) a.mean[row] = mean;
    if (a.rstd != nullptr) a.rstd[row] = rstd;
  }

  const W* w = static_cast<const W*>(a.weight);
  const W* b = static_cast<const W*>(a.bias);
  T* y = static_cast<T*>(a.y) + row * a.y_stride;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t e = (j * G + lane) * E;
    typename X::wide f = widen<T, E>(raw[j]);
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
    for (int i = 0; i < E; ++i) f[i] = (f[i] - mean) * rstd;
    if (w != nullptr) f *= widen<W, E>(load_row<W, E, false>(w, e, dim));
    if (b != nullptr) f += widen<W, E>(load_row<W, E, false>(b, e, dim));
    store_row<T, E>(y, e, dim, narrow<T, E>(f));
  }
}

// Rows too long for the registers: a workgroup reads its row three times,
// after the first from the caches.
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
  group_sum<1024, 1>(sum, slots[0]);
  const float mean = sum[0] * inv_dim;

  float sq[1], factor = 1.0f;
  for (int turn = 1;; turn = 0) {
    sq[0] = 0.0f;
    for (uint32_t e = threadIdx.x * E; e < dim; e += kStep) {
      const typename X::wide f = (widen<T, E>(load_row<T, E, false>(x, e, dim)) - mean) * factor;
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (e + i < dim) sq[0] = fmaf(f[i], f[i], sq[0]);
    }
    group_sum<1024, 1>(sq, slots[turn]);
    if (!squares_overflow(sq[0], mean, factor)) break;
    factor = kScaleDown;
  }
  const float rstd = factor / sqrtf(sq[0] * inv_dim + a.eps * factor * factor);
  if (threadIdx.x == 0) {
    if (a.mean != nullptr) a.mean[row] = mean;
    if (a.rstd != nullptr) a.rstd[row] = rstd;
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
    for (int i = 0; i < E; ++i) f[i] = (f[i] - mean) * rstd;
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
template <class T, int E, bool CK>
__device__ __forceinline__ Input<T, E, CK> load_input(const NormGradArgs& a, uint64_t row, uint32_t e, uint32_t dim) {
  Input<T, E, CK> v;
  if constexpr (CK) {
    v.q = load_row<int8_t, E>(a.codes + row * a.dim, e, dim);
    v.scale = e < dim ? a.scales[row * ck_blocks(a.dim) + e / kCkBlock] : 127u;
  } else {
    v.x = load_row<T, E>(static_cast<const T*>(a.x) + row * a.x_stride, e, dim);
  }
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

// Each group of G lanes takes every (groups)-th row; its next row is loaded
// before the current one's sums are exchanged.  dw and db are summed per
// workgroup over its rows in order, then over workgroups by norm_sum_kernel:
// a fixed order, whatever the timing.
template <class T, class W, int G, int EPL, bool CK>
__global__ __launch_bounds__(G > kThreads ? G : kThreads) void norm_grad_kernel(NormGradArgs a, uint32_t pitch) {
  constexpr int E = 16 / sizeof(T);
  constexpr int V = EPL / E;
  constexpr int kRows = G >= kThreads ? 1 : kThreads / G;
  typedef Vec<T, E> X;
  __shared__ float slots[2][2][16];
  __shared__ float join[kRows > 1 ? kRows * G * EPL : 1];
  const uint32_t lane = threadIdx.x % G;
  const uint32_t sub = kRows > 1 ? threadIdx.x / G : 0;
  const uint32_t dim = static_cast<uint32_t>(a.dim);
  const uint64_t step = static_cast<uint64_t>(gridDim.x) * kRows;
  const T* dy = static_cast<const T*>(a.dy);
  T* dx = static_cast<T*>(a.dx);
  const float inv_dim = 1.0f / static_cast<float>(dim);

  typename X::wide w[V], dw[V], db[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint32_t e = (j * G + lane) * E;
#pragma unroll
    for (int i = 0; i < E; ++i) w[j][i] = 1.0f;
    if (a.weight != nullptr) w[j] = widen<W, E>(load_row<W, E, false>(static_cast<const W*>(a.weight), e, dim));
    dw[j] = 0.0f;
    db[j] = 0.0f;
  }

  uint64_t row = static_cast<uint64_t>(blockIdx.x) * kRows + sub;
  typename X::type next_dy[V];
  Input<T, E, CK> next_x[V];
  float next_mean = 0.0f, next_rstd = 0.0f;
  if (row < a.rows) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t e = (j * G + lane) * E;
      next_x[j] = load_input<T, E, CK>(a, row, e, dim);
      next_dy[j] = load_row<T, E>(dy + row * a.dy_stride, e, dim);
    }
    next_mean = a.mean[row];
    next_rstd = a.rstd[row];
  }
  uint32_t turn = 0;
  for (; row < a.rows; row += step, turn ^= 1u) {
    typename X::wide xhat[V], g[V];
    const float mean = next_mean, rstd = next_rstd;
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const typename X::wide d = widen<T, E>(next_dy[j]);
      xhat[j] = (input_value<T, E, CK>(next_x[j]) - mean) * rstd;
      g[j] = d * w[j];
      db[j] += d;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        dw[j][i] = fmaf(d[i], xhat[j][i], dw[j][i]);
        s[0] += g[j][i];
        s[1] = fmaf(g[j][i], xhat[j][i], s[1]);
      }
    }
    if (row + step < a.rows) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint32_t e = (j * G + lane) * E;
        next_x[j] = load_input<T, E, CK>(a, row + step, e, dim);
        next_dy[j] = load_row<T, E>(dy + (row + step) * a.dy_stride, e, dim);
      }
      next_mean = a.mean[row + step];
      next_rstd = a.rstd[row + step];
    }
    group_sum<G, 2>(s, slots[turn]);
    const float c1 = s[0] * inv_dim, c2 = s[1] * inv_dim;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      typename X::wide f;
#pragma unroll
      for (int i = 0; i < E; ++i) f[i] = (g[j][i] - fmaf(xhat[j][i], c2, c1)) * rstd;
      store_row<T, E>(dx + row * a.dx_stride, (j * G + lane) * E, dim, narrow<T, E>(f));
    }
  }

  // One partial row of dw and one of db for each workgroup.
  float* part = a.partial + static_cast<uint64_t>(blockIdx.x) * 2 * pitch;
#pragma unroll
  for (int k = 0; k < 2; ++k, part += pitch) {
    if constexpr (kRows > 1) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < E; ++i) join[sub * (G * EPL) + (j * G + lane) * E + i] = k == 0 ? dw[j][i] : db[j][i];
      __syncthreads();
      for (uint32_t e = threadIdx.x; e < dim; e += kThreads) {
        float t = 0.0f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) t += join[r * (G * EPL) + e];
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
  const uint32_t e = (blockIdx.x % column_groups * kThreads + threadIdx.x) * E;
  const uint32_t p = blockIdx.x / column_groups;
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

// dw and db from the workgroups' partial rows: 64 columns a workgroup, wave w
// takes partial rows w, w + 16, ...; no rows at all give zeros.
template <class W>
__global__ __launch_bounds__(1024) void norm_sum_kernel(const float* partial, uint32_t pitch, uint32_t parts,
                                                        uint32_t dim, W* dweight, W* dbias) {
  __shared__ float join[16][64];
  W* out = blockIdx.y == 0 ? dweight : dbias;
  if (out == nullptr) return;
  const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const uint32_t e = blockIdx.x * 64 + lane;
  float t = 0.0f;
  if (e < dim) {
    const float* p = partial + blockIdx.y * pitch + e;
#pragma unroll 8
    for (uint32_t r = wave; r < parts; r += 16) t += p[static_cast<uint64_t>(r) * 2 * pitch];
  }
  join[wave][lane] = t;
  __syncthreads();
  if (wave == 0 && e < dim) {
    float s = 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r) s += join[r][lane];
    out[e] = static_cast<W>(s);
  }
}

// ------------------------------------------------------------ checkpoints
// L lanes share a row's chunk of 8 * L elements (a power of two, at least 4:
// a block's lanes stay together), so short rows share a wave.
template <class T>
__global__ __launch_bounds__(kThreads) void pack_kernel(PackArgs a, uint32_t lanes, uint32_t chunks) {
  const uint64_t thread = block_id() * kThreads + threadIdx.x;
  const uint64_t item = thread / lanes;
  const uint64_t row = item / chunks;
  const uint32_t dim = static_cast<uint32_t>(a.dim);
  if (row >= a.rows) return;  // all the lanes of an item
  const uint32_t e = (static_cast<uint32_t>(item % chunks) * lanes + static_cast<uint32_t>(thread % lanes)) * 8;
  const T* x = static_cast<const T*>(a.x) + row * a.stride;
  const typename Vec<T, 8>::wide f = widen<T, 8>(load_row<T, 8>(x, e, dim));
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, ck_magnitude(f[i]));
  const uint32_t byte = ck_scale_byte(ck_largest<4>(m));
  const float inverse = ck_inverse(byte);
  typename Vec<int8_t, 8>::type q;
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = ck_code(f[i], inverse);
  store_row<int8_t, 8>(a.codes + row * a.dim, e, dim, q);
  if (e % kCkBlock == 0 && e < dim) a.scales[row * ck_blocks(a.dim) + e / kCkBlock] = static_cast<uint8_t>(byte);
}

template <class T>
__global__ __launch_bounds__(kThreads) void unpack_kernel(PackArgs a, uint32_t lanes, uint32_t chunks) {
  const uint64_t thread = block_id() * kThreads + threadIdx.x;
  const uint64_t item = thread / lanes;
  const uint64_t row = item / chunks;
  const uint32_t dim = static_cast<uint32_t>(a.dim);
  const uint32_t e = (static_cast<uint32_t>(item % chunks) * lanes + static_cast<uint32_t>(thread % lanes)) * 8;
  if (row >= a.rows || e >= dim) return;
  const typename Vec<int8_t, 8>::type q = load_row<int8_t, 8>(a.codes + row * a.dim, e, dim);
  const float step = ck_step(a.scales[row * ck_blocks(a.dim) + e / kCkBlock]);
  const typename Vec<T, 8>::wide f = __builtin_convertvector(q, typename Vec<T, 8>::wide) * step;
  store_row<T, 8>(static_cast<T*>(a.out) + row * a.stride, e, dim, narrow<T, 8>(f));
}

template <class T>
hipError_t checkpoint(const PackArgs& a, bool pack, hipStream_t s) {
  uint32_t lanes = 4;
  while (lanes < 64 && lanes * 8 < a.dim) lanes *= 2;
  const uint64_t chunks = (a.dim + lanes * 8 - 1) / (lanes * 8);
  const uint64_t grid = (a.rows * chunks * lanes + kThreads - 1) / kThreads;
  const dim3 g = grid_of(grid);
  return launch(pack ? pack_kernel<T> : unpack_kernel<T>, g, kThreads, 0, s, a, lanes, static_cast<uint32_t>(chunks));
}

// --------------------------------------------------------------- launches
template <class T, class W, int G, int EPL>
hipError_t norm_go(const NormArgs& a, hipStream_t s) {
  constexpr uint32_t kRows = G >= kThreads ? 1 : kThreads / G;
  const uint64_t grid = (a.rows + kRows - 1) / kRows;
  return launch(norm_kernel<T, W, G, EPL>, grid_of(grid), G > kThreads ? G : kThreads, 0, s, a);
}

template <class T, class W>
hipError_t norm(const NormArgs& a, hipStream_t s) {
  // A wave per row where there are rows for every wave slot of the chip's
  // first fill; with fewer, four waves share a row and it is done sooner.
  if (a.rows >= 2048) {
    if (a.dim <= 512) return norm_go<T, W, 64, 8>(a, s);
    if (a.dim <= 1024) return norm_go<T, W, 64, 16>(a, s);
    if (a.dim <= 2048) return norm_go<T, W, 64, 32>(a, s);
    if (a.dim <= 4096) return norm_go<T, W, 64, 64>(a, s);
  }
  if (a.dim <= 2048) return norm_go<T, W, 256, 8>(a, s);
  if (a.dim <= 4096) return norm_go<T, W, 256, 16>(a, s);
  if (a.dim <= 8192) return norm_go<T, W, 256, 32>(a, s);
  if (a.dim <= 16384) return norm_go<T, W, 256, 64>(a, s);
  if (a.dim <= 32768) return norm_go<T, W, 1024, 32>(a, s);
  return launch(norm_long_kernel<T, W>, grid_of(a.rows), 1024, 0, s, a);
}

uint32_t grad_pitch(uint64_t dim) { return static_cast<uint32_t>((dim + 15) / 16 * 16); }
uint32_t grad_parts(uint64_t rows) { return static_cast<uint32_t>(rows < kGradGroups ? rows : kGradGroups); }

template <class T, class W, int G, int EPL, bool CK>
hipError_t grad_go(const NormGradArgs& a, uint32_t pitch, uint32_t* parts, hipStream_t s) {
  constexpr uint32_t kRows = G >= kThreads ? 1 : kThreads / G;
  const uint32_t need = static_cast<uint32_t>((a.rows + kRows - 1) / kRows < kGradGroups ? (a.rows + kRows - 1) / kRows
                                                                                         : kGradGroups);
  *parts = need;
  return launch(norm_grad_kernel<T, W, G, EPL, CK>, dim3(need), G > kThreads ? G : kThreads, 0, s, a, pitch);
}

template <class T, class W, bool CK>
hipError_t norm_grad(const NormGradArgs& a, hipStream_t s) {
  const uint32_t pitch = grad_pitch(a.dim);
  uint32_t parts = 0;
  hipError_t e = hipSuccess;
  if (a.rows != 0) {
    if (a.dim <= 512) {
      e = grad_go<T, W, 64, 8, CK>(a, pitch, &parts, s);
    } else if (a.dim <= 1024) {
      e = grad_go<T, W, 64, 16, CK>(a, pitch, &parts, s);
    } else if (a.dim <= 2048) {
      e = grad_go<T, W, 256, 8, CK>(a, pitch, &parts, s);
    } else if (a.dim <= 4096) {
      e = grad_go<T, W, 256, 16, CK>(a, pitch, &parts, s);
    } else if (a.dim <= 8192) {
      e = grad_go<T, W, 512, 16, CK>(a, pitch, &parts, s);
    } else if (a.dim <= 16384) {
      e = grad_go<T, W, 1024, 16, CK>(a, pitch, &parts, s);
    } else {
      parts = grad_parts(a.rows);
      const uint32_t per = kThreads * (16 / sizeof(T));
      const uint32_t columns = static_cast<uint32_t>((a.dim + per - 1) / per);
      e = launch(norm_columns_kernel<T, CK>, dim3(columns * parts), kThreads, 0, s, a, pitch, parts, columns);
      if (e != hipSuccess) return e;
      e = launch(norm_grad_long_kernel<T, W, CK>, grid_of(a.rows), 1024, 0, s, a);
    }
  }
  if (e != hipSuccess || (a.dweight == nullptr && a.dbias == nullptr)) return e;
  return launch(norm_sum_kernel<W>, dim3(static_cast<uint32_t>((a.dim + 63) / 64), 2), 1024, 0, s, a.partial, pitch,
                parts, static_cast<uint32_t>(a.dim), static_cast<W*>(a.dweight), static_cast<W*>(a.dbias));
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
