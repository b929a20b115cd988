// Products that are stored as they are, and copies of matrices as 16-bit parts.
#include "product_store.h"

namespace rsx {
namespace {

struct Store {
  typedef StoreArgs Args;
  template <class T, class TILE>
  static __device__ __forceinline__ void run(const ProductArgs& p, const Where& w, const StoreArgs& e,
                                             const f32x4 (&acc)[TILE::TN][TILE::TM], RSX_LDS char* lds) {
    staged<TILE, false>(w, acc, lds, [&](uint32_t m, uint32_t n, f32x8 v) {
      if (m >= p.m || n >= p.n) return;
      if (e.partial) {
        put<float, 8>(e.partial + (static_cast<uint64_t>(w.split) * p.m + m) * p.n, n, p.n, v);
      } else {
        if (e.add) v += get<float, 8>(e.add + static_cast<uint64_t>(m) * p.n, n, p.n);
        if (e.accumulate) v += get_as<8>(e.type, e.out, m * e.ld, n, p.n);
        put_as<8>(e.type, e.out, m * e.ld, n, p.n, v);
      }
    });
  }
};

// The cuts' sums, added in their order.
__global__ __launch_bounds__(256) void reduce_splits(const float* partial, uint32_t splits, uint32_t m, uint32_t n, StoreArgs e) {
  const uint32_t chunks = (n + 3) / 4;
  const uint64_t t = block_id() * 256 + threadIdx.x;
  if (t >= static_cast<uint64_t>(m) * chunks) return;
  const uint64_t row = t / chunks;
  const uint32_t c = static_cast<uint32_t>(t % chunks) * 4;
  f32x4 v = get<float, 4>(partial + row * n, c, n);
  for (uint32_t s = 1; s < splits; ++s) v += get<float, 4>(partial + (s * static_cast<uint64_t>(m) + row) * n, c, n);
  if (e.add) v += get<float, 4>(e.add + row * n, c, n);
  if (e.accumulate) v += get_as<4>(e.type, e.out, row * e.ld, c, n);
  put_as<4>(e.type, e.out, row * e.ld, c, n, v);
}

template <class T, int LA, int LB>
hipError_t store(const ProductArgs& p, const StoreArgs& e, bool large, hipStream_t s) {
  return large ? launch_tiles<T, Large, LA, LB, false, false, Store>(p, e, s)
               : launch_tiles<T, Middle, LA, LB, false, false, Store>(p, e, s);
}
template <class T>
hipError_t store(Layouts l, const ProductArgs& p, const StoreArgs& e, bool large, hipStream_t s) {
  return l == kNT ? store<T, kRow, kRow>(p, e, large, s)
                  : l == kNN ? store<T, kRow, kCol>(p, e, large, s) : store<T, kCol, kCol>(p, e, large, s);
}

// A workgroup moves one stretch of 2048 elements of a row, eight a lane.
template <class S, class T>
__global__ __launch_bounds__(256) void copy_parts(const S* src, uint64_t ld, uint32_t rows, uint32_t cols, uint32_t groups, Parts dst) {
  const uint64_t id = block_id();
  const uint64_t row = id / groups;
  const uint32_t c = static_cast<uint32_t>(id % groups) * 2048 + threadIdx.x * 8;
  if (row >= rows || c >= dst.ld) return;
  typename Vec<float, 8>::type v = __builtin_convertvector((load_row<S, 8, false>(src + row * ld, c, cols)), typename Vec<float, 8>::type);
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if (i >= dst.count) break;
    const auto h = __builtin_convertvector(v, typename Vec<T, 8>::type);
    *reinterpret_cast<typename Vec<T, 8>::type*>(static_cast<T*>(dst.part[i]) + row * dst.ld + c) = h;
    const auto back = __builtin_convertvector(h, typename Vec<float, 8>::type);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = fabsf(back[e]) < INFINITY ? v[e] - back[e] : 0.0f;
  }
}
template <class S, class T>
hipError_t copy(const Matrix& m, const Parts& dst, hipStream_t s) {
  const uint32_t groups = static_cast<uint32_t>((dst.ld + 2047) / 2048);
  return launch(copy_parts<S, T>, grid_of(m.rows * groups), 256, 0, s, static_cast<const S*>(m.p), m.ld,
                static_cast<uint32_t>(m.rows), static_cast<uint32_t>(m.cols), groups, dst);
}

}  // namespace

uint32_t store_splits(uint64_t m, uint64_t n, uint64_t steps) {
  if (m == 0 || n == 0 || large_tiles(m, n, 1, false)) return 1;
  const uint64_t tiles = ((m + 127) / 128) * ((n + 127) / 128);
  // Two middle tiles a CU; a cut of fewer than 8 steps is mostly its beginning and its end.
  uint64_t splits = 2 * kCus / tiles;
  if (splits > steps / 8) splits = steps / 8;
  if (splits > 16) splits = 16;
  return splits < 2 ? 1 : static_cast<uint32_t>(splits);
}

hipError_t launch_store(bool half, Layouts l, ProductArgs p, StoreArgs e, void* ws, hipStream_t s) {
  if (p.m == 0 || p.n == 0) return hipSuccess;
  p.batch = 1;
  const bool large = large_tiles(p.m, p.n, 1, false);
  p.splits = store_splits(p.m, p.n, p.nseg * ((p.k + static_cast<uint64_t>(kStep) - 1) / kStep));
  e.partial = p.splits > 1 ? static_cast<float*>(ws) : nullptr;
  const hipError_t st = half ? store<f16_t>(l, p, e, large, s) : store<bf16_t>(l, p, e, large, s);
  if (st != hipSuccess || p.splits == 1) return st;
  const uint64_t groups = (static_cast<uint64_t>(p.m) * ((p.n + 3) / 4) + 255) / 256;
  return launch(reduce_splits, grid_of(groups), 256, 0, s, static_cast<const float*>(ws), p.splits, p.m, p.n, e);
}

hipError_t launch_copy(const Matrix& m, int type, const Parts& dst, bool half, hipStream_t s) {
  if (m.rows == 0 || m.cols == 0) return hipSuccess;
  if (half) return copy<f16_t, f16_t>(m, dst, s);  // no fp32 matrix is cut into fp16 parts here
  return type == RSX_FLOAT32 ? copy<float, bf16_t>(m, dst, s)
                             : type == RSX_BFLOAT16 ? copy<bf16_t, bf16_t>(m, dst, s) : copy<f16_t, bf16_t>(m, dst, s);
}

}  // namespace rsx
