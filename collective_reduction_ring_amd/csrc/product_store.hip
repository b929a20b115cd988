// Products that are stored as they are, and copies of matrices as 16-bit parts.
#include "product_store.h"

namespace rsx {
namespace {

struct Store {
  typedef StoreArgs Args;
  template <class T, class TILE, int N>
  static __device__ __forceinline__ void run(const ProductArgs& p, const Where& w, const StoreArgs& e,
                                             const f32x4 (&acc)[TILE::TN][N], uint32_t i0, RSX_LDS char* lds) {
    void* out = w.batch ? e.out2 : e.out;
    const uint64_t ld = w.batch ? e.ld2 : e.ld;
    staged<TILE, false, N>(w, acc, i0, lds, [&](uint32_t m, uint32_t n, f32x8 v) {
      if (m >= p.m || n >= p.n) return;
      if (e.add) v += get<float, 8>(e.add + static_cast<uint64_t>(m) * p.n, n, p.n);
      if (e.row) v *= e.row[m];
      if (e.accumulate) v += get_as<8>(e.type, out, m * ld, n, p.n);
      put_as<8>(e.type, out, m * ld, n, p.n, v);
    });
  }
};

template <class T>
hipError_t store(Layouts l, const ProductArgs& p, const Schedule& c, const StoreArgs& e, void* ws, hipStream_t s) {
  return l == kNT   ? launch_product<T, kRow, kRow, false, false, Store>(p, c, ws, e, s)
         : l == kNN ? launch_product<T, kRow, kCol, false, false, Store>(p, c, ws, e, s)
                    : launch_product<T, kCol, kCol, false, false, Store>(p, c, ws, e, s);
}

// A workgroup moves one stretch of 2048 elements of a row, eight a lane.
constexpr uint64_t kStretch = 2048;
template <class S, class T>
__global__ __launch_bounds__(256) void copy_parts(const Copies c) {
  uint64_t id = block_id();
  int i = 0;
  while (i < c.n && id >= c.begin[i + 1]) ++i;
  if (i == c.n) return;
  id -= c.begin[i];
  const Matrix from = c.from[i];
  const Parts to = c.to[i];
  const uint64_t groups = (to.ld + kStretch - 1) / kStretch, row = id / groups;
  const uint32_t col = static_cast<uint32_t>(id % groups * kStretch) + threadIdx.x * 8;
  if (col >= to.ld) return;
  f32x8 v = __builtin_convertvector((load_row<S, 8, false>(static_cast<const S*>(from.p) + row * from.ld, col, static_cast<uint32_t>(from.cols))), f32x8);
  take_parts<T, 8>(v, to.count, [&](int k, typename Vec<T, 8>::type h) {
    *reinterpret_cast<typename Vec<T, 8>::type*>(static_cast<T*>(k == 0 ? to.part[0] : k == 1 ? to.part[1] : to.part[2]) + row * to.ld + col) = h;
  });
}

}  // namespace

// The times are in units of a large tile's step with every CU at one, 1.75 us: what
// the chip's power allows, so that fewer tiles at a time run faster, but not in
// proportion.  A CU holds one large tile at a time, two middle or four small ones.
// A tile begins and ends in two to three steps' time.  Cut tiles cost their sums'
// way through memory (a large tile's are 256 KB) and two more launches.
Schedule schedule(uint64_t m, uint64_t n, uint64_t batch, uint64_t steps, bool triangle, bool small) {
  Schedule best = {1, 0, 0, 0};
  if (m == 0 || n == 0 || batch == 0) return best;
  constexpr uint64_t kSide[3] = {256, 128, 64}, kHeld[3] = {1, 2, 4};
  constexpr double kLeast[3] = {0.5, 0.28, 0.14}, kMost[3] = {1.0, 0.56, 0.45}, kEnds[3] = {2.5, 2.0, 1.5}, kPiece[3] = {0.4, 0.25, 0.15};
  double least = 1e300;
  for (int i = 0; i < (small ? 3 : 2); ++i) {
    const uint64_t tm = (m + kSide[i] - 1) / kSide[i], tn = (n + kSide[i] - 1) / kSide[i], slots = kHeld[i] * kCus;
    const uint64_t tiles = (triangle ? tm * (tm + 1) / 2 : tm * tn) * batch, rest = tiles % slots, rounds = tiles / slots;
    // of `count` tiles at a time
    auto rate = [&](uint64_t count) {
      return kLeast[i] + (kMost[i] - kLeast[i]) * static_cast<double>(count) / static_cast<double>(slots);
    };
    const double s = static_cast<double>(steps), whole = static_cast<double>(rounds) * (kMost[i] * s + kEnds[i]);
    const double apart = whole + (rest ? rate(rest) * s + kEnds[i] : 0.0);
    if (apart < least) {
      least = apart;
      best = {i, static_cast<uint32_t>(tiles), 0, 0};
    }
    uint64_t cuts = rest ? slots / rest : 0;
    cuts = cuts > steps / 4 ? steps / 4 : cuts;  // a piece of fewer steps is mostly its ends
    cuts = cuts > 16 ? 16 : cuts;
    if (cuts < 2) continue;
    const double cut = whole + rate(rest * cuts) * (s / static_cast<double>(cuts)) + kEnds[i] + 3.0 + kPiece[i] * static_cast<double>(cuts);
    if (cut < least) {
      least = cut;
      best = {i, static_cast<uint32_t>(tiles - rest), static_cast<uint32_t>(cuts), rest * cuts * kSide[i] * kSide[i] * 4};
    }
  }
  return best;
}

hipError_t launch_store(bool half, Layouts l, ProductArgs p, const StoreArgs& e, void* ws, hipStream_t s) {
  if (p.m == 0 || p.n == 0) return hipSuccess;
  const Schedule c = store_schedule(p.m, p.n, p.k, p.nseg, p.batch);
  return half ? store<f16_t>(l, p, c, e, ws, s) : store<bf16_t>(l, p, c, e, ws, s);
}

hipError_t launch_copies(Copies& c, int type, bool half, hipStream_t s) {
  c.begin[0] = 0;
  for (int i = 0; i < c.n; ++i) c.begin[i + 1] = c.begin[i] + c.from[i].rows * ((c.to[i].ld + kStretch - 1) / kStretch);
  if (c.n == 0) return hipSuccess;
  // no fp32 matrix is cut into fp16 parts here
  return launch(half                    ? copy_parts<f16_t, f16_t>
                : type == RSX_FLOAT32  ? copy_parts<float, bf16_t>
                : type == RSX_BFLOAT16 ? copy_parts<bf16_t, bf16_t> : copy_parts<f16_t, bf16_t>,
                grid_of(c.begin[c.n]), 256, 0, s, c);
}

}  // namespace rsx
