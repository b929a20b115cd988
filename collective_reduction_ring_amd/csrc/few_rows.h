// Products of few rows with a large matrix, a decoding step's: the matrix is
// read once, straight into the lanes that multiply it, and the time is the
// memory's.
//
// A workgroup takes 16 * RG of the matrix's rows and its waves share k out
// in turns of U steps; their sums meet in LDS.  (131072 x 4096 bf16: eight waves and
// turns of four steps 185 us, 5.8 TB/s; four and eight 191, with streamed loads,
// which fetch a cache line again for its other half, 221; sixteen and two 176, but
// 264 with the softmax's registers.)  A step is one matrix
// instruction of 32 k (16 bits) or four of 4 k (fp32, whose products stay fp32
// here): a lane's 16 bytes of a row are its k, in the matrix and in x alike.
#pragma once

#include "product.h"

namespace rsx {

struct FewArgs {
  const void* x;
  const void* w;
  const void* w2;  // second matrix of a double product
  uint64_t ldx, ldw, ldw2;
  uint32_t n, rows, k;  // rows of x, of the matrix; length of either
  uint32_t cuts;        // workgroups that share a group of rows' k; 0 is 1
  uint64_t rest;        // SPLIT: elements from x to its second part, which is multiplied as well
};
// Which of them this one is.
__device__ __forceinline__ uint32_t few_cut(const FewArgs& p) { return p.cuts ? static_cast<uint32_t>(block_id() % p.cuts) : 0; }

constexpr int kFewWaves = 8;
constexpr uint32_t kFewRows = 64;  // rows of x that this form takes at most

template <class T>
struct FewFrag {
  static constexpr int N = 16 / sizeof(T);
  typedef typename Vec<T, N>::type type;
};
__device__ __forceinline__ f32x4 few_mma(FewFrag<float>::type w, FewFrag<float>::type x, f32x4 c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(w[i], x[i], c, 0, 0, 0);
  return c;
}
__device__ __forceinline__ f32x4 few_mma(FewFrag<bf16_t>::type w, FewFrag<bf16_t>::type x, f32x4 c) { return mma(w, x, c); }
__device__ __forceinline__ f32x4 few_mma(FewFrag<f16_t>::type w, FewFrag<f16_t>::type x, f32x4 c) { return mma(w, x, c); }

// v[g][t] for the waves t mod kFewWaves: lane l has x row 16 t + l % 16 and matrix
// rows first + 16 g + 4 (l / 16) .. + 3 (g from RG on: the second matrix's).
template <class T, int NT, int RG, bool DUAL, bool SPLIT, class EPILOGUE>
__global__ __launch_bounds__(64 * kFewWaves, 4) void few_rows_kernel(const FewArgs p, const typename EPILOGUE::Args e) {
  constexpr int NM = DUAL ? 2 * RG : RG, N = FewFrag<T>::N, S = 4 * N, NX = SPLIT ? 2 * NT : NT;
  constexpr int U = NM + NX <= 5 ? 4 : NM + NX <= 8 ? 2 : 1;  // a turn's loads in registers: 80 at most, beside the sums
  typedef typename FewFrag<T>::type V;
  __shared__ f32x4 sums[kFewWaves][NM][NT][64];
  const uint32_t l = threadIdx.x % 64, wave = uniform(threadIdx.x / 64), r = l % 16, g = l / 16;
  const uint32_t cuts = p.cuts ? p.cuts : 1, cut = few_cut(p);
  const uint64_t group = block_id() / cuts;
  if (group * (16 * RG) >= p.rows) return;
  const uint32_t first = static_cast<uint32_t>(group) * (16 * RG);
  const T* wr[NM];
  const T* xr[NX];
#pragma unroll
  for (int m = 0; m < NM; ++m) {
    const uint64_t row = min(first + m % RG * 16 + r, p.rows - 1);
    wr[m] = (m < RG ? static_cast<const T*>(p.w) + row * p.ldw : static_cast<const T*>(p.w2) + row * p.ldw2) + g * N;
  }
#pragma unroll
  for (int t = 0; t < NX; ++t)
    xr[t] = static_cast<const T*>(p.x) + (t < NT ? 0 : p.rest) + static_cast<uint64_t>(min(t % NT * 16 + r, p.n - 1)) * p.ldx + g * N;
  f32x4 acc[NM][NT];
#pragma unroll
  for (int m = 0; m < NM; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[m][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  // the waves of all cuts take turns
  const uint32_t turns = p.k / (U * S), all = kFewWaves * cuts, me = cut * kFewWaves + wave;
  const uint32_t mine = turns > me ? (turns - me + all - 1) / all : 0;
  // Workgroups begin in different places of the rows: row strides are often powers of two, and in step all would
  // ask the same memory channels.
  uint32_t at = mine ? static_cast<uint32_t>(group % mine) : 0;
  for (uint32_t i = 0; i < mine; ++i) {
    const uint32_t turn = me + at * all;
    at = at + 1 < mine ? at + 1 : 0;
    V w[U][NM], x[U][NX];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int m = 0; m < NM; ++m) w[u][m] = load_kept<T, N>(wr[m] + (turn * U + u) * S);
#pragma unroll
      for (int t = 0; t < NX; ++t) x[u][t] = load_kept<T, N>(xr[t] + (turn * U + u) * S);
    }
    __builtin_amdgcn_sched_barrier(0);  // a turn's loads are all on their way before the first is waited for
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int t = 0; t < NX; ++t) acc[m][t % NT] = few_mma(w[u][m], x[u][t], acc[m][t % NT]);
  }
  for (uint32_t step = turns * U + me; step * S < p.k; step += all) {
    // what is left of a row, element by element where it ends in a lane's 16 bytes
    const uint32_t k = step * S + g * N;
    V x[NX];
#pragma unroll
    for (int t = 0; t < NX; ++t) x[t] = load_row<T, N, false>(xr[t] - g * N, k, p.k);
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      const V w = load_row<T, N, false>(wr[m] - g * N, k, p.k);
#pragma unroll
      for (int t = 0; t < NX; ++t) acc[m][t % NT] = few_mma(w, x[t], acc[m][t % NT]);
    }
  }
#pragma unroll
  for (int m = 0; m < NM; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) sums[wave][m][t][l] = acc[m][t];
  __syncthreads();
  for (int t = wave; t < NT; t += kFewWaves) {
    f32x4 v[NM];
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      v[m] = sums[0][m][t][l];
#pragma unroll
      for (int i = 1; i < kFewWaves; ++i) v[m] += sums[i][m][t][l];
    }
    EPILOGUE::template few<T, RG>(p, e, t * 16 + r, first + g * 4, v);
  }
}

template <class T, int RG, bool DUAL, class EPILOGUE, bool SPLIT = false>
hipError_t launch_few(const FewArgs& p, const typename EPILOGUE::Args& e, hipStream_t s) {
  const dim3 grid = grid_of((static_cast<uint64_t>(p.rows) + 16 * RG - 1) / (16 * RG) * (p.cuts ? p.cuts : 1));
  if (p.n <= 16) return launch(few_rows_kernel<T, 1, RG, DUAL, SPLIT, EPILOGUE>, grid, 64 * kFewWaves, 0, s, p, e);
  if (p.n <= 32) return launch(few_rows_kernel<T, 2, RG, DUAL, SPLIT, EPILOGUE>, grid, 64 * kFewWaves, 0, s, p, e);
  return launch(few_rows_kernel<T, 4, RG, DUAL, SPLIT, EPILOGUE>, grid, 64 * kFewWaves, 0, s, p, e);
}

}  // namespace rsx
