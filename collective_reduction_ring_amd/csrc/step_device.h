// Device helpers of the training-step operators: typed vectors of a row, wave
// and group sums, and the 8-bit block format of a checkpoint.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "step_internal.h"

namespace rsx {

// Launch of a kernel; the status of this launch alone.
template <class P>
struct Given {
  typedef P type;
};
template <class... P>
hipError_t launch(void (*kernel)(P...), dim3 grid, uint32_t threads, uint32_t lds, hipStream_t s,
                  typename Given<P>::type... a) {
  void* args[] = {static_cast<void*>(&a)...};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(threads), args, lds, s);
}

typedef __bf16 bf16_t;
typedef _Float16 f16_t;

// Index of the workgroup in a grid_of grid.
__device__ __forceinline__ uint64_t block_id() {
  return static_cast<uint64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
}

// N elements of T.  Rows start at any element and have any length, so a
// vector access assumes element alignment only; the global memory
// instructions take any such address in one access.
template <class T, int N>
struct Vec {
  typedef T type __attribute__((ext_vector_type(N)));
  typedef T loose __attribute__((ext_vector_type(N), aligned(sizeof(T))));
  typedef float wide __attribute__((ext_vector_type(N)));
};

// Streamed: read or written once, so it passes the caches by.
template <class T, int N>
__device__ __forceinline__ typename Vec<T, N>::type load_once(const T* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const typename Vec<T, N>::loose*>(p));
}
template <class T, int N>
__device__ __forceinline__ typename Vec<T, N>::type load_kept(const T* p) {
  return *reinterpret_cast<const typename Vec<T, N>::loose*>(p);
}
template <class T, int N>
__device__ __forceinline__ void store_once(T* p, typename Vec<T, N>::type v) {
  __builtin_nontemporal_store(static_cast<typename Vec<T, N>::loose>(v),
                              reinterpret_cast<typename Vec<T, N>::loose*>(p));
}

// Vector at element e of a row of `dim`; elements past the row's end are 0,
// and are not touched.  `ONCE`: a streamed load.
template <class T, int N, bool ONCE = true>
__device__ __forceinline__ typename Vec<T, N>::type load_row(const T* row, uint32_t e, uint32_t dim) {
  typename Vec<T, N>::type v = {};
  if (e + N <= dim) {
    v = ONCE ? load_once<T, N>(row + e) : load_kept<T, N>(row + e);
  } else if (e < dim) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (e + i < dim) v[i] = row[e + i];
  }
  return v;
}
template <class T, int N>
__device__ __forceinline__ void store_row(T* row, uint32_t e, uint32_t dim, typename Vec<T, N>::type v) {
  if (e + N <= dim) {
    store_once<T, N>(row + e, v);
  } else if (e < dim) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (e + i < dim) row[e + i] = v[i];
  }
}

// The same for rows of at least N elements, in two steps: a vector that does
// not fit is loaded from the row's end (load_in), and moved into place when it
// is used (in_place).  Loads by element, or a move at once, wait for the load:
// every row of a width that fills no vector then has no other row on its way
// (gradient of 32767 rows of 4095 bf16: 356 and 214 us).
template <class T, int N, bool ONCE = true>
__device__ __forceinline__ typename Vec<T, N>::type load_in(const T* row, uint32_t e, uint32_t dim) {
  const T* p = row + min(e, dim - N);
  return ONCE ? load_once<T, N>(p) : load_kept<T, N>(p);
}
template <class T, int N>
__device__ __forceinline__ typename Vec<T, N>::type in_place(typename Vec<T, N>::type v, uint32_t e, uint32_t dim) {
  constexpr int kBytes = static_cast<int>(sizeof(T)) * N;
  typedef typename Vec<T, N>::type V;
  typedef uint64_t Two __attribute__((ext_vector_type(2)));
  const uint32_t by = min(e - min(e, dim - N), static_cast<uint32_t>(N));
  if (__ballot(by != 0) == 0) return v;
  const uint32_t bits = by * static_cast<uint32_t>(sizeof(T)) * 8;
  auto down = [](Two u, uint32_t n) {  // n <= 128
    const uint64_t lo = n == 0 ? u[0] : n < 64 ? (u[0] >> n) | (u[1] << (64 - n)) : n < 128 ? u[1] >> (n - 64) : 0;
    return Two{lo, n < 64 ? u[1] >> n : 0};
  };
  if constexpr (kBytes == 16) {
    return __builtin_bit_cast(V, down(__builtin_bit_cast(Two, v), bits));
  } else if constexpr (kBytes == 8) {
    return __builtin_bit_cast(V, bits < 64 ? __builtin_bit_cast(uint64_t, v) >> bits : 0);
  } else {
    static_assert(kBytes == 4, "");
    return __builtin_bit_cast(V, bits < 32 ? __builtin_bit_cast(uint32_t, v) >> bits : 0u);
  }
}
// Both steps for vectors of 32 bytes too.
template <class T, int N, bool ONCE>
__device__ __forceinline__ typename Vec<T, N>::type load_wide(const T* row, uint32_t e, uint32_t dim) {
  if constexpr (sizeof(T) * N <= 16) {
    return load_in<T, N, ONCE>(row, e, dim);
  } else {
    return __builtin_shufflevector(load_in<T, N / 2, ONCE>(row, e, dim), load_in<T, N / 2, ONCE>(row, e + N / 2, dim), 0, 1, 2, 3,
                                   4, 5, 6, 7);
  }
}
template <class T, int N>
__device__ __forceinline__ typename Vec<T, N>::type wide_in_place(typename Vec<T, N>::type v, uint32_t e, uint32_t dim) {
  if constexpr (sizeof(T) * N <= 16) {
    return in_place<T, N>(v, e, dim);
  } else {
    return __builtin_shufflevector(in_place<T, N / 2>(__builtin_shufflevector(v, v, 0, 1, 2, 3), e, dim),
                                   in_place<T, N / 2>(__builtin_shufflevector(v, v, 4, 5, 6, 7), e + N / 2, dim), 0, 1, 2, 3, 4, 5,
                                   6, 7);
  }
}
// Both at once, through the caches.
template <class T, int N>
__device__ __forceinline__ typename Vec<T, N>::type load_pair(const T* row, uint32_t e, uint32_t dim) {
  return wide_in_place<T, N>(load_wide<T, N, false>(row, e, dim), e, dim);
}

// v, as far as the compiler knows another value each time: what is computed
// from it in a loop stays in the loop, instead of in registers before it.
template <class V>
__device__ __forceinline__ V fresh(V v) {
  asm volatile("" : "+v"(v));
  return v;
}

template <class T, int N>
__device__ __forceinline__ typename Vec<T, N>::wide widen(typename Vec<T, N>::type v) {
  return __builtin_convertvector(v, typename Vec<T, N>::wide);
}
// Rounded to nearest even, once.
template <class T, int N>
__device__ __forceinline__ typename Vec<T, N>::type narrow(typename Vec<T, N>::wide v) {
  return __builtin_convertvector(v, typename Vec<T, N>::type);
}

// ---------------------------------------------------------------- waves
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
constexpr int kSwap1 = 0xB1;        // quad_perm [1,0,3,2]
constexpr int kSwap2 = 0x4E;        // quad_perm [2,3,0,1]
constexpr int kHalfMirror = 0x141;  // within 8 lanes
constexpr int kMirror = 0x140;      // within 16 lanes

// Sum over the 64 lanes, the same in every lane: a tree of fixed order.
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<kSwap1>(v);
  v += dpp<kSwap2>(v);
  v += dpp<kHalfMirror>(v);
  v += dpp<kMirror>(v);
  return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp<kSwap1>(v));
  v = fmaxf(v, dpp<kSwap2>(v));
  v = fmaxf(v, dpp<kHalfMirror>(v));
  v = fmaxf(v, dpp<kMirror>(v));
  return fmaxf(fmaxf(lane_value(v, 0), lane_value(v, 16)), fmaxf(lane_value(v, 32), lane_value(v, 48)));
}

// Barrier for LDS exchange alone: loads from and stores to global memory stay
// in flight across it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// For values that are the same in the whole wave, but not to the compiler.
__device__ __forceinline__ uint32_t uniform(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(v)));
}
__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
  return (static_cast<uint64_t>(uniform(static_cast<uint32_t>(v >> 32))) << 32) | uniform(static_cast<uint32_t>(v));
}
// Set bits of m below this lane's.
__device__ __forceinline__ uint32_t lanes_below(uint64_t m) {
  return __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(m >> 32), __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(m), 0));
}
// Which of the rows of a workgroup, G lanes each, is this lane's.
template <int G, int K>
__device__ __forceinline__ uint32_t sub_row() {
  if constexpr (G >= K) return 0;
  if constexpr (G >= 64) return uniform(threadIdx.x / G);
  return threadIdx.x / G;
}

// Sums over the G lanes that share a row, the same in each of them.  Up to
// G = 64 in a wave, no LDS.  Otherwise every thread of the workgroup takes
// part, and `slot` is an array that no sum still in use shares (callers
// alternate between arrays, one barrier each).
template <int G, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float (*slot)[16]) {
  static_assert(G == 16 || G == 32 || G % 64 == 0, "");
  if constexpr (G < 64) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] += dpp<kSwap1>(v[i]);
      v[i] += dpp<kSwap2>(v[i]);
      v[i] += dpp<kHalfMirror>(v[i]);
      v[i] += dpp<kMirror>(v[i]);
      if constexpr (G == 32)  // lane ^ 16
        v[i] += __builtin_bit_cast(float, __builtin_amdgcn_ds_swizzle(__builtin_bit_cast(int, v[i]), 0x401f));
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  }
  if constexpr (G > 64) {
    const int wave = threadIdx.x / 64, first = wave / (G / 64) * (G / 64);
    if (threadIdx.x % 64 == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) slot[i][wave] = v[i];
    }
    lds_barrier();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < G / 64; ++w) t += slot[i][first + w];
      v[i] = t;
    }
  }
}

// ------------------------------------------------- 8-bit block format
// 32 consecutive elements of a row share one power of two.  With E the
// exponent of their largest magnitude (2^E <= m < 2^(E+1)), an element x is
// kept as q = rint(x / 2^(E-6)), clamped to [-127, 127], and stands for
// q * 2^(E-6): at most half a step off, or one step where |q| would be 128.
// Both scalings are by powers of two, so the rounding to q is the only one.
// The scale byte holds E - 6 + 127; blocks of magnitude below 2^-120 use byte
// 0 (a step of 2^-127).  A block that holds an infinity or a NaN gets byte 255
// and comes back as NaN throughout: 8 bits hide no divergence.
constexpr uint32_t kCkBad = 255;

__device__ __forceinline__ uint32_t ck_scale_byte(float largest) {
  const uint32_t e = __builtin_bit_cast(uint32_t, largest) >> 23;  // largest >= 0
  return e == 255u ? kCkBad : e > 6u ? e - 6u : 0u;
}
__device__ __forceinline__ float ck_step(uint32_t byte) {
  const uint32_t b = byte == 0u ? 0x00400000u : byte == kCkBad ? 0x7fc00000u : byte << 23;
  return __builtin_bit_cast(float, b);
}
// 1 / ck_step; 0 for a bad block.
__device__ __forceinline__ float ck_inverse(uint32_t byte) {
  return byte == kCkBad ? 0.0f : __builtin_bit_cast(float, (254u - byte) << 23);
}
__device__ __forceinline__ int8_t ck_code(float x, float inverse) {
  // A bad block has codes of 0, and -127 for its infinities and NaNs, which times 0
  // are NaN and left to the clamp; its byte says that no code of it counts.
  return static_cast<int8_t>(fminf(fmaxf(__builtin_rintf(x * inverse), -127.0f), 127.0f));
}

// Largest magnitude over the lanes that share a block: LANES = 32 / elements
// per lane, consecutive and aligned.  A NaN counts as an infinity.
template <int LANES>
__device__ __forceinline__ float ck_largest(float m) {
  static_assert(LANES == 4 || LANES == 8, "a lane holds 8 or 4 elements of a block");
  m = fmaxf(m, dpp<kSwap1>(m));
  m = fmaxf(m, dpp<kSwap2>(m));
  if constexpr (LANES == 8) m = fmaxf(m, dpp<kHalfMirror>(m));
  return m;
}
__device__ __forceinline__ float ck_magnitude(float x) {
  const float a = fabsf(x);
  return a == a ? a : INFINITY;
}

}  // namespace rsx
