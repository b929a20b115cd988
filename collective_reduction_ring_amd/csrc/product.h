// Tile products on the matrix cores: what the feed-forward block, the log
// probabilities from hidden states and the orthogonalised update share.
//
// A product is C[m][n] = sum over segments s and k of A_s[m][k] * B_s[n][k],
// with 16-bit elements (bf16 or fp16) and fp32 sums.  Segments are products
// that add up in the registers: the two halves of a feed-forward gradient, and
// the parts of values that 16 bits do not hold.  An fp32 value is the sum of
// three bf16 values exactly, or of two fp16 values within 2^-22 of itself as
// long as its size is known, and the product of two such sums is a few
// products of parts at the 16-bit rate, sixteen times the rate of fp32 matrix
// instructions: six products of parts (bf16) by the rates 2.6 times as fast as
// one in fp32, three (fp16) 5.3 times; as measured (1230 TFLOP/s here, 153 of the
// library's fp32 product, 8192^3) 1.3 and 2.7 times.
//
// An operand is either "row" (k side by side) or "col" (m or n side by side,
// one k row after another); a col tile is turned by the LDS's transposing
// reads, so that no operand has to be transposed in memory.
#pragma once

#include "step_device.h"

namespace rsx {

constexpr int kRow = 0, kCol = 1;
constexpr int kMaxSegments = 12;
constexpr uint32_t kStep = 64;  // k of one step: 128 bytes of a row, one cache line

struct Segment {
  const void* a;
  const void* b;
  const void* b2;  // second matrix of a double product
  uint64_t lda, ldb, ldb2;
};

struct ProductArgs {
  Segment seg[kMaxSegments];
  uint64_t batch_a, batch_b;  // elements from one matrix of a stack to the next
  uint32_t m, n, k;
  uint32_t nseg, seg_steps;   // segments; steps of each
  uint32_t tiles_m, tiles_n;
  uint32_t batch;
  uint32_t tiles;             // of one matrix: all, or those on and below the diagonal
  uint32_t full, cuts;        // tiles that a workgroup has whole; workgroups that share the steps of each other one
  float* pieces;              // a tile's sums for each of those
};

template <class T>
struct Frag;
template <>
struct Frag<bf16_t> {
  typedef bf16_t type __attribute__((ext_vector_type(8)));
  typedef bf16_t half __attribute__((ext_vector_type(4)));
};
template <>
struct Frag<f16_t> {
  typedef f16_t type __attribute__((ext_vector_type(8)));
  typedef f16_t half __attribute__((ext_vector_type(4)));
};
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mma(Frag<bf16_t>::type a, Frag<bf16_t>::type b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(Frag<f16_t>::type a, Frag<f16_t>::type b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

#define RSX_LDS __attribute__((address_space(3)))

// Four 16-bit elements of a col tile, turned: of 16 lanes, lane i gives the
// address of elements 4 (i % 4) .. + 3 of k row i / 4, and gets element i of k
// rows 0 .. 3.
template <class T>
__device__ __forceinline__ typename Frag<T>::half turned(RSX_LDS const char* p) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(typename Frag<T>::half,
                            __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<RSX_LDS s16x4*>(const_cast<RSX_LDS char*>(p))));
}

// A tile of BM x BN of C: WM x WN waves, each TM x 16 rows by TN x 16 columns.
template <int BM_, int BN_, int WM_, int WN_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int kThreads = 64 * WM * WN;
  static constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
  static constexpr int kBytesA = BM * kStep, kBytesB = BN * kStep * 2;  // of a piece
};

// LDS of two steps: six arrays, which the compiler can tell apart, so that it
// lets a read of one pass loads into the others.
struct Stage {
  RSX_LDS char *a0, *a1, *b;
};
#define RSX_PRODUCT_LDS(TILE, first, second)                                                                              \
  __shared__ __attribute__((aligned(1024))) char lds_a00[TILE::kBytesA], lds_a01[TILE::kBytesA], lds_b0[TILE::kBytesB];   \
  __shared__ __attribute__((aligned(1024))) char lds_a10[TILE::kBytesA], lds_a11[TILE::kBytesA], lds_b1[TILE::kBytesB];   \
  const Stage first = {(RSX_LDS char*)lds_a00, (RSX_LDS char*)lds_a01, (RSX_LDS char*)lds_b0};                            \
  const Stage second = {(RSX_LDS char*)lds_a10, (RSX_LDS char*)lds_a11, (RSX_LDS char*)lds_b1}

// A tile's place in LDS.  B's tile is one piece; A's is two, one for the first
// and one for the second half of every wave's rows, which are read one after
// the other and loaded again as soon as each has been read.  Row r of piece h is
// the tile's row of wave row r / HR, at h * HR + r % HR.  A row piece holds 64 k
// of a row side by side, a col piece all rows of a k.  Either is made of 16-byte
// chunks, moved within their 128 bytes or more so that lanes that read one column
// meet other banks: row pieces keep chunk c of row r at c ^ (r % 8), col pieces
// chunk c of k at c ^ 2 turn(k): the lanes of a transposing read that meet in a
// cycle are of k .. k + 3 and k + 8 .. k + 11, 32 bytes each.
template <int LAYOUT, int ROWS>
struct Piece {
  static constexpr int kBytes = ROWS * kStep * 2;
  static constexpr int kChunks = LAYOUT == kRow ? 8 : ROWS / 8;  // of an LDS row
  static_assert(LAYOUT == kRow || kChunks >= 8, "");
  static __device__ __forceinline__ uint32_t turn(uint32_t k) {
    // rows of 128 bytes: the k's lowest bit is a bank's already
    return kChunks == 8 ? (k >> 1 & 1) | (k >> 2 & 2) : (k & 3) | (k >> 1 & 4);
  }
  static __device__ __forceinline__ uint32_t moved(uint32_t row) { return LAYOUT == kRow ? row & 7 : turn(row) << 1; }
};

// Loads of one operand's pieces, straight into LDS: each lane moves 16 bytes, a
// wave's 64 lanes fill 1 KB in order, and which chunk a lane asks for says what
// goes there.  The buffer's range gives zeros past the last row (row) or the
// last k (col), `beyond` past the last k of a row.  DUAL: of each 64 rows, 32 are
// of the first matrix and the same 32 of the second.
template <int LAYOUT, int ROWS, int THREADS, int PIECES, int HR, bool DUAL>
struct Loader {
  typedef Piece<LAYOUT, ROWS / PIECES> P;
  static constexpr int kLoads = P::kBytes / (THREADS * 16);  // of a piece
  static constexpr int kRowsPerLoad = THREADS / P::kChunks;
  static constexpr bool kBoth = DUAL && kRowsPerLoad == 32;  // loads alternate; otherwise half of the waves has each matrix
  static_assert(kLoads >= 1 && (!DUAL || (LAYOUT == kRow && PIECES == 1 && (kRowsPerLoad == 64 || kRowsPerLoad == 32))), "");
  const char* base[kBoth ? 2 : 1];
  uint32_t stride[kBoth ? 2 : 1];  // bytes
  uint32_t side;                   // rows but the last (row), bytes of the last k row (col)
  uint32_t offset[PIECES][kLoads];
  uint32_t chunk;

  // first: the tile's first row, of `count`; step: the first k step.
  __device__ __forceinline__ void open(const void* m1, uint64_t ld1, const void* m2, uint64_t ld2, uint32_t first, uint32_t count,
                                       uint32_t step) {
    const uint32_t t = threadIdx.x, r = t / P::kChunks;
    chunk = (t % P::kChunks) ^ P::moved(r);
    static_assert(LAYOUT == kRow ? kRowsPerLoad % 8 == 0 : kRowsPerLoad % 16 == 0, "");
    if (DUAL && !kBoth && uniform(t / 64) >= THREADS / 128) {
      m1 = m2;
      ld1 = ld2;
    }
    open_one(0, m1, ld1, first, step);
    if constexpr (kBoth) open_one(1, m2, ld2, first, step);
    side = LAYOUT == kRow ? min(static_cast<uint32_t>(DUAL ? ROWS / 2 : ROWS), count - first) - 1 : (count - first) * 2;
#pragma unroll
    for (int h = 0; h < PIECES; ++h)
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint32_t q = r + i * kRowsPerLoad;  // LDS row
        if constexpr (LAYOUT == kRow) {
          const uint32_t row = kBoth ? r + i / 2 * 32 : DUAL ? r % 32 + i * 32 : tile_row(h, q);
          offset[h][i] = row * stride[kBoth ? i % 2 : 0] + chunk * 16;
        } else {
          offset[h][i] = q * stride[0] + tile_row(h, chunk * 8) * 2;
        }
      }
  }
  static __device__ __forceinline__ uint32_t tile_row(int h, uint32_t r) {
    return PIECES == 1 ? r : r / HR * (2 * HR) + h * HR + r % HR;
  }
  __device__ __forceinline__ void open_one(int i, const void* m, uint64_t ld, uint32_t first, uint32_t step) {
    const uint64_t at = LAYOUT == kRow ? first * ld + step * kStep : step * kStep * ld + first;
    base[i] = static_cast<const char*>(m) + at * 2;
    stride[i] = static_cast<uint32_t>(ld) * 2;
  }
  // left: k from this step's first on; 0 for a step past the last one (all zeros).
  // Loads from .. to - 1 of a piece.
  __device__ __forceinline__ void issue(RSX_LDS char* lds, int h, int from, int to, uint32_t left) const {
    const uint32_t wave = uniform(threadIdx.x / 64);
    const uint32_t beyond = LAYOUT == kRow && chunk * 8 >= left ? 0xffffffffu : 0u;
    __amdgpu_buffer_rsrc_t r[kBoth ? 2 : 1];
#pragma unroll
    for (int i = 0; i < (kBoth ? 2 : 1); ++i) {
      const uint32_t bytes = LAYOUT == kRow ? side * stride[i] + left * 2 : (min(kStep, left) - 1) * stride[i] + side;
      r[i] = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base[i]), 0, left != 0 ? bytes : 0, 0x00027000);
    }
#pragma unroll
    for (int i = from; i < to; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r[kBoth ? i % 2 : 0],
                                               reinterpret_cast<RSX_LDS void*>(lds + wave * 1024 + i * (THREADS * 16)), 16,
                                               static_cast<int>(offset[h][i] | beyond), 0, 0, 0);
  }
  __device__ __forceinline__ void advance() {
#pragma unroll
    for (int i = 0; i < (kBoth ? 2 : 1); ++i)
      base[i] += LAYOUT == kRow ? kStep * 2 : static_cast<uint64_t>(stride[i]) * kStep;
  }
};

// One operand's fragments of a step's half kk (32 k): 16 rows each, from row
// `first` of the piece on.
template <class T, int LAYOUT, int ROWS>
struct Reader {
  typedef Piece<LAYOUT, ROWS> P;
  uint32_t at;  // this lane's byte in the piece
  __device__ __forceinline__ explicit Reader(uint32_t first) {
    const uint32_t l = threadIdx.x % 64, g = l / 16, i = l % 16;
    if constexpr (LAYOUT == kRow) {
      at = (first + i) * 128 + ((g ^ (l & 7)) << 4);
    } else {
      const uint32_t k = 8 * g + i / 4;
      at = k * (ROWS * 2) + (((first / 16) ^ P::turn(k)) * 32) + (i % 4) * 8;
    }
  }
  __device__ __forceinline__ typename Frag<T>::type get(RSX_LDS const char* lds, int kk, int j) const {
    if constexpr (LAYOUT == kRow) {
      return *reinterpret_cast<RSX_LDS const typename Frag<T>::type*>(lds + (at ^ (kk * 64)) + j * 2048);
    } else {
      const uint32_t a = at ^ (j * 32);
      const auto lo = turned<T>(lds + a + kk * (32 * ROWS * 2));
      const auto hi = turned<T>(lds + a + kk * (32 * ROWS * 2) + 4 * ROWS * 2);
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

// Which tile of C a workgroup has: consecutive workgroups go to the eight XCDs
// in turn, and each XCD has an L2 of its own, so an XCD takes a run of tiles;
// in a run, eight tile rows share each tile column's operand.
__device__ __forceinline__ uint32_t xcd_run(uint32_t id, uint32_t total) {
  const uint32_t each = total / 8, more = total % 8, x = id % 8;
  return x * each + min(x, more) + id / 8;
}

template <int N>
struct Int {
  static constexpr int value = N;
};

struct Where {
  uint32_t m0, n0, batch;
};

// Tile t of all matrices'.
template <class TILE, bool DUAL, bool TRIANGLE>
__device__ __forceinline__ Where where_of(const ProductArgs& p, uint32_t t) {
  Where w;
  w.batch = t / p.tiles;
  t %= p.tiles;
  uint32_t i, j;
  constexpr uint32_t kGroup = 8;
  if (TRIANGLE) {
    // Before row i are i (i + 1) / 2 tiles; the root says which row t would be in, row after row, and with it the group.
    auto before = [](uint32_t row) { return static_cast<uint32_t>(static_cast<uint64_t>(row) * (row + 1) / 2); };
    auto row_of = [&](uint32_t x) {
      uint32_t r = static_cast<uint32_t>((sqrtf(8.0f * static_cast<float>(x) + 1.0f) - 1.0f) * 0.5f);  // off by one at most
      while (before(r) > x) --r;
      while (before(r + 1) <= x) ++r;
      return r;
    };
    const uint32_t first = row_of(t) / kGroup * kGroup, rows = min(kGroup, p.tiles_m - first);
    t -= before(first);
    if (t < rows * first) {  // the group's columns up to the diagonal's block
      i = first + t % rows;
      j = t / rows;
    } else {
      t -= rows * first;
      i = row_of(t);
      j = first + t - before(i);
      i += first;
    }
  } else {
    const uint32_t group = t / (kGroup * p.tiles_n), first = group * kGroup, rows = min(kGroup, p.tiles_m - first);
    t -= group * kGroup * p.tiles_n;
    i = first + t % rows;
    j = t / rows;
  }
  w.m0 = uniform(i * TILE::BM);
  w.n0 = uniform(j * (DUAL ? TILE::BN / 2 : TILE::BN));
  w.batch = uniform(w.batch);
  return w;
}

// The sums of a tile.  acc[j][i]: lane l has row m = 16 i + l % 16 of its wave's
// rows and columns n = 16 j + 4 (l / 16) .. + 3: four that lie side by side.  (Of a
// double product, j below TN / 2 is the first matrix, the others the second.)
//
// Two steps are in LDS.  A step has four phases, a quarter of its matrix
// instructions each: the first and second halves of the wave's rows, of each the
// two halves of the step's k.  Fragments are read one phase ahead, over the two
// barriers too.  After the first barrier all waves have read B and A's first
// piece, after the second A's second piece; both are loaded again for the step
// after the next, a quarter of the loads in each phase: loads wait for each other
// where they start, and what waits with them is the matrix instructions behind
// them (8192^3: 918 us with six of eight loads in one phase, 894 so).
//
// The matrix instructions are busy 71% of the time at about 1.75 GHz, and what makes
// them busier lowers the clock (the library's product: 87% at 1.55 GHz).  8192^3 bf16
// 1220 to 1250 TFLOP/s, whichever side k is on; with long k in the operators 1390 to
// 1457.  (The library's product: 1517 with k side by side in both, 1383 in one,
// 1194 in neither.)  Four waves of 128 x 128 each: 1091 TFLOP/s, fewer waves to
// change over to; instructions of 32 x 32 x 16: busier, at 1.62 GHz, 5% slower.
template <class T, class TILE, int LA, int LB, bool DUAL>
__device__ __forceinline__ void tile_product(const ProductArgs& p, const Where& w, uint32_t begin, uint32_t end, const Stage& st0,
                                             const Stage& st1, f32x4 (&acc)[TILE::TN][TILE::TM]) {
  constexpr int TM = TILE::TM, TN = TILE::TN, THREADS = TILE::kThreads, H = TM / 2;
  typedef Loader<LA, TILE::BM, THREADS, 2, H * 16, false> LoadA;
  typedef Loader<LB, TILE::BN, THREADS, 1, 0, DUAL> LoadB;
  constexpr int NA = LoadA::kLoads, NB = LoadB::kLoads / 2;  // loads of a phase
  static_assert(TM % 2 == 0 && LoadB::kLoads % 2 == 0 && 2 * NA + 2 * NB <= 15, "");
  const uint32_t wave = uniform(threadIdx.x / 64);
  LoadA load_a;
  LoadB load_b;
  const Reader<T, LA, TILE::BM / 2> read_a((wave / TILE::WN) * (H * 16));
  const Reader<T, LB, TILE::BN> read_b((wave % TILE::WN) * (TN * 16));
#pragma unroll
  for (int j = 0; j < TN; ++j)
#pragma unroll
    for (int i = 0; i < TM; ++i) acc[j][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  uint32_t s = begin / p.seg_steps, k = begin % p.seg_steps, ahead = begin;
  auto open = [&]() {
    const Segment& g = p.seg[s];
    load_a.open(static_cast<const char*>(g.a) + w.batch * p.batch_a * 2, g.lda, nullptr, 0, w.m0, LA == kRow ? p.m : (p.m + 7) & ~7u, k);
    load_b.open(static_cast<const char*>(g.b) + w.batch * p.batch_b * 2, g.ldb, g.b2, g.ldb2, w.n0, LB == kRow ? p.n : (p.n + 7) & ~7u, k);
  };
  // Quarter q of a step's loads.
  const uint32_t whole = (p.k + 7) & ~7u;  // rows are filled with zeros to a multiple of 16 bytes
  auto fetch = [&](const Stage& st, int q) {
    const uint32_t left_a = ahead < end ? (LA == kRow ? whole : p.k) - k * kStep : 0;
    const uint32_t left_b = ahead < end ? (LB == kRow ? whole : p.k) - k * kStep : 0;
    if (q < 2) load_b.issue(st.b, 0, q * NB, (q + 1) * NB, left_b);
    if (q == 2) load_a.issue(st.a0, 0, 0, NA, left_a);
    if (q == 3) load_a.issue(st.a1, 1, 0, NA, left_a);
  };
  auto advance = [&]() {
    ++ahead;
    load_a.advance();
    load_b.advance();
    if (++k == p.seg_steps && ahead < end) {
      k = 0;
      ++s;
      open();
    }
  };
  typename Frag<T>::type a[2][H], b[2][TN];
  auto get_a = [&](RSX_LDS const char* lds, int kk) {
#pragma unroll
    for (int i = 0; i < H; ++i) a[kk][i] = read_a.get(lds, kk, i);
  };
  auto get_b = [&](RSX_LDS const char* lds, int kk) {
#pragma unroll
    for (int j = 0; j < TN; ++j) b[kk][j] = read_b.get(lds, kk, j);
  };
  constexpr int kReadA = (LA == kRow ? 1 : 2) * H, kReadB = (LB == kRow ? 1 : 2) * TN;
  auto multiply = [&](int h, int kk, int reads) {
#pragma unroll
    for (int i = 0; i < H; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[j][h * H + i] = mma(b[kk][j], a[kk][i], acc[j][h * H + i]);
    // The order of a phase: its reads between its first matrix instructions, its loads apart.
    constexpr int kAll = H * TN, kFirst = kAll / 2;
#pragma unroll
    for (int i = 0; i < reads; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      if (i * kFirst / reads != (i + 1) * kFirst / reads) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x010, NA - NA / 2, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, kAll / 4, 0);
    __builtin_amdgcn_sched_group_barrier(0x010, NA / 2, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, kAll, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  // All but the last FLYING loads are there, and this wave's reads are done.
  // (A fence here would have the compiler wait for all loads.)
  auto meet = [&](auto flying) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070 | decltype(flying)::value);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  auto step = [&](const Stage& here, const Stage& next) {
    get_b(here.b, 1);
    get_a(here.a0, 1);
    fetch(next, 3);
    multiply(0, 0, kReadA + kReadB);
    advance();
    meet(Int<2 * NA + 2 * NB>());
    get_a(here.a1, 0);
    fetch(here, 0);
    multiply(0, 1, kReadA);
    get_a(here.a1, 1);
    fetch(here, 1);
    multiply(1, 0, kReadA);
    meet(Int<NA + 2 * NB>());
    get_b(next.b, 0);
    get_a(next.a0, 0);
    fetch(here, 2);
    multiply(1, 1, kReadA + kReadB);
  };
  open();
#pragma unroll
  for (int q = 0; q < 4; ++q) fetch(st0, q);
  advance();
#pragma unroll
  for (int q = 0; q < 3; ++q) fetch(st1, q);
  meet(Int<2 * NA + 2 * NB>());
  get_b(st0.b, 0);
  get_a(st0.a0, 0);
  // Of an odd number of steps, one more is of zeros: a way out in the middle cost
  // the sums' registers twice.
  for (uint32_t at = begin; at < end; at += 2) {
    step(st0, st1);
    step(st1, st0);
  }
  // Loads of steps past the last one still land in LDS: before anything else is there, and before it is another workgroup's.
  __builtin_amdgcn_s_waitcnt(0);
}

// ------------------------------------------------------------ epilogues
typedef float f32x8 __attribute__((ext_vector_type(8)));

// Where a lane's sums belong: acc[j][i] is row(i), columns col(j) .. + 3.
template <class TILE>
struct Place {
  uint32_t m, n;
  __device__ __forceinline__ explicit Place(const Where& w) {
    const uint32_t l = threadIdx.x % 64, wave = threadIdx.x / 64;
    m = w.m0 + wave / TILE::WN * (TILE::TM * 16) + l % 16;
    n = w.n0 + wave % TILE::WN * (TILE::TN * 16) + l / 16 * 4;
  }
  __device__ __forceinline__ uint32_t row(int i) const { return m + i * 16; }
  __device__ __forceinline__ uint32_t col(int j) const { return n + j * 16; }
};

// The sums through LDS, 16 rows of each wave at a time, so that a lane has eight
// columns that lie side by side and a row's 64 columns are eight lanes': whole
// cache lines for the loads and stores of an epilogue, and its code once.
// f(row, column, v), or of a double product f(row, column, v, v2).  A wave's
// patch is its own; 16-byte chunks are moved by the row, against bank conflicts.
// acc holds N of the wave's TM groups of 16 rows, from group i0 on.
//
// With g, f returns values that go back to LDS, and g(row, column, v) has eight
// rows' of one column, from that row on: for stores of the transpose, 16 bytes a
// lane and two lanes side by side.  (One by one from f: 88 us for 74, of 144 large
// tiles of a symmetric product of 32 steps.)
struct NotTurned {};
template <class TILE, bool DUAL, int N, class F, class G = NotTurned>
__device__ __forceinline__ void staged(const Where& w, const f32x4 (&acc)[TILE::TN][N], uint32_t i0, RSX_LDS char* lds, F f, G g = {},
                                       bool turn = true) {
  constexpr bool TURNED = !__is_same(G, NotTurned);
  constexpr int COLS = TILE::TN * 16, CHUNKS = COLS / 4, WIDTH = DUAL ? COLS / 2 : COLS, LANES = WIDTH / 8, ROWS = 64 / LANES;
  static_assert(TILE::WM * TILE::WN * 16 * COLS * 4 <= TILE::kBytesB, "");
  const uint32_t l = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
  RSX_LDS char* patch = lds + wave * (16 * COLS * 4);
  auto chunk = [&](uint32_t row, uint32_t c) { return reinterpret_cast<RSX_LDS f32x4*>(patch + row * (COLS * 4) + ((c ^ (row % CHUNKS)) * 16)); };
  __syncthreads();
#pragma nounroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int q = 0; q < N; ++q)
      if (q == i) {
#pragma unroll
        for (int j = 0; j < TILE::TN; ++j) *chunk(l % 16, j * 4 + l / 16) = acc[j][q];
      }
    __builtin_amdgcn_wave_barrier();
    const uint32_t c = l % LANES;
#pragma nounroll
    for (uint32_t r = l / LANES; r < 16; r += ROWS) {
      const uint32_t row = w.m0 + wave / TILE::WN * (TILE::TM * 16) + (i0 + i) * 16 + r, col = w.n0 + wave % TILE::WN * WIDTH + c * 8;
      const f32x8 v = __builtin_shufflevector(*chunk(r, 2 * c), *chunk(r, 2 * c + 1), 0, 1, 2, 3, 4, 5, 6, 7);
      if constexpr (DUAL) {
        f(row, col, v,
          __builtin_shufflevector(*chunk(r, CHUNKS / 2 + 2 * c), *chunk(r, CHUNKS / 2 + 2 * c + 1), 0, 1, 2, 3, 4, 5, 6, 7));
      } else if constexpr (TURNED) {
        const f32x8 back = f(row, col, v);
        if (turn) {
          *chunk(r, 2 * c) = __builtin_shufflevector(back, back, 0, 1, 2, 3);
          *chunk(r, 2 * c + 1) = __builtin_shufflevector(back, back, 4, 5, 6, 7);
        }
      } else {
        f(row, col, v);
      }
    }
    __builtin_amdgcn_wave_barrier();
    if constexpr (TURNED) {
      if (turn) {
#pragma nounroll
        for (uint32_t t = l; t < 2 * COLS; t += 64) {
          const uint32_t x = t / 2, r = t % 2 * 8;
          f32x8 v;
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = reinterpret_cast<RSX_LDS const float*>(chunk(r + e, x / 4))[x % 4];
          g(w.m0 + wave / TILE::WN * (TILE::TM * 16) + (i0 + i) * 16 + r, w.n0 + wave % TILE::WN * WIDTH + x, v);
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
}

// N elements of a row; past the row's end nothing is touched.
template <class T, int N>
__device__ __forceinline__ void put(T* row, uint32_t c, uint32_t n, typename Vec<float, N>::type v) {
  const auto h = __builtin_convertvector(v, typename Vec<T, N>::type);
  if (c + N <= n) {
    *reinterpret_cast<typename Vec<T, N>::loose*>(row + c) = h;
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (c + e < n) row[c + e] = h[e];
  }
}
template <class T, int N>
__device__ __forceinline__ typename Vec<float, N>::type get(const T* row, uint32_t c, uint32_t n) {
  typedef typename Vec<float, N>::type V;
  if (c + N <= n) return __builtin_convertvector(*reinterpret_cast<const typename Vec<T, N>::loose*>(row + c), V);
  V v = {};
#pragma unroll
  for (int e = 0; e < N; ++e)
    if (c + e < n) v[e] = static_cast<float>(row[c + e]);
  return v;
}
template <int N>
__device__ __forceinline__ void put_as(int type, void* p, uint64_t at, uint32_t c, uint32_t n, typename Vec<float, N>::type v) {
  if (type == RSX_FLOAT32) put<float, N>(static_cast<float*>(p) + at, c, n, v);
  else if (type == RSX_BFLOAT16) put<bf16_t, N>(static_cast<bf16_t*>(p) + at, c, n, v);
  else put<f16_t, N>(static_cast<f16_t*>(p) + at, c, n, v);
}
template <int N>
__device__ __forceinline__ typename Vec<float, N>::type get_as(int type, const void* p, uint64_t at, uint32_t c, uint32_t n) {
  if (type == RSX_FLOAT32) return get<float, N>(static_cast<const float*>(p) + at, c, n);
  if (type == RSX_BFLOAT16) return get<bf16_t, N>(static_cast<const bf16_t*>(p) + at, c, n);
  return get<f16_t, N>(static_cast<const f16_t*>(p) + at, c, n);
}

// A matrix of values kept as sums of 16-bit parts, rows of `ld` elements (a
// multiple of 8) with zeros behind the last column.
struct Parts {
  void* part[3];
  uint64_t ld;
  int count;
};

// N values as `count` parts, rounded to nearest each, by f(which, part).
// A value that bf16 rounds to infinity has bf16's largest as a part.  An infinity
// is the last part's, which is multiplied with first parts alone, and 1 with its
// sign is the first part: with an infinity in the first part, its products with the
// other matrix's lower parts, which may be 0 or of the other sign, would be NaN.
// (fp16's parts are of values within its range.)
template <class T, int N, class F>
__device__ __forceinline__ void take_parts(typename Vec<float, N>::type v, int count, F f) {
  typedef typename Vec<T, N>::type V;
  typedef typename Vec<float, N>::type W;
  if (__is_same(T, bf16_t) && count > 1) {
    float most = 0.0f;
#pragma unroll
    for (int e = 0; e < N; ++e) most = fmaxf(most, fabsf(v[e]));
    if (most >= 0x1.ffp127f) {
#pragma nounroll
      for (int i = 0; i < count; ++i) {
        W back = __builtin_convertvector(__builtin_convertvector(v, V), W);
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (i + 1 < count && fabsf(back[e]) == INFINITY)
            back[e] = copysignf(fabsf(v[e]) < INFINITY ? 0x1.fep127f : i == 0 ? 1.0f : 0.0f, v[e]);
        f(i, __builtin_convertvector(back, V));
        v -= back;
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if (i >= count) break;
    const V h = __builtin_convertvector(v, V);
    f(i, h);
    const W back = __builtin_convertvector(h, W);
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = __is_same(T, bf16_t) || fabsf(back[e]) < INFINITY ? v[e] - back[e] : 0.0f;
  }
}
template <class T, int N>
__device__ __forceinline__ void put_parts(const Parts& p, uint64_t row, uint32_t c, uint32_t n, typename Vec<float, N>::type v) {
  const uint64_t at = row * p.ld + c;
  if (p.count == 0 || c >= ((n + 7) & ~7u)) return;
#pragma unroll
  for (int e = 0; e < N; ++e)
    if (c + e >= n) v[e] = 0.0f;
  take_parts<T, N>(v, p.count, [&](int i, typename Vec<T, N>::type h) {
    *reinterpret_cast<typename Vec<T, N>::type*>(static_cast<T*>(i == 0 ? p.part[0] : i == 1 ? p.part[1] : p.part[2]) + at) = h;
  });
}
template <class T, int N>
__device__ __forceinline__ typename Vec<float, N>::type get_parts(const Parts& p, uint64_t row, uint32_t c) {
  typedef typename Vec<float, N>::type V;
  V v = {};
#pragma unroll
  for (int i = 2; i >= 0; --i)
    if (i < p.count)
      v += __builtin_convertvector(*reinterpret_cast<const typename Vec<T, N>::type*>(static_cast<const T*>(p.part[i]) + row * p.ld + c), V);
  return v;
}

// A tile's sums as they lie in the lanes.
template <class TILE>
__device__ __forceinline__ f32x4* sums_at(const ProductArgs& p, uint32_t slot) {
  return reinterpret_cast<f32x4*>(p.pieces) + static_cast<uint64_t>(slot) * (TILE::TN * TILE::TM * TILE::kThreads) + threadIdx.x;
}
template <class T, class TILE, int LA, int LB, bool DUAL, bool TRIANGLE, class EPILOGUE>
__global__ __launch_bounds__(TILE::kThreads, 2) void full_tiles(const ProductArgs p, const typename EPILOGUE::Args e) {
#ifdef __HIP_DEVICE_COMPILE__  // the host's compiler takes no part in the body
  const uint64_t id = block_id();
  if (id >= p.full) return;
  RSX_PRODUCT_LDS(TILE, st0, st1);
  const Where w = where_of<TILE, DUAL, TRIANGLE>(p, xcd_run(static_cast<uint32_t>(id), p.full));
  f32x4 acc[TILE::TN][TILE::TM];
  tile_product<T, TILE, LA, LB, DUAL>(p, w, 0, p.nseg * p.seg_steps, st0, st1, acc);
  EPILOGUE::template run<T, TILE, TILE::TM>(p, w, e, acc, 0, st0.b);
#endif
}

// The tiles past the last full round of the CUs, few of them: `cuts` workgroups
// have a stretch of each one's steps, all of them in step (the first stretches of
// all tiles, then the second ones), so that what their rows and columns have in
// common is read once.  Another launch adds a tile's pieces in their order and
// has its epilogue.  (The tiles' steps laid end to end and shared out evenly, any
// number of tiles, were slower than an unfilled round: workgroups at different k
// share nothing in the L2.)
template <class T, class TILE, int LA, int LB, bool DUAL, bool TRIANGLE>
__global__ __launch_bounds__(TILE::kThreads, 2) void cut_tiles(const ProductArgs p) {
#ifdef __HIP_DEVICE_COMPILE__
  const uint64_t id = block_id();
  const uint32_t rest = p.tiles * p.batch - p.full, total = p.nseg * p.seg_steps;
  if (id >= static_cast<uint64_t>(rest) * p.cuts) return;
  RSX_PRODUCT_LDS(TILE, st0, st1);
  const uint32_t slot = xcd_run(static_cast<uint32_t>(id), rest * p.cuts), cut = slot / rest;
  const Where w = where_of<TILE, DUAL, TRIANGLE>(p, p.full + slot % rest);
  f32x4 acc[TILE::TN][TILE::TM];
  tile_product<T, TILE, LA, LB, DUAL>(p, w, static_cast<uint32_t>(static_cast<uint64_t>(total) * cut / p.cuts),
                                      static_cast<uint32_t>(static_cast<uint64_t>(total) * (cut + 1) / p.cuts), st0, st1, acc);
  f32x4* q = sums_at<TILE>(p, slot);
#pragma unroll
  for (int j = 0; j < TILE::TN; ++j)
#pragma unroll
    for (int i = 0; i < TILE::TM; ++i) q[(j * TILE::TM + i) * TILE::kThreads] = acc[j][i];
#endif
}

// A workgroup for each group of 16 rows of the tile's waves.
template <class T, class TILE, bool DUAL, bool TRIANGLE, class EPILOGUE>
__global__ __launch_bounds__(TILE::kThreads, 2) void finish_tiles(const ProductArgs p, const typename EPILOGUE::Args e) {
#ifdef __HIP_DEVICE_COMPILE__
  const uint64_t id = block_id();
  const uint32_t rest = p.tiles * p.batch - p.full;
  if (id >= static_cast<uint64_t>(rest) * TILE::TM) return;
  __shared__ __attribute__((aligned(1024))) char lds[TILE::kBytesB];
  const uint32_t tile = static_cast<uint32_t>(id / TILE::TM), i0 = static_cast<uint32_t>(id % TILE::TM);
  const Where w = where_of<TILE, DUAL, TRIANGLE>(p, p.full + tile);
  f32x4 acc[TILE::TN][1];
#pragma unroll
  for (int j = 0; j < TILE::TN; ++j) acc[j][0] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (uint32_t cut = 0; cut < p.cuts; ++cut) {
    const f32x4* q = sums_at<TILE>(p, cut * rest + tile) + i0 * TILE::kThreads;
#pragma unroll
    for (int j = 0; j < TILE::TN; ++j) acc[j][0] += q[j * TILE::TM * TILE::kThreads];
  }
  EPILOGUE::template run<T, TILE, 1>(p, w, e, acc, i0, (RSX_LDS char*)lds);
#endif
}

// ------------------------------------------------------------- host side
typedef Tile<256, 256, 2, 4> Large;
typedef Tile<128, 128, 2, 2> Middle;
typedef Tile<64, 64, 2, 2> Small;

// One operand: parts of a matrix with a common row stride.
struct Operand {
  const void* part[3];
  uint64_t ld;
};

// Products of the parts i of A and j of B, the smallest first.  What is left out,
// i + j from the larger count on, is below the last part's own rounding.
inline void add_segments(ProductArgs& p, const Operand& a, int parts_a, const Operand& b, int parts_b, const Operand* b2 = nullptr) {
  for (int sum = (parts_a > parts_b ? parts_a : parts_b) - 1; sum >= 0; --sum)
    for (int i = sum; i >= 0; --i)
      if (i < parts_a && sum - i < parts_b)
        p.seg[p.nseg++] = {a.part[i], b.part[sum - i], b2 ? b2->part[sum - i] : nullptr, a.ld, b.ld, b2 ? b2->ld : 0};
}
// How many.
inline uint64_t segments_of(int parts_a, int parts_b) {
  ProductArgs p = {};
  add_segments(p, {}, parts_a, {}, parts_b);
  return p.nseg;
}

// How a product m x n of `steps` steps is spread over the CUs: the tile, and how
// many tiles a workgroup has whole; the others' steps are cut.
struct Schedule {
  int tile;  // 0 large, 1 middle, 2 small
  uint32_t full, cuts;
  uint64_t bytes;  // of the pieces' sums
};
Schedule schedule(uint64_t m, uint64_t n, uint64_t batch, uint64_t steps, bool triangle, bool small);

// Sets what a schedule says; n as the schedule's (of a double product, both matrices' columns).
template <class TILE>
void set_tiles(ProductArgs& p, const Schedule& c, void* pieces, bool dual, bool triangle) {
  const uint32_t bn = dual ? TILE::BN / 2 : TILE::BN;
  p.seg_steps = p.k == 0 ? 1 : (p.k + kStep - 1) / kStep;
  p.tiles_m = (p.m + TILE::BM - 1) / TILE::BM;
  p.tiles_n = (p.n + bn - 1) / bn;
  p.tiles = static_cast<uint32_t>(triangle ? static_cast<uint64_t>(p.tiles_m) * (p.tiles_m + 1) / 2
                                           : static_cast<uint64_t>(p.tiles_m) * p.tiles_n);
  p.full = c.full;
  p.cuts = c.cuts;
  p.pieces = static_cast<float*>(pieces);
}

template <class T, class TILE, int LA, int LB, bool DUAL, bool TRIANGLE, class EPILOGUE>
hipError_t launch_tiles(ProductArgs p, const Schedule& c, void* pieces, const typename EPILOGUE::Args& e, hipStream_t s) {
  set_tiles<TILE>(p, c, pieces, DUAL, TRIANGLE);
  if (p.full != 0) {
    const hipError_t st = launch(full_tiles<T, TILE, LA, LB, DUAL, TRIANGLE, EPILOGUE>, grid_of(p.full), TILE::kThreads, 0, s, p, e);
    if (st != hipSuccess) return st;
  }
  const uint32_t rest = p.tiles * p.batch - p.full;
  if (rest == 0) return hipSuccess;
  const hipError_t st = launch(cut_tiles<T, TILE, LA, LB, DUAL, TRIANGLE>, grid_of(static_cast<uint64_t>(rest) * p.cuts), TILE::kThreads, 0, s, p);
  if (st != hipSuccess) return st;
  return launch(finish_tiles<T, TILE, DUAL, TRIANGLE, EPILOGUE>, grid_of(static_cast<uint64_t>(rest) * TILE::TM), TILE::kThreads, 0, s, p,
                e);
}
template <class T, int LA, int LB, bool DUAL, bool TRIANGLE, class EPILOGUE>
hipError_t launch_product(const ProductArgs& p, const Schedule& c, void* pieces, const typename EPILOGUE::Args& e, hipStream_t s) {
  return c.tile == 0 ? launch_tiles<T, Large, LA, LB, DUAL, TRIANGLE, EPILOGUE>(p, c, pieces, e, s)
                     : launch_tiles<T, Middle, LA, LB, DUAL, TRIANGLE, EPILOGUE>(p, c, pieces, e, s);
}

}  // namespace rsx
