// Embedding lookup with scaling, and its gradient: by sorted tokens, or for few
// tokens each by its own search.
//
//   out[i, :]  = scale * table[t_i, :]          t_i = tokens[i] - first
//   grad[v, :] = (grad[v, :] +) scale * sum of dout[i, :] over the i with t_i = v
//
// A token outside [0, vocab) gives a row of zeros and no gradient.
#include <algorithm>

#include "step_device.h"

namespace rsx {
namespace {

constexpr int kThreads = 256;

template <class I>
__device__ __forceinline__ uint64_t token_row(const void* tokens, uint64_t i, int64_t first) {
  // Unsigned: a token below `first` wraps to a row far past any table's end.
  return static_cast<uint64_t>(static_cast<int64_t>(static_cast<const I*>(tokens)[i])) - static_cast<uint64_t>(first);
}
__device__ __forceinline__ uint64_t token_row(const void* tokens, uint64_t i, int64_t first, int wide) {
  return wide ? token_row<int64_t>(tokens, i, first) : token_row<int32_t>(tokens, i, first);
}
// Rows of tokens i, i + step, ..., all asked for at once: with the test of
// `wide` around each, those of 4 bytes would be waited for in turn.  Past `last`: of that.
template <int N>
__device__ __forceinline__ void token_rows(const void* tokens, uint32_t i, uint32_t step, uint32_t last, int64_t first,
                                           int wide, uint64_t (&rows)[N]) {
  if (wide) {
#pragma unroll
    for (int j = 0; j < N; ++j) rows[j] = token_row<int64_t>(tokens, min(i + j * step, last), first);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) rows[j] = token_row<int32_t>(tokens, min(i + j * step, last), first);
  }
}

// Elements of a vector of the gradient: 16 bytes of the wider type, so that
// each of a wave's accesses covers one unbroken span on either side.
template <class T, class U>
constexpr int kVector = sizeof(T) == 4 || sizeof(U) == 4 ? 4 : 8;

// Lanes that one row of `dim` fills, a power of two up to a wave.
inline uint32_t lanes_of(uint64_t dim, uint32_t e) {
  uint32_t lanes = 1;
  while (lanes < 64 && static_cast<uint64_t>(lanes) * e < dim) lanes *= 2;
  return lanes;
}

// ---------------------------------------------------------------- lookup
// A wave copies V vectors per lane of one row: 64 * V * E elements.  A vector
// has 16 bytes of the output, which is streamed; the table's side goes through
// the caches, where pieces join (fp32 to bf16, 16384 rows of 4096: 47.4 us; by
// 16 bytes of the table 49.2).
template <class T, class U, int V>
__global__ __launch_bounds__(kThreads) void lookup_kernel(EmbedArgs a, uint32_t chunks) {
  constexpr int E = 16 / sizeof(U);
  const uint32_t lane = threadIdx.x % 64;
  const uint64_t item = uniform64(block_id() * (kThreads / 64) + threadIdx.x / 64);
  const uint64_t i = item / chunks;
  if (i >= a.n) return;
  const uint32_t dim = static_cast<uint32_t>(a.dim);
  const uint32_t base = static_cast<uint32_t>(item - i * chunks) * (64 * V * E) + lane * E;
  const uint64_t row = uniform64(token_row(a.tokens, i, a.first, a.wide));
  U* out = static_cast<U*>(a.out) + i * a.out_stride;
  typename Vec<T, E>::type v[V] = {};
  if (row < a.vocab) {
    const T* src = static_cast<const T*>(a.table) + row * a.table_stride;
    // Kept: frequent tokens' rows are read again from the caches.
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = load_wide<T, E, false>(src, base + j * 64 * E, dim);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t e = base + j * 64 * E;
      store_row<U, E>(out, e, dim, narrow<U, E>(widen<T, E>(wide_in_place<T, E>(v[j], e, dim)) * a.scale));
    }
  } else {
    const typename Vec<U, E>::type zero = {};
#pragma unroll
    for (int j = 0; j < V; ++j) store_row<U, E>(out, base + j * 64 * E, dim, zero);
  }
}

// Rows of at most half a wave: `lanes` lanes to a row, 64 / lanes rows to a wave.
template <class T, class U>
__global__ __launch_bounds__(kThreads) void lookup_narrow_kernel(EmbedArgs a, uint32_t lanes) {
  constexpr int E = 16 / sizeof(U);
  const uint64_t thread = block_id() * kThreads + threadIdx.x;
  const uint64_t i = thread / lanes;
  const uint32_t dim = static_cast<uint32_t>(a.dim);
  const uint32_t e = static_cast<uint32_t>(thread % lanes) * E;
  if (i >= a.n || e >= dim) return;
  const uint64_t row = token_row(a.tokens, i, a.first, a.wide);
  typename Vec<T, E>::wide f = 0.0f;
  if (row < a.vocab) {
    const T* src = static_cast<const T*>(a.table) + row * a.table_stride;
    f = widen<T, E>(dim >= E ? load_pair<T, E>(src, e, dim) : load_row<T, E, false>(src, e, dim)) * a.scale;
  }
  store_row<U, E>(static_cast<U*>(a.out) + i * a.out_stride, e, dim, narrow<U, E>(f));
}

template <class T, class U, int V>
hipError_t lookup_go(const EmbedArgs& a, hipStream_t s) {
  constexpr int E = 16 / sizeof(U);
  const uint64_t chunks = (a.dim + 64 * V * E - 1) / (64 * V * E);
  const uint64_t grid = (a.n * chunks + kThreads / 64 - 1) / (kThreads / 64);
  return launch(lookup_kernel<T, U, V>, grid_of(grid), kThreads, 0, s, a, static_cast<uint32_t>(chunks));
}

template <class T, class U>
hipError_t lookup(const EmbedArgs& a, hipStream_t s) {
  const uint32_t lanes = lanes_of(a.dim, 16 / sizeof(U));
  if (lanes < 64)
    return launch(lookup_narrow_kernel<T, U>, grid_of((a.n * lanes + kThreads - 1) / kThreads), kThreads, 0, s, a, lanes);
  // No more vectors than the row has (65536 rows of 300 bf16: 15 us, with four
  // 24); one where there is little to do.
  constexpr uint64_t kSpan = 64 * (16 / sizeof(U));
  if (a.n * a.dim < (1u << 22) || a.dim <= kSpan) return lookup_go<T, U, 1>(a, s);
  return a.dim <= 2 * kSpan ? lookup_go<T, U, 2>(a, s) : lookup_go<T, U, 4>(a, s);
}

// ------------------------------------------------------------------- sort
// Stable sort of (row, position) pairs by row, so that a row's positions come
// in increasing order and its sum has one order on every run.  Least
// significant digit first, kDigit bits a pass; a token outside the table has
// the row `vocab` and goes last.
//
// Within a workgroup each wave owns a contiguous part of its tile and counts
// its rows by digit; a scan over (digit, wave) turns the counts into each
// wave's first place for each digit; then every wave takes its part 64
// entries at a time, and an entry's place is the digit's next place plus the
// number of earlier lanes with that digit, found by one compare per bit.
constexpr int kDigit = 9;
constexpr int kBins = 1 << kDigit;
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr uint32_t kSmallSort = 8192;  // tokens that one workgroup sorts in its LDS
constexpr uint32_t kMaxTiles = 64;     // of a larger sort

// Lanes of the wave whose digit equals this lane's, among `valid`.  Sign masks
// and compares by hand take 4 instructions a bit (plain shifts and selects
// become 11), and these are most of what a sort in one workgroup runs.
__device__ __forceinline__ uint64_t same_digit(uint32_t d, uint64_t valid) {
  uint32_t lo = static_cast<uint32_t>(valid), hi = static_cast<uint32_t>(valid >> 32);
#pragma unroll
  for (int b = 0; b < kDigit; ++b) {
    const uint32_t bit = static_cast<uint32_t>(__builtin_amdgcn_sbfe(static_cast<int>(d), b, 1));  // 0 or all ones
    const uint64_t set = __builtin_amdgcn_uicmp(bit, 0u, 33);                                     // lanes where it is not 0
    lo &= ~(static_cast<uint32_t>(set) ^ bit);
    hi &= ~(static_cast<uint32_t>(set >> 32) ^ bit);
  }
  return (static_cast<uint64_t>(hi) << 32) | lo;
}

// Exclusive scan over (digit, wave) of counts[wave][digit] in place, on top of
// `base` for each digit (null: none); every thread of the workgroup calls it.
__device__ void scan_counts(uint32_t (*counts)[kBins], uint32_t* totals, const uint32_t* base) {
  const uint32_t t = threadIdx.x;
  uint32_t sum = 0;
  if (t < kBins) {
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = counts[w][t];
      counts[w][t] = sum;
      sum += c;
    }
  }
  if (base == nullptr) {
    // Inclusive scan of the digits' totals: a wave shuffle scan, then the
    // kBins / 64 waves' sums.
    uint32_t v = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t o = __shfl_up(v, d);
      if (t % 64 >= static_cast<uint32_t>(d)) v += o;
    }
    if (t < kBins && t % 64 == 63) totals[t / 64] = v;
    __syncthreads();
    if (t < kBins) {
      uint32_t before = v - sum;
      for (uint32_t w = 0; w < t / 64; ++w) before += totals[w];
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) counts[w][t] += before;
    }
  } else if (t < kBins) {
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) counts[w][t] += base[t];
  }
  __syncthreads();
}

// Rows that no token names are zeroed beside the sort and the sums: those have
// few workgroups or wait for scattered loads, the zeros are nothing but
// stores, so each hides the other.  A workgroup takes a group of `rows` rows;
// those that a token names are marked as bits of `named`.
constexpr uint32_t kNamedWords = kSortWaves * kBins;  // marks that a workgroup holds in LDS
// Bytes of a group that scans, about: half of it and twice of it take 49.3 and
// 51.7 us for 8192 x 1024 bf16 into 50000 fp32 rows (this 49.3), 119.4 and 120 for
// 4000 x 4096 fp32 into 32000 (117.4), 30.0 and 31.1 for 700 x 1024 bf16 into 50000
// (29.8).
constexpr uint32_t kScanGroup = 3u << 17;
constexpr uint32_t kZeroGroup = 1u << 15;  // bytes of one that does not
// Bytes that a small sort has time for, about, and the joins; the rest is zeroed
// beside the sums.  For 8000 tokens and more (us, with 64 MB, 128 and 256): 1024 columns into
// 50000 fp32 rows 53.7, 49.3, 52.7; 2048 bf16 into 130000 126.8, 122.0, 120.0; 512
// into 400000 fp32 rows 179.3, 170.8, 168.8.  Fewer tokens sort in less time, and 32
// MB would be better: 700 x 1024 into 50000 bf16 rows 25.8 for 29.8, 2000 into 32000
// fp32 rows 32.7 for 35.5.  The joins with none, 24 and 48 MB: 65536 x 4096 into
// 131072 bf16 rows 322, 319.5, 318.3; 8192 x 1024 into 50000 50.8, 49.3, 49.6.
constexpr uint64_t kSortZeros = 128000000;
constexpr uint64_t kJoinZeros = 24000000;
constexpr uint32_t kPlanes = 4;            // sets of marks of the whole table, each from a part of the tokens
struct ZeroPlan {
  const uint32_t* named;  // marks of the whole table, kPlanes times `words`; null: not there
  uint64_t words;
  uint32_t rows, lanes;   // rows of a group; lanes that share a row
  uint32_t magic;         // 2^32 / dim + 1 of a table without gaps, else 0
  uint64_t first, end;    // groups of this launch
};
// Marks of rows v0 .. v0 + rows in LDS, from a scan of tokens begin .. n.
__device__ void mark_rows(const EmbedGradArgs& a, uint64_t v0, uint32_t rows, uint32_t* named, uint32_t begin, uint32_t n) {
  for (uint32_t i = threadIdx.x; i < (rows + 31) / 32; i += kSortThreads) named[i] = 0;
  __syncthreads();
  constexpr int kAhead = 8;
  for (uint32_t i0 = begin + threadIdx.x; i0 < n; i0 += kAhead * kSortThreads) {
    uint64_t r[kAhead];
    token_rows(a.tokens, i0, kSortThreads, n - 1, a.first, a.wide, r);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) r[j] -= v0;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i0 + j * kSortThreads >= n || r[j] >= rows) continue;
      // A frequent token's mark is there already; setting it again would queue.
      const uint32_t word = static_cast<uint32_t>(r[j]) / 32, bit = 1u << (r[j] % 32);
      if ((__hip_atomic_load(&named[word], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP) & bit) == 0)
        atomicOr(&named[word], bit);
    }
  }
  __syncthreads();
}
template <class B>
__device__ __forceinline__ void zero_rows(const EmbedGradArgs& a, const ZeroPlan& z, uint64_t v0, uint32_t rows,
                                          const uint32_t* named, uint32_t planes, uint64_t bit0) {
  constexpr int E = 16 / sizeof(B);
  const uint32_t dim = static_cast<uint32_t>(a.dim);
  const typename Vec<B, E>::type zero = {};
  for (uint32_t r = threadIdx.x / z.lanes; r < rows; r += blockDim.x / z.lanes) {
    const uint64_t bit = bit0 + r;
    uint32_t word = named[bit / 32];
    for (uint32_t p = 1; p < planes; ++p) word |= named[p * z.words + bit / 32];
    if ((word >> (bit % 32)) & 1u) continue;
    B* g = static_cast<B*>(a.grad) + (v0 + r) * a.grad_stride;
    for (uint32_t e = threadIdx.x % z.lanes * E; e < dim; e += z.lanes * E) store_row<B, E>(g, e, dim, zero);
  }
}
// The same of a table without gaps, as one run of 16-byte vectors from a cache
// line's start: rows of any width fill every lane and every line.
template <class B>
__device__ __forceinline__ void zero_run(const EmbedGradArgs& a, const ZeroPlan& z, uint64_t v0, uint32_t rows,
                                         const uint32_t* named) {
  constexpr uint32_t E = 16 / sizeof(B);
  const uint32_t dim = static_cast<uint32_t>(a.dim), n = rows * dim;
  B* g = static_cast<B*>(a.grad) + v0 * a.dim;
  auto row_of = [&](uint32_t e) {
    uint32_t r = __umulhi(e, z.magic);  // the row, or one more
    if (r * dim > e) --r;
    return r;
  };
  auto is_named = [&](uint32_t r) { return (named[r / 32] >> (r % 32)) & 1u; };
  const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(g) % 128 / sizeof(B));
  const typename Vec<B, static_cast<int>(E)>::type zero = {};
  for (uint32_t q = threadIdx.x; q * E < n + off; q += blockDim.x) {
    if (q * E + E <= off) continue;  // before the run
    const uint32_t e = q * E - off;  // wraps where the vector starts before it
    const uint32_t first = q * E < off ? 0u : e, last = min(e + E, n);  // elements of this vector
    uint32_t r = row_of(first);
    uint32_t some = is_named(r);
    for (uint32_t end = (r + 1) * dim; end < last && some == 0; end += dim) some = is_named(++r);
    if (some == 0 && last - first == E) {
      store_once<B, static_cast<int>(E)>(g + e, zero);
    } else {
      for (uint32_t i = first; i < last; ++i)
        if (!is_named(row_of(i))) g[i] = static_cast<B>(0);
    }
  }
}
// Group z.first + block, from the marks of the table or, without, of its own.
template <class B>
__device__ __forceinline__ void zero_group(const EmbedGradArgs& a, const ZeroPlan& z, uint64_t block, uint32_t* lds) {
  const uint64_t group = z.first + block, v0 = group * z.rows;
  if (group >= z.end) return;
  const uint32_t rows = static_cast<uint32_t>(min(static_cast<uint64_t>(z.rows), a.vocab - v0));
  if (z.named != nullptr) return zero_rows<B>(a, z, v0, rows, z.named, kPlanes, v0);
  mark_rows(a, v0, rows, lds, 0, static_cast<uint32_t>(a.n));
  if (z.magic != 0) return zero_run<B>(a, z, v0, rows, lds);
  zero_rows<B>(a, z, v0, rows, lds, 1, 0);
}

// The whole sort of at most kSmallSort tokens in one workgroup.  A lane has its
// 8 entries in registers; they are counted and ranked in one go, an entry's
// rank in its wave being its digit's count so far (8000 tokens of a vocabulary
// of 30000, two passes: 17.0 us, counted by atomics first 19.3; one pass for a
// vocabulary of 500: 13.3 and 11.7).  Bound by the instructions of one CU.
template <class B>
__global__ __launch_bounds__(kSortThreads) void sort_small_kernel(EmbedGradArgs a, int bits, uint32_t* keys,
                                                                  uint32_t* places, ZeroPlan z) {
  constexpr uint32_t kMine = kSmallSort / kSortThreads;
  __shared__ uint32_t key[kSmallSort];
  __shared__ uint16_t place[kSmallSort];
  __shared__ uint32_t counts[kSortWaves][kBins];
  __shared__ uint32_t totals[kBins / 64];
  if (block_id() != 0) return zero_group<B>(a, z, block_id() - 1, &counts[0][0]);
  const uint32_t n = static_cast<uint32_t>(a.n);
  const uint32_t lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
  const uint32_t part = ((n + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;  // entries of a wave, at most 64 * kMine
  const uint32_t begin = min(wave * part, n), end = min(begin + part, n);
  uint64_t rows[kMine];
  token_rows(a.tokens, begin + lane, 64, n - 1, a.first, a.wide, rows);
  uint32_t k[kMine], p[kMine], rank[kMine];
#pragma unroll
  for (uint32_t j = 0; j < kMine; ++j) {
    k[j] = rows[j] < a.vocab ? static_cast<uint32_t>(rows[j]) : static_cast<uint32_t>(a.vocab);
    p[j] = begin + j * 64 + lane;
  }
  for (int shift = 0; shift < bits; shift += kDigit) {
    for (uint32_t i = lane; i < kBins; i += 64) counts[wave][i] = 0;  // the wave's own
    if (shift != 0) {
#pragma unroll
      for (uint32_t j = 0; j < kMine; ++j) {
        const uint32_t i = min(begin + j * 64 + lane, n - 1);
        k[j] = key[i];
        p[j] = place[i];
      }
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (uint32_t j = 0; j < kMine; ++j) {
      if (begin + j * 64 >= end) continue;  // the same for the wave
      const bool there = begin + j * 64 + lane < end;
      const uint32_t d = (k[j] >> shift) % kBins;
      const uint64_t mates = same_digit(d, __ballot(there));
      const uint32_t before = lanes_below(mates);
      const uint32_t c = there ? counts[wave][d] : 0u;
      rank[j] = c + before;
      __builtin_amdgcn_wave_barrier();
      if (there && before == 0) counts[wave][d] = c + static_cast<uint32_t>(__popcll(mates));
      __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    scan_counts(counts, totals, nullptr);
    const bool last = shift + kDigit >= bits;
#pragma unroll
    for (uint32_t j = 0; j < kMine; ++j) {
      if (begin + j * 64 + lane >= end) continue;
      const uint32_t to = counts[wave][(k[j] >> shift) % kBins] + rank[j];
      if (last) {
        keys[to] = k[j];
        places[to] = p[j];
      } else {
        key[to] = k[j];
        place[to] = static_cast<uint16_t>(p[j]);
      }
    }
    __syncthreads();
  }
}

// Digit counts of each tile: hist[tile][digit].  The first pass also marks the
// named rows (`marks`, `marked` rows to a workgroup), later ones zero groups.
template <class B>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(EmbedGradArgs a, const uint32_t* keys_in, int shift,
                                                                  uint32_t tile, uint32_t tiles, uint32_t* hist,
                                                                  uint32_t* marks, uint32_t marked, ZeroPlan z) {
  __shared__ uint32_t counts[kNamedWords];
  if (block_id() >= tiles) {
    if (marks == nullptr) return zero_group<B>(a, z, block_id() - tiles, nullptr);
    const uint32_t plane = static_cast<uint32_t>((block_id() - tiles) % kPlanes);
    const uint64_t v0 = (block_id() - tiles) / kPlanes * marked;
    if (v0 >= a.vocab) return;
    const uint32_t rows = static_cast<uint32_t>(min(static_cast<uint64_t>(marked), a.vocab - v0));
    const uint32_t all = static_cast<uint32_t>(a.n), part = (all + kPlanes - 1) / kPlanes;
    mark_rows(a, v0, rows, counts, plane * part, min((plane + 1) * part, all));
    for (uint32_t i = threadIdx.x; i < (rows + 31) / 32; i += kSortThreads) marks[plane * z.words + v0 / 32 + i] = counts[i];
    return;
  }
  const uint32_t n = static_cast<uint32_t>(a.n);
  if (threadIdx.x < kBins) counts[threadIdx.x] = 0;
  __syncthreads();
  const uint32_t begin = blockIdx.x * tile, end = min(n - begin, tile) + begin;
  for (uint32_t i = begin + threadIdx.x; i < end; i += kSortThreads) {
    uint32_t k;
    if (keys_in != nullptr) {
      k = keys_in[i];
    } else {
      const uint64_t row = token_row(a.tokens, i, a.first, a.wide);
      k = row < a.vocab ? static_cast<uint32_t>(row) : static_cast<uint32_t>(a.vocab);
    }
    atomicAdd(&counts[(k >> shift) % kBins], 1u);
  }
  __syncthreads();
  if (threadIdx.x < kBins) hist[blockIdx.x * kBins + threadIdx.x] = counts[threadIdx.x];
}

// One pass: every tile's entries to their places.  Each workgroup adds up the
// tiles' counts by itself, so a pass is two launches.
template <class B>
__global__ __launch_bounds__(kSortThreads) void sort_move_kernel(EmbedGradArgs a, const uint32_t* keys_in,
                                                                 const uint32_t* places_in, int shift, uint32_t tile,
                                                                 uint32_t tiles, const uint32_t* hist,
                                                                 uint32_t* keys_out, uint32_t* places_out, ZeroPlan z) {
  __shared__ uint32_t counts[kSortWaves][kBins];
  __shared__ uint32_t base[2][kBins], sums[kBins];
  __shared__ uint32_t totals[kBins / 64];
  if (block_id() >= tiles) return zero_group<B>(a, z, block_id() - tiles, nullptr);
  const uint32_t n = static_cast<uint32_t>(a.n), t = threadIdx.x;
  const uint32_t lane = t % 64, wave = t / 64;
  const uint32_t tile_begin = blockIdx.x * tile, tile_end = min(n - tile_begin, tile) + tile_begin;
  const uint32_t part = tile / kSortWaves;  // a multiple of 64
  const uint32_t begin = min(tile_begin + wave * part, tile_end), end = min(begin + part, tile_end);
  auto key_at = [&](uint32_t i) {
    if (keys_in != nullptr) return keys_in[i];
    const uint64_t row = token_row(a.tokens, i, a.first, a.wide);
    return row < a.vocab ? static_cast<uint32_t>(row) : static_cast<uint32_t>(a.vocab);
  };
  auto place_at = [&](uint32_t i) { return places_in != nullptr ? places_in[i] : i; };
  // The first 64 entries of each wave, all of them up to 65536 tokens, are
  // asked for before anything else.
  const uint32_t first_key = begin + lane < end ? key_at(begin + lane) : 0u;
  const uint32_t first_place = begin + lane < end ? place_at(begin + lane) : 0u;
  for (uint32_t i = t; i < kSortWaves * kBins; i += kSortThreads) (&counts[0][0])[i] = 0;
  // The tiles' counts of a digit, half of them to each half of the workgroup,
  // all on their way at once.
  static_assert(kSortThreads == 2 * kBins && kMaxTiles % 2 == 0, "");
  const uint32_t bin = t % kBins, half = t / kBins;
  uint32_t c[kMaxTiles / 2];
#pragma unroll
  for (uint32_t j = 0; j < kMaxTiles / 2; ++j) {
    const uint32_t b = half * (kMaxTiles / 2) + j;
    c[j] = b < tiles ? hist[b * kBins + bin] : 0u;
  }
  uint32_t before = 0, total = 0;
#pragma unroll
  for (uint32_t j = 0; j < kMaxTiles / 2; ++j) {
    before += half * (kMaxTiles / 2) + j < blockIdx.x ? c[j] : 0u;
    total += c[j];
  }
  base[half][bin] = before;
  if (half != 0) sums[bin] = total;
  __syncthreads();
  if (half == 0) total += sums[bin];
  uint32_t v = total;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_up(v, d);
    if (lane >= static_cast<uint32_t>(d)) v += o;
  }
  if (half == 0 && lane == 63) totals[wave] = v;
  __syncthreads();
  if (half == 0) {
    uint32_t start = v - total + base[0][t] + base[1][t];
    for (uint32_t w = 0; w < wave; ++w) start += totals[w];
    base[0][t] = start;
  }
  for (uint32_t i = begin + lane; i < end; i += 64) {
    const uint32_t k = i < begin + 64 ? first_key : key_at(i);
    atomicAdd(&counts[wave][(k >> shift) % kBins], 1u);
  }
  __syncthreads();
  scan_counts(counts, totals, base[0]);
  for (uint32_t at = begin; at < end; at += 64) {
    const uint32_t i = at + lane;
    const bool there = i < end;
    const uint32_t k = at == begin ? first_key : there ? key_at(i) : 0u;
    const uint32_t p = at == begin ? first_place : there ? place_at(i) : 0u;
    const uint32_t d = (k >> shift) % kBins;
    const uint64_t mates = same_digit(d, __ballot(there));
    const uint32_t rank = lanes_below(mates);
    uint32_t to = 0;
    if (there) to = counts[wave][d] + rank;
    __builtin_amdgcn_wave_barrier();
    if (there && rank == 0) counts[wave][d] += static_cast<uint32_t>(__popcll(mates));
    __builtin_amdgcn_wave_barrier();
    if (there) {
      keys_out[to] = k;
      places_out[to] = p;
    }
  }
}

// ---------------------------------------------------------------- gradient
// The sorted entries are cut into chunks of `chunk`; a wave sums a chunk's
// rows over 64 * E columns in fp32.  A run of equal rows that lies in its
// chunk is stored at once.  The part of a run that came from an earlier chunk
// goes to head[chunk], the first part of one that goes on to tail[chunk];
// join_kernel adds a run's tail and the heads after it, in order.  So a
// frequent token is spread over many waves and the order of its sum is fixed.
constexpr uint32_t kZeroRows = 64;  // most rows of a group that reads its marks off the sorted entries

// LDS that a workgroup of the sums reserves and does not use: four to a CU
// leave the memory's pages in better order than eight.  Gradients of many wide
// rows gain by it, narrow and few rows lose nothing or nearly so (us, with 32 KiB
// and without): 65536 x 4096 bf16 into 131072 rows 318.6 and 321; 8000 x 4096 fp32
// into 30000 126.2 and 128.2; 65536 x 1024 fp32 into 50000 114.5 and 116.1;
// 65536 x 512 bf16 into fp32 66.4 and 65.3; 65536 x 64 to 256 and 700 to 4000
// tokens equal.
constexpr uint32_t kSumReserve = 32768;

// Keys are below 2^32 - 1 (vocab < 2^31), so this equals none of them.
constexpr uint32_t kNoKey = 0xffffffffu;

// First entry in [lo, n) with a key of at least v (n if none), by a 64-way
// search of the whole wave.
__device__ __forceinline__ uint32_t first_at_least(const uint32_t* keys, uint32_t lo, uint32_t n, uint32_t v) {
  const uint32_t lane = threadIdx.x % 64;
  uint32_t hi = n;  // every key before lo is < v, every key from hi on >= v
  while (lo < hi) {
    const uint32_t step = (hi - lo + 63) / 64;
    const uint64_t at = lo + static_cast<uint64_t>(lane) * step;
    const uint64_t under = __ballot(at < hi && keys[at < n ? at : n - 1] < v);
    const uint32_t c = static_cast<uint32_t>(__popcll(under));
    if (c == 0) break;
    hi = static_cast<uint32_t>(min(static_cast<uint64_t>(hi), lo + static_cast<uint64_t>(c) * step));
    lo += (c - 1) * step + 1;
  }
  return lo;
}

// Zeros once the entries are sorted, without marks of the table: which of the
// rows v0 .. v0 + rows are named is read off the entries from the first at or
// past v0, a workgroup's width at a time; where one row fills that width, on
// to the next.
struct SortedZeros {
  uint64_t first, end;  // rows of this launch
  uint32_t rows;        // of a workgroup, at most kZeroRows
};
inline uint64_t zero_blocks(const SortedZeros& z) { return (z.end - z.first + z.rows - 1) / z.rows; }
template <class U>
__device__ void zero_sorted_rows(const EmbedGradArgs& a, const uint32_t* keys, const ZeroPlan& plan, const SortedZeros& z,
                                 uint64_t block) {
  __shared__ uint32_t named[kZeroRows / 32];
  const uint64_t first_row = z.first + block * z.rows;
  if (first_row >= z.end) return;
  const uint32_t rows = static_cast<uint32_t>(min(static_cast<uint64_t>(z.rows), z.end - first_row));
  const uint32_t n = static_cast<uint32_t>(a.n), v0 = static_cast<uint32_t>(first_row);
  uint32_t at = first_at_least(keys, 0, n, v0);
  if (threadIdx.x < kZeroRows / 32) named[threadIdx.x] = 0;
  __syncthreads();
  while (at < n) {  // the same for the whole workgroup
    const uint32_t i = at + threadIdx.x;
    const uint32_t k = i < n ? keys[i] : kNoKey;
    if (k - v0 < rows) atomicOr(&named[(k - v0) / 32], 1u << ((k - v0) % 32));
    const uint32_t last = at + blockDim.x - 1;
    if (last >= n) break;
    const uint32_t kl = keys[last];
    if (kl - v0 >= rows) break;
    at = kl == keys[at] ? first_at_least(keys, last, n, kl + 1) : last + 1;
  }
  __syncthreads();
  if (plan.magic != 0) return zero_run<U>(a, plan, first_row, rows, named);
  zero_rows<U>(a, plan, first_row, rows, named, 1, 0);
}
// The zeros of a launch beside its own work, from marks or without.
template <class U>
__device__ __forceinline__ void zeros_beside(const EmbedGradArgs& a, const uint32_t* keys, const ZeroPlan& z,
                                             const SortedZeros& sorted, uint64_t block) {
  if (z.named != nullptr) return zero_group<U>(a, z, block, nullptr);
  zero_sorted_rows<U>(a, keys, z, sorted, block);
}

template <class U, int E>
__device__ __forceinline__ void put_sum(const EmbedGradArgs& a, uint32_t row, uint32_t e, uint32_t dim,
                                        typename Vec<float, E>::type sum) {
  U* g = static_cast<U*>(a.grad) + row * a.grad_stride;
  sum *= a.scale;
  if (a.accumulate) sum += widen<U, E>(load_row<U, E>(g, e, dim));
  store_row<U, E>(g, e, dim, narrow<U, E>(sum));
}

// A wave's 64 * E columns of a partial row, four floats of each lane at a
// time, so that its accesses are unbroken; pitch is a multiple of 512.
template <int E>
__device__ __forceinline__ void put_part(float* row, uint32_t column, typename Vec<float, E>::type v) {
  float* p = row + column * (64 * E) + threadIdx.x % 64 * 4;
#pragma unroll
  for (int h = 0; h < E / 4; ++h) {
    typename Vec<float, 4>::type q;
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = v[h * 4 + i];
    *reinterpret_cast<typename Vec<float, 4>::type*>(p + h * 256) = q;
  }
}
template <int E>
__device__ __forceinline__ typename Vec<float, E>::type get_part(const float* row, uint32_t column) {
  const float* p = row + column * (64 * E) + threadIdx.x % 64 * 4;
  typename Vec<float, E>::type v;
#pragma unroll
  for (int h = 0; h < E / 4; ++h) {
    const typename Vec<float, 4>::type q = *reinterpret_cast<const typename Vec<float, 4>::type*>(p + h * 256);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[h * 4 + i] = q[i];
  }
  return v;
}

template <class T, class U>
__global__ __launch_bounds__(kThreads) void sum_kernel(EmbedGradArgs a, const uint32_t* keys, const uint32_t* places,
                                                       float* head, float* tail, uint32_t chunk, uint32_t chunks,
                                                       uint32_t columns, uint64_t sum_groups, uint64_t pitch,
                                                       ZeroPlan z, SortedZeros sorted) {
  constexpr int E = kVector<T, U>;
  const uint64_t block = block_id();
  if (block >= sum_groups) return zeros_beside<U>(a, keys, z, sorted, block - sum_groups);
  const uint32_t n = static_cast<uint32_t>(a.n), dim = static_cast<uint32_t>(a.dim);
  const uint32_t lane = threadIdx.x % 64;
  const uint64_t item = uniform64(block * (kThreads / 64) + threadIdx.x / 64);
  const uint32_t c = static_cast<uint32_t>(item / columns);
  const uint32_t column = static_cast<uint32_t>(item - static_cast<uint64_t>(c) * columns);
  const uint32_t e = column * (64 * E) + lane * E;
  if (c >= chunks) return;  // whole waves; no barrier follows
  const uint32_t begin = c * chunk, end = min(n - begin, chunk) + begin;
  const uint32_t vocab = static_cast<uint32_t>(a.vocab);
  const uint32_t key_before = begin != 0 ? keys[begin - 1] : kNoKey;
  const uint32_t key_after = end < n ? keys[end] : kNoKey;
  const T* dout = static_cast<const T*>(a.dout);

  typename Vec<float, E>::type sum = {};
  uint32_t run = keys[begin];
  bool from_before = run == key_before;
  constexpr int kAhead = 8;  // rows in flight
  for (uint32_t at = begin; at < end; at += 64) {
    // Lane i holds entry at + i.
    const uint32_t count = min(end - at, 64u);
    const uint32_t mine = at + min(lane, count - 1);
    const uint32_t k = keys[mine], p = places[mine];
    for (uint32_t i0 = 0; i0 < count; i0 += kAhead) {
      typename Vec<T, E>::type v[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const uint32_t i = min(i0 + j, count - 1);
        const uint64_t place = static_cast<uint32_t>(__builtin_amdgcn_readlane(p, i));
        const T* row = dout + place * a.dout_stride;
        v[j] = dim >= E ? load_in<T, E>(row, e, dim) : load_row<T, E>(row, e, dim);
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (i0 + j >= count) break;
        const uint32_t key = __builtin_amdgcn_readlane(k, i0 + j);
        if (key != run) {
          if (from_before)
            put_part<E>(head + c * pitch, column, sum);
          else
            put_sum<U, E>(a, run, e, dim, sum);
          run = key;
          from_before = false;
          sum = 0.0f;
        }
        if (run == vocab) return;  // tokens outside the table are last: nothing to sum
        sum += widen<T, E>(dim >= E ? in_place<T, E>(v[j], e, dim) : v[j]);
      }
    }
  }
  if (from_before)
    put_part<E>(head + c * pitch, column, sum);
  else if (run == key_after)
    put_part<E>(tail + c * pitch, column, sum);
  else
    put_sum<U, E>(a, run, e, dim, sum);
}

// A run that starts in chunk c and goes on: its tail, then the heads of the
// following chunks while they begin with its row.  The K waves of a workgroup
// take an equal part of the chunks each and are added in order.
template <class U, int E, int K>
__global__ __launch_bounds__(K * 64) void join_kernel(EmbedGradArgs a, const uint32_t* keys, const float* head,
                                                      const float* tail, uint32_t chunk, uint32_t columns,
                                                      uint64_t pitch, uint64_t joins, ZeroPlan z, SortedZeros sorted) {
  __shared__ float part[K][64 * E];
  const uint32_t n = static_cast<uint32_t>(a.n), dim = static_cast<uint32_t>(a.dim);
  const uint32_t lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
  const uint64_t block = block_id();
  if (block >= joins) return zeros_beside<U>(a, keys, z, sorted, block - joins);
  const uint32_t c = static_cast<uint32_t>(block / columns);
  const uint32_t chunks = (n + chunk - 1) / chunk;
  const uint32_t next = (c + 1) * chunk;
  const uint32_t run = keys[next - 1];
  // Not a run that goes on, or not one that starts in this chunk.
  if (run == static_cast<uint32_t>(a.vocab) || keys[next] != run || (c != 0 && keys[c * chunk - 1] == run)) return;
  // Chunks after c that begin with the run's row: from c + 1 on, a 64-way search.
  uint32_t lo = c + 1, hi = chunks;  // chunk lo begins with it, chunk hi (if there) does not
  while (hi - lo > 1) {
    const uint32_t step = (hi - lo + 63) / 64;
    const uint64_t at = lo + static_cast<uint64_t>(lane) * step;
    const uint64_t with = __ballot(at < hi && keys[(at < hi ? at : lo) * chunk] == run);
    const uint32_t k = static_cast<uint32_t>(__popcll(with));  // at least lane 0
    hi = static_cast<uint32_t>(min(static_cast<uint64_t>(hi), lo + static_cast<uint64_t>(k) * step));
    lo += (k - 1) * step;
  }
  const uint32_t heads = lo - c;
  const uint32_t column = static_cast<uint32_t>(block - static_cast<uint64_t>(c) * columns);
  const uint32_t e = column * (64 * E) + lane * E;
  const uint32_t share = (heads + K - 1) / K;
  const uint32_t begin = min(wave * share, heads), end = min(begin + share, heads);
  typename Vec<float, E>::type sum = {};
  if (wave == 0) sum = get_part<E>(tail + c * pitch, column);
  const float* h = head + (static_cast<uint64_t>(c) + 1) * pitch;
  constexpr int kAhead = 8;
  for (uint32_t i0 = begin; i0 < end; i0 += kAhead) {
    typename Vec<float, E>::type v[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) v[j] = get_part<E>(h + min(i0 + j, end - 1) * pitch, column);
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (i0 + j < end) sum += v[j];
  }
#pragma unroll
  for (int i = 0; i < E; ++i) part[wave][lane * E + i] = sum[i];
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int w = 1; w < K; ++w)
#pragma unroll
    for (int i = 0; i < E; ++i) sum[i] += part[w][lane * E + i];
  put_sum<U, E>(a, run, e, dim, sum);
}

// Few tokens need no sort, and one launch does it all: a workgroup takes token
// i and 64 * E columns, and is done if an earlier token names the same row;
// else it sums the rows of i and of the later tokens with that row, in fp32.
// Each wave has 64 of the tokens, and the waves are added in order.  Further
// workgroups zero rows, marked from the same tokens.  Bound by the one launch
// and its waits: a token, its row, the store.  Against the sort, the sums and
// the joins, bf16: 250 tokens of 64 columns 5.5 us, so 16.2; 500 of 512 6.8 and
// 16.5; 500 of 1024 into 32000 rows 16.9 and 23.6; 500 times one token of 1024
// 11.1 and 15.0.  Every workgroup looks at every token, so that many tokens or
// columns are better sorted: 1000 of 1024 took 41.4 and 24.7, 500 of 4096 20.4
// and 18.1 (32000 waves), 500 of 2048 12.7 and 16.7 (16000).
constexpr uint32_t kDirect = 512;
constexpr uint64_t kDirectWaves = 1u << 14;  // most waves
constexpr uint32_t kDirectRows = 2048;  // most rows of a group of zeros
constexpr int kDirectAhead = 16;        // rows in flight

// Adds the rows of the first N tokens in `set`, counted from `base`, and takes
// them out of it.
template <class T, int E, int N>
__device__ __forceinline__ void add_rows(const T* dout, uint64_t stride, uint32_t base, uint64_t* set, uint32_t e,
                                         uint32_t dim, typename Vec<float, E>::type* sum) {
  typename Vec<T, E>::type v[N];
  uint64_t left = *set;
  uint32_t i = 0;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    if (left != 0) i = static_cast<uint32_t>(__builtin_ctzll(left));
    left &= left - 1;  // of 0: 0
    v[j] = load_in<T, E>(dout + (base + i) * stride, e, dim);
  }
  // Each load is issued before the first is waited for: without this the
  // compiler moves one to its use, behind the test, and they wait in turn.
  typedef uint32_t Words __attribute__((ext_vector_type(sizeof(T) * E / 4)));
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = __builtin_bit_cast(typename Vec<T, E>::type, fresh(__builtin_bit_cast(Words, v[j])));
#pragma unroll
  for (int j = 0; j < N; ++j) {
    if (*set == 0) break;
    *set &= *set - 1;
    *sum += widen<T, E>(in_place<T, E>(v[j], e, dim));
  }
}

template <class T, class U>
__global__ __launch_bounds__(kDirect) void direct_kernel(EmbedGradArgs a, uint32_t columns, uint64_t sums, ZeroPlan z) {
  constexpr int E = kVector<T, U>;
  typedef typename Vec<float, E>::type Sum;
  __shared__ uint32_t key[kDirect];
  __shared__ uint32_t named[kDirectRows / 32];
  extern __shared__ __attribute__((aligned(16))) char lds[];  // a sum of each thread
  Sum* part = reinterpret_cast<Sum*>(lds);
  const uint32_t n = static_cast<uint32_t>(a.n), dim = static_cast<uint32_t>(a.dim);
  const uint32_t vocab = static_cast<uint32_t>(a.vocab);
  const uint64_t block = block_id();
  for (uint32_t i = threadIdx.x; i < n; i += blockDim.x) {
    const uint64_t row = token_row(a.tokens, i, a.first, a.wide);
    key[i] = row < vocab ? static_cast<uint32_t>(row) : vocab;
  }
  if (block >= sums) {
    const uint64_t first_row = (block - sums) * z.rows;
    const uint32_t rows = first_row < vocab ? static_cast<uint32_t>(min(static_cast<uint64_t>(z.rows), vocab - first_row)) : 0u;
    const uint32_t v0 = static_cast<uint32_t>(first_row);
    for (uint32_t i = threadIdx.x; i < kDirectRows / 32; i += blockDim.x) named[i] = 0;
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < n; i += blockDim.x)
      if (key[i] - v0 < rows) atomicOr(&named[(key[i] - v0) / 32], 1u << ((key[i] - v0) % 32));
    __syncthreads();
    if (rows == 0) return;
    if (z.magic != 0) return zero_run<U>(a, z, first_row, rows, named);
    return zero_rows<U>(a, z, first_row, rows, named, 1, 0);
  }
  __syncthreads();
  const uint32_t lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
  const uint32_t mine = static_cast<uint32_t>(block / columns);
  const uint32_t e = static_cast<uint32_t>(block - static_cast<uint64_t>(mine) * columns) * (64 * E) + lane * E;
  const uint32_t run = uniform(key[mine]);
  if (run == vocab) return;
  auto same = [&](uint32_t base) { return __ballot(base + lane < n && key[min(base + lane, n - 1)] == run); };
  uint32_t waves = 0;  // that have such tokens
  for (uint32_t base = 0; base < n; base += 64) {
    const uint64_t set = same(base);
    if (set == 0) continue;
    // The first of them all: the same test in every wave.
    if (waves == 0 && base + static_cast<uint32_t>(__builtin_ctzll(set)) < mine) return;
    waves |= 1u << (base / 64);
  }
  Sum sum = {};
  const T* dout = static_cast<const T*>(a.dout);
  const uint32_t base = wave * 64;
  uint64_t set = same(base);
  if (dim < E) {
    for (; set != 0; set &= set - 1)
      sum += widen<T, E>(load_row<T, E>(dout + (base + static_cast<uint32_t>(__builtin_ctzll(set))) * a.dout_stride, e, dim));
  }
  while (set != 0) {
    if ((set & (set - 1)) == 0) {
      add_rows<T, E, 1>(dout, a.dout_stride, base, &set, e, dim, &sum);
    } else {
      add_rows<T, E, kDirectAhead>(dout, a.dout_stride, base, &set, e, dim, &sum);
    }
  }
  if ((waves & (waves - 1)) != 0) {
    part[threadIdx.x] = sum;
    __syncthreads();
    if (wave != 0) return;
    for (uint32_t w = 1; w < blockDim.x / 64; ++w) sum += part[w * 64 + lane];  // zeros where it has none
  } else if ((waves >> wave) != 1) {
    return;
  }
  put_sum<U, E>(a, run, e, dim, sum);
}

// Sizes of the sort and of the sums, the same for the workspace and the launch.
struct GradPlan {
  uint32_t tile, tiles;    // sort
  uint32_t chunk, chunks;  // sums
  uint64_t pitch;          // floats between partial rows
  uint64_t keys, places, keys2, places2, hist, marks, head, tail, total;  // byte offsets
};
// Tokens up to which a scan marks the named rows.
constexpr uint64_t kScanTokens = 1u << 17;

GradPlan grad_plan(uint64_t vocab, uint64_t dim, uint64_t n) {
  GradPlan p;
  // Tiles of whole 64-entry steps for each of the 16 waves.
  const uint64_t unit = kSortThreads;
  p.tile = static_cast<uint32_t>(((n + kMaxTiles - 1) / kMaxTiles + unit - 1) / unit * unit);
  if (p.tile == 0) p.tile = unit;
  p.tiles = static_cast<uint32_t>((n + p.tile - 1) / p.tile);
  // Long chunks have few partial rows, short ones fill the chip: about 4096
  // waves of 512 columns.
  const uint64_t columns = (dim + 511) / 512;
  p.chunk = 8;
  while (p.chunk < 128 && n * columns > static_cast<uint64_t>(p.chunk) * 4096) p.chunk *= 2;
  p.chunks = static_cast<uint32_t>((n + p.chunk - 1) / p.chunk);
  p.pitch = columns * 512;
  uint64_t at = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  p.keys = take(n * 4);
  p.places = take(n * 4);
  p.keys2 = take(n * 4);
  p.places2 = take(n * 4);
  p.hist = take(static_cast<uint64_t>(p.tiles) * kBins * 4);
  p.marks = take(n > kSmallSort && n <= kScanTokens ? (vocab + 31) / 32 * kPlanes * 4 : 0);
  p.head = take(p.chunks * p.pitch * 4);
  p.tail = take(p.chunks * p.pitch * 4);
  p.total = at;
  return p;
}

// The sort, with zeros of the unnamed rows beside it where z->rows is not 0;
// z->end is where the sums' launch goes on.
template <class B>
hipError_t sort(const EmbedGradArgs& a, const GradPlan& p, ZeroPlan* z, hipStream_t s) {
  char* ws = static_cast<char*>(a.ws);
  uint32_t* keys = reinterpret_cast<uint32_t*>(ws + p.keys);
  uint32_t* places = reinterpret_cast<uint32_t*>(ws + p.places);
  uint32_t* keys2 = reinterpret_cast<uint32_t*>(ws + p.keys2);
  uint32_t* places2 = reinterpret_cast<uint32_t*>(ws + p.places2);
  uint32_t* hist = reinterpret_cast<uint32_t*>(ws + p.hist);
  uint32_t* marks = reinterpret_cast<uint32_t*>(ws + p.marks);
  int bits = 1;
  while (bits < 32 && (a.vocab >> bits) != 0) ++bits;  // rows run up to `vocab` itself
  const uint64_t groups = z->rows != 0 ? (a.vocab + z->rows - 1) / z->rows : 0;
  if (a.n <= kSmallSort) {
    // as many as are done with the sort; the rest beside the sums and the joins
    z->end = std::min(groups, (kSortZeros + a.dim * sizeof(B) * z->rows) / (a.dim * sizeof(B) * std::max(z->rows, 1u)));
    return launch(sort_small_kernel<B>, grid_of(1 + groups), kSortThreads, 0, s, a, bits, keys, places, *z);
  }
  // Marks by one workgroup on each of the CUs that the sort leaves, and 256 KiB
  // of zeros for each, which are about done with the sort's step.
  constexpr uint64_t kBeside = 192;
  uint64_t marked = ((a.vocab * kPlanes + kBeside - 1) / kBeside + 31) / 32 * 32;
  marked = std::min<uint64_t>(marked, kNamedWords * 32);
  const uint64_t marking = groups != 0 ? (a.vocab + marked - 1) / marked * kPlanes : 0;
  const uint64_t beside_groups = kBeside * 8;
  const int passes = (bits + kDigit - 1) / kDigit;
  const uint32_t *kin = nullptr, *pin = nullptr;
  uint32_t *kout = passes % 2 ? keys : keys2, *pout = passes % 2 ? places : places2;
  for (int pass = 0; pass < passes; ++pass) {
    const int shift = pass * kDigit;
    if (pass != 0) z->end = std::min(groups, z->first + beside_groups);
    const uint64_t beside = pass == 0 ? marking : z->end - z->first;
    hipError_t e = launch(sort_count_kernel<B>, grid_of(p.tiles + beside), kSortThreads, 0, s, a, kin, shift, p.tile,
                          p.tiles, hist, pass == 0 && groups != 0 ? marks : nullptr, static_cast<uint32_t>(marked), *z);
    if (e != hipSuccess) return e;
    if (groups != 0) z->named = marks;
    z->first = z->end;
    z->end = std::min(groups, z->first + beside_groups);
    e = launch(sort_move_kernel<B>, grid_of(p.tiles + z->end - z->first), kSortThreads, 0, s, a, kin, pin, shift, p.tile,
               p.tiles, hist, kout, pout, *z);
    if (e != hipSuccess) return e;
    z->first = z->end;
    kin = kout;
    pin = pout;
    kout = kout == keys ? keys2 : keys;
    pout = pout == places ? places2 : places;
  }
  return hipSuccess;
}

template <class T, class U>
hipError_t grad(const EmbedGradArgs& a, hipStream_t s) {
  constexpr int E = kVector<T, U>;
  const uint32_t columns = static_cast<uint32_t>((a.dim + 64 * E - 1) / (64 * E));
  const uint64_t row_bytes = a.dim * sizeof(U);
  const bool small = a.n <= kSmallSort;
  // The direct sums' waves: one to 64 tokens, at least four.
  const uint64_t waves = std::max<uint64_t>(4, (a.n + 63) / 64);
  const bool direct = a.n <= kDirect && a.n * columns * waves <= kDirectWaves;
  ZeroPlan z = {nullptr, (a.vocab + 31) / 32, 0, lanes_of(a.dim, 16 / sizeof(U)), 0, 0, 0};
  // Runs of less than 2^31 elements, with few named rows in between; rows of
  // many lanes are as good by row, unless a group has few of them or they share
  // lines (4000 rows of 3353 into 42879 fp32 rows: 133 us, by row 154).
  if (small && a.grad_stride == a.dim && a.dim != 1 && (row_bytes < 4096 || direct || row_bytes % 128 != 0))
    z.magic = static_cast<uint32_t>((1ull << 32) / a.dim + 1);
  if (direct) {
    // Groups of zeros of up to 32 KiB, of small tables less.
    const uint64_t bytes = std::min<uint64_t>(kZeroGroup, std::max<uint64_t>(4096, a.vocab * row_bytes / 2048));
    z.rows = static_cast<uint32_t>(std::max<uint64_t>(1, std::min<uint64_t>(bytes / row_bytes, kDirectRows)));
    const uint64_t sums = a.n * columns, groups = a.accumulate ? 0 : (a.vocab + z.rows - 1) / z.rows;
    if (sums + groups == 0) return hipSuccess;
    const uint32_t threads = static_cast<uint32_t>(waves) * 64;
    return launch(direct_kernel<T, U>, grid_of(sums + groups), threads, threads * E * 4, s, a, columns, sums, z);
  }
  const GradPlan p = grad_plan(a.vocab, a.dim, a.n);
  char* ws = static_cast<char*>(a.ws);
  const uint32_t* keys = reinterpret_cast<const uint32_t*>(ws + p.keys);
  const uint32_t* places = reinterpret_cast<const uint32_t*>(ws + p.places);
  float* head = reinterpret_cast<float*>(ws + p.head);
  float* tail = reinterpret_cast<float*>(ws + p.tail);
  if (!a.accumulate && a.n <= kScanTokens) {
    // Where a group scans the tokens by itself, rounds of a workgroup to each CU
    // but the sort's own, all of one size, of about kScanGroup.  Else short:
    // groups of 32 KiB sweep the table in order, groups of 256 KiB are 2048
    // places that are written at once (336 and 353 us for the gradient of 65536
    // rows of 4096 bf16 in a table of 131072).
    uint64_t rows = kZeroGroup / row_bytes;
    if (small) {
      const uint64_t slots = kCus - 1;
      const uint64_t bytes = std::min<uint64_t>(a.vocab * row_bytes, kSortZeros);
      const uint64_t rounds = (bytes + slots * kScanGroup - 1) / (slots * kScanGroup);
      rows = (bytes / row_bytes + slots * rounds - 1) / (slots * rounds);
    }
    z.rows = static_cast<uint32_t>(std::max<uint64_t>(1, std::min<uint64_t>(rows, kNamedWords * 32)));
  }
  const hipError_t sorting = sizeof(U) == 4 ? sort<uint32_t>(a, p, &z, s) : sort<uint16_t>(a, p, &z, s);
  if (sorting != hipSuccess) return sorting;
  const uint64_t sums = (static_cast<uint64_t>(p.chunks) * columns + kThreads / 64 - 1) / (kThreads / 64);
  const uint64_t joins = p.chunks < 2 ? 0 : static_cast<uint64_t>(p.chunks - 1) * columns;
  // What the sort has left of the zeros: beside the joins what is done with
  // them, the other beside the sums.
  uint64_t zeros = 0, last_zeros = 0;  // workgroups
  ZeroPlan last_z = z;
  SortedZeros sorted = {0, 0, static_cast<uint32_t>(std::max<uint64_t>(1, std::min<uint64_t>(kZeroRows, 2 * kZeroGroup / row_bytes)))};
  SortedZeros last_sorted = sorted;
  if (z.named != nullptr) {
    const uint64_t groups = (a.vocab + z.rows - 1) / z.rows;
    z.first = z.end;
    z.end = groups - (joins != 0 ? std::min<uint64_t>(groups - z.first, kJoinZeros / kZeroGroup) : 0);
    last_z.first = z.end;
    last_z.end = groups;
    zeros = z.end - z.first;
    last_zeros = last_z.end - last_z.first;
  } else if (!a.accumulate) {
    sorted.first = std::min<uint64_t>(a.vocab, z.end * z.rows);
    sorted.end = a.vocab - (joins != 0 ? std::min<uint64_t>(a.vocab - sorted.first, kJoinZeros / row_bytes) : 0);
    last_sorted.first = sorted.end;
    last_sorted.end = a.vocab;
    zeros = zero_blocks(sorted);
    last_zeros = zero_blocks(last_sorted);
  }
  const hipError_t e = launch(sum_kernel<T, U>, grid_of(sums + zeros), kThreads, kSumReserve, s, a, keys, places, head, tail, p.chunk,
                              p.chunks, columns, sums, p.pitch, z, sorted);
  if (e != hipSuccess || joins == 0) return e;
  // Most workgroups find no run to join: few waves each where they are many.
  const auto join = joins > 4000 ? join_kernel<U, E, 4> : join_kernel<U, E, 8>;
  return launch(join, grid_of(joins + last_zeros), joins > 4000 ? 256u : 512u, 0, s, a, keys, head, tail, p.chunk, columns,
                p.pitch, joins, last_z, last_sorted);
}

}  // namespace

hipError_t launch_embedding(const EmbedArgs& a, hipStream_t s) {
  switch (a.table_type * 16 + a.out_type) {
    case RSX_FLOAT32 * 16 + RSX_FLOAT32:
      return lookup<float, float>(a, s);
    case RSX_FLOAT32 * 16 + RSX_BFLOAT16:
      return lookup<float, bf16_t>(a, s);
    case RSX_FLOAT32 * 16 + RSX_FLOAT16:
      return lookup<float, f16_t>(a, s);
    case RSX_BFLOAT16 * 16 + RSX_FLOAT32:
      return lookup<bf16_t, float>(a, s);
    case RSX_BFLOAT16 * 16 + RSX_BFLOAT16:
      return lookup<bf16_t, bf16_t>(a, s);
    case RSX_BFLOAT16 * 16 + RSX_FLOAT16:
      return lookup<bf16_t, f16_t>(a, s);
    case RSX_FLOAT16 * 16 + RSX_FLOAT32:
      return lookup<f16_t, float>(a, s);
    case RSX_FLOAT16 * 16 + RSX_BFLOAT16:
      return lookup<f16_t, bf16_t>(a, s);
    default:
      return lookup<f16_t, f16_t>(a, s);
  }
}

// Of few tokens too, which use none: the rule that callers see has no step in it.
uint64_t embedding_grad_ws(uint64_t vocab, uint64_t dim, uint64_t n) { return grad_plan(vocab, dim, n).total; }

hipError_t launch_embedding_grad(const EmbedGradArgs& a, hipStream_t s) {
  switch (a.dout_type * 16 + a.grad_type) {
    case RSX_FLOAT32 * 16 + RSX_FLOAT32:
      return grad<float, float>(a, s);
    case RSX_FLOAT32 * 16 + RSX_BFLOAT16:
      return grad<float, bf16_t>(a, s);
    case RSX_FLOAT32 * 16 + RSX_FLOAT16:
      return grad<float, f16_t>(a, s);
    case RSX_BFLOAT16 * 16 + RSX_FLOAT32:
      return grad<bf16_t, float>(a, s);
    case RSX_BFLOAT16 * 16 + RSX_BFLOAT16:
      return grad<bf16_t, bf16_t>(a, s);
    case RSX_BFLOAT16 * 16 + RSX_FLOAT16:
      return grad<bf16_t, f16_t>(a, s);
    case RSX_FLOAT16 * 16 + RSX_FLOAT32:
      return grad<f16_t, float>(a, s);
    case RSX_FLOAT16 * 16 + RSX_BFLOAT16:
      return grad<f16_t, bf16_t>(a, s);
    default:
      return grad<f16_t, f16_t>(a, s);
  }
}

}  // namespace rsx
