// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   out[i, :]  = scale * table[t_i, :]          t_i = tokens[i] - first
//   grad[v, :] = (grad[v, :] +) scale * sum of dout[i, :] over the i with t_i = v
//
// A token outside [0, vocab) gives a row of zeros and no gradient.
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

__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<int>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<int>(v >> 32));
  return (static_cast<uint64_t>(hi) << 32) | lo;
}

// ---------------------------------------------------------------- lookup
// A wave copies V vectors per lane of one row: 64 * V * E elements.
template <class T, class U, int V>
__global__ __launch_bounds__(kThreads) void lookup_kernel(EmbedArgs a, uint32_t chunks) {
  constexpr int E = sizeof(T) == 4 && sizeof(U) == 4 ? 4 : 8;
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
    for (int j = 0; j < V; ++j) v[j] = load_row<T, E, false>(src, base + j * 64 * E, dim);
#pragma unroll
    for (int j = 0; j < V; ++j)
      store_row<U, E>(out, base + j * 64 * E, dim, narrow<U, E>(widen<T, E>(v[j]) * a.scale));
  } else {
    const typename Vec<U, E>::type zero = {};
#pragma unroll
    for (int j = 0; j < V; ++j) store_row<U, E>(out, base + j * 64 * E, dim, zero);
  }
}

template <class T, class U, int V>
hipError_t lookup_go(const EmbedArgs& a, hipStream_t s) {
  constexpr int E = sizeof(T) == 4 && sizeof(U) == 4 ? 4 : 8;
  const uint64_t chunks = (a.dim + 64 * V * E - 1) / (64 * V * E);
  const uint64_t grid = (a.n * chunks + kThreads / 64 - 1) / (kThreads / 64);
  return launch(lookup_kernel<T, U, V>, grid_of(grid), kThreads, 0, s, a, static_cast<uint32_t>(chunks));
}

template <class T, class U>
hipError_t lookup(const EmbedArgs& a, hipStream_t s) {
  return a.n * a.dim < (1u << 22) ? lookup_go<T, U, 1>(a, s) : lookup_go<T, U, 4>(a, s);
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
// number of earlier lanes with that digit, found by one ballot per bit.
constexpr int kDigit = 9;
constexpr int kBins = 1 << kDigit;
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr uint32_t kSmallSort = 8192;  // tokens that one workgroup sorts in its LDS

// Lanes of the wave whose digit equals this lane's, among `valid`.
__device__ __forceinline__ uint64_t same_digit(uint32_t d, uint64_t valid) {
  uint64_t m = valid;
#pragma unroll
  for (int b = 0; b < kDigit; ++b) {
    const uint64_t set = __ballot((d >> b) & 1u);
    m &= ((d >> b) & 1u) ? set : ~set;
  }
  return m;
}
__device__ __forceinline__ uint32_t lanes_below(uint64_t m) {
  return __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(m >> 32), __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(m), 0));
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

// The whole sort of at most kSmallSort tokens in one workgroup.
__global__ __launch_bounds__(kSortThreads) void sort_small_kernel(EmbedGradArgs a, int bits, uint32_t* keys,
                                                                  uint32_t* places) {
  __shared__ uint32_t key[2][kSmallSort];
  __shared__ uint16_t place[2][kSmallSort];
  __shared__ uint32_t counts[kSortWaves][kBins];
  __shared__ uint32_t totals[kBins / 64];
  const uint32_t n = static_cast<uint32_t>(a.n);
  const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const uint32_t part = ((n + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;  // entries of a wave
  const uint32_t begin = min(wave * part, n), end = min(begin + part, n);
  for (uint32_t i = threadIdx.x; i < n; i += kSortThreads) {
    const uint64_t row = token_row(a.tokens, i, a.first, a.wide);
    key[0][i] = row < a.vocab ? static_cast<uint32_t>(row) : static_cast<uint32_t>(a.vocab);
    place[0][i] = static_cast<uint16_t>(i);
  }
  int from = 0;
  for (int shift = 0; shift < bits; shift += kDigit, from ^= 1) {
    for (uint32_t i = threadIdx.x; i < kSortWaves * kBins; i += kSortThreads) (&counts[0][0])[i] = 0;
    __syncthreads();
    for (uint32_t i = begin + lane; i < end; i += 64) atomicAdd(&counts[wave][(key[from][i] >> shift) % kBins], 1u);
    __syncthreads();
    scan_counts(counts, totals, nullptr);
    const bool last = shift + kDigit >= bits;
    for (uint32_t at = begin; at < end; at += 64) {
      const uint32_t i = at + lane;
      const bool there = i < end;
      const uint32_t k = there ? key[from][i] : 0u;
      const uint32_t p = there ? place[from][i] : 0u;
      const uint32_t d = (k >> shift) % kBins;
      const uint64_t mates = same_digit(d, __ballot(there));
      const uint32_t rank = lanes_below(mates);
      uint32_t to = 0;
      if (there) to = counts[wave][d] + rank;
      __builtin_amdgcn_wave_barrier();
      if (there && rank == 0) counts[wave][d] += static_cast<uint32_t>(__popcll(mates));
      __builtin_amdgcn_wave_barrier();
      if (there) {
        if (last) {
          keys[to] = k;
          places[to] = p;
        } else {
          key[from ^ 1][to] = k;
          place[from ^ 1][to] = static_cast<uint16_t>(p);
        }
      }
    }
    __syncthreads();
  }
}

// Digit counts of each tile: hist[tile][digit].
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(EmbedGradArgs a, const uint32_t* keys_in, int shift,
                                                                  uint32_t tile, uint32_t* hist) {
  __shared__ uint32_t counts[kBins];
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
__global__ __launch_bounds__(kSortThreads) void sort_move_kernel(EmbedGradArgs a, const uint32_t* keys_in,
                                                                 const uint32_t* places_in, int shift, uint32_t tile,
                                                                 const uint32_t* hist, uint32_t* keys_out,
                                                                 uint32_t* places_out) {
  __shared__ uint32_t counts[kSortWaves][kBins];
  __shared__ uint32_t base[kBins];
  __shared__ uint32_t totals[kBins / 64];
  const uint32_t n = static_cast<uint32_t>(a.n), t = threadIdx.x;
  const uint32_t lane = t % 64, wave = t / 64;
  for (uint32_t i = t; i < kSortWaves * kBins; i += kSortThreads) (&counts[0][0])[i] = 0;
  uint32_t before = 0, total = 0;
  if (t < kBins) {
#pragma unroll 8
    for (uint32_t b = 0; b < gridDim.x; ++b) {
      const uint32_t c = hist[b * kBins + t];
      before += b < blockIdx.x ? c : 0u;
      total += c;
    }
  }
  uint32_t v = total;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_up(v, d);
    if (lane >= static_cast<uint32_t>(d)) v += o;
  }
  if (t < kBins && lane == 63) totals[wave] = v;
  __syncthreads();
  if (t < kBins) {
    uint32_t start = v - total + before;
    for (uint32_t w = 0; w < wave; ++w) start += totals[w];
    base[t] = start;
  }
  const uint32_t tile_begin = blockIdx.x * tile, tile_end = min(n - tile_begin, tile) + tile_begin;
  const uint32_t part = tile / kSortWaves;  // a multiple of 64
  const uint32_t begin = min(tile_begin + wave * part, tile_end), end = min(begin + part, tile_end);
  auto key_at = [&](uint32_t i) {
    if (keys_in != nullptr) return keys_in[i];
    const uint64_t row = token_row(a.tokens, i, a.first, a.wide);
    return row < a.vocab ? static_cast<uint32_t>(row) : static_cast<uint32_t>(a.vocab);
  };
  for (uint32_t i = begin + lane; i < end; i += 64) atomicAdd(&counts[wave][(key_at(i) >> shift) % kBins], 1u);
  __syncthreads();
  scan_counts(counts, totals, base);
  for (uint32_t at = begin; at < end; at += 64) {
    const uint32_t i = at + lane;
    const bool there = i < end;
    const uint32_t k = there ? key_at(i) : 0u;
    const uint32_t p = !there ? 0u : places_in != nullptr ? places_in[i] : i;
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
// Rows that no token names are zeroed by the workgroups after those
// (kZeroRows rows each), unless the gradient accumulates.
constexpr uint32_t kZeroRows = 64;

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

template <class U, int E>
__device__ __forceinline__ void put_sum(const EmbedGradArgs& a, uint32_t row, uint32_t e, uint32_t dim,
                                        typename Vec<U, E>::wide sum) {
  U* g = static_cast<U*>(a.grad) + row * a.grad_stride;
  sum *= a.scale;
  if (a.accumulate) sum += widen<U, E>(load_row<U, E>(g, e, dim));
  store_row<U, E>(g, e, dim, narrow<U, E>(sum));
}

template <class T, class U, int E>
__global__ __launch_bounds__(kThreads) void sum_kernel(EmbedGradArgs a, const uint32_t* keys, const uint32_t* places,
                                                       float* head, float* tail, uint32_t chunk, uint32_t chunks,
                                                       uint32_t columns, uint64_t sum_groups, uint64_t pitch) {
  __shared__ uint32_t named[kZeroRows];
  const uint32_t n = static_cast<uint32_t>(a.n), dim = static_cast<uint32_t>(a.dim);
  const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  typedef typename Vec<T, E>::wide Wide;
  const uint64_t block = block_id();
  if (block >= sum_groups) {
    // Which of the rows v0 .. v0 + 63 are named: the entries from the first
    // at or past v0, a workgroup's width at a time; where one row fills that
    // width, on to the next row.
    const uint64_t first_row = (block - sum_groups) * kZeroRows;
    if (first_row >= a.vocab) return;
    const uint32_t v0 = static_cast<uint32_t>(first_row);
    uint32_t at = first_at_least(keys, 0, n, v0);
    if (threadIdx.x < kZeroRows) named[threadIdx.x] = 0;
    __syncthreads();
    while (at < n) {  // the same for the whole workgroup
      const uint32_t i = at + threadIdx.x;
      const uint32_t k = i < n ? keys[i] : kNoKey;
      if (k - v0 < kZeroRows) named[k - v0] = 1;
      const uint32_t last = at + kThreads - 1;
      if (last >= n) break;
      const uint32_t kl = keys[last];
      if (kl - v0 >= kZeroRows) break;
      at = kl == keys[at] ? first_at_least(keys, last, n, kl + 1) : last + 1;
    }
    __syncthreads();
    const typename Vec<U, E>::type zero = {};
    for (uint32_t r = wave; r < kZeroRows && v0 + r < a.vocab; r += kThreads / 64) {
      if (named[r]) continue;
      U* g = static_cast<U*>(a.grad) + (v0 + r) * a.grad_stride;
      for (uint32_t e = lane * E; e < dim; e += 64 * E) store_row<U, E>(g, e, dim, zero);
    }
    return;
  }

  const uint64_t item = uniform64(block * (kThreads / 64) + wave);
  const uint32_t c = static_cast<uint32_t>(item / columns);
  const uint32_t e = static_cast<uint32_t>(item - static_cast<uint64_t>(c) * columns) * (64 * E) + lane * E;
  if (c >= chunks) return;  // whole waves; no barrier follows
  const uint32_t begin = c * chunk;
  const uint32_t count = min(n - begin, chunk);
  const uint32_t vocab = static_cast<uint32_t>(a.vocab);
  // Lane i holds entry begin + i, lane 63 the entry before the chunk, lane
  // `count` the one after it (chunk <= 32).
  uint32_t k = kNoKey, p = 0;
  if (lane <= count && begin + lane < n) {
    k = keys[begin + lane];
    p = places[begin + lane];
  }
  if (lane == 63 && begin != 0) k = keys[begin - 1];
  const uint32_t key_before = __builtin_amdgcn_readlane(k, 63);
  const uint32_t key_after = __builtin_amdgcn_readlane(k, count);
  const T* dout = static_cast<const T*>(a.dout);

  Wide sum = 0.0f;
  uint32_t run = __builtin_amdgcn_readlane(k, 0);
  bool from_before = run == key_before;
  constexpr int kAhead = 8;
  for (uint32_t i0 = 0; i0 < count; i0 += kAhead) {
    typename Vec<T, E>::type v[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const uint32_t i = min(i0 + j, count - 1);
      const uint64_t place = static_cast<uint32_t>(__builtin_amdgcn_readlane(p, i));
      v[j] = load_row<T, E>(dout + place * a.dout_stride, e, dim);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i0 + j >= count) break;
      const uint32_t key = __builtin_amdgcn_readlane(k, i0 + j);
      if (key != run) {
        if (from_before)
          store_row<float, E>(head + c * pitch, e, dim, sum);
        else
          put_sum<U, E>(a, run, e, dim, sum);
        run = key;
        from_before = false;
        sum = 0.0f;
      }
      if (run == vocab) return;  // tokens outside the table are last: nothing to sum
      sum += widen<T, E>(v[j]);
    }
  }
  if (from_before)
    store_row<float, E>(head + c * pitch, e, dim, sum);
  else if (run == key_after)
    store_row<float, E>(tail + c * pitch, e, dim, sum);
  else
    put_sum<U, E>(a, run, e, dim, sum);
}

// A run that starts in chunk c and goes on: its tail, then the heads of the
// following chunks while they begin with its row.  The four waves of a
// workgroup take a quarter of the chunks each and are added in order.
template <class U, int E>
__global__ __launch_bounds__(kThreads) void join_kernel(EmbedGradArgs a, const uint32_t* keys, const float* head,
                                                        const float* tail, uint32_t chunk, uint32_t columns,
                                                        uint64_t pitch) {
  __shared__ float part[kThreads / 64][64 * E];
  const uint32_t n = static_cast<uint32_t>(a.n), dim = static_cast<uint32_t>(a.dim);
  const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const uint64_t block = block_id();
  const uint32_t c = static_cast<uint32_t>(block / columns);
  const uint32_t chunks = (n + chunk - 1) / chunk;
  if (block / columns >= chunks - 1) return;  // the last chunk starts no run that goes on
  const uint32_t next = (c + 1) * chunk;
  const uint32_t run = keys[next - 1];
  // Not a run that goes on, or not one that starts in this chunk.
  if (run == static_cast<uint32_t>(a.vocab) || keys[next] != run || (c != 0 && keys[c * chunk - 1] == run)) return;
  uint32_t heads = 0;  // chunks after c that begin with the run's row
  for (;;) {
    const uint64_t at = static_cast<uint64_t>(c) + 1 + heads + lane;
    const uint64_t m = __ballot(at < chunks && keys[at < chunks ? at * chunk : 0] == run);
    const uint32_t more = m == ~0ull ? 64u : static_cast<uint32_t>(__builtin_ctzll(~m));
    heads += more;
    if (more < 64) break;
  }
  const uint32_t e = static_cast<uint32_t>(block - static_cast<uint64_t>(c) * columns) * (64 * E) + lane * E;
  const uint32_t quarter = (heads + 3) / 4;
  const uint32_t begin = min(wave * quarter, heads), end = min(begin + quarter, heads);
  typename Vec<float, E>::type sum = {};
  if (wave == 0) sum = load_row<float, E>(tail + c * pitch, e, dim);
  const float* h = head + (c + 1) * pitch;
#pragma unroll 8
  for (uint32_t i = begin; i < end; ++i) sum += load_row<float, E>(h + i * pitch, e, dim);
#pragma unroll
  for (int i = 0; i < E; ++i) part[wave][lane * E + i] = sum[i];
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w)
#pragma unroll
    for (int i = 0; i < E; ++i) sum[i] += part[w][lane * E + i];
  put_sum<U, E>(a, run, e, dim, sum);
}

// Sizes of the sort and of the sums, the same for the workspace and the launch.
struct GradPlan {
  uint32_t tile, tiles;    // sort
  uint32_t chunk, chunks;  // sums
  uint64_t pitch;          // floats between partial rows
  uint64_t keys, places, keys2, places2, hist, head, tail, total;  // byte offsets
};
GradPlan grad_plan(uint64_t dim, uint64_t n) {
  GradPlan p;
  // About 64 tiles, of whole 64-entry steps for each of the 16 waves.
  const uint64_t unit = kSortThreads;
  p.tile = static_cast<uint32_t>(((n + 63) / 64 + unit - 1) / unit * unit);
  if (p.tile == 0) p.tile = unit;
  p.tiles = static_cast<uint32_t>((n + p.tile - 1) / p.tile);
  // Chunks short enough that a small batch still fills the chip.
  p.chunk = n >= 32768 ? 32u : n >= 8192 ? 16u : 8u;
  p.chunks = static_cast<uint32_t>((n + p.chunk - 1) / p.chunk);
  p.pitch = (dim + 15) / 16 * 16;
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
  p.head = take(p.chunks * p.pitch * 4);
  p.tail = take(p.chunks * p.pitch * 4);
  p.total = at;
  return p;
}

template <class T, class U>
hipError_t grad(const EmbedGradArgs& a, hipStream_t s) {
  constexpr int E = sizeof(T) == 4 ? 4 : 8;
  const GradPlan p = grad_plan(a.dim, a.n);
  char* ws = static_cast<char*>(a.ws);
  uint32_t* keys = reinterpret_cast<uint32_t*>(ws + p.keys);
  uint32_t* places = reinterpret_cast<uint32_t*>(ws + p.places);
  uint32_t* keys2 = reinterpret_cast<uint32_t*>(ws + p.keys2);
  uint32_t* places2 = reinterpret_cast<uint32_t*>(ws + p.places2);
  uint32_t* hist = reinterpret_cast<uint32_t*>(ws + p.hist);
  float* head = reinterpret_cast<float*>(ws + p.head);
  float* tail = reinterpret_cast<float*>(ws + p.tail);
  int bits = 1;
  while (bits < 32 && (a.vocab >> bits) != 0) ++bits;  // rows run up to `vocab` itself
  hipError_t e = hipSuccess;
  if (a.n == 0) {
    // nothing to sort or sum
  } else if (a.n <= kSmallSort) {
    e = launch(sort_small_kernel, dim3(1), kSortThreads, 0, s, a, bits, keys, places);
    if (e != hipSuccess) return e;
  } else {
    const uint32_t *kin = nullptr, *pin = nullptr;
    uint32_t *kout = ((bits + kDigit - 1) / kDigit) % 2 ? keys : keys2, *pout = kout == keys ? places : places2;
    for (int shift = 0; shift < bits; shift += kDigit) {
      e = launch(sort_count_kernel, dim3(p.tiles), kSortThreads, 0, s, a, kin, shift, p.tile, hist);
      if (e != hipSuccess) return e;
      e = launch(sort_move_kernel, dim3(p.tiles), kSortThreads, 0, s, a, kin, pin, shift, p.tile, hist, kout, pout);
      if (e != hipSuccess) return e;
      kin = kout;
      pin = pout;
      kout = kout == keys ? keys2 : keys;
      pout = pout == places ? places2 : places;
    }
  }
  const uint32_t columns = static_cast<uint32_t>((a.dim + 64 * E - 1) / (64 * E));
  const uint64_t sums = (static_cast<uint64_t>(p.chunks) * columns + kThreads / 64 - 1) / (kThreads / 64);
  const uint64_t zeros = a.accumulate ? 0 : (a.vocab + kZeroRows - 1) / kZeroRows;
  if (sums + zeros == 0) return hipSuccess;
  e = launch(sum_kernel<T, U, E>, grid_of(sums + zeros), kThreads, 0, s, a, keys, places, head, tail, p.chunk, p.chunks,
             columns, sums, p.pitch);
  if (e != hipSuccess || p.chunks < 2) return e;
  return launch(join_kernel<U, E>, grid_of(static_cast<uint64_t>(p.chunks - 1) * columns), kThreads, 0, s, a, keys, head,
                tail, p.chunk, columns, p.pitch);
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

uint64_t embedding_grad_ws(uint64_t dim, uint64_t n) { return grad_plan(dim, n).total; }

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
