// Log probabilities of given tokens, with the entropy and the most likely
// alternatives, and their gradient.
//
//   lse = log sum exp z,  log p_j = z_j - lse,
//   logprob = log p_token,  entropy H = -sum p_j log p_j,
//   dz_j = g (delta(j, token) - p_j) - h p_j (log p_j + H)
//   for gradients g of the log probability and h of the entropy.
//
// The forward pass reads a row once: each lane keeps a running maximum m, the
// sum s of 2^u and the sum t of 2^u u, u = (z - m) log2 e, all in fp32.  Then
// lse = m + ln s and H = ln s - t ln 2 / s, a sum of two terms that are not
// negative, so nothing cancels.  The instructions bound it nearly as much as
// the reads do, so u is one: z log2 e - r, with r = m log2 e rounded; what the
// rounding took is put back once, at the end.  A masked logit (-inf) adds nothing; a row of
// nothing else has lse = -inf, log probabilities of -inf, entropy 0 and a
// gradient of 0.  lse alone is a rounding of lse's size off (2^-10 at 16384), and
// so is each p that a gradient takes from it; lse_rest keeps what that took.
// A row with a NaN or +inf has NaN for lse, log probabilities,
// entropy and gradient.  A token outside the row has log probability 0 and no
// gradient through it.
#include "step_device.h"

namespace rsx {
namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ uint64_t token_at(const void* tokens, uint64_t i, int wide) {
  return wide ? static_cast<uint64_t>(static_cast<const int64_t*>(tokens)[i])
              : static_cast<uint64_t>(static_cast<int64_t>(static_cast<const int32_t*>(tokens)[i]));
}

// ------------------------------------------------------- softmax statistics
struct Stats {
  float m, s, t;
};
constexpr float kLeast = -1e30f;  // stands in for u = -inf where u is a factor

// The maximum that u is taken against: 0 while there is none.
__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? 0.0f : m; }

// `a` against the larger maximum m.
__device__ __forceinline__ Stats rebase(const Stats& a, float m) {
  const float d = (a.m - reference(m)) * kLog2e;
  const float f = __builtin_amdgcn_exp2f(d);
  const float dd = fmaxf(d, kLeast);
  return {m, a.s * f, (a.t + dd * a.s) * f};
}
__device__ __forceinline__ Stats merge(const Stats& a, const Stats& b) {
  const float m = fmaxf(a.m, b.m);
  const Stats x = rebase(a, m), y = rebase(b, m);
  return {m, x.s + y.s, x.t + y.t};
}
__device__ __forceinline__ Stats wave_merge(Stats a) {
  const float m = wave_max(a.m);
  const Stats x = rebase(a, m);
  return {m, wave_sum(x.s), wave_sum(x.t)};
}

// --------------------------------------------------------- top alternatives
// A candidate as one integer: its value in order (a NaN below every number,
// -0 equal to +0) in the high half, the complement of its index in the low
// half, so that of equal values the lower index is the larger candidate.  0
// is no candidate.
__device__ __forceinline__ uint32_t value_order(float z) {
  const uint32_t b = __builtin_bit_cast(uint32_t, z + 0.0f);
  const uint32_t o = b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
  return z == z ? o : 1u;
}
__device__ __forceinline__ float order_value(uint32_t o) {
  const uint32_t b = o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu);
  return o == 1u ? __builtin_bit_cast(float, 0x7fc00000u) : __builtin_bit_cast(float, b);
}
__device__ __forceinline__ uint64_t candidate(uint32_t order, uint32_t index) {
  return (static_cast<uint64_t>(order) << 32) | (0xffffffffu - index);
}
// A wave's candidates, a list in LDS.  What passes `least`, a bound that the
// top-th largest is known to pass, is put at its end, all lanes' at once; a
// list that is full is cut to its `top` largest, whose last is the new bound.
// (Kept sorted, each candidate is an insertion of its own, and the waves of a CU
// queue for its scalar unit: 2050 rows of 14528 fp16 with 16 alternatives took
// 43 us, this way 29.)
constexpr uint32_t kList = 128;
struct Best {
  uint64_t* list;
  uint64_t least;
  uint32_t n;
};
// Orders the wave's own LDS accesses.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}
// The list's `top` largest, in order; all are different.
__device__ void cut_list(Best& b, uint32_t lane, uint32_t top) {
  wave_fence();
  uint64_t mine[kList / 64];
  uint32_t rank[kList / 64] = {};
#pragma unroll
  for (uint32_t k = 0; k < kList / 64; ++k) mine[k] = k * 64 + lane < b.n ? b.list[k * 64 + lane] : 0ull;
#pragma unroll 8
  for (uint32_t j = 0; j < b.n; ++j) {
    const uint64_t other = b.list[j];
#pragma unroll
    for (uint32_t k = 0; k < kList / 64; ++k) rank[k] += other > mine[k] ? 1u : 0u;
  }
  wave_fence();
#pragma unroll
  for (uint32_t k = 0; k < kList / 64; ++k)
    if (mine[k] != 0 && rank[k] < top) b.list[rank[k]] = mine[k];
  wave_fence();
  if (b.n < top) return;
  b.n = top;
  const uint64_t last = b.list[top - 1];
  const uint64_t bound = uniform64(last);
  b.least = bound > b.least ? bound : b.least;
}
// A lower bound of the top-th largest of the lanes' values, its upper 16 bits
// one at a time (of 16-bit logits the others follow from the sign).
__device__ __forceinline__ uint32_t lanes_nth(uint32_t v, uint32_t top) {
  uint64_t alive = ~0ull;
  uint32_t found = 0, need = top;
#pragma unroll
  for (int bit = 31; bit >= 16; --bit) {
    const uint64_t set = __ballot((v >> bit) & 1u) & alive;
    const uint32_t c = static_cast<uint32_t>(__popcll(set));
    if (c >= need) {
      alive = set;
      found |= 1u << bit;
    } else {
      need -= c;
      alive &= ~set;
    }
  }
  return found;
}

// ---------------------------------------------------------------- forward
constexpr int kUnroll = 4;  // vectors of a step, with as many on their way

struct Partial {
  float m, s, t, pad;
};

// A row (or a slice of one) as single elements up to the first 16-byte
// boundary, whole vectors, and single elements again: accesses that are off a
// boundary cost a quarter of the rate.
template <class T>
struct Cut {
  static constexpr int E = 16 / sizeof(T);
  uint32_t head, vectors, tail;
  const T* middle;
  __device__ __forceinline__ Cut(const T* row, const void* align, uint32_t n) {
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(align) / sizeof(T)) % E;
    head = min((E - off) % E, n);
    vectors = (n - head) / E;
    tail = n - head - vectors * E;
    middle = row + head;
  }
  // Threads 0 .. head - 1 and E .. E + tail - 1 have a single element each;
  // its index, or `n` and more for none.
  __device__ __forceinline__ uint32_t single(uint32_t thread) const {
    if (thread < head) return thread;
    const uint32_t i = thread - E;
    return thread >= E && i < tail ? head + vectors * E + i : 0xffffffffu;
  }
};

__device__ __forceinline__ float logit_at(const LogprobArgs& a, uint64_t at) {
  return a.type == RSX_FLOAT32    ? static_cast<const float*>(a.logits)[at]
         : a.type == RSX_BFLOAT16 ? static_cast<float>(static_cast<const bf16_t*>(a.logits)[at])
                                  : static_cast<float>(static_cast<const f16_t*>(a.logits)[at]);
}

// What a row's results need of its token; asked for before the row is read.
struct Token {
  bool there;
  float z;
};
__device__ __forceinline__ Token row_token(const LogprobArgs& a, uint64_t row) {
  const uint64_t tok = token_at(a.tokens, row, a.wide);
  const bool there = tok < a.vocab;
  return {there, there ? logit_at(a, row * a.stride + tok) : 0.0f};
}
// A row's maximum and the logarithm of its sum: lse in two parts.
struct Level {
  float m, ln_s;
};
__device__ __forceinline__ bool all_masked(const Stats& st) { return st.s == 0.0f && st.m == -INFINITY; }
__device__ __forceinline__ Level level_of(const Stats& st) {
  // The maximum's own term is 1, but for roundings.
  return {st.m, all_masked(st) ? -INFINITY : logf(st.s < 1.0f ? 1.0f : st.s)};
}
// (z - m) - ln s keeps more digits than z - lse where the maximum is large.
__device__ __forceinline__ float log_prob(const Level& l, float z) {
  return l.ln_s == -INFINITY ? -INFINITY : (z - l.m) - l.ln_s;
}
__device__ __forceinline__ void finish_row(const LogprobArgs& a, uint64_t row, const Stats& st, const Token& tok) {
  const bool none = all_masked(st);
  const Level l = level_of(st);
  a.logprob[row] = tok.there ? log_prob(l, tok.z) : 0.0f;
  const float lse = none ? -INFINITY : l.m + l.ln_s;
  a.lse[row] = lse;
  if (a.lse_rest != nullptr) {
    // What the rounding took from the sum of m and ln s, exactly.
    const float ln_s = lse - l.m;
    a.lse_rest[row] = fabsf(lse) < INFINITY ? (l.m - (lse - ln_s)) + (l.ln_s - ln_s) : 0.0f;
  }
  // u is not positive, but for roundings
  const float s = st.s < 1.0f ? 1.0f : st.s, t = st.t > 0.0f ? 0.0f : st.t;
  if (a.entropy != nullptr) a.entropy[row] = none ? 0.0f : l.ln_s - t * kLn2 / s;
}

// A lane's statistics on the way.  `r` stands for m log2 e, for m of at least
// -kFar: what lies further down is taken against -kFar.  The rounding of r goes
// through the exponential, so it has to be small: up to |m| = kFar it is at most
// 1, and it doubles with |m| (439 at 1e10, where 2^off is no fp32 number).  A row
// whose maximum itself is beyond +-kFar (all of it masked by -1e9, for one) is
// summed again, against the maximum.
constexpr float kFar = 0x1p24f;
struct Running {
  float m, r, s, t;
};
__device__ __forceinline__ float scaled(float m) { return fmaxf(m, -kFar) * kLog2e; }
__device__ __forceinline__ void raise(Running& a, float m) {
  // The old r against the new one as it is held, rounded: a contracted product
  // leaves the rounding in the sums so far (up to a factor of 2^(1/4) at m = 2^22).
#pragma clang fp contract(off)
  const float r = scaled(m), d = fmaxf(a.r - r, kLeast), f = __builtin_amdgcn_exp2f(d);
  a.t = fmaf(d, a.s, a.t) * f;
  a.s *= f;
  a.r = r;
  a.m = m;
}
__device__ __forceinline__ void add(Running& a, float z) {
  const float u = fmaf(z, kLog2e, -a.r);
  const float p = __builtin_amdgcn_exp2f(u);
  a.s += p;
  a.t = fmaf(p, fmaxf(u, kLeast), a.t);
}
// The same sums against m itself, or against -kFar for an m below.
__device__ __forceinline__ Stats settled(const Running& a) {
  if (a.m < -kFar) return {a.m == -INFINITY ? a.m : -kFar, a.s, a.t};  // r is exact there
  const float off = fmaf(a.m, kLog2e, -a.r), f = __builtin_amdgcn_exp2f(-off);
  return {a.m, a.s * f, fmaf(-off, a.s, a.t) * f};
}
__device__ __forceinline__ bool is_far(float m) { return fabsf(m) >= kFar && fabsf(m) < INFINITY; }
// For a maximum that is known.
__device__ __forceinline__ void add_against(Stats& a, float z) {
  const float u = (z - a.m) * kLog2e;
  const float p = __builtin_amdgcn_exp2f(u);
  a.s += p;
  a.t = fmaf(p, fmaxf(u, kLeast), a.t);
}

// The smallest logit that may pass `least`.  Numbers alone are compared so; as
// long as a NaN may pass, it has to go by candidates.
__device__ __forceinline__ float passing(uint64_t least) {
  return order_value(static_cast<uint32_t>(least >> 32));
}
__device__ __forceinline__ bool nan_passes(uint64_t least) { return (least >> 32) <= 1u; }

// An element of each lane, as candidates.
__device__ __forceinline__ void offer(Best& best, float z, uint32_t index, bool there, uint32_t lane, uint32_t top) {
  const uint64_t c = there ? candidate(value_order(z), index) : 0ull;
  uint64_t who = __ballot(c > best.least);
  if (who == 0) return;
  if (best.n + static_cast<uint32_t>(__popcll(who)) > kList) {
    cut_list(best, lane, top);
    who = __ballot(c > best.least);
  }
  if (c > best.least) best.list[best.n + lanes_below(who)] = c;
  best.n += static_cast<uint32_t>(__popcll(who));
}

// Workgroup (row, slice): the statistics and best candidates of `slice`
// elements; with one slice to a row, the row's results.  K waves, steps of U
// vectors.
template <class T, bool TOP, int K, int U>
__global__ __launch_bounds__(K * 64) void logprob_kernel(LogprobArgs a, uint32_t slices, uint32_t slice,
                                                         Partial* partial, uint64_t* best_out) {
  constexpr int E = 16 / sizeof(T);
  typedef Vec<T, E> X;
  __shared__ Stats wave_stats[K];
  __shared__ uint64_t wave_best[TOP ? K : 1][TOP ? kList : 1];
  __shared__ typename X::type staged[TOP ? K : 1][U][TOP ? 64 : 1];
  const uint64_t block = block_id();
  const uint64_t row = block / slices;
  if (row >= a.rows) return;
  const uint32_t part = static_cast<uint32_t>(block - row * slices);
  const uint32_t lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
  const uint32_t begin = part * slice;
  const uint32_t n = min(slice, static_cast<uint32_t>(a.vocab) - begin);
  const T* z = static_cast<const T*>(a.logits) + row * a.stride + begin;
  const Cut<T> cut(z, z, n);
  const uint32_t top = a.top;
  Token token = {false, 0.0f};
  if (slices == 1 && threadIdx.x == 0) token = row_token(a, row);
  const uint32_t one = cut.single(threadIdx.x);
  float alone = one < n ? static_cast<float>(z[one]) : -INFINITY;

  Running st = {-INFINITY, scaled(-INFINITY), 0.0f, 0.0f};
  Best best = {wave_best[TOP ? wave : 0], 0ull, 0u};
  // A step is U vectors of each lane; those past the end read as masked.
  constexpr uint32_t kGroup = 64 * U;
  typename X::type next[U];
  auto load = [&](uint32_t base) {
    const T* p = cut.middle + static_cast<uint64_t>(base + lane) * E;
    if (base + kGroup <= cut.vectors) {  // the same for the wave
#pragma unroll
      for (int j = 0; j < U; ++j) next[j] = load_once<T, E>(p + j * 64 * E);
    } else {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        next[j] = static_cast<T>(-INFINITY);
        if (base + j * 64 + lane < cut.vectors) next[j] = load_once<T, E>(p + j * 64 * E);
      }
    }
  };
  uint32_t base = wave * kGroup;
  if (base < cut.vectors) load(base);
  for (; base < cut.vectors; base += K * kGroup) {
    typename X::type raw[U];
#pragma unroll
    for (int j = 0; j < U; ++j) raw[j] = next[j];
    if (base + K * kGroup < cut.vectors) load(base + K * kGroup);
    float most = static_cast<float>(raw[0][0]);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const typename X::wide f = widen<T, E>(raw[j]);
#pragma unroll
      for (int i = 0; i < E; ++i) most = fmaxf(most, f[i]);
    }
    if (most > st.m) raise(st, most);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const typename X::wide f = widen<T, E>(raw[j]);
#pragma unroll
      for (int i = 0; i < E; ++i) add(st, f[i]);
    }
    if constexpr (TOP) {
      if (nan_passes(best.least) || __ballot(most >= passing(best.least))) {
        // The top-th largest of the lanes' maxima so far, elements of their own,
        // is a lower bound of the top-th largest.  A maximum of -inf may stand
        // for NaNs (which fmaxf passes over) or for the fill past the slice's
        // end, and counts as the lowest order; lanes that are past the end
        // altogether have no element.
        const uint32_t sure = st.m > -INFINITY ? value_order(st.m) : 1u;
        const uint32_t bound = lanes_nth(wave * kGroup + lane < cut.vectors ? sure : 0u, top);
        const uint64_t least = bound <= 1u ? 0ull : candidate(bound, 0xffffffffu) - 1;
        if (least > best.least) best.least = least;
        // A lane's elements that may pass, as bits.
        const float pass = passing(best.least);
        const bool any = nan_passes(best.least);
        uint32_t mine = 0;
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const typename X::wide f = widen<T, E>(raw[j]);
          uint32_t bits = 0;
#pragma unroll
          for (int i = 0; i < E; ++i) bits |= (any || f[i] >= pass ? 1u : 0u) << i;
          if (base + j * 64 + lane < cut.vectors) mine |= bits << (j * E);
        }
        if (__ballot(mine != 0)) {
          // All lanes offer one element at a time, by number: through LDS.
          const uint32_t first = begin + cut.head + (base + lane) * E;
          typename X::type(&stage)[U][TOP ? 64 : 1] = staged[wave];
#pragma unroll
          for (int j = 0; j < U; ++j) stage[j][lane] = raw[j];
          wave_fence();
          do {
            const uint32_t t = mine != 0 ? static_cast<uint32_t>(__builtin_ctz(mine)) : 0u;
            const float z = static_cast<float>(reinterpret_cast<const T*>(&stage[t / E][lane])[t % E]);
            offer(best, z, first + t / E * (64 * E) + t % E, mine != 0, lane, top);
            mine &= mine - 1;
          } while (__ballot(mine != 0));
          wave_fence();
        }
      }
    }
  }
  if (wave == 0) {
    if (alone > st.m) raise(st, alone);
    add(st, alone);
    if constexpr (TOP) offer(best, alone, begin + one, one < n, lane, top);
  }

  Stats own = wave_merge(settled(st));
  if (lane == 0) wave_stats[wave] = own;
  if constexpr (TOP) {
    if (best.n > top) cut_list(best, lane, top);
    if (lane >= best.n && lane < top) best.list[lane] = 0ull;  // none
  }
  __syncthreads();
  Stats all = wave_stats[0];
#pragma unroll
  for (int w = 1; w < K; ++w) all = merge(all, wave_stats[w]);
  if (is_far(all.m)) {  // the same for the workgroup
    const float most = wave_max(st.m);
    __syncthreads();
    if (lane == 0) wave_stats[wave].m = most;
    __syncthreads();
    Stats c = {wave_stats[0].m, 0.0f, 0.0f};
#pragma unroll
    for (int w = 1; w < K; ++w) c.m = fmaxf(c.m, wave_stats[w].m);
    for (uint32_t v = threadIdx.x; v < cut.vectors; v += K * 64) {
      const typename X::wide f = widen<T, E>(load_kept<T, E>(cut.middle + static_cast<uint64_t>(v) * E));
#pragma unroll
      for (int i = 0; i < E; ++i) add_against(c, f[i]);
    }
    if (one < n) add_against(c, alone);
    c.s = wave_sum(c.s);
    c.t = wave_sum(c.t);
    __syncthreads();
    if (lane == 0) wave_stats[wave] = c;
    __syncthreads();
    all = wave_stats[0];
#pragma unroll
    for (int w = 1; w < K; ++w) {
      all.s += wave_stats[w].s;
      all.t += wave_stats[w].t;
    }
  }
  if (threadIdx.x == 0) {
    if (slices == 1)
      finish_row(a, row, all, token);
    else
      partial[block] = {all.m, all.s, all.t, 0.0f};
  }
  if constexpr (TOP) {
    const Level level = level_of(all);
    // A candidate's rank is the number of larger ones; all are different but
    // for 0, which is none.
    for (uint32_t i = threadIdx.x; i < K * top; i += K * 64) {
      const uint64_t c = wave_best[i / top][i % top];
      uint32_t rank = 0, found = 0;
#pragma unroll
      for (int w = 0; w < K; ++w)
#pragma unroll 4
        for (uint32_t j = 0; j < top; ++j) {
          const uint64_t other = wave_best[w][j];
          rank += other > c ? 1u : 0u;
          found += other != 0 ? 1u : 0u;
        }
      if (c != 0 && rank < top) {
        if (slices == 1) {
          a.top_token[row * top + rank] = static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(c));
          a.top_logprob[row * top + rank] = log_prob(level, order_value(static_cast<uint32_t>(c >> 32)));
        } else {
          best_out[block * top + rank] = c;
        }
      }
      // Fewer candidates than `top` in this slice: the rest is none.
      if (slices > 1 && i < top && i >= found) best_out[block * top + i] = 0ull;
    }
  }
}

// A row's slices joined in order.
constexpr int kJoinThreads = 512;
constexpr uint32_t kMaxSlices = 64;
constexpr uint32_t kMaxJoin = 1024;  // candidates, each compared with every other
__global__ __launch_bounds__(kJoinThreads) void logprob_join_kernel(LogprobArgs a, uint32_t slices,
                                                                    const Partial* partial, const uint64_t* best) {
  __shared__ uint64_t cand[kMaxJoin];
  __shared__ uint32_t ranks[kMaxJoin];
  __shared__ Level row_level;
  const uint64_t row = block_id();
  if (row >= a.rows) return;
  const uint32_t top = a.top, n = slices * top;
  Token token = {false, 0.0f};
  if (threadIdx.x == 0) token = row_token(a, row);
  Stats st = {-INFINITY, 0.0f, 0.0f};
  for (uint32_t i = threadIdx.x; i < n; i += kJoinThreads) {
    cand[i] = best[row * n + i];
    ranks[i] = 0;
  }
  if (threadIdx.x < 64) {  // slices <= 64: one wave has them all
    if (threadIdx.x < slices) {
      const Partial p = partial[row * slices + threadIdx.x];
      st = {p.m, p.s, p.t};
    }
    st = wave_merge(st);
    if (threadIdx.x == 0) row_level = level_of(st);
  }
  __syncthreads();
  // A candidate's rank is the number of larger ones, counted in parts.
  constexpr uint32_t kPart = 64;
  const uint32_t parts = (n + kPart - 1) / kPart;
  for (uint32_t i = threadIdx.x; i < n * parts; i += kJoinThreads) {
    const uint32_t who = i % n, first = i / n * kPart, last = min(first + kPart, n);
    const uint64_t c = cand[who];
    uint32_t rank = 0;
#pragma unroll 8
    for (uint32_t j = first; j < last; ++j) rank += cand[j] > c ? 1u : 0u;
    if (rank != 0) atomicAdd(&ranks[who], rank);
  }
  __syncthreads();
  const Level level = row_level;
  for (uint32_t i = threadIdx.x; i < n; i += kJoinThreads) {
    const uint64_t c = cand[i];
    const uint32_t rank = ranks[i];
    if (c == 0 || rank >= top) continue;
    a.top_token[row * top + rank] = static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(c));
    a.top_logprob[row * top + rank] = log_prob(level, order_value(static_cast<uint32_t>(c >> 32)));
  }
  if (threadIdx.x == 0) finish_row(a, row, st, token);  // the token's logit is the last to come
}

// Slices of a row.  Enough workgroups for the chip, none below one step of its
// four waves, and no more than the join takes in one go.  Where steps of
// kUnroll vectors leave CUs idle, half as long ones.
constexpr uint32_t kWantGroups = 1024;
struct Slices {
  uint32_t count, length;
  bool brief;
};
Slices slices_of(uint64_t rows, uint64_t vocab, uint32_t top) {
  uint64_t step = 4 * 64 * kUnroll * 8;  // elements of 16 bits; twice that of fp32
  const bool brief = rows * ((vocab + step - 1) / step) < kCus;
  if (brief) step /= 2;
  uint64_t n = rows == 0 ? 1 : (kWantGroups + rows - 1) / rows;
  const uint64_t most = (vocab + step - 1) / step;
  // A row of few steps is done before a second launch could join its slices
  // (372 rows of 19893 bf16: 8 us whole, 11 in slices; 9 rows of 28928 with 16
  // alternatives, 8 half steps: 20 and 13).
  if (most <= 4) return {1u, static_cast<uint32_t>(vocab), brief};
  n = n < most ? n : most;
  const uint64_t room = top > kMaxJoin / kMaxSlices ? kMaxJoin / top : kMaxSlices;
  n = n < room ? n : room;
  n = n > 0 ? n : 1;
  uint64_t length = (vocab + n - 1) / n;
  length = (length + step - 1) / step * step;
  return {static_cast<uint32_t>((vocab + length - 1) / length), static_cast<uint32_t>(length), brief};
}

// One wave to a row where a wave's step holds most of it and there are rows
// enough: four have barriers, and three of them little to do.
constexpr uint64_t kWaveRow = 4096;
constexpr uint64_t kWaveRows = 1024;

template <class T>
hipError_t logprobs(const LogprobArgs& a, hipStream_t s) {
  const Slices sl = slices_of(a.rows, a.vocab, a.top);
  const uint64_t grid = a.rows * sl.count;
  Partial* partial = static_cast<Partial*>(a.ws);
  uint64_t* best = reinterpret_cast<uint64_t*>(static_cast<char*>(a.ws) + (grid * sizeof(Partial) + 255) / 256 * 256);
  const dim3 g = grid_of(grid);
  if (a.vocab <= kWaveRow && a.rows >= kWaveRows)  // one slice
    return launch(a.top != 0 ? logprob_kernel<T, true, 1, kUnroll> : logprob_kernel<T, false, 1, kUnroll>, g, 64, 0, s, a,
                  sl.count, sl.length, partial, best);
  const auto kernel = sl.brief ? (a.top != 0 ? logprob_kernel<T, true, 4, kUnroll / 2> : logprob_kernel<T, false, 4, kUnroll / 2>)
                               : (a.top != 0 ? logprob_kernel<T, true, 4, kUnroll> : logprob_kernel<T, false, 4, kUnroll>);
  const hipError_t e = launch(kernel, g, kThreads, 0, s, a, sl.count, sl.length, partial, best);
  if (e != hipSuccess || sl.count == 1) return e;
  return launch(logprob_join_kernel, grid_of(a.rows), kJoinThreads, 0, s, a, sl.count, partial, best);
}

// --------------------------------------------------------------- gradient
// Workgroup (row, tile) of kThreads * kUnroll vectors; those of the gradient
// lie on 16-byte boundaries.  The first tile has the row's single elements too.
template <class T>
__global__ __launch_bounds__(kThreads) void logprob_grad_kernel(LogprobGradArgs a, uint32_t tiles) {
  constexpr int E = 16 / sizeof(T);
  typedef Vec<T, E> X;
  const uint64_t block = block_id();
  const uint64_t row = block / tiles;
  if (row >= a.rows) return;
  const uint32_t tile = static_cast<uint32_t>(block - row * tiles);
  const uint32_t base = tile * (kThreads * kUnroll) + threadIdx.x;
  const uint32_t vocab = static_cast<uint32_t>(a.vocab);
  const T* z = static_cast<const T*>(a.logits) + row * a.stride;
  T* dz = static_cast<T*>(a.dlogits) + row * a.dstride;
  const Cut<T> cut(z, dz, vocab);
  T* out = dz + cut.head;
  typename X::type raw[kUnroll];
#pragma unroll
  for (int j = 0; j < kUnroll; ++j)
    if (base + j * kThreads < cut.vectors)
      raw[j] = load_once<T, E>(cut.middle + static_cast<uint64_t>(base + j * kThreads) * E);
  const uint32_t one = tile == 0 ? cut.single(threadIdx.x) : 0xffffffffu;
  const float alone = one < vocab ? static_cast<float>(z[one]) : 0.0f;
  const float lse = a.lse[row], rest = a.lse_rest != nullptr ? a.lse_rest[row] : 0.0f;
  const uint64_t tok = token_at(a.tokens, row, a.wide);
  const uint32_t mine = tok < a.vocab ? static_cast<uint32_t>(tok) : 0xffffffffu;  // no element's index
  const float g = tok < a.vocab ? a.dlogprob[row] : 0.0f;
  const float h = a.dentropy != nullptr ? a.dentropy[row] : 0.0f;
  const float c = a.dentropy != nullptr ? fmaf(h, a.entropy[row], g) : g;  // dz_j = -p_j (c + h log p_j)
  const bool none = lse == -INFINITY;
  auto gradient = [&](float v, uint32_t e) {
    const float lp = (v - lse) - rest;
    const float p = __builtin_amdgcn_exp2f(lp * kLog2e);
    // Of no weight, no gradient: h log p may be past fp32, and 0 times that a NaN.
    float d = p == 0.0f ? 0.0f : -p * fmaf(h, lp, c);
    if (mine == e) d += g;
    return none ? 0.0f : d;
  };
#pragma unroll
  for (int j = 0; j < kUnroll; ++j) {
    const uint32_t v = base + j * kThreads;
    if (v >= cut.vectors) break;
    typename X::wide f = widen<T, E>(raw[j]);
#pragma unroll
    for (int i = 0; i < E; ++i) f[i] = gradient(f[i], cut.head + v * E + i);
    store_once<T, E>(out + static_cast<uint64_t>(v) * E, narrow<T, E>(f));
  }
  if (one < vocab) dz[one] = static_cast<T>(gradient(alone, one));
}

template <class T>
hipError_t logprobs_grad(const LogprobGradArgs& a, hipStream_t s) {
  const uint64_t per = kThreads * kUnroll * (16 / sizeof(T));
  const uint64_t tiles = (a.vocab + per - 1) / per;
  return launch(logprob_grad_kernel<T>, grid_of(a.rows * tiles), kThreads, 0, s, a, static_cast<uint32_t>(tiles));
}

}  // namespace

uint64_t token_logprobs_ws(uint64_t rows, uint64_t vocab, uint32_t top) {
  const Slices sl = slices_of(rows, vocab, top);
  if (sl.count <= 1) return 0;
  return (rows * sl.count * sizeof(Partial) + 255) / 256 * 256 + rows * sl.count * top * sizeof(uint64_t);
}

hipError_t launch_token_logprobs(const LogprobArgs& a, hipStream_t s) {
  if (a.type == RSX_FLOAT32) return logprobs<float>(a, s);
  return a.type == RSX_BFLOAT16 ? logprobs<bf16_t>(a, s) : logprobs<f16_t>(a, s);
}
hipError_t launch_token_logprobs_grad(const LogprobGradArgs& a, hipStream_t s) {
  if (a.type == RSX_FLOAT32) return logprobs_grad<float>(a, s);
  return a.type == RSX_BFLOAT16 ? logprobs_grad<bf16_t>(a, s) : logprobs_grad<f16_t>(a, s);
}

}  // namespace rsx
