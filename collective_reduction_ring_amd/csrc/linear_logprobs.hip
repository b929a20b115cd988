// Log probabilities of tokens from hidden states, z = scale * h W^T, and their
// gradient, without the logits in memory.
//
// Forward: each tile of the product leaves, for each of its rows, the largest
// logit, the sum of exp(z - largest) and that sum weighted by z - largest; a
// second launch joins a row's tiles.
//
// Gradient: the vocabulary is taken in pieces.  A piece's logits are multiplied
// again, and the tile's epilogue makes of them
//   dz_j = scale * (g (delta(j, token) - p_j) - d p_j (log p_j + entropy)),
// the operand of two products, dW = dz^T h for the piece's rows (each complete)
// and dh += dz W.  That is 4/3 of the operations of keeping all logits, and
// memory for one piece.
//
// What is rounded: dz, as an operand, to bf16; with fp16 matrices it is two bf16
// parts, and so are the matrices, since probabilities of large vocabularies lie
// below fp16's range; with fp32 all is three.  Most of a row's dz is its token's.
// Each row is divided by about that before it is rounded, dz = c dz', so that the
// token's is 1 and keeps all its digits: dhidden = c (dz' W) is as good as
// its own rounding, and dW = dz'^T (c h) has the rounding of c h, one by one.
// Rounded as it is, a row's dz would be off by one error in all its elements, and
// where all rows have one weight, all rows by the same.
//
// The time is the tile products', for few rows the memory's.  4096 x 131072 x 4096
// bf16: forward 3160 us (1392 TFLOP/s); each of four pieces' dz 902, dW 845 and dh
// 755 (1457 TFLOP/s).  8 rows: 191 us, 5.6 TB/s.
#include "few_rows.h"
#include "product_store.h"

namespace rsx {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ int64_t token_at(const void* tokens, int wide, uint32_t i) {
  return wide ? static_cast<const int64_t*>(tokens)[i] : static_cast<const int32_t*>(tokens)[i];
}

// Of some of a row's logits: the largest, and the sums over them of e and of
// e * (z - largest), e = exp(z - largest).
struct Some {
  float most, sum, gap;
};
__device__ __forceinline__ float less(float z, float most) { return most == -INFINITY ? z : z - most; }
__device__ __forceinline__ Some joined(const Some& a, const Some& b) {
  const float m = fmaxf(a.most, b.most);
  const float da = less(a.most, m), db = less(b.most, m);
  const float ea = __builtin_amdgcn_exp2f(da * kLog2e), eb = __builtin_amdgcn_exp2f(db * kLog2e);
  // an empty part has sums of 0 (or of NaN, which stay in the sum); so far below the other that e is 0, d may be -inf
  Some r = {m, 0.0f, 0.0f};
  r.sum = (a.most == -INFINITY ? a.sum : a.sum * ea) + (b.most == -INFINITY ? b.sum : b.sum * eb);
  r.gap = (ea == 0.0f ? 0.0f : (a.gap + a.sum * da) * ea) + (eb == 0.0f ? 0.0f : (b.gap + b.sum * db) * eb);
  return r;
}
__device__ __forceinline__ Some across(const Some& a, int lanes) {
  return joined(a, {__shfl_xor(a.most, lanes), __shfl_xor(a.sum, lanes), __shfl_xor(a.gap, lanes)});
}

struct SoftmaxArgs {
  float4* some;   // [row][tile]
  float* picked;  // the token's logit, of rows that have one
  const void* tokens;
  uint32_t tiles;
  int wide;
  float scale;
};

struct Softmax {
  typedef SoftmaxArgs Args;
  // N groups of four logits of one row, at columns c(j).  EDGE: those from `vocab` on do not count.
  template <bool EDGE, int N, class C>
  static __device__ __forceinline__ Some take(const SoftmaxArgs& e, const f32x4 (&v)[N], C c, uint32_t vocab) {
    float z[4 * N];
    Some s = {-INFINITY, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        z[4 * j + x] = v[j][x] * e.scale;
        if (EDGE && c(j) + x >= vocab) z[4 * j + x] = -INFINITY;
        s.most = fmaxf(s.most, z[4 * j + x]);
      }
    const float from = s.most == -INFINITY ? 0.0f : s.most;
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) {
      const float d = z[i] - from, x = __builtin_amdgcn_exp2f(d * kLog2e);
      s.sum += x;
      s.gap += x * fmaxf(d, -1e30f);  // 0 for a logit of minus infinity; a NaN shows in the sum
    }
    return s;
  }
  // The token's logit, where this lane has it.
  template <int N, class C>
  static __device__ __forceinline__ void pick(const SoftmaxArgs& e, const f32x4 (&v)[N], C c, int64_t token, uint32_t row) {
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (c(j) + x == token) e.picked[row] = v[j][x] * e.scale;
  }
  template <class T, class TILE, int N>
  static __device__ __forceinline__ void run(const ProductArgs& p, const Where& w, const SoftmaxArgs& e,
                                             const f32x4 (&acc)[TILE::TN][N], uint32_t i0, RSX_LDS char* lds) {
    const Place<TILE> at(w);
    const uint32_t l = threadIdx.x % 64, wave = threadIdx.x / 64;
    const uint32_t first = w.n0 + uniform(wave) % TILE::WN * (TILE::TN * 16);  // this wave's columns
    const bool edge = first + TILE::TN * 16 > p.n;
    RSX_LDS float* part = reinterpret_cast<RSX_LDS float*>(lds);  // [wave column][row of the tile][3]
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t row = at.row(i0 + i);
      const int64_t token = row < p.m ? token_at(e.tokens, e.wide, row) : -1;
      f32x4 v[TILE::TN];
#pragma unroll
      for (int j = 0; j < TILE::TN; ++j) v[j] = acc[j][i];
      auto column = [&](int j) { return at.col(j); };
      const bool mine = token >= first && token < min(first + TILE::TN * 16, p.n);
      if (__ballot(mine) != 0) pick(e, v, column, mine ? token : -1, row);
      Some s = edge ? take<true>(e, v, column, p.n) : take<false>(e, v, column, p.n);
      s = across(across(s, 16), 32);
      if (l < 16) {
        RSX_LDS float* to = part + ((wave % TILE::WN) * TILE::BM + (row - w.m0)) * 3;
        to[0] = s.most;
        to[1] = s.sum;
        to[2] = s.gap;
      }
    }
    __syncthreads();
    for (uint32_t r = threadIdx.x; r < TILE::BM && w.m0 + r < p.m; r += TILE::kThreads) {
      if (N < TILE::TM && r / 16 % TILE::TM != i0) continue;
      Some s = {part[r * 3], part[r * 3 + 1], part[r * 3 + 2]};
#pragma unroll
      for (int i = 1; i < TILE::WN; ++i) {
        RSX_LDS const float* q = part + (i * TILE::BM + r) * 3;
        s = joined(s, {q[0], q[1], q[2]});
      }
      e.some[static_cast<uint64_t>(w.m0 + r) * e.tiles + w.n0 / TILE::BN] = float4{s.most, s.sum, s.gap, 0.0f};
    }
  }
  template <class T, int RG>
  static __device__ __forceinline__ void few(const FewArgs& p, const SoftmaxArgs& e, uint32_t row, uint32_t c, const f32x4 (&v)[RG]) {
    const int64_t token = row < p.n ? token_at(e.tokens, e.wide, row) : -1;
    auto column = [&](int j) { return c + 16 * j; };
    pick(e, v, column, token >= 0 && token < p.rows ? token : -1, row);
    Some s = take<true>(e, v, column, p.rows);
    s = across(across(s, 16), 32);
    if (row < p.n && threadIdx.x % 64 < 16)
      e.some[static_cast<uint64_t>(row) * e.tiles + c / (16 * RG)] = float4{s.most, s.sum, s.gap, 0.0f};
  }
};

struct JoinArgs {
  const float4* some;
  const float* picked;
  const void* tokens;
  float* logprob;
  float* entropy;
  float* lse;
  float* lse_rest;
  uint32_t rows, tiles;
  uint64_t vocab;
  int wide;
};

// One workgroup a row.
__global__ __launch_bounds__(256) void join_tiles(const JoinArgs a) {
  const uint64_t row = block_id();
  if (row >= a.rows) return;
  __shared__ float part[4][3];
  Some s = {-INFINITY, 0.0f, 0.0f};
  for (uint32_t i = threadIdx.x; i < a.tiles; i += 256) {
    const float4 q = a.some[row * a.tiles + i];
    s = joined(s, {q.x, q.y, q.z});
  }
#pragma unroll
  for (int lanes = 1; lanes < 64; lanes *= 2) s = across(s, lanes);
  if (threadIdx.x % 64 == 0) {
    part[threadIdx.x / 64][0] = s.most;
    part[threadIdx.x / 64][1] = s.sum;
    part[threadIdx.x / 64][2] = s.gap;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
#pragma unroll
  for (int i = 1; i < 4; ++i) s = joined(s, {part[i][0], part[i][1], part[i][2]});
  const int64_t token = token_at(a.tokens, a.wide, static_cast<uint32_t>(row));
  const bool there = token >= 0 && static_cast<uint64_t>(token) < a.vocab;
  const bool none = s.most == -INFINITY && s.sum == 0.0f;
  const float ln = logf(s.sum);
  const float lse = none ? -INFINITY : s.most + ln;
  a.lse[row] = lse;
  if (a.lse_rest) {  // what the rounding of the sum took, from the larger and the smaller of the two
    const float big = fabsf(s.most) >= fabsf(ln) ? s.most : ln, small = fabsf(s.most) >= fabsf(ln) ? ln : s.most;
    a.lse_rest[row] = fabsf(lse) < INFINITY ? small - (lse - big) : 0.0f;
  }
  a.logprob[row] = !there ? 0.0f : none ? -INFINITY : (a.picked[row] - s.most) - ln;
  if (a.entropy) a.entropy[row] = none ? 0.0f : ln - s.gap / s.sum;
}

// What a row of dz is made of, but for its logits.
struct RowArgs {
  const void* tokens;
  const float* lse;
  const float* lse_rest;
  const float* entropy;
  const float* dlogprob;
  const float* dentropy;
  uint64_t vocab;
  float scale;
  int wide;
};
struct Row {
  int64_t token;  // -1: none in the vocabulary
  float lse, rest, g, d, h;
  __device__ __forceinline__ Row(const RowArgs& e, uint32_t i) {
    token = token_at(e.tokens, e.wide, i);
    if (token < 0 || static_cast<uint64_t>(token) >= e.vocab) token = -1;
    lse = e.lse[i];
    rest = e.lse_rest ? e.lse_rest[i] : 0.0f;
    g = token >= 0 ? e.dlogprob[i] : 0.0f;
    d = e.dentropy ? e.dentropy[i] : 0.0f;
    h = e.dentropy ? e.entropy[i] : 0.0f;
  }
  // The gradient in logit z.
  __device__ __forceinline__ float dz(float z, bool hit) const {
    const float lp = (z - lse) - rest, p = __builtin_amdgcn_exp2f(lp * kLog2e), own = hit ? g : 0.0f;
    if (lse == -INFINITY) return 0.0f;
    return p == 0.0f ? own : own - p * (g + d * (lp + h));
  }
};

// Each row's factor c, and c h in parts: a workgroup a row.  c is scale times the
// token's dz, or what bounds dz where that is small beside it or not there.
template <class S>
__global__ __launch_bounds__(256) void scale_rows(const S* hidden, uint64_t ld, const S* weight, uint64_t wld, uint32_t rows, uint32_t dim,
                                                  RowArgs e, float* factor, Parts to) {
  const uint64_t i = block_id();
  if (i >= rows) return;
  __shared__ float part[4];
  const Row row(e, static_cast<uint32_t>(i));
  const S* h = hidden + i * ld;
  float sum = 0.0f;
  if (row.token >= 0) {
    const S* w = weight + row.token * wld;
    for (uint64_t c = threadIdx.x * 8; c < dim; c += 2048) {
      const auto a = load_row<S, 8, false>(h, static_cast<uint32_t>(c), dim), b = load_row<S, 8, false>(w, static_cast<uint32_t>(c), dim);
#pragma unroll
      for (int x = 0; x < 8; ++x) sum = fmaf(static_cast<float>(a[x]), static_cast<float>(b[x]), sum);
    }
  }
  sum = wave_sum(sum);
  if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = sum;
  __syncthreads();
  const float most = fabsf(row.g) + fabsf(row.d);
  float c = row.token >= 0 ? row.dz(((part[0] + part[1]) + (part[2] + part[3])) * e.scale, true) : most;
  // (not of a NaN, which is to show)
  if (fabsf(c) < most * (row.d == 0.0f ? 0x1p-20f : 0x1p-3f)) c = most;
  c = row.lse == -INFINITY || most == 0.0f ? 0.0f : c * e.scale;  // without a gradient, a row adds nothing whatever it holds
  if (c != 0.0f && fabsf(c) < 1e-30f) c = 1e-30f;  // so that 1 / c and the parts of c h are in range
  if (threadIdx.x == 0) factor[i] = c;
  if (to.count == 0) return;
  for (uint64_t x = threadIdx.x * 8; x < dim; x += 2048) {
    f32x8 v = __builtin_convertvector((load_row<S, 8, false>(h, static_cast<uint32_t>(x), dim)), f32x8) * c;
    if (c == 0.0f) v = f32x8{};  // whatever h is
    put_parts<bf16_t, 8>(to, i, static_cast<uint32_t>(x), dim, v);
  }
}

struct DzArgs {
  RowArgs row;
  const float* factor;
  Parts dz;
  uint64_t first;  // the piece's first row of the matrix
};

struct Dz {
  typedef DzArgs Args;
  template <class T, class TILE, int N>
  static __device__ __forceinline__ void run(const ProductArgs& p, const Where& w, const DzArgs& e,
                                             const f32x4 (&acc)[TILE::TN][N], uint32_t i0, RSX_LDS char* lds) {
    staged<TILE, false, N>(w, acc, i0, lds, [&](uint32_t i, uint32_t c, f32x8 v) {
      if (i >= p.m) return;
      Row row(e.row, i);
      const float f = e.factor[i], by = f == 0.0f ? 0.0f : e.row.scale / f;
      if (f == 0.0f) row.lse = -INFINITY;  // a row without a gradient, whatever it holds
      const uint64_t hit = row.token >= 0 ? static_cast<uint64_t>(row.token) - e.first : ~0ull;
#pragma unroll
      for (int x = 0; x < 8; ++x) v[x] = row.dz(v[x] * e.row.scale, c + x == hit) * by;
      put_parts<bf16_t, 8>(e.dz, i, c, p.n, v);
    });
  }
};

#define RSX_TRY(x)                        \
  do {                                    \
    const hipError_t st_ = (x);           \
    if (st_ != hipSuccess) return st_;    \
  } while (0)

ProductArgs sizes(uint64_t m, uint64_t n, uint64_t k) {
  ProductArgs p = {};
  p.m = static_cast<uint32_t>(m);
  p.n = static_cast<uint32_t>(n);
  p.k = static_cast<uint32_t>(k);
  p.batch = 1;
  return p;
}

// Whether a call takes the few-row form: 16-bit matrices that the tiles read in
// place are faster there from 17 rows on (65536 x 4096 bf16: 99 us for 16 rows and
// 113 to 120 for 17 to 128 in tiles, 129 for 32 here); others would be copied first.
bool few_form(const LinearLogprobArgs& a) { return a.rows <= (a.type == RSX_FLOAT32 || a.copies ? kFewRows : 16); }

constexpr int kFewGroups = 2;  // of 16 matrix rows: with one, x is read from L2 as often as the matrix from memory

struct Forward {
  Prepared hidden, weight;
  float4* some;
  float* picked;
  uint32_t tiles;
  bool few;
  Schedule spread;
  void* pieces;
};
Forward plan(const LinearLogprobArgs& a, Arena& ws) {
  Forward f = {};
  const int n = a.type == RSX_FLOAT32 ? 3 : 1;
  const bool half = a.type == RSX_FLOAT16;
  f.few = few_form(a);
  f.spread = schedule(a.rows, a.vocab, 1, steps_of(a.dim, segments_of(n, n)), false, false);
  const uint64_t width = f.few ? 16 * kFewGroups : f.spread.tile == 0 ? Large::BN : Middle::BN;
  f.tiles = static_cast<uint32_t>((a.vocab + width - 1) / width);
  if (!f.few) {
    f.hidden = take_operand(ws, a.hidden, a.type, n, half, a.copies);
    f.weight = take_operand(ws, a.weight, a.type, n, half, a.copies);
    f.pieces = ws.take(f.spread.bytes);
  }
  f.some = static_cast<float4*>(ws.take(a.rows * f.tiles * sizeof(float4)));
  f.picked = static_cast<float*>(ws.take(a.rows * 4));
  return f;
}

// Columns of a piece: 2^27 elements of dz (256 MB of bf16: the Infinity Cache's
// size), at least 16 tiles, and at most what the tile loads' offsets reach over.
uint64_t piece(uint64_t rows, uint64_t vocab) {
  uint64_t n = ((1ull << 27) / (rows ? rows : 1)) & ~4095ull;
  n = n < 4096 ? 4096 : n > (1ull << 20) ? 1ull << 20 : n;
  return n < vocab ? n : vocab;
}

struct Backward {
  Prepared hidden, weight;  // of the logits' product
  Prepared weight2;         // of dhidden's
  Parts scaled;             // rows of hidden times their factors
  Parts dz;
  float* factor;
  int parts;  // of the operands in the gradients' products
  float* sum;  // dhidden so far
  void* split;
  uint64_t piece;
};
Backward plan(const LinearLogprobGradArgs& a, Arena& ws) {
  Backward b = {};
  const bool half = a.type == RSX_FLOAT16;
  const int n = a.type == RSX_FLOAT32 ? 3 : 1, n2 = half ? 2 : n;
  b.parts = n2;
  b.hidden = take_operand(ws, a.hidden, a.type, n, half, a.copies);
  b.weight = take_operand(ws, a.weight, a.type, n, half, a.copies);
  b.weight2 = b.weight;
  if (half && a.dhidden) b.weight2 = take_operand(ws, a.weight, a.type, n2, false, a.copies);
  if (a.dweight) b.scaled = take_parts(ws, a.rows, a.dim, n2);
  b.factor = static_cast<float*>(ws.take(a.rows * 4));
  b.piece = piece(a.rows, a.vocab);
  b.dz = take_parts(ws, a.rows, b.piece, n2);
  if (a.dhidden && b.piece < a.vocab) b.sum = static_cast<float*>(ws.take(a.rows * a.dim * 4));
  const uint64_t segs = segments_of(n2, n2);
  uint64_t split = 0;
  const uint64_t last = b.piece ? a.vocab % b.piece : 0;  // the last piece is cut in its own way
  for (const uint64_t v : {b.piece, last}) {
    if (v == 0) continue;
    const uint64_t h = a.dhidden ? store_ws(a.rows, a.dim, v, segs) : 0, w = a.dweight ? store_ws(v, a.dim, a.rows, segs) : 0;
    const uint64_t z = schedule(a.rows, v, 1, steps_of(a.dim, segments_of(n, n)), false, false).bytes;
    split = split < h ? h : split;
    split = split < w ? w : split;
    split = split < z ? z : split;
  }
  b.split = ws.take(split);
  return b;
}

template <class S>
hipError_t factors(const LinearLogprobGradArgs& a, const Backward& b, const RowArgs& row, hipStream_t s) {
  return launch(scale_rows<S>, grid_of(a.rows), 256, 0, s, static_cast<const S*>(a.hidden.p), a.hidden.ld, static_cast<const S*>(a.weight.p),
                a.weight.ld, static_cast<uint32_t>(a.rows), static_cast<uint32_t>(a.dim), row, b.factor, b.scaled);
}

}  // namespace

uint64_t linear_logprobs_ws(const LinearLogprobArgs& a) {
  Arena ws(nullptr);
  plan(a, ws);
  if (!a.copies) return ws.at;
  // what is right for matrices that are copied is right for others too
  LinearLogprobArgs b = a;
  b.copies = false;
  Arena other(nullptr);
  plan(b, other);
  return ws.at > other.at ? ws.at : other.at;
}

hipError_t launch_linear_logprobs(const LinearLogprobArgs& a, hipStream_t s) {
  Arena ws(a.ws);
  const Forward f = plan(a, ws);
  const bool half = a.type == RSX_FLOAT16;
  const SoftmaxArgs e = {f.some, f.picked, a.tokens, f.tiles, a.wide, a.scale};
  if (f.few) {
    const FewArgs p = {a.hidden.p, a.weight.p, nullptr, a.hidden.ld, a.weight.ld, 0, static_cast<uint32_t>(a.rows),
                       static_cast<uint32_t>(a.vocab), static_cast<uint32_t>(a.dim)};
    RSX_TRY((a.type == RSX_FLOAT32 ? launch_few<float, kFewGroups, false, Softmax>(p, e, s)
             : half                ? launch_few<f16_t, kFewGroups, false, Softmax>(p, e, s)
                                   : launch_few<bf16_t, kFewGroups, false, Softmax>(p, e, s)));
  } else {
    Copies c = {};
    fill_operand(c, f.hidden, a.hidden);
    fill_operand(c, f.weight, a.weight);
    RSX_TRY(launch_copies(c, a.type, half, s));
    ProductArgs p = sizes(a.rows, a.vocab, a.dim);
    const int n = a.type == RSX_FLOAT32 ? 3 : 1;
    add_segments(p, f.hidden.op, n, f.weight.op, n);
    RSX_TRY((half ? launch_product<f16_t, kRow, kRow, false, false, Softmax>(p, f.spread, f.pieces, e, s)
                  : launch_product<bf16_t, kRow, kRow, false, false, Softmax>(p, f.spread, f.pieces, e, s)));
  }
  return launch(join_tiles, grid_of(a.rows), 256, 0, s,
                {f.some, f.picked, a.tokens, a.logprob, a.entropy, a.lse, a.lse_rest, static_cast<uint32_t>(a.rows), f.tiles,
                 a.vocab, a.wide});
}

uint64_t linear_logprobs_grad_ws(const LinearLogprobGradArgs& a) {
  Arena ws(nullptr);
  plan(a, ws);
  return ws.at;
}

hipError_t launch_linear_logprobs_grad(const LinearLogprobGradArgs& a, hipStream_t s) {
  const bool half = a.type == RSX_FLOAT16;
  const int n = a.type == RSX_FLOAT32 ? 3 : 1;
  Arena ws(a.ws);
  const Backward b = plan(a, ws);
  Copies copies = {};
  fill_operand(copies, b.hidden, a.hidden);
  fill_operand(copies, b.weight, a.weight);
  RSX_TRY(launch_copies(copies, a.type, half, s));
  if (half && a.dhidden) {
    Copies c = {};
    fill_operand(c, b.weight2, a.weight);
    RSX_TRY(launch_copies(c, a.type, false, s));
  }
  const RowArgs row = {a.tokens, a.lse, a.lse_rest, a.entropy, a.dlogprob, a.dentropy, a.vocab, a.scale, a.wide};
  if (a.rows)
    RSX_TRY(a.type == RSX_FLOAT32    ? factors<float>(a, b, row, s)
            : a.type == RSX_BFLOAT16 ? factors<bf16_t>(a, b, row, s) : factors<f16_t>(a, b, row, s));
  const uint64_t es = a.weight_type == RSX_FLOAT32 ? 4 : 2;
  for (uint64_t first = 0; first < a.vocab; first += b.piece) {
    const uint64_t v = a.vocab - first < b.piece ? a.vocab - first : b.piece;
    auto rows_from = [&](Operand o) {
      for (const void*& part : o.part)
        if (part) part = static_cast<const char*>(part) + first * o.ld * 2;
      return o;
    };
    if (a.rows) {
      ProductArgs p = sizes(a.rows, v, a.dim);
      add_segments(p, b.hidden.op, n, rows_from(b.weight.op), n);
      const DzArgs e = {row, b.factor, b.dz, first};
      const Schedule c = schedule(a.rows, v, 1, steps_of(a.dim, p.nseg), false, false);
      RSX_TRY((half ? launch_product<f16_t, kRow, kRow, false, false, Dz>(p, c, b.split, e, s)
                    : launch_product<bf16_t, kRow, kRow, false, false, Dz>(p, c, b.split, e, s)));
    }
    if (a.dweight) {
      ProductArgs p = sizes(v, a.dim, a.rows);
      add_segments(p, operand(b.dz), b.parts, operand(b.scaled), b.parts);
      void* to = static_cast<char*>(a.dweight) + first * a.dweight_ld * es;
      RSX_TRY(launch_store(false, kTN, p, {to, a.dweight_ld, a.weight_type, nullptr, nullptr, a.accumulate}, b.split, s));
    }
    if (a.dhidden) {
      ProductArgs p = sizes(a.rows, a.dim, v);
      add_segments(p, operand(b.dz), b.parts, rows_from(b.weight2.op), b.parts);
      const bool last = first + v == a.vocab;
      const float* add = first ? b.sum : nullptr;
      const StoreArgs e = last ? StoreArgs{a.dhidden, a.dhidden_ld, a.type, add, b.factor, 0}
                               : StoreArgs{b.sum, a.dim, RSX_FLOAT32, add, nullptr, 0};
      RSX_TRY(launch_store(false, kNN, p, e, b.split, s));
    }
  }
  return hipSuccess;
}

}  // namespace rsx
