// Internal launch interface of the operators that are matrix products
// (feed-forward block, log probabilities from hidden states, orthogonalised
// updates), between their C-ABI layer (product_abi.hip) and their kernels.
// Not installed.
#pragma once

#include "step_internal.h"

namespace rsx {

// Widths (elements of a row) that the product kernels' 32-bit offsets in a tile
// cover, whatever the row stride of a copy is.
constexpr uint64_t kMaxWidth = 1ull << 22;

// Workspace handed out front to back, 256-byte aligned; with a null base it
// counts.
struct Arena {
  char* base;
  uint64_t at = 0;
  explicit Arena(void* p) : base(static_cast<char*>(p)) {}
  void* take(uint64_t bytes) {
    char* p = base ? base + at : nullptr;
    at += (bytes + 255) & ~255ull;
    return p;
  }
};

// A caller's matrix: rows of `cols` elements, `ld` elements apart.
struct Matrix {
  const void* p;
  uint64_t rows, cols, ld;
};

// Whether the tile loads can read a 16-bit matrix where it is: 16-byte chunks
// that start on 16-byte boundaries and do not reach over a row's end.
inline bool in_place(const Matrix& m) {
  return (reinterpret_cast<uintptr_t>(m.p) & 15) == 0 && m.cols % 8 == 0 && (m.rows <= 1 || (m.ld % 8 == 0 && m.ld >= m.cols && m.ld < kMaxWidth));
}

// ---------------------------------------------------------- feed-forward
struct FeedForwardArgs {
  Matrix x, w_gate, w_up, w_down;
  void* out;
  uint64_t out_ld;
  float* gate;  // kept for the gradient; null: not kept
  float* up;
  uint64_t rows, dim, hidden;
  int act, type;
  bool copies;  // some matrix cannot be read in place
  void* ws;
};
uint64_t feed_forward_ws(const FeedForwardArgs& a);
hipError_t launch_feed_forward(const FeedForwardArgs& a, hipStream_t s);

struct FeedForwardGradArgs {
  Matrix dout, x, w_gate, w_up, w_down;
  const float* gate;
  const float* up;
  void* dx;  // null: no gradient of x
  void* dw_gate;  // null: none of the weights
  void* dw_up;
  void* dw_down;
  uint64_t dx_ld, dw_gate_ld, dw_up_ld, dw_down_ld;
  uint64_t rows, dim, hidden;
  int act, type, weight_type, accumulate;
  bool copies;
  void* ws;
};
uint64_t feed_forward_grad_ws(const FeedForwardGradArgs& a);
hipError_t launch_feed_forward_grad(const FeedForwardGradArgs& a, hipStream_t s);

// ------------------------------------- log probabilities from hidden states
struct LinearLogprobArgs {
  Matrix hidden, weight;
  const void* tokens;
  float* logprob;
  float* entropy;   // may be null
  float* lse;
  float* lse_rest;  // may be null
  uint64_t rows, vocab, dim;
  float scale;
  int type, wide;
  bool copies;
  void* ws;
};
uint64_t linear_logprobs_ws(const LinearLogprobArgs& a);
hipError_t launch_linear_logprobs(const LinearLogprobArgs& a, hipStream_t s);

struct LinearLogprobGradArgs {
  Matrix hidden, weight;
  const void* tokens;
  const float* lse;
  const float* lse_rest;  // may be null
  const float* entropy;   // null with dentropy
  const float* dlogprob;
  const float* dentropy;  // may be null
  void* dhidden;          // may be null
  void* dweight;          // may be null
  uint64_t dhidden_ld, dweight_ld;
  uint64_t rows, vocab, dim;
  float scale;
  int type, weight_type, wide, accumulate;
  bool copies;
  void* ws;
};
uint64_t linear_logprobs_grad_ws(const LinearLogprobGradArgs& a);
hipError_t launch_linear_logprobs_grad(const LinearLogprobGradArgs& a, hipStream_t s);

// ------------------------------------------------- orthogonalised updates
struct NewtonSchulzArgs {
  const void* x;
  void* out;
  uint64_t batch, rows, cols, x_ld, out_ld, x_batch, out_batch;
  int steps, type;
  float a, b, c, eps;
  void* ws;
};
uint64_t newton_schulz_ws(uint64_t batch, uint64_t rows, uint64_t cols);
hipError_t launch_newton_schulz(const NewtonSchulzArgs& a, hipStream_t s);

}  // namespace rsx
