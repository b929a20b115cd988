// Internal launch interface of the training-step operators (embedding, layer
// norm, 8-bit checkpoints, token log probabilities), between their C-ABI layer
// (step_abi.hip) and their kernels.  Not installed.
#pragma once

#include "rsx_internal.h"

namespace rsx {

// MI355X's CUs; the kernels that loop over rows size their grids by it.
constexpr uint32_t kCus = 256;

// Bytes a buffer may span: far above the card's memory, and low enough that no
// launch grid below overflows.
constexpr uint64_t kMaxSpan = 1ull << 45;

// Grid of `n` workgroups as x * y: HIP counts the work-items of one dimension
// in 32 bits.  Workgroups past the last one have nothing to do.
constexpr uint64_t kGridX = 1ull << 20;
inline dim3 grid_of(uint64_t n) {
  if (n <= kGridX) return dim3(static_cast<uint32_t>(n));
  return dim3(static_cast<uint32_t>(kGridX), static_cast<uint32_t>((n + kGridX - 1) / kGridX));
}

// ------------------------------------------------------------- embedding
struct EmbedArgs {
  const void* table;
  const void* tokens;
  void* out;
  uint64_t table_stride, out_stride;  // elements between rows
  uint64_t n;                         // tokens
  uint64_t vocab, dim;
  int64_t first;                      // token id of the table's first row
  float scale;
  int table_type, out_type, wide;     // wide: tokens are int64
};
hipError_t launch_embedding(const EmbedArgs& a, hipStream_t s);

struct EmbedGradArgs {
  const void* dout;
  const void* tokens;
  void* grad;
  uint64_t dout_stride, grad_stride;
  uint64_t n, vocab, dim;
  int64_t first;
  float scale;
  int dout_type, grad_type, wide, accumulate;
  void* ws;
};
// Workspace of the gradient, in bytes.
uint64_t embedding_grad_ws(uint64_t vocab, uint64_t dim, uint64_t n);
hipError_t launch_embedding_grad(const EmbedGradArgs& a, hipStream_t s);

// ------------------------------------------------------------ layer norm
// Elements of a row that share one scale byte of a checkpoint.
constexpr uint32_t kCkBlock = 32;
constexpr uint64_t ck_blocks(uint64_t dim) { return dim / kCkBlock + (dim % kCkBlock != 0); }

struct NormArgs {
  const void* x;
  const void* weight;  // may be null
  const void* bias;    // may be null
  void* y;
  float* mean;         // may be null
  float* rstd;         // may be null
  int8_t* codes;       // checkpoint of x; null without one
  uint8_t* scales;
  uint64_t x_stride, y_stride, rows, dim;
  float eps;
  int type, weight_type;
};
hipError_t launch_layer_norm(const NormArgs& a, hipStream_t s);

struct NormGradArgs {
  const void* dy;
  const void* x;       // null: the row comes from codes and scales
  const int8_t* codes;
  const uint8_t* scales;
  const float* mean;
  const float* rstd;
  const void* weight;  // may be null
  void* dx;
  void* dweight;       // may be null
  void* dbias;         // may be null
  float* partial;      // workspace
  uint64_t dy_stride, x_stride, dx_stride, rows, dim;
  int type, weight_type;
};
uint64_t layer_norm_grad_ws(uint64_t rows, uint64_t dim);
hipError_t launch_layer_norm_grad(const NormGradArgs& a, hipStream_t s);

struct PackArgs {
  const void* x;
  void* out;
  int8_t* codes;
  uint8_t* scales;
  uint64_t stride, rows, dim;  // stride of x (pack) or out (unpack)
  int type;
};
hipError_t launch_checkpoint_pack(const PackArgs& a, hipStream_t s);
hipError_t launch_checkpoint_unpack(const PackArgs& a, hipStream_t s);

// ------------------------------------------------- token log probabilities
struct LogprobArgs {
  const void* logits;
  const void* tokens;
  float* logprob;
  float* entropy;      // may be null
  float* lse;
  float* lse_rest;     // may be null
  float* top_logprob;
  int32_t* top_token;
  void* ws;
  uint64_t stride, rows, vocab;
  uint32_t top;
  int type, wide;
};
uint64_t token_logprobs_ws(uint64_t rows, uint64_t vocab, uint32_t top);
hipError_t launch_token_logprobs(const LogprobArgs& a, hipStream_t s);

struct LogprobGradArgs {
  const void* logits;
  const void* tokens;
  const float* lse;
  const float* lse_rest;  // may be null
  const float* entropy;   // null with dentropy
  const float* dlogprob;
  const float* dentropy;  // may be null
  void* dlogits;
  uint64_t stride, dstride, rows, vocab;
  int type, wide;
};
hipError_t launch_token_logprobs_grad(const LogprobGradArgs& a, hipStream_t s);

}  // namespace rsx
