// C ABI of the operators that are matrix products (declared in include/rsx.h):
// argument validation and aliasing rules.  Every check runs before the first
// HIP call.
#include "areas.h"
#include "product_internal.h"

namespace rsx {
namespace {

bool act_known(int act) { return act >= RSX_ACT_SILU && act <= RSX_ACT_RELU; }

// A weight gradient is of the weights' type or fp32.
size_t grad_size(int type, int weight_type) { return weight_type == type || weight_type == RSX_FLOAT32 ? float_size(weight_type) : 0; }

// 128 x 128 tiles of the products m x n that a call launches: few enough for one grid.
bool tiles_fit(uint64_t m, uint64_t n) { return ((m + 127) / 128) * ((n + 63) / 64) < (1ull << 30); }

bool copies(std::initializer_list<Matrix> all) {
  for (const Matrix& m : all)
    if (m.rows != 0 && m.cols != 0 && !in_place(m)) return true;
  return false;
}

}  // namespace
}  // namespace rsx

using namespace rsx;

extern "C" {

size_t rsx_feed_forward_workspace_size(size_t rows, size_t dim, size_t hidden, rsx_dtype_t type, int copies) {
  if (rows > kMaxSize || dim >= kMaxWidth || hidden >= kMaxWidth || float_size(type) == 0 || rows == 0 || dim == 0) return 0;
  return feed_forward_ws({{nullptr, rows, dim, dim}, {nullptr, hidden, dim, dim}, {nullptr, hidden, dim, dim},
                          {nullptr, dim, hidden, hidden}, nullptr, 0, nullptr, nullptr, rows, dim, hidden, 0, type, copies != 0, nullptr});
}

rsx_status_t rsx_feed_forward(const void* x, size_t x_stride, const void* w_gate, size_t gate_stride,
                              const void* w_up, size_t up_stride, const void* w_down,
                              size_t down_stride, void* out, size_t out_stride, float* gate, float* up,
                              size_t rows, size_t dim, size_t hidden, rsx_activation_t activation,
                              rsx_dtype_t type, void* workspace, size_t workspace_bytes,
                              hipStream_t stream) {
  const size_t es = float_size(type);
  if (es == 0) return RSX_ERR_INVALID_TYPE;
  if (!act_known(activation)) return RSX_ERR_INVALID_OP;
  if (rows > kMaxSize || dim >= kMaxWidth || hidden >= kMaxWidth || !tiles_fit(rows, dim) || !tiles_fit(rows, 2 * hidden))
    return RSX_ERR_UNSUPPORTED;
  if ((gate == nullptr) != (up == nullptr)) return RSX_ERR_INVALID_ARGUMENT;
  Areas m;
  m.write(out, rows, dim, out_stride, es);
  m.read(x, rows, dim, x_stride, es);
  m.read(w_gate, hidden, dim, gate_stride, es);
  m.read(w_up, hidden, dim, up_stride, es);
  m.read(w_down, dim, hidden, down_stride, es);
  if (gate != nullptr) {
    m.write(gate, rows, hidden, hidden, 4);
    m.write(up, rows, hidden, hidden, 4);
  }
  const Matrix mx = {x, rows, dim, x_stride}, mg = {w_gate, hidden, dim, gate_stride}, mu = {w_up, hidden, dim, up_stride},
               md = {w_down, dim, hidden, down_stride};
  const bool move = copies({mx, mg, mu, md});
  m.workspace(workspace, workspace_bytes, rsx_feed_forward_workspace_size(rows, dim, hidden, type, move));
  const rsx_status_t st = m.status();
  if (st != RSX_SUCCESS || rows == 0 || dim == 0) return st;
  return hip_status(launch_feed_forward({mx, mg, mu, md, out, out_stride, gate, up, rows, dim, hidden, activation, type, move, workspace},
                                        stream));
}

size_t rsx_feed_forward_grad_workspace_size(size_t rows, size_t dim, size_t hidden, rsx_dtype_t type, int copies) {
  if (rows > kMaxSize || dim >= kMaxWidth || hidden >= kMaxWidth || float_size(type) == 0 || dim == 0) return 0;
  void* some = &copies;  // every gradient is wanted
  return feed_forward_grad_ws({{nullptr, rows, dim, dim}, {nullptr, rows, dim, dim}, {nullptr, hidden, dim, dim}, {nullptr, hidden, dim, dim},
                               {nullptr, dim, hidden, hidden}, nullptr, nullptr, some, some, some, some, 0, 0, 0, 0, rows, dim, hidden, 0,
                               type, type, 0, copies != 0, nullptr});
}

rsx_status_t rsx_feed_forward_grad(const void* dout, size_t dout_stride, const void* x, size_t x_stride,
                                   const void* w_gate, size_t gate_stride, const void* w_up,
                                   size_t up_stride, const void* w_down, size_t down_stride,
                                   const float* gate, const float* up, void* dx, size_t dx_stride,
                                   void* dw_gate, size_t dw_gate_stride, void* dw_up,
                                   size_t dw_up_stride, void* dw_down, size_t dw_down_stride,
                                   size_t rows, size_t dim, size_t hidden,
                                   rsx_activation_t activation, rsx_dtype_t type,
                                   rsx_dtype_t weight_grad_type, int accumulate, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream) {
  const size_t es = float_size(type), gs = grad_size(type, weight_grad_type);
  if (es == 0 || gs == 0) return RSX_ERR_INVALID_TYPE;
  if (!act_known(activation)) return RSX_ERR_INVALID_OP;
  if (rows > kMaxSize || dim >= kMaxWidth || hidden >= kMaxWidth || !tiles_fit(rows, dim) || !tiles_fit(rows, hidden) ||
      !tiles_fit(dim, hidden))
    return RSX_ERR_UNSUPPORTED;
  if ((dw_gate == nullptr) != (dw_up == nullptr) || (dw_gate == nullptr) != (dw_down == nullptr)) return RSX_ERR_INVALID_ARGUMENT;
  Areas m;
  m.read(dout, rows, dim, dout_stride, es);
  m.read(x, rows, dim, x_stride, es);
  m.read(w_gate, hidden, dim, gate_stride, es);
  m.read(w_up, hidden, dim, up_stride, es);
  m.read(w_down, dim, hidden, down_stride, es);
  m.read(gate, rows, hidden, hidden, 4);
  m.read(up, rows, hidden, hidden, 4);
  if (dx != nullptr) m.write(dx, rows, dim, dx_stride, es);
  if (dw_gate != nullptr) {
    m.write(dw_gate, hidden, dim, dw_gate_stride, gs);
    m.write(dw_up, hidden, dim, dw_up_stride, gs);
    m.write(dw_down, dim, hidden, dw_down_stride, gs);
  }
  const Matrix my = {dout, rows, dim, dout_stride}, mx = {x, rows, dim, x_stride}, mg = {w_gate, hidden, dim, gate_stride},
               mu = {w_up, hidden, dim, up_stride}, md = {w_down, dim, hidden, down_stride};
  const bool move = copies({my, mx, mg, mu, md});
  m.workspace(workspace, workspace_bytes, rsx_feed_forward_grad_workspace_size(rows, dim, hidden, type, move));
  const rsx_status_t st = m.status();
  if (st != RSX_SUCCESS || dim == 0 || (dx == nullptr && dw_gate == nullptr)) return st;
  return hip_status(launch_feed_forward_grad({my, mx, mg, mu, md, gate, up, dx, dw_gate, dw_up, dw_down, dx_stride, dw_gate_stride,
                                              dw_up_stride, dw_down_stride, rows, dim, hidden, activation, type, weight_grad_type,
                                              accumulate != 0, move, workspace},
                                             stream));
}

size_t rsx_linear_logprobs_workspace_size(size_t rows, size_t vocab, size_t dim, rsx_dtype_t type, int copies) {
  if (rows > kMaxSize || vocab > kMaxSize || dim >= kMaxWidth || float_size(type) == 0 || rows == 0 || vocab == 0) return 0;
  return linear_logprobs_ws({{nullptr, rows, dim, dim}, {nullptr, vocab, dim, dim}, nullptr, nullptr, nullptr, nullptr, nullptr, rows, vocab,
                             dim, 1.0f, type, 0, copies != 0, nullptr});
}

rsx_status_t rsx_linear_logprobs(const void* hidden, size_t hidden_stride, const void* weight,
                                 size_t weight_stride, rsx_dtype_t type, const void* tokens,
                                 rsx_dtype_t token_type, size_t rows, size_t vocab, size_t dim,
                                 float scale, float* logprob, float* entropy, float* lse,
                                 float* lse_rest, void* workspace, size_t workspace_bytes,
                                 hipStream_t stream) {
  const size_t es = float_size(type), is = token_size(token_type);
  if (es == 0 || is == 0) return RSX_ERR_INVALID_TYPE;
  if (rows > kMaxSize || vocab > kMaxSize || dim >= kMaxWidth || !tiles_fit(rows, vocab)) return RSX_ERR_UNSUPPORTED;
  if (vocab == 0) return RSX_ERR_INVALID_ARGUMENT;
  Areas m;
  m.read(hidden, rows, dim, hidden_stride, es);
  m.read(weight, vocab, dim, weight_stride, es);
  m.read_flat(tokens, rows, is);
  m.write_flat(logprob, rows, 4);
  if (entropy != nullptr) m.write_flat(entropy, rows, 4);
  m.write_flat(lse, rows, 4);
  if (lse_rest != nullptr) m.write_flat(lse_rest, rows, 4);
  const Matrix mh = {hidden, rows, dim, hidden_stride}, mw = {weight, vocab, dim, weight_stride};
  const bool move = copies({mh, mw});
  m.workspace(workspace, workspace_bytes, rsx_linear_logprobs_workspace_size(rows, vocab, dim, type, move));
  const rsx_status_t st = m.status();
  if (st != RSX_SUCCESS || rows == 0) return st;
  return hip_status(launch_linear_logprobs({mh, mw, tokens, logprob, entropy, lse, lse_rest, rows, vocab, dim, scale, type,
                                            token_type == RSX_INT64, move, workspace},
                                           stream));
}

size_t rsx_linear_logprobs_grad_workspace_size(size_t rows, size_t vocab, size_t dim, rsx_dtype_t type, int copies) {
  if (rows > kMaxSize || vocab > kMaxSize || dim >= kMaxWidth || float_size(type) == 0 || vocab == 0 || dim == 0) return 0;
  void* some = &copies;  // both gradients are wanted
  return linear_logprobs_grad_ws({{nullptr, rows, dim, dim}, {nullptr, vocab, dim, dim}, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                  some, some, 0, 0, rows, vocab, dim, 1.0f, type, type, 0, 0, copies != 0, nullptr});
}

rsx_status_t rsx_linear_logprobs_grad(const void* hidden, size_t hidden_stride, const void* weight,
                                      size_t weight_stride, rsx_dtype_t type, const void* tokens,
                                      rsx_dtype_t token_type, const float* lse,
                                      const float* lse_rest, const float* entropy,
                                      const float* dlogprob, const float* dentropy, void* dhidden,
                                      size_t dhidden_stride, void* dweight, size_t dweight_stride,
                                      rsx_dtype_t dweight_type, int accumulate, size_t rows,
                                      size_t vocab, size_t dim, float scale, void* workspace,
                                      size_t workspace_bytes, hipStream_t stream) {
  const size_t es = float_size(type), is = token_size(token_type), gs = grad_size(type, dweight_type);
  if (es == 0 || is == 0 || gs == 0) return RSX_ERR_INVALID_TYPE;
  if (rows > kMaxSize || vocab > kMaxSize || dim >= kMaxWidth || !tiles_fit(rows, vocab) || !tiles_fit(vocab, dim) ||
      !tiles_fit(rows, dim))
    return RSX_ERR_UNSUPPORTED;
  if (vocab == 0) return RSX_ERR_INVALID_ARGUMENT;
  Areas m;
  m.read(hidden, rows, dim, hidden_stride, es);
  m.read(weight, vocab, dim, weight_stride, es);
  m.read_flat(tokens, rows, is);
  m.read_flat(lse, rows, 4);
  if (lse_rest != nullptr) m.read_flat(lse_rest, rows, 4);
  m.read_flat(dlogprob, rows, 4);
  if (dentropy != nullptr) {
    m.read_flat(dentropy, rows, 4);
    m.read_flat(entropy, rows, 4);
  }
  if (dhidden != nullptr) m.write(dhidden, rows, dim, dhidden_stride, es);
  if (dweight != nullptr) m.write(dweight, vocab, dim, dweight_stride, gs);
  const Matrix mh = {hidden, rows, dim, hidden_stride}, mw = {weight, vocab, dim, weight_stride};
  const bool move = copies({mh, mw});
  m.workspace(workspace, workspace_bytes, rsx_linear_logprobs_grad_workspace_size(rows, vocab, dim, type, move));
  const rsx_status_t st = m.status();
  if (st != RSX_SUCCESS || dim == 0 || (dhidden == nullptr && dweight == nullptr)) return st;
  return hip_status(launch_linear_logprobs_grad({mh, mw, tokens, lse, lse_rest, entropy, dlogprob, dentropy, dhidden, dweight,
                                                 dhidden_stride, dweight_stride, rows, vocab, dim, scale, type, dweight_type,
                                                 token_type == RSX_INT64, accumulate != 0, move, workspace},
                                                stream));
}

size_t rsx_newton_schulz_workspace_size(size_t batch, size_t rows, size_t cols) {
  if (batch > 65535 || rows >= kMaxWidth || cols >= kMaxWidth || batch == 0 || rows == 0 || cols == 0) return 0;
  return newton_schulz_ws(batch, rows, cols);
}

rsx_status_t rsx_newton_schulz(const void* x, size_t x_stride, size_t x_matrix, void* out,
                               size_t out_stride, size_t out_matrix, size_t batch, size_t rows,
                               size_t cols, int steps, float a, float b, float c, float eps,
                               rsx_dtype_t type, void* workspace, size_t workspace_bytes,
                               hipStream_t stream) {
  const size_t es = float_size(type);
  if (es == 0) return RSX_ERR_INVALID_TYPE;
  if (batch > 65535 || rows >= kMaxWidth || cols >= kMaxWidth || x_matrix > kMaxSpan / es || out_matrix > kMaxSpan / es ||
      rows * cols > kMaxSpan / 4 / (batch ? batch : 1) || x_stride > kMaxSpan / es || out_stride > kMaxSpan / es)
    return RSX_ERR_UNSUPPORTED;
  // a matrix's span is in range before it is made of rows and stride: the product may wrap
  if (rows > 1 && (x_stride > kMaxSpan / es / rows || out_stride > kMaxSpan / es / rows)) return RSX_ERR_UNSUPPORTED;
  if (steps < 1 || !(eps >= 0.0f)) return RSX_ERR_INVALID_ARGUMENT;
  const bool some = rows != 0 && cols != 0;
  Areas m;
  if (some) {
    m.bad = x_stride < cols && x_stride != 0;
    m.bad = m.bad || out_stride < cols;
    // One matrix of a stack is one "row" here; of matrices side by side, one row of all of them.
    auto beside = [&](size_t stride, size_t each) { return each >= cols && each < (rows - 1) * stride + cols && (batch - 1) * each + cols <= stride; };
    if (batch > 1 && beside(x_stride, x_matrix)) m.read(x, rows, (batch - 1) * x_matrix + cols, x_stride, es);
    else m.read(x, batch, (rows - 1) * x_stride + cols, batch > 1 ? x_matrix : (rows - 1) * x_stride + cols, es);
    if (batch > 1 && beside(out_stride, out_matrix)) m.write(out, rows, (batch - 1) * out_matrix + cols, out_stride, es);
    else m.write(out, batch, (rows - 1) * out_stride + cols, batch > 1 ? out_matrix : (rows - 1) * out_stride + cols, es);
  }
  m.workspace(workspace, workspace_bytes, rsx_newton_schulz_workspace_size(batch, rows, cols));
  // x has been read before the first value of out is written, so they may be one
  const rsx_status_t st = m.status(x_stride == out_stride ? 1 : 0);
  if (st != RSX_SUCCESS || batch == 0 || !some) return st;
  return hip_status(launch_newton_schulz({x, out, batch, rows, cols, x_stride, out_stride, x_matrix, out_matrix, steps, type, a, b, c, eps,
                                          workspace},
                                         stream));
}

}  // extern "C"
