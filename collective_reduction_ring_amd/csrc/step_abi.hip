// C ABI of the training-step operators (declared in include/rsx.h): argument
// validation and aliasing rules.  Every check runs before the first HIP call.
#include "areas.h"

using namespace rsx;

extern "C" {

rsx_status_t rsx_embedding(const void* table, size_t table_stride, size_t vocab, size_t dim,
                           rsx_dtype_t table_type, const void* tokens, size_t ntokens,
                           rsx_dtype_t token_type, int64_t first, float scale, void* out,
                           size_t out_stride, rsx_dtype_t out_type, hipStream_t stream) {
  const size_t ts = float_size(table_type), os = float_size(out_type), is = token_size(token_type);
  if (ts == 0 || os == 0 || is == 0) return RSX_ERR_INVALID_TYPE;
  if (vocab > kMaxSize || dim > kMaxSize || ntokens > kMaxSize) return RSX_ERR_UNSUPPORTED;
  if (ids_wrap(first, vocab)) return RSX_ERR_INVALID_ARGUMENT;
  Areas m;
  m.read(table, vocab, dim, table_stride, ts);
  m.read_flat(tokens, ntokens, is);
  m.write(out, ntokens, dim, out_stride, os);
  const rsx_status_t st = m.status();
  if (st != RSX_SUCCESS || ntokens == 0 || dim == 0) return st;
  return hip_status(launch_embedding({table, tokens, out, table_stride, out_stride, ntokens, vocab, dim, first, scale,
                                      table_type, out_type, token_type == RSX_INT64},
                                     stream));
}

size_t rsx_embedding_grad_workspace_size(size_t ntokens, size_t vocab, size_t dim) {
  if (ntokens > kMaxSize || vocab > kMaxSize || dim > kMaxSize || ntokens == 0 || dim == 0) return 0;
  return embedding_grad_ws(vocab, dim, ntokens);
}

rsx_status_t rsx_embedding_grad(const void* dout, size_t dout_stride, rsx_dtype_t dout_type,
                                const void* tokens, size_t ntokens, rsx_dtype_t token_type,
                                int64_t first, float scale, void* grad, size_t grad_stride,
                                size_t vocab, size_t dim, rsx_dtype_t grad_type, int accumulate,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const size_t ds = float_size(dout_type), gs = float_size(grad_type), is = token_size(token_type);
  if (ds == 0 || gs == 0 || is == 0) return RSX_ERR_INVALID_TYPE;
  if (vocab > kMaxSize || dim > kMaxSize || ntokens > kMaxSize) return RSX_ERR_UNSUPPORTED;
  if (ids_wrap(first, vocab)) return RSX_ERR_INVALID_ARGUMENT;
  Areas m;
  m.write(grad, vocab, dim, grad_stride, gs);
  m.read(dout, ntokens, dim, dout_stride, ds);
  m.read_flat(tokens, ntokens, is);
  m.workspace(workspace, workspace_bytes, rsx_embedding_grad_workspace_size(ntokens, vocab, dim));
  const rsx_status_t st = m.status();
  if (st != RSX_SUCCESS || vocab == 0 || dim == 0) return st;
  return hip_status(launch_embedding_grad({dout, tokens, grad, dout_stride, grad_stride, ntokens, vocab, dim, first,
                                           scale, dout_type, grad_type, token_type == RSX_INT64, accumulate != 0,
                                           workspace},
                                          stream));
}

rsx_status_t rsx_layer_norm(const void* x, size_t x_stride, const void* weight, const void* bias,
                            void* y, size_t y_stride, float* mean, float* rstd, int8_t* codes,
                            uint8_t* scales, size_t rows, size_t dim, float eps, rsx_dtype_t type,
                            rsx_dtype_t weight_type, hipStream_t stream) {
  const size_t es = float_size(type), ws = float_size(weight_type);
  if (es == 0 || ws == 0 || (weight_type != type && weight_type != RSX_FLOAT32)) return RSX_ERR_INVALID_TYPE;
  if (rows > kMaxSize || dim > kMaxSize) return RSX_ERR_UNSUPPORTED;
  if ((codes == nullptr) != (scales == nullptr)) return RSX_ERR_INVALID_ARGUMENT;
  Areas m;
  m.write(y, rows, dim, y_stride, es);
  m.read(x, rows, dim, x_stride, es);
  if (weight != nullptr) m.read_flat(weight, dim, ws);
  if (bias != nullptr) m.read_flat(bias, dim, ws);
  if (mean != nullptr) m.write_flat(mean, rows, 4);
  if (rstd != nullptr) m.write_flat(rstd, rows, 4);
  if (codes != nullptr) {
    m.write(codes, rows, dim, dim, 1);
    m.write(scales, rows, ck_blocks(dim), ck_blocks(dim), 1);
  }
  const rsx_status_t st = m.status(1);
  if (st != RSX_SUCCESS || rows == 0 || dim == 0) return st;
  return hip_status(launch_layer_norm({x, weight, bias, y, mean, rstd, codes, scales, x_stride, y_stride, rows, dim, eps,
                                       type, weight_type},
                                      stream));
}

size_t rsx_layer_norm_grad_workspace_size(size_t rows, size_t dim) {
  if (rows > kMaxSize || dim > kMaxSize || rows == 0 || dim == 0) return 0;
  return layer_norm_grad_ws(rows, dim);
}

rsx_status_t rsx_layer_norm_grad(const void* dy, size_t dy_stride, const void* x, size_t x_stride,
                                 const int8_t* codes, const uint8_t* scales, const float* mean,
                                 const float* rstd, const void* weight, void* dx, size_t dx_stride,
                                 void* dweight, void* dbias, size_t rows, size_t dim,
                                 rsx_dtype_t type, rsx_dtype_t weight_type, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
  const size_t es = float_size(type), ws = float_size(weight_type);
  if (es == 0 || ws == 0 || (weight_type != type && weight_type != RSX_FLOAT32)) return RSX_ERR_INVALID_TYPE;
  if (rows > kMaxSize || dim > kMaxSize) return RSX_ERR_UNSUPPORTED;
  Areas m;
  m.write(dx, rows, dim, dx_stride, es);
  m.read(dy, rows, dim, dy_stride, es);
  if (x != nullptr) {
    if (codes != nullptr || scales != nullptr) return RSX_ERR_INVALID_ARGUMENT;
    m.read(x, rows, dim, x_stride, es);
  } else {
    m.read(codes, rows, dim, dim, 1);
    m.read(scales, rows, ck_blocks(dim), ck_blocks(dim), 1);
  }
  m.read_flat(mean, rows, 4);
  m.read_flat(rstd, rows, 4);
  if (weight != nullptr) m.read_flat(weight, dim, ws);
  if (dweight != nullptr) m.write_flat(dweight, dim, ws);
  if (dbias != nullptr) m.write_flat(dbias, dim, ws);
  m.workspace(workspace, workspace_bytes, rsx_layer_norm_grad_workspace_size(rows, dim));
  const rsx_status_t st = m.status(x != nullptr ? 2 : 1);
  if (st != RSX_SUCCESS || dim == 0) return st;
  return hip_status(launch_layer_norm_grad({dy, x, codes, scales, mean, rstd, weight, dx, dweight, dbias,
                                            static_cast<float*>(workspace), dy_stride, x_stride, dx_stride, rows, dim,
                                            type, weight_type},
                                           stream));
}

rsx_status_t rsx_checkpoint_pack(const void* x, size_t x_stride, int8_t* codes, uint8_t* scales,
                                 size_t rows, size_t dim, rsx_dtype_t type, hipStream_t stream) {
  const size_t es = float_size(type);
  if (es == 0) return RSX_ERR_INVALID_TYPE;
  if (rows > kMaxSize || dim > kMaxSize) return RSX_ERR_UNSUPPORTED;
  Areas m;
  m.read(x, rows, dim, x_stride, es);
  m.write(codes, rows, dim, dim, 1);
  m.write(scales, rows, ck_blocks(dim), ck_blocks(dim), 1);
  const rsx_status_t st = m.status();
  if (st != RSX_SUCCESS || rows == 0 || dim == 0) return st;
  return hip_status(launch_checkpoint_pack({x, nullptr, codes, scales, x_stride, rows, dim, type}, stream));
}

rsx_status_t rsx_checkpoint_unpack(const int8_t* codes, const uint8_t* scales, void* out,
                                   size_t out_stride, size_t rows, size_t dim, rsx_dtype_t type,
                                   hipStream_t stream) {
  const size_t es = float_size(type);
  if (es == 0) return RSX_ERR_INVALID_TYPE;
  if (rows > kMaxSize || dim > kMaxSize) return RSX_ERR_UNSUPPORTED;
  Areas m;
  m.read(codes, rows, dim, dim, 1);
  m.read(scales, rows, ck_blocks(dim), ck_blocks(dim), 1);
  m.write(out, rows, dim, out_stride, es);
  const rsx_status_t st = m.status();
  if (st != RSX_SUCCESS || rows == 0 || dim == 0) return st;
  return hip_status(launch_checkpoint_unpack(
      {nullptr, out, const_cast<int8_t*>(codes), const_cast<uint8_t*>(scales), out_stride, rows, dim, type}, stream));
}

size_t rsx_token_logprobs_workspace_size(size_t rows, size_t vocab, int top) {
  if (rows > kMaxSize || vocab > kMaxSize || top < 0 || top > RSX_TOP_MAX || rows == 0 || vocab == 0) return 0;
  return token_logprobs_ws(rows, vocab, static_cast<uint32_t>(top));
}

rsx_status_t rsx_token_logprobs(const void* logits, size_t stride, rsx_dtype_t type,
                                const void* tokens, rsx_dtype_t token_type, size_t rows,
                                size_t vocab, int top, float* logprob, float* entropy, float* lse,
                                float* top_logprob, int32_t* top_token, void* workspace,
                                size_t workspace_bytes, hipStream_t stream) {
  return rsx_token_logprobs_rest(logits, stride, type, tokens, token_type, rows, vocab, top, logprob, entropy, lse, nullptr,
                                 top_logprob, top_token, workspace, workspace_bytes, stream);
}

rsx_status_t rsx_token_logprobs_rest(const void* logits, size_t stride, rsx_dtype_t type,
                                     const void* tokens, rsx_dtype_t token_type, size_t rows,
                                     size_t vocab, int top, float* logprob, float* entropy,
                                     float* lse, float* lse_rest, float* top_logprob,
                                     int32_t* top_token, void* workspace, size_t workspace_bytes,
                                     hipStream_t stream) {
  const size_t es = float_size(type), is = token_size(token_type);
  if (es == 0 || is == 0) return RSX_ERR_INVALID_TYPE;
  if (rows > kMaxSize || vocab > kMaxSize) return RSX_ERR_UNSUPPORTED;
  if (vocab == 0 || top < 0 || top > RSX_TOP_MAX || static_cast<size_t>(top) > vocab) return RSX_ERR_INVALID_ARGUMENT;
  Areas m;
  m.read(logits, rows, vocab, stride, es);
  m.read_flat(tokens, rows, is);
  m.write_flat(logprob, rows, 4);
  if (entropy != nullptr) m.write_flat(entropy, rows, 4);
  m.write_flat(lse, rows, 4);
  if (lse_rest != nullptr) m.write_flat(lse_rest, rows, 4);
  if (top != 0) {
    m.write_flat(top_logprob, rows * static_cast<size_t>(top), 4);
    m.write_flat(top_token, rows * static_cast<size_t>(top), 4);
  }
  m.workspace(workspace, workspace_bytes, rsx_token_logprobs_workspace_size(rows, vocab, top));
  const rsx_status_t st = m.status();
  if (st != RSX_SUCCESS || rows == 0) return st;
  return hip_status(launch_token_logprobs({logits, tokens, logprob, entropy, lse, lse_rest, top_logprob, top_token,
                                           workspace, stride, rows, vocab, static_cast<uint32_t>(top), type,
                                           token_type == RSX_INT64},
                                          stream));
}

rsx_status_t rsx_token_logprobs_grad(const void* logits, size_t stride, rsx_dtype_t type,
                                     const void* tokens, rsx_dtype_t token_type, const float* lse,
                                     const float* entropy, const float* dlogprob,
                                     const float* dentropy, void* dlogits, size_t dlogits_stride,
                                     size_t rows, size_t vocab, hipStream_t stream) {
  return rsx_token_logprobs_grad_rest(logits, stride, type, tokens, token_type, lse, nullptr, entropy, dlogprob, dentropy,
                                      dlogits, dlogits_stride, rows, vocab, stream);
}

rsx_status_t rsx_token_logprobs_grad_rest(const void* logits, size_t stride, rsx_dtype_t type,
                                          const void* tokens, rsx_dtype_t token_type,
                                          const float* lse, const float* lse_rest,
                                          const float* entropy, const float* dlogprob,
                                          const float* dentropy, void* dlogits,
                                          size_t dlogits_stride, size_t rows, size_t vocab,
                                          hipStream_t stream) {
  const size_t es = float_size(type), is = token_size(token_type);
  if (es == 0 || is == 0) return RSX_ERR_INVALID_TYPE;
  if (rows > kMaxSize || vocab > kMaxSize) return RSX_ERR_UNSUPPORTED;
  if (vocab == 0) return RSX_ERR_INVALID_ARGUMENT;
  Areas m;
  m.write(dlogits, rows, vocab, dlogits_stride, es);
  m.read(logits, rows, vocab, stride, es);
  m.read_flat(tokens, rows, is);
  m.read_flat(lse, rows, 4);
  if (lse_rest != nullptr) m.read_flat(lse_rest, rows, 4);
  m.read_flat(dlogprob, rows, 4);
  if (dentropy != nullptr) {
    m.read_flat(dentropy, rows, 4);
    m.read_flat(entropy, rows, 4);
  }
  const rsx_status_t st = m.status(1);
  if (st != RSX_SUCCESS || rows == 0) return st;
  return hip_status(launch_token_logprobs_grad({logits, tokens, lse, lse_rest, entropy, dlogprob, dentropy, dlogits,
                                                stride, dlogits_stride, rows, vocab, type, token_type == RSX_INT64},
                                               stream));
}

}  // extern "C"
