// C ABI of the training-step operators (include/tide.h): argument checks and
// workspace sizes of the 8-bit activation checkpoints, of the weight gradient
// that reads them and of the vocabulary loss.  Host code only; the kernels are
// in checkpoint.hip, weight_grad.hip and vocab_loss.hip.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <string>

#include "tide_internal.h"
#include "training.h"

namespace {

using tide::kMaxElems;
using tide::kMaxFeatures;
using tide::kMaxTokens;

tide_status hip_status(int rc, const char* what) {
  if (rc == 0) return TIDE_OK;
  return tide::set_error(TIDE_ERR_HIP, std::string(what) + ": " + hipGetErrorString(hipError_t(rc)));
}

tide_status invalid(const std::string& why) { return tide::set_error(TIDE_ERR_INVALID, why); }

// A rows x cols matrix with rows `stride` elements apart.
tide_status check_matrix(const char* name, int64_t rows, int64_t cols, int64_t stride) {
  const std::string n(name);
  if (rows < 0 || cols < 0) return invalid(n + ": negative size");
  if (rows > kMaxTokens || cols > kMaxFeatures || stride > kMaxFeatures)
    return tide::set_error(TIDE_ERR_RANGE, n + ": more than 2^31 - 1 rows, or a row or row stride above 2^22 elements");
  if (stride < cols) return invalid(n + ": the row stride is smaller than the row");
  if (rows > 0 && (cols + 63) / 64 * 64 > kMaxElems / rows)
    return tide::set_error(TIDE_ERR_RANGE, n + ": more than 2^34 elements, with rows filled up to a multiple of 64");
  return TIDE_OK;
}

tide_status check_pointer(const char* name, const void* p, uintptr_t align) {
  if (p == nullptr) return invalid(std::string(name) + " must not be NULL");
  if (reinterpret_cast<uintptr_t>(p) & (align - 1))
    return tide::set_error(TIDE_ERR_ALIGN, std::string(name) + " is not " + std::to_string(align) + "-byte aligned");
  return TIDE_OK;
}

tide_status check_dtype(const char* name, int32_t dtype) {
  if (dtype != TIDE_DTYPE_BF16 && dtype != TIDE_DTYPE_F32)
    return invalid(std::string(name) + " must be TIDE_DTYPE_BF16 or TIDE_DTYPE_F32");
  return TIDE_OK;
}

tide_status check_format(int32_t format) {
  if (format != TIDE_CODE_E4M3 && format != TIDE_CODE_INT8)
    return invalid("format must be TIDE_CODE_E4M3 or TIDE_CODE_INT8");
  return TIDE_OK;
}

tide_status check_workspace(const void* workspace, int64_t given, int64_t need) {
  if (need == 0) return TIDE_OK;
  tide_status st = check_pointer("workspace", workspace, 256);
  if (st != TIDE_OK) return st;
  if (given < need)
    return invalid("the workspace holds " + std::to_string(given) + " bytes, the call needs " + std::to_string(need));
  return TIDE_OK;
}

#define TIDE_TRY(expr)                   \
  do {                                   \
    const tide_status st_ = (expr);      \
    if (st_ != TIDE_OK) return st_;      \
  } while (0)

uintptr_t size_of(int32_t dtype) { return dtype == TIDE_DTYPE_F32 ? 4 : 2; }

// Checks shared by the pack and the unpack; *call is filled in.
tide_status checkpoint_call(const char* name, const void* x, int32_t dtype, int64_t rows, int64_t cols,
                            int64_t row_stride, int32_t format, const void* codes, const void* scales,
                            tide::PackCall* call) {
  TIDE_TRY(check_dtype("dtype", dtype));
  TIDE_TRY(check_format(format));
  TIDE_TRY(check_matrix(name, rows, cols, row_stride));
  if (rows > 0 && cols > 0) {
    TIDE_TRY(check_pointer(name, x, size_of(dtype)));
    TIDE_TRY(check_pointer("codes", codes, 16));
    TIDE_TRY(check_pointer("scales", scales, 1));
  }
  *call = tide::PackCall{x,
                         dtype == TIDE_DTYPE_F32,
                         rows,
                         cols,
                         row_stride,
                         format == TIDE_CODE_INT8,
                         const_cast<void*>(codes),
                         const_cast<void*>(scales)};
  return TIDE_OK;
}

tide_status check_weight_grad(const void* dy, int64_t rows, int64_t outs, int64_t dy_stride, int64_t ins) {
  TIDE_TRY(check_matrix("dy", rows, outs, dy_stride));
  TIDE_TRY(check_matrix("codes", rows, ins, ins));
  TIDE_TRY(check_matrix("dw", outs, ins, ins));
  if (rows > 0 && outs > 0 && ins > 0) TIDE_TRY(check_pointer("dy", dy, 2));
  return TIDE_OK;
}

int64_t weight_grad_bytes(const void* dy, int64_t rows, int64_t outs, int64_t dy_stride, int64_t ins) {
  if (outs == 0 || ins == 0) return 0;
  const tide::WeightGradPlan p = tide::plan_weight_grad(rows, outs, ins, tide::rows_aligned(dy, dy_stride, outs));
  return p.dy_bytes + p.partial_bytes;
}

tide_status check_vocab_loss(const void* hidden, int64_t hidden_stride, const void* weight, int64_t weight_stride,
                             int64_t tokens, int64_t hidden_size, int64_t vocab) {
  TIDE_TRY(check_matrix("hidden", tokens, hidden_size, hidden_stride));
  TIDE_TRY(check_matrix("weight", vocab, hidden_size, weight_stride));
  if (vocab > kMaxFeatures || tokens > tide::kMaxLossTokens)
    return tide::set_error(TIDE_ERR_RANGE, "more than 2^24 tokens, or a vocabulary above 2^22");
  if (vocab < 1 || hidden_size < 1) return invalid("the vocabulary and the hidden size must be at least 1");
  if (tokens > 0) {
    TIDE_TRY(check_pointer("hidden", hidden, 2));
    TIDE_TRY(check_pointer("weight", weight, 2));
  }
  return TIDE_OK;
}

tide::VocabLossCall vocab_loss_call(const void* hidden, int64_t hidden_stride, const void* weight,
                                    int64_t weight_stride, int64_t tokens, int64_t hidden_size, int64_t vocab) {
  tide::VocabLossCall c{};
  c.h = hidden;
  c.h_ld = hidden_stride;
  c.w = weight;
  c.w_ld = weight_stride;
  c.tokens = tokens;
  c.hidden = hidden_size;
  c.vocab = vocab;
  return c;
}

}  // namespace

extern "C" {

tide_status tide_checkpoint_layout(int64_t cols, int64_t* code_cols, int64_t* scale_cols) {
  return tide::guarded([&]() -> tide_status {
    tide::clear_error();
    TIDE_TRY(check_matrix("checkpoint", 0, cols, cols));
    const int64_t blocks = (cols + tide::kPackBlock - 1) / tide::kPackBlock;
    if (code_cols) *code_cols = blocks * tide::kPackBlock;
    if (scale_cols) *scale_cols = blocks;
    return TIDE_OK;
  });
}

tide_status tide_checkpoint_pack(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t row_stride,
                                 int32_t format, void* codes, void* scales, void* stream) {
  return tide::guarded([&]() -> tide_status {
    tide::clear_error();
    tide::PackCall c;
    TIDE_TRY(checkpoint_call("x", x, dtype, rows, cols, row_stride, format, codes, scales, &c));
    if (rows == 0 || cols == 0) return TIDE_OK;
    return hip_status(tide::launch_pack(c, stream), "checkpoint_pack_kernel launch");
  });
}

tide_status tide_checkpoint_unpack(const void* codes, const void* scales, int32_t format, int64_t rows, int64_t cols,
                                   void* out, int32_t dtype, int64_t row_stride, void* stream) {
  return tide::guarded([&]() -> tide_status {
    tide::clear_error();
    tide::PackCall c;
    TIDE_TRY(checkpoint_call("out", out, dtype, rows, cols, row_stride, format, codes, scales, &c));
    if (rows == 0 || cols == 0) return TIDE_OK;
    return hip_status(tide::launch_unpack(c, stream), "checkpoint_unpack_kernel launch");
  });
}

tide_status tide_checkpoint_weight_grad_workspace(const uint16_t* dy, int64_t rows, int64_t out_features,
                                                  int64_t dy_stride, int64_t in_features, int64_t* bytes) {
  return tide::guarded([&]() -> tide_status {
    tide::clear_error();
    if (bytes == nullptr) return invalid("bytes must not be NULL");
    TIDE_TRY(check_weight_grad(dy, rows, out_features, dy_stride, in_features));
    *bytes = weight_grad_bytes(dy, rows, out_features, dy_stride, in_features);
    return TIDE_OK;
  });
}

tide_status tide_checkpoint_weight_grad(const uint16_t* dy, int64_t rows, int64_t out_features, int64_t dy_stride,
                                        const void* codes, const void* scales, int32_t format, int64_t in_features,
                                        void* dw, int32_t dw_dtype, float alpha, int32_t accumulate, void* workspace,
                                        int64_t workspace_bytes, void* stream) {
  return tide::guarded([&]() -> tide_status {
    tide::clear_error();
    TIDE_TRY(check_format(format));
    TIDE_TRY(check_dtype("dw_dtype", dw_dtype));
    if (accumulate != 0 && accumulate != 1) return invalid("accumulate must be 0 or 1");
    TIDE_TRY(check_weight_grad(dy, rows, out_features, dy_stride, in_features));
    if (out_features == 0 || in_features == 0) return TIDE_OK;
    TIDE_TRY(check_pointer("dw", dw, size_of(dw_dtype)));
    if (rows > 0) {
      TIDE_TRY(check_pointer("codes", codes, 16));
      TIDE_TRY(check_pointer("scales", scales, 1));
    }
    TIDE_TRY(check_workspace(workspace, workspace_bytes,
                             weight_grad_bytes(dy, rows, out_features, dy_stride, in_features)));
    tide::WeightGradCall c;
    c.dy = dy;
    c.dy_ld = dy_stride;
    c.codes = codes;
    c.scales = static_cast<const uint8_t*>(scales);
    c.tokens = rows;
    c.outs = out_features;
    c.ins = in_features;
    c.int8 = format == TIDE_CODE_INT8;
    c.f32 = dw_dtype == TIDE_DTYPE_F32;
    c.accumulate = accumulate;
    c.alpha = alpha;
    c.dw = dw;
    return hip_status(tide::launch_weight_grad(c, workspace, stream), "weight_grad_kernel launch");
  });
}

tide_status tide_vocab_loss_workspace(const uint16_t* hidden, int64_t hidden_stride, const uint16_t* weight,
                                      int64_t weight_stride, int64_t tokens, int64_t hidden_size, int64_t vocab,
                                      int32_t gradients, int32_t dweight_dtype, int64_t* bytes) {
  return tide::guarded([&]() -> tide_status {
    tide::clear_error();
    if (bytes == nullptr) return invalid("bytes must not be NULL");
    if (gradients != 0 && gradients != 1) return invalid("gradients must be 0 or 1");
    TIDE_TRY(check_dtype("dweight_dtype", dweight_dtype));
    TIDE_TRY(check_vocab_loss(hidden, hidden_stride, weight, weight_stride, tokens, hidden_size, vocab));
    tide::VocabLossCall c = vocab_loss_call(hidden, hidden_stride, weight, weight_stride, tokens, hidden_size, vocab);
    c.dhidden_wanted = gradients == 1;
    c.dw_f32 = dweight_dtype == TIDE_DTYPE_F32;
    *bytes = tide::vocab_loss_bytes(c);
    return TIDE_OK;
  });
}

tide_status tide_vocab_loss(const uint16_t* hidden, int64_t hidden_stride, const uint16_t* weight,
                            int64_t weight_stride, const int64_t* targets, int64_t tokens, int64_t hidden_size,
                            int64_t vocab, float* loss, float* lse, void* workspace, int64_t workspace_bytes,
                            void* stream) {
  return tide::guarded([&]() -> tide_status {
    tide::clear_error();
    TIDE_TRY(check_vocab_loss(hidden, hidden_stride, weight, weight_stride, tokens, hidden_size, vocab));
    tide::VocabLossCall c = vocab_loss_call(hidden, hidden_stride, weight, weight_stride, tokens, hidden_size, vocab);
    if (tokens == 0) return TIDE_OK;
    TIDE_TRY(check_pointer("targets", targets, 8));
    TIDE_TRY(check_pointer("loss", loss, 4));
    if (lse) TIDE_TRY(check_pointer("lse", lse, 4));
    TIDE_TRY(check_workspace(workspace, workspace_bytes, tide::vocab_loss_bytes(c)));
    c.targets = targets;
    c.loss = loss;
    c.lse = lse;
    return hip_status(tide::launch_vocab_loss(c, workspace, stream), "vocabulary loss launch");
  });
}

tide_status tide_vocab_loss_grad(const uint16_t* hidden, int64_t hidden_stride, const uint16_t* weight,
                                 int64_t weight_stride, const int64_t* targets, const float* grad_loss,
                                 int64_t tokens, int64_t hidden_size, int64_t vocab, float* loss, float* lse,
                                 uint16_t* dhidden, void* dweight, int32_t dweight_dtype, int32_t accumulate,
                                 void* workspace, int64_t workspace_bytes, void* stream) {
  return tide::guarded([&]() -> tide_status {
    tide::clear_error();
    TIDE_TRY(check_dtype("dweight_dtype", dweight_dtype));
    if (accumulate != 0 && accumulate != 1) return invalid("accumulate must be 0 or 1");
    TIDE_TRY(check_vocab_loss(hidden, hidden_stride, weight, weight_stride, tokens, hidden_size, vocab));
    TIDE_TRY(check_pointer("dweight", dweight, size_of(dweight_dtype)));
    tide::VocabLossCall c = vocab_loss_call(hidden, hidden_stride, weight, weight_stride, tokens, hidden_size, vocab);
    c.dhidden_wanted = true;
    c.dw = dweight;
    c.dw_f32 = dweight_dtype == TIDE_DTYPE_F32;
    c.accumulate = accumulate;
    if (tokens > 0) {
      TIDE_TRY(check_pointer("targets", targets, 8));
      TIDE_TRY(check_pointer("grad_loss", grad_loss, 4));
      TIDE_TRY(check_pointer("loss", loss, 4));
      if (lse) TIDE_TRY(check_pointer("lse", lse, 4));
      TIDE_TRY(check_pointer("dhidden", dhidden, 2));
      TIDE_TRY(check_workspace(workspace, workspace_bytes, tide::vocab_loss_bytes(c)));
    }
    c.targets = targets;
    c.grad_loss = grad_loss;
    c.loss = loss;
    c.lse = lse;
    c.dhidden = dhidden;
    return hip_status(tide::launch_vocab_loss(c, workspace, stream), "vocabulary loss launch");
  });
}

}  // extern "C"
