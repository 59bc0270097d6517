// C ABI of the training-step operators (include/tide.h): argument checks and
// workspace sizes of the 8-bit activation checkpoints, of the weight gradient
// that reads them, of the vocabulary loss, of layer norm, of the gated block and
// of the orthogonalised updates.  Host code only; the kernels are in the .hip
// files of those names.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <string>
#include <utility>
#include <vector>

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

// Rows of `bytes` each, `pitch` apart.
struct Area {
  const char* name;
  uintptr_t at;
  int64_t rows, bytes, pitch;

  bool empty() const { return at == 0 || rows == 0 || bytes == 0; }
  bool solid() const { return rows == 1 || pitch == bytes; }
  uintptr_t end() const { return at + uintptr_t((rows - 1) * pitch + bytes); }
};
Area matrix_area(const char* name, const void* p, int64_t rows, int64_t cols, int64_t stride, uintptr_t size) {
  return Area{name, reinterpret_cast<uintptr_t>(p), rows, cols * int64_t(size), stride * int64_t(size)};
}
Area vector_area(const char* name, const void* p, int64_t n, uintptr_t size) {
  return matrix_area(name, p, 1, n, n, size);
}

// Whether two areas share a byte.  Of two with gaps between their rows and different
// pitches only those that start together are known to.
bool overlap(const Area& a, const Area& b) {
  if (a.empty() || b.empty() || a.at >= b.end() || b.at >= a.end()) return false;
  if (a.at == b.at) return true;
  if (a.at > b.at) return overlap(b, a);
  const int64_t off = int64_t(b.at - a.at);
  if (b.solid()) {
    // a's last row that starts before b ends, from the first that ends behind b's start
    const int64_t first = off < a.bytes ? 0 : (off - a.bytes) / a.pitch + 1;
    return first < a.rows && a.at + uintptr_t(first * a.pitch) < b.end();
  }
  if (a.solid()) return true;  // b's first row starts in it
  if (a.pitch != b.pitch) return false;
  // b's rows start `in` bytes after the start of a's from row `row` on
  const int64_t row = off / a.pitch, in = off % a.pitch;
  return in < a.bytes || (in + b.bytes > a.pitch && row + 1 < a.rows);
}

// No output (the first `outs` of the areas) may share memory with another area.
tide_status check_apart(std::initializer_list<Area> areas, size_t outs) {
  const Area* all = areas.begin();
  for (size_t i = 0; i < outs; ++i)
    for (size_t j = i + 1; j < areas.size(); ++j)
      if (overlap(all[i], all[j])) return invalid(std::string(all[i].name) + " overlaps " + all[j].name);
  return TIDE_OK;
}

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

// Checks shared by layer norm and its gradients; *call is filled in.
tide_status layer_norm_call(const void* x, int32_t x_dtype, int64_t x_stride, const char* y_name, int32_t y_dtype,
                            int64_t y_stride, int64_t rows, int64_t cols, const void* weight, const void* bias,
                            int32_t affine_dtype, tide::LayerNormCall* call) {
  TIDE_TRY(check_dtype("x_dtype", x_dtype));
  TIDE_TRY(check_dtype((std::string(y_name) + "_dtype").c_str(), y_dtype));
  TIDE_TRY(check_dtype("affine_dtype", affine_dtype));
  TIDE_TRY(check_matrix("x", rows, cols, x_stride));
  TIDE_TRY(check_matrix(y_name, rows, cols, y_stride));
  if (cols < 1) return invalid("a row must hold at least one value");
  if (weight) TIDE_TRY(check_pointer("weight", weight, size_of(affine_dtype)));
  if (bias) TIDE_TRY(check_pointer("bias", bias, size_of(affine_dtype)));
  if (rows > 0) TIDE_TRY(check_pointer("x", x, size_of(x_dtype)));
  *call = tide::LayerNormCall{};
  call->x = x;
  call->x_ld = x_stride;
  call->x_f32 = x_dtype == TIDE_DTYPE_F32;
  call->y_f32 = y_dtype == TIDE_DTYPE_F32;
  call->y_ld = y_stride;
  call->weight = weight;
  call->bias = bias;
  call->affine_f32 = affine_dtype == TIDE_DTYPE_F32;
  call->rows = rows;
  call->cols = cols;
  return TIDE_OK;
}

// Checks shared by the gated block, its gradients and its workspace; *call is
// filled in.
tide_status gated_call(const uint16_t* x, int64_t x_stride, const uint16_t* w_gate, int64_t gate_stride,
                       const uint16_t* w_up, int64_t up_stride, int64_t tokens, int64_t hidden_size, int64_t ffn_size,
                       int32_t activation, const uint16_t* gates, int64_t gates_stride, bool grad,
                       tide::GatedCall* call) {
  if (activation != TIDE_ACT_SILU && activation != TIDE_ACT_GELU)
    return invalid("activation must be TIDE_ACT_SILU or TIDE_ACT_GELU");
  TIDE_TRY(check_matrix("x", tokens, hidden_size, x_stride));
  TIDE_TRY(check_matrix("w_gate", ffn_size, hidden_size, gate_stride));
  TIDE_TRY(check_matrix("w_up", ffn_size, hidden_size, up_stride));
  if (hidden_size < 1 || ffn_size < 1) return invalid("the hidden sizes must be at least 1");
  if (ffn_size > kMaxFeatures / 2) return tide::set_error(TIDE_ERR_RANGE, "an inner size above 2^21");
  // (the gradients' workspace holds dg and du, which are as large)
  if (gates || grad) TIDE_TRY(check_matrix("gates", tokens, 2 * ffn_size, gates ? gates_stride : 2 * ffn_size));
  if (tokens > 0) {
    TIDE_TRY(check_pointer("x", x, 2));
    TIDE_TRY(check_pointer("w_gate", w_gate, 2));
    TIDE_TRY(check_pointer("w_up", w_up, 2));
    if (gates) TIDE_TRY(check_pointer("gates", gates, 2));
  }
  *call = tide::GatedCall{};
  call->x = x;
  call->x_ld = x_stride;
  call->w_gate = w_gate;
  call->gate_ld = gate_stride;
  call->w_up = w_up;
  call->up_ld = up_stride;
  call->tokens = tokens;
  call->hidden = hidden_size;
  call->ffn = ffn_size;
  call->gelu = activation == TIDE_ACT_GELU;
  call->gates = const_cast<uint16_t*>(gates);
  call->gates_ld = gates_stride;
  call->grad = grad;
  return TIDE_OK;
}

tide_status check_orthogonalize(int32_t count, int64_t rows, int64_t cols, int64_t x_stride, int64_t out_stride,
                                int32_t steps) {
  if (count < 0) return invalid("a negative number of matrices");
  TIDE_TRY(check_matrix("x", rows, cols, x_stride));
  TIDE_TRY(check_matrix("out", rows, cols, out_stride));
  if (rows > kMaxFeatures) return tide::set_error(TIDE_ERR_RANGE, "more than 2^22 rows");
  const int64_t small = std::min(rows, cols);
  TIDE_TRY(check_matrix("the smaller side's square", small, small, small));
  if (steps < 1 || steps > 64) return invalid("steps must be in [1, 64]");
  return TIDE_OK;
}

// The largest magnitude of p(t) = a + b t + c t^2 over [0, top].
double largest_factor(double a, double b, double c, double top) {
  double most = std::max(std::abs(a), std::abs(a + top * (b + top * c)));
  const double at = c != 0 ? -b / (2 * c) : -1;
  if (at > 0 && at < top) most = std::max(most, std::abs(a + at * (b + at * c)));
  return most;
}

// Whether the steps keep every entry of their matrices in the range that fp16
// operands times 2^12 hold (16, with room for roundings): a matrix's entries are
// at most its largest singular value, which the polynomials bound.
tide_status check_coefficients(double a, double b, double c, int32_t steps) {
  if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return invalid("the coefficients must be finite");
  constexpr double kRoom = 14.0;
  double top = 1.0;  // the largest singular value there may be
  for (int32_t k = 0; k < steps; ++k) {
    const double t = top * top;
    bool fits = t <= kRoom && largest_factor(a, b, c, t) <= kRoom && largest_factor(0, b, c, t) <= kRoom;
    if (fits) {
      // s (a + b s^2 + c s^4) over [0, top]: its ends and where a + 3 b t + 5 c t^2 = 0
      auto value = [&](double u) { return u >= 0 && u <= t ? std::sqrt(u) * std::abs(a + u * (b + u * c)) : 0.0; };
      double next = value(t);
      const double d = 9 * b * b - 20 * a * c;
      if (c != 0 && d >= 0) {
        next = std::max(next, value((-3 * b + std::sqrt(d)) / (10 * c)));
        next = std::max(next, value((-3 * b - std::sqrt(d)) / (10 * c)));
      } else if (c == 0 && b != 0) {
        next = std::max(next, value(-a / (3 * b)));
      }
      top = next;
      fits = top * top <= kRoom;
    }
    if (!fits) return invalid("with these coefficients the steps leave the range that their fp16 operands hold");
  }
  return TIDE_OK;
}

// No output twice, and none that shares memory with another output or another
// matrix's input (its own has been read when it is written).
tide_status check_distinct(const void* const* x, uintptr_t x_size, int64_t x_stride, uint16_t* const* out,
                           int64_t out_stride, int32_t count, int64_t rows, int64_t cols) {
  auto place = [](const char* list, int32_t i) { return std::string(list) + "[" + std::to_string(i) + "]"; };
  auto area = [&](const void* p, int64_t stride, uintptr_t size) { return matrix_area("", p, rows, cols, stride, size); };
  std::vector<std::pair<uintptr_t, int32_t>> at(count);
  for (int32_t i = 0; i < count; ++i) at[i] = {reinterpret_cast<uintptr_t>(out[i]), i};
  std::sort(at.begin(), at.end());
  for (int32_t i = 1; i < count; ++i)
    if (at[i].first == at[i - 1].first)
      return invalid(place("out", at[i - 1].second) + " and " + place("out", at[i].second) + " are the same matrix");
  for (int32_t i = 0; i < count; ++i) {
    const Area a = area(out[at[i].second], out_stride, 2);
    for (int32_t j = i + 1; j < count && at[j].first < a.end(); ++j)
      if (overlap(a, area(out[at[j].second], out_stride, 2)))
        return invalid(place("out", at[i].second) + " overlaps " + place("out", at[j].second));
  }
  const uintptr_t span = area(out[0], out_stride, 2).end() - reinterpret_cast<uintptr_t>(out[0]);
  for (int32_t i = 0; i < count; ++i) {
    const Area a = area(x[i], x_stride, x_size);
    auto near = std::lower_bound(at.begin(), at.end(), std::make_pair(a.at > span ? a.at - span : 0, int32_t(0)));
    for (; near != at.end() && near->first < a.end(); ++near)
      if (near->second != i && overlap(a, area(out[near->second], out_stride, 2)))
        return invalid(place("out", near->second) + (near->first == a.at ? " is " : " overlaps ") + place("x", i));
  }
  return TIDE_OK;
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

tide_status tide_layer_norm(const void* x, int32_t x_dtype, int64_t x_stride, int64_t rows, int64_t cols,
                            const void* weight, const void* bias, int32_t affine_dtype, float eps, void* out,
                            int32_t out_dtype, int64_t out_stride, float* mean, float* rstd, void* stream) {
  return tide::guarded([&]() -> tide_status {
    tide::clear_error();
    tide::LayerNormCall c;
    TIDE_TRY(layer_norm_call(x, x_dtype, x_stride, "out", out_dtype, out_stride, rows, cols, weight, bias, affine_dtype,
                             &c));
    if (!(eps >= 0)) return invalid("eps must not be negative");
    if (rows == 0) return TIDE_OK;
    TIDE_TRY(check_pointer("out", out, size_of(out_dtype)));
    if (mean) TIDE_TRY(check_pointer("mean", mean, 4));
    if (rstd) TIDE_TRY(check_pointer("rstd", rstd, 4));
    c.eps = eps;
    c.out = out;
    c.mean = mean;
    c.rstd = rstd;
    if (mean != nullptr && mean == rstd) return invalid("mean and rstd are the same vector");
    const uintptr_t affine = size_of(affine_dtype);
    TIDE_TRY(check_apart({matrix_area("out", out, rows, cols, out_stride, size_of(out_dtype)), vector_area("mean", mean, rows, 4),
                          vector_area("rstd", rstd, rows, 4), matrix_area("x", x, rows, cols, x_stride, size_of(x_dtype)),
                          vector_area("weight", weight, cols, affine), vector_area("bias", bias, cols, affine)},
                         3));
    return hip_status(tide::launch_layer_norm(c, nullptr, stream), "layer norm launch");
  });
}

tide_status tide_layer_norm_grad_workspace(int32_t x_dtype, int32_t dout_dtype, int64_t rows, int64_t cols,
                                           int64_t* bytes) {
  return tide::guarded([&]() -> tide_status {
    tide::clear_error();
    if (bytes == nullptr) return invalid("bytes must not be NULL");
    tide::LayerNormCall c;
    const float here = 0.0f;  // stands for tensors
    TIDE_TRY(layer_norm_call(&here, x_dtype, cols, "dout", dout_dtype, cols, rows, cols, nullptr, nullptr, TIDE_DTYPE_F32,
                             &c));
    c.dweight = const_cast<float*>(&here);
    *bytes = tide::layer_norm_grad_bytes(c);
    return TIDE_OK;
  });
}

tide_status tide_layer_norm_grad(const void* dout, int32_t dout_dtype, int64_t dout_stride, const void* x,
                                 int32_t x_dtype, int64_t x_stride, int64_t rows, int64_t cols, const void* weight,
                                 int32_t affine_dtype, const float* mean, const float* rstd, void* dx,
                                 int64_t dx_stride, void* dweight, void* dbias, int32_t accumulate, void* workspace,
                                 int64_t workspace_bytes, void* stream) {
  return tide::guarded([&]() -> tide_status {
    tide::clear_error();
    tide::LayerNormCall c;
    TIDE_TRY(layer_norm_call(x, x_dtype, x_stride, "dout", dout_dtype, dout_stride, rows, cols, weight, nullptr,
                             affine_dtype, &c));
    if (accumulate != 0 && accumulate != 1) return invalid("accumulate must be 0 or 1");
    TIDE_TRY(check_matrix("dx", rows, cols, dx_stride));
    if (dweight) TIDE_TRY(check_pointer("dweight", dweight, size_of(affine_dtype)));
    if (dbias) TIDE_TRY(check_pointer("dbias", dbias, size_of(affine_dtype)));
    c.grad = true;
    c.dweight = dweight;
    c.dbias = dbias;
    c.accumulate = accumulate;
    if (rows > 0) {
      TIDE_TRY(check_pointer("dout", dout, size_of(dout_dtype)));
      TIDE_TRY(check_pointer("mean", mean, 4));
      TIDE_TRY(check_pointer("rstd", rstd, 4));
      TIDE_TRY(check_pointer("dx", dx, size_of(x_dtype)));
      TIDE_TRY(check_workspace(workspace, workspace_bytes, tide::layer_norm_grad_bytes(c)));
    }
    c.dout = dout;
    c.mean = const_cast<float*>(mean);
    c.rstd = const_cast<float*>(rstd);
    c.dx = dx;
    c.dx_ld = dx_stride;
    if (rows > 0 && dweight != nullptr && dweight == dbias) return invalid("dweight and dbias are the same vector");
    const uintptr_t affine = size_of(affine_dtype);
    if (rows > 0)
      TIDE_TRY(check_apart({matrix_area("dx", dx, rows, cols, dx_stride, size_of(x_dtype)), vector_area("dweight", dweight, cols, affine),
                            vector_area("dbias", dbias, cols, affine),
                            matrix_area("dout", dout, rows, cols, dout_stride, size_of(dout_dtype)),
                            matrix_area("x", x, rows, cols, x_stride, size_of(x_dtype)), vector_area("weight", weight, cols, affine),
                            vector_area("mean", mean, rows, 4), vector_area("rstd", rstd, rows, 4)},
                           3));
    return hip_status(tide::launch_layer_norm(c, workspace, stream), "layer norm gradient launch");
  });
}

tide_status tide_gated_block_workspace(const uint16_t* x, int64_t x_stride, const uint16_t* w_gate, int64_t gate_stride,
                                       const uint16_t* w_up, int64_t up_stride, int64_t tokens, int64_t hidden_size,
                                       int64_t ffn_size, int32_t gradients, const uint16_t* gates, int64_t* bytes) {
  return tide::guarded([&]() -> tide_status {
    tide::clear_error();
    if (bytes == nullptr) return invalid("bytes must not be NULL");
    if (gradients != 0 && gradients != 1) return invalid("gradients must be 0 or 1");
    tide::GatedCall c;
    TIDE_TRY(gated_call(x, x_stride, w_gate, gate_stride, w_up, up_stride, tokens, hidden_size, ffn_size, TIDE_ACT_SILU,
                        gates, 2 * ffn_size, gradients == 1, &c));
    if (gradients == 0) TIDE_TRY(check_matrix("out", tokens, ffn_size, ffn_size));
    *bytes = tide::gated_block_bytes(c);
    return TIDE_OK;
  });
}

tide_status tide_gated_block(const uint16_t* x, int64_t x_stride, const uint16_t* w_gate, int64_t gate_stride,
                             const uint16_t* w_up, int64_t up_stride, int64_t tokens, int64_t hidden_size,
                             int64_t ffn_size, int32_t activation, uint16_t* out, int64_t out_stride, uint16_t* gates,
                             int64_t gates_stride, void* workspace, int64_t workspace_bytes, void* stream) {
  return tide::guarded([&]() -> tide_status {
    tide::clear_error();
    tide::GatedCall c;
    TIDE_TRY(gated_call(x, x_stride, w_gate, gate_stride, w_up, up_stride, tokens, hidden_size, ffn_size, activation,
                        gates, gates_stride, false, &c));
    TIDE_TRY(check_matrix("out", tokens, ffn_size, out_stride));
    if (tokens == 0) return TIDE_OK;
    TIDE_TRY(check_pointer("out", out, 2));
    TIDE_TRY(check_workspace(workspace, workspace_bytes, tide::gated_block_bytes(c)));
    TIDE_TRY(check_apart({matrix_area("out", out, tokens, ffn_size, out_stride, 2),
                          matrix_area("gates", gates, tokens, 2 * ffn_size, gates_stride, 2),
                          matrix_area("x", x, tokens, hidden_size, x_stride, 2),
                          matrix_area("w_gate", w_gate, ffn_size, hidden_size, gate_stride, 2),
                          matrix_area("w_up", w_up, ffn_size, hidden_size, up_stride, 2)},
                         2));
    c.out = out;
    c.out_ld = out_stride;
    return hip_status(tide::launch_gated_block(c, workspace, stream), "gated block launch");
  });
}

tide_status tide_gated_block_grad(const uint16_t* dout, int64_t dout_stride, const uint16_t* x, int64_t x_stride,
                                  const uint16_t* w_gate, int64_t gate_stride, const uint16_t* w_up, int64_t up_stride,
                                  int64_t tokens, int64_t hidden_size, int64_t ffn_size, int32_t activation,
                                  const uint16_t* gates, int64_t gates_stride, uint16_t* dx, int64_t dx_stride,
                                  void* dw_gate, void* dw_up, int32_t dw_dtype, int32_t accumulate, void* workspace,
                                  int64_t workspace_bytes, void* stream) {
  return tide::guarded([&]() -> tide_status {
    tide::clear_error();
    TIDE_TRY(check_dtype("dw_dtype", dw_dtype));
    if (accumulate != 0 && accumulate != 1) return invalid("accumulate must be 0 or 1");
    tide::GatedCall c;
    TIDE_TRY(gated_call(x, x_stride, w_gate, gate_stride, w_up, up_stride, tokens, hidden_size, ffn_size, activation,
                        gates, gates_stride, true, &c));
    TIDE_TRY(check_matrix("dout", tokens, ffn_size, dout_stride));
    TIDE_TRY(check_matrix("dx", tokens, hidden_size, dx_stride));
    TIDE_TRY(check_pointer("dw_gate", dw_gate, size_of(dw_dtype)));
    TIDE_TRY(check_pointer("dw_up", dw_up, size_of(dw_dtype)));
    if (tokens > 0) {
      TIDE_TRY(check_pointer("dout", dout, 2));
      TIDE_TRY(check_pointer("dx", dx, 2));
      TIDE_TRY(check_workspace(workspace, workspace_bytes, tide::gated_block_bytes(c)));
    }
    c.dout = dout;
    c.dout_ld = dout_stride;
    c.dx = dx;
    c.dx_ld = dx_stride;
    c.dw_gate = dw_gate;
    c.dw_up = dw_up;
    c.dw_f32 = dw_dtype == TIDE_DTYPE_F32;
    c.accumulate = accumulate;
    if (tokens > 0 && dw_gate == dw_up) return invalid("dw_gate and dw_up are the same matrix");
    if (tokens > 0)
      TIDE_TRY(check_apart({matrix_area("dx", dx, tokens, hidden_size, dx_stride, 2),
                            matrix_area("dw_gate", dw_gate, ffn_size, hidden_size, hidden_size, size_of(dw_dtype)),
                            matrix_area("dw_up", dw_up, ffn_size, hidden_size, hidden_size, size_of(dw_dtype)),
                            matrix_area("dout", dout, tokens, ffn_size, dout_stride, 2),
                            matrix_area("x", x, tokens, hidden_size, x_stride, 2),
                            matrix_area("w_gate", w_gate, ffn_size, hidden_size, gate_stride, 2),
                            matrix_area("w_up", w_up, ffn_size, hidden_size, up_stride, 2),
                            matrix_area("gates", gates, tokens, 2 * ffn_size, gates_stride, 2)},
                           3));
    return hip_status(tide::launch_gated_block(c, workspace, stream), "gated block gradient launch");
  });
}

tide_status tide_orthogonalize_workspace(int32_t count, int64_t rows, int64_t cols, int32_t steps, int64_t* bytes) {
  return tide::guarded([&]() -> tide_status {
    tide::clear_error();
    if (bytes == nullptr) return invalid("bytes must not be NULL");
    TIDE_TRY(check_orthogonalize(count, rows, cols, cols, cols, steps));
    tide::OrthogonalCall c{};
    c.count = count;
    c.rows = rows;
    c.cols = cols;
    c.steps = steps;
    *bytes = tide::orthogonalize_bytes(c);
    return TIDE_OK;
  });
}

tide_status tide_orthogonalize(const void* const* x, int32_t x_dtype, int64_t x_stride, uint16_t* const* out,
                               int64_t out_stride, int32_t count, int64_t rows, int64_t cols, int32_t steps, float a,
                               float b, float c, float eps, void* workspace, int64_t workspace_bytes, void* stream) {
  return tide::guarded([&]() -> tide_status {
    tide::clear_error();
    TIDE_TRY(check_dtype("x_dtype", x_dtype));
    TIDE_TRY(check_orthogonalize(count, rows, cols, x_stride, out_stride, steps));
    TIDE_TRY(check_coefficients(a, b, c, steps));
    if (!(eps >= 0)) return invalid("eps must not be negative");
    if (count == 0 || rows == 0 || cols == 0) return TIDE_OK;
    if (x == nullptr || out == nullptr) return invalid("x and out must not be NULL");
    for (int32_t i = 0; i < count; ++i) {
      const std::string n = "[" + std::to_string(i) + "]";
      TIDE_TRY(check_pointer(("x" + n).c_str(), x[i], size_of(x_dtype)));
      TIDE_TRY(check_pointer(("out" + n).c_str(), out[i], 2));
    }
    TIDE_TRY(check_distinct(x, size_of(x_dtype), x_stride, out, out_stride, count, rows, cols));
    tide::OrthogonalCall o{};
    o.x = x;
    o.x_f32 = x_dtype == TIDE_DTYPE_F32;
    o.x_ld = x_stride;
    o.out = reinterpret_cast<void* const*>(out);
    o.out_ld = out_stride;
    o.count = count;
    o.rows = rows;
    o.cols = cols;
    o.steps = steps;
    o.a = a;
    o.b = b;
    o.c = c;
    o.eps = eps;
    TIDE_TRY(check_workspace(workspace, workspace_bytes, tide::orthogonalize_bytes(o)));
    return hip_status(tide::launch_orthogonalize(o, workspace, stream), "orthogonalized update launch");
  });
}

}  // extern "C"
