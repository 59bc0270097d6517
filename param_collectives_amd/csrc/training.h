// Private types of the training-step operators: the 8-bit activation
// checkpoints (checkpoint.hip), the weight gradient that reads them
// (weight_grad.hip), the vocabulary loss (vocab_loss.hip) and their C ABI
// (training.cpp).
#pragma once

#include <cstdint>

namespace tide {

constexpr int64_t kPackBlock = 32;                      // values that share an exponent byte
constexpr int64_t kMaxFeatures = int64_t(1) << 22;      // features, hidden size, vocabulary, row pitch: 32-bit tile offsets
constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 1;  // tokens (rows)
constexpr int64_t kMaxLossTokens = int64_t(1) << 24;    // tokens of one vocabulary loss
// Elements of one matrix: a launch counts its threads in 32 bits, and the
// element-wise kernels give a thread at least 4.
constexpr int64_t kMaxElems = int64_t(1) << 34;

struct PackCall {
  const void* x;  // pack: source; unpack: destination
  int32_t f32;
  int64_t rows, cols, ld;
  int32_t int8;
  void* codes;
  void* scales;
};

struct WeightGradCall {
  const void* dy;
  int64_t dy_ld;
  const void* codes;
  const uint8_t* scales;
  int64_t tokens, outs, ins;
  int32_t int8, f32, accumulate;
  float alpha;
  void* dw;
};

// How a weight gradient is cut into tiles and splits, and its workspace:
// dy_bytes of aligned rows (when dY's are not), then partial_bytes.
struct WeightGradPlan {
  bool big;  // 256 x 256 tiles
  int64_t tiles_m, tiles_n, splits, split_k, dy_ld, dy_bytes, partial_bytes;
};

struct VocabLossCall {
  const void* h;  // tokens x hidden bf16, rows h_ld apart
  int64_t h_ld;
  const void* w;  // vocab x hidden bf16, rows w_ld apart
  int64_t w_ld;
  const int64_t* targets;
  int64_t tokens, hidden, vocab;
  float* loss;
  float* lse;  // may be null
  // the gradients, where wanted
  bool dhidden_wanted;
  const float* grad_loss;
  void* dhidden;
  void* dw;
  int32_t dw_f32, accumulate;
};

// Whether rows of `cols` bf16 elements, `ld` apart from p, all start and end on
// 16 bytes: the tiles then read them in place, 16 bytes at a time and never
// past a row's end.
bool rows_aligned(const void* p, int64_t ld, int64_t cols);
WeightGradPlan plan_weight_grad(int64_t tokens, int64_t outs, int64_t ins, bool aligned);

// Workgroups of a tile kernel with `items` tiles of side x side: as many as the
// 256 CUs hold at once (by their LDS), each taking one item after another.
inline unsigned resident_groups(int64_t items, int64_t side) {
  const int64_t most = side == 256 ? 256 : side == 128 ? 512 : 1024;
  return unsigned(items < most ? items : most);
}

// Launches; each returns the hipError_t as int.
int launch_pack(const PackCall& c, void* stream);
int launch_unpack(const PackCall& c, void* stream);
int launch_weight_grad(const WeightGradCall& c, void* workspace, void* stream);
int64_t vocab_loss_bytes(const VocabLossCall& c);  // its workspace
int launch_vocab_loss(const VocabLossCall& c, void* workspace, void* stream);
int launch_align_rows(const void* src, int64_t src_ld, int64_t rows, int64_t cols, void* dst, int64_t ld,
                      void* stream);

}  // namespace tide
