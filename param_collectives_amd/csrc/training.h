// Private types of the training-step operators: the 8-bit activation
// checkpoints (checkpoint.hip), the weight gradient that reads them
// (weight_grad.hip), the vocabulary loss (vocab_loss.hip), layer norm
// (layer_norm.hip), the gated block (gated_block.hip), orthogonalised updates
// (orthogonalize.hip) and their C ABI (training.cpp).
#pragma once

#include <cstdint>

namespace tide {

constexpr int64_t kPackBlock = 32;                      // values that share an exponent byte
constexpr int64_t kMaxFeatures = int64_t(1) << 22;      // features, hidden size, vocabulary, row pitch: 32-bit tile offsets
constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 1;  // tokens (rows)
constexpr int64_t kMaxLossTokens = int64_t(1) << 24;    // tokens of one vocabulary loss
// Elements of one matrix with its rows filled up to a multiple of 64, the widest
// pitch a copy of it may get: a launch counts its threads in 32 bits, and the
// element-wise kernels give a thread 8.
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

constexpr int kBK = 32;  // k per step of the matrix products

// How a product's tiles go to the resident workgroups (slots): whole rounds of
// tiles as they are, and the rest of them in splits of `per` steps of k each,
// whose fp32 partial sums are joined afterwards.  Items [0, full) are tiles,
// the others (tiles - full) * splits pieces.
struct Cut {
  uint32_t tiles, full, splits, per, items;
};

#ifdef __HIPCC__
#define TIDE_BOTH __host__ __device__
#else
#define TIDE_BOTH
#endif

// Workgroups of tiles of a side that the 256 CUs hold at once, by their LDS: two a
// CU of 128, one of 256 or, with as many loads on their way, of 64.
TIDE_BOTH inline int64_t tile_slots(int64_t side) { return side == 128 ? 512 : 256; }

// The rest is split so that its pieces fill a round, or not at all, whichever is
// estimated to end first: a round takes its steps (0.72 us each for a 256 x 256
// tile a CU, 0.45 us for two of 128 x 128) and about 11 more, the join about 5 us,
// and each piece 0.1 or 0.03 us for its partial sums.  Large tiles that are more
// than half a round, too many to be split in one, may fill two or three: the loss
// with gradients of 4096 x 2560 x 50000, whose dH has 160, takes 2.83 instead of
// 3.30 ms (and half a round, 96 tiles, 2% more in two rounds than in one).
TIDE_BOTH inline int64_t most_rounds(int64_t side) { return side == 256 ? 3 : 1; }

TIDE_BOTH inline Cut cut_tiles(int64_t all, int64_t all_steps, int64_t side) {
  const uint32_t tiles = uint32_t(all), steps = uint32_t(all_steps), slots = uint32_t(tile_slots(side));
  const uint32_t rest = tiles % slots, longest = steps / (side == 256 ? 32 : 16);  // splits, by the shortest piece
  Cut c{tiles, tiles, 1, steps, tiles};
  if (rest == 0) return c;
  // in 64ths of a step
  const uint32_t round = 11 * 64, join = (side == 256 ? 7 : 11) * 64, piece = side == 256 ? 9 : 4;
  uint32_t best = steps * 64 + round;
  for (uint32_t r = 1; r <= uint32_t(most_rounds(side)); ++r) {
    uint32_t splits = r * slots / rest;
    splits = splits < longest ? splits : longest;
    if (splits < 2) continue;
    const uint32_t per = (steps + splits - 1) / splits;
    splits = (steps + per - 1) / per;
    const uint32_t n = rest * splits, cost = (n + slots - 1) / slots * (per * 64 + round) + join + n * piece;
    if (cost >= best) continue;
    best = cost;
    c = Cut{tiles, tiles - rest, splits, per, tiles - rest + n};
    if (r == 1) break;
  }
  return c;
}

inline int64_t partial_bytes(const Cut& c, int64_t side) {
  return c.splits > 1 ? int64_t(c.items - c.full) * side * side * 4 : 0;
}

// About what a product of that cut takes, in us, for the choice of the tile.
inline double cut_cost(const Cut& c, int64_t steps, int64_t side) {
  const double step = side == 256 ? 0.72 : 0.45, tile = side == 256 ? 8.0 : 5.0;
  const int64_t slots = tile_slots(side), rounds = (c.full + slots - 1) / slots, more = (c.items - c.full + slots - 1) / slots;
  return double(rounds) * (double(steps) * step + tile) + double(more) * (double(c.per) * step + tile) +
         (c.splits > 1 ? 5.0 + 0.4e-6 * double(partial_bytes(c, side)) : 0.0);
}

// A product's tiles: the side (a small tile's is that of its rows) and the cut that
// are estimated to end first.  tiles(side) counts them.  Tiles of 64 are not split (a
// step of them takes `small_step` us, a tile about 4 more: fitted to the two sizes
// that follow) and read operands below 4 GiB.  (509 tokens, 2048 x 768, gated block's
// gradients: 43 us with them, 46 without; 512 x 2048 orthogonalized 147 and 187 us.)
struct Tiling {
  int64_t side = 256;
  Cut cut{};
};
template <typename F>
inline Tiling tiling_of(int64_t steps, int64_t operand_bytes, F tiles, double small_step = 0.15) {
  Tiling best;
  double least = 0;
  for (int64_t side : {256, 128, 64}) {
    Tiling t;
    t.side = side;
    const int64_t n = tiles(side);
    double cost;
    if (side == 64) {
      if (operand_bytes >= int64_t(1) << 31) break;
      t.cut = Cut{uint32_t(n), uint32_t(n), 1, uint32_t(steps), uint32_t(n)};
      cost = double((n + 255) / 256) * (double(steps) * small_step + 4.0);
    } else {
      t.cut = cut_tiles(n, steps, side);
      cost = cut_cost(t.cut, steps, side);
    }
    if (side == 256 || cost < least) {
      best = t;
      least = cost;
    }
  }
  return best;
}

// How a weight gradient is laid out, and its workspace: dy_bytes of aligned
// rows (when dY's are not), then partial_bytes.
struct WeightGradPlan {
  int64_t side;  // of its tiles
  Cut cut;
  int64_t tiles_m, tiles_n, dy_ld, dy_bytes, partial_bytes;
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

struct LayerNormCall {
  const void* x;
  int64_t x_ld;
  int32_t x_f32, y_f32;  // of x and dx, of out and dout
  const void* weight;    // may be null, as bias
  const void* bias;
  int32_t affine_f32;
  int64_t rows, cols;
  float eps;
  void* out;
  int64_t y_ld;  // of out or dout
  float* mean;   // may be null in the forward pass
  float* rstd;
  // the gradients
  bool grad;
  const void* dout;
  void* dx;
  int64_t dx_ld;
  void* dweight;  // may be null, as dbias
  void* dbias;
  int32_t accumulate;
};

struct GatedCall {
  const void* x;  // tokens x hidden bf16, rows x_ld apart
  int64_t x_ld;
  const void* w_gate;  // ffn x hidden bf16 each
  int64_t gate_ld;
  const void* w_up;
  int64_t up_ld;
  int64_t tokens, hidden, ffn;
  int32_t gelu;
  void* gates;  // tokens x 2 ffn bf16; written by the forward pass, read for the gradients; or null
  int64_t gates_ld;
  void* out;
  int64_t out_ld;
  // the gradients
  bool grad;
  const void* dout;
  int64_t dout_ld;
  void* dx;
  int64_t dx_ld;
  void* dw_gate;
  void* dw_up;
  int32_t dw_f32, accumulate;
};

struct OrthogonalCall {
  const void* const* x;  // `count` matrices of rows x cols, rows x_ld apart
  int32_t x_f32;
  int64_t x_ld;
  void* const* out;  // bf16
  int64_t out_ld;
  int32_t count;
  int64_t rows, cols;
  int32_t steps;
  float a, b, c, eps;
};

// Whether rows of `cols` bf16 elements, `ld` apart from p, all start and end on
// 16 bytes: the tiles then read them in place, 16 bytes at a time and never
// past a row's end.
bool rows_aligned(const void* p, int64_t ld, int64_t cols);
WeightGradPlan plan_weight_grad(int64_t tokens, int64_t outs, int64_t ins, bool aligned);

// Workgroups of a tile kernel with `items` tiles of side x side: as many as the
// 256 CUs hold at once (by their LDS), each taking one item after another.
inline unsigned resident_groups(int64_t items, int64_t side) {
  return unsigned(items < tile_slots(side) ? items : tile_slots(side));
}

// Launches; each returns the hipError_t as int.
int launch_pack(const PackCall& c, void* stream);
int launch_unpack(const PackCall& c, void* stream);
int launch_weight_grad(const WeightGradCall& c, void* workspace, void* stream);
int64_t vocab_loss_bytes(const VocabLossCall& c);  // its workspace
int launch_vocab_loss(const VocabLossCall& c, void* workspace, void* stream);
int64_t layer_norm_grad_bytes(const LayerNormCall& c);
int launch_layer_norm(const LayerNormCall& c, void* workspace, void* stream);
int launch_align_rows(const void* src, int64_t src_ld, int64_t rows, int64_t cols, void* dst, int64_t ld,
                      void* stream, int64_t out_rows = 0);
int64_t gated_block_bytes(const GatedCall& c);  // its workspace
int launch_gated_block(const GatedCall& c, void* workspace, void* stream);
int64_t orthogonalize_bytes(const OrthogonalCall& c);  // its workspace
int launch_orthogonalize(const OrthogonalCall& c, void* workspace, void* stream);

}  // namespace tide
