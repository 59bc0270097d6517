// Weight gradient of a linear layer from its activation checkpoint:
//   dW[o][i] = alpha sum_t dY[t][o] X[t][i]  (+ the old dW)
// with dY bf16 and X in the packed 8-bit form (checkpoint.hip), widened to bf16 on
// its way into LDS (gemm.h): the products are exact, so there is no rounding but
// the sums' and the result's.  The tokens are k, and both operands have their k
// as rows, so fragments are read from LDS with the transposing read.
//
// Bound by issue: the codes' widening and the staging take the slots between the
// matrix instructions, which are busy 49% of the cycles at 8192 x 4096 x 14336
// (and LDS for 31%).  Measured there, tokens x outs x ins, over two cards: 830 to
// 885 us from int8 into fp32 (1090 to 1160 TFLOP/s), 745 to 805 us from e4m3;
// 4096^3 from e4m3 105 to 116 us (1190 to 1300; a plain library product of bf16
// matrices reaches 1060 in this orientation).  Small ones are bound by latency:
// 509 x 768 x 2048 takes 10 us, 0.45 us a step of 32 tokens.
//
// Few tiles and many tokens are split along the tokens (training.h); the pieces'
// fp32 sums are joined in order, so results do not change from run to run.
#include "gemm.h"
#include "tide_internal.h"
#include "training.h"

namespace {

using namespace tide;

struct WeightGradArgs {
  Operand dy, x;
  int64_t outs, ins, tokens;
  Cut cut;
  float* partial;    // a slot of a tile for each piece of the cut
  void* dw;
  float alpha;
  int32_t f32, accumulate;
  uint32_t tiles_m, tiles_n;
};

template <Code CODE, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM* WN * 64, 2) void weight_grad_kernel(WeightGradArgs a) {
  using G = Gemm<Form::kCols, Form::kPacked, CODE, BM, BN, WM, WN>;
  __shared__ __align__(16) char lds0[G::kStage];
  __shared__ __align__(16) char lds1[G::kStage];
  __shared__ __align__(16) char lds2[G::kStage];
  __shared__ __align__(16) char lds3[G::kStage];
  // One tile a workgroup: with the next tile's loads under the epilogue, as in
  // the vocabulary loss, the codes' registers spill (measured 2-18% slower).
  const Piece p = piece_of<false>(a.cut, blockIdx.x, a.tokens);
  uint32_t tm, tn;
  tile_of(p.tile, a.tiles_m, a.tiles_n, 4, &tm, &tn);
  const int64_t m0 = int64_t(tm) * BM, n0 = int64_t(tn) * BN;
  G g;
  g.setup();
  g.open(a.dy, a.x, m0, n0, p.k_first, p.k_end, lds0, lds1, lds2);
  g.loop(lds0, lds1, lds2, lds3);
  if (p.slot >= 0)
    g.write(slot_target<BM>(a.partial, p.slot, a.outs - m0), 0, 0, lds3, [] {});
  else
    g.write(Target{a.dw, a.ins, a.outs, a.ins, nullptr, nullptr, a.alpha, a.f32, a.accumulate}, m0, n0, lds3,
            [] {});
}

template <int SIDE>
__global__ __launch_bounds__(256) void join_weight_grad_kernel(WeightGradArgs a) {
  constexpr uint32_t kParts = SIDE * SIDE / 2048;
  join_tile<SIDE>(a.partial, a.cut, a.tiles_m, a.tiles_n, blockIdx.x / kParts, blockIdx.x % kParts,
                  Target{a.dw, a.ins, a.outs, a.ins, nullptr, nullptr, a.alpha, a.f32, a.accumulate});
}

// Rows of any pitch and alignment -> rows of pitch `ld` (a multiple of 8)
// that start on 16 bytes, filled up with zeros (51658 x 3611: 126 us, 5.9 TB/s; one
// element at a time 215 us).
__global__ __launch_bounds__(256) void align_rows_kernel(const uint16_t* src, int64_t src_ld, int64_t rows,
                                                         int64_t cols, uint16_t* dst, int64_t ld) {
  const int64_t groups = ld / 8, i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= rows * groups) return;
  const int64_t r = i / groups, c = (i - r * groups) * 8;
  *reinterpret_cast<u32x4*>(dst + r * ld + c) = eight_of(src + r * src_ld + c, cols - c);
}

}  // namespace

namespace tide {

bool rows_aligned(const void* p, int64_t ld, int64_t cols) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0 && cols % 8 == 0;
}

int launch_align_rows(const void* src, int64_t src_ld, int64_t rows, int64_t cols, void* dst, int64_t ld,
                      void* stream) {
  const int64_t n = rows * (ld / 8);
  if (n == 0) return 0;
  hipLaunchKernelGGL(align_rows_kernel, dim3(unsigned((n + 255) / 256)), dim3(256), 0,
                     static_cast<hipStream_t>(stream), static_cast<const uint16_t*>(src), src_ld, rows, cols,
                     static_cast<uint16_t*>(dst), ld);
  return int(hipGetLastError());
}

WeightGradPlan plan_weight_grad(int64_t tokens, int64_t outs, int64_t ins, bool aligned) {
  const int64_t steps = (tokens + kBK - 1) / kBK;
  const int64_t big = (outs + 255) / 256 * ((ins + 255) / 256), small = (outs + 127) / 128 * ((ins + 127) / 128);
  const Cut cb = cut_tiles(big, steps, 256), cs = cut_tiles(small, steps, 128);
  WeightGradPlan p;
  p.side = cut_cost(cb, steps, 256) <= cut_cost(cs, steps, 128) ? 256 : 128;
  p.cut = p.side == 256 ? cb : cs;
  p.tiles_m = (outs + p.side - 1) / p.side;
  p.tiles_n = (ins + p.side - 1) / p.side;
  p.dy_ld = (outs + 63) / 64 * 64;
  p.dy_bytes = aligned ? 0 : (tokens * p.dy_ld * 2 + 255) / 256 * 256;
  p.partial_bytes = partial_bytes(p.cut, p.side);
  return p;
}

int launch_weight_grad(const WeightGradCall& c, void* workspace, void* stream) {
  const bool aligned = rows_aligned(c.dy, c.dy_ld, c.outs);
  const WeightGradPlan p = plan_weight_grad(c.tokens, c.outs, c.ins, aligned);
  char* ws = static_cast<char*>(workspace);
  hipStream_t st = static_cast<hipStream_t>(stream);
  WeightGradArgs a;
  a.dy = Operand{c.dy, nullptr, c.dy_ld, 0, c.outs};
  if (!aligned) {
    const int rc = launch_align_rows(c.dy, c.dy_ld, c.tokens, c.outs, ws, p.dy_ld, stream);
    if (rc != 0) return rc;
    a.dy.base = ws;
    a.dy.ld = p.dy_ld;
  }
  const int64_t blocks = (c.ins + 31) / 32;
  a.x = Operand{c.codes, c.scales, blocks * 32, blocks, c.ins};
  a.outs = c.outs;
  a.ins = c.ins;
  a.tokens = c.tokens;
  a.cut = p.cut;
  a.partial = reinterpret_cast<float*>(ws + p.dy_bytes);
  a.dw = c.dw;
  a.alpha = c.alpha;
  a.f32 = c.f32;
  a.accumulate = c.accumulate;
  a.tiles_m = uint32_t(p.tiles_m);
  a.tiles_n = uint32_t(p.tiles_n);
  const dim3 grid(p.cut.items);
  if (p.side == 256) {
    if (c.int8)
      hipLaunchKernelGGL((weight_grad_kernel<Code::kInt8, 256, 256, 2, 4>), grid, dim3(512), 0, st, a);
    else
      hipLaunchKernelGGL((weight_grad_kernel<Code::kE4m3, 256, 256, 2, 4>), grid, dim3(512), 0, st, a);
  } else {
    if (c.int8)
      hipLaunchKernelGGL((weight_grad_kernel<Code::kInt8, 128, 128, 2, 2>), grid, dim3(256), 0, st, a);
    else
      hipLaunchKernelGGL((weight_grad_kernel<Code::kE4m3, 128, 128, 2, 2>), grid, dim3(256), 0, st, a);
  }
  const int rc = int(hipGetLastError());
  if (rc != 0 || p.cut.splits == 1) return rc;
  const unsigned rest = p.cut.tiles - p.cut.full;
  if (p.side == 256)
    hipLaunchKernelGGL(join_weight_grad_kernel<256>, dim3(rest * 32), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(join_weight_grad_kernel<128>, dim3(rest * 8), dim3(256), 0, st, a);
  return int(hipGetLastError());
}

}  // namespace tide
