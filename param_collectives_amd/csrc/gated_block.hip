// The gated feed-forward block on MI355X (gfx950): for tokens x (T x D) and
// weights Wg, Wu (F x D each)
//   g = x Wg^T,  u = x Wu^T,  h = act(g) u
// and, from dh,
//   dg = dh u act'(g),  du = dh act(g)
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x.
//
// Forward: a tile holds the products with the same columns of both weights (the
// B side of a tile is half Wg's rows, half Wu's), and a wave those that belong
// together, so that h leaves the accumulators in the one launch and g and u are
// written only where the backward pass is to have them.
//
// Backward: dg and du, side by side in rounded bf16, are the operand of the other
// products.  They come from kept g and u in a pass over them, or, where only x was
// kept, from the forward pass's product again, whose epilogue then reads dh: the
// unrounded sums go in, and nothing but dg and du is written.  dx is one product
// over 2 F values of k, the two weights stacked; dWg and dWu are one launch.
//
// Bound by the matrix cores and their power: 8192 tokens, 4096 x 14336 1.52 to 1.57
// ms (1240 TFLOP/s; the cores busy 71% of its cycles), the gradients from x 4.4 ms
// (1310 TFLOP/s), of 4096 tokens, 5120 x 13824 from kept gates 1.83 ms (1270).  Starting
// the next tile's loads before a tile's whole epilogue gains nothing (-1.7% to +0.5%),
// nor does leaving a tile's stores on their way behind them (-1.5% to 0).
//
// Up to 16 tokens, the weights' traffic is all that counts (few_gated_kernel).
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "gemm.h"
#include "training.h"

namespace {

using namespace tide;

// Both activations are z sigma(k(z)) (GELU in its tanh form: (1 + tanh y) / 2 =
// sigma(2 y)), with 1 - sigma(k) = sigma(k) exp(-k): neither cancels at either end.
// Where exp(-k) leaves fp32, sigma is 0.
constexpr float kLog2e = 1.44269504088896340736f, kRoot = 1.59576912160573071176f, kCube = 0.044715f;

__device__ __forceinline__ float act_value(float z, int32_t gelu) {
  const float k = gelu ? kRoot * z * (1.0f + kCube * (z * z)) : z;
  return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-k * kLog2e));
}

// The activation and its derivative.
struct Act {
  float value, slope;
};
__device__ __forceinline__ Act activate(float z, int32_t gelu) {
  const float z2 = z * z;
  const float k = gelu ? kRoot * z * (1.0f + kCube * z2) : z;
  const float e = __builtin_amdgcn_exp2f(-k * kLog2e), s = __builtin_amdgcn_rcpf(1.0f + e);
  float more = z * (s * (s * e));
  if (gelu) more *= kRoot * (1.0f + 3.0f * kCube * z2);
  // both ends, where the factors are 0 and infinite: sigma (1 - sigma) is 0
  if (s == 0.0f || e == 0.0f) more = 0.0f;
  return Act{z * s, s + more};
}

// What becomes of g and u.
struct Finish {
  int64_t rows, cols;  // T, F
  int32_t gelu;
  // forward
  uint16_t* out;
  int64_t out_ld;
  uint16_t* gates;  // g, then u at column F; or null
  int64_t gates_ld;
  // backward
  const uint16_t* dout;  // null: forward
  int64_t dout_ld;
  uint16_t* dgates;  // dg, then du at column `half`; rows 2 * half apart
  int64_t half;      // F filled up to a multiple of 32
};

// 8 values to p, of which `left` exist.
__device__ __forceinline__ void put_eight(uint16_t* p, u32x4 v, int64_t left) {
  if (left >= 8) {
    *reinterpret_cast<any_u32x4*>(p) = v;
    return;
  }
#pragma unroll
  for (int j = 0; j < 7; ++j)
    if (j < left) p[j] = uint16_t(v[j >> 1] >> (16 * (j & 1)));
}

// g, u -> h of 8 columns.
__device__ __forceinline__ u32x4 eight_out(int32_t gelu, f32x4v g0, f32x4v g1, f32x4v u0, f32x4v u1) {
  float h[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) h[j] = act_value(j < 4 ? g0[j & 3] : g1[j & 3], gelu) * (j < 4 ? u0[j & 3] : u1[j & 3]);
  return u32x4{two_bf16(h[0], h[1]), two_bf16(h[2], h[3]), two_bf16(h[4], h[5]), two_bf16(h[6], h[7])};
}
__device__ __forceinline__ u32x4 eight_bf16(f32x4v lo, f32x4v hi) {
  return u32x4{two_bf16(lo[0], lo[1]), two_bf16(lo[2], lo[3]), two_bf16(hi[0], hi[1]), two_bf16(hi[2], hi[3])};
}
// g, u, dh (bf16) -> dg and du of 8 columns, of which `left` exist: zeros for the
// rest, which fill up k.
__device__ __forceinline__ void eight_dgates(int32_t gelu, f32x4v g0, f32x4v g1, f32x4v u0, f32x4v u1, u32x4 d,
                                             int64_t left, u32x4* dg, u32x4* du) {
  float a[8], b[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float dh = (j & 1) ? high_bf16(d[j >> 1]) : low_bf16(d[j >> 1]);
    const Act act = activate(j < 4 ? g0[j & 3] : g1[j & 3], gelu);
    a[j] = dh * (j < 4 ? u0[j & 3] : u1[j & 3]) * act.slope;
    b[j] = dh * act.value;
  }
  if (left < 8) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j >= left) a[j] = b[j] = 0.0f;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    (*dg)[j] = two_bf16(a[2 * j], a[2 * j + 1]);
    (*du)[j] = two_bf16(b[2 * j], b[2 * j + 1]);
  }
}

// Columns n .. n + 7 of row m, which exists.
__device__ __forceinline__ void finish(const Finish& f, int64_t m, int64_t n, f32x4v g0, f32x4v g1, f32x4v u0,
                                       f32x4v u1) {
  const int64_t left = f.cols - n;
  if (f.dout == nullptr) {
    if (left <= 0) return;
    put_eight(f.out + m * f.out_ld + n, eight_out(f.gelu, g0, g1, u0, u1), left);
    if (f.gates == nullptr) return;
    put_eight(f.gates + m * f.gates_ld + n, eight_bf16(g0, g1), left);
    put_eight(f.gates + m * f.gates_ld + f.cols + n, eight_bf16(u0, u1), left);
    return;
  }
  if (n >= f.half) return;
  u32x4 dg, du;
  eight_dgates(f.gelu, g0, g1, u0, u1, eight_of(f.dout + m * f.dout_ld + n, left), left, &dg, &du);
  uint16_t* p = f.dgates + m * 2 * f.half + n;
  *reinterpret_cast<u32x4*>(p) = dg;
  *reinterpret_cast<u32x4*>(p + f.half) = du;
}

// ------------------------------------------------------------ g and u

struct GatedArgs {
  Operand x, w;
  int64_t depth;
  Cut cut;
  float* partial;
  uint32_t tiles_m, tiles_n;
  uint32_t* queue;  // null: every workgroup has its one item
  Finish f;
};

// A lane's columns of both products lie side by side in its accumulators (Form::kPair):
// the epilogue takes no LDS, its stores are 16 bytes a lane, 64 a row, from one
// shared address and the lane's offset, and dh's rows are asked for before the
// first is used.  GRAD: dg and du instead of h.  WHOLE: k is whole steps (tiles of 64
// rows take any).
template <bool GRAD, bool WHOLE, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM* WN * 64, BM == 64 ? 1 : 2) void gated_kernel(GatedArgs a) {
  using G = std::conditional_t<BM == 64, DeepGemm<Form::kRows, Form::kPair, BM, BN, WM, WN, false, 2>,
                               Gemm<Form::kRows, Form::kPair, Code::kE4m3, BM, BN, WM, WN, false, WHOLE>>;
  __shared__ __align__(16) char lds0[G::kStage];
  __shared__ __align__(16) char lds1[G::kStage];
  __shared__ __align__(16) char lds2[G::kStage];
  __shared__ __align__(16) char lds3[G::kStage];
  __shared__ uint32_t turn;
  static_assert(G::kFN == 4 && BN / WN == 64, "8 columns a lane");
  Queue q;
  uint32_t item = blockIdx.x;
  if (a.queue) item = first_item(q, a.queue, a.cut.items, &turn);
  if (item == kNoItem) return;
  int64_t m0, n0, slot;
  G g;
  g.setup();
  auto open = [&](uint32_t item) {
    const Piece p = piece_of<false>(a.cut, item, a.depth);
    uint32_t tm, tn;
    tile_of(p.tile, a.tiles_m, a.tiles_n, 4, &tm, &tn);
    m0 = int64_t(tm) * BM;
    n0 = int64_t(tn) * (BN / 2);
    slot = p.slot;
    g.open(a.x, a.w, m0, n0, p.k_first, p.k_end, lds0, lds1, lds2, lds3);
  };
  const int32_t gelu = a.f.gelu;
  open(item);
  while (item != kNoItem) {
    g.loop(lds0, lds1, lds2, lds3);
    const uint32_t k = a.queue ? q.ask() : 0;
    const int64_t s1 = slot;
    // this wave's part of the tile: rows from m1, 16 at a time, columns from n1; this lane's row and columns of it
    const int64_t m1 = m0 + g.wm * (BM / WM), n1 = n0 + g.wn * 32;
    g.renew_lane();
    const uint32_t row = g.lane & 15, col = uint32_t(g.lane >> 4) * 8;
    const int64_t left = a.f.cols - n1 - col, rows = a.f.rows - m1 - row;
    u32x4 d[GRAD ? G::kFM : 1];
    if constexpr (GRAD) {
      if (s1 < 0) {
        const uint16_t* from = a.f.dout + m1 * a.f.dout_ld + n1;
        uint32_t at = row * uint32_t(a.f.dout_ld) + col;
#pragma unroll
        for (int i = 0; i < G::kFM; ++i) {
          d[i] = u32x4{0, 0, 0, 0};
          if (16 * i < rows) d[i] = eight_of(from + at, left);
          at += 16 * uint32_t(a.f.dout_ld);
        }
      }
    }
    // the rows come in order, and the places go on with them
    const uint32_t ld = GRAD ? uint32_t(2 * a.f.half) : uint32_t(a.f.out_ld);
    uint16_t* const to = GRAD ? a.f.dgates + m1 * 2 * a.f.half + n1 : a.f.out + m1 * a.f.out_ld + n1;
    uint16_t* const kept = a.f.gates + m1 * a.f.gates_ld + n1;
    uint32_t at = row * ld + col, kept_at = row * uint32_t(a.f.gates_ld) + col;
#pragma unroll
    for (int i = 0; i < G::kFM; ++i) {
      const f32x4v g0 = g.acc[i][0], g1 = g.acc[i][1], u0 = g.acc[i][2], u1 = g.acc[i][3];
      if (s1 >= 0) {
        float* p = a.partial + s1 * BM * BN + (g.wm * (BM / WM) + 16 * i + row) * BN + g.wn * 32 + col;
        *reinterpret_cast<f32x4v*>(p) = g0;
        *reinterpret_cast<f32x4v*>(p + 4) = g1;
        *reinterpret_cast<f32x4v*>(p + BN / 2) = u0;
        *reinterpret_cast<f32x4v*>(p + BN / 2 + 4) = u1;
      } else if constexpr (GRAD) {
        if (16 * i < rows && col + n1 < a.f.half) {
          u32x4 dg, du;
          eight_dgates(gelu, g0, g1, u0, u1, d[i], left, &dg, &du);
          *reinterpret_cast<u32x4*>(to + at) = dg;
          *reinterpret_cast<u32x4*>(to + a.f.half + at) = du;
        }
      } else if (16 * i < rows && left > 0) {
        put_eight(to + at, eight_out(gelu, g0, g1, u0, u1), left);
        if (a.f.gates) {
          put_eight(kept + kept_at, eight_bf16(g0, g1), left);
          put_eight(kept + a.f.cols + kept_at, eight_bf16(u0, u1), left);
        }
      }
      at += 16 * ld;
      kept_at += 16 * uint32_t(a.f.gates_ld);
      if (i == G::kFM / 2 - 1) {
        item = a.queue ? next_item(q, k, &turn) : kNoItem;
        if (item != kNoItem) open(item);
      }
    }
  }
}

// Joins the partial sums of g and u and finishes them, 8 columns a thread.
template <int SIDE>
__global__ __launch_bounds__(256) void join_gated_kernel(GatedArgs a) {
  constexpr uint32_t kParts = SIDE * SIDE / 2 / 2048;
  const uint32_t r = blockIdx.x / kParts, i = blockIdx.x % kParts * 256 + threadIdx.x;
  const uint32_t row = i / (SIDE / 16), col = i % (SIDE / 16) * 8;
  uint32_t tm, tn;
  tile_of(a.cut.full + r, a.tiles_m, a.tiles_n, 4, &tm, &tn);
  const int64_t m = int64_t(tm) * SIDE + row, n = int64_t(tn) * (SIDE / 2) + col;
  if (m >= a.f.rows || n >= a.f.half) return;
  f32x4v g0, g1, u0, u1;
  join_eight<SIDE>(a.partial, a.cut, r, row, col, &g0, &g1);
  join_eight<SIDE>(a.partial, a.cut, r, row, SIDE / 2 + col, &u0, &u1);
  finish(a.f, m, n, g0, g1, u0, u1);
}

// dg and du from kept g and u.
__global__ __launch_bounds__(256) void kept_gates_kernel(const uint16_t* gates, int64_t ld, Finish f) {
  const int64_t groups = f.half / 8, i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t m = i / groups, n = (i - m * groups) * 8;
  if (m >= f.rows) return;
  const uint16_t* p = gates + m * ld + n;
  const u32x4 g = eight_of(p, f.cols - n), u = eight_of(p + f.cols, f.cols - n);
  finish(f, m, n, f32x4v{low_bf16(g[0]), high_bf16(g[0]), low_bf16(g[1]), high_bf16(g[1])},
         f32x4v{low_bf16(g[2]), high_bf16(g[2]), low_bf16(g[3]), high_bf16(g[3])},
         f32x4v{low_bf16(u[0]), high_bf16(u[0]), low_bf16(u[1]), high_bf16(u[1])},
         f32x4v{low_bf16(u[2]), high_bf16(u[2]), low_bf16(u[3]), high_bf16(u[3])});
}

// Up to 16 tokens: a workgroup has 16 columns, and its waves split k; each reads
// its part of the 16 rows of both weights straight into registers, and the
// tokens' states, which every workgroup reads, from the caches.  Rows may start
// anywhere: nothing is copied first.  Bound by the bytes on their way: 1 token, 4096 x
// 14336 43 us (5.4 TB/s), 16 tokens 51, 1 token, 8192 x 28672 156 us (6.0 TB/s).  (With
// 4 waves 48, 53.5 and 155 us, with 16 50, 59 and 176; loads of 8 steps at once
// spill, 110 us.)  Two sets of loads take turns, and each workgroup starts at a place
// of its own in its rows, so that they do not ask the same channels at one time.
constexpr int kFewWaves = 8;
__global__ __launch_bounds__(kFewWaves * 64, 4) void few_gated_kernel(const uint16_t* x, int64_t x_ld,
                                                                      const uint16_t* gate, int64_t gate_ld,
                                                                      const uint16_t* up, int64_t up_ld, int64_t depth,
                                                                      Finish f) {
  constexpr int kDeep = 4;  // steps whose loads go out together
  __shared__ f32x4v part[2][kFewWaves][64];
  const int lane = threadIdx.x & 63, wave = wave_index(), r = lane & 15, g = lane >> 4;
  const int64_t n0 = int64_t(blockIdx.x) * 16;
  // rows past the end read the last one: their results are dropped
  const int64_t v = n0 + r < f.cols ? n0 + r : f.cols - 1, t = r < f.rows ? r : f.rows - 1;
  const uint16_t* wg = gate + v * gate_ld + 8 * g;
  const uint16_t* wu = up + v * up_ld + 8 * g;
  const uint16_t* xt = x + t * x_ld + 8 * g;
  typedef bf16x8 any_bf16x8 __attribute__((aligned(2)));
  auto load = [](const uint16_t* p) -> bf16x8 { return *(const TIDE_GLOBAL any_bf16x8*)p; };
  const int64_t whole = depth / 32, per = (whole + kFewWaves - 1) / kFewWaves;
  int64_t s = wave * per;
  const int64_t end = s + per < whole ? s + per : whole;
  f32x4v ag = f32x4v{0.f, 0.f, 0.f, 0.f}, au = ag;
  struct Steps {
    bf16x8 g[kDeep], u[kDeep], x[kDeep];
  } even, odd;
  auto fetch = [&](Steps& to, int64_t at) {
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      to.g[i] = load(wg + (at + i) * 32);
      to.u[i] = load(wu + (at + i) * 32);
      to.x[i] = load(xt + (at + i) * 32);
    }
    __builtin_amdgcn_sched_barrier(0);  // all of them on their way before the first product
  };
  auto multiply = [&](const Steps& w) {
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      ag = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.g[i], w.x[i], ag, 0, 0, 0);
      au = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.u[i], w.x[i], au, 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  const int64_t blocks = end > s ? (end - s) / kDeep : 0;
  if (blocks > 0) {
    int64_t b = blockIdx.x % blocks;
    auto next = [&] {
      const int64_t at = s + b * kDeep;
      b = b + 1 == blocks ? 0 : b + 1;
      return at;
    };
    fetch(even, next());
    int64_t n = 1;
    for (; n + 2 <= blocks; n += 2) {
      fetch(odd, next());
      multiply(even);
      fetch(even, next());
      multiply(odd);
    }
    if (n < blocks) {
      fetch(odd, next());
      multiply(even);
      multiply(odd);
    } else {
      multiply(even);
    }
    s += blocks * kDeep;
  }
  for (; s < end; ++s) {
    const bf16x8 bg = load(wg + s * 32), bu = load(wu + s * 32), bx = load(xt + s * 32);
    ag = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bg, bx, ag, 0, 0, 0);
    au = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bu, bx, au, 0, 0, 0);
  }
  if (wave == kFewWaves - 1 && whole * 32 < depth) {
    const int64_t k = whole * 32, left = depth - k - 8 * g;
    auto some = [&](const uint16_t* p) {
      const u32x4 b = eight_of(p + k, left);
      bf16x8 o;
      __builtin_memcpy(&o, &b, 16);
      return o;
    };
    const bf16x8 bg = some(wg), bu = some(wu), bx = some(xt);
    ag = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bg, bx, ag, 0, 0, 0);
    au = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bu, bx, au, 0, 0, 0);
  }
  part[0][wave][lane] = ag;
  part[1][wave][lane] = au;
  __syncthreads();
  // a lane holds of token r the columns n0 + 4 g + 0..3; 32 threads take 8 columns each
  if (threadIdx.x >= 32) return;
  const int token = threadIdx.x & 15, pair = threadIdx.x >> 4;
  if (token >= f.rows) return;
  f32x4v sum[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sum[i] = f32x4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kFewWaves; ++k) sum[i] = add4(sum[i], part[i >> 1][k][token + 16 * (2 * pair + (i & 1))]);
  }
  finish(f, token, n0 + 8 * pair, sum[0], sum[1], sum[2], sum[3]);
}

// ------------------------------------------------------------ dx, dWg and dWu

// One or two products of the same sizes: the second's tiles follow the first's,
// with its own A, `shift` bytes on, and its own target.
struct GradArgs {
  Operand a, b;
  int64_t depth;
  int64_t shift;
  Target to[2];
  Cut cut;
  float* partial;
  uint32_t tiles_m, tiles_n;  // of one product
  int32_t products;
  uint32_t* queue;  // null: every workgroup has its one item
};

__device__ __forceinline__ uint32_t grad_tile(const GradArgs& a, uint32_t tile, uint32_t* tm, uint32_t* tn) {
  tile_of(tile, a.tiles_m * a.products, a.tiles_n, 4, tm, tn);
  const uint32_t second = *tm >= a.tiles_m ? 1 : 0;
  *tm -= second * a.tiles_m;
  return second;
}

template <Form FA, Form FB, int SIDE, int WM, int WN>
__global__ __launch_bounds__(WM* WN * 64, SIDE == 64 ? 1 : 2) void gated_grad_kernel(GradArgs a) {
  using G = std::conditional_t<SIDE == 64, DeepGemm<FA, FB, SIDE, SIDE, WM, WN, false, 4>,
                               Gemm<FA, FB, Code::kE4m3, SIDE, SIDE, WM, WN, false, FB == Form::kStack>>;
  __shared__ __align__(16) char lds0[G::kStage];
  __shared__ __align__(16) char lds1[G::kStage];
  __shared__ __align__(16) char lds2[G::kStage];
  __shared__ __align__(16) char lds3[G::kStage];
  __shared__ __align__(16) char own[own_rows<G, SIDE>()];
  __shared__ uint32_t turn;
  Queue q;
  uint32_t item = blockIdx.x;
  if (a.queue) item = first_item(q, a.queue, a.cut.items, &turn);
  if (item == kNoItem) return;
  int64_t m0, n0, slot;
  uint32_t second;
  G g;
  g.setup();
  auto open = [&](uint32_t item) {
    const Piece p = piece_of<FB == Form::kStack>(a.cut, item, a.depth);
    uint32_t tm, tn;
    second = grad_tile(a, p.tile, &tm, &tn);
    m0 = int64_t(tm) * SIDE;
    n0 = int64_t(tn) * SIDE;
    slot = p.slot;
    Operand left = a.a;
    left.base = static_cast<const char*>(left.base) + second * a.shift;
    g.open(left, a.b, m0, n0, p.k_first, p.k_end, lds0, lds1, lds2, lds3);
  };
  open(item);
  while (item != kNoItem) {
    g.loop(lds0, lds1, lds2, lds3);
    const uint32_t k = a.queue ? q.ask() : 0;
    const Target t = slot >= 0 ? slot_target<SIDE>(a.partial, slot, a.to[0].rows - m0) : second ? a.to[1] : a.to[0];
    const int64_t m1 = slot >= 0 ? 0 : m0, n1 = slot >= 0 ? 0 : n0;
    g.write_rows(t, m1, n1, SIDE == 64 ? own : lds3, [&] {
      item = a.queue ? next_item(q, k, &turn) : kNoItem;
      if (item != kNoItem) open(item);
    });
  }
}

template <int SIDE>
__global__ __launch_bounds__(256) void join_grad_kernel(GradArgs a) {
  constexpr uint32_t kParts = SIDE * SIDE / 2048;
  const uint32_t r = blockIdx.x / kParts, i = blockIdx.x % kParts * 256 + threadIdx.x;
  const uint32_t row = i / (SIDE / 8), col = i % (SIDE / 8) * 8;
  uint32_t tm, tn;
  const uint32_t second = grad_tile(a, a.cut.full + r, &tm, &tn);
  const int64_t m = int64_t(tm) * SIDE + row, n = int64_t(tn) * SIDE + col;
  if (m >= a.to[0].rows || n >= a.to[0].cols) return;
  f32x4v lo, hi;
  join_eight<SIDE>(a.partial, a.cut, r, row, col, &lo, &hi);
  put_some(second ? a.to[1] : a.to[0], m, n, lo, hi);
}

__global__ __launch_bounds__(256) void clear_words_kernel(uint32_t* p, uint32_t n) {
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  if (i < n) p[i] = 0;
}

// No tokens: the weights' gradients are 0.
__global__ __launch_bounds__(256) void clear_gradients_kernel(uint16_t* a, uint16_t* b, int64_t n) {
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) a[i] = b[i] = 0;
}

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

int64_t tiles_on(int64_t n, int64_t side) { return (n + side - 1) / side; }
// Columns of g and u in a tile (32 in the narrow ones).
int64_t pair_columns(int64_t side) { return side == 64 ? 64 : side / 2; }

constexpr int64_t kFew = 16;       // tokens that few_gated_kernel takes: one product's rows
constexpr uint32_t kProducts = 3;  // g and u; dx; dWg and dWu

// Where one call's workspace keeps what.
struct Layout {
  bool few = false, narrow = false, copy_x = false, copy_w = false, gates = false;  // gates: g and u are formed
  int64_t ld = 0, half = 0, depth = 0;
  Tiling fwd, dx, dw;
  bool queued = false;
  // byte offsets
  int64_t queues = 0, x = 0, w = 0, dgates = 0, partial = 0, bytes = 0;
};

Layout layout_of(const GatedCall& c) {
  Layout L;
  L.gates = !c.grad || c.gates == nullptr;
  L.few = c.tokens <= kFew;
  L.half = up(c.ffn, 32);
  L.ld = up(c.hidden, 64);
  if (L.gates && !L.few)
    L.fwd = tiling_of((c.hidden + kBK - 1) / kBK, 0,  // k along the rows of both
                      [&](int64_t side) { return tiles_on(c.tokens, side) * tiles_on(c.ffn, pair_columns(side)); }, 0.2);
  // Small tiles' steps take the time of their LDS accesses.  As long as all of them are
  // on CUs of their own, tiles of half the columns, of two waves, take less (17 tokens,
  // 2048 x 768 10.7 us instead of 13.6); with more tiles the wide ones, which read
  // less (64 tokens, 4096 x 14336 53 us instead of 70).
  if (const int64_t n = tiles_on(c.tokens, 64) * tiles_on(c.ffn, 32); L.fwd.side == 64 && n <= tile_slots(64)) {
    L.narrow = true;
    L.fwd.cut.items = L.fwd.cut.tiles = L.fwd.cut.full = uint32_t(n);
  }
  // Tiles read rows that start and end on 16 bytes, those of 256 whole steps of k too:
  // a short last one spills their registers (8192 tokens, 4104 x 14336 2190 us, with
  // the copies, which are filled up with zeros, 1620), the smaller tiles' not (700,
  // 1016 x 2000 15 us, with the copies 28).  dx reads the weights one behind the
  // other.
  const bool tiles = c.grad || !L.few;
  const bool steps = !(L.gates && !L.few) || L.fwd.side < 256 || c.hidden % kBK == 0;
  L.depth = steps ? c.hidden : up(c.hidden, kBK);
  const bool w_aligned = steps && rows_aligned(c.w_gate, c.gate_ld, c.hidden) && rows_aligned(c.w_up, c.up_ld, c.hidden) &&
                         c.gate_ld == c.up_ld;
  L.copy_x = tiles && !(steps && rows_aligned(c.x, c.x_ld, c.hidden));
  L.copy_w = tiles && (!w_aligned || (c.grad && c.ffn % kBK != 0));
  int64_t at = 0, partial = 0;
  auto take = [&](int64_t n) {
    const int64_t here = at;
    at += up(n, 256);
    return here;
  };
  auto also = [&](const Tiling& t) {
    const int64_t n = partial_bytes(t.cut, t.side);
    partial = n > partial ? n : partial;
    L.queued |= t.cut.items > tile_slots(t.side);
  };
  if (L.gates && !L.few) also(L.fwd);
  if (c.grad) {
    const int64_t w_ld = L.copy_w ? L.ld : c.gate_ld, x_ld = L.copy_x ? L.ld : c.x_ld;
    const int64_t wide = 2 * L.half > x_ld ? 2 * L.half : x_ld;
    L.dx = tiling_of(2 * L.half / kBK, L.half * w_ld * 2, [&](int64_t side) { return tiles_on(c.tokens, side) * tiles_on(c.hidden, side); });
    L.dw = tiling_of((c.tokens + kBK - 1) / kBK, c.tokens * wide * 2,
                     [&](int64_t side) { return 2 * tiles_on(c.ffn, side) * tiles_on(c.hidden, side); });
    also(L.dx);
    also(L.dw);
  }
  if (L.queued) L.queues = take(kProducts * kQueueWords * kQueuePitch * 4);
  if (L.copy_x) L.x = take(c.tokens * L.ld * 2);
  if (L.copy_w) L.w = take(2 * L.half * L.ld * 2);
  if (c.grad) L.dgates = take(c.tokens * 2 * L.half * 2);
  if (partial > 0) L.partial = take(partial);
  L.bytes = at;
  return L;
}

#define TIDE_LAUNCHED()                       \
  do {                                        \
    const int rc_ = int(hipGetLastError());   \
    if (rc_ != 0) return rc_;                 \
  } while (0)

template <Form FA, Form FB>
int launch_grad(GradArgs a, const Tiling& t, float* partial, uint32_t* queue, hipStream_t st) {
  a.cut = t.cut;
  a.partial = partial;
  a.tiles_m = uint32_t(tiles_on(a.to[0].rows, t.side));
  a.tiles_n = uint32_t(tiles_on(a.to[0].cols, t.side));
  a.queue = t.cut.items > tile_slots(t.side) ? queue : nullptr;
  const dim3 grid(resident_groups(t.cut.items, t.side));
  if (t.side == 256)
    hipLaunchKernelGGL((gated_grad_kernel<FA, FB, 256, 2, 4>), grid, dim3(512), 0, st, a);
  else if (t.side == 128)
    hipLaunchKernelGGL((gated_grad_kernel<FA, FB, 128, 2, 2>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((gated_grad_kernel<FA, FB, 64, 2, 2>), grid, dim3(256), 0, st, a);
  TIDE_LAUNCHED();
  if (t.cut.splits == 1) return 0;
  const unsigned rest = t.cut.tiles - t.cut.full;
  if (t.side == 256)
    hipLaunchKernelGGL(join_grad_kernel<256>, dim3(rest * 32), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(join_grad_kernel<128>, dim3(rest * 8), dim3(256), 0, st, a);
  return int(hipGetLastError());
}

}  // namespace

namespace tide {

int64_t gated_block_bytes(const GatedCall& c) { return c.tokens > 0 && c.ffn > 0 ? layout_of(c).bytes : 0; }

int launch_gated_block(const GatedCall& c, void* workspace, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  if (c.tokens == 0) {
    if (!c.grad || c.accumulate || c.ffn == 0) return 0;
    hipLaunchKernelGGL(clear_gradients_kernel, dim3(2048), dim3(256), 0, st, static_cast<uint16_t*>(c.dw_gate),
                       static_cast<uint16_t*>(c.dw_up), c.ffn * c.hidden * (c.dw_f32 ? 2 : 1));
    return int(hipGetLastError());
  }
  const Layout L = layout_of(c);
  uint32_t* queues = reinterpret_cast<uint32_t*>(ws + L.queues);
  float* partial = reinterpret_cast<float*>(ws + L.partial);
  if (L.queued) {
    constexpr uint32_t kWords = kProducts * kQueueWords * kQueuePitch;
    hipLaunchKernelGGL(clear_words_kernel, dim3((kWords + 255) / 256), dim3(256), 0, st, queues, kWords);
    TIDE_LAUNCHED();
  }
  Operand x{c.x, nullptr, c.x_ld, 0, c.tokens}, w{c.w_gate, nullptr, c.gate_ld, 0, c.ffn};
  w.second = c.w_up;
  if (L.copy_x) {
    const int rc = launch_align_rows(c.x, c.x_ld, c.tokens, c.hidden, ws + L.x, L.ld, stream);
    if (rc != 0) return rc;
    x.base = ws + L.x;
    x.ld = L.ld;
  }
  if (L.copy_w) {
    char* to = ws + L.w;
    char* up_to = to + L.half * L.ld * 2;
    int rc = launch_align_rows(c.w_gate, c.gate_ld, c.ffn, c.hidden, to, L.ld, stream, L.half);
    if (rc == 0) rc = launch_align_rows(c.w_up, c.up_ld, c.ffn, c.hidden, up_to, L.ld, stream, L.half);
    if (rc != 0) return rc;
    w.base = to;
    w.second = up_to;
    w.ld = L.ld;
  }
  Finish f{};
  f.rows = c.tokens;
  f.cols = c.ffn;
  f.gelu = c.gelu;
  f.half = L.half;
  if (c.grad) {
    f.dout = static_cast<const uint16_t*>(c.dout);
    f.dout_ld = c.dout_ld;
    f.dgates = reinterpret_cast<uint16_t*>(ws + L.dgates);
  } else {
    f.out = static_cast<uint16_t*>(c.out);
    f.out_ld = c.out_ld;
    f.gates = static_cast<uint16_t*>(c.gates);
    f.gates_ld = c.gates_ld;
  }
  if (!L.gates) {
    const int64_t n = c.tokens * (L.half / 8);
    hipLaunchKernelGGL(kept_gates_kernel, dim3(unsigned((n + 255) / 256)), dim3(256), 0, st,
                       static_cast<const uint16_t*>(c.gates), c.gates_ld, f);
    TIDE_LAUNCHED();
  } else if (L.few) {
    // the caller's own rows: they may start anywhere
    const unsigned grid = unsigned((c.grad ? L.half : c.ffn) + 15) / 16;
    const uint16_t *xp = static_cast<const uint16_t*>(c.x), *gate = static_cast<const uint16_t*>(c.w_gate),
                   *up_w = static_cast<const uint16_t*>(c.w_up);
    hipLaunchKernelGGL(few_gated_kernel, dim3(grid), dim3(kFewWaves * 64), 0, st, xp, c.x_ld, gate, c.gate_ld, up_w,
                       c.up_ld, c.hidden, f);
    TIDE_LAUNCHED();
  } else {
    GatedArgs a;
    a.x = x;
    a.w = w;
    a.depth = L.depth;
    a.cut = L.fwd.cut;
    a.partial = partial;
    a.tiles_m = uint32_t(tiles_on(c.tokens, L.fwd.side));
    a.tiles_n = uint32_t(tiles_on(c.ffn, L.narrow ? 32 : pair_columns(L.fwd.side)));
    a.queue = a.cut.items > tile_slots(L.fwd.side) ? queues : nullptr;
    a.f = f;
    const dim3 grid(resident_groups(a.cut.items, L.fwd.side));
#define TIDE_GATED(WHOLE, BM, BN, WN)                                                                \
  do {                                                                                               \
    if (c.grad)                                                                                      \
      hipLaunchKernelGGL((gated_kernel<true, WHOLE, BM, BN, 2, WN>), grid, dim3(128 * WN), 0, st, a); \
    else                                                                                             \
      hipLaunchKernelGGL((gated_kernel<false, WHOLE, BM, BN, 2, WN>), grid, dim3(128 * WN), 0, st, a); \
  } while (0)
    if (L.fwd.side == 256)
      TIDE_GATED(true, 256, 256, 4);
    else if (L.fwd.side == 128 && L.depth % kBK == 0)
      TIDE_GATED(true, 128, 128, 2);
    else if (L.fwd.side == 128)
      TIDE_GATED(false, 128, 128, 2);
    else if (L.narrow)
      TIDE_GATED(true, 64, 64, 1);
    else
      TIDE_GATED(true, 64, 128, 2);
#undef TIDE_GATED
    TIDE_LAUNCHED();
    if (a.cut.splits > 1) {
      const unsigned rest = a.cut.tiles - a.cut.full;
      if (L.fwd.side == 256)
        hipLaunchKernelGGL(join_gated_kernel<256>, dim3(rest * 16), dim3(256), 0, st, a);
      else
        hipLaunchKernelGGL(join_gated_kernel<128>, dim3(rest * 4), dim3(256), 0, st, a);
      TIDE_LAUNCHED();
    }
  }
  if (!c.grad) return 0;

  GradArgs d{};
  d.a = Operand{f.dgates, nullptr, 2 * L.half, 0, c.tokens};
  d.b = w;
  d.b.extent = c.hidden;
  d.b.split = L.half / kBK;
  d.depth = 2 * L.half;
  d.products = 1;
  d.to[0] = d.to[1] = Target{c.dx, c.dx_ld, c.tokens, c.hidden, nullptr, nullptr, 1.0f, 0, 0};
  int rc = launch_grad<Form::kRows, Form::kStack>(d, L.dx, partial, queues + kQueueWords * kQueuePitch, st);
  if (rc != 0) return rc;
  GradArgs v{};
  v.a = Operand{f.dgates, nullptr, 2 * L.half, 0, c.ffn};
  v.b = x;
  v.b.extent = c.hidden;
  v.depth = c.tokens;
  v.shift = L.half * 2;
  v.products = 2;
  v.to[0] = Target{c.dw_gate, c.hidden, c.ffn, c.hidden, nullptr, nullptr, 1.0f, c.dw_f32, c.accumulate};
  v.to[1] = v.to[0];
  v.to[1].base = c.dw_up;
  return launch_grad<Form::kCols, Form::kCols>(v, L.dw, partial, queues + 2 * kQueueWords * kQueuePitch, st);
}

}  // namespace tide
