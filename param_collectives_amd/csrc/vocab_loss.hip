// Cross entropy of an output projection over a large vocabulary on MI355X
// (gfx950), with its gradients: for tokens t with hidden states H, projection
// rows W and targets,
//   z[t][v] = sum_d H[t][d] W[v][d]
//   lse[t]  = log sum_v exp z[t][v],   loss[t] = lse[t] - z[t][target]
//   dz[t][v] = g[t] (exp(z[t][v] - lse[t]) - [v = target])
//   dH = dz W,   dW = dz^T H.
// The logits are formed tile by tile in the matrix cores' fp32 accumulators
// and never written.  The loss keeps of each tile row its maximum and its sum
// of exponentials, and joins them over the vocabulary's tiles.  The gradients
// need every logit twice more; recomputing them would add a third to the three
// products' work, so the tile also leaves exp(z - tile row's maximum), which lies in
// [0, 1], in 16 bits (rounded by at most 2^-11, eight times finer than the bf16 it
// becomes; see two_powers), for a bounded piece of the tokens at a time.  A pass
// over that piece turns it into dz in bf16, the operand of the two
// products; the target's entry is expm1(-loss), since exp(z - lse) - 1 would lose a
// confident token's gradient to rounding.  What
// is rounded to bf16 is dz over the largest |g|, which comes back as a factor of
// the products' fp32 sums: g of a mean over n tokens is 1/n for all of them,
// and its own rounding (up to 2^-8, the same in every entry) would not average
// out (measured: the gradients' error of 0.0032 in the 2-norm falls to 0.0019,
// 0.0017 of it from the results' own rounding).
//
// Bound by the matrix cores and their power: at 4096 x 4096 x 128000 (tokens x
// hidden x vocabulary) the three products run 66 to 80% of the cycles, with the
// clock down to 1.75 GHz, and take 3.4, 2.9 to 3.2 and 3.2 of 9.9 ms (9.8 to 10.3 ms
// over the cards; 1250 to 1310 TFLOP/s); turning the logits into dz takes 0.33 ms at
// 6.3 TB/s.  The loss of 4096 x 4096 x 65536 takes 1.65 to 1.75 ms.  At up to 64
// tokens the weights' traffic is the bound (few_logits_kernel), in between a
// tile's latency: a step of 32 k takes 0.45 us with 128 x 128 tiles, 0.72 us with
// 256 x 256 ones.
//
// Tokens whose target lies outside the vocabulary are left out: nothing in their
// rows (a padded batch's NaN) reaches the others.  Where tokens are listed, those
// rows are never read; the loss of at most 256 tokens reads them with the others,
// and what a tile's row holds stays in its row.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gemm.h"
#include "training.h"

namespace {

using namespace tide;

constexpr float kLog2e = 1.44269504088896340736f;

// exp(z - m) for the tile row's maximum m; nothing but -inf in the row: 0.  (The
// difference first: a multiple of m by itself overflows where a mask has left a
// tile row nothing but the lowest numbers.)
__device__ __forceinline__ float reference(float m) { return m == -__builtin_inff() ? 0.0f : m; }
__device__ __forceinline__ float power(float z, float ref) { return __builtin_amdgcn_exp2f((z - ref) * kLog2e); }

// A token's loss from its row's maximum, the sum of exp(z - maximum) (at least 1,
// the maximum's own) and the target's logit.  The two logits' difference is taken
// first: lse - z_t, each rounded by itself, is noise where the target is likely
// (up to 4e-6 at logits of 40 and 4e-5 at 500, and below 0 for some of them).
__device__ __forceinline__ float token_loss(float top, float sum, float target_z) {
  return (top - target_z) + logf(sum);
}

// Two numbers of [0, 1] in 16 bits each: 6 bits of exponent and 10 of fraction, the
// middle bits of the fp32 number over 2^64, whose sign and two high exponent bits
// are 0.  Above 2^-62 they are rounded by at most 2^-11 of themselves, below by
// 2^-73.  (A word that is unlikely for every token gets its whole gradient from
// such entries: of fp16 numbers, times 2^15, those below 2^-29 lose bits and those
// below 2^-40 are 0.)
constexpr float kPowerUnit = 0x1p64f;
__device__ __forceinline__ uint32_t two_powers(float a, float b) {
  const uint32_t x = (__float_as_uint(a * (1.0f / kPowerUnit)) << 3) + 0x8000u;
  const uint32_t y = (__float_as_uint(b * (1.0f / kPowerUnit)) << 3) + 0x8000u;
  return __builtin_amdgcn_perm(y, x, 0x07060302u);
}
// The number in the low 16 bits, over kPowerUnit.
__device__ __forceinline__ float power_value(uint32_t bits) { return __uint_as_float((bits & 0xFFFFu) << 13); }

constexpr uint32_t kQueues = 3;  // of a piece's three products

// Rows of this piece that hold a token: the piece covers the listed tokens
// [first, first + piece).
__device__ __forceinline__ int64_t rows_of(const int32_t* count, int64_t first, int64_t piece) {
  int64_t n = int64_t(__builtin_amdgcn_readfirstlane(*count)) - first;
  n = n < piece ? n : piece;
  return n > 0 ? n : 0;
}

// ------------------------------------------------------------ the token list

// Lists the tokens that count, in order, and clears the loss and lse of the
// others; clears the queues; the largest |grad_loss| of the tokens that count goes
// to *scale (1 where that is 0 or not finite).  One workgroup: a pass per 1024
// tokens.
__global__ __launch_bounds__(1024) void list_tokens_kernel(const int64_t* targets, int64_t tokens, int64_t vocab,
                                                           const float* grad_loss, int32_t* list, int32_t* count,
                                                           float* scale, float* loss, float* lse, uint32_t* queues) {
  __shared__ int32_t wave_sum[16];
  __shared__ uint32_t wave_top[16];
  uint32_t top = 0;  // magnitudes compare as their bits, NaN above all
  if (threadIdx.x < kQueues * kQueueWords) queues[threadIdx.x * kQueuePitch] = 0;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  int32_t before = 0;
  for (int64_t t0 = 0; t0 < tokens; t0 += 1024) {
    const int64_t t = t0 + threadIdx.x;
    const int64_t v = t < tokens ? targets[t] : -1;
    const bool keep = v >= 0 && v < vocab;
    const uint64_t mask = __ballot(keep);
    if (lane == 0) wave_sum[wave] = int32_t(__popcll(mask));
    __syncthreads();
    int32_t at = before, total = 0;
    for (int w = 0; w < 16; ++w) {
      if (w < wave) at += wave_sum[w];
      total += wave_sum[w];
    }
    if (keep) {
      list[at + int32_t(__popcll(mask & ((uint64_t(1) << lane) - 1)))] = int32_t(t);
      if (grad_loss) {
        const uint32_t g = __float_as_uint(grad_loss[t]) & 0x7FFFFFFFu;
        top = top > g ? top : g;
      }
    } else if (t < tokens) {
      loss[t] = 0.0f;
      if (lse) lse[t] = 0.0f;
    }
    before += total;
    __syncthreads();
  }
  if (grad_loss) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t o = uint32_t(__shfl_xor(int(top), d));
      top = top > o ? top : o;
    }
    if (lane == 0) wave_top[wave] = top;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    *count = before;
    if (grad_loss) {
      for (int w = 0; w < 16; ++w) top = top > wave_top[w] ? top : wave_top[w];
      *scale = top == 0 || top >= 0x7F800000u ? 1.0f : __uint_as_float(top);
    }
  }
}

// The listed tokens' hidden states, row after row, each filled up with zeros
// to a pitch that is a multiple of 64; and zeros in the rows of dH (if any)
// whose tokens are not listed.
__global__ __launch_bounds__(256) void gather_rows_kernel(const uint16_t* hidden, int64_t ld, int64_t cols,
                                                          const int32_t* list, const int32_t* count, uint16_t* out,
                                                          int64_t out_ld, int64_t tokens,
                                                          const int64_t* targets, int64_t vocab, uint16_t* dhidden) {
  const int64_t groups = out_ld / 8, i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t r = i / groups, c = (i - r * groups) * 8;
  if (r >= tokens) return;
  if (dhidden) {
    const int64_t target = targets[r];
    if (target < 0 || target >= vocab) {
      for (int64_t j = c; j < c + 8 && j < cols; ++j) dhidden[r * cols + j] = 0;
    }
  }
  if (r >= *count) return;
  *reinterpret_cast<u32x4*>(out + r * out_ld + c) = eight_of(hidden + int64_t(list[r]) * ld + c, cols - c);
}

// ------------------------------------------------------------ logits

struct LogitsArgs {
  Operand h, w;            // h.extent is not used: the rows of the piece are
  const int32_t* count;    // null: every one of `tokens` rows is a token, in order
  const int32_t* list;
  const int64_t* targets;
  int64_t tokens, vocab, depth;
  int64_t first, piece;
  float2* stats;           // [row of the piece][vocabulary tile]: maximum, sum of the powers
  float* target_z;         // [row of the piece]
  uint16_t* e;             // [row of the piece][e_ld]: the powers in 16 bits, or null
  int64_t e_ld;
  uint32_t tiles_n;
  uint32_t* queue;         // null: every workgroup has its one tile
};

template <int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM* WN * 64, 2) void logits_kernel(LogitsArgs a) {
  using G = Gemm<Form::kRows, Form::kRows, Code::kE4m3, BM, BN, WM, WN>;
  __shared__ __align__(16) char lds0[G::kStage];
  __shared__ __align__(16) char lds1[G::kStage];
  __shared__ __align__(16) char lds2[G::kStage];
  __shared__ __align__(16) char lds3[G::kStage];
  // Per row of the tile: its waves' maxima and sums, and the target's column
  // (of the tile that runs and of the next).
  __shared__ float peak[WN][BM];
  __shared__ float sums[WN][BM];
  __shared__ int32_t aim[2][BM];
  constexpr int kFM = G::kFM, kFN = G::kFN, kRowsWave = BM / WM, kColsWave = BN / WN;
  const int64_t rows = a.count ? rows_of(a.count, a.first, a.piece) : a.tokens;
  const uint32_t tiles_m = uint32_t((rows + BM - 1) / BM), items = tiles_m * a.tiles_n;
  __shared__ uint32_t turn;
  Queue q;
  uint32_t item = blockIdx.x < items ? blockIdx.x : kNoItem;
  if (a.queue) item = first_item(q, a.queue, items, &turn);
  if (item == kNoItem) return;
  a.h.base = static_cast<const uint16_t*>(a.h.base) + a.first * a.h.ld;
  a.h.extent = rows;
  int64_t m0, n0;
  uint32_t tn;
  G g;
  g.setup();
  auto open = [&](uint32_t item) {
    uint32_t tm;
    tile_of(item, tiles_m, a.tiles_n, 4, &tm, &tn);
    m0 = int64_t(tm) * BM;
    n0 = int64_t(tn) * BN;
    g.open(a.h, a.w, m0, n0, 0, a.depth, lds0, lds1, lds2);
  };
  auto take_aim = [&](int set) {
    for (int row = g.tid; row < BM; row += G::kThreads) {
      int64_t col = -1;
      if (m0 + row < rows) col = a.targets[a.count ? a.list[a.first + m0 + row] : m0 + row] - n0;
      aim[set][row] = col >= 0 && col < BN ? int32_t(col) : -1;
    }
  };
  open(item);
  take_aim(0);
  for (int set = 0; item != kNoItem; set ^= 1) {
    g.loop(lds0, lds1, lds2, lds3);
    const uint32_t k = a.queue ? q.ask() : 0;
    const int64_t m1 = m0, n1 = n0;
    const uint32_t t1 = tn;

    // A lane holds of row 16 i + lane % 16 the columns 16 j + 4 (lane / 16) + r.
    // The tile row's maximum and sum go over its lanes, then over the WN waves.
    const int col0 = g.wn * kColsWave + 4 * (g.lane >> 4), row0 = g.wm * kRowsWave + (g.lane & 15);
    if (a.vocab - n1 < BN) {
      const int left = int(a.vocab - n1);
#pragma unroll
      for (int i = 0; i < kFM; ++i)
#pragma unroll
        for (int j = 0; j < kFN; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (col0 + 16 * j + r >= left) g.acc[i][j][r] = -__builtin_inff();
    }
#pragma unroll
    for (int i = 0; i < kFM; ++i) {
      float m = g.acc[i][0][0];
#pragma unroll
      for (int j = 0; j < kFN; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) m = fmaxf(m, g.acc[i][j][r]);
      m = fmaxf(m, other_16(m));
      m = fmaxf(m, other_32(m));
      if (g.lane < 16) peak[g.wn][row0 + 16 * i] = m;
    }
    lds_barrier();
#pragma unroll
    for (int i = 0; i < kFM; ++i) {
      const int row = row0 + 16 * i;
      const int at = aim[set][row] - col0;
      if (__any(at >= 0 && at < kColsWave)) {
        // the target's logit, before it becomes an exponential
#pragma unroll
        for (int j = 0; j < kFN; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (at == 16 * j + r) a.target_z[m1 + row] = g.acc[i][j][r];
      }
      float m = peak[0][row];
#pragma unroll
      for (int w = 1; w < WN; ++w) m = fmaxf(m, peak[w][row]);
      const float c = reference(m);
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < kFN; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float x = power(g.acc[i][j][r], c);
          g.acc[i][j][r] = x;
          s += x;
        }
      s += other_16(s);
      s += other_32(s);
      if (g.lane < 16) sums[g.wn][row] = s;
    }
    if (a.queue) {
      item = next_item(q, k, &turn);
      if (item != kNoItem) open(item);
    } else {
      item = kNoItem;
      lds_barrier();
    }
    for (int row = g.tid; row < BM; row += G::kThreads) {
      if (m1 + row >= rows) continue;
      float m = peak[0][row], s = sums[0][row];
#pragma unroll
      for (int w = 1; w < WN; ++w) {
        m = fmaxf(m, peak[w][row]);
        s += sums[w][row];
      }
      a.stats[(m1 + row) * a.tiles_n + t1] = make_float2(m, s);
    }
    if (a.e) {
      // the pitch is a multiple of 64: a group of 8 columns is in or out
      auto put = [&](int r, int c, f32x4v lo, f32x4v hi) {
        const u32x4 v = u32x4{two_powers(lo[0], lo[1]), two_powers(lo[2], lo[3]), two_powers(hi[0], hi[1]),
                              two_powers(hi[2], hi[3])};
        *reinterpret_cast<u32x4*>(a.e + (m1 + r) * a.e_ld + n1 + c) = v;
      };
      if (m1 + BM <= rows && n1 + BN <= a.e_ld) {
        g.template each<true>(lds3, put, [] {});
      } else {
        g.template each<false>(lds3, [&](int r, int c, f32x4v lo, f32x4v hi) {
          if (m1 + r < rows && n1 + c < a.e_ld) put(r, c, lo, hi);
        }, [] {});
      }
    }
    if (item != kNoItem) take_aim(set ^ 1);
  }
}

// The same for up to 16 NT tokens, where the weights' traffic is all that
// counts: a wave reads the fragments of 16 vocabulary rows straight into
// registers, a block of 256 k ahead (8 KiB a wave, 16 MiB over the GPU).  The
// states' blocks come through LDS, two in turn, for the four waves of a workgroup
// (each wave reading them for itself, which the L1 does not hold, took 44 us
// instead of 31 for 17 x 2048 x 32000 from cold caches).  Row r's 16 bytes c are
// kept at c ^ (r & 15): the fragment reads touch all banks once.
// A block's states are started before its weights, and the compiler must not mix
// them: the wait before a barrier lets the kSteps youngest loads go on, which
// have to be the weights', for the states are read by the other waves too.
template <int NT>
__global__ __launch_bounds__(256) void few_logits_kernel(LogitsArgs a) {
  constexpr int kDeep = 256, kSteps = kDeep / 32, kLoads = 2 * NT;
  __shared__ __align__(16) char h0[16 * NT * kDeep * 2];
  __shared__ __align__(16) char h1[16 * NT * kDeep * 2];
  __shared__ float peak[4][16 * NT];
  __shared__ float sums[4][16 * NT];
  const int64_t rows = a.count ? rows_of(a.count, a.first, a.piece) : a.tokens;
  if (rows == 0) return;
  const int lane = threadIdx.x & 63, wave = wave_index(), r = lane & 15, g = lane >> 4;
  const int64_t n0 = int64_t(blockIdx.x) * 64 + wave * 16;
  // rows past the end read the last one: their results are dropped
  const int64_t v = n0 + r < a.vocab ? n0 + r : a.vocab - 1;
  const char* w = static_cast<const char*>(a.w.base) + v * a.w.ld * 2 + g * 16;
  const char* h = static_cast<const char*>(a.h.base) + a.first * a.h.ld * 2;
  uint32_t off[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int lin = i * 256 + int(threadIdx.x), row = lin >> 5, c = (lin & 31) ^ (row & 15);
    off[i] = uint32_t(row < rows ? row : int(rows) - 1) * uint32_t(a.h.ld * 2) + uint32_t(c * 16);
  }
  auto load = [](const char* p) { return *(const TIDE_GLOBAL bf16x8*)p; };
  auto states = [&](char* to, int64_t block) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) load_to_lds(uniform(h + block * kDeep * 2), off[i], to + (i * 256 + wave * 64) * 16);
  };
  f32x4v acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = f32x4v{0.f, 0.f, 0.f, 0.f};
  const int64_t blocks = a.depth / kDeep;
  bf16x8 w0[kSteps], w1[kSteps];
  auto weights = [&](bf16x8* to, int64_t block) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) to[i] = load(w + block * kDeep * 2 + i * 64);
  };
  auto multiply = [&](const char* now, const bf16x8* wf) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const bf16x8 hf = *reinterpret_cast<const bf16x8*>(now + ((16 * t + r) * 32 + ((4 * i + g) ^ r)) * 16);
        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[i], hf, acc[t], 0, 0, 0);
      }
  };
  auto block = [&](const char* now, char* next, const bf16x8* wf, bf16x8* wn, int64_t b) {
    wait_loads<kSteps, true>();  // this block's states are older than its weights
    bare_barrier();
    states(next, b + 1);
    __builtin_amdgcn_sched_barrier(0);
    weights(wn, b + 1);
    __builtin_amdgcn_sched_barrier(0);
    multiply(now, wf);
  };
  auto last = [&](const char* now, const bf16x8* wf) {
    wait_loads<kSteps, true>();
    bare_barrier();
    multiply(now, wf);
  };
  if (blocks > 0) {
    states(h0, 0);
    __builtin_amdgcn_sched_barrier(0);
    weights(w0, 0);
    __builtin_amdgcn_sched_barrier(0);
    int64_t b = 0;
    for (; b + 2 < blocks; b += 2) {
      block(h0, h1, w0, w1, b);
      block(h1, h0, w1, w0, b + 1);
    }
    if (b + 1 < blocks) {
      block(h0, h1, w0, w1, b);
      last(h1, w1);
    } else {
      last(h0, w0);
    }
  }
  for (int64_t k = blocks * kDeep; k < a.depth; k += 32) {
    const bool in = k + 8 * g < a.depth;  // k counts in eights
    const bf16x8 zero = {};
    const bf16x8 wv = in ? load(w + k * 2) : zero;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int64_t row = 16 * t + r < rows ? 16 * t + r : rows - 1;
      const bf16x8 hv = in ? load(h + row * a.h.ld * 2 + (k + 8 * g) * 2) : zero;
      acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, hv, acc[t], 0, 0, 0);
    }
  }

  // A lane holds of token 16 t + r the vocabulary rows n0 + 4 g + 0..3.
  const int64_t left = a.vocab - n0 - 4 * g;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float m = -__builtin_inff();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= left) acc[t][j] = -__builtin_inff();
      m = fmaxf(m, acc[t][j]);
    }
    m = fmaxf(m, other_16(m));
    m = fmaxf(m, other_32(m));
    if (lane < 16) peak[wave][16 * t + r] = m;
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int row = 16 * t + r;
    if (row < rows) {
      const int64_t at = a.targets[a.count ? a.list[a.first + row] : row] - n0 - 4 * g;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (at == j && j < left) a.target_z[row] = acc[t][j];
    }
    float m = peak[0][row];
#pragma unroll
    for (int w4 = 1; w4 < 4; ++w4) m = fmaxf(m, peak[w4][row]);
    const float c = reference(m);
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      acc[t][j] = power(acc[t][j], c);
      s += acc[t][j];
    }
    s += other_16(s);
    s += other_32(s);
    if (lane < 16) sums[wave][row] = s;
    if (a.e && row < rows && n0 + 4 * g < a.e_ld)
      *reinterpret_cast<u32x2*>(a.e + row * a.e_ld + n0 + 4 * g) =
          u32x2{two_powers(acc[t][0], acc[t][1]), two_powers(acc[t][2], acc[t][3])};
  }
  __syncthreads();
  for (int row = threadIdx.x; row < rows; row += 256) {
    float m = peak[0][row], s = sums[0][row];
#pragma unroll
    for (int w4 = 1; w4 < 4; ++w4) {
      m = fmaxf(m, peak[w4][row]);
      s += sums[w4][row];
    }
    a.stats[row * a.tiles_n + blockIdx.x] = make_float2(m, s);
  }
}

// Joins a row's tiles: one workgroup per row.  (m, s) stands for s exp(m), and a
// tile of nothing but -inf, (-inf, 0), for nothing.  Each
// thread takes four tiles at a time, so that their loads overlap (a wave per row
// that read the tiles twice took 4.8 us for 17 rows of 500).  Clears the queues, which
// no workgroup uses by now.
__global__ __launch_bounds__(256) void join_rows_kernel(const float2* stats, uint32_t tiles, const int32_t* count,
                                                        const int32_t* list, const int64_t* targets, int64_t vocab,
                                                        int64_t tokens, int64_t first, int64_t piece,
                                                        const float* target_z, float2* row_sum, float* loss,
                                                        float* lse, uint32_t* queues) {
  constexpr float kLowest = -3.402823466e38f;  // finite: the difference of two of them is 0
  __shared__ float2 wave_part[4];
  // the logits' queue for the next piece, the others' for this one
  if (blockIdx.x == 0 && queues && threadIdx.x < kQueues * kQueueWords) queues[threadIdx.x * kQueuePitch] = 0;
  const int64_t row = blockIdx.x;
  const int64_t rows = count ? rows_of(count, first, piece) : tokens;
  if (row >= rows) return;
  const int lane = threadIdx.x & 63;
  const float2* p = stats + row * tiles;
  float m = kLowest, s = 0.0f;
  for (uint32_t t = threadIdx.x; t < tiles; t += 1024) {
    float2 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = t + 256 * j < tiles ? p[t + 256 * j] : make_float2(kLowest, 0.0f);
    float top = m;
#pragma unroll
    for (int j = 0; j < 4; ++j) top = fmaxf(top, v[j].x);
    s *= __builtin_amdgcn_exp2f((m - top) * kLog2e);
#pragma unroll
    for (int j = 0; j < 4; ++j) s += v[j].y * __builtin_amdgcn_exp2f((v[j].x - top) * kLog2e);
    m = top;
  }
  float top = m;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
  s *= __builtin_amdgcn_exp2f((m - top) * kLog2e);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
  if (lane == 0) wave_part[threadIdx.x >> 6] = make_float2(top, s);
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < 4; ++w) top = fmaxf(top, wave_part[w].x);
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) s += wave_part[w].y * __builtin_amdgcn_exp2f((wave_part[w].x - top) * kLog2e);
    const int64_t token = count ? list[first + row] : row;
    const int64_t target = targets[token];
    const bool keep = target >= 0 && target < vocab;
    if (row_sum) row_sum[row] = make_float2(top, s);
    loss[token] = keep ? token_loss(top, s, target_z[row]) : 0.0f;
    if (lse) lse[token] = keep ? top + logf(s) : 0.0f;
  }
}

// ------------------------------------------------------------ gradients

// The piece's exponentials (two_powers) -> dz / *scale (bf16), in place; the columns from the
// vocabulary's end to the row's pitch become 0.  A workgroup takes 2048
// columns of a row.
__global__ __launch_bounds__(256) void logit_grad_kernel(uint16_t* e, int64_t e_ld, int64_t vocab, const float2* stats,
                                                         uint32_t tiles, uint32_t tile_cols, const int32_t* count,
                                                         const int32_t* list, const int64_t* targets, int64_t first,
                                                         int64_t piece, const float* target_z, const float2* row_sum,
                                                         const float* grad_loss, const float* scale) {
  const int64_t row = blockIdx.y + int64_t(blockIdx.z) * 32768;
  const int64_t rows = rows_of(count, first, piece);
  if (row >= rows) return;
  const int64_t c = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (c >= e_ld) return;
  const int32_t token = list[first + row];
  const float2 sum = row_sum[row];
  const float g = grad_loss[token] / *scale;
  const int64_t target = targets[token];
  u32x4* p = reinterpret_cast<u32x4*>(e + row * e_ld + c);
  uint32_t out[4] = {0, 0, 0, 0};
  if (c < vocab) {
    const u32x4 w = *p;
    const float tile_max = stats[row * tiles + uint32_t(c) / tile_cols].x;
    const float f = __builtin_amdgcn_exp2f((tile_max - sum.x) * kLog2e) * (kPowerUnit / sum.y * g);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float v = power_value(w[j >> 1] >> (16 * (j & 1))) * f;
      if (c + j == target) v = g * expm1f(-token_loss(sum.x, sum.y, target_z[row]));
      if (c + j >= vocab) v = 0.0f;
      out[j >> 1] |= bf16_bits_of(v) << (16 * (j & 1));
    }
  }
  *p = u32x4{out[0], out[1], out[2], out[3]};
}

struct HiddenGradArgs {
  Operand dz, w;
  const int32_t* count;
  const float* scale;
  const int32_t* list;
  int64_t first, piece, hidden, vocab;
  float* partial;  // a slot of a tile for each piece of the cut, which the tokens that count decide
  uint16_t* dhidden;
  uint32_t tiles_n;
  uint32_t* queue;
};

template <int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM* WN * 64, 2) void hidden_grad_kernel(HiddenGradArgs a) {
  using G = Gemm<Form::kRows, Form::kCols, Code::kE4m3, BM, BN, WM, WN>;
  __shared__ __align__(16) char lds0[G::kStage];
  __shared__ __align__(16) char lds1[G::kStage];
  __shared__ __align__(16) char lds2[G::kStage];
  __shared__ __align__(16) char lds3[G::kStage];
  const int64_t rows = rows_of(a.count, a.first, a.piece);
  const uint32_t tiles_m = uint32_t((rows + BM - 1) / BM);
  const Cut cut = cut_tiles(tiles_m * a.tiles_n, (a.vocab + kBK - 1) / kBK, BM);
  __shared__ uint32_t turn;
  Queue q;
  uint32_t item = first_item(q, a.queue, cut.items, &turn);
  if (item == kNoItem) return;
  a.dz.extent = rows;
  const Target out{a.dhidden, a.hidden, rows, a.hidden, a.list + a.first, nullptr, *a.scale, 0, 0};
  int64_t m0, n0, slot;
  G g;
  g.setup();
  auto open = [&](uint32_t item) {
    const Piece p = piece_of<true>(cut, item, a.vocab);
    uint32_t tm, tn;
    tile_of(p.tile, tiles_m, a.tiles_n, 4, &tm, &tn);
    m0 = int64_t(tm) * BM;
    n0 = int64_t(tn) * BN;
    slot = p.slot;
    g.open(a.dz, a.w, m0, n0, p.k_first, p.k_end, lds0, lds1, lds2);
  };
  open(item);
  while (item != kNoItem) {
    g.loop(lds0, lds1, lds2, lds3);
    const uint32_t k = q.ask();
    const int64_t m1 = slot >= 0 ? 0 : m0, n1 = slot >= 0 ? 0 : n0;
    const Target t = slot >= 0 ? slot_target<BM>(a.partial, slot, rows - m0) : out;
    g.write(t, m1, n1, lds3, [&] {
      item = next_item(q, k, &turn);
      if (item != kNoItem) open(item);
    });
  }
}

template <int SIDE>
__global__ __launch_bounds__(256) void join_hidden_kernel(HiddenGradArgs a) {
  constexpr uint32_t kParts = SIDE * SIDE / 2048;
  const int64_t rows = rows_of(a.count, a.first, a.piece);
  const uint32_t tiles_m = uint32_t((rows + SIDE - 1) / SIDE);
  const Cut cut = cut_tiles(tiles_m * a.tiles_n, (a.vocab + kBK - 1) / kBK, SIDE);
  if (cut.splits == 1) return;
  for (uint32_t i = blockIdx.x; i < (cut.tiles - cut.full) * kParts; i += gridDim.x)
    join_tile<SIDE>(a.partial, cut, tiles_m, a.tiles_n, i / kParts, i % kParts,
                    Target{a.dhidden, a.hidden, rows, a.hidden, a.list + a.first, nullptr, *a.scale, 0, 0});
}

__global__ __launch_bounds__(256) void clear_kernel(uint16_t* p, int64_t n) {
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) p[i] = 0;
}

struct VocabGradArgs {
  Operand dz, h;
  const int32_t* count;
  const float* scale;
  int64_t first, piece, hidden, vocab;
  const float* sum_in;  // the earlier pieces' sums, or null
  float* sum_out;       // not the last piece: where the sums go on, or null
  void* dw;
  int32_t f32, accumulate;
  uint32_t tiles_m, tiles_n;
  uint32_t* queue;
};

template <int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM* WN * 64, 2) void vocab_grad_kernel(VocabGradArgs a) {
  using G = Gemm<Form::kCols, Form::kCols, Code::kE4m3, BM, BN, WM, WN>;
  __shared__ __align__(16) char lds0[G::kStage];
  __shared__ __align__(16) char lds1[G::kStage];
  __shared__ __align__(16) char lds2[G::kStage];
  __shared__ __align__(16) char lds3[G::kStage];
  __shared__ uint32_t turn;
  Queue q;
  uint32_t item = first_item(q, a.queue, a.tiles_m * a.tiles_n, &turn);
  if (item == kNoItem) return;
  const int64_t rows = rows_of(a.count, a.first, a.piece);
  a.h.base = static_cast<const uint16_t*>(a.h.base) + a.first * a.h.ld;
  const float scale = *a.scale;
  int64_t m0, n0;
  G g;
  g.setup();
  const Target t = a.sum_out ? Target{a.sum_out, a.hidden, a.vocab, a.hidden, nullptr, a.sum_in, 1.0f, 1, 0}
                             : Target{a.dw, a.hidden, a.vocab, a.hidden, nullptr, a.sum_in, scale, a.f32, a.accumulate};
  auto open = [&](uint32_t item) {
    uint32_t tm, tn;
    tile_of(item, a.tiles_m, a.tiles_n, 4, &tm, &tn);
    m0 = int64_t(tm) * BM;
    n0 = int64_t(tn) * BN;
    g.open(a.dz, a.h, m0, n0, 0, rows, lds0, lds1, lds2);
  };
  open(item);
  while (item != kNoItem) {
    g.loop(lds0, lds1, lds2, lds3);
    const uint32_t k = q.ask();
    const int64_t m1 = m0, n1 = n0;
    g.write(t, m1, n1, lds3, [&] {
      item = next_item(q, k, &turn);
      if (item != kNoItem) open(item);
    });
  }
}

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// The tile of a product that is not cut: 256, unless fewer than 192 of them leave
// CUs without one, or one side is at most 128, where half a tile would be
// filling (a loss of 109 x 2048 x 50000 50 -> 42 us; for a third of filling, 339
// or 300 tokens, 128 is still 15% slower than 256).
int tile_side(int64_t rows, int64_t cols) {
  return (rows + 255) / 256 * ((cols + 255) / 256) >= 192 && rows > 128 && cols > 128 ? 256 : 128;
}

// Where one call's workspace keeps what.
struct Layout {
  int64_t piece = 0, pieces = 0;
  int64_t h_ld = 0, w_ld = 0, e_ld = 0;
  bool listed = false;  // tokens are listed and their states gathered
  int rows = 256, cols = 256;  // tile of the logits; up to 64 tokens (rows 16 to 64) without LDS
  int64_t tiles_n = 0;
  int side_h = 256;     // of dH's tiles
  bool h_splits = false;  // whether they may be split
  int side_w = 256;     // of dW's tiles
  bool sums = false;    // dW's sums go over the pieces in the workspace
  // byte offsets
  int64_t list = 0, count = 0, queues = 0, h = 0, w = 0, stats = 0, target_z = 0, row_sum = 0, e = 0, partial = 0, dw_sums = 0,
          bytes = 0;
};

Layout layout_of(const VocabLossCall& c) {
  Layout L;
  const bool grad = c.dhidden_wanted;
  L.h_ld = up(c.hidden, 64);
  L.e_ld = up(c.vocab, 64);
  // A piece's exponentials take at most 2 GiB (and at least one tile of rows);
  // without them a piece is 32768 tokens.  (And at most 2^22 rows, each of which
  // gets a workgroup: a launch counts its threads in 32 bits.)
  int64_t most = grad ? (int64_t(1) << 31) / (L.e_ld * 2) / 256 * 256 : 32768;
  if (most > int64_t(1) << 22) most = int64_t(1) << 22;
  if (most < 256) most = 256;
  L.piece = c.tokens < most ? c.tokens : most;
  L.pieces = L.piece > 0 ? (c.tokens + L.piece - 1) / L.piece : 1;
  // One tile of rows gains nothing from leaving tokens out of a loss.
  L.listed = grad || c.tokens > 256 || !rows_aligned(c.h, c.h_ld, c.hidden);
  L.rows = L.piece <= 64 ? int(up(L.piece, 16)) : tile_side(L.piece, c.vocab);
  L.cols = L.piece <= 64 ? 64 : L.rows;
  L.tiles_n = (c.vocab + L.cols - 1) / L.cols;
  int64_t at = 0;
  auto take = [&](int64_t n) {
    const int64_t here = at;
    at += up(n, 256);
    return here;
  };
  if (L.listed) {
    L.count = take(8);  // and the scale
    L.queues = take(kQueues * kQueueWords * kQueuePitch * 4);
    L.list = take(c.tokens * 4);
    L.h = take(c.tokens * L.h_ld * 2);
  }
  if (!rows_aligned(c.w, c.w_ld, c.hidden)) {
    L.w_ld = L.h_ld;
    L.w = take(c.vocab * L.w_ld * 2);
  }
  L.stats = take(L.piece * L.tiles_n * 8);
  L.target_z = take(L.piece * 4);
  if (grad) {
    L.row_sum = take(L.piece * 8);
    L.e = take(L.piece * L.e_ld * 2);
    // The cut itself waits for the number of tokens that count.  Its partial
    // sums take no more slots than the rounds of its pieces, nor than every tile
    // split as far as may be.
    const int64_t steps = (c.vocab + kBK - 1) / kBK;
    const int64_t big = (L.piece + 255) / 256 * ((c.hidden + 255) / 256);
    const int64_t small = (L.piece + 127) / 128 * ((c.hidden + 127) / 128);
    L.side_h = cut_cost(cut_tiles(big, steps, 256), steps, 256) <= cut_cost(cut_tiles(small, steps, 128), steps, 128)
                   ? 256
                   : 128;
    const int64_t most = L.side_h == 256 ? big * (steps / 32) : small * (steps / 16);
    const int64_t room = most_rounds(L.side_h) * tile_slots(L.side_h);
    const int64_t slots = most < room ? most : room;
    // one tile is split if any number of them is
    L.h_splits = cut_tiles(1, steps, L.side_h).splits > 1;
    if (L.h_splits) L.partial = take(slots * L.side_h * L.side_h * 4);
    L.side_w = tile_side(c.vocab, c.hidden);
    L.sums = L.pieces > 1 && !c.dw_f32;
    if (L.sums) L.dw_sums = take(c.vocab * c.hidden * 4);
  }
  L.bytes = at;
  return L;
}

#define TIDE_LAUNCHED()                       \
  do {                                        \
    const int rc_ = int(hipGetLastError());   \
    if (rc_ != 0) return rc_;                 \
  } while (0)

}  // namespace

namespace tide {

int64_t vocab_loss_bytes(const VocabLossCall& c) { return c.tokens > 0 ? layout_of(c).bytes : 0; }

int launch_vocab_loss(const VocabLossCall& c, void* workspace, void* stream) {
  if (c.tokens == 0) {
    if (!c.dhidden_wanted || c.accumulate) return 0;
    const int64_t bytes = c.vocab * c.hidden * (c.dw_f32 ? 4 : 2);
    hipLaunchKernelGGL(clear_kernel, dim3(2048), dim3(256), 0,
                       static_cast<hipStream_t>(stream), static_cast<uint16_t*>(c.dw), bytes / 2);
    return int(hipGetLastError());
  }
  const Layout L = layout_of(c);
  char* ws = static_cast<char*>(workspace);
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool grad = c.dhidden_wanted;
  const int64_t* targets = c.targets;
  int32_t* count = L.listed ? reinterpret_cast<int32_t*>(ws + L.count) : nullptr;
  float* scale = L.listed ? reinterpret_cast<float*>(count + 1) : nullptr;
  uint32_t* queues = L.listed ? reinterpret_cast<uint32_t*>(ws + L.queues) : nullptr;
  int32_t* list = L.listed ? reinterpret_cast<int32_t*>(ws + L.list) : nullptr;
  Operand h{c.h, nullptr, c.h_ld, 0, c.tokens}, w{c.w, nullptr, c.w_ld, 0, c.vocab};
  if (L.listed) {
    hipLaunchKernelGGL(list_tokens_kernel, dim3(1), dim3(1024), 0, st, targets, c.tokens, c.vocab,
                       c.grad_loss, list, count, scale, c.loss, c.lse, queues);
    TIDE_LAUNCHED();
    uint16_t* rows = reinterpret_cast<uint16_t*>(ws + L.h);
    const int64_t n = c.tokens * (L.h_ld / 8);
    hipLaunchKernelGGL(gather_rows_kernel, dim3(unsigned((n + 255) / 256)), dim3(256), 0, st,
                       static_cast<const uint16_t*>(c.h), c.h_ld, c.hidden, list, count, rows, L.h_ld,
                       c.tokens, targets, c.vocab,
                       grad ? static_cast<uint16_t*>(c.dhidden) : nullptr);
    TIDE_LAUNCHED();
    h.base = rows;
    h.ld = L.h_ld;
  }
  if (!rows_aligned(c.w, c.w_ld, c.hidden)) {
    const int rc = launch_align_rows(c.w, c.w_ld, c.vocab, c.hidden, ws + L.w, L.w_ld, stream);
    if (rc != 0) return rc;
    w.base = ws + L.w;
    w.ld = L.w_ld;
  }
  float2* stats = reinterpret_cast<float2*>(ws + L.stats);
  float* target_z = reinterpret_cast<float*>(ws + L.target_z);
  float2* row_sum = grad ? reinterpret_cast<float2*>(ws + L.row_sum) : nullptr;
  uint16_t* e = grad ? reinterpret_cast<uint16_t*>(ws + L.e) : nullptr;
  for (int64_t p = 0; p < L.pieces; ++p) {
    const int64_t first = p * L.piece;
    LogitsArgs a;
    a.h = h;
    a.w = w;
    a.count = count;
    a.list = list;
    a.targets = targets;
    a.tokens = c.tokens;
    a.vocab = c.vocab;
    a.depth = c.hidden;
    a.first = first;
    a.piece = L.piece;
    a.stats = stats;
    a.target_z = target_z;
    a.e = e;
    a.e_ld = L.e_ld;
    a.tiles_n = uint32_t(L.tiles_n);
    const int64_t tiles = (L.piece + L.rows - 1) / L.rows * L.tiles_n;
    a.queue = queues;
    const dim3 grid(L.listed ? resident_groups(tiles, L.rows) : unsigned(tiles));
    if (L.rows == 256)
      hipLaunchKernelGGL((logits_kernel<256, 256, 2, 4>), grid, dim3(512), 0, st, a);
    else if (L.rows == 128)
      hipLaunchKernelGGL((logits_kernel<128, 128, 2, 2>), grid, dim3(256), 0, st, a);
    else if (L.rows == 64)
      hipLaunchKernelGGL(few_logits_kernel<4>, dim3(a.tiles_n), dim3(256), 0, st, a);
    else if (L.rows == 48)
      hipLaunchKernelGGL(few_logits_kernel<3>, dim3(a.tiles_n), dim3(256), 0, st, a);
    else if (L.rows == 32)
      hipLaunchKernelGGL(few_logits_kernel<2>, dim3(a.tiles_n), dim3(256), 0, st, a);
    else
      hipLaunchKernelGGL(few_logits_kernel<1>, dim3(a.tiles_n), dim3(256), 0, st, a);
    TIDE_LAUNCHED();
    hipLaunchKernelGGL(join_rows_kernel, dim3(unsigned(L.piece)), dim3(256), 0, st, stats, a.tiles_n, count,
                       list, targets, c.vocab, c.tokens, first, L.piece, target_z, row_sum, c.loss, c.lse,
                       queues);
    TIDE_LAUNCHED();
    if (!grad) continue;
    const int64_t rows_z = L.piece < 32768 ? L.piece : 32768;
    hipLaunchKernelGGL(logit_grad_kernel,
                       dim3(unsigned((L.e_ld + 2047) / 2048), unsigned(rows_z), unsigned((L.piece + 32767) / 32768)),
                       dim3(256), 0, st, e, L.e_ld, c.vocab, stats, a.tiles_n, uint32_t(L.cols), count, list, targets,
                       first, L.piece, target_z, row_sum, c.grad_loss, scale);
    TIDE_LAUNCHED();
    HiddenGradArgs d;
    d.dz = Operand{e, nullptr, L.e_ld, 0, L.piece};
    d.w = w;
    d.w.extent = c.hidden;
    d.count = count;
    d.scale = scale;
    d.list = list;
    d.first = first;
    d.piece = L.piece;
    d.hidden = c.hidden;
    d.vocab = c.vocab;
    d.partial = reinterpret_cast<float*>(ws + L.partial);
    d.dhidden = static_cast<uint16_t*>(c.dhidden);
    d.tiles_n = uint32_t((c.hidden + L.side_h - 1) / L.side_h);
    d.queue = queues + kQueueWords * kQueuePitch;
    // as many workgroups as fit, where there may be pieces: the cut waits for the tokens that count
    const int64_t tiles_h = (L.piece + L.side_h - 1) / L.side_h * d.tiles_n;
    const dim3 grid_h(L.h_splits ? unsigned(tile_slots(L.side_h)) : resident_groups(tiles_h, L.side_h));
    if (L.side_h == 256)
      hipLaunchKernelGGL((hidden_grad_kernel<256, 256, 2, 4>), grid_h, dim3(512), 0, st, d);
    else
      hipLaunchKernelGGL((hidden_grad_kernel<128, 128, 2, 2>), grid_h, dim3(256), 0, st, d);
    TIDE_LAUNCHED();
    if (L.h_splits) {
      if (L.side_h == 256)
        hipLaunchKernelGGL(join_hidden_kernel<256>, dim3(1024), dim3(256), 0, st, d);
      else
        hipLaunchKernelGGL(join_hidden_kernel<128>, dim3(1024), dim3(256), 0, st, d);
      TIDE_LAUNCHED();
    }
    VocabGradArgs v;
    v.dz = Operand{e, nullptr, L.e_ld, 0, c.vocab};
    v.h = h;
    v.h.extent = c.hidden;
    v.count = count;
    v.scale = scale;
    v.first = first;
    v.piece = L.piece;
    v.hidden = c.hidden;
    v.vocab = c.vocab;
    float* sums = L.sums ? reinterpret_cast<float*>(ws + L.dw_sums) : nullptr;
    v.sum_in = p > 0 ? sums : nullptr;
    v.sum_out = p + 1 < L.pieces ? sums : nullptr;
    v.dw = c.dw;
    v.queue = queues + 2 * kQueueWords * kQueuePitch;
    v.f32 = c.dw_f32;
    v.accumulate = c.accumulate || (p > 0 && !L.sums);
    const int64_t side_w = L.side_w;
    v.tiles_m = uint32_t((c.vocab + side_w - 1) / side_w);
    v.tiles_n = uint32_t((c.hidden + side_w - 1) / side_w);
    const dim3 grid_w(resident_groups(int64_t(v.tiles_m) * v.tiles_n, side_w));
    if (L.side_w == 256)
      hipLaunchKernelGGL((vocab_grad_kernel<256, 256, 2, 4>), grid_w, dim3(512), 0, st, v);
    else
      hipLaunchKernelGGL((vocab_grad_kernel<128, 128, 2, 2>), grid_w, dim3(256), 0, st, v);
    TIDE_LAUNCHED();
  }
  return 0;
}

}  // namespace tide
