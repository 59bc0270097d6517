// Orthogonalised updates on MI355X (gfx950): a matrix X is taken towards U V^T of
// its singular value decomposition by a few steps of
//   X <- X / (|X| + eps)                       (the Frobenius norm)
//   G = X X^T,  P = a I + b G + c G^2,  X <- P X    (X^T X and X P for tall ones)
// so that every singular value s goes to s (a + b s^2 + c s^4) a step.  G and P
// are symmetric: only the tiles on and below the diagonal are formed, and written
// twice.
//
// Bound by the matrix cores: m (m + 1) n + m^2 (m + 1) + 2 m^2 n operations a
// step, m the smaller side.  The operands of the products are fp16, whose rate is
// bf16's: all entries of X, G and P are below 16, and kept times 2^12 they are
// normal numbers down to 2^-26, rounded by at most 2^-11.  bf16's roundings come
// out as errors of 1 to 3% in the 2-norm where a few directions are strong: what
// the first roundings of X leave in the weak directions is raised with them.  For
// the same reason the first kExact steps add a times the rest of X's rounding, a
// second fp16: 0.1% instead of 0.4% (a simulation in 64 bits with these roundings).
// From then on the weak directions are large enough.  A bf16 X has no rest at the
// start: it is scaled by a power of two, and what the norm is more than that goes
// into the first step's factors.
//
// Measured: one of 14336 x 4096 in fp32 4.3 ms (920 TFLOP/s), 128 of 2048 x 768 4.3 to
// 5.1 ms (600 to 510): their products have 24 and 64 steps of k, and what a tile takes
// beside them (X's rest read, X and its rest written, G and P written twice) is as
// much again; G and P of 32 at a time are 192 tiles, which leave 64 CUs idle.
//
// The norm is summed in fp64, which no entry's square leaves.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "gemm.h"
#include "training.h"

namespace {

using namespace tide;

constexpr int kExact = 3;               // steps whose a X keeps the rest of X's rounding
constexpr float kUnit = 4096.0f;        // entries are kept times this
constexpr float kRest = 2048.0f;        // and the rest of a rounding times this as well
constexpr int64_t kMost = 64;           // matrices of a piece, whose addresses go with the launch
constexpr int64_t kSumBlocks = 1024;    // workgroups that share a matrix's norm, at most

typedef float f32x8v __attribute__((ext_vector_type(8)));

__device__ __forceinline__ u32x4 eight_f16(f32x8v v) { return __builtin_bit_cast(u32x4, __builtin_convertvector(v, f16x8)); }
__device__ __forceinline__ f32x8v f16_values(u32x4 v) {
  return __builtin_convertvector(__builtin_bit_cast(f16x8, v), f32x8v);
}
__device__ __forceinline__ f32x8v join_quads(f32x4v lo, f32x4v hi) {
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}
// Eight values and the rests of their roundings.
__device__ __forceinline__ void split_eight(f32x8v v, u32x4* hi, u32x4* lo) {
  *hi = eight_f16(v);
  const f32x8v h = f16_values(*hi);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = (v[j] - h[j]) * kRest;
  *lo = eight_f16(v);
}

// Rows and columns of the workspace's matrices are filled up with zeros to a
// multiple of this, the k of a step.
__host__ __device__ __forceinline__ int64_t padded(int64_t n) { return (n + kBK - 1) / kBK * kBK; }

struct Pointers {
  void* p[kMost];
};

// Sixteens of rows that an epilogue loads ahead, a power of two less one: its
// operations on one take 0.3 us, a load one or two.
constexpr int kAhead = 3;

template <Form FA, Form FB, int SIDE, int WM, int WN>
using Products = std::conditional_t<SIDE == 64, DeepGemm<FA, FB, SIDE, SIDE, WM, WN, true, 4>,
                                    Gemm<FA, FB, Code::kE4m3, SIDE, SIDE, WM, WN, true, true>>;

// ------------------------------------------------------------ the norm

struct StartArgs {
  Pointers x;
  int32_t f32;
  int64_t ld, rows, cols;
  double* sums;    // [matrix][gridDim.x]
  float* factors;  // [matrix]: X over its norm is this times what is kept
  uint32_t* queues;
  uint32_t queue_words;
  float eps;
  uint16_t* hi;  // [matrix][rows][pitch]
  uint16_t* lo;
  int64_t pitch, matrix;
};

// 8 values of a row from column c, as fp32; zeros past its end.
__device__ __forceinline__ f32x8v eight_values(const StartArgs& a, const void* x, int64_t r, int64_t c) {
  f32x8v v;
  const int64_t left = a.cols - c;
  if (a.f32) {
    const float* p = static_cast<const float*>(x) + r * a.ld + c;
    if (left >= 8) {
      const f32x4v l = *reinterpret_cast<const any_f32x4*>(p), h = *reinterpret_cast<const any_f32x4*>(p + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = j < 4 ? l[j & 3] : h[j & 3];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = j < left ? p[j] : 0.0f;
    }
  } else {
    const u32x4 w = eight_of(static_cast<const uint16_t*>(x) + r * a.ld + c, left);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (j & 1) ? high_bf16(w[j >> 1]) : low_bf16(w[j >> 1]);
  }
  return v;
}

// The sum of squares of a workgroup's share of matrix blockIdx.y.  Clears the
// queues of the launches that follow.
__global__ __launch_bounds__(256) void square_sums_kernel(StartArgs a) {
  __shared__ double part[4];
  for (uint32_t i = (blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x; i < a.queue_words;
       i += gridDim.x * gridDim.y * 256)
    a.queues[i] = 0;
  const void* x = a.x.p[blockIdx.y];
  const int64_t groups = (a.cols + 7) / 8, all = a.rows * groups;
  double s = 0;
  const int64_t step = int64_t(gridDim.x) * 256;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < all; i += 4 * step) {
    f32x8v v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t at = i + k * step, r = at / groups;
      v[k] = f32x8v{};
      if (at < all) v[k] = eight_values(a, x, r, (at - r * groups) * 8);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) s += double(v[k][j]) * double(v[k][j]);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) a.sums[blockIdx.y * gridDim.x + blockIdx.x] = part[0] + part[1] + part[2] + part[3];
}

// X over its norm, times kUnit, but for a factor in [1, 2), in fp16, and of an fp32 X
// the rest in another; zeros around it.  The product is taken in fp64: its factor may
// lie outside fp32's range.
__global__ __launch_bounds__(256) void normalize_kernel(StartArgs a, int32_t blocks) {
  __shared__ double factor;
  if (threadIdx.x < 64) {
    double s = 0;
    for (int i = threadIdx.x; i < blocks; i += 64) s += a.sums[int64_t(blockIdx.y) * blocks + i];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
    if (threadIdx.x == 0) {
      const double f = double(kUnit) / (sqrt(s) + double(a.eps));
      // (a norm that is 0, infinite or NaN: all that is not 0 becomes NaN, or all)
      const bool plain = f > 0 && f < __builtin_inf();
      factor = plain ? ldexp(1.0, ilogb(f)) : f;
      if (blockIdx.x == 0) a.factors[blockIdx.y] = plain ? float(f / ldexp(1.0, ilogb(f))) : 1.0f;
    }
  }
  __syncthreads();
  const double f = factor;
  const void* x = a.x.p[blockIdx.y];
  const int64_t groups = a.pitch / 8, all = padded(a.rows) * groups;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < all; i += int64_t(gridDim.x) * 256) {
    const int64_t r = i / groups, c = (i - r * groups) * 8;
    f32x8v v = {};
    if (r < a.rows) v = eight_values(a, x, r, c);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = r < a.rows && c + j < a.cols ? float(double(v[j]) * f) : 0.0f;
    u32x4 hi, lo;
    split_eight(v, &hi, &lo);
    const int64_t at = int64_t(blockIdx.y) * a.matrix + r * a.pitch + c;
    *reinterpret_cast<u32x4*>(a.hi + at) = hi;
    if (a.f32) *reinterpret_cast<u32x4*>(a.lo + at) = lo;
  }
}

// ------------------------------------------------------------ G and P

// alpha S + beta G (+ diagonal), S = A A^T of each matrix.
struct SymmetricArgs {
  Operand a;
  int64_t a_matrix;  // elements from matrix to matrix
  int64_t depth;
  Cut cut;
  float* partial;
  uint32_t tiles;  // of a matrix
  uint32_t* queue;
  const uint16_t* g;  // or null
  uint16_t* out;      // size x size each (columns to padded(size)), rows `ld` apart, `matrix` elements from one to the next
  int64_t size, ld, matrix;
  float alpha, beta, diagonal;
  const float* factors;  // of A, or null: 1

  __device__ __forceinline__ float scale(int64_t z) const { return factors ? factors[z] * factors[z] * alpha : alpha; }
  // The values of 8 columns of row m from column n, whose G (if any) is `old`.
  __device__ __forceinline__ f32x8v value(float scale, int64_t m, int64_t n, f32x4v lo, f32x4v hi, u32x4 old) const {
    f32x8v v = join_quads(lo, hi);
    const f32x8v o = f16_values(old);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = scale * v[j] + (g ? beta * o[j] : 0.0f);
    if (diagonal != 0.0f) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (m == n + j) v[j] += diagonal;
    }
    if (n + 8 > size) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (n + j >= size) v[j] = 0.0f;
    }
    return v;
  }
};

// The matrix and the tile (row >= column) of tile t of all matrices.
__device__ __forceinline__ void symmetric_tile(const SymmetricArgs& a, uint32_t t, int64_t* z, uint32_t* tm,
                                               uint32_t* tn) {
  const uint32_t u = nth_of_share(t, a.cut.tiles), k = u / a.tiles, i = u - k * a.tiles;
  uint32_t row = uint32_t((sqrtf(8.0f * float(i) + 1.0f) - 1.0f) * 0.5f);
  while (row * (row + 1) / 2 > i) --row;
  while ((row + 1) * (row + 2) / 2 <= i) ++row;
  *z = __builtin_amdgcn_readfirstlane(k);
  *tm = __builtin_amdgcn_readfirstlane(row);
  *tn = __builtin_amdgcn_readfirstlane(i - row * (row + 1) / 2);
}

template <Form F, int SIDE, int WM, int WN>
__global__ __launch_bounds__(WM* WN * 64, SIDE == 64 ? 1 : 2) void symmetric_kernel(SymmetricArgs a) {
  using G = Products<F, F, SIDE, WM, WN>;
  __shared__ __align__(16) char lds0[G::kStage];
  __shared__ __align__(16) char lds1[G::kStage];
  __shared__ __align__(16) char lds2[G::kStage];
  __shared__ __align__(16) char lds3[G::kStage];
  __shared__ __align__(16) char own[own_rows<G, SIDE>()];
  char* const rows_lds = SIDE == 64 ? own : lds3;  // the epilogue's
  __shared__ uint32_t turn;
  Queue q;
  uint32_t item = blockIdx.x;
  if (a.queue) item = first_item(q, a.queue, a.cut.items, &turn);
  if (item == kNoItem) return;
  int64_t m0, n0, slot, z;
  G g;
  g.setup();
  auto open = [&](uint32_t item) {
    const Piece p = piece_of<false>(a.cut, item, a.depth);
    uint32_t tm, tn;
    symmetric_tile(a, p.tile, &z, &tm, &tn);
    m0 = int64_t(tm) * SIDE;
    n0 = int64_t(tn) * SIDE;
    slot = p.slot;
    Operand x = a.a;
    x.base = static_cast<const uint16_t*>(x.base) + z * a.a_matrix;
    g.open(x, x, m0, n0, p.k_first, p.k_end, lds0, lds1, lds2, lds3);
  };
  open(item);
  while (item != kNoItem) {
    g.loop(lds0, lds1, lds2, lds3);
    const uint32_t k = a.queue ? q.ask() : 0;
    const int64_t m1 = m0, n1 = n0, s1 = slot;
    const float scale = a.scale(z);
    g.renew_lane();
    const uint32_t row = g.lane / G::kRowGroups, ld = uint32_t(a.ld);
    // the rows come in order, and the places go on with them
    uint32_t at = (g.wm * (SIDE / WM) + row) * ld + uint32_t(g.column()), ahead = at;
    const int64_t rows = a.size - m1 - row, left = padded(a.size) - n1 - g.column();
    const int64_t first = z * a.matrix + m1 * a.ld + n1;
    uint16_t* const mirrored = a.out + z * a.matrix + n1 * a.ld + m1;
    // G's values of the rows that come next
    constexpr int kRows = 64 / G::kRowGroups, kCalls = 16 / kRows;  // rows of a call, calls of 16 rows
    u32x4 old[kAhead + 1][kCalls];
    auto before = [&](int i) {
      if (a.g == nullptr || s1 >= 0) return;
#pragma unroll
      for (int b = i == 0 ? 0 : i + kAhead - 1; b < i + kAhead && b < G::kFM; ++b)
#pragma unroll
        for (int q = 0; q < kCalls; ++q) {
          const int r = g.wm * (SIDE / WM) + b * 16 + q * kRows;
          if (r < rows && left > 0) old[b & kAhead][q] = *reinterpret_cast<const u32x4*>(a.g + first + ahead);
          ahead += kRows * ld;
        }
    };
    // rows of the mirrored tile are this one's columns
    const uint32_t m_at = uint32_t(g.mirror_column()) * ld + uint32_t(g.lane & 1) * 8;
    const int64_t m_rows = a.size - n1 - g.mirror_column(), m_left = a.size - m1 - (g.lane & 1) * 8;
    const int64_t m_pad = padded(a.size) - a.size;
    g.each_mirrored(
        rows_lds, s1 < 0 && m1 != n1, before,
        [&](int r, int i, int q, f32x4v& lo, f32x4v& hi) {
          if (s1 >= 0) return put_slot<SIDE>(a.partial, s1, r + row, g.column(), lo, hi);
          const f32x8v v = a.value(scale, m1 + r + row, n1 + g.column(), lo, hi, a.g ? old[i & kAhead][q] : u32x4{0, 0, 0, 0});
          if (r < rows && left > 0) *reinterpret_cast<u32x4*>(a.out + first + at) = eight_f16(v);
          at += kRows * ld;
          lo = __builtin_shufflevector(v, v, 0, 1, 2, 3);
          hi = __builtin_shufflevector(v, v, 4, 5, 6, 7);
        },
        [&](int r, int q, f32x4v lo, f32x4v hi) {
          f32x8v v = join_quads(lo, hi);
          const int64_t some = m_left - r;  // the tile below this one's rows may end inside the group
          if (some < 8) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (j >= some) v[j] = 0.0f;
          }
          if (32 * q < m_rows && some > -m_pad)
            *reinterpret_cast<u32x4*>(mirrored + r + (m_at + 32 * q * ld)) = eight_f16(v);
        },
        [&] {
          item = a.queue ? next_item(q, k, &turn) : kNoItem;
          if (item != kNoItem) open(item);
        });
  }
}

// Few and small matrices, k along the rows: a workgroup has a tile of 32 x 32 and its
// waves split k, each reading its steps of the rows straight into registers, eight of
// them on their way.  Taken where every tile has a CU (512 x 2048 orthogonalized
// takes 136 us, by tiles of 64 through LDS 143; 60 of 64 x 128 86 for 101; 16 of 256 x
// 256, whose 576 tiles are too many, 107 either way).  The first product of tall
// matrices, whose k runs down the columns, keeps the tiles of 64, which transpose as
// they read: 2048 x 512 takes 141 us, 60 of 128 x 64 94.  What is left is the launches':
// one that only waits for the last one's results takes 4 us of the 8 a launch.
constexpr int kFewWaves = 8;
__global__ __launch_bounds__(kFewWaves * 64) void few_symmetric_kernel(SymmetricArgs a) {
  constexpr int kDeep = 4;  // steps whose loads go out together
  __shared__ f32x4v part[kFewWaves][4][64];
  __shared__ float values[32][33];
  const int lane = threadIdx.x & 63, wave = wave_index(), r = lane & 15, g = lane >> 4;
  int64_t z;
  uint32_t tm, tn;
  symmetric_tile(a, blockIdx.x, &z, &tm, &tn);
  const int64_t m0 = int64_t(tm) * 32, n0 = int64_t(tn) * 32;
  // rows past the end read the last one: their results are dropped
  const uint16_t* rows = static_cast<const uint16_t*>(a.a.base) + z * a.a_matrix + 8 * g;
  const uint16_t* from[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = (i < 2 ? m0 : n0) + 16 * (i & 1) + r;
    from[i] = rows + (row < a.size ? row : a.size - 1) * a.a.ld;
  }
  const int64_t steps = a.depth / kBK, per = (steps + kFewWaves - 1) / kFewWaves, first = wave * per;
  const int64_t end = first + per < steps ? first + per : steps;
  f32x4v acc[2][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i >> 1][i & 1] = f32x4v{0.f, 0.f, 0.f, 0.f};
  struct Steps {
    f16x8 x[kDeep][4];
  } even, odd;
  auto fetch = [&](Steps& to, int64_t s) {
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const int64_t at = (s + u < end ? s + u : end - 1) * kBK;
#pragma unroll
      for (int i = 0; i < 4; ++i) to.x[u][i] = *(const TIDE_GLOBAL f16x8*)(from[i] + at);
    }
    __builtin_amdgcn_sched_barrier(0);  // all of them on their way before the first product
  };
  auto multiply = [&](const Steps& w, int64_t s) {
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      if (s + u >= end) break;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w.x[u][2 + j], w.x[u][i], acc[i][j], 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  if (first < end) {
    fetch(even, first);
    for (int64_t s = first; s < end; s += 2 * kDeep) {
      if (s + kDeep < end) fetch(odd, s + kDeep);
      multiply(even, s);
      if (s + kDeep >= end) break;
      if (s + 2 * kDeep < end) fetch(even, s + 2 * kDeep);
      multiply(odd, s + kDeep);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) part[wave][i][lane] = acc[i >> 1][i & 1];
  __syncthreads();
  // a lane holds of row m0 + 16 i + r the columns n0 + 16 j + 4 g + 0..3; 128 threads take 8 columns each
  if (threadIdx.x < 128) {
    const int row = threadIdx.x / 4, col = threadIdx.x % 4 * 8, i = row / 16 * 2 + col / 16;
    const int at = (row & 15) + (col & 15) / 4 * 16;
    const int64_t m = m0 + row, n = n0 + col;
    f32x8v v = {};
    if (m < a.size) {
      f32x4v lo = part[0][i][at], hi = part[0][i][at + 16];
#pragma unroll
      for (int k = 1; k < kFewWaves; ++k) {
        lo = add4(lo, part[k][i][at]);
        hi = add4(hi, part[k][i][at + 16]);
      }
      const int64_t to = z * a.matrix + m * a.ld + n;
      v = a.value(a.scale(z), m, n, lo, hi, a.g ? *reinterpret_cast<const u32x4*>(a.g + to) : u32x4{0, 0, 0, 0});
      *reinterpret_cast<u32x4*>(a.out + to) = eight_f16(v);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) values[row][col + j] = v[j];
  }
  if (tm == tn) return;
  __syncthreads();
  if (threadIdx.x >= 128) return;
  const int n = threadIdx.x / 4, m = threadIdx.x % 4 * 8;
  if (n0 + n >= a.size) return;
  f32x8v v;
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = values[m + j][n];
  *reinterpret_cast<u32x4*>(a.out + z * a.matrix + (n0 + n) * a.ld + m0 + m) = eight_f16(v);
}

// A part of a tile is 32 rows of 64 columns.
template <int SIDE>
__global__ __launch_bounds__(256) void join_symmetric_kernel(SymmetricArgs a) {
  constexpr uint32_t kParts = SIDE * SIDE / 2048;
  __shared__ float values[32][65];
  const uint32_t r = blockIdx.x / kParts, part = blockIdx.x % kParts;
  const uint32_t r0 = part / (SIDE / 64) * 32, c0 = part % (SIDE / 64) * 64;
  int64_t z;
  uint32_t tm, tn;
  symmetric_tile(a, a.cut.full + r, &z, &tm, &tn);
  const int64_t m0 = int64_t(tm) * SIDE, n0 = int64_t(tn) * SIDE;
  const uint32_t row = threadIdx.x / 8, col = threadIdx.x % 8 * 8;
  if (m0 + r0 >= padded(a.size) || n0 + c0 >= padded(a.size)) return;  // the whole part
  const int64_t m1 = m0 + r0 + row, n1 = n0 + c0 + col;
  f32x8v v = {};
  if (m1 < a.size && n1 < padded(a.size)) {
    f32x4v lo, hi;
    join_eight<SIDE>(a.partial, a.cut, r, r0 + row, c0 + col, &lo, &hi);
    const int64_t at = z * a.matrix + m1 * a.ld + n1;
    v = a.value(a.scale(z), m1, n1, lo, hi, a.g ? *reinterpret_cast<const u32x4*>(a.g + at) : u32x4{0, 0, 0, 0});
    *reinterpret_cast<u32x4*>(a.out + at) = eight_f16(v);
  }
  if (tm == tn) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) values[row][col + j] = v[j];
  __syncthreads();
  const uint32_t n = threadIdx.x / 4, m = threadIdx.x % 4 * 8;
  const int64_t m2 = n0 + c0 + n, n2 = m0 + r0 + m;
  if (m2 >= a.size || n2 >= padded(a.size)) return;
  // (zeros where the rows of this part end)
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = values[m + j][n];
  *reinterpret_cast<u32x4*>(a.out + z * a.matrix + m2 * a.ld + n2) = eight_f16(v);
}

// ------------------------------------------------------------ P X

struct UpdateArgs {
  Operand a, b;
  int64_t a_matrix, b_matrix;  // elements from matrix to matrix
  int64_t depth;
  Cut cut;
  float* partial;
  uint32_t tiles_m, tiles_n;
  uint32_t* queue;
  int64_t rows, cols, ld, matrix;
  int32_t rest;  // what lo holds of X is added
  uint16_t* lo;
  const float* factors;  // of X, or null: 1
  float coefficient;
  uint16_t* next;  // X's next, or null: the last step's result goes to out
  int32_t keep;    // the rest of its rounding goes to lo
  Pointers out;
  int64_t out_ld;

  // The next X times kUnit, of 8 columns, the rest of whose own X is y (or zeros);
  // f: factors' of the matrix.
  __device__ __forceinline__ float factor(int64_t z) const { return factors ? factors[z] : 1.0f; }
  __device__ __forceinline__ f32x8v value(float f, f32x4v l, f32x4v h, u32x4 y) const {
    const float scale = f * (1.0f / kUnit), more = f * coefficient * (1.0f / kRest);
    f32x8v v = join_quads(l, h);
    const f32x8v b = f16_values(y);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = scale * v[j] + (rest ? more * b[j] : 0.0f);
    return v;
  }
  // Its 8 columns, of which `left` exist (0 of a row that fills up), to places in
  // next, lo or out.
  __device__ __forceinline__ void put(f32x8v v, int64_t left, uint16_t* to_next, uint16_t* to_lo, uint16_t* to_out) const {
    if (next) {
      if (left < 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j >= left) v[j] = 0.0f;
      }
      if (!keep) {
        *reinterpret_cast<u32x4*>(to_next) = eight_f16(v);
        return;
      }
      u32x4 x, y;
      split_eight(v, &x, &y);
      *reinterpret_cast<u32x4*>(to_next) = x;
      *reinterpret_cast<u32x4*>(to_lo) = y;
      return;
    }
    u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = two_bf16(v[2 * j] * (1.0f / kUnit), v[2 * j + 1] * (1.0f / kUnit));
    if (left >= 8) {
      *reinterpret_cast<any_u32x4*>(to_out) = w;
      return;
    }
#pragma unroll
    for (int j = 0; j < 7; ++j)
      if (j < left) to_out[j] = uint16_t(w[j >> 1] >> (16 * (j & 1)));
  }
};

__device__ __forceinline__ void update_tile(const UpdateArgs& a, uint32_t t, int64_t* z, uint32_t* tm, uint32_t* tn) {
  const uint32_t tiles = a.tiles_m * a.tiles_n, u = nth_of_share(t, a.cut.tiles), k = u / tiles, i = u - k * tiles;
  const uint32_t band = i / (4 * a.tiles_n), in = i - band * 4 * a.tiles_n;
  const uint32_t rows = band * 4 + 4 <= a.tiles_m ? 4 : a.tiles_m - band * 4;
  *z = __builtin_amdgcn_readfirstlane(k);
  *tm = __builtin_amdgcn_readfirstlane(band * 4 + in % rows);
  *tn = __builtin_amdgcn_readfirstlane(in / rows);
}

template <Form FB, int SIDE, int WM, int WN>
__global__ __launch_bounds__(WM* WN * 64, SIDE == 64 ? 1 : 2) void update_kernel(UpdateArgs a) {
  using G = Products<Form::kRows, FB, SIDE, WM, WN>;
  __shared__ __align__(16) char lds0[G::kStage];
  __shared__ __align__(16) char lds1[G::kStage];
  __shared__ __align__(16) char lds2[G::kStage];
  __shared__ __align__(16) char lds3[G::kStage];
  __shared__ __align__(16) char own[own_rows<G, SIDE>()];
  char* const rows_lds = SIDE == 64 ? own : lds3;  // the epilogue's
  __shared__ uint32_t turn;
  Queue q;
  uint32_t item = blockIdx.x;
  if (a.queue) item = first_item(q, a.queue, a.cut.items, &turn);
  if (item == kNoItem) return;
  int64_t m0, n0, slot, z;
  G g;
  g.setup();
  auto open = [&](uint32_t item) {
    const Piece p = piece_of<false>(a.cut, item, a.depth);
    uint32_t tm, tn;
    update_tile(a, p.tile, &z, &tm, &tn);
    m0 = int64_t(tm) * SIDE;
    n0 = int64_t(tn) * SIDE;
    slot = p.slot;
    Operand x = a.a, y = a.b;
    x.base = static_cast<const uint16_t*>(x.base) + z * a.a_matrix;
    y.base = static_cast<const uint16_t*>(y.base) + z * a.b_matrix;
    g.open(x, y, m0, n0, p.k_first, p.k_end, lds0, lds1, lds2, lds3);
  };
  open(item);
  while (item != kNoItem) {
    g.loop(lds0, lds1, lds2, lds3);
    const uint32_t k = a.queue ? q.ask() : 0;
    const int64_t m1 = m0, n1 = n0, s1 = slot;
    g.renew_lane();
    const uint32_t row = g.lane / G::kRowGroups;
    // the rows come in order, and the places go on with them
    const uint32_t ld = uint32_t(a.ld), out_ld = uint32_t(a.out_ld), r0 = g.wm * (SIDE / WM) + row;
    uint32_t at = r0 * ld + uint32_t(g.column()), ahead = at, out_at = r0 * out_ld + uint32_t(g.column());
    const int64_t rows = a.rows - m1 - row, left = a.cols - n1 - g.column();
    const int64_t row_pad = padded(a.rows) - a.rows, col_pad = padded(a.cols) - a.cols;
    const int64_t first = z * a.matrix + m1 * a.ld + n1;
    uint16_t* out = static_cast<uint16_t*>(a.out.p[z]) + m1 * a.out_ld + n1;
    const float factor = a.factor(z);
    // what is left of X in the rows that come next
    constexpr int kRows = 64 / G::kRowGroups, kCalls = 16 / kRows;  // rows of a call, calls of 16 rows
    u32x4 y[kAhead + 1][kCalls];
    auto before = [&](int i) {
      if (!a.rest || s1 >= 0) return;
#pragma unroll
      for (int b = i == 0 ? 0 : i + kAhead - 1; b < i + kAhead && b < G::kFM; ++b)
#pragma unroll
        for (int q = 0; q < kCalls; ++q) {
          const int r = g.wm * (SIDE / WM) + b * 16 + q * kRows;
          if (r < rows && left > 0) y[b & kAhead][q] = *reinterpret_cast<const u32x4*>(a.lo + first + ahead);
          ahead += kRows * ld;
        }
    };
    g.each_rows(
        rows_lds, before,
        [&](int r, int i, int q, f32x4v lo, f32x4v hi) {
          if (s1 >= 0) return put_slot<SIDE>(a.partial, s1, r + row, g.column(), lo, hi);
          const uint32_t here = at, out_here = out_at;
          at += kRows * ld;
          out_at += kRows * out_ld;
          if (r - rows >= row_pad || left <= -col_pad) return;
          a.put(a.value(factor, lo, hi, a.rest ? y[i & kAhead][q] : u32x4{0, 0, 0, 0}), r < rows ? left : 0, a.next + first + here,
                a.lo + first + here, out + out_here);
        },
        [&] {
          item = a.queue ? next_item(q, k, &turn) : kNoItem;
          if (item != kNoItem) open(item);
        });
  }
}

template <int SIDE>
__global__ __launch_bounds__(256) void join_update_kernel(UpdateArgs a) {
  constexpr uint32_t kParts = SIDE * SIDE / 2048;
  const uint32_t r = blockIdx.x / kParts, i = blockIdx.x % kParts * 256 + threadIdx.x;
  const uint32_t row = i / (SIDE / 8), col = i % (SIDE / 8) * 8;
  int64_t z;
  uint32_t tm, tn;
  update_tile(a, a.cut.full + r, &z, &tm, &tn);
  const int64_t m = int64_t(tm) * SIDE + row, n = int64_t(tn) * SIDE + col;
  if (m >= padded(a.rows) || n >= padded(a.cols)) return;
  f32x4v lo = {}, hi = {};
  if (m < a.rows) join_eight<SIDE>(a.partial, a.cut, r, row, col, &lo, &hi);
  const int64_t at = z * a.matrix + m * a.ld + n;
  u32x4 y = u32x4{0, 0, 0, 0};
  if (a.rest && m < a.rows && n < a.cols) y = *reinterpret_cast<const u32x4*>(a.lo + at);
  a.put(a.value(a.factor(z), lo, hi, y), m < a.rows ? a.cols - n : 0, a.next + at, a.lo + at, static_cast<uint16_t*>(a.out.p[z]) + m * a.out_ld + n);
}

// ------------------------------------------------------------ launches

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Where one call's workspace keeps what, of `piece` matrices at a time.
struct Layout {
  bool tall = false;
  int64_t piece = 0, small = 0, pitch = 0, small_pitch = 0, matrix = 0, small_matrix = 0;
  int64_t sum_blocks = 0, copy_blocks = 0;  // workgroups of a matrix
  int64_t partial_bytes = 0;
  // byte offsets
  int64_t sums = 0, factors = 0, queues = 0, x0 = 0, x1 = 0, lo = 0, g = 0, p = 0, partial = 0, bytes = 0;
};

struct Tilings {
  Tiling gram, square, update;
};
int64_t steps_of(int64_t depth) { return padded(depth) / kBK; }
Tilings tilings_of(const OrthogonalCall& c, const Layout& L, int64_t count) {
  const int64_t large = c.rows > c.cols ? c.rows : c.cols;
  auto triangle = [&](int64_t side) {
    const int64_t t = (L.small + side - 1) / side;
    return count * t * (t + 1) / 2;
  };
  Tilings t;
  t.gram = tiling_of(steps_of(large), L.matrix * 2, triangle);
  t.square = tiling_of(steps_of(L.small), L.small_matrix * 2, triangle);
  t.update = tiling_of(steps_of(L.small), L.matrix * 2, [&](int64_t side) { return count * ((c.rows + side - 1) / side) * ((c.cols + side - 1) / side); });
  return t;
}

Layout layout_of(const OrthogonalCall& c) {
  Layout L;
  L.tall = c.rows > c.cols;
  L.small = L.tall ? c.cols : c.rows;
  L.pitch = up(c.cols, 64);
  L.small_pitch = up(L.small, 64);
  L.matrix = padded(c.rows) * L.pitch;
  L.small_matrix = L.small * L.small_pitch;
  const int64_t each = 3 * L.matrix * 2 + 2 * L.small_matrix * 2;
  // (With 256, 384, 512 MiB and 1 GiB 128 of 2048 x 768 take 5.38, 4.96, 5.10 and 4.90
  // ms, 64 of 2048 x 1408 7.54, 7.61, 7.00 and 7.11, 40 of 4096 x 1024 4.61, 4.68, 4.35
  // and 4.16: how a piece's tiles fill whole rounds decides.  384 MiB is as fast for
  // the first, and the memory is the caller's.)
  L.piece = (int64_t(3) << 27) / each;
  L.piece = L.piece < 1 ? 1 : L.piece > kMost ? kMost : L.piece;
  if (L.piece > c.count) L.piece = c.count;
  // pieces of one size, the last one's rest apart
  const int64_t pieces = (c.count + L.piece - 1) / L.piece;
  L.piece = (c.count + pieces - 1) / pieces;
  const int64_t groups = (padded(c.rows) * (L.pitch / 8) + 255) / 256;
  L.sum_blocks = 2048 / L.piece;
  if (L.sum_blocks > kSumBlocks) L.sum_blocks = kSumBlocks;
  if (L.sum_blocks > (groups + 3) / 4) L.sum_blocks = (groups + 3) / 4;  // of four groups a thread
  L.copy_blocks = 8192 / L.piece;
  if (L.copy_blocks > groups) L.copy_blocks = groups;
  const int64_t last = c.count - (pieces - 1) * L.piece;
  for (int64_t n : {L.piece, last}) {
    const Tilings t = tilings_of(c, L, n);
    for (const Tiling& one : {t.gram, t.square, t.update}) {
      const int64_t bytes = partial_bytes(one.cut, one.side);
      L.partial_bytes = bytes > L.partial_bytes ? bytes : L.partial_bytes;
    }
  }
  int64_t at = 0;
  auto take = [&](int64_t n) {
    const int64_t here = at;
    at += up(n, 256);
    return here;
  };
  L.sums = take(L.piece * L.sum_blocks * 8);
  L.factors = take(L.piece * 4);
  L.queues = take(3 * c.steps * kQueueWords * kQueuePitch * 4);
  L.x0 = take(L.piece * L.matrix * 2);
  L.x1 = take(L.piece * L.matrix * 2);
  L.lo = take(L.piece * L.matrix * 2);
  L.g = take(L.piece * L.small_matrix * 2);
  L.p = take(L.piece * L.small_matrix * 2);
  if (L.partial_bytes > 0) L.partial = take(L.partial_bytes);
  L.bytes = at;
  return L;
}

#define TIDE_LAUNCHED()                       \
  do {                                        \
    const int rc_ = int(hipGetLastError());   \
    if (rc_ != 0) return rc_;                 \
  } while (0)

template <Form F>
int launch_symmetric(SymmetricArgs a, const Tiling& t, int64_t count, uint32_t* queue, hipStream_t st) {
  a.cut = t.cut;
  a.tiles = uint32_t(t.cut.tiles / count);
  const int64_t on_side = (a.size + 31) / 32, few = count * on_side * (on_side + 1) / 2;
  if (F == Form::kRows && t.side == 64 && few <= tile_slots(64)) {
    a.cut.tiles = uint32_t(few);
    a.tiles = uint32_t(few / count);
    hipLaunchKernelGGL(few_symmetric_kernel, dim3(unsigned(few)), dim3(kFewWaves * 64), 0, st, a);
    return int(hipGetLastError());
  }
  a.queue = t.cut.items > tile_slots(t.side) ? queue : nullptr;
  const dim3 grid(resident_groups(t.cut.items, t.side));
  if (t.side == 256)
    hipLaunchKernelGGL((symmetric_kernel<F, 256, 2, 4>), grid, dim3(512), 0, st, a);
  else if (t.side == 128)
    hipLaunchKernelGGL((symmetric_kernel<F, 128, 2, 2>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((symmetric_kernel<F, 64, 2, 2>), grid, dim3(256), 0, st, a);
  TIDE_LAUNCHED();
  if (t.cut.splits == 1) return 0;
  const unsigned rest = t.cut.tiles - t.cut.full;
  if (t.side == 256)
    hipLaunchKernelGGL(join_symmetric_kernel<256>, dim3(rest * 32), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(join_symmetric_kernel<128>, dim3(rest * 8), dim3(256), 0, st, a);
  return int(hipGetLastError());
}

template <Form FB>
int launch_update(UpdateArgs a, const Tiling& t, uint32_t* queue, hipStream_t st) {
  a.cut = t.cut;
  a.tiles_m = uint32_t((a.rows + t.side - 1) / t.side);
  a.tiles_n = uint32_t((a.cols + t.side - 1) / t.side);
  a.queue = t.cut.items > tile_slots(t.side) ? queue : nullptr;
  const dim3 grid(resident_groups(t.cut.items, t.side));
  if (t.side == 256)
    hipLaunchKernelGGL((update_kernel<FB, 256, 2, 4>), grid, dim3(512), 0, st, a);
  else if (t.side == 128)
    hipLaunchKernelGGL((update_kernel<FB, 128, 2, 2>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((update_kernel<FB, 64, 2, 2>), grid, dim3(256), 0, st, a);
  TIDE_LAUNCHED();
  if (t.cut.splits == 1) return 0;
  const unsigned rest = t.cut.tiles - t.cut.full;
  if (t.side == 256)
    hipLaunchKernelGGL(join_update_kernel<256>, dim3(rest * 32), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL(join_update_kernel<128>, dim3(rest * 8), dim3(256), 0, st, a);
  return int(hipGetLastError());
}

int run_piece(const OrthogonalCall& c, const Layout& L, int64_t first, int64_t count, char* ws, hipStream_t st) {
  uint32_t* queues = reinterpret_cast<uint32_t*>(ws + L.queues);
  uint16_t* now = reinterpret_cast<uint16_t*>(ws + L.x0);
  uint16_t* next = reinterpret_cast<uint16_t*>(ws + L.x1);
  uint16_t* lo = reinterpret_cast<uint16_t*>(ws + L.lo);
  uint16_t* gram = reinterpret_cast<uint16_t*>(ws + L.g);
  uint16_t* poly = reinterpret_cast<uint16_t*>(ws + L.p);
  float* partial = reinterpret_cast<float*>(ws + L.partial);
  StartArgs s{};
  Pointers out{};
  for (int64_t i = 0; i < count; ++i) {
    s.x.p[i] = const_cast<void*>(c.x[first + i]);
    out.p[i] = c.out[first + i];
  }
  s.f32 = c.x_f32;
  s.ld = c.x_ld;
  s.rows = c.rows;
  s.cols = c.cols;
  s.sums = reinterpret_cast<double*>(ws + L.sums);
  s.factors = reinterpret_cast<float*>(ws + L.factors);
  s.queues = queues;
  s.queue_words = uint32_t(3 * c.steps * kQueueWords * kQueuePitch);
  s.eps = c.eps;
  s.hi = now;
  s.lo = lo;
  s.pitch = L.pitch;
  s.matrix = L.matrix;
  hipLaunchKernelGGL(square_sums_kernel, dim3(unsigned(L.sum_blocks), unsigned(count)), dim3(256), 0, st, s);
  TIDE_LAUNCHED();
  hipLaunchKernelGGL(normalize_kernel, dim3(unsigned(L.copy_blocks), unsigned(count)), dim3(256), 0, st, s,
                     int32_t(L.sum_blocks));
  TIDE_LAUNCHED();
  const Tilings t = tilings_of(c, L, count);
  for (int32_t k = 0; k < c.steps; ++k) {
    const bool last = k + 1 == c.steps;
    const float* factors = k == 0 ? s.factors : nullptr;
    uint32_t* q = queues + 3 * k * kQueueWords * kQueuePitch;
    SymmetricArgs g{};
    g.a = Operand{now, nullptr, L.pitch, 0, L.small};
    g.a_matrix = L.matrix;
    g.depth = padded(L.tall ? c.rows : c.cols);
    g.partial = partial;
    g.out = gram;
    g.size = L.small;
    g.ld = L.small_pitch;
    g.matrix = L.small_matrix;
    g.alpha = 1.0f / kUnit;
    g.factors = factors;
    int rc = L.tall ? launch_symmetric<Form::kCols>(g, t.gram, count, q, st)
                    : launch_symmetric<Form::kRows>(g, t.gram, count, q, st);
    if (rc != 0) return rc;
    g.a = Operand{gram, nullptr, L.small_pitch, 0, L.small};
    g.a_matrix = L.small_matrix;
    g.depth = padded(L.small);
    g.factors = nullptr;
    g.g = gram;
    g.out = poly;
    g.alpha = c.c / kUnit;
    g.beta = c.b;
    g.diagonal = c.a * kUnit;
    rc = launch_symmetric<Form::kRows>(g, t.square, count, q + kQueueWords * kQueuePitch, st);
    if (rc != 0) return rc;
    UpdateArgs u{};
    u.depth = padded(L.small);
    u.partial = partial;
    u.rows = c.rows;
    u.cols = c.cols;
    u.ld = L.pitch;
    u.matrix = L.matrix;
    u.rest = k == 0 ? c.x_f32 : k < kExact;
    u.factors = factors;
    u.lo = lo;
    u.coefficient = c.a;
    u.next = last ? nullptr : next;
    u.keep = k + 1 < kExact;
    u.out = out;
    u.out_ld = c.out_ld;
    if (L.tall) {
      u.a = Operand{now, nullptr, L.pitch, 0, c.rows};
      u.a_matrix = L.matrix;
      u.b = Operand{poly, nullptr, L.small_pitch, 0, L.small};
      u.b_matrix = L.small_matrix;
      rc = launch_update<Form::kRows>(u, t.update, q + 2 * kQueueWords * kQueuePitch, st);
    } else {
      u.a = Operand{poly, nullptr, L.small_pitch, 0, L.small};
      u.a_matrix = L.small_matrix;
      u.b = Operand{now, nullptr, L.pitch, 0, c.cols};
      u.b_matrix = L.matrix;
      rc = launch_update<Form::kCols>(u, t.update, q + 2 * kQueueWords * kQueuePitch, st);
    }
    if (rc != 0) return rc;
    uint16_t* const old = now;
    now = next;
    next = old;
  }
  return 0;
}

}  // namespace

namespace tide {

int64_t orthogonalize_bytes(const OrthogonalCall& c) {
  return c.count > 0 && c.rows > 0 && c.cols > 0 ? layout_of(c).bytes : 0;
}

int launch_orthogonalize(const OrthogonalCall& c, void* workspace, void* stream) {
  if (c.count == 0 || c.rows == 0 || c.cols == 0) return 0;
  const Layout L = layout_of(c);
  for (int64_t first = 0; first < c.count; first += L.piece) {
    const int64_t n = c.count - first < L.piece ? c.count - first : L.piece;
    const int rc = run_piece(c, L, first, n, static_cast<char*>(workspace), static_cast<hipStream_t>(stream));
    if (rc != 0) return rc;
  }
  return 0;
}

}  // namespace tide
