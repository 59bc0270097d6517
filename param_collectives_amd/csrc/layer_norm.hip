// Layer norm over the rows of a matrix and its gradients on MI355X (gfx950):
//   mean = sum x / n,  rstd = 1 / sqrt(sum (x - mean)^2 / n + eps)
//   y = (x - mean) rstd w + b
//   xh = (x - mean) rstd,  g = dy w
//   dx = rstd (g - sum g / n - xh sum (g xh) / n)
//   dw = sum over rows of dy xh,  db = sum over rows of dy.
//
// Bound by HBM.  A row stays in the registers of the threads that share it (a
// wave, or a workgroup of 256 to 1024), so that every value is read once: the
// mean, the squares around it and the result come from there.  A thread takes 16
// bytes of the wider type at a time, neighbouring threads neighbouring ones, and
// holds the same columns of each row that its workgroup walks: weight and bias
// are read once, and the sums of dw and db go on in registers, fp32, until the
// workgroup's last row.  They are then written for a second launch, which adds
// them over the workgroups in order.
//
// The squares are taken around the mean as rounded, whose error (the mean of
// what is left) is taken back from both: a mean far above the deviations costs
// the rounding of x alone.
//
// Rows too long for the registers are read two or three times, by loops.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gemm.h"
#include "training.h"

namespace {

using namespace tide;

struct NormArgs {
  const void* x;
  int64_t x_ld;
  const void* dy;  // gradients only
  int64_t dy_ld;
  void* out;       // y or dx
  int64_t out_ld;
  const void* weight;  // or null: 1
  const void* bias;    // or null: 0
  float* mean;         // the gradients read them
  float* rstd;
  float* partial;      // gradients: [workgroup][2][cols]
  int64_t rows;
  int32_t cols, affine_f32;
  float eps;
};

// U neighbouring values of a row, as they lie in memory: 8 or 16 bytes of bf16
// or 16 of fp32.
template <bool F32, int U>
struct Raw {
  static_assert(U == 4 || U == 8, "values of a thread");
  static constexpr int kWords = U * (F32 ? 4 : 2) / 4;
  uint32_t w[kWords];

  // Of which `left` exist (any number): zeros for the rest.
  __device__ __forceinline__ void load(const void* row, int64_t c, int left) {
    if (left >= U) {
      if constexpr (kWords == 4) {
        typedef any_u32x4 __attribute__((may_alias)) vec;
        const vec* p = reinterpret_cast<const vec*>(static_cast<const char*>(row) + c * (F32 ? 4 : 2));
        const u32x4 v = __builtin_nontemporal_load(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = v[i];
      } else {
        typedef u32x2 __attribute__((aligned(2), may_alias)) vec;
        const vec* p = reinterpret_cast<const vec*>(static_cast<const char*>(row) + c * (F32 ? 4 : 2));
        const u32x2 v = __builtin_nontemporal_load(p);
        w[0] = v[0];
        w[1] = v[1];
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
#pragma unroll
    for (int i = 0; i < U - 1; ++i) {
      if (i >= left) break;
      if constexpr (F32)
        w[i] = static_cast<const uint32_t*>(row)[c + i];
      else
        w[i / 2] |= uint32_t(static_cast<const uint16_t*>(row)[c + i]) << (16 * (i & 1));
    }
  }

  __device__ __forceinline__ float value(int i) const {
    if constexpr (F32) return __uint_as_float(w[i]);
    return (i & 1) ? high_bf16(w[i / 2]) : low_bf16(w[i / 2]);
  }

  __device__ __forceinline__ void set(const float* v) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = F32 ? __float_as_uint(v[i]) : two_bf16(v[2 * i], v[2 * i + 1]);
  }

  __device__ __forceinline__ void store(void* row, int64_t c, int left) const {
    if (left >= U) {
      if constexpr (kWords == 4) {
        typedef any_u32x4 __attribute__((may_alias)) vec;
        __builtin_nontemporal_store(u32x4{w[0], w[1], w[2], w[3]},
                                    reinterpret_cast<vec*>(static_cast<char*>(row) + c * (F32 ? 4 : 2)));
      } else {
        typedef u32x2 __attribute__((aligned(2), may_alias)) vec;
        __builtin_nontemporal_store(u32x2{w[0], w[1]},
                                    reinterpret_cast<vec*>(static_cast<char*>(row) + c * (F32 ? 4 : 2)));
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < U - 1; ++i) {
      if (i >= left) break;
      if constexpr (F32)
        static_cast<uint32_t*>(row)[c + i] = w[i];
      else
        static_cast<uint16_t*>(row)[c + i] = uint16_t(w[i / 2] >> (16 * (i & 1)));
    }
  }
};

template <bool F32>
constexpr int64_t kSize = F32 ? 4 : 2;

__device__ __forceinline__ float affine(const void* p, int32_t f32, int64_t c, float none) {
  if (p == nullptr) return none;
  return f32 ? static_cast<const float*>(p)[c] : low_bf16(static_cast<const uint16_t*>(p)[c]);
}

// The sum over a wave, in every lane.
template <int CTRL>
__device__ __forceinline__ float with_lane(float v) {
  return v + __uint_as_float(__builtin_amdgcn_update_dpp(0, int(__float_as_uint(v)), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = with_lane<0xB1>(v);   // lane ^ 1
  v = with_lane<0x4E>(v);   // lane ^ 2
  v = with_lane<0x141>(v);  // the other four of eight
  v = with_lane<0x140>(v);  // the other eight of sixteen
  v += other_16(v);
  return v + other_32(v);
}

// Two sums over the threads that share a row, in every one of them.  `turn`
// alternates between two sets of words, so that one barrier a sum is enough.
template <int SHARE>
struct RowSum {
  static constexpr int kWaves = SHARE / 64;
  float2 (*words)[kWaves > 1 ? kWaves : 1];
  int turn = 0;

  __device__ __forceinline__ float2 operator()(float a, float b) {
    a = wave_sum(a);
    b = wave_sum(b);
    if constexpr (kWaves > 1) {
      if ((threadIdx.x & 63) == 0) words[turn][wave_index()] = make_float2(a, b);
      __syncthreads();
      a = b = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float2 v = words[turn][w];
        a += v.x;
        b += v.y;
      }
      turn ^= 1;
    }
    return make_float2(a, b);
  }
};

// SHARE threads share a row of up to SHARE * U * J values; a workgroup of BLOCK
// threads walks BLOCK / SHARE rows at a time.
template <int SHARE>
constexpr int kBlock = SHARE < 256 ? 256 : SHARE;

template <bool XF32, bool YF32, int SHARE, int J>
__global__ __launch_bounds__(kBlock<SHARE>) void layer_norm_kernel(NormArgs a) {
  constexpr int U = XF32 || YF32 ? 4 : 8, kRows = kBlock<SHARE> / SHARE;
  __shared__ float2 words[2][SHARE / 64];
  RowSum<SHARE> sum{words};
  const int t = threadIdx.x % SHARE;
  const float n = float(a.cols);
  float w[J * U], b[J * U];
  int left[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = (j * SHARE + t) * U;
    left[j] = a.cols - c;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      w[j * U + i] = i < left[j] ? affine(a.weight, a.affine_f32, c + i, 1.0f) : 0.0f;
      b[j * U + i] = i < left[j] ? affine(a.bias, a.affine_f32, c + i, 0.0f) : 0.0f;
    }
  }
  const int64_t step = int64_t(gridDim.x) * kRows;
  int64_t r = int64_t(blockIdx.x) * kRows + threadIdx.x / SHARE;
  Raw<XF32, U> next[J];
  auto fetch = [&](int64_t row) {
    const char* p = static_cast<const char*>(a.x) + row * a.x_ld * kSize<XF32>;
#pragma unroll
    for (int j = 0; j < J; ++j) next[j].load(p, (j * SHARE + t) * U, left[j]);
  };
  if (r < a.rows) fetch(r);
  // a row's threads leave together: with more than one wave a row, a workgroup has one
  for (; r < a.rows; r += step) {
    float x[J * U];
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < U; ++i) x[j * U + i] = next[j].value(i);
    if (r + step < a.rows) fetch(r + step);
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < J * U; ++k) s += x[k];
    const float mean = sum(s, 0.0f).x / n;
    float off = 0.0f, squares = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float& v = x[j * U + i];
        v = i < left[j] ? v - mean : 0.0f;
        off += v;
        squares += v * v;
      }
    const float2 both = sum(off, squares);
    off = both.x / n;
    const float var = fmaxf(both.y / n - off * off, 0.0f);
    // a NaN of the row must come out: the maximum would drop it
    const float rstd = 1.0f / sqrtf((both.y != both.y ? both.y : var) + a.eps);
    char* out = static_cast<char*>(a.out) + r * a.out_ld * kSize<YF32>;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float y[U];
#pragma unroll
      for (int i = 0; i < U; ++i) y[i] = (x[j * U + i] - off) * rstd * w[j * U + i] + b[j * U + i];
      Raw<YF32, U> v;
      v.set(y);
      v.store(out, (j * SHARE + t) * U, left[j]);
    }
    if (t == 0) {
      if (a.mean) a.mean[r] = mean + off;
      if (a.rstd) a.rstd[r] = rstd;
    }
  }
}

template <bool XF32, bool YF32, int SHARE, int J>
__global__ __launch_bounds__(kBlock<SHARE>) void layer_norm_grad_kernel(NormArgs a) {
  constexpr int U = XF32 || YF32 ? 4 : 8, kRows = kBlock<SHARE> / SHARE;
  __shared__ float2 words[2][SHARE / 64];
  RowSum<SHARE> sum{words};
  const int t = threadIdx.x % SHARE;
  const float n = float(a.cols);
  float w[J * U], dw[J * U], db[J * U];
  int left[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = (j * SHARE + t) * U;
    left[j] = a.cols - c;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      w[j * U + i] = i < left[j] ? affine(a.weight, a.affine_f32, c + i, 1.0f) : 0.0f;
      dw[j * U + i] = db[j * U + i] = 0.0f;
    }
  }
  const int64_t step = int64_t(gridDim.x) * kRows;
  int64_t r = int64_t(blockIdx.x) * kRows + threadIdx.x / SHARE;
  Raw<XF32, U> next_x[J];
  Raw<YF32, U> next_dy[J];
  float next_mean = 0.0f, next_rstd = 0.0f;
  auto fetch = [&](int64_t row) {
    const char* px = static_cast<const char*>(a.x) + row * a.x_ld * kSize<XF32>;
    const char* py = static_cast<const char*>(a.dy) + row * a.dy_ld * kSize<YF32>;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      next_x[j].load(px, (j * SHARE + t) * U, left[j]);
      next_dy[j].load(py, (j * SHARE + t) * U, left[j]);
    }
    next_mean = a.mean[row];
    next_rstd = a.rstd[row];
  };
  if (r < a.rows) fetch(r);
  for (; r < a.rows; r += step) {
    float xh[J * U], g[J * U];
    const float mean = next_mean, rstd = next_rstd;
    float s = 0.0f, sx = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int k = j * U + i;
        const float dy = next_dy[j].value(i);
        xh[k] = i < left[j] ? (next_x[j].value(i) - mean) * rstd : 0.0f;
        g[k] = dy * w[k];
        dw[k] += dy * xh[k];
        db[k] += dy;
        s += g[k];
        sx += g[k] * xh[k];
      }
    if (r + step < a.rows) fetch(r + step);
    const float2 both = sum(s, sx);
    s = both.x / n;
    sx = both.y / n;
    char* out = static_cast<char*>(a.out) + r * a.out_ld * kSize<XF32>;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float d[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int k = j * U + i;
        d[i] = rstd * (g[k] - s - xh[k] * sx);
      }
      Raw<XF32, U> v;
      v.set(d);
      v.store(out, (j * SHARE + t) * U, left[j]);
    }
  }
  if (a.partial == nullptr) return;
  float* p = a.partial + int64_t(blockIdx.x) * 2 * a.cols;
  if constexpr (kRows > 1) {
    // the waves' sums, one after the other
    __shared__ float all[2 * SHARE * U * J];
    for (int turn = 0; turn < kRows; ++turn) {
      if (int(threadIdx.x) / SHARE == turn) {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int i = 0; i < U; ++i) {
            const int k = j * U + i, at = (k * SHARE + t) * 2;
            if (turn > 0) {
              dw[k] += all[at];
              db[k] += all[at + 1];
            }
            all[at] = dw[k];
            all[at + 1] = db[k];
          }
      }
      __syncthreads();
    }
    if (int(threadIdx.x) / SHARE != kRows - 1) return;
  }
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (i < left[j]) {
        const int c = (j * SHARE + t) * U + i;
        p[c] = dw[j * U + i];
        p[a.cols + c] = db[j * U + i];
      }
}

// The sums of dw and db over the workgroups: kSlices threads a column, each
// adding its share of the workgroups in order, then one the shares.
constexpr int kSlices = 16, kJoinCols = 64;
__global__ __launch_bounds__(kSlices* kJoinCols) void join_affine_kernel(const float* partial, int64_t groups,
                                                                         int64_t cols, void* dw, void* db,
                                                                         int32_t f32, int32_t accumulate) {
  __shared__ float part[2][kSlices][kJoinCols];
  const int k = threadIdx.x % kJoinCols, slice = threadIdx.x / kJoinCols;
  const int64_t c = int64_t(blockIdx.x) * kJoinCols + k;
  float a = 0.0f, b = 0.0f;
  if (c < cols) {
    const int64_t per = (groups + kSlices - 1) / kSlices, g0 = slice * per, g1 = g0 + per < groups ? g0 + per : groups;
#pragma unroll 4
    for (int64_t g = g0; g < g1; ++g) {
      a += partial[g * 2 * cols + c];
      b += partial[(g * 2 + 1) * cols + c];
    }
  }
  part[0][slice][k] = a;
  part[1][slice][k] = b;
  __syncthreads();
  if (slice > 1 || c >= cols) return;
  void* out = slice == 0 ? dw : db;
  if (out == nullptr) return;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kSlices; ++i) s += part[slice][i][k];
  if (f32) {
    float* o = static_cast<float*>(out) + c;
    *o = accumulate ? *o + s : s;
  } else {
    uint16_t* o = static_cast<uint16_t*>(out) + c;
    *o = uint16_t(bf16_bits_of(accumulate ? low_bf16(*o) + s : s));
  }
}

// ------------------------------------------------------------ rows of any length

constexpr int kWideBlock = 1024, kWideU = 4;

template <bool F32>
__device__ __forceinline__ float at(const void* row, int64_t c) {
  return F32 ? static_cast<const float*>(row)[c] : low_bf16(static_cast<const uint16_t*>(row)[c]);
}

template <bool XF32, bool YF32>
__global__ __launch_bounds__(kWideBlock) void wide_norm_kernel(NormArgs a) {
  __shared__ float2 words[2][kWideBlock / 64];
  RowSum<kWideBlock> sum{words};
  const float n = float(a.cols);
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const char* x = static_cast<const char*>(a.x) + r * a.x_ld * kSize<XF32>;
    char* out = static_cast<char*>(a.out) + r * a.out_ld * kSize<YF32>;
    auto each = [&](auto f) {
      for (int64_t c = int64_t(threadIdx.x) * kWideU; c < a.cols; c += kWideBlock * kWideU) {
        const int left = a.cols - c < kWideU ? int(a.cols - c) : kWideU;
        Raw<XF32, kWideU> v;
        v.load(x, c, left);
        f(v, c, left);
      }
    };
    float s = 0.0f;
    each([&](const Raw<XF32, kWideU>& v, int64_t, int) {
#pragma unroll
      for (int i = 0; i < kWideU; ++i) s += v.value(i);
    });
    const float mean = sum(s, 0.0f).x / n;
    float off = 0.0f, squares = 0.0f;
    each([&](const Raw<XF32, kWideU>& v, int64_t, int left) {
#pragma unroll
      for (int i = 0; i < kWideU; ++i) {
        const float d = i < left ? v.value(i) - mean : 0.0f;
        off += d;
        squares += d * d;
      }
    });
    const float2 both = sum(off, squares);
    off = both.x / n;
    const float var = fmaxf(both.y / n - off * off, 0.0f);
    const float rstd = 1.0f / sqrtf((both.y != both.y ? both.y : var) + a.eps);
    each([&](const Raw<XF32, kWideU>& v, int64_t c, int left) {
      float y[kWideU];
#pragma unroll
      for (int i = 0; i < kWideU; ++i)
        y[i] = i < left ? (v.value(i) - mean - off) * rstd * affine(a.weight, a.affine_f32, c + i, 1.0f) +
                              affine(a.bias, a.affine_f32, c + i, 0.0f)
                        : 0.0f;
      Raw<YF32, kWideU> o;
      o.set(y);
      o.store(out, c, left);
    });
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = mean + off;
      if (a.rstd) a.rstd[r] = rstd;
    }
  }
}

template <bool XF32, bool YF32>
__global__ __launch_bounds__(kWideBlock) void wide_norm_grad_kernel(NormArgs a) {
  __shared__ float2 words[2][kWideBlock / 64];
  RowSum<kWideBlock> sum{words};
  const float n = float(a.cols);
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const char* x = static_cast<const char*>(a.x) + r * a.x_ld * kSize<XF32>;
    const char* dy = static_cast<const char*>(a.dy) + r * a.dy_ld * kSize<YF32>;
    char* out = static_cast<char*>(a.out) + r * a.out_ld * kSize<XF32>;
    const float mean = a.mean[r], rstd = a.rstd[r];
    auto each = [&](auto f) {
      for (int64_t c = int64_t(threadIdx.x) * kWideU; c < a.cols; c += kWideBlock * kWideU) {
        const int left = a.cols - c < kWideU ? int(a.cols - c) : kWideU;
        Raw<XF32, kWideU> vx;
        Raw<YF32, kWideU> vy;
        vx.load(x, c, left);
        vy.load(dy, c, left);
        float xh[kWideU], g[kWideU];
#pragma unroll
        for (int i = 0; i < kWideU; ++i) {
          xh[i] = i < left ? (vx.value(i) - mean) * rstd : 0.0f;
          g[i] = i < left ? vy.value(i) * affine(a.weight, a.affine_f32, c + i, 1.0f) : 0.0f;
        }
        f(xh, g, c, left);
      }
    };
    float s = 0.0f, sx = 0.0f;
    each([&](const float* xh, const float* g, int64_t, int) {
#pragma unroll
      for (int i = 0; i < kWideU; ++i) {
        s += g[i];
        sx += g[i] * xh[i];
      }
    });
    const float2 both = sum(s, sx);
    s = both.x / n;
    sx = both.y / n;
    each([&](const float* xh, const float* g, int64_t c, int left) {
      float d[kWideU];
#pragma unroll
      for (int i = 0; i < kWideU; ++i) d[i] = rstd * (g[i] - s - xh[i] * sx);
      Raw<XF32, kWideU> o;
      o.set(d);
      o.store(out, c, left);
    });
  }
}

// dw and db of a strip of columns over a slice of the rows (blockIdx.y).
template <bool XF32, bool YF32>
__global__ __launch_bounds__(256) void wide_affine_kernel(NormArgs a) {
  const int64_t c = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (c >= a.cols) return;
  float dw = 0.0f, db = 0.0f;
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
    const float x = at<XF32>(static_cast<const char*>(a.x) + r * a.x_ld * kSize<XF32>, c);
    const float dy = at<YF32>(static_cast<const char*>(a.dy) + r * a.dy_ld * kSize<YF32>, c);
    dw += dy * ((x - a.mean[r]) * a.rstd[r]);
    db += dy;
  }
  float* p = a.partial + int64_t(blockIdx.y) * 2 * a.cols;
  p[c] = dw;
  p[a.cols + c] = db;
}

// ------------------------------------------------------------ launches

struct Shape {
  int share, j;  // threads of a row and their pieces; share 0: any length
  int64_t groups;
};

Shape shape_of(const LayerNormCall& c, bool grad) {
  const int64_t u = c.x_f32 || c.y_f32 ? 4 : 8;
  Shape s{0, 0, 0};
  for (int share : {64, 256, 512, 1024}) {
    if (c.cols <= share * u * 2) {
      s.share = share;
      s.j = c.cols <= share * u ? 1 : 2;
      break;
    }
  }
  if (s.share == 0) {
    s.groups = c.rows < 512 ? c.rows : 512;
    return s;
  }
  const int64_t block = s.share < 256 ? 256 : s.share, at_once = block / s.share;
  const int64_t need = (c.rows + at_once - 1) / at_once, most = 256 * (2048 / block) / (grad ? 2 : 1);
  s.groups = need < most ? need : most;
  return s;
}

template <bool XF32, bool YF32>
int launch(const LayerNormCall& c, const Shape& s, const NormArgs& a, bool grad, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(s.groups));
#define TIDE_NORM(SHARE, J)                                                                                     \
  do {                                                                                                          \
    if (grad)                                                                                                   \
      hipLaunchKernelGGL((layer_norm_grad_kernel<XF32, YF32, SHARE, J>), grid, dim3(kBlock<SHARE>), 0, st, a); \
    else                                                                                                        \
      hipLaunchKernelGGL((layer_norm_kernel<XF32, YF32, SHARE, J>), grid, dim3(kBlock<SHARE>), 0, st, a);      \
  } while (0)
  if (s.share == 64 && s.j == 1)
    TIDE_NORM(64, 1);
  else if (s.share == 64)
    TIDE_NORM(64, 2);
  else if (s.share == 256 && s.j == 1)
    TIDE_NORM(256, 1);
  else if (s.share == 256)
    TIDE_NORM(256, 2);
  else if (s.share == 512)
    TIDE_NORM(512, 2);  // one piece would have fitted 256 threads
  else if (s.share == 1024)
    TIDE_NORM(1024, 2);
  else if (!grad)
    hipLaunchKernelGGL((wide_norm_kernel<XF32, YF32>), grid, dim3(kWideBlock), 0, st, a);
  else {
    hipLaunchKernelGGL((wide_norm_grad_kernel<XF32, YF32>), grid, dim3(kWideBlock), 0, st, a);
    const int rc = int(hipGetLastError());
    if (rc != 0 || a.partial == nullptr) return rc;
    hipLaunchKernelGGL((wide_affine_kernel<XF32, YF32>), dim3(unsigned((c.cols + 255) / 256), unsigned(s.groups)),
                       dim3(256), 0, st, a);
  }
#undef TIDE_NORM
  return int(hipGetLastError());
}

}  // namespace

namespace tide {

int64_t layer_norm_grad_bytes(const LayerNormCall& c) {
  if (c.rows == 0 || (c.dweight == nullptr && c.dbias == nullptr)) return 0;
  return (shape_of(c, true).groups * 2 * c.cols * 4 + 255) / 256 * 256;
}

int launch_layer_norm(const LayerNormCall& c, void* workspace, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool sums = c.grad && (c.dweight != nullptr || c.dbias != nullptr);
  Shape s{0, 0, 0};
  NormArgs a;
  a.x = c.x;
  a.x_ld = c.x_ld;
  a.dy = c.dout;
  a.dy_ld = c.y_ld;
  a.out = c.grad ? c.dx : c.out;
  a.out_ld = c.grad ? c.dx_ld : c.y_ld;
  a.weight = c.weight;
  a.bias = c.bias;
  a.mean = c.mean;
  a.rstd = c.rstd;
  a.partial = sums ? static_cast<float*>(workspace) : nullptr;
  a.rows = c.rows;
  a.cols = int32_t(c.cols);
  a.affine_f32 = c.affine_f32;
  a.eps = c.eps;
  if (c.rows > 0) {
    s = shape_of(c, c.grad);
    const int rc = c.x_f32 ? (c.y_f32 ? launch<true, true>(c, s, a, c.grad, st) : launch<true, false>(c, s, a, c.grad, st))
                           : (c.y_f32 ? launch<false, true>(c, s, a, c.grad, st)
                                      : launch<false, false>(c, s, a, c.grad, st));
    if (rc != 0) return rc;
  }
  if (!sums) return 0;
  // no rows: the sums are 0
  hipLaunchKernelGGL(join_affine_kernel, dim3(unsigned((c.cols + kJoinCols - 1) / kJoinCols)),
                     dim3(kSlices * kJoinCols), 0, st, a.partial, s.groups, c.cols, c.dweight, c.dbias, c.affine_f32,
                     c.accumulate);
  return int(hipGetLastError());
}

}  // namespace tide
