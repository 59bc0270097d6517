// Layer norm over the rows of a matrix and its gradients on MI355X (gfx950):
//   mean = sum x / n,  rstd = 1 / sqrt(sum (x - mean)^2 / n + eps)
//   y = (x - mean) rstd w + b
//   xh = (x - mean) rstd,  g = dy w
//   dx = rstd (g - sum g / n - xh sum (g xh) / n)
//   dw = sum over rows of dy xh,  db = sum over rows of dy.
//
// Bound by HBM.  A row stays in the registers of the threads that share it (16
// lanes, a wave, or a workgroup of 256 to 1024), so that every value is read once:
// the mean, the squares around it and the result come from there.  A thread takes 16 bytes
// of the wider type at a time, neighbouring threads neighbouring ones, and holds
// the same columns of each row that its workgroup walks: weight and bias are read
// once, and the sums of dw and db go on in registers, fp32, until the workgroup's
// last row.  They are then written for a second launch, which adds them over the
// workgroups in order.  While a row is worked on, the next two are on their way:
// the barriers of a row's sums wait for LDS only.
//
// A row's values are summed in fp64 (bf16's in a thread in fp32, as 32nds: they
// hardly round there, and stay in range) and the mean is kept in two fp32: a mean far
// above the deviations costs the rounding of x alone.  The squares' sum and the
// gradients' two are fp32: in a thread, whose values are added up piece by piece (at
// most 12 additions for each), and over the threads (at most 22).  (In fp64 over the
// threads the gradients spill: 16384 bf16 rows of 8192 204 us instead of 154.)
//
// Measured: 8191 rows of 5120, fp32 to bf16, 42 to 44 us (5.7 to 6.0 TB/s); gradients
// of 16384 rows of 8192 in bf16 155 us (5.2 TB/s), of 262144 rows of 128 45 us (4.5
// TB/s, two launches; the forward pass 28 us); a few rows 3 us of kernel in a call of
// 4.5.
//
// Rows too long for the registers are read three times, by loops, and take 3 to 6
// times what their bytes do once: 4096 rows of 18432 in bf16 292 us, their gradients
// 404, 512 of 65536 in fp32 143 and 320.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

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

  __device__ __forceinline__ void load(const void* row, uint32_t c) {
    const char* p = static_cast<const char*>(row) + c * (F32 ? 4 : 2);
    if constexpr (kWords == 4) {
      typedef any_u32x4 __attribute__((may_alias)) vec;
      const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const vec*>(p));
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = v[i];
    } else {
      typedef u32x2 __attribute__((aligned(2), may_alias)) vec;
      const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const vec*>(p));
      w[0] = v[0];
      w[1] = v[1];
    }
  }
  __device__ __forceinline__ void store(void* row, uint32_t c) const {
    char* p = static_cast<char*>(row) + c * (F32 ? 4 : 2);
    if constexpr (kWords == 4) {
      typedef any_u32x4 __attribute__((may_alias)) vec;
      __builtin_nontemporal_store(u32x4{w[0], w[1], w[2], w[3]}, reinterpret_cast<vec*>(p));
    } else {
      typedef u32x2 __attribute__((aligned(2), may_alias)) vec;
      __builtin_nontemporal_store(u32x2{w[0], w[1]}, reinterpret_cast<vec*>(p));
    }
  }
  // The same of the first `left` values; zeros for the rest.
  __device__ __forceinline__ void load_some(const void* row, int64_t c, int left) {
    if (left >= U) return load(static_cast<const char*>(row) + c * (F32 ? 4 : 2), 0);
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
  __device__ __forceinline__ void store_some(void* row, int64_t c, int left) const {
    if (left >= U) return store(static_cast<char*>(row) + c * (F32 ? 4 : 2), 0);
#pragma unroll
    for (int i = 0; i < U - 1; ++i) {
      if (i >= left) break;
      if constexpr (F32)
        static_cast<uint32_t*>(row)[c + i] = w[i];
      else
        static_cast<uint16_t*>(row)[c + i] = uint16_t(w[i / 2] >> (16 * (i & 1)));
    }
  }

  // New to the compiler: what was worked out from it is not kept.
  __device__ __forceinline__ void renewed() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) renew(w[i]);
  }

  __device__ __forceinline__ float value(int i) const {
    if constexpr (F32) return __uint_as_float(w[i]);
    return (i & 1) ? high_bf16(w[i / 2]) : low_bf16(w[i / 2]);
  }

  __device__ __forceinline__ void set(const float* v) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = F32 ? __float_as_uint(v[i]) : two_bf16(v[2 * i], v[2 * i + 1]);
  }
};

template <bool F32>
constexpr int64_t kSize = F32 ? 4 : 2;

// The U columns of piece j of thread t of SHARE.  A row's last piece may be short:
// its thread takes the last U columns instead, of which the first `again` are its
// neighbour's too.  Both write them, the same values; sums leave them out.
struct Columns {
  uint32_t first;
  int again;  // U: there are none
};
template <int U, int SHARE>
__device__ __forceinline__ Columns columns_of(int cols, int j, int t) {
  const int c = (j * SHARE + t) * U, over = c + U - cols;
  return Columns{uint32_t(over > 0 ? cols - U : c), over <= 0 ? 0 : over < U ? over : U};
}

// Column c's weight or bias.
__device__ __forceinline__ float affine(const void* p, int32_t f32, int64_t c, float none) {
  if (p == nullptr) return none;
  return f32 ? static_cast<const float*>(p)[c] : low_bf16(static_cast<const uint16_t*>(p)[c]);
}

// U neighbouring ones.
template <int U>
__device__ __forceinline__ void affine_values(const void* p, int32_t f32, uint32_t c, float none, float* v) {
  if (p == nullptr) {
#pragma unroll
    for (int i = 0; i < U; ++i) v[i] = none;
  } else if (f32) {
#pragma unroll
    for (int i = 0; i < U; i += 4) {
      Raw<true, 4> r;
      r.load(p, c + i);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[i + k] = r.value(k);
    }
  } else {
    Raw<false, U> r;
    r.load(p, c);
#pragma unroll
    for (int i = 0; i < U; ++i) v[i] = r.value(i);
  }
}

// The sum over 16 neighbouring lanes or a wave, in every one of them: within 16
// lanes, then lane 15 of a row of lanes to the next one and lane 31 to the upper
// half.
template <int CTRL, int ROWS>
__device__ __forceinline__ float moved(float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, int(__float_as_uint(v)), CTRL, ROWS, 0xF, true));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double moved(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = uint32_t(__builtin_amdgcn_update_dpp(0, int(b), CTRL, ROWS, 0xF, true));
  const uint32_t hi = uint32_t(__builtin_amdgcn_update_dpp(0, int(b >> 32), CTRL, ROWS, 0xF, true));
  return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}
__device__ __forceinline__ float last_lane(float v) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}
__device__ __forceinline__ double last_lane(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, uint64_t(uint32_t(__builtin_amdgcn_readlane(uint32_t(b >> 32), 63))) << 32 |
                                        uint32_t(__builtin_amdgcn_readlane(uint32_t(b), 63)));
}
template <int LANES, typename T>
__device__ __forceinline__ T lanes_sum(T v) {
  v += moved<0xB1, 0xF>(v);   // lane ^ 1
  v += moved<0x4E, 0xF>(v);   // lane ^ 2
  v += moved<0x141, 0xF>(v);  // the other four of eight
  v += moved<0x140, 0xF>(v);  // the other eight of sixteen
  if constexpr (LANES == 16) return v;
  v += moved<0x142, 0xA>(v);
  v += moved<0x143, 0xC>(v);
  return last_lane(v);
}

// N sums over the threads that share a row, in every one of them.  `turn` alternates
// between two sets of words, so that one barrier a sum is enough; it waits for LDS
// only, not for the rows on their way.
template <int SHARE>
struct RowSum {
  static constexpr int kWaves = SHARE < 64 ? 1 : SHARE / 64;
  double (*words)[2][kWaves];
  int turn = 0;

  template <int N, typename T>
  __device__ __forceinline__ void operator()(T* v) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = lanes_sum<SHARE < 64 ? SHARE : 64>(v[k]);
    if constexpr (kWaves > 1) {
      T(*w)[kWaves] = reinterpret_cast<T(*)[kWaves]>(words[turn]);
      if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int k = 0; k < N; ++k) w[k][wave_index()] = v[k];
      }
      lds_barrier();
#pragma unroll
      for (int k = 0; k < N; ++k) {
        v[k] = w[k][0];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) v[k] += w[k][i];
      }
      turn ^= 1;
    }
  }
};

// SHARE threads share a row of up to SHARE * U * J values; a workgroup of BLOCK
// threads walks BLOCK / SHARE rows at a time.
template <int SHARE>
constexpr int kBlock = SHARE < 256 ? 256 : SHARE;

// A mean in two parts, and 1 / sqrt(var + eps).
struct Stats {
  float mean, rest, rstd;
};
__device__ __forceinline__ Stats mean_of(double sum, double per_value) {
  const double m = sum * per_value;
  const float mean = float(m);
  // (infinite or NaN: nothing is left)
  return Stats{mean, float(m - double(mean)), 0.0f};
}
// From the mean square around m.mean, whose own mean is m.rest.
__device__ __forceinline__ float rstd_of(float square, float rest, float eps) {
  const float var = square - rest * rest;
  return 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + eps);
}

// The same for all lanes of a wave but where they share several rows.
template <int SHARE>
__device__ __forceinline__ int64_t first_row() {
  static_assert(SHARE == 16 || SHARE == 64 || SHARE == kBlock<SHARE>, "rows of a workgroup");
  if constexpr (SHARE == 16) return int64_t(blockIdx.x) * (kBlock<SHARE> / SHARE) + threadIdx.x / SHARE;
  return SHARE == 64 ? int64_t(blockIdx.x) * (kBlock<SHARE> / SHARE) + wave_index() : int64_t(blockIdx.x);
}

template <int SHARE>
__device__ __forceinline__ char* row_at(const void* p, int64_t bytes) {
  const char* row = static_cast<const char*>(p) + bytes;
  return const_cast<char*>(SHARE < 64 ? row : uniform(row));
}

// One row after another through SETS sets of registers: use(k, row) is called
// for every row of this thread with the set that fetch(k, row) filled, SETS - 1
// rows ahead.
template <int SETS, typename F, typename U>
__device__ __forceinline__ void walk(int64_t r, int64_t step, int64_t rows, F fetch, U use) {
  constexpr int kAhead = SETS - 1;
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (r + k * step < rows) fetch(k, r + k * step);
  while (r < rows) {
#pragma unroll
    for (int k = 0; k < SETS; ++k) {
      if (r + kAhead * step < rows) fetch((k + kAhead) % SETS, r + kAhead * step);
      if (r < rows) use(k, r);
      r += step;
    }
  }
}
// Two sets of that many registers where three would be more than `most`.
constexpr int sets_of(int words, int most) { return 3 * words > most ? 2 : 3; }

template <bool XF32, bool YF32, int SHARE, int J>
__global__ __launch_bounds__(kBlock<SHARE>) void layer_norm_kernel(NormArgs a) {
  constexpr int U = XF32 || YF32 ? 4 : 8, kRows = kBlock<SHARE> / SHARE;
  __shared__ double words[2][2][RowSum<SHARE>::kWaves];
  RowSum<SHARE> sum{words};
  const int t = threadIdx.x % SHARE;
  const double per_value = 1.0 / double(a.cols);
  float w[J * U], b[J * U];
  Columns at[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    at[j] = columns_of<U, SHARE>(a.cols, j, t);
    affine_values<U>(a.weight, a.affine_f32, at[j].first, 1.0f, w + j * U);
    affine_values<U>(a.bias, a.affine_f32, at[j].first, 0.0f, b + j * U);
  }
  constexpr int kSet = sets_of(J * Raw<XF32, U>::kWords, 96);
  Raw<XF32, U> x[kSet][J];
  walk<kSet>(
      first_row<SHARE>(), int64_t(gridDim.x) * kRows, a.rows,
      [&](int set, int64_t row) {
        const char* p = row_at<SHARE>(a.x, row * a.x_ld * kSize<XF32>);
#pragma unroll
        for (int j = 0; j < J; ++j)
          if (at[j].again < U) x[set][j].load(p, at[j].first);
      },
      [&](int set, int64_t row) {
        // a row's threads leave together: with more than one wave a row, a workgroup has one
        // add(sum, value) over a thread's values, piece by piece
        auto sum_of = [&](auto none, auto add) {
          auto s = none;
#pragma unroll
          for (int j = 0; j < J; ++j) {
            auto piece = none;
            if (at[j].again == 0) {
#pragma unroll
              for (int i = 0; i < U; ++i) piece = add(piece, x[set][j].value(i));
            } else if (at[j].again < U) {
#pragma unroll
              for (int i = 1; i < U; ++i)
                if (i >= at[j].again) piece = add(piece, x[set][j].value(i));
            }
            s += piece;
          }
          return s;
        };
        // (of bf16 in fp64 65536 rows of 2048 take 107 us instead of 105)
        double total[1];
        if constexpr (XF32)
          total[0] = sum_of(0.0, [](double s, float v) { return s + double(v); });
        else
          total[0] = 32.0 * double(sum_of(0.0f, [](float s, float v) { return fmaf(v, 1.0f / 32.0f, s); }));
        sum.template operator()<1>(total);
        Stats m = mean_of(total[0], per_value);
        float square[1] = {sum_of(0.0f, [&](float s, float v) {
          const float d = v - m.mean;
          return s + d * d;
        })};
        sum.template operator()<1>(square);
#pragma unroll
        for (int j = 0; j < J; ++j) x[set][j].renewed();
        m.rstd = rstd_of(square[0] / float(a.cols), m.rest, a.eps);
        const float back = -m.rest * m.rstd;
        char* out = row_at<SHARE>(a.out, row * a.out_ld * kSize<YF32>);
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (at[j].again == U) continue;
          float y[U];
#pragma unroll
          for (int i = 0; i < U; ++i)
            y[i] = fmaf(fmaf(x[set][j].value(i) - m.mean, m.rstd, back), w[j * U + i], b[j * U + i]);
          Raw<YF32, U> v;
          v.set(y);
          v.store(out, at[j].first);
        }
        if (t == 0) {
          if (a.mean) a.mean[row] = m.mean;
          if (a.rstd) a.rstd[row] = m.rstd;
        }
      });
}

template <bool XF32, bool YF32, int SHARE, int J>
__global__ __launch_bounds__(kBlock<SHARE>, 4) void layer_norm_grad_kernel(NormArgs a) {
  constexpr int U = XF32 || YF32 ? 4 : 8, kRows = kBlock<SHARE> / SHARE;
  __shared__ double words[2][2][RowSum<SHARE>::kWaves];
  RowSum<SHARE> sum{words};
  const int t = threadIdx.x % SHARE;
  const float per_value = 1.0f / float(a.cols);
  float w[J * U], dw[J * U], db[J * U];
  Columns at[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    at[j] = columns_of<U, SHARE>(a.cols, j, t);
    affine_values<U>(a.weight, a.affine_f32, at[j].first, 1.0f, w + j * U);
#pragma unroll
    for (int i = 0; i < U; ++i) dw[j * U + i] = db[j * U + i] = 0.0f;
  }
  // (1024 threads' rows of more than 8192 columns with fp32 are not fetched ahead: 4096
  // of 12288 114 us instead of 123, of 14336 138 instead of 300, which spills)
  constexpr int kSet = SHARE == 1024 && U == 4 && J > 2
                           ? 1
                           : sets_of(J * (Raw<XF32, U>::kWords + Raw<YF32, U>::kWords), 24);
  Raw<XF32, U> x[kSet][J];
  Raw<YF32, U> y[kSet][J];
  float mean[kSet], rstd[kSet];
  walk<kSet>(
      first_row<SHARE>(), int64_t(gridDim.x) * kRows, a.rows,
      [&](int set, int64_t row) {
        const char* px = row_at<SHARE>(a.x, row * a.x_ld * kSize<XF32>);
        const char* py = row_at<SHARE>(a.dy, row * a.dy_ld * kSize<YF32>);
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (at[j].again == U) continue;
          x[set][j].load(px, at[j].first);
          y[set][j].load(py, at[j].first);
        }
        mean[set] = a.mean[row];
        rstd[set] = a.rstd[row];
      },
      [&](int set, int64_t row) {
        float s = 0.0f, sx = 0.0f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (at[j].again == U) continue;
          float gs = 0.0f, gx = 0.0f;
#pragma unroll
          for (int i = 0; i < U; ++i) {
            const int k = j * U + i;
            const float dy = y[set][j].value(i), xh = (x[set][j].value(i) - mean[set]) * rstd[set], g = dy * w[k];
            dw[k] = fmaf(dy, xh, dw[k]);
            db[k] += dy;
            gs += g;
            gx = fmaf(g, xh, gx);
          }
          if (at[j].again > 0) {
            gs = gx = 0.0f;
#pragma unroll
            for (int i = 1; i < U; ++i) {
              if (i < at[j].again) continue;
              const float g = y[set][j].value(i) * w[j * U + i];
              gs += g;
              gx = fmaf(g, (x[set][j].value(i) - mean[set]) * rstd[set], gx);
            }
          }
          s += gs;
          sx += gx;
          __builtin_amdgcn_sched_barrier(0);
        }
        float both[2] = {s, sx};
        sum.template operator()<2>(both);
        // (kept from above, the values would take twice the rows' registers)
#pragma unroll
        for (int j = 0; j < J; ++j) {
          x[set][j].renewed();
          y[set][j].renewed();
        }
        s = both[0] * per_value;
        sx = -both[1] * per_value;
        char* out = row_at<SHARE>(a.out, row * a.out_ld * kSize<XF32>);
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (at[j].again == U) continue;
          float d[U];
#pragma unroll
          for (int i = 0; i < U; ++i) {
            const float xh = (x[set][j].value(i) - mean[set]) * rstd[set];
            d[i] = rstd[set] * fmaf(xh, sx, fmaf(y[set][j].value(i), w[j * U + i], -s));
          }
          Raw<XF32, U> v;
          v.set(d);
          v.store(out, at[j].first);
          __builtin_amdgcn_sched_barrier(0);
        }
      });
  if (a.partial == nullptr) return;
  float* p = a.partial + int64_t(blockIdx.x) * 2 * a.cols;
  if constexpr (kRows > 1) {
    // the sums of a wave's rows, then those of the waves, one after the other
    if constexpr (SHARE < 64) {
#pragma unroll
      for (int k = 0; k < J * U; ++k)
#pragma unroll
        for (int lanes = SHARE; lanes < 64; lanes *= 2) {
          dw[k] += __shfl_xor(dw[k], lanes);
          db[k] += __shfl_xor(db[k], lanes);
        }
    }
    __shared__ float all[2 * SHARE * U * J];
    constexpr int kWaves = kBlock<SHARE> / 64;
    for (int turn = 0; turn < kWaves; ++turn) {
      if (int(threadIdx.x) / 64 == turn && int(threadIdx.x) % 64 < SHARE) {
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
    if (int(threadIdx.x) / 64 != kWaves - 1 || int(threadIdx.x) % 64 >= SHARE) return;
  }
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (i >= at[j].again) {
        const uint32_t c = at[j].first + i;
        p[c] = dw[j * U + i];
        p[a.cols + c] = db[j * U + i];
      }
}

// The sums of dw and db over the workgroups: kSlices threads a column, each
// adding its share of the workgroups in order, then one the shares.
constexpr int kSlices = 16, kJoinCols = 64, kAtOnce = 16;  // loads on their way
__global__ __launch_bounds__(kSlices* kJoinCols) void join_affine_kernel(const float* partial, int64_t groups,
                                                                         int64_t cols, void* dw, void* db,
                                                                         int32_t f32, int32_t accumulate) {
  __shared__ float part[2][kSlices][kJoinCols];
  const int k = threadIdx.x % kJoinCols, slice = threadIdx.x / kJoinCols;
  const int64_t c = int64_t(blockIdx.x) * kJoinCols + k;
  float a = 0.0f, b = 0.0f;
  if (c < cols) {
    const int64_t per = (groups + kSlices - 1) / kSlices, g0 = slice * per, g1 = g0 + per < groups ? g0 + per : groups;
    const float* p = partial + g0 * 2 * cols + c;
    int64_t left = g1 - g0;
    for (; left > 0; left -= kAtOnce, p += kAtOnce * 2 * cols) {
      float v[kAtOnce], w[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int64_t at = (i < left ? i : 0) * 2 * cols;
        v[i] = p[at];
        w[i] = p[at + cols];
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        a += i < left ? v[i] : 0.0f;
        b += i < left ? w[i] : 0.0f;
      }
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
  __shared__ double words[2][2][kWideBlock / 64];
  RowSum<kWideBlock> sum{words};
  const double per_value = 1.0 / double(a.cols);
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const char* x = static_cast<const char*>(a.x) + r * a.x_ld * kSize<XF32>;
    char* out = static_cast<char*>(a.out) + r * a.out_ld * kSize<YF32>;
    auto each = [&](auto f) {
      for (int64_t c = int64_t(threadIdx.x) * kWideU; c < a.cols; c += kWideBlock * kWideU) {
        const int left = a.cols - c < kWideU ? int(a.cols - c) : kWideU;
        Raw<XF32, kWideU> v;
        v.load_some(x, c, left);
        f(v, c, left);
      }
    };
    // a row may be long: the threads' own sums are fp64 too
    double total[1] = {0.0};
    each([&](const Raw<XF32, kWideU>& v, int64_t, int) {
#pragma unroll
      for (int i = 0; i < kWideU; ++i) total[0] += double(v.value(i));
    });
    sum.template operator()<1>(total);
    Stats m = mean_of(total[0], per_value);
    total[0] = 0.0;
    each([&](const Raw<XF32, kWideU>& v, int64_t, int left) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < kWideU; ++i) {
        const float d = v.value(i) - m.mean;
        if (i < left) s += d * d;
      }
      total[0] += double(s);
    });
    sum.template operator()<1>(total);
    m.rstd = rstd_of(float(total[0] * per_value), m.rest, a.eps);
    each([&](const Raw<XF32, kWideU>& v, int64_t c, int left) {
      float y[kWideU];
#pragma unroll
      for (int i = 0; i < kWideU; ++i)
        y[i] = i < left ? (v.value(i) - m.mean - m.rest) * m.rstd * affine(a.weight, a.affine_f32, c + i, 1.0f) +
                              affine(a.bias, a.affine_f32, c + i, 0.0f)
                        : 0.0f;
      Raw<YF32, kWideU> o;
      o.set(y);
      o.store_some(out, c, left);
    });
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[r] = m.mean;
      if (a.rstd) a.rstd[r] = m.rstd;
    }
  }
}

template <bool XF32, bool YF32>
__global__ __launch_bounds__(kWideBlock) void wide_norm_grad_kernel(NormArgs a) {
  __shared__ double words[2][2][kWideBlock / 64];
  RowSum<kWideBlock> sum{words};
  const double per_value = 1.0 / double(a.cols);
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
        vx.load_some(x, c, left);
        vy.load_some(dy, c, left);
        float xh[kWideU], g[kWideU];
#pragma unroll
        for (int i = 0; i < kWideU; ++i) {
          xh[i] = i < left ? (vx.value(i) - mean) * rstd : 0.0f;
          g[i] = i < left ? vy.value(i) * affine(a.weight, a.affine_f32, c + i, 1.0f) : 0.0f;
        }
        f(xh, g, c, left);
      }
    };
    double both[2] = {0.0, 0.0};
    each([&](const float* xh, const float* g, int64_t, int) {
      float s = 0.0f, sx = 0.0f;
#pragma unroll
      for (int i = 0; i < kWideU; ++i) {
        s += g[i];
        sx += g[i] * xh[i];
      }
      both[0] += double(s);
      both[1] += double(sx);
    });
    sum.template operator()<2>(both);
    const float s = float(both[0] * per_value), sx = float(both[1] * per_value);
    each([&](const float* xh, const float* g, int64_t c, int left) {
      float d[kWideU];
#pragma unroll
      for (int i = 0; i < kWideU; ++i) d[i] = rstd * (g[i] - s - xh[i] * sx);
      Raw<XF32, kWideU> o;
      o.set(d);
      o.store_some(out, c, left);
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

// As few threads a row as hold it in so many values each that several rows are worked
// on in a CU and few threads wait for each other.  That many are 32, 16 of 16 lanes'
// and a wave's, and for the gradients, which hold three more values for each, 16 of
// bf16 and 12 where there is fp32: 16 spill (8192 fp32 rows of 4096 116 us instead of
// 74, 4096 of 8192 124 instead of 79).  16 lanes have 8 of the gradients' (65536 rows of
// 200 126 us with 16 and 34 by a wave).  By 16 lanes 262144 rows of 128 take 28 us, by
// a wave 79, their gradients 45 and 75.  1024 threads have 16 of either (4096
// fp32 rows of 14336 138 us; by loops 376).
// A workgroup of the gradients leaves two fp32 sums a column, so there is at most one
// for 64 rows, for 32 where a wave or all of it shares a row (one for 16: 16384 rows
// of 2048 84 us instead of 74), but one a CU; and no more than 512 of 256 threads (1024
// of 16 lanes' a row: 65536 bf16 rows of 2048 149 us and not 167 with 1024 of them, 32768
// of 8192 by 512 threads 282 and not 292 with 512, 262144 of 128 by 16 lanes 46 and 50
// with 512).  The forward pass has 512 too, whose threads start seldom, where a thread
// has enough values on its way (8191 fp32 rows of 5120 42 us, 47 with 1024, 55 with 256),
// and 1024 where it has 8 at most (65536 bf16 rows of 2048 104 us, 143 with 512).
Shape shape_of(const LayerNormCall& c, bool grad) {
  const int64_t u = c.x_f32 || c.y_f32 ? 4 : 8;
  Shape s{0, 0, 0};
  for (int share : {16, 64, 256, 512, 1024}) {
    const int64_t most = (!grad ? share <= 64 ? 16 : 32 : share == 16 ? 8 : u == 4 && share < 1024 ? 12 : 16) / u;
    if (!grad && share == 1024) break;
    if (c.cols >= u && c.cols <= share * u * most) {
      s.share = share;
      s.j = int((c.cols + share * u - 1) / (share * u));
      break;
    }
  }
  if (s.share == 0) {
    s.groups = c.rows < 512 ? c.rows : 512;
    return s;
  }
  const int64_t block = s.share < 256 ? 256 : s.share, at_once = block / s.share;
  const int64_t need = (c.rows + at_once - 1) / at_once;
  int64_t most = ((grad ? s.share > 16 : s.j * u > 8) ? 512 : 1024) * 256 / block;
  if (grad) {
    const int64_t each = s.share == 16 ? 4 : s.share == 64 ? 8 : 32;
    if (most > need / each) most = need / each;
    if (most < 256) most = 256;
  }
  s.groups = need < most ? need : most;
  return s;
}

template <bool XF32, bool YF32>
int launch_wide(const LayerNormCall& c, const Shape& s, const NormArgs& a, bool grad, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(s.groups));
  if (!grad) {
    hipLaunchKernelGGL((wide_norm_kernel<XF32, YF32>), grid, dim3(kWideBlock), 0, st, a);
    return int(hipGetLastError());
  }
  hipLaunchKernelGGL((wide_norm_grad_kernel<XF32, YF32>), grid, dim3(kWideBlock), 0, st, a);
  const int rc = int(hipGetLastError());
  if (rc != 0 || a.partial == nullptr) return rc;
  hipLaunchKernelGGL((wide_affine_kernel<XF32, YF32>), dim3(unsigned((c.cols + 255) / 256), unsigned(s.groups)),
                     dim3(256), 0, st, a);
  return int(hipGetLastError());
}

template <bool XF32, bool YF32>
int launch(const LayerNormCall& c, const Shape& s, const NormArgs& a, bool grad, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(s.groups));
  if (s.share == 0) return launch_wide<XF32, YF32>(c, s, a, grad, st);
  constexpr int kPer = XF32 || YF32 ? 2 : 1;  // pieces of 8 values
  constexpr int kMore = kPer == 2 ? 3 : 2;
#define TIDE_NORM(KERNEL, SHARE, J) hipLaunchKernelGGL((KERNEL<XF32, YF32, SHARE, J>), grid, dim3(kBlock<SHARE>), 0, st, a)
  if (grad) {
    if (s.share == 16)
      TIDE_NORM(layer_norm_grad_kernel, 16, kPer);
    else if (s.share == 64 && s.j <= kPer)
      TIDE_NORM(layer_norm_grad_kernel, 64, kPer);
    else if (s.share == 64)
      TIDE_NORM(layer_norm_grad_kernel, 64, kMore);
    else if (s.share == 256 && s.j <= kPer)
      TIDE_NORM(layer_norm_grad_kernel, 256, kPer);
    else if (s.share == 256)
      TIDE_NORM(layer_norm_grad_kernel, 256, kMore);
    else if (s.share == 512 && s.j <= kPer)
      TIDE_NORM(layer_norm_grad_kernel, 512, kPer);
    else if (s.share == 512)
      TIDE_NORM(layer_norm_grad_kernel, 512, kMore);
    else if (s.j <= kPer)
      TIDE_NORM(layer_norm_grad_kernel, 1024, kPer);
    else if (s.j <= kMore)
      TIDE_NORM(layer_norm_grad_kernel, 1024, kMore);
    else
      TIDE_NORM(layer_norm_grad_kernel, 1024, 2 * kPer);
  } else {
    if (s.share == 16 && s.j <= kPer)
      TIDE_NORM(layer_norm_kernel, 16, kPer);
    else if (s.share == 16)
      TIDE_NORM(layer_norm_kernel, 16, 2 * kPer);
    else if (s.share == 64 && s.j <= kPer)
      TIDE_NORM(layer_norm_kernel, 64, kPer);
    else if (s.share == 64)
      TIDE_NORM(layer_norm_kernel, 64, 2 * kPer);
    else if (s.share == 512)
      TIDE_NORM(layer_norm_kernel, 512, 4 * kPer);
    else if (s.j <= kPer)
      TIDE_NORM(layer_norm_kernel, 256, kPer);
    else if (s.j <= 2 * kPer)
      TIDE_NORM(layer_norm_kernel, 256, 2 * kPer);
    else if (s.j <= 3 * kPer)
      TIDE_NORM(layer_norm_kernel, 256, 3 * kPer);
    else
      TIDE_NORM(layer_norm_kernel, 256, 4 * kPer);
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
