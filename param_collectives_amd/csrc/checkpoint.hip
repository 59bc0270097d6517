// Activation checkpoints in 8 bits on MI355X (gfx950): a row-major bf16 or
// fp32 matrix is kept as one byte of code per value and one exponent byte per
// block of 32 values of a row, and restored from them.
//
// A block's exponent byte b stands for 2^(b - 127), the smallest power of two
// u with max |x| <= 448 u (e4m3 codes) or <= 127.5 u (int8 codes), b held in
// [10, 246] or [10, 248]; a value's code is x / u rounded to nearest even and
// saturated at 448 or 127.  The division is exact, so each value has this one
// rounding: at most 2^-4 of the value (or u 2^-10) for e4m3, half of u for
// int8.  A block that holds a NaN or an infinity gets b = 255 and comes back
// as NaN.  b >= 10 keeps every non-zero u q a normal bf16 number, so restoring
// rounds nothing, in bf16 either.
//
// Both kernels are bound by HBM.  A lane takes 16 bytes of values, 8 of bf16 or
// 4 of fp32, and 4 or 8 lanes a block, whose maximum goes through two or three
// cross-lane steps.  The values are read and written with the non-temporal hint
// (they pass once), so every access has to cover whole lines.  Measured from
// cold caches: 8192 x 14336 bf16 packed and restored in 108 us, 6.6 TB/s (138 us
// with plain accesses), 4095 x 5120 fp32 in 34 us, 6.2 TB/s (47 us; 54 us with
// the hint and 8 fp32 values a lane).  Rows that do not start on 16 bytes are
// accessed the same way: 8192 x 14335 bf16 packed in 61 us and restored in 53
// (141 and 168 us one value at a time).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gemm.h"
#include "training.h"

namespace {

using namespace tide;

template <bool F32>
constexpr int kUnit = F32 ? 4 : 8;  // values of a lane
template <bool F32>
constexpr int kSweeps = F32 ? 4 : 2;  // units of a thread
constexpr uint32_t kLowest = 10, kNotFinite = 255;

struct PackArgs {
  void* x;
  int64_t ld;
  uint8_t* codes;
  uint8_t* scales;
  int64_t units;       // of the matrix
  uint32_t row_units;  // of a row, whole blocks
  uint64_t magic;      // ceil(2^44 / row_units)
  int32_t cols;
};

// Row and unit of the row of this thread's unit `i` of the workgroup that
// starts at unit `first`.
__device__ __forceinline__ void locate(const PackArgs& a, int64_t first_row, uint32_t first_unit, uint32_t i,
                                       int64_t* row, uint32_t* unit) {
  // n is below row_units + 2^11 and row_units at most 2^20: the product is
  // below 2^55 and the quotient exact
  const uint32_t n = first_unit + i;
  const uint32_t q = uint32_t((uint64_t(n) * a.magic) >> 44);
  *row = first_row + q;
  *unit = n - q * a.row_units;
}

template <bool F32>
__device__ __forceinline__ void load_unit(const void* x, int64_t at, int left, float* v) {
  if constexpr (F32) {
    const float* p = static_cast<const float*>(x) + at;
    if (left >= 4) {
      const f32x4v w = __builtin_nontemporal_load(reinterpret_cast<const any_f32x4*>(p));
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = w[j];
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = j < left ? p[j] : 0.0f;
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(x) + at;
    if (left >= 8) {
      const u32x4 w = __builtin_nontemporal_load(reinterpret_cast<const any_u32x4*>(p));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = j < left ? __uint_as_float(uint32_t(p[j]) << 16) : 0.0f;
    }
  }
}

// The largest value of this lane's group of 4 (EIGHT: 8) lanes.
template <bool EIGHT>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  uint32_t o = uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0xB1, 0xF, 0xF, true));  // lanes 1 0 3 2
  v = v > o ? v : o;
  o = uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0x4E, 0xF, 0xF, true));  // lanes 2 3 0 1
  v = v > o ? v : o;
  if constexpr (EIGHT) {
    o = uint32_t(__builtin_amdgcn_mov_dpp(int(v), 0x141, 0xF, 0xF, true));  // lanes 7 6 5 4 3 2 1 0
    v = v > o ? v : o;
  }
  return v;
}

template <Code CODE>
__device__ __forceinline__ uint32_t exponent_byte(uint32_t top) {
  // top: the bits of the block's largest magnitude, 1.f 2^(e - 127)
  constexpr uint32_t kShift = CODE == Code::kE4m3 ? 8 : 6;                      // 448 = 1.75 2^8, 127.5 = 1.992.. 2^6
  constexpr uint32_t kLimit = CODE == Code::kE4m3 ? 0x600000u : 0x7F0000u;      // their fractions
  constexpr uint32_t kHighest = CODE == Code::kE4m3 ? 246u : 248u;
  if (top >= 0x7F800000u) return kNotFinite;
  int32_t b = int32_t(top >> 23) - int32_t(kShift) + ((top & 0x7FFFFFu) > kLimit ? 1 : 0);
  b = b > int32_t(kLowest) ? b : int32_t(kLowest);
  return uint32_t(b) < kHighest ? uint32_t(b) : kHighest;
}

template <bool F32, Code CODE>
__global__ __launch_bounds__(256) void checkpoint_pack_kernel(PackArgs a) {
  constexpr int U = kUnit<F32>, S = kSweeps<F32>, kWords = U / 4;
  const int64_t base = int64_t(blockIdx.x) * (256 * S);
  const int64_t row0 = base / a.row_units;
  const uint32_t unit0 = uint32_t(base - row0 * a.row_units);
  float v[S][U];
  int64_t row[S];
  uint32_t unit[S];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const uint32_t i = s * 256 + threadIdx.x;
    locate(a, row0, unit0, i, &row[s], &unit[s]);
    const int c = int(unit[s]) * U;
    // lanes past the end (whole blocks of them) read nothing
    load_unit<F32>(a.x, row[s] * a.ld + c, base + i < a.units ? a.cols - c : 0, v[s]);
  }
#pragma unroll
  for (int s = 0; s < S; ++s) {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const uint32_t m = __float_as_uint(v[s][j]) & 0x7FFFFFFFu;
      top = top > m ? top : m;
    }
    const uint32_t b = exponent_byte<CODE>(group_max<F32>(top));
    const float r = __uint_as_float((254u - (b == kNotFinite ? kLowest : b)) << 23);  // 2^(127 - b)
    uint32_t w[kWords];
#pragma unroll
    for (int h = 0; h < kWords; ++h) {
      float y[4];
      constexpr float kTop = CODE == Code::kE4m3 ? 448.0f : 127.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = __builtin_amdgcn_fmed3f(v[s][4 * h + j] * r, -kTop, kTop);
      if constexpr (CODE == Code::kE4m3) {
        int p = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
        w[h] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], p, true));
        if (b == kNotFinite) w[h] = 0x7F7F7F7Fu;
      } else {
        // 1.5 2^23 + y rounds y to an integer (to nearest even) in the low byte
        uint32_t q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = __float_as_uint(y[j] + 12582912.0f);
        const uint32_t lo = __builtin_amdgcn_perm(q[1], q[0], 0x0C0C0400u);
        const uint32_t hi = __builtin_amdgcn_perm(q[3], q[2], 0x04000C0Cu);
        w[h] = b == kNotFinite ? 0u : lo | hi;
      }
    }
    if (base + s * 256 + threadIdx.x < a.units) {
      uint8_t* to = a.codes + (row[s] * a.row_units + unit[s]) * U;
      if constexpr (F32)
        *reinterpret_cast<uint32_t*>(to) = w[0];
      else
        *reinterpret_cast<u32x2*>(to) = u32x2{w[0], w[kWords - 1]};
      if (unit[s] % (32 / U) == 0) a.scales[row[s] * (a.row_units / (32 / U)) + unit[s] / (32 / U)] = uint8_t(b);
    }
  }
}

template <bool F32, Code CODE>
__global__ __launch_bounds__(256) void checkpoint_unpack_kernel(PackArgs a) {
  constexpr int U = kUnit<F32>, S = kSweeps<F32>, kWords = U / 4;
  const int64_t base = int64_t(blockIdx.x) * (256 * S);
  const int64_t row0 = base / a.row_units;
  const uint32_t unit0 = uint32_t(base - row0 * a.row_units);
  uint32_t w[S][kWords];
  uint32_t b[S];
  int64_t row[S];
  uint32_t unit[S];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const uint32_t i = s * 256 + threadIdx.x;
    locate(a, row0, unit0, i, &row[s], &unit[s]);
    if (base + i < a.units) {
      const uint8_t* from = a.codes + (row[s] * a.row_units + unit[s]) * U;
      if constexpr (F32) {
        w[s][0] = *reinterpret_cast<const uint32_t*>(from);
      } else {
        const u32x2 p = *reinterpret_cast<const u32x2*>(from);
        w[s][0] = p[0];
        w[s][kWords - 1] = p[1];
      }
      b[s] = a.scales[row[s] * (a.row_units / (32 / U)) + unit[s] / (32 / U)];
    }
  }
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int c = int(unit[s]) * U;
    if (base + s * 256 + threadIdx.x >= a.units || c >= a.cols) continue;
    const int left = a.cols - c;
    const int64_t at = row[s] * a.ld + c;
    if constexpr (F32) {
      const u32x2 h = widen4<CODE>(w[s][0], b[s]);
      const f32x4v f = f32x4v{__uint_as_float(h[0] << 16), __uint_as_float(h[0] & 0xFFFF0000u),
                              __uint_as_float(h[1] << 16), __uint_as_float(h[1] & 0xFFFF0000u)};
      float* p = static_cast<float*>(a.x) + at;
      if (left >= 4) {
        __builtin_nontemporal_store(f, reinterpret_cast<any_f32x4*>(p));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < left) p[j] = f[j];
      }
    } else {
      const u32x2 lo = widen4<CODE>(w[s][0], b[s]), hi = widen4<CODE>(w[s][kWords - 1], b[s]);
      const u32x4 h = u32x4{lo.x, lo.y, hi.x, hi.y};
      uint16_t* p = static_cast<uint16_t*>(a.x) + at;
      if (left >= 8) {
        __builtin_nontemporal_store(h, reinterpret_cast<any_u32x4*>(p));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < left) p[j] = uint16_t(h[j >> 1] >> (16 * (j & 1)));
      }
    }
  }
}

template <bool PACK, bool F32, Code CODE>
void launch_as(const PackArgs& a, unsigned grid, hipStream_t st) {
  if constexpr (PACK)
    hipLaunchKernelGGL((checkpoint_pack_kernel<F32, CODE>), dim3(grid), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((checkpoint_unpack_kernel<F32, CODE>), dim3(grid), dim3(256), 0, st, a);
}

template <bool PACK>
int launch(const PackCall& c, void* stream) {
  PackArgs a;
  const int64_t blocks = (c.cols + kPackBlock - 1) / kPackBlock;
  a.x = const_cast<void*>(c.x);
  a.ld = c.ld;
  a.codes = static_cast<uint8_t*>(c.codes);
  a.scales = static_cast<uint8_t*>(c.scales);
  const int64_t unit = c.f32 ? kUnit<true> : kUnit<false>, sweep = 256 * (c.f32 ? kSweeps<true> : kSweeps<false>);
  a.row_units = uint32_t(blocks * (kPackBlock / unit));
  a.units = c.rows * int64_t(a.row_units);
  a.magic = ((uint64_t(1) << 44) + a.row_units - 1) / a.row_units;
  a.cols = int32_t(c.cols);
  const unsigned grid = unsigned((a.units + sweep - 1) / sweep);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (c.f32) {
    if (c.int8)
      launch_as<PACK, true, Code::kInt8>(a, grid, st);
    else
      launch_as<PACK, true, Code::kE4m3>(a, grid, st);
  } else {
    if (c.int8)
      launch_as<PACK, false, Code::kInt8>(a, grid, st);
    else
      launch_as<PACK, false, Code::kE4m3>(a, grid, st);
  }
  return int(hipGetLastError());
}

}  // namespace

namespace tide {

int launch_pack(const PackCall& c, void* stream) { return launch<true>(c, stream); }
int launch_unpack(const PackCall& c, void* stream) { return launch<false>(c, stream); }

}  // namespace tide
