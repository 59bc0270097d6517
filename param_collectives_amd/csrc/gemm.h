// The matrix-product core of the training-step operators (weight_grad.hip,
// vocab_loss.hip) on MI355X (gfx950): one workgroup computes a BM x BN tile of
//   C[m][n] = sum_k A(m, k) B(k, n)
// with bf16 operands and fp32 sums on the matrix cores (16x16x32 products).
//
// An operand is read in one of three forms:
//   Form::kRows    its rows are C's rows (columns), k runs along them;
//   Form::kCols    its rows are the values of k, C's rows (columns) run along
//                  them;
//   Form::kPacked  as kCols, in the packed 8-bit form (codes and one exponent
//                  byte per block of 32), widened while it is staged.
// Tiles go to LDS, kRows and kCols ones by loads that write LDS directly (16
// bytes a lane).  Those loads fill LDS in lane order, so the bank swizzle is
// made by choosing which 16 bytes a lane fetches:
//   kRows tile [rows][64 k], 8 chunks of 16 bytes a row: chunk c of row r is
//     kept at slot c ^ (r & 7), and the 16-byte fragment reads of 8
//     consecutive rows touch all 64 banks once;
//   kCols, kPacked tile [64 k][rows]: chunk c of row k is kept at
//     c ^ 2 f(k), f(k) made of bits 0, 1 and 3 of k; a fragment is read by the
//     transposing LDS read, whose 32 lanes touch 8 rows k of 32 bytes each.
// The products take the n side first, so a lane holds 4 consecutive n of one m.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace tide {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4v __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

#define TIDE_GLOBAL __attribute__((address_space(1)))
#define TIDE_LDS __attribute__((address_space(3)))

enum class Form { kRows, kCols, kPacked };
enum class Code { kE4m3, kInt8 };

constexpr int kBK = 64;  // k per staged step

struct Operand {
  const void* base;       // bf16 values, or codes (kPacked); 16-byte aligned
  const uint8_t* scales;  // kPacked: [k][scale_ld]
  int64_t ld;             // elements from row to row, a multiple of 8 (kPacked: of 32)
  int64_t scale_ld;
  int64_t extent;         // rows (columns) of C that exist on this side
};

// 8 zero values for the lanes whose k lies past the end.
static __device__ __align__(16) const uint32_t g_zero16[4] = {0, 0, 0, 0};

__device__ __forceinline__ void load_to_lds(const void* g, void* lds) {
  __builtin_amdgcn_global_load_lds((const TIDE_GLOBAL void*)g, (TIDE_LDS void*)lds, 16, 0, 0);
}

// Every load to LDS or registers of this wave has arrived (vmcnt(0) on gfx9;
// expcnt and lgkmcnt are left at their maxima).
__device__ __forceinline__ void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0F70); }

// The same for every lane: keeps a base address in scalar registers, apart
// from the lanes' offsets (the loads take both).
template <typename T>
__device__ __forceinline__ const T* uniform(const T* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(v)), hi = __builtin_amdgcn_readfirstlane(uint32_t(v >> 32));
  return reinterpret_cast<const T*>(uint64_t(hi) << 32 | lo);
}

// Makes a value new to the compiler: what is computed from it stays where it
// is written (hoisted out of the step loop, the addresses of two stages'
// fragments would not fit the registers).
__device__ __forceinline__ uint32_t renew(uint32_t& v) {
  asm("" : "+v"(v));
  return v;
}

__device__ __forceinline__ int wave_index() { return __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6); }

__device__ __forceinline__ int col_swizzle(int k) { return ((k & 3) | ((k >> 1) & 4)) << 1; }

__device__ __forceinline__ bf16x2 bits_as_bf16x2(uint32_t v) {
  bf16x2 r;
  __builtin_memcpy(&r, &v, 4);
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_as_bits(bf16x2 v) {
  uint32_t r;
  __builtin_memcpy(&r, &v, 4);
  return r;
}

// Four codes (the bytes of w) times 2^(scale byte - 127), as bf16.  The
// product is exact: a code has at most 7 significant bits and the packing
// keeps every value a normal bf16 number.  A scale byte of 255 gives NaN.
template <Code CODE>
__device__ __forceinline__ u32x2 widen4(uint32_t w, uint32_t scale_byte) {
  u32x2 r;
  if constexpr (CODE == Code::kE4m3) {
    const float s = __uint_as_float(scale_byte << 23);
    r.x = bf16x2_as_bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false));
    r.y = bf16x2_as_bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true));
  } else {
    const float s = __uint_as_float(scale_byte == 255u ? 0x7FC00000u : scale_byte << 23);
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = float(int32_t(w << (24 - 8 * i)) >> 24) * s;
    // exact values: their upper halves are the bf16 numbers
    r.x = __builtin_amdgcn_perm(__float_as_uint(f[1]), __float_as_uint(f[0]), 0x07060302u);
    r.y = __builtin_amdgcn_perm(__float_as_uint(f[3]), __float_as_uint(f[2]), 0x07060302u);
  }
  return r;
}

// One operand side of the tile: ROWS rows (columns) of C, FRAGS x 16 of them a
// wave's, THREADS threads.
template <Form FORM, Code CODE, int ROWS, int FRAGS, int THREADS>
struct Side {
  static constexpr int kBytes = ROWS * kBK * 2;
  static constexpr int kLoads = kBytes / 16 / THREADS;  // 16-byte loads of a thread per step
  static constexpr int kRowChunks = FORM == Form::kRows ? 8 : ROWS / 8;
  static constexpr int kUnits = ROWS / 16;                // kPacked: 16-code units of a row
  static constexpr int kPasses = kBK * kUnits / THREADS;  // kPacked: units of a thread per step

  const char* base;        // of the tile's first row (kRows) or column, k = 0
  const uint8_t* scales;
  int64_t step;            // bytes from one step of 64 k to the next
  int64_t scale_step;
  uint32_t off[FORM == Form::kPacked ? kPasses : kLoads];  // byte offset of each load at its step's base
  uint32_t scale_off[FORM == Form::kPacked ? kPasses : 1];
  u32x4 held[FORM == Form::kPacked ? kPasses : 1];  // kPacked: codes on their way to LDS
  uint32_t held_scale[FORM == Form::kPacked ? kPasses : 1];
  uint32_t put[FORM == Form::kPacked ? kPasses : 1];  // where each unit goes in the tile

  __device__ __forceinline__ void init(const Operand& o, int64_t first, int tid) {
    // rows (columns) past the end read the last one: their results are dropped
    const int64_t last = o.extent - 1 - first;
    if constexpr (FORM == Form::kRows) {
      base = static_cast<const char*>(o.base) + first * o.ld * 2;
      step = kBK * 2;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int lin = i * THREADS + tid, r = lin >> 3, c = (lin & 7) ^ (r & 7);
        const int rr = r <= last ? r : int(last);
        off[i] = uint32_t(rr) * uint32_t(o.ld * 2) + uint32_t(c * 16);
      }
    } else if constexpr (FORM == Form::kCols) {
      base = static_cast<const char*>(o.base) + first * 2;
      step = o.ld * (kBK * 2);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int lin = i * THREADS + tid, k = lin / kRowChunks, c = (lin % kRowChunks) ^ col_swizzle(k);
        off[i] = uint32_t(k) * uint32_t(o.ld * 2) + (c * 8 <= last ? uint32_t(c * 16) : 0u);
      }
    } else {
      base = static_cast<const char*>(o.base) + first;
      scales = o.scales + first / 32;
      step = o.ld * kBK;
      scale_step = o.scale_ld * kBK;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int lin = i * THREADS + tid, k = lin / kUnits, u = lin % kUnits;
        const bool in = u * 16 <= last;
        off[i] = uint32_t(k) * uint32_t(o.ld) + (in ? uint32_t(u * 16) : 0u);
        scale_off[i] = uint32_t(k) * uint32_t(o.scale_ld) + (in ? uint32_t(u >> 1) : 0u);
        put[i] = uint32_t((k * kRowChunks + ((2 * u) ^ col_swizzle(k))) * 16);
      }
    }
  }

  // Start the loads of step s into `lds` (kPacked: into registers).  TAIL:
  // only `left` < 64 values of k remain, the rest is staged as zeros (k
  // counts in eights on a kRows side, whose rows are zero from there to the
  // next multiple of 8).
  template <bool TAIL>
  __device__ __forceinline__ void fetch(char* lds, int64_t s, int left, int tid) {
    const char* at = uniform(base + s * step);
    if constexpr (FORM == Form::kPacked) {
      const uint8_t* sc = uniform(scales + s * scale_step);
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int k = (i * THREADS + tid) / kUnits;
        if (!TAIL || k < left) {
          held[i] = *(const TIDE_GLOBAL u32x4*)(at + renew(off[i]));
          held_scale[i] = *(const TIDE_GLOBAL uint8_t*)(sc + renew(scale_off[i]));
        } else {
          held[i] = u32x4{0, 0, 0, 0};
          held_scale[i] = 127;
        }
      }
    } else {
      const int wave_base = wave_index() * 64;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const char* src = at + renew(off[i]);
        if constexpr (TAIL) {
          const int lin = i * THREADS + tid;
          const int k = FORM == Form::kRows ? ((lin & 7) ^ ((lin >> 3) & 7)) * 8 : lin / kRowChunks;
          if (k >= left) src = reinterpret_cast<const char*>(g_zero16);
        }
        load_to_lds(src, lds + (i * THREADS + wave_base) * 16);
      }
    }
  }

  // kPacked: widen what fetch() loaded and write it to LDS.
  __device__ __forceinline__ void settle(char* lds, int tid) {
    if constexpr (FORM == Form::kPacked) {
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        char* to = lds + renew(put[i]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x2 lo = widen4<CODE>(held[i][2 * h], held_scale[i]);
          const u32x2 hi = widen4<CODE>(held[i][2 * h + 1], held_scale[i]);
          *reinterpret_cast<u32x4*>(to + 16 * h) = u32x4{lo.x, lo.y, hi.x, hi.y};
        }
      }
    }
  }

  // Where this lane's fragments of a wave's FRAGS x 16 rows (columns) from r0
  // (a multiple of 16 FRAGS) start in the tile.
  static constexpr int kSpots = FORM == Form::kRows ? 2 : FRAGS;
  static __device__ __forceinline__ void spots(uint32_t* at, int r0, int lane) {
    if constexpr (FORM == Form::kRows) {
      const int r = r0 + (lane & 15);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) at[kk] = uint32_t((r * 8 + ((4 * kk + (lane >> 4)) ^ (r & 7))) * 16);
    } else {
      // a transposing read gives lane l of 16 the values of column l in the
      // four rows k of which lanes 4j .. 4j+3 point at 4 columns each
      const int k = 8 * (lane >> 4) + ((lane & 15) >> 2);
#pragma unroll
      for (int i = 0; i < FRAGS; ++i) {
        const int col = r0 + 16 * i + 4 * (lane & 3);
        at[i] = uint32_t((k * kRowChunks + ((col >> 3) ^ col_swizzle(k))) * 16 + (col & 4) * 2);
      }
    }
  }

  // Fragment i: rows (columns) 16 i + 0..15, k = 32 kk + 8 (lane / 16) + 0..7.
  static __device__ __forceinline__ bf16x8 fragment(const char* lds, uint32_t* at, int i, int kk) {
    if constexpr (FORM == Form::kRows) {
      return *reinterpret_cast<const bf16x8*>(lds + renew(at[kk]) + i * 2048);
    } else {
      // rows k, k + 4 and k + 32 share their swizzle
      const char* p = lds + renew(at[i]) + kk * 32 * kRowChunks * 16;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TIDE_LDS s16x4*)p);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TIDE_LDS s16x4*)(p + 4 * kRowChunks * 16));
      bf16x8 r;
      __builtin_memcpy(&r, &lo, 8);
      __builtin_memcpy(reinterpret_cast<char*>(&r) + 8, &hi, 8);
      return r;
    }
  }
};

// The tile loop.  WM x WN waves, each holding an (BM / WM) x (BN / WN) part.
template <Form FA, Form FB, Code CODE, int BM, int BN, int WM, int WN>
struct Gemm {
  static constexpr int kThreads = WM * WN * 64;
  static constexpr int kFM = BM / WM / 16, kFN = BN / WN / 16;  // fragments of a wave
  using SA = Side<FA, CODE, BM, kFM, kThreads>;
  using SB = Side<FB, CODE, BN, kFN, kThreads>;
  static constexpr int kStage = SA::kBytes + SB::kBytes;
  static constexpr int kLds = 2 * kStage;

  f32x4v acc[kFM][kFN];
  int tid, lane, wm, wn;
  uint32_t at_a[SA::kSpots], at_b[SB::kSpots];

  __device__ __forceinline__ void multiply(const char* la, const char* lb) {
#pragma unroll
    for (int kk = 0; kk < kBK / 32; ++kk) {
      bf16x8 b[kFN];
#pragma unroll
      for (int j = 0; j < kFN; ++j) b[j] = SB::fragment(lb, at_b, j, kk);
#pragma unroll
      for (int i = 0; i < kFM; ++i) {
        const bf16x8 a = SA::fragment(la, at_a, i, kk);
#pragma unroll
        for (int j = 0; j < kFN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j], a, acc[i][j], 0, 0, 0);
      }
    }
  }

  // Sums k over [k_first, k_end) (k_first a multiple of 64) into acc.  `lds0`
  // and `lds1` hold kStage bytes each.
  __device__ __forceinline__ void run(const Operand& a, const Operand& b, int64_t m0, int64_t n0, int64_t k_first,
                                      int64_t k_end, char* lds0, char* lds1) {
    tid = threadIdx.x;
    lane = tid & 63;
    wm = wave_index() / WN;
    wn = wave_index() % WN;
#pragma unroll
    for (int i = 0; i < kFM; ++i)
#pragma unroll
      for (int j = 0; j < kFN; ++j) acc[i][j] = f32x4v{0.f, 0.f, 0.f, 0.f};
    if (k_end <= k_first) return;
    SA::spots(at_a, wm * (BM / WM), lane);
    SB::spots(at_b, wn * (BN / WN), lane);
    SA sa;
    SB sb;
    sa.init(a, m0, tid);
    sb.init(b, n0, tid);
    const int64_t s_first = k_first / kBK, whole = k_end / kBK;
    const int left = int(k_end - whole * kBK);
    auto settle = [&](char* lds) {
      sa.settle(lds, tid);
      sb.settle(lds + SA::kBytes, tid);
    };
    // A short last step goes first, so that the loop's steps are all whole;
    // the stage it takes makes the last step's the second.
    const int64_t steps = whole - s_first + (left ? 1 : 0);
    const bool even = (steps & 1) == 0;
    char* first_stage = even ? lds0 : lds1;
    int64_t s = s_first;
    if (left) {
      sa.template fetch<true>(first_stage, whole, left, tid);
      sb.template fetch<true>(first_stage + SA::kBytes, whole, left, tid);
    } else {
      sa.template fetch<false>(first_stage, s, 0, tid);
      sb.template fetch<false>(first_stage + SA::kBytes, s, 0, tid);
      ++s;
    }
    settle(first_stage);
    // One barrier a step: once past it, this step's tiles are in LDS and every
    // wave has read the other stage's tiles of the step before.
    auto one = [&](char* now, char* next) {
      wait_loads();
      __syncthreads();
      sa.template fetch<false>(next, s, 0, tid);
      sb.template fetch<false>(next + SA::kBytes, s, 0, tid);
      ++s;
      __builtin_amdgcn_sched_barrier(0);  // the loads start before the products
      multiply(now, now + SA::kBytes);
      settle(next);
    };
    if (even) one(lds0, lds1);
    while (s < whole) {
      one(lds1, lds0);
      one(lds0, lds1);
    }
    wait_loads();
    __syncthreads();
    multiply(lds1, lds1 + SA::kBytes);
  }

  // f(m, n, values of columns n .. n+3) for every group of four this wave
  // holds.  The groups pass through this wave's 16 rows of LDS (the stages are
  // free by then), so that 16 lanes hand over 64 neighbouring columns of a row.
  template <typename F>
  __device__ __forceinline__ void each(int64_t m0, int64_t n0, char* lds0, F f) {
    constexpr int kCols = BN / WN, kPitch = kCols + 4, kGroups = kCols / 4;
    static_assert(WM * WN * 16 * kPitch * 4 <= kStage, "epilogue rows");
    float* rows = reinterpret_cast<float*>(lds0) + wave_index() * 16 * kPitch;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kFM; ++i) {
#pragma unroll
      for (int j = 0; j < kFN; ++j)
        *reinterpret_cast<f32x4v*>(rows + (lane & 15) * kPitch + j * 16 + 4 * (lane >> 4)) = acc[i][j];
#pragma unroll 1
      for (int q = lane; q < 16 * kGroups; q += 64) {
        const int r = q / kGroups, c = (q % kGroups) * 4;
        f(m0 + wm * (BM / WM) + i * 16 + r, n0 + wn * kCols + c,
          *reinterpret_cast<const f32x4v*>(rows + r * kPitch + c));
      }
    }
  }
};

__device__ __forceinline__ uint32_t bf16_bits_of(float v) {
  const __bf16 b = __bf16(v);  // round to nearest even
  uint16_t r;
  __builtin_memcpy(&r, &b, 2);
  return r;
}

// alpha s (+ old) for the `n` values v of one row from element `at`, rounded
// once to the output's type (fp32 or bf16).
__device__ __forceinline__ void store_values(void* out, int32_t f32, int32_t accumulate, float alpha, int64_t at, int n,
                                           f32x4v v) {
  if (f32) {
    float* d = static_cast<float*>(out) + at;
    if (n == 4 && (reinterpret_cast<uintptr_t>(d) & 15) == 0) {
      f32x4v r;
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = alpha * v[i];
      if (accumulate) {
        const f32x4v old = *reinterpret_cast<const f32x4v*>(d);
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = old[i] + r[i];
      }
      *reinterpret_cast<f32x4v*>(d) = r;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) d[i] = accumulate ? d[i] + alpha * v[i] : alpha * v[i];
    }
  } else {
    uint16_t* d = static_cast<uint16_t*>(out) + at;
    if (n == 4 && (reinterpret_cast<uintptr_t>(d) & 7) == 0) {
      float r[4];
      u32x2 old = u32x2{0, 0};
      if (accumulate) old = *reinterpret_cast<const u32x2*>(d);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float o = __uint_as_float(i & 1 ? old[i >> 1] & 0xFFFF0000u : old[i >> 1] << 16);
        r[i] = accumulate ? o + alpha * v[i] : alpha * v[i];
      }
      *reinterpret_cast<u32x2*>(d) =
          u32x2{bf16_bits_of(r[0]) | bf16_bits_of(r[1]) << 16, bf16_bits_of(r[2]) | bf16_bits_of(r[3]) << 16};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) {
          const float r = alpha * v[i];
          d[i] = uint16_t(bf16_bits_of(accumulate ? __uint_as_float(uint32_t(d[i]) << 16) + r : r));
        }
    }
  }
}

// The splits' values of `n` elements from element `at`, added in order.
__device__ __forceinline__ f32x4v sum_splits(const float* partial, int32_t splits, int64_t elems, int64_t at, int n) {
  f32x4v s = f32x4v{0.f, 0.f, 0.f, 0.f};
  for (int32_t k = 0; k < splits; ++k) {
    const float* p = partial + int64_t(k) * elems + at;
    if (n == 4 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
      const f32x4v v = *reinterpret_cast<const f32x4v*>(p);
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] += v[j];
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < n) s[j] += p[j];
    }
  }
  return s;
}

// Workgroups go round-robin over the 8 XCDs, each with an L2 of its own: XCD x
// takes a contiguous share of the tiles, in an order that walks `group` tile
// rows before it moves to the next tile column, so that what an XCD works on
// at one time shares operand tiles.
__device__ __forceinline__ void tile_of(uint32_t bid, uint32_t tiles_m, uint32_t tiles_n, uint32_t group, uint32_t* tm,
                                        uint32_t* tn) {
  const uint32_t total = tiles_m * tiles_n, x = bid & 7, each = total >> 3, more = total & 7;
  const uint32_t t = x * each + (x < more ? x : more) + (bid >> 3);
  const uint32_t band = t / (group * tiles_n), in = t - band * group * tiles_n;
  const uint32_t rows = band * group + group <= tiles_m ? group : tiles_m - band * group;
  *tm = __builtin_amdgcn_readfirstlane(band * group + in % rows);
  *tn = __builtin_amdgcn_readfirstlane(in / rows);
}

}  // namespace tide
