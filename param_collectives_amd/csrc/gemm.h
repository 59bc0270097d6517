// The matrix-product core of the training-step operators (weight_grad.hip,
// vocab_loss.hip, gated_block.hip, orthogonalize.hip) on MI355X (gfx950): one
// workgroup computes a BM x BN tile of
//   C[m][n] = sum_k A(m, k) B(k, n)
// with bf16 (or, on request, fp16) operands and fp32 sums on the matrix cores
// (16x16x32 products).
//
// An operand is read in one of five forms:
//   Form::kRows    its rows are C's rows (columns), k runs along them;
//   Form::kPair    as kRows, from two matrices: a tile's first half of rows are
//                  the one's, the second half the same rows of the other, and a
//                  wave holds the products of both for its share of them;
//   Form::kCols    its rows are the values of k, C's rows (columns) run along
//                  them;
//   Form::kStack   as kCols, from two matrices: the values of k go on in the
//                  second after `split` steps;
//   Form::kPacked  as kCols, in the packed 8-bit form (codes and one exponent
//                  byte per block of 32), widened while it is staged.
// Tiles go to LDS, all but kPacked ones by loads that write LDS directly (16
// bytes a lane).  Those loads fill LDS in lane order, so the bank swizzle is
// made by choosing which 16 bytes a lane fetches:
//   kRows, kPair tile [rows][32 k], 4 chunks of 16 bytes a row: chunk c of row r is
//     kept at c ^ f(r), f(r) = -(r / 4) mod 4.  A 16-byte fragment read goes
//     through the 64 banks 16 lanes at a time, not neighbours but lanes 0-3,
//     12-15 and 20-27, then the rest of 0-31, and so on: f gives each such
//     group 16 different places (r / 4 mod 4 does not: measured, bank conflicts
//     in 21% of a kernel's cycles);
//   kCols, kStack, kPacked tile [32 k][rows]: chunk c of row k is kept at
//     c ^ 2 f(k), f(k) made of bits 0, 1 and 3 of k (of 64 columns, whose rows
//     are half a turn of the banks, of bits 1 and 3); a fragment is read by the
//     transposing LDS read, whose 32 lanes touch 8 rows k of 32 bytes each.
// The products take the n side first, so a lane holds 4 consecutive n of one m.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "training.h"

namespace tide {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x2v __attribute__((ext_vector_type(2)));
typedef float f32x4v __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// 16 bytes of a caller's matrix, aligned to its elements only: global memory
// takes such accesses whole.
typedef u32x4 any_u32x4 __attribute__((aligned(2)));
typedef f32x4v any_f32x4 __attribute__((aligned(4)));

#define TIDE_GLOBAL __attribute__((address_space(1)))
#define TIDE_LDS __attribute__((address_space(3)))

enum class Form { kRows, kPair, kCols, kStack, kPacked };
enum class Code { kE4m3, kInt8 };

constexpr int kStages = 4;  // LDS stages a tile's steps go round

struct Operand {
  const void* base;       // bf16 (fp16) values, or codes (kPacked); 16-byte aligned
  const uint8_t* scales;  // kPacked: [k][scale_ld]
  int64_t ld;             // elements from row to row, a multiple of 8 (kPacked: of 32)
  int64_t scale_ld;
  int64_t extent;         // rows (columns) of C that exist on this side
  const void* second = nullptr;  // kPair, kStack: the other matrix, of the same layout
  int64_t split = 0;             // kStack: steps of k in the first
};

// 8 zero values for the lanes whose k lies past the end.
static __device__ __align__(16) const uint32_t g_zero16[4] = {0, 0, 0, 0};

// 16 bytes a lane from its own address to LDS, in lane order.
__device__ __forceinline__ void load_to_lds(const void* g, void* lds) {
  __builtin_amdgcn_global_load_lds((const TIDE_GLOBAL void*)g, (TIDE_LDS void*)lds, 16, 0, 0);
}

// The same from a shared base and the lane's offset.  (A buffer load: the
// compiler takes the global load above for an access to LDS as well, and then
// waits for all of a wave's LDS reads where it could wait for the oldest.)
__device__ __forceinline__ void load_to_lds(const void* base, uint32_t offset, void* lds) {
  const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, -1, 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (TIDE_LDS void*)lds, 16, int(offset), 0, 0, 0);
}

// The same with an offset that all lanes share.
__device__ __forceinline__ void load_to_lds(const void* base, uint32_t offset, uint32_t shared, void* lds) {
  const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, -1, 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (TIDE_LDS void*)lds, 16, int(offset), int(shared), 0, 0);
}

// Waits until at most N of this wave's loads (to LDS or registers) are still
// on their way and, with LGKM, until its LDS accesses are done.
template <int N, bool LGKM>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "the counter's bits");
  __builtin_amdgcn_s_waitcnt((LGKM ? 0x0070 : 0x0F70) | (N & 15) | (N >> 4) << 14);
}

// A barrier that waits for nothing but the other waves: what must have arrived
// before it is waited for by wait_loads.
__device__ __forceinline__ void bare_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

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

// The value 16 (32) lanes away: lane XOR 16 (32).
__device__ __forceinline__ float other_16(float v) {
  const uint32_t b = __float_as_uint(v);
  const auto p = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  return __uint_as_float((threadIdx.x & 16) ? p[0] : p[1]);
}
__device__ __forceinline__ float other_32(float v) {
  const uint32_t b = __float_as_uint(v);
  const auto p = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return __uint_as_float((threadIdx.x & 32) ? p[0] : p[1]);
}

__device__ __forceinline__ int row_swizzle(int r) { return -(r >> 2) & 3; }
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
// wave's, THREADS threads.  LEAN: where fragments start is worked out at each
// read, from one register (see Gemm).
template <Form FORM, Code CODE, int ROWS, int FRAGS, int THREADS, bool LEAN>
struct Side {
  static constexpr bool kPacked = FORM == Form::kPacked, kPair = FORM == Form::kPair, kStack = FORM == Form::kStack;
  static constexpr bool kAlong = FORM == Form::kRows || kPair;  // k runs along the rows
  static constexpr int kBytes = ROWS * kBK * 2;
  static constexpr int kRowChunks = kAlong ? kBK / 8 : ROWS / 8;
  // What a thread moves per step: 16-byte loads to LDS, or units of 16 codes.
  static constexpr int kParts = kPacked ? kBK * (ROWS / 16) / THREADS : kBytes / 16 / THREADS;
  static constexpr int kLoads = kPacked ? 2 * kParts : kParts;  // a unit's codes and its exponent byte
  static_assert(kParts >= 1, "tile too small for its threads");
  // kPair: the parts of the first matrix are half of them
  static_assert(!kPair || (kParts % 2 == 0 && FRAGS % 2 == 0), "halves of a tile");

  const char* base;        // of the tile's first row (kRows) or column, k = 0
  const uint8_t* scales;
  int64_t step;            // bytes from one step of k to the next
  int64_t scale_step;
  uint32_t off[kParts];    // byte offset of each part at its step's base
  uint32_t scale_off[kPacked ? kParts : 1];
  uint32_t put[kPacked ? kParts : 1];  // where each unit goes in the tile
  const char* second;  // kPair, kStack: `base` of the other matrix
  int64_t split;       // kStack

  // kPacked: codes on their way to LDS
  struct Held {
    u32x4 codes[kPacked ? kParts : 1];
    uint32_t scale[kPacked ? kParts : 1];
  };

  // (kPair: a fragment's rows 4 b .. 4 b + 3 are the tile's 8 b .. 8 b + 3, or the
  // four after them, so that a lane holds 8 neighbouring columns of C; the swizzle
  // goes with the fragment's rows.)
  static __device__ __forceinline__ int swizzle_of_k(int k) {
    return ROWS == 64 ? (k & 2) | ((k >> 1) & 4) : col_swizzle(k);
  }
  static __device__ __forceinline__ int swizzle(int r) { return row_swizzle(kPair ? r >> 1 : r); }
  static __device__ __forceinline__ int part_k(int lin) {
    return kAlong ? ((lin & 3) ^ swizzle(lin >> 2)) * 8 : lin / (kPacked ? ROWS / 16 : kRowChunks);
  }

  __device__ __forceinline__ void init(const Operand& o, int64_t first, int tid) {
    // rows (columns) past the end read the last one: their results are dropped
    const int64_t last = o.extent - 1 - first;
    if constexpr (kAlong) {
      base = static_cast<const char*>(o.base) + first * o.ld * 2;
      if constexpr (kPair) second = static_cast<const char*>(o.second) + first * o.ld * 2;
      step = kBK * 2;
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        const int lin = i * THREADS + tid, r = (lin >> 2) % (kPair ? ROWS / 2 : ROWS);
        const int rr = r <= last ? r : int(last);
        off[i] = uint32_t(rr) * uint32_t(o.ld * 2) + uint32_t(part_k(lin) * 2);
      }
    } else if constexpr (!kPacked) {
      base = static_cast<const char*>(o.base) + first * 2;
      if constexpr (kStack) {
        second = static_cast<const char*>(o.second) + first * 2;
        split = o.split;
      }
      step = o.ld * (kBK * 2);
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        const int lin = i * THREADS + tid, k = part_k(lin), c = (lin % kRowChunks) ^ swizzle_of_k(k);
        off[i] = uint32_t(k) * uint32_t(o.ld * 2) + (c * 8 <= last ? uint32_t(c * 16) : 0u);
      }
    } else {
      base = static_cast<const char*>(o.base) + first;
      scales = o.scales + first / 32;
      step = o.ld * kBK;
      scale_step = o.scale_ld * kBK;
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        const int lin = i * THREADS + tid, k = part_k(lin), u = lin % (ROWS / 16);
        const bool in = u * 16 <= last;
        off[i] = uint32_t(k) * uint32_t(o.ld) + (in ? uint32_t(u * 16) : 0u);
        scale_off[i] = uint32_t(k) * uint32_t(o.scale_ld) + (in ? uint32_t(u >> 1) : 0u);
        put[i] = uint32_t((k * kRowChunks + ((2 * u) ^ swizzle_of_k(k))) * 16);
      }
    }
  }

  // Where part i of step s starts.
  __device__ __forceinline__ const char* at_step(int64_t s, int i) const {
    if constexpr (kPair) return uniform((i < kParts / 2 ? base : second) + s * step);
    if constexpr (kStack) return uniform(s < split ? base + s * step : second + (s - split) * step);
    return uniform(base + s * step);
  }

  // Start the loads of step s into `lds` (kPacked: into `held`).  TAIL: only
  // `left` < 32 values of k remain (none, for an empty step), the rest is
  // staged as zeros (k counts in eights where it runs along the rows, which are
  // zero from there to the next multiple of 8).
  template <bool TAIL>
  __device__ __forceinline__ void fetch(char* lds, Held& held, int64_t s, int left, int tid) {
    if constexpr (kPacked) {
      const char* at = at_step(s, 0);
      const uint8_t* sc = uniform(scales + s * scale_step);
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        if (!TAIL || part_k(i * THREADS + tid) < left) {
          held.codes[i] = *(const TIDE_GLOBAL u32x4*)(at + renew(off[i]));
          held.scale[i] = *(const TIDE_GLOBAL uint8_t*)(sc + renew(scale_off[i]));
        } else {
          held.codes[i] = u32x4{0, 0, 0, 0};
          held.scale[i] = 127;
        }
      }
    } else {
      const int wave_base = wave_index() * 64;
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        const char* at = at_step(s, i);
        char* to = lds + (i * THREADS + wave_base) * 16;
        if constexpr (TAIL)
          load_to_lds(part_k(i * THREADS + tid) < left ? at + off[i] : reinterpret_cast<const char*>(g_zero16), to);
        else
          load_to_lds(at, off[i], to);
      }
    }
  }

  // Part i of a whole step's loads to LDS.
  __device__ __forceinline__ void fetch_part(char* lds, int64_t s, int i) {
    load_to_lds(at_step(s, i), off[i], lds + (i * THREADS + wave_index() * 64) * 16);
  }

  // The same for an operand of less than 4 GiB: what all lanes share goes into the
  // instruction's own offset, and little is computed for a load.
  __device__ __forceinline__ void fetch_near(char* lds, uint32_t s, int i) {
    char* to = lds + (i * THREADS + wave_index() * 64) * 16;
    if constexpr (kPair)
      load_to_lds(i < kParts / 2 ? base : second, off[i], s * uint32_t(step), to);
    else if constexpr (kStack) {
      const bool in = int64_t(s) < split;
      load_to_lds(in ? base : second, off[i], (in ? s : s - uint32_t(split)) * uint32_t(step), to);
    } else
      load_to_lds(base, off[i], s * uint32_t(step), to);
  }

  // kPacked: widen what fetch() loaded, halves [h0, h1) of each unit, and write
  // it to LDS.
  __device__ __forceinline__ void settle(char* lds, const Held& held, int h0 = 0, int h1 = 2) {
    if constexpr (kPacked) {
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        char* to = lds + renew(put[i]);
#pragma unroll
        for (int h = h0; h < h1; ++h) {
          const u32x2 lo = widen4<CODE>(held.codes[i][2 * h], held.scale[i]);
          const u32x2 hi = widen4<CODE>(held.codes[i][2 * h + 1], held.scale[i]);
          *reinterpret_cast<u32x4*>(to + 16 * h) = u32x4{lo.x, lo.y, hi.x, hi.y};
        }
      }
    }
  }

  // Where this lane's fragments of a wave's FRAGS x 16 rows (columns) from r0
  // (a multiple of 16 FRAGS) start in the tile.
  static constexpr int kSpots = kAlong || LEAN ? 1 : FRAGS;
  static __device__ __forceinline__ void spots(uint32_t* at, int r0, int lane) {
    if constexpr (kAlong) {
      const int r = kPair ? r0 / 2 + 2 * (lane & 12) + (lane & 3) : r0 + (lane & 15);
      at[0] = uint32_t((r * kRowChunks + ((lane >> 4) ^ swizzle(r))) * 16);
    } else {
      // a transposing read gives lane l of 16 the values of column l in the
      // four rows k of which lanes 4j .. 4j+3 point at 4 columns each
      const int k = 8 * (lane >> 4) + ((lane & 15) >> 2), col = r0 + 4 * (lane & 3);
      const uint32_t first = uint32_t((k * kRowChunks + ((col >> 3) ^ swizzle_of_k(k))) * 16 + (col & 4) * 2);
#pragma unroll
      for (int i = 0; i < kSpots; ++i) at[i] = spot(first, i);
    }
  }
  // 16 i columns on are 2 i chunks, bits that are 0 before the swizzle.
  static __device__ __forceinline__ uint32_t spot(uint32_t first, int i) { return first ^ uint32_t(i * 32); }

  // Fragment i: rows (columns) 16 i + 0..15, k = 8 (lane / 16) + 0..7.  (kPair: the
  // second half of the fragments are the second matrix's, and of 32 rows two
  // fragments have every other four.)
  static __device__ __forceinline__ bf16x8 fragment(const char* lds, uint32_t* at, int i) {
    if constexpr (kAlong) {
      constexpr int kHalf = FRAGS / 2;
      const int j = kPair ? i % kHalf : i, r = kPair ? i / kHalf * (ROWS / 2) + j / 2 * 32 + j % 2 * 4 : j * 16;
      return *reinterpret_cast<const bf16x8*>(lds + renew(at[0]) + r * kRowChunks * 16);
    } else {
      // rows k and k + 4 share their swizzle
      const char* p = lds + (LEAN ? spot(renew(at[0]), i) : renew(at[i]));
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TIDE_LDS s16x4*)p);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TIDE_LDS s16x4*)(p + 4 * kRowChunks * 16));
      bf16x8 r;
      __builtin_memcpy(&r, &lo, 8);
      __builtin_memcpy(reinterpret_cast<char*>(&r) + 8, &hi, 8);
      return r;
    }
  }
};

__device__ __forceinline__ uint32_t bf16_bits_of(float v) {
  const __bf16 b = __bf16(v);  // round to nearest even
  uint16_t r;
  __builtin_memcpy(&r, &b, 2);
  return r;
}
// (One instruction for both.)
__device__ __forceinline__ uint32_t two_bf16(float a, float b) {
  return bf16x2_as_bits(__builtin_convertvector((f32x2v{a, b}), bf16x2));
}
__device__ __forceinline__ float low_bf16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float high_bf16(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }
__device__ __forceinline__ f32x4v add4(f32x4v a, f32x4v b) {
#pragma unroll
  for (int j = 0; j < 4; ++j) b[j] = a[j] + b[j];
  return b;
}

// 8 bf16 values from s, of which `left` exist (any number): zeros for the rest.
__device__ __forceinline__ u32x4 eight_of(const uint16_t* s, int64_t left) {
  if (left >= 8) return *reinterpret_cast<const any_u32x4*>(s);
  u32x4 v;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] = (2 * j < left ? uint32_t(s[2 * j]) : 0u) | (2 * j + 1 < left ? uint32_t(s[2 * j + 1]) : 0u) << 16;
  return v;
}

// Where a product goes: alpha (add + s) (+ old), rounded once to fp32 or bf16.
struct Target {
  void* base;
  int64_t ld, rows, cols;
  const int32_t* row_map;  // the row of `base` (and `add`) that each row goes to, or null
  const float* add;        // as `base`, or null
  float alpha;
  int32_t f32, accumulate;
};

// Writes 8 columns of row m from column n, all of them in range.
__device__ __forceinline__ void put_vectors(const Target& t, int64_t m, int64_t n, f32x4v lo, f32x4v hi) {
  const int64_t at = (t.row_map ? int64_t(t.row_map[m]) : m) * t.ld + n;
  if (t.add) {
    lo = add4(*reinterpret_cast<const any_f32x4*>(t.add + at), lo);
    hi = add4(*reinterpret_cast<const any_f32x4*>(t.add + at + 4), hi);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    lo[j] = t.alpha * lo[j];
    hi[j] = t.alpha * hi[j];
  }
  if (t.f32) {
    float* d = static_cast<float*>(t.base) + at;
    if (t.accumulate) {
      lo = add4(*reinterpret_cast<const any_f32x4*>(d), lo);
      hi = add4(*reinterpret_cast<const any_f32x4*>(d + 4), hi);
    }
    *reinterpret_cast<any_f32x4*>(d) = lo;
    *reinterpret_cast<any_f32x4*>(d + 4) = hi;
  } else {
    any_u32x4* d = reinterpret_cast<any_u32x4*>(static_cast<uint16_t*>(t.base) + at);
    if (t.accumulate) {
      const u32x4 o = *d;
      lo = add4(f32x4v{low_bf16(o[0]), high_bf16(o[0]), low_bf16(o[1]), high_bf16(o[1])}, lo);
      hi = add4(f32x4v{low_bf16(o[2]), high_bf16(o[2]), low_bf16(o[3]), high_bf16(o[3])}, hi);
    }
    *d = u32x4{two_bf16(lo[0], lo[1]), two_bf16(lo[2], lo[3]), two_bf16(hi[0], hi[1]), two_bf16(hi[2], hi[3])};
  }
}

// The same, of those in range, which at the row's end go one by one.
__device__ __forceinline__ void put_some(const Target& t, int64_t m, int64_t n, f32x4v lo, f32x4v hi) {
  if (m >= t.rows || n >= t.cols) return;
  if (n + 8 <= t.cols) return put_vectors(t, m, n, lo, hi);
  const int64_t at = (t.row_map ? int64_t(t.row_map[m]) : m) * t.ld + n;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (n + j >= t.cols) continue;
    float v = j < 4 ? lo[j & 3] : hi[j & 3];
    if (t.add) v = t.add[at + j] + v;
    v = t.alpha * v;
    if (t.f32) {
      float* d = static_cast<float*>(t.base) + at + j;
      *d = t.accumulate ? *d + v : v;
    } else {
      uint16_t* d = static_cast<uint16_t*>(t.base) + at + j;
      *d = uint16_t(bf16_bits_of(t.accumulate ? low_bf16(*d) + v : v));
    }
  }
}

// Orders this wave's LDS accesses for all its lanes: what a lane wrote before is
// read by the others after, and the other way round.  (The LDS serves a wave in
// order; it is the compiler that must not swap accesses of different lanes.)
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Waits for this wave's LDS accesses, then for the other waves (not for loads).
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_s_waitcnt(0xC07F);
  bare_barrier();
}

// The tile loop.  WM x WN waves, each holding an (BM / WM) x (BN / WN) part.  A
// workgroup takes one tile after another: open() starts a tile's first loads,
// loop() sums it into acc, and while acc is used comes the next tile's open(), so
// that its loads (but codes) pass under the rest of the epilogue.
//
// Step i's tiles lie in stage i mod 4.  While a wave multiplies step i it
// starts the loads of step i + 3 and reads the first fragments of step i + 1,
// so that one barrier a step is enough and no product waits behind it: past
// it, step i + 1 has arrived for all waves, and all are done with the stage
// that step i + 3 goes to.  (Packed codes are loaded 4 steps ahead into
// registers and written to LDS 2 steps ahead.)  The whole steps are filled up
// to a multiple of 4 with empty ones, which go first; a short last step goes
// before them all, from the last stage.  WHOLE: there is never a short one (the
// second place where sums are formed costs registers: without it the sums of a
// 256 x 256 tile of two kRows sides are not spilled).
template <Form FA, Form FB, Code CODE, int BM, int BN, int WM, int WN, bool F16 = false, bool WHOLE = false>
struct Gemm {
  static constexpr int kThreads = WM * WN * 64;
  static constexpr int kFM = BM / WM / 16, kFN = BN / WN / 16;  // fragments of a wave
  static constexpr bool kPacked = FA == Form::kPacked || FB == Form::kPacked;
  // With e4m3 codes the fragments' addresses no longer fit the registers beside
  // the products' sums (spilled in the step loop: 12% slower); with int8 codes
  // there is no time to work them out (3% slower), nor need without codes.
  static constexpr bool kLean = kPacked && CODE == Code::kE4m3;
  // Codes are widened beside the products, e4m3 ones half a unit at a time with a
  // row of products between the halves (4096^3: 107.4 -> 105.5 us; 8192 x 4096 x
  // 14336: 773 -> 762 us), int8 ones at once (in halves 846 -> 853 us).
  static constexpr int kHalves = kPacked && CODE == Code::kE4m3 ? 2 : 1;
  using SA = Side<FA, CODE, BM, kFM, kThreads, kLean>;
  using SB = Side<FB, CODE, BN, kFN, kThreads, kLean>;
  static constexpr int kStage = SA::kBytes + SB::kBytes;  // bytes of each of the four stages

  f32x4v acc[kFM][kFN];
  int tid, lane, wm, wn;

  SA sa;
  SB sb;
  uint32_t at_a[SA::kSpots], at_b[SB::kSpots];
  int64_t s;       // the running step, in 32 k; below `first`: an empty one
  int64_t first, whole, rounds;
  int left;

  __device__ __forceinline__ void setup() {
    tid = threadIdx.x;
    lane = tid & 63;
    wm = wave_index() / WN;
    wn = wave_index() % WN;
    SA::spots(at_a, wm * (BM / WM), lane);
    SB::spots(at_b, wn * (BN / WN), lane);
  }

  // What an epilogue computes from the lane from here on is not worked out before
  // the sums, whose registers it would take.
  __device__ __forceinline__ void renew_lane() { asm("" : "+v"(lane)); }

  static __device__ __forceinline__ f32x4v product(bf16x8 n, bf16x8 m, f32x4v sum) {
    if constexpr (F16)
      return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, n), __builtin_bit_cast(f16x8, m), sum, 0, 0,
                                                    0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(n, m, sum, 0, 0, 0);
  }

  // Loads to LDS of step s + ahead < s + 3.
  __device__ __forceinline__ void fetch_early(char* lds, int ahead) {
    typename SA::Held na;
    typename SB::Held nb;
    if (s + ahead < first) {
      if (!SA::kPacked) sa.template fetch<true>(lds, na, first, 0, tid);
      if (!SB::kPacked) sb.template fetch<true>(lds + SA::kBytes, nb, first, 0, tid);
    } else {
      if (!SA::kPacked) sa.template fetch<false>(lds, na, s + ahead, 0, tid);
      if (!SB::kPacked) sb.template fetch<false>(lds + SA::kBytes, nb, s + ahead, 0, tid);
    }
  }

  // Starts the tile at (m0, n0), k in [k_first, k_end) (k_first a multiple of
  // 32), in the first three stages, which no wave uses any more.
  __device__ __forceinline__ void open(const Operand& a, const Operand& b, int64_t m0, int64_t n0, int64_t k_first,
                                       int64_t k_end, char* l0, char* l1, char* l2, char* = nullptr) {
    sa.init(a, m0, tid);
    sb.init(b, n0, tid);
    first = k_first / kBK;
    whole = k_end > k_first ? k_end / kBK : first;
    left = !WHOLE && k_end > k_first ? int(k_end - whole * kBK) : 0;
    rounds = (whole - first + 3) / 4;
    s = whole - rounds * 4;
    if (rounds == 0) return;
    fetch_early(l0, 0);
    fetch_early(l1, 1);
    fetch_early(l2, 2);
  }

  // Sums the opened tile into acc.  All waves are done with the stages then.
  __device__ __forceinline__ void loop(char* l0, char* l1, char* l2, char* l3) {
    bf16x8 fb[kFN], fa[2];
    typename SA::Held ha[2];  // packed sides: codes of an even and an odd step
    typename SB::Held hb[2];
    // Codes of step s + ahead < s + 4.
    auto codes_early = [&](int ahead, typename SA::Held& na, typename SB::Held& nb) {
      if (s + ahead < first) {
        if (SA::kPacked) sa.template fetch<true>(nullptr, na, first, 0, tid);
        if (SB::kPacked) sb.template fetch<true>(nullptr, nb, first, 0, tid);
      } else {
        if (SA::kPacked) sa.template fetch<false>(nullptr, na, s + ahead, 0, tid);
        if (SB::kPacked) sb.template fetch<false>(nullptr, nb, s + ahead, 0, tid);
      }
    };
    auto settle = [&](char* lds, int set, int h) {
      sa.settle(lds, ha[set], h * 2 / kHalves, (h + 1) * 2 / kHalves);
      sb.settle(lds + SA::kBytes, hb[set], h * 2 / kHalves, (h + 1) * 2 / kHalves);
    };

    auto begin = [&](const char* lds) {
#pragma unroll
      for (int i = 0; i < 2; ++i) fa[i] = SA::fragment(lds, at_a, i);
#pragma unroll
      for (int j = 0; j < kFN; ++j) fb[j] = SB::fragment(lds + SA::kBytes, at_b, j);
    };
    // Loads to LDS of step s + 3, kPerRow of them after a row.  (Started together at
    // the step's head they hold its products up, 4% of a large product's time.)
    constexpr int kPartsA = SA::kPacked ? 0 : SA::kParts, kParts = kPartsA + (SB::kPacked ? 0 : SB::kParts);
    constexpr int kPerRow = (kParts + kFM - 1) / kFM;
    // codes are loaded after row kFM / 2 - 1 or a later one
    static_assert(!kPacked || (kParts + kPerRow - 1) / kPerRow <= kFM / 2, "loads to LDS before codes");
    // Multiplies the step in `now`, whose first fragments have been read;
    // MORE: reads the first ones of the step in `next`.  A fragment is read two
    // rows of products before its own; part(i) follows row i, halfway(h) the
    // middle ones.
    auto multiply = [&](const char* now, const char* next, bool more, auto part, auto halfway) {
      bf16x8 nb[kFN], a[kFM + 2];
      a[0] = fa[0];
      a[1] = fa[1];
#pragma unroll
      for (int i = 0; i < kFM; ++i) {
        if (i + 2 < kFM)
          a[i + 2] = SA::fragment(now, at_a, i + 2);
        else if (more)
          a[i + 2] = SA::fragment(next, at_a, i + 2 - kFM);
        if (more) {
#pragma unroll
          for (int j = 0; j < kFN; ++j)
            if (i == (j * kFM) / kFN) nb[j] = SB::fragment(next + SA::kBytes, at_b, j);
        }
#pragma unroll
        for (int j = 0; j < kFN; ++j) acc[i][j] = product(fb[j], a[i], acc[i][j]);
        part(i);
        // A step's loads to LDS come before its codes', as the next waits count
        // them.  (Not between them everywhere: with 256 x 256 tiles of int8 codes
        // it costs spilled registers, and there a row of products lies between.)
        if (kPacked && i == kFM / 2 - 1 && i * kPerRow < kParts) __builtin_amdgcn_sched_barrier(0);
        if (i == kFM / 2 - kHalves) halfway(0);
        if (kHalves == 2 && i == kFM / 2) halfway(1);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (more) {
        fa[0] = a[kFM];
        fa[1] = a[kFM + 1];
#pragma unroll
        for (int j = 0; j < kFN; ++j) fb[j] = nb[j];
      }
    };
    // Loads a wave starts after those to LDS of step i + 1, by the beginning of
    // step i: step i + 2's, and the codes of steps i + 2 and i + 3.
    constexpr int kCodeLoads = (SA::kPacked ? SA::kLoads : 0) + (SB::kPacked ? SB::kLoads : 0);
    constexpr int kAfter = SA::kLoads + SB::kLoads + kCodeLoads;
    // Those that follow row i.
    auto load = [&](char* to3, int i) {
#pragma unroll
      for (int n = i * kPerRow; n < (i + 1) * kPerRow; ++n) {
        if (n < kPartsA)
          sa.fetch_part(to3, s + 3, n);
        else if (n < kParts)
          sb.fetch_part(to3 + SA::kBytes, s + 3, n - kPartsA);
      }
    };
    auto step = [&](char* now, char* next, char* to2, char* to3, int set) {
      wait_loads<kAfter, kPacked>();
      bare_barrier();
      multiply(now, next, true, [&](int i) { load(to3, i); }, [&](int h) {
        settle(to2, set, h);
        if (h + 1 < kHalves) return;
        if (SA::kPacked) sa.template fetch<false>(nullptr, ha[set], s + 4, 0, tid);
        if (SB::kPacked) sb.template fetch<false>(nullptr, hb[set], s + 4, 0, tid);
      });
      ++s;
    };

    // every first load on its way before the first is waited for
    typename SA::Held ta, ea[2];
    typename SB::Held tb, eb[2];
    if (!WHOLE && left) {
      lds_barrier();  // the last stage may have served an epilogue
      sa.template fetch<true>(l3, ta, whole, left, tid);
      sb.template fetch<true>(l3 + SA::kBytes, tb, whole, left, tid);
    }
    if (kPacked && rounds > 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) codes_early(i, ea[i], eb[i]);
#pragma unroll
      for (int i = 0; i < 2; ++i) codes_early(2 + i, ha[i], hb[i]);
    }
    if (!WHOLE && left) {
      sa.settle(l3, ta);
      sb.settle(l3 + SA::kBytes, tb);
    }
    if (kPacked && rounds > 0) {
      sa.settle(l0, ea[0]);
      sb.settle(l0 + SA::kBytes, eb[0]);
      sa.settle(l1, ea[1]);
      sb.settle(l1 + SA::kBytes, eb[1]);
    }
#pragma unroll
    for (int i = 0; i < kFM; ++i)
#pragma unroll
      for (int j = 0; j < kFN; ++j) acc[i][j] = f32x4v{0.f, 0.f, 0.f, 0.f};
    wait_loads<0, true>();
    bare_barrier();
    if (!WHOLE && left) {
      begin(l3);
      multiply(l3, l3, false, [](int) {}, [](int) {});
    }
    if (rounds > 0) {
      begin(l0);
      for (int64_t r = 1; r < rounds; ++r) {
        step(l0, l1, l2, l3, 0);
        step(l1, l2, l3, l0, 1);
        step(l2, l3, l0, l1, 0);
        step(l3, l0, l1, l2, 1);
      }
      wait_loads<kAfter, kPacked>();
      bare_barrier();
      multiply(l0, l1, true, [&](int i) { load(l3, i); }, [&](int h) { settle(l2, 0, h); });
      wait_loads<SA::kLoads + SB::kLoads, kPacked>();  // what was started after step i + 1's: codes and the last step's
      bare_barrier();
      multiply(l1, l2, true, [](int) {}, [&](int h) { settle(l3, 1, h); });
      wait_loads<0, kPacked>();
      bare_barrier();
      multiply(l2, l3, true, [](int) {}, [](int) {});
      multiply(l3, l3, false, [](int) {}, [](int) {});
    }
    lds_barrier();
  }

  // f(row, column, values of 8 columns from that one) for every group of eight
  // this wave holds, rows and columns counted in the tile.  The groups pass
  // through this wave's 16 rows of the last stage, so that the lanes hand over
  // neighbouring columns of a row; the 16 bytes g of row r are kept at g ^ r,
  // which spreads the rows over the banks.
  // halfway() comes after half of the rows.
  template <bool UNROLL, typename F, typename H>
  __device__ __forceinline__ void each(char* lds, F f, H halfway) {
    constexpr int kCols = BN / WN, kQuads = kCols / 4, kMask = kQuads - 1, kGroups = kCols / 8;
    static_assert(WM * WN * 16 * kCols * 4 <= kStage && (kQuads & kMask) == 0, "epilogue rows");
    float* rows = reinterpret_cast<float*>(lds) + wave_index() * 16 * kCols;
#pragma unroll
    for (int i = 0; i < kFM; ++i) {
      const int w = lane & 15;
#pragma unroll
      for (int j = 0; j < kFN; ++j)
        *reinterpret_cast<f32x4v*>(rows + w * kCols + ((4 * j + (lane >> 4)) ^ (w & kMask)) * 4) = acc[i][j];
      wave_order();
      auto group = [&](int q) {
        const int r = q / kGroups, c = q % kGroups;
        f(wm * (BM / WM) + i * 16 + r, wn * kCols + c * 8,
          *reinterpret_cast<const f32x4v*>(rows + r * kCols + ((2 * c) ^ (r & kMask)) * 4),
          *reinterpret_cast<const f32x4v*>(rows + r * kCols + ((2 * c + 1) ^ (r & kMask)) * 4));
      };
      if constexpr (UNROLL && 16 * kGroups % 64 == 0) {
#pragma unroll
        for (int q = 0; q < 16 * kGroups / 64; ++q) group(lane + 64 * q);
      } else {
#pragma unroll 1
        for (int q = lane; q < 16 * kGroups; q += 64) group(q);
      }
      wave_order();
      if (i == kFM / 2 - 1) halfway();
    }
  }

  // f(row, values of 8 columns) for every group of eight this wave holds, 8 rows
  // at a time: the group is column() of row `row` + lane / 8, `row` the same for
  // all lanes, so that addresses take one scalar addition.  before(i) comes two
  // calls of f ahead of the 2 i-th.
  static constexpr int kRowGroups = BN / WN / 8;
  static_assert(64 % kRowGroups == 0, "groups of a row");
  __device__ __forceinline__ int column() const { return wn * (BN / WN) + lane % kRowGroups * 8; }
  template <typename P, typename F, typename H>
  __device__ __forceinline__ void each_rows(char* lds, P before, F f, H halfway) {
    constexpr int kCols = BN / WN, kMask = kCols / 4 - 1, kRows = 64 / kRowGroups;
    static_assert(WM * WN * 16 * kCols * 4 <= kStage, "epilogue rows");
    float* rows = reinterpret_cast<float*>(lds) + wave_index() * 16 * kCols;
    const int w = lane & 15, c = lane % kRowGroups;
    before(0);
#pragma unroll
    for (int i = 0; i < kFM; ++i) {
#pragma unroll
      for (int j = 0; j < kFN; ++j)
        *reinterpret_cast<f32x4v*>(rows + w * kCols + ((4 * j + (lane >> 4)) ^ (w & kMask)) * 4) = acc[i][j];
      if (i + 1 < kFM) before(i + 1);
      wave_order();
#pragma unroll
      for (int q = 0; q < 16 / kRows; ++q) {
        const int r = q * kRows + lane / kRowGroups;
        f(wm * (BM / WM) + i * 16 + q * kRows, i, q,
          *reinterpret_cast<const f32x4v*>(rows + r * kCols + ((2 * c) ^ (r & kMask)) * 4),
          *reinterpret_cast<const f32x4v*>(rows + r * kCols + ((2 * c + 1) ^ (r & kMask)) * 4));
      }
      wave_order();
      if (i == kFM / 2 - 1) halfway();
    }
  }

  // The same, where f may change the values; with `mirror` also t(row, q, values of 8
  // rows of a column) of the changed values: rows `row` + 0..7 or, in the odd lanes,
  // 8..15, of column mirror_column() + 32 q.
  __device__ __forceinline__ int mirror_column() const { return wn * (BN / WN) + (lane >> 1); }
  template <typename P, typename F, typename T, typename H>
  __device__ __forceinline__ void each_mirrored(char* lds, bool mirror, P before, F f, T t, H halfway) {
    constexpr int kCols = BN / WN, kMask = kCols / 4 - 1, kRows = 64 / kRowGroups;
    static_assert(kCols % 32 == 0 && WM * WN * 16 * kCols * 4 <= kStage, "epilogue rows");
    float* rows = reinterpret_cast<float*>(lds) + wave_index() * 16 * kCols;
    const int w = lane & 15, c = lane % kRowGroups;
    before(0);
#pragma unroll
    for (int i = 0; i < kFM; ++i) {
#pragma unroll
      for (int j = 0; j < kFN; ++j)
        *reinterpret_cast<f32x4v*>(rows + w * kCols + ((4 * j + (lane >> 4)) ^ (w & kMask)) * 4) = acc[i][j];
      if (i + 1 < kFM) before(i + 1);
      wave_order();
#pragma unroll
      for (int q = 0; q < 16 / kRows; ++q) {
        const int r = q * kRows + lane / kRowGroups;
        f32x4v* p0 = reinterpret_cast<f32x4v*>(rows + r * kCols + ((2 * c) ^ (r & kMask)) * 4);
        f32x4v* p1 = reinterpret_cast<f32x4v*>(rows + r * kCols + ((2 * c + 1) ^ (r & kMask)) * 4);
        f32x4v lo = *p0, hi = *p1;
        f(wm * (BM / WM) + i * 16 + q * kRows, i, q, lo, hi);
        if (mirror) {
          *p0 = lo;
          *p1 = hi;
        }
      }
      wave_order();
      if (mirror) {
        const int r0 = (lane & 1) * 8;
#pragma unroll
        for (int q = 0; q < kCols / 32; ++q) {
          const int n = (lane >> 1) + 32 * q;
          f32x4v lo, hi;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float v = rows[(r0 + j) * kCols + ((n >> 2) ^ ((r0 + j) & kMask)) * 4 + (n & 3)];
            if (j < 4)
              lo[j & 3] = v;
            else
              hi[j & 3] = v;
          }
          t(wm * (BM / WM) + i * 16, q, lo, hi);
        }
        wave_order();
      }
      if (i == kFM / 2 - 1) halfway();
    }
  }

  // Writes the tile at (m0, n0) to `t`, which has no row map, adds nothing and takes
  // the sums as they are: as write(), with fewer instructions.
  template <typename H>
  __device__ __forceinline__ void write_rows(const Target& t, int64_t m0, int64_t n0, char* lds, H halfway) {
    const int64_t n1 = n0 + column(), left = t.cols - n1;
    const uint32_t row = lane / kRowGroups, ld = uint32_t(t.ld);
    // the rows come in order: the place goes on with them (a product for each row's
    // would be worked out for all of them beforehand, and spilled)
    uint32_t at = (wm * (BM / WM) + row) * ld + uint32_t(column());
    const int64_t first = m0 * t.ld + n0;
    const int64_t rows = t.rows - m0 - row;
    each_rows(
        lds, [](int) {},
        [&](int r, int, int, f32x4v lo, f32x4v hi) {
          const uint32_t here = at;
          at += (64 / kRowGroups) * ld;
          if (r >= rows || left <= 0) return;
          if (left < 8) return put_some(t, m0 + r + row, n1, lo, hi);
          if (t.f32) {
            any_f32x4* d = reinterpret_cast<any_f32x4*>(static_cast<float*>(t.base) + first + here);
            if (t.accumulate) {
              lo = add4(d[0], lo);
              hi = add4(d[1], hi);
            }
            d[0] = lo;
            d[1] = hi;
          } else {
            any_u32x4* d = reinterpret_cast<any_u32x4*>(static_cast<uint16_t*>(t.base) + first + here);
            if (t.accumulate) {
              const u32x4 o = *d;
              lo = add4(f32x4v{low_bf16(o[0]), high_bf16(o[0]), low_bf16(o[1]), high_bf16(o[1])}, lo);
              hi = add4(f32x4v{low_bf16(o[2]), high_bf16(o[2]), low_bf16(o[3]), high_bf16(o[3])}, hi);
            }
            *d = u32x4{two_bf16(lo[0], lo[1]), two_bf16(lo[2], lo[3]), two_bf16(hi[0], hi[1]), two_bf16(hi[2], hi[3])};
          }
        },
        halfway);
  }

  // Writes the tile at (m0, n0) to `t`.
  template <typename H>
  __device__ __forceinline__ void write(const Target& t, int64_t m0, int64_t n0, char* lds, H halfway) {
    if (n0 + BN <= t.cols)
      each<true>(
          lds,
          [&](int r, int c, f32x4v lo, f32x4v hi) {
            if (m0 + r < t.rows) put_vectors(t, m0 + r, n0 + c, lo, hi);
          },
          halfway);
    else
      each<false>(
          lds, [&](int r, int c, f32x4v lo, f32x4v hi) { put_some(t, m0 + r, n0 + c, lo, hi); }, halfway);
  }
};

// The same for small tiles of few products, whose time is that of their loads on
// their way: a stage is U steps, so up to 3 U of them are, a barrier comes once in U
// steps, and a stage's fragments are read while the one before is multiplied.  The
// steps are filled up to a multiple of U with empty ones; they and a short last step,
// filled up with zeros, go first, so that the loop starts whole ones only.  The
// stages' places are chosen so that the last one ends a turn of the four: open()
// may fill any of them, and the epilogue needs LDS of its own.  (512 x 2048
// orthogonalized by tiles of 64 took 187 us where they were 128, and a stage's
// fragments read ahead 4% less; of 64 x 128 tiles three steps a stage instead of two,
// 108 KB on their way, 2% more: what bounds a step is its LDS traffic.)
template <Form FA, Form FB, int BM, int BN, int WM, int WN, bool F16, int U>
struct DeepGemm : Gemm<FA, FB, Code::kE4m3, BM, BN, WM, WN, F16, true> {
  using Base = Gemm<FA, FB, Code::kE4m3, BM, BN, WM, WN, F16, true>;
  using typename Base::SA;
  using typename Base::SB;
  using Base::kFM;
  using Base::kFN;
  using Base::sa;
  using Base::sb;
  using Base::acc;
  using Base::tid;
  using Base::s;
  using Base::first;
  using Base::whole;
  using Base::rounds;
  using Base::left;
  static constexpr int kStage = U * Base::kStage;
  static constexpr int kRows = Base::kStage;                    // bytes of the epilogue's LDS
  static constexpr int kLoads = U * (SA::kLoads + SB::kLoads);  // of a stage

  uint32_t skip;  // places of the first turn that no stage takes

  // Step `step` of one of the first three stages.  Below `first`: the short last step,
  // just below it, or an empty one; from `whole` on: empty.
  __device__ __forceinline__ void fetch_step(char* stage, int u, int64_t step) {
    typename SA::Held na;
    typename SB::Held nb;
    char *la = stage + u * SA::kBytes, *lb = stage + U * SA::kBytes + u * SB::kBytes;
    if (step >= first && step < whole) {
      sa.template fetch<false>(la, na, step, 0, tid);
      sb.template fetch<false>(lb, nb, step, 0, tid);
    } else {
      const bool tail = left > 0 && step + 1 == first;
      sa.template fetch<true>(la, na, tail ? whole : first, tail ? left : 0, tid);
      sb.template fetch<true>(lb, nb, tail ? whole : first, tail ? left : 0, tid);
    }
  }
  // Load n of a whole stage's.
  __device__ __forceinline__ void fetch_part(char* stage, uint32_t step, int n) {
    constexpr int kEach = SA::kParts + SB::kParts;
    const int u = n / kEach, i = n % kEach;
    if (i < SA::kParts)
      sa.fetch_near(stage + u * SA::kBytes, step + u, i);
    else
      sb.fetch_near(stage + U * SA::kBytes + u * SB::kBytes, step + u, i - SA::kParts);
  }

  __device__ __forceinline__ void open(const Operand& a, const Operand& b, int64_t m0, int64_t n0, int64_t k_first,
                                       int64_t k_end, char* l0, char* l1, char* l2, char* l3) {
    sa.init(a, m0, tid);
    sb.init(b, n0, tid);
    first = k_first / kBK;
    whole = k_end > k_first ? k_end / kBK : first;
    left = k_end > k_first ? int(k_end - whole * kBK) : 0;
    const int64_t steps = whole - first + (left > 0 ? 1 : 0), stages = (steps + U - 1) / U;
    rounds = (stages + 3) / 4;
    skip = uint32_t(-stages) & 3;
    s = whole - stages * U;
    if (rounds == 0) return;
    // always three stages, so that the waits count the same loads
#pragma unroll 1
    for (uint32_t t = 0; t < 3; ++t) {
      const uint32_t place = (skip + t) & 3;
      char* const to = place == 0 ? l0 : place == 1 ? l1 : place == 2 ? l2 : l3;
#pragma unroll 1
      for (int u = 0; u < U; ++u) fetch_step(to, u, s + int(t) * U + u);
    }
  }

  __device__ __forceinline__ void loop(char* l0, char* l1, char* l2, char* l3) {
    struct Fragments {
      bf16x8 a[U][kFM], b[U][kFN];
    } even, odd;
    auto read = [&](Fragments& f, const char* stage, int u) {
#pragma unroll
      for (int i = 0; i < kFM; ++i) f.a[u][i] = SA::fragment(stage + u * SA::kBytes, Base::at_a, i);
#pragma unroll
      for (int j = 0; j < kFN; ++j) f.b[u][j] = SB::fragment(stage + U * SA::kBytes + u * SB::kBytes, Base::at_b, j);
    };
    auto read_all = [&](Fragments& f, const char* stage) {
#pragma unroll
      for (int u = 0; u < U; ++u) read(f, stage, u);
    };
    // Multiplies a stage and reads the next one; LOAD: starts the loads of the one
    // three stages on.
    auto stage = [&](const Fragments& now, Fragments& next, const char* from, char* to3, bool load, bool more) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (more) read(next, from, u);
        if (load) {
#pragma unroll
          for (int n = u * kLoads / U; n < (u + 1) * kLoads / U; ++n) fetch_part(to3, uint32_t(s) + 3 * U, n);
        }
#pragma unroll
        for (int i = 0; i < kFM; ++i)
#pragma unroll
          for (int j = 0; j < kFN; ++j) acc[i][j] = Base::product(now.b[u][j], now.a[u][i], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
      }
      s += U;
    };
    // Before a stage: the next one has arrived for all waves, and what this wave read
    // of this one (whose place the loads after it go to) has come back.
    auto ready = [&](bool last) {
      if (last)
        wait_loads<0, true>();
      else
        wait_loads<kLoads, true>();
      bare_barrier();
    };
#pragma unroll
    for (int i = 0; i < kFM; ++i)
#pragma unroll
      for (int j = 0; j < kFN; ++j) acc[i][j] = f32x4v{0.f, 0.f, 0.f, 0.f};
    if (rounds > 0) {
      wait_loads<2 * kLoads, true>();
      bare_barrier();
      if (skip == 0)
        read_all(even, l0);
      else if (skip == 1)
        read_all(odd, l1);
      else if (skip == 2)
        read_all(even, l2);
      else
        read_all(odd, l3);
      uint32_t over = skip;
      for (int64_t r = 1; r < rounds; ++r) {
        if (over == 0) {
          ready(false);
          stage(even, odd, l1, l3, true, true);
        }
        if (over <= 1) {
          ready(false);
          stage(odd, even, l2, l0, true, true);
        }
        if (over <= 2) {
          ready(false);
          stage(even, odd, l3, l1, true, true);
        }
        ready(false);
        stage(odd, even, l0, l2, true, true);
        over = 0;
      }
      if (over == 0) {
        ready(false);
        stage(even, odd, l1, l3, true, true);
      }
      if (over <= 1) {
        ready(false);
        stage(odd, even, l2, nullptr, false, true);
      }
      if (over <= 2) {
        ready(true);
        stage(even, odd, l3, nullptr, false, true);
      }
      stage(odd, even, nullptr, nullptr, false, false);
    }
    lds_barrier();
  }
};

// Bytes of LDS that an epilogue needs beside the stages.
template <typename G, int SIDE>
constexpr int own_rows() {
  if constexpr (SIDE == 64)
    return G::kRows;
  else
    return 16;
}

// The items of a launch (tiles, or pieces of them) are handed out by queues: one
// word for each of the 8 XCDs, cleared before the launch, counts the items that
// were taken of the XCD's share, item 8 k + x being XCD x's k-th.  A workgroup
// takes from its own XCD's share, whose neighbours its L2 holds, and when that is
// used up from the others'.  So the CUs that a kernel beside this one or a
// stream's CU mask leaves free get all the work: with a fixed share for each of
// 256 workgroups, those without a CU began when the others ended (measured: 58%
// slower on a stream of 240 CUs).  The words lie apart: on one line, 512 workgroups'
// requests took 35 us one after the other.
constexpr uint32_t kNoItem = ~0u;
constexpr uint32_t kQueueWords = 8, kQueuePitch = 64;  // of a queue; from word to word

struct Queue {
  uint32_t* words;
  uint32_t items, x;

  __device__ __forceinline__ void setup(uint32_t* queue, uint32_t n) {
    words = queue;
    items = n;
    asm volatile("s_getreg_b32 %0, hwreg(HW_REG_XCC_ID)" : "=s"(x));
    x &= 7;
  }
  __device__ __forceinline__ uint32_t share(uint32_t of) const { return (items >> 3) + (of < (items & 7) ? 1u : 0u); }
  // The first wave's: its first lane asks for an item of the own share, and the
  // wave settles what ask() gave.  Whether the others' shares have items left is
  // looked up for all of them at once (asked for one after the other, the last
  // look of each workgroup took 10 us).
  __device__ __forceinline__ uint32_t ask() { return threadIdx.x == 0 ? atomicAdd(words + x * kQueuePitch, 1u) : 0u; }
  __device__ __forceinline__ uint32_t settle(uint32_t asked) {
    uint32_t k = __builtin_amdgcn_readfirstlane(asked), used = 0;
    while (k >= share(x)) {
      used |= 1u << x;
      const uint32_t lane = threadIdx.x;
      const bool left = lane < kQueueWords && __hip_atomic_load(words + lane * kQueuePitch, __ATOMIC_RELAXED,
                                                                __HIP_MEMORY_SCOPE_AGENT) < share(lane);
      const uint32_t open = uint32_t(__ballot(left)) & ~used;
      if (open == 0) return kNoItem;
      x = (x + __builtin_ctz((open | open << 8) >> x)) & 7;
      k = __builtin_amdgcn_readfirstlane(ask());
    }
    return 8 * k + x;
  }
};

// A workgroup's first item of a queue.
__device__ __forceinline__ uint32_t first_item(Queue& q, uint32_t* words, uint32_t items, uint32_t* turn) {
  q.setup(words, items);
  if (wave_index() == 0) {
    const uint32_t got = q.settle(q.ask());
    if (threadIdx.x == 0) *turn = got;
  }
  __syncthreads();
  const uint32_t item = __builtin_amdgcn_readfirstlane(*turn);
  __syncthreads();
  return item;
}

// The workgroup's next item, which was asked for as k (at the end of a tile's
// sums: earlier, a workgroup would take what one that is still to start should
// have).
__device__ __forceinline__ uint32_t next_item(Queue& q, uint32_t k, uint32_t* turn) {
  if (wave_index() == 0) {
    const uint32_t got = q.settle(k);
    if (threadIdx.x == 0) *turn = got;
  }
  lds_barrier();
  return __builtin_amdgcn_readfirstlane(*turn);
}

// Item 8 k + x of `total` -> the k-th of XCD x's share, the shares contiguous.
__device__ __forceinline__ uint32_t nth_of_share(uint32_t item, uint32_t total) {
  const uint32_t x = item & 7, each = total >> 3, more = total & 7;
  return x * each + (x < more ? x : more) + (item >> 3);
}

// The tile of an item: XCD x's share of the tiles is contiguous, in an order
// that walks `group` tile rows before it moves to the next tile column, so that
// what an XCD works on at one time shares operand tiles.  (A group of 4 measured
// against 2, 8 and 16 on 4096 x 128000 x 4096: 1.5%, 1.5% and 6% faster.)
__device__ __forceinline__ void tile_of(uint32_t bid, uint32_t tiles_m, uint32_t tiles_n, uint32_t group, uint32_t* tm,
                                        uint32_t* tn) {
  const uint32_t t = nth_of_share(bid, tiles_m * tiles_n);
  const uint32_t band = t / (group * tiles_n), in = t - band * group * tiles_n;
  const uint32_t rows = band * group + group <= tiles_m ? group : tiles_m - band * group;
  *tm = __builtin_amdgcn_readfirstlane(band * group + in % rows);
  *tn = __builtin_amdgcn_readfirstlane(in / rows);
}

// The tile, and the range of steps, of an item of a cut (training.h).  RANGES: an
// XCD's share of the pieces is contiguous with the splits outside, so it reads a
// range of k of both operands once, instead of some tiles' whole k (for dH, whose
// operands are large: the loss with gradients of 667 x 2048 x 50001, 240 pieces,
// 508 -> 485 us).  Otherwise the XCD keeps its tiles (weight gradients: no different
// at 8192 x 4096 x 14336, and 22.6 instead of 25.0 us at 2048 x 768 x 2048).
struct Piece {
  uint32_t tile;
  int64_t k_first, k_end;  // of a depth of k
  int64_t slot;            // of its partial sums; -1: it is a whole tile
};
template <bool RANGES>
__device__ __forceinline__ Piece piece_of(const Cut& c, uint32_t item, int64_t depth) {
  if (item < c.full) return Piece{item, 0, depth, -1};
  const uint32_t rest = c.tiles - c.full, i = item - c.full, q = RANGES ? nth_of_share(i, c.items - c.full) : i;
  const uint32_t split = q / rest;
  uint32_t r = q - split * rest;
  if constexpr (RANGES) {
    // neighbours: tile full + 8 j + x is x's j-th (tile_of)
    const uint32_t u = r, each = rest >> 3, more = rest & 7, large = more * (each + 1);
    const uint32_t x = u < large ? u / (each + 1) : more + (u - large) / each;
    r = 8 * (u < large ? u - x * (each + 1) : (u - large) - (x - more) * each) + x;
  }
  const int64_t k0 = int64_t(split) * c.per * kBK, k1 = k0 + int64_t(c.per) * kBK;
  return Piece{c.full + r, k0, k1 < depth ? k1 : depth, c.splits > 1 ? int64_t(split) * rest + r : -1};
}

// Where the partial sums of a slot go, of a tile of which `rows` exist.
template <int SIDE>
__device__ __forceinline__ Target slot_target(float* partial, int64_t slot, int64_t rows) {
  return Target{partial + slot * SIDE * SIDE, SIDE, rows < SIDE ? rows : SIDE, SIDE, nullptr, nullptr, 1.0f, 1, 0};
}

// 8 columns from `col` of row `row` of a slot.
template <int SIDE>
__device__ __forceinline__ void put_slot(float* partial, int64_t slot, int row, int col, f32x4v lo, f32x4v hi) {
  float* p = partial + slot * SIDE * SIDE + row * SIDE + col;
  *reinterpret_cast<f32x4v*>(p) = lo;
  *reinterpret_cast<f32x4v*>(p + 4) = hi;
}

// The partial sums of 8 columns from `col` of row `row` of tile full + r (of a cut
// with splits), added in order of the splits.
template <int SIDE>
__device__ __forceinline__ void join_eight(const float* partial, const Cut& c, uint32_t r, uint32_t row, uint32_t col,
                                           f32x4v* lo, f32x4v* hi) {
  const float* p = partial + int64_t(r) * SIDE * SIDE + row * SIDE + col;
  f32x4v l = f32x4v{0.f, 0.f, 0.f, 0.f}, h = l;
#pragma unroll 4
  for (uint32_t k = 0; k < c.splits; ++k, p += int64_t(c.tiles - c.full) * SIDE * SIDE) {
    l = add4(l, *reinterpret_cast<const f32x4v*>(p));
    h = add4(h, *reinterpret_cast<const f32x4v*>(p + 4));
  }
  *lo = l;
  *hi = h;
}

// Joins the partial sums of tile full + r (of a cut with splits), in order of
// the splits, into `t`: `part` of the SIDE * SIDE / 2048 parts of a tile.
template <int SIDE>
__device__ __forceinline__ void join_tile(const float* partial, const Cut& c, uint32_t tiles_m, uint32_t tiles_n,
                                          uint32_t r, uint32_t part, const Target& t) {
  const uint32_t g = part * 256 + threadIdx.x, row = g / (SIDE / 8), col = g % (SIDE / 8) * 8;
  uint32_t tm, tn;
  tile_of(c.full + r, tiles_m, tiles_n, 4, &tm, &tn);
  const int64_t m = int64_t(tm) * SIDE + row, n = int64_t(tn) * SIDE + col;
  if (m >= t.rows || n >= t.cols) return;
  f32x4v lo, hi;
  join_eight<SIDE>(partial, c, r, row, col, &lo, &hi);
  put_some(t, m, n, lo, hi);
}

}  // namespace tide
