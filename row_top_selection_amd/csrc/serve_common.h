// serve_common.h - what the serving operators' kernels share: matrix
// instruction wrappers, asynchronous copies from memory to LDS, LDS swizzle,
// and the host's argument checks.
#ifndef DSATOPK_SERVE_COMMON_H_
#define DSATOPK_SERVE_COMMON_H_

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dsatopk.h"

namespace dsatopk_serve {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 fp16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 fp16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 fp16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

using lds_u32 = __attribute__((address_space(3))) uint32_t;
using lds_i16x4 = __attribute__((address_space(3))) i16x4;
using global_u32 = const __attribute__((address_space(1))) uint32_t;

// How attention scales its softmax's weights before it rounds them to a 16-bit
// type: by a reference 2^kLift below a maximum of the row's scores, which is
// kept until a lane's weights add up to more than kMost (in wide_tiles.h, to more
// than a bound of its own). bfloat16 has fp32's
// exponents, so that every weight is off by at most 2^-8 of itself wherever
// it lies. Half precision ends 14 (with fewer bits: 24) binary orders below 1
// and 16 above: weights up to kMost, its largest number, stay finite, and one is
// off by at most 2^-11 of itself or 2^-25, half of the last step, where that is
// more: 2^-35 of the row's largest weight, which is 2^kLift at least. From 1
// down it would lose bits of weights 10 nats below the maximum, and all of
// those 18 below, which can be most of an output: many tokens beside one of
// large score and small value.
constexpr float kBf16Lift = 0.0f, kBf16Most = 256.0f;
constexpr float kFp16Lift = 10.0f, kFp16Most = 65504.0f;

// A 16-bit float type's matrix instructions. In all of them lane l holds
// row (A) or column (B) l % 32 (l % 16), and along the contraction the
// lane group l / 32 (l / 16) holds consecutive elements; the result has
// column l % 32 (l % 16) and rows 8 * (i / 4) + 4 * (l / 32) + i % 4
// (4 * (l / 16) + i) in its i-th register.
struct Bf16 {
  static constexpr float kLift = kBf16Lift, kMost = kBf16Most;
  static __device__ __forceinline__ f32x16 mma32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 mma16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 mma16_half(u32x2 a, u32x2 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(i16x4, a),
                                                     __builtin_bit_cast(i16x4, b), c, 0, 0, 0);
  }
  // Two floats, each rounded to nearest even, in one word.
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    bf16x2 v = {(__bf16)x, (__bf16)y};
    return __builtin_bit_cast(uint32_t, v);
  }
  static __device__ __forceinline__ void unpack(uint32_t w, float& x, float& y) {
    x = __builtin_bit_cast(float, w << 16);
    y = __builtin_bit_cast(float, w & 0xffff0000u);
  }
};

struct Fp16 {
  static constexpr float kLift = kFp16Lift, kMost = kFp16Most;
  static __device__ __forceinline__ f32x16 mma32(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(fp16x8, a),
                                                  __builtin_bit_cast(fp16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 mma16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(fp16x8, a),
                                                  __builtin_bit_cast(fp16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 mma16_half(u32x2 a, u32x2 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x16f16(__builtin_bit_cast(fp16x4, a),
                                                 __builtin_bit_cast(fp16x4, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    fp16x2 v = {(_Float16)x, (_Float16)y};
    return __builtin_bit_cast(uint32_t, v);
  }
  static __device__ __forceinline__ void unpack(uint32_t w, float& x, float& y) {
    const fp16x2 v = __builtin_bit_cast(fp16x2, w);
    x = (float)v[0];
    y = (float)v[1];
  }
};

// 16 bytes a lane from memory straight into LDS: lane l's bytes go to
// lds + 16 * l (lds is the wave's, the global address each lane's own).
// Completion is counted with the vector loads (wait_copies). The compiler takes
// it for an access of LDS as well: while one is under way, each of its waits for
// an LDS read is a wait for all that have been issued.
__device__ __forceinline__ void copy_to_lds(const void* global, char* lds) {
  __builtin_amdgcn_global_load_lds((global_u32*)(uintptr_t)global, (lds_u32*)lds, 16, 0, 0);
}

// 16 bytes from memory (said to be memory: a pointer that may come from
// either of two places would otherwise be loaded as one that may be LDS).
__device__ __forceinline__ u32x4 load16(const char* global) {
  return *reinterpret_cast<const __attribute__((address_space(1))) u32x4*>((uintptr_t)global);
}

// Until every load and copy of this wave has arrived.
__device__ __forceinline__ void wait_copies() {
  __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt 0, the other counters unbounded
  asm volatile("" ::: "memory");       // LDS reads stay behind it
}

// Until all but this wave's last n loads and copies have arrived.
template <int n>
__device__ __forceinline__ void wait_copies_but() {
  static_assert(n >= 0 && n < 64, "six bits of the count, the low four first, the others on top");
  __builtin_amdgcn_s_waitcnt(0x0f70 | (n & 15) | (n >> 4 << 14));
  asm volatile("" ::: "memory");
}

// Copies of all waves visible to all waves (each waits for its own first).
__device__ __forceinline__ void copies_barrier() {
  wait_copies();
  __syncthreads();
}

// Four 16-bit elements down a column of an LDS tile: the 16 lanes of a
// group point at 4 rows x 4 chunks of 8 bytes (lane i: row i / 4, chunk
// i % 4), and lane i gets column i of those 16, rows 0 .. 3.
__device__ __forceinline__ u32x2 read_columns(const char* lds) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)lds));
}

// Where row t of an LDS tile keeps its 16-byte chunk c: chunk c ^ swizzle of
// t, so that the lanes of a read share none of the 64 banks (256 bytes). (The stores
// of the scores' widened 8-bit heads do: a fifth of that kernel's LDS cycles.)
// Each has 16 different values over 16 rows, for row reads (16 lanes: 16
// rows, one chunk), and more than that for column reads:
//   swizzle16: rows 8a .. 8a + 7 differ in bits 1 .. 3, for 32 lanes that
//   read 8 rows x 2 chunks (products of 16 columns);
//   swizzle32: rows 4a .. 4a + 3 differ in bits 2 and 3, for 32 lanes that
//   read 4 rows x 4 chunks (products of 32 columns);
//   swizzle8, for rows of 8 chunks: two rows fill the banks, and the 8 even
//   and the 8 odd of 16 rows each have 8 different values.
__device__ __forceinline__ constexpr int swizzle16(int t) { return ((t & 7) << 1) | ((t >> 3) & 1); }
__device__ __forceinline__ constexpr int swizzle32(int t) { return ((t & 3) << 2) | ((t >> 2) & 3); }
__device__ __forceinline__ constexpr int swizzle8(int t) { return (t >> 1) & 7; }

// x, as a value that what follows is computed from anew: addresses made of
// it take instructions in the loop instead of registers across it.
__device__ __forceinline__ int here(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// The value of lane ^ 32.
__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32); }

// The last g with key(g) <= x, of the rising keys of n (n at least 1, key(0) <=
// x): 64 keys at a time, the same in all lanes of a wave.
template <class Key>
__device__ __forceinline__ int32_t last_below(int32_t n, int64_t x, int lane, Key key) {
  int32_t at = 0;
  while (n > 1) {
    const int32_t step = (n + 63) / 64;
    const int32_t i = lane * step;
    const int32_t in = (int32_t)__popcll(__ballot(i < n && key(at + i) <= x));
    const int32_t skip = in > 1 ? (in - 1) * step : 0;
    at += skip;
    n = min(step, n - skip);
  }
  return __builtin_amdgcn_readfirstlane(at);
}

// Bytes that stand in for cache entries which a call may not read (no page,
// past a row's end).
constexpr int kZeroBytes = 2048;
static __device__ __align__(256) const uint32_t zero_words[kZeroBytes / 4] = {};
__device__ __forceinline__ const char* zero_row() {
  return reinterpret_cast<const char*>(zero_words);
}

inline bool pow2(int64_t v) { return v >= 1 && (v & (v - 1)) == 0; }

inline int log2_of(int64_t v) {
  int b = 0;
  while ((int64_t(1) << b) < v) ++b;
  return b;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

template <class P>
int launch(void (*fn)(P), dim3 grid, dim3 block, P p, void* stream) {
  void* args[] = {&p};
  return hipLaunchKernel(reinterpret_cast<const void*>(fn), grid, block, args, 0,
                         (hipStream_t)stream) == hipSuccess
             ? DSATOPK_OK
             : DSATOPK_ERR_HIP;
}

}  // namespace dsatopk_serve

#endif  // DSATOPK_SERVE_COMMON_H_
