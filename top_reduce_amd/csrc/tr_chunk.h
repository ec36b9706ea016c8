// 16-byte pieces of operand rows, alike for bf16 and fp32 (gfx950, wave64).
//
// Every product here is "NT": activation rows and weight rows both run along
// the reduction dimension. A lane holds one 16-byte chunk of a row: lane l the
// row l % 16 and, of four neighbouring chunks, chunk l / 16. For bf16 that is
// the operand of one 16x16x32 MFMA. For fp32 the four elements of the chunk
// feed four 16x16x4 MFMAs: MFMA s takes element s of every lane, so the four
// cover the 16 k of the chunks once each (in another order, the same for both
// operands). Either way lane (g, r) = (l / 16, l % 16) ends with
// sum_k A[4 g + i][k] B[r][k], i = 0..3.
#pragma once

#include "tr_device.h"

namespace tr {

constexpr float kMaxFloat = 3.4028234664e38f;   // the largest finite fp32

template <bool kF32>
struct Elem;
template <>
struct Elem<false> {
  typedef uint16_t type;
  static constexpr int kBytes = 2, kChunk = 8;   // elements in 16 bytes
};
template <>
struct Elem<true> {
  typedef float type;
  static constexpr int kBytes = 4, kChunk = 4;
};

template <bool kF32>
__device__ __forceinline__ floatx4 mma16(const u32x4& a, const u32x4& b, floatx4 c) {
  if constexpr (kF32) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[s]), __uint_as_float(b[s]), c, 0,
                                               0, 0);
    return c;
  } else {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
}

__device__ __forceinline__ u32x4 load16(const char* p) {
  return *reinterpret_cast<const u32x4*>(p);
}

// 16 bytes that need not start on 16: one load, as global memory takes any
// alignment.
__device__ __forceinline__ u32x4 load16_odd(const void* p) {
  typedef uint32_t Odd __attribute__((ext_vector_type(4), aligned(2)));
  return *static_cast<const Odd*>(p);
}

// The 16 bytes at element k of a row of n elements that need not start on 16
// bytes; zero past n. Near the end the row's last 16 bytes are read, and shifted.
template <bool kF32>
__device__ __forceinline__ u32x4 load16_any(const typename Elem<kF32>::type* row, int k, int n) {
  constexpr int kC = Elem<kF32>::kChunk;
  if (n >= kC) {
    const int at = min(k, n - kC), over = k - at;
    const u32x4 v = load16_odd(row + at);
    if (over == 0) return v;
    const unsigned __int128 all = __builtin_bit_cast(unsigned __int128, v);
    return __builtin_bit_cast(u32x4, over < kC ? all >> (over * Elem<kF32>::kBytes * 8) : 0);
  }
  u32x4 v = {0, 0, 0, 0};
  if constexpr (kF32) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (k + i < n) v[i] = __float_as_uint(row[k + i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = k + 2 * i < n ? row[k + 2 * i] : 0;
      const uint32_t hi = k + 2 * i + 1 < n ? row[k + 2 * i + 1] : 0;
      v[i] = lo | (hi << 16);
    }
  }
  return v;
}

// Lane i < the number of tokens in `mask` (the same in every lane): the token of
// rank i.
__device__ __forceinline__ int tokens_by_rank(uint64_t mask) {
  const int lane = lane_id();
  // lane t of the mask sends t to the lane of its rank, the others to lane 63,
  // which counts with 64 tokens only
  return __builtin_amdgcn_ds_permute(((mask >> lane) & 1 ? popc_below(mask) : 63) * 4, lane);
}

// Two floats rounded to bf16 (nearest even) by one hardware conversion; lo in
// bits 0..15.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
  const bf16x2 v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
  return __builtin_bit_cast(uint32_t, v);
}

// v as two bf16 numbers, hi + lo with 16 significant bits: what is to be rounded to
// the first one. A number past bf16's range (not past fp32's) has the largest of bf16
// as its first one, and its rest in the second.
__device__ __forceinline__ float first_bf16(float v) {
  constexpr float kMaxBf16 = 3.38953139e38f;
  return fabsf(v) <= kMaxFloat ? fminf(fmaxf(v, -kMaxBf16), kMaxBf16) : v;
}
// The second one, given the first. Of an infinity or a NaN it is 0, not NaN.
__device__ __forceinline__ float second_bf16(float v, float hi) { return fabsf(hi) <= kMaxFloat ? v - hi : 0.0f; }

// Four floats as two bf16 numbers each, packed like cvt_bf16x2.
__device__ __forceinline__ void split_bf16(const floatx4& v, uint2& hi, uint2& lo) {
  hi = uint2{cvt_bf16x2(first_bf16(v[0]), first_bf16(v[1])), cvt_bf16x2(first_bf16(v[2]), first_bf16(v[3]))};
  lo = uint2{cvt_bf16x2(second_bf16(v[0], __uint_as_float(hi.x << 16)),
                        second_bf16(v[1], __uint_as_float(hi.x & 0xffff0000u))),
             cvt_bf16x2(second_bf16(v[2], __uint_as_float(hi.y << 16)),
                        second_bf16(v[3], __uint_as_float(hi.y & 0xffff0000u)))};
}

// silu(g) * u in fp32. bf16 results take the hardware exponential and
// reciprocal (about 1 ulp of fp32 each, far below their own rounding); fp32
// results the exact division. silu first: g u alone may be past fp32 where the
// result is not (g = -64, u = 2e38), and times a reciprocal of 0 would be NaN.
template <bool kF32>
__device__ __forceinline__ float swiglu(float g, float u) {
  if constexpr (kF32) return g / (1.0f + expf(-g)) * u;
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

// Stores the four neighbouring outputs v of a row at column col, those below
// n only; `vec`: the row's start and col allow one wide store.
template <bool kF32>
__device__ __forceinline__ void store4(typename Elem<kF32>::type* row, int64_t col, int64_t n,
                                       bool vec, const floatx4& v) {
  if constexpr (kF32) {
    if (vec && col + 4 <= n) {
      *reinterpret_cast<floatx4*>(row + col) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (col + i < n) row[col + i] = v[i];
    }
  } else {
    const uint32_t p[2] = {cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3])};
    if (vec && col + 4 <= n) {
      *reinterpret_cast<uint2*>(row + col) = uint2{p[0], p[1]};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (col + i < n) row[col + i] = static_cast<uint16_t>(p[i >> 1] >> (16 * (i & 1)));
    }
  }
}

}  // namespace tr
