// Numbers in blocks of 32 with a scale each (gfx950, wave64).
//
// A row of K numbers (K a multiple of 32) is K elements of 8 bits (e4m3: 4 bits of
// exponent, 3 of mantissa, no infinities) or 4 (e2m1: 0, 1/2, 1, 3/2, 2, 3, 4, 6 and a
// sign; the number at an even k in the low half of its byte), and K / 32 scale bytes
// (e8m0: byte b is 2^(b - 127), 255 is NaN). The scale of a block is the smallest power
// of two, 2^-127 at least, that brings its largest magnitude to 448 (6) or below, so no
// element saturates; elements are rounded to nearest, ties to even. In 8 bits an element
// that is not finite is NaN and has no part in the scale; in 4 bits, which have no NaN,
// it makes its block's scale NaN.
#pragma once

#include "tr_chunk.h"

namespace tr {

constexpr int kMxBlock = 32;

// The scale byte of a block whose largest finite magnitude is `top`: the exponent of
// top, less that of 448 = 1.75 2^8 (6 = 1.5 2^2), and one more where top's mantissa is
// past 1.75 (1.5), by a carry out of the mantissa.
template <int kBits>
__device__ __forceinline__ int mx_scale_byte(float top) {
  const int u = static_cast<int>(__float_as_uint(top));
  const int b = kBits == 8 ? ((u + 0x1fffff) >> 23) - 8 : ((u + 0x3fffff) >> 23) - 2;
  return max(b, 0);
}

// 2^-(b - 127) of a scale byte that mx_scale_byte gives (at most 253).
__device__ __forceinline__ float mx_inverse(int b) { return __uint_as_float(static_cast<uint32_t>(254 - b) << 23); }

// |v|, 0 where v is not finite.
__device__ __forceinline__ float mx_magnitude(float v) {
  const float a = fabsf(v);
  return a <= kMaxFloat ? a : 0.0f;
}

// Four floats, already scaled, as four bytes of e4m3.
__device__ __forceinline__ uint32_t mx_pack8(float a, float b, float c, float d) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true));
}

// The float that scales a block's elements, for the conversions: their scale operand
// is an fp32 number of which the exponent counts, 2^-127 being a subnormal one.
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  return __uint_as_float(max(byte << 23, 0x00400000u));
}

typedef float floatx2 __attribute__((ext_vector_type(2)));

// Elements 2 i, 2 i + 1 of a dword of e2m1 (i < 4) or e4m3 (i < 2), scaled, as two bf16
// (exact: at most 4 significant bits; infinite from 2^128 on, below 2^-133 by bf16's steps) or
// two floats.
template <int kBits, int kI>
__device__ __forceinline__ uint32_t mx_pair_bf16(uint32_t v, float scale) {
  if constexpr (kBits == 4)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, kI));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, scale, kI != 0));
}
// Eight elements of 4 bits.
__device__ __forceinline__ u32x4 widen4(uint32_t v, float scale) {
  return u32x4{mx_pair_bf16<4, 0>(v, scale), mx_pair_bf16<4, 1>(v, scale), mx_pair_bf16<4, 2>(v, scale),
               mx_pair_bf16<4, 3>(v, scale)};
}
template <int kBits, int kI>
__device__ __forceinline__ floatx2 mx_pair_f32(uint32_t v, float scale) {
  if constexpr (kBits == 4)
    return __builtin_bit_cast(floatx2, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, scale, kI));
  else
    return __builtin_bit_cast(floatx2, __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(v, scale, kI != 0));
}

// Cache policies of loads to LDS: the ordinary one, and that of what is read once. Weights
// that the 256 MiB behind the L2s cannot hold from call to call are read so.
constexpr int kKept = 0, kOnce = 2;
inline bool read_once(int64_t weight_bytes) { return weight_bytes > (int64_t{256} << 20); }

#if defined(__HIP_DEVICE_COMPILE__)
constexpr int kRawBuffer = 0x00020000;        // word 3 of a buffer resource: raw, 32-bit data
constexpr uint32_t kPast = 0x80000000u;       // an offset past every buffer here: reads 0
typedef __attribute__((address_space(3))) void lds_void;
typedef const __attribute__((address_space(1))) void global_void;

// s_waitcnt immediate: at most n vector loads in flight, with lgkm no LDS access.
__host__ __device__ constexpr int waitcnt_vm(int n, bool lgkm) {
  return (n & 15) | ((n >> 4) << 14) | (7 << 4) | ((lgkm ? 0 : 15) << 8);
}

// A barrier for LDS that leaves loads to LDS in flight (the caller has waited for those
// that it needs).
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Eight floats as three times eight bf16 that add up to them: their upper 16 bits, the upper 16
// of what is left, and the rest (24 significant bits are 8, 8 and 8). Beside bf16 weights three
// matrix instructions count every product in full, at five times the rate of the fp32 ones.
// What is not finite is the first part alone. A number below 2^-110 may have bits below the
// smallest bf16, 2^-133, which its third part cannot hold: they are in the lower halves of the
// remainders' words (`below`), which are 0 otherwise; split_rest makes numbers of them.
struct Split {
  u32x4 top, mid, low;
  uint32_t below;
};
// Whether a number of the wave's has bits left, by what its lanes have of `below`.
__device__ __forceinline__ bool any_below(uint32_t below) { return __any((below & 0xffffu) != 0) != 0; }
typedef uint32_t u32x8 __attribute__((ext_vector_type(8)));
typedef float floatx8 __attribute__((ext_vector_type(8)));
__device__ __forceinline__ u32x4 upper_halves(const u32x8& v) {
  return u32x4{__builtin_amdgcn_perm(v[1], v[0], 0x07060302u), __builtin_amdgcn_perm(v[3], v[2], 0x07060302u),
               __builtin_amdgcn_perm(v[5], v[4], 0x07060302u), __builtin_amdgcn_perm(v[7], v[6], 0x07060302u)};
}
__device__ __forceinline__ Split split_bf16(const u32x4& lo, const u32x4& hi) {
  u32x8 a = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  const floatx8 x = __builtin_bit_cast(floatx8, a);
  u32x8 b = __builtin_bit_cast(u32x8, x - __builtin_bit_cast(floatx8, a & 0xffff0000u));
  u32x8 c = __builtin_bit_cast(u32x8, __builtin_bit_cast(floatx8, b) - __builtin_bit_cast(floatx8, b & 0xffff0000u));
  auto all = [](const u32x8& v) { return (v[0] | v[1] | v[2]) | (v[3] | v[4] | v[5]) | (v[6] | v[7]); };
  uint32_t below = all(c);
  // What is not finite has NaN as its remainder. (Of finite numbers of 2^16 and more, too, the
  // remainders' exponents may come to all ones together: nothing changes for them.)
  if (__any((below & 0x7f800000u) == 0x7f800000u)) {
    const u32x8 size = a & 0x7fffffffu;
    const u32x8 finite = __builtin_bit_cast(u32x8, size < 0x7f800000u), nan = __builtin_bit_cast(u32x8, size > 0x7f800000u);
    a |= nan & 0x00400000u;
    b &= finite;
    c &= finite;
    below = all(c);
  }
  return {upper_halves(a), upper_halves(b), upper_halves(c), below};
}

// What split_bf16 leaves of the same eight floats, 16 bits at most each, times 2^64: `top` and
// `mid` (low is 0). Their weights are scaled by scale_down's 2^-64; where a scale is too small for
// that, the products are below 2^-190.
__device__ __forceinline__ Split split_rest(const u32x4& lo, const u32x4& hi) {
  const u32x8 a = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  const u32x8 b = __builtin_bit_cast(u32x8, __builtin_bit_cast(floatx8, a) - __builtin_bit_cast(floatx8, a & 0xffff0000u));
  const u32x8 c = __builtin_bit_cast(u32x8, __builtin_bit_cast(floatx8, b) - __builtin_bit_cast(floatx8, b & 0xffff0000u));
  const u32x8 finite = __builtin_bit_cast(u32x8, (a & 0x7fffffffu) < 0x7f800000u);
  const floatx8 d = __builtin_bit_cast(floatx8, c & 0x8000ffffu & finite) * 0x1p64f;
  const u32x8 e = __builtin_bit_cast(u32x8, d);
  const floatx8 f = d - __builtin_bit_cast(floatx8, e & 0xffff0000u);
  return {upper_halves(e), upper_halves(__builtin_bit_cast(u32x8, f)), u32x4{0, 0, 0, 0}, 0};
}
// A block's scale (mx_scale) times 2^-64, 2^-127 at least.
__device__ __forceinline__ float scale_down(float scale) {
  const int u = static_cast<int>(__float_as_uint(scale));
  return __uint_as_float(u >= 0x7f800000 ? u : max(u - (64 << 23), 0x00400000));
}

// Eight scale bytes of a row, blocks at .. at + 7, as they lie in memory (at least 8
// blocks: the row's last eight at most), and with 0 for those past the last.
__device__ __forceinline__ uint2 load_scale8(const uint8_t* p, int at, int blocks) {
  typedef uint32_t Odd __attribute__((ext_vector_type(2), aligned(1)));
  const Odd v = *(const __attribute__((address_space(1))) Odd*)(p + min(at, blocks - 8));
  return uint2{v[0], v[1]};
}
__device__ __forceinline__ uint2 scale8(uint2 v, int at, int blocks) {
  const int over = at - min(at, blocks - 8);
  const uint64_t all = (static_cast<uint64_t>(v.y) << 32 | v.x) >> (8 * over & 63);
  return over < 8 ? uint2{static_cast<uint32_t>(all), static_cast<uint32_t>(all >> 32)} : uint2{0, 0};
}

// The scales of kRows rows, 4 kWords bytes of each a k-tile, for a block of kWaves waves: in
// LDS for the k-tiles next to come. A load of a few bytes costs a CU about as much as one of
// a line of 128, which it is one of, and brings that line along: so a turn's rows, one of
// kTurns in order, get 16 bytes each, for kTurns k-tiles. Against every row's own bytes at
// every k-tile: 8 experts of a row, 7168 x 4096, 46 -> 39 us (38 with one row's scales for
// all); 32 of 32 rows 191 -> 158. 32 bytes a turn took more than they saved (42).
template <int kWords, int kRows, int kWaves>
struct ScaleRing {
  static constexpr int kBytes = 4 * kWords, kTurns = 16 / kBytes, kSlots = 2 * kTurns;
  static constexpr int kPart = kRows / (kTurns * kWaves);      // rows of a wave's turn
  static constexpr int kSize = kSlots * kRows * kWords;        // words of LDS
  static_assert(kRows % (kTurns * kWaves) == 0 && kPart <= kWave, "turns");
  struct Window {
    uint2 lo, hi;
  };
  const uint8_t* row[kTurns];      // scales of this lane's row of each turn
  int blocks, first, lane;         // first: of a wave's rows in a turn

  __device__ __forceinline__ static int row_of(int turn, int wave, int lane) {
    return turn * (kRows / kTurns) + wave * kPart + min(lane, kPart - 1);
  }
  // of the rows whose turn k-tile kt is, for k-tiles kt .. kt + kTurns - 1
  __device__ __forceinline__ void load(Window& w, int kt) const {
    const int t = kt & (kTurns - 1);
    const uint8_t* p = row[0];
#pragma unroll
    for (int i = 1; i < kTurns; ++i) {
      const uint8_t* q = row[i];
      asm("" : "+v"(q));      // (chosen among registers, not by an index into memory)
      p = t == i ? q : p;
    }
    load_from(w, p, kt);
  }
  __device__ __forceinline__ void store(const Window& w, uint32_t* ring, int kt) const {
    store_to(w, ring, kt & (kTurns - 1), kt);
  }
  // of a row of turn t (before its first turn, too)
  __device__ __forceinline__ void load_from(Window& w, const uint8_t* p, int kt) const {
    w.lo = load_scale8(p, kt * kBytes, blocks);
    w.hi = load_scale8(p, kt * kBytes + 8, blocks);
  }
  __device__ __forceinline__ void store_to(const Window& w, uint32_t* ring, int t, int kt) const {
    if (lane >= kPart) return;
    const int r = t * (kRows / kTurns) + first + lane;
    uint2 lo = w.lo, hi = w.hi;
    if (kt * kBytes + 16 > blocks) lo = scale8(lo, kt * kBytes, blocks), hi = scale8(hi, kt * kBytes + 8, blocks);
    if constexpr (kWords == 1) {
      const uint32_t v[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
      for (int i = 0; i < 4; ++i) slot(ring, kt + i)[r] = v[i];
    } else {
      reinterpret_cast<uint2*>(slot(ring, kt))[r] = lo;
      reinterpret_cast<uint2*>(slot(ring, kt + 1))[r] = hi;
    }
  }
  // kWords words of every row for k-tile kt
  __device__ __forceinline__ static uint32_t* slot(uint32_t* ring, int kt) {
    return ring + (kt & (kSlots - 1)) * (kRows * kWords);
  }
};
#endif

template <int k>
struct Index {
  static constexpr int value = k;
};

// Between matrix instructions and the first read of what they wrote: with 19 wait states
// after a v_mfma_scale_f32_32x32x64_f8f6f4, which is what the compiler leaves, the last of
// its 16 registers has been read before it was written. `acc`, and what later calls name,
// is read after 48.
__device__ __forceinline__ void settle(floatx16& acc) {
  asm volatile("s_nop 15\n\ts_nop 15\n\ts_nop 15" : "+a"(acc));
}
__device__ __forceinline__ void settled(floatx16& acc) { asm volatile("" : "+a"(acc)); }

}  // namespace tr
