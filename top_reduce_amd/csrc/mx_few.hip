// Products with weights in blocks of 32 with scales (tr_mx.h), for few rows.
//
//   y[r][n] = sum over k of x[r][k] w[n][k]          x: blocks of 8 bits, bf16 or fp32
//
// for the rows of each expert's segment, or for all rows of one matrix. With SwiGLU
// rows [0, N / 2) of w are gate and the others up, and the result silu(g) u.
//
// Bound by reading the weights. An element times its block's scale is a bf16 number, so
// both operands are widened in registers, two by one conversion, and multiplied by bf16
// matrix instructions: every product is exact and the sums are fp32 (the matrix
// instructions that take the blocks as they are drop what is 2^-13 below the largest of
// eight products; here, where the weights' bytes take the time, they would save nothing).
// With x in fp32 the weights are widened to fp32.
//
// A block takes 16 kGroups rows of w; its waves share the k-tiles of 128 and add their
// sums in LDS in a fixed order. Lane l = 16 g + r of a wave holds, of each group, row r's
// block g of a k-tile (16 or 32 bytes), so the four lanes of a row read 64 or 128 bytes
// in a row, and of x the same block of row r.
#include "tr_internal.h"
#include "tr_mx.h"

namespace tr {
namespace {

constexpr int kWaves = 4;
constexpr int kTile = 128;

enum { kRowsMx = 0, kRowsBf16 = 1, kRowsF32 = 2 };

// One lane's block of a row: elements of kBits, and the scale byte.
template <int kBits>
struct MxBlock {
  u32x4 v[kBits / 4];
  uint32_t s;
  __device__ __forceinline__ void load(const uint8_t* q, const uint8_t* sc, int block) {
    const u32x4* p = reinterpret_cast<const u32x4*>(q + static_cast<int64_t>(block) * (4 * kBits));
#pragma unroll
    for (int i = 0; i < kBits / 4; ++i) v[i] = p[i];
    s = sc[block];
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kBits / 4; ++i) v[i] = u32x4{0, 0, 0, 0};
    s = 127;
  }
  // elements [8 i, 8 i + 8) as bf16
  template <int kI>
  __device__ __forceinline__ u32x4 bf16() const {
    const float f = mx_scale(s);
    if constexpr (kBits == 4) {
      const uint32_t d = v[0][kI];
      return u32x4{mx_pair_bf16<4, 0>(d, f), mx_pair_bf16<4, 1>(d, f), mx_pair_bf16<4, 2>(d, f),
                   mx_pair_bf16<4, 3>(d, f)};
    } else {
      const uint32_t d = v[kI / 2][2 * (kI & 1)], e = v[kI / 2][2 * (kI & 1) + 1];
      return u32x4{mx_pair_bf16<8, 0>(d, f), mx_pair_bf16<8, 1>(d, f), mx_pair_bf16<8, 0>(e, f),
                   mx_pair_bf16<8, 1>(e, f)};
    }
  }
  // elements [4 i, 4 i + 4) as floats
  template <int kI>
  __device__ __forceinline__ u32x4 f32() const {
    const float f = mx_scale(s);
    floatx2 a, b;
    if constexpr (kBits == 4) {
      const uint32_t d = v[0][kI / 2];
      a = mx_pair_f32<4, 2 * (kI & 1)>(d, f);
      b = mx_pair_f32<4, 2 * (kI & 1) + 1>(d, f);
    } else {
      const uint32_t d = v[kI / 4][kI & 3];
      a = mx_pair_f32<8, 0>(d, f);
      b = mx_pair_f32<8, 1>(d, f);
    }
    return u32x4{__float_as_uint(a[0]), __float_as_uint(a[1]), __float_as_uint(b[0]), __float_as_uint(b[1])};
  }
};

// One lane's 32 numbers of a row of x.
template <int kRows>
struct RowBlock;
template <>
struct RowBlock<kRowsMx> : MxBlock<8> {
  template <int kI>
  __device__ __forceinline__ u32x4 operand() const {
    return bf16<kI>();
  }
};
template <int kChunks>
struct PlainBlock {
  u32x4 v[kChunks];
  __device__ __forceinline__ void load(const uint8_t* q, const uint8_t*, int block) {
    const u32x4* p = reinterpret_cast<const u32x4*>(q + static_cast<int64_t>(block) * (16 * kChunks));
#pragma unroll
    for (int i = 0; i < kChunks; ++i) v[i] = p[i];
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) v[i] = u32x4{0, 0, 0, 0};
  }
  template <int kI>
  __device__ __forceinline__ u32x4 operand() const {
    return v[kI];
  }
};
template <>
struct RowBlock<kRowsBf16> : PlainBlock<4> {};
template <>
struct RowBlock<kRowsF32> : PlainBlock<8> {};

struct FewArgs {
  const uint8_t* x;        // rows of x: elements
  const uint8_t* xs;       // their scales (kRowsMx)
  const uint8_t* w;        // [E, N, K]
  const uint8_t* ws;       // [E, N, K / 32]
  const int* offsets;      // [E + 1], or NULL: one matrix, rows [0, R)
  const int* rows;         // [R] rows of x, or NULL: the same
  void* y;                 // [R, No]; bf16, or fp32 with kRowsF32, or 8 bits
  uint8_t* ys;             // [R, No / 32] scales of y in 8 bits
  int64_t T;               // rows of x
  int R;
  int K, N;
  int most;                // experts with more rows are another kernel's
};

// One k-tile of a wave's operands.
template <int kBits, int kRows, int kGroups, int kNT>
struct TileData {
  MxBlock<kBits> w[kGroups];
  RowBlock<kRows> x[kNT];
};

template <int kI, int kBits, int kRows, int kGroups, int kNT>
__device__ __forceinline__ void multiply(const TileData<kBits, kRows, kGroups, kNT>& t, floatx4 (&acc)[kGroups][kNT]) {
  constexpr int kSteps = kRows == kRowsF32 ? 8 : 4;
  if constexpr (kI < kSteps) {
    u32x4 b[kNT];
#pragma unroll
    for (int n = 0; n < kNT; ++n) b[n] = t.x[n].template operand<kI>();
#pragma unroll
    for (int m = 0; m < kGroups; ++m) {
      u32x4 a;
      if constexpr (kRows == kRowsF32) a = t.w[m].template f32<kI>();
      else a = t.w[m].template bf16<kI>();
#pragma unroll
      for (int n = 0; n < kNT; ++n) acc[m][n] = mma16<kRows == kRowsF32>(a, b[n], acc[m][n]);
    }
    multiply<kI + 1>(t, acc);
  }
}

// Rows [first, first + 16 kNT) of the result, those below `end`, times 16 kGroups rows
// of w: group m has rows wrow(m) .. + 15.
template <int kBits, int kRows, int kGroups, int kNT, bool kSwiglu, bool kMxOut>
__device__ __forceinline__ void few_strip(const FewArgs& a, int e, int first, int end, int strip, float* part) {
  constexpr int kOuts = kSwiglu ? 8 * kGroups : 16 * kGroups;   // outputs of a strip
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r = lane & 15, g = lane >> 4;
  const int No = kSwiglu ? a.N / 2 : a.N;
  const int n0 = strip * kOuts;
  const int blocks = a.K / kMxBlock;
  const int64_t wbytes = static_cast<int64_t>(a.K) * kBits / 8;
  const uint8_t* wq[kGroups];
  const uint8_t* wsc[kGroups];
#pragma unroll
  for (int m = 0; m < kGroups; ++m) {
    // rows past the last are the last again: their outputs are not stored
    constexpr int kHalf = kSwiglu ? kGroups / 2 : kGroups;
    const int n = min(n0 + (m % kHalf) * 16 + r, No - 1) + (m < kHalf ? 0 : No);
    const int64_t row = static_cast<int64_t>(e) * a.N + n;
    wq[m] = a.w + row * wbytes;
    wsc[m] = a.ws + row * blocks;
  }
  constexpr int kXBytes = kRows == kRowsMx ? 1 : kRows == kRowsBf16 ? 2 : 4;
  const uint8_t* xq[kNT];
  const uint8_t* xsc[kNT];
#pragma unroll
  for (int n = 0; n < kNT; ++n) {
    int64_t row = min(first + n * 16 + r, end - 1);
    if (a.rows) row = a.rows[row];
    row = max(int64_t{0}, min(row, a.T - 1));
    xq[n] = a.x + row * a.K * kXBytes;
    xsc[n] = a.xs + row * blocks;
  }
  floatx4 acc[kGroups][kNT];
#pragma unroll
  for (int m = 0; m < kGroups; ++m)
#pragma unroll
    for (int n = 0; n < kNT; ++n) acc[m][n] = floatx4{0, 0, 0, 0};

  const int whole = a.K / kTile;
  TileData<kBits, kRows, kGroups, kNT> t[2];
  auto load = [&](auto& d, int kt) {
    const int b = kt * 4 + g;
#pragma unroll
    for (int m = 0; m < kGroups; ++m) d.w[m].load(wq[m], wsc[m], b);
#pragma unroll
    for (int n = 0; n < kNT; ++n) d.x[n].load(xq[n], xsc[n], b);
  };
  if (wave < whole) {
    load(t[0], wave);
    for (int kt = wave; kt < whole; kt += 2 * kWaves) {
      // (past the last: the last again, not used)
      load(t[1], min(kt + kWaves, whole - 1));
      multiply<0>(t[0], acc);
      load(t[0], min(kt + 2 * kWaves, whole - 1));
      if (kt + kWaves < whole) multiply<0>(t[1], acc);
    }
  }
  if (wave == whole % kWaves && blocks % 4) {   // the blocks of a last, partial k-tile
    const int b = whole * 4 + g;
    if (b < blocks) {
      load(t[0], whole);
    } else {
#pragma unroll
      for (int m = 0; m < kGroups; ++m) t[0].w[m].clear();
#pragma unroll
      for (int n = 0; n < kNT; ++n) t[0].x[n].clear();
    }
    multiply<0>(t[0], acc);
  }

  // part[wave][row][group][16]: the waves' sums
  constexpr int kPitch = 16 * kGroups + 4;
  float* mine = part + wave * (16 * kNT * kPitch);
#pragma unroll
  for (int m = 0; m < kGroups; ++m)
#pragma unroll
    for (int n = 0; n < kNT; ++n)
      *reinterpret_cast<floatx4*>(mine + (n * 16 + r) * kPitch + m * 16 + 4 * g) = acc[m][n];
  __syncthreads();
  // four neighbouring outputs a thread; eight threads are a block of 32
  for (int i = threadIdx.x; i < 16 * kNT * (kOuts / 4); i += kWaves * kWave) {
    const int row = i / (kOuts / 4), c = (i % (kOuts / 4)) * 4;
    auto total = [&](int col) {
      floatx4 s = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < kWaves; ++w)
        s += *reinterpret_cast<const floatx4*>(part + (w * 16 * kNT + row) * kPitch + col);
      return s;
    };
    floatx4 v = total(c);
    if constexpr (kSwiglu) {
      const floatx4 u = total(c + kOuts);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = swiglu<false>(v[j], u[j]);
    }
    const int64_t out = first + row;
    if constexpr (kMxOut) {
      float top = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) top = fmaxf(top, mx_magnitude(v[j]));
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 8));
      const int b = mx_scale_byte<8>(top);
      const float inv = mx_inverse(b);
      if (out < end && n0 + c < No) {
        const int64_t at = out * No + n0 + c;
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.y) + at) =
            mx_pack8(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
        if ((c & 31) == 0) a.ys[at / kMxBlock] = static_cast<uint8_t>(b);
      }
    } else {
      constexpr bool kF32 = kRows == kRowsF32;
      typedef typename Elem<kF32>::type Out;
      if (out < end)
        store4<kF32>(static_cast<Out*>(a.y) + out * No, n0 + c, No, No % 4 == 0, v);
    }
  }
  __syncthreads();
}

template <int kBits, int kRows, int kGroups, int kNT, bool kSwiglu, bool kMxOut>
__global__ __launch_bounds__(kWaves* kWave) void few_products(FewArgs a) {
  __shared__ float part[kWaves * 16 * kNT * (16 * kGroups + 4)];
  const int e = blockIdx.y;
  int begin = 0, end = a.R;
  if (a.offsets) {
    begin = max(0, min(a.offsets[e], a.R));
    end = max(begin, min(a.offsets[e + 1], a.R));
  }
  if (end - begin > a.most) return;
  for (int first = begin; first < end; first += 16 * kNT)
    few_strip<kBits, kRows, kGroups, kNT, kSwiglu, kMxOut>(a, e, first, end, blockIdx.x, part);
}

template <int kBits, int kRows, int kNT, bool kSwiglu, bool kMxOut>
void launch(const FewArgs& a, int E, hipStream_t st) {
  constexpr int kGroups = kSwiglu && kMxOut ? 4 : 2;
  constexpr int kOuts = kSwiglu ? 8 * kGroups : 16 * kGroups;
  const int No = kSwiglu ? a.N / 2 : a.N;
  const dim3 grid(static_cast<uint32_t>(cdiv(No, kOuts)), static_cast<uint32_t>(E));
  few_products<kBits, kRows, kGroups, kNT, kSwiglu, kMxOut><<<grid, kWaves * kWave, 0, st>>>(a);
}

template <int kBits, int kRows, bool kSwiglu, bool kMxOut>
void launch_rows(const FewArgs& a, int E, hipStream_t st) {
  if (a.R <= 16) launch<kBits, kRows, 1, kSwiglu, kMxOut>(a, E, st);
  else launch<kBits, kRows, 4, kSwiglu, kMxOut>(a, E, st);
}

template <int kBits>
void launch_experts(const tr_expert_desc& d, const FewArgs& a, hipStream_t st) {
  if (d.swiglu && d.out) launch_rows<kBits, kRowsMx, true, true>(a, d.E, st);
  else if (d.swiglu) launch_rows<kBits, kRowsMx, true, false>(a, d.E, st);
  else if (d.out) launch_rows<kBits, kRowsMx, false, true>(a, d.E, st);
  else launch_rows<kBits, kRowsMx, false, false>(a, d.E, st);
}

}  // namespace

hipError_t expert_few(const tr_expert_desc& d, const void* x, const void* xs, const void* w, const void* ws,
                      const int* offsets, const int* rows, void* y, void* ys, int most, hipStream_t st) {
  const FewArgs a{static_cast<const uint8_t*>(x), static_cast<const uint8_t*>(xs),
                  static_cast<const uint8_t*>(w), static_cast<const uint8_t*>(ws), offsets, rows, y,
                  static_cast<uint8_t*>(ys), d.T, static_cast<int>(d.R), static_cast<int>(d.K),
                  static_cast<int>(d.N), most};
  if (d.bits == 4) launch_experts<4>(d, a, st);
  else launch_experts<8>(d, a, st);
  return hipGetLastError();
}

hipError_t linear_mx4(const tr_linear4_desc& d, const void* x, const void* w, const void* ws, void* y,
                      hipStream_t st) {
  const FewArgs a{static_cast<const uint8_t*>(x), nullptr, static_cast<const uint8_t*>(w),
                  static_cast<const uint8_t*>(ws), nullptr, nullptr, y, nullptr, d.T,
                  static_cast<int>(d.T), static_cast<int>(d.K), static_cast<int>(d.N), 0x7fffffff};
  if (d.dtype == TR_F32) launch_rows<4, kRowsF32, false, false>(a, 1, st);
  else launch_rows<4, kRowsBf16, false, false>(a, 1, st);
  return hipGetLastError();
}

}  // namespace tr
