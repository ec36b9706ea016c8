// Products with weights in blocks of 32 with scales (tr_mx.h), for few rows.
//
//   y[r][n] = sum over k of x[r][k] w[n][k]          x: blocks of 8 bits, bf16 or fp32
//
// for the rows of each expert's segment, or for all rows of one matrix. With SwiGLU
// rows [0, N / 2) of w are gate and the others up, and the result silu(g) u.
//
// Bound by reading the weights. An element times its block's scale is a bf16 number, so
// both operands are widened in registers, two by one conversion, and multiplied by bf16
// matrix instructions: every product is exact and the sums are fp32 (numbers of 2^128 and more
// are infinite, those of 8 bits below 2^-133 go by bf16's steps; the matrix
// instructions that take the blocks as they are drop what is 2^-13 below the largest of
// eight products; here, where the weights' bytes take the time, they would save nothing).
// A number of x in fp32 is three of bf16 (split_bf16) in stream_products; few_products widens
// the weights to fp32.
//
// A block takes 16 kGroups rows of w; its waves share K and add their sums in LDS in a
// fixed order. Lane l = 16 g + r of a wave multiplies row r of w by row r of x, of which it
// has the same numbers.
//
// A vector load costs a CU about four cycles for every line of 128 bytes that it touches:
// 16 rows of 64 bytes, as the matrix instruction's lanes hold them, come at 40 KB/us a CU.
// So rows go to LDS by whole lines, without registers, and the operands are read from
// there (stream_products); what that does not take, few_products loads by lanes (32 experts, K =
// 224, N = 4096, 64 / 8192 rows: 32 / 124 us, where reading and multiplying take 5 / 16). 1 row, 7168
// x 7168 in 4 bits: 7.7 us (3.5 TB/s with a launch's first and last loads in it), 16 rows of 8
// bits by weights of 8 12.7; 5 rows in fp32, 1440 x 1001, 7.1, the host's.
#include "tr_internal.h"
#include "tr_mx.h"

namespace tr {
namespace {

constexpr int kFewWaves = 4;
constexpr int kTile = 128;

enum { kRowsMx = 0, kRowsBf16 = 1, kRowsF32 = 2 };

// One lane's 32 numbers of a row's k-tile: elements of kBits, and the k-tile's four scale
// bytes. kSpread (8 bits): 16 from 16 g on and 16 from 64 + 16 g on; else block g.
template <int kBits, bool kSpread = kBits == 8>
struct MxBlock {
  static constexpr int kStep = kSpread ? 64 : 16;     // bytes from v[i] to v[i + 1]
  u32x4 v[kBits / 4];
  uint32_t s;
  // q: the row from this lane's first byte on
  __device__ __forceinline__ void load(const uint8_t* q, const uint8_t* sc, int kt) {
    typedef uint32_t Odd __attribute__((aligned(1)));
#pragma unroll
    for (int i = 0; i < kBits / 4; ++i)
      v[i] = *reinterpret_cast<const u32x4*>(q + static_cast<int64_t>(kt) * (16 * kBits) + kStep * i);
    s = *reinterpret_cast<const Odd*>(sc + kt * 4);
  }
  // the last, partial k-tile: the row has `left` blocks in it; others are 0
  __device__ __forceinline__ void load_part(const uint8_t* q, const uint8_t* sc, int kt, int left, int g) {
#pragma unroll
    for (int i = 0; i < kBits / 4; ++i) {
      v[i] = u32x4{0, 0, 0, 0};
      if ((kSpread ? 2 * i + (g >> 1) : g) < left)
        v[i] = *reinterpret_cast<const u32x4*>(q + static_cast<int64_t>(kt) * (16 * kBits) + kStep * i);
    }
    s = 0;
    for (int b = 0; b < left; ++b) s |= static_cast<uint32_t>(sc[kt * 4 + b]) << (8 * b);
  }
  // the scale of v[i]
  __device__ __forceinline__ float scale(int i, int g) const {
    return mx_scale((s >> (kSpread ? 16 * i + 8 * (g >> 1) : 8 * g)) & 255);
  }
  // elements [8 i, 8 i + 8) as bf16
  template <int kI>
  __device__ __forceinline__ u32x4 bf16(int g) const {
    if constexpr (kBits == 4) {
      const float f = scale(0, g);
      const uint32_t d = v[0][kI];
      return u32x4{mx_pair_bf16<4, 0>(d, f), mx_pair_bf16<4, 1>(d, f), mx_pair_bf16<4, 2>(d, f),
                   mx_pair_bf16<4, 3>(d, f)};
    } else {
      const float f = scale(kI / 2, g);
      const uint32_t d = v[kI / 2][2 * (kI & 1)], e = v[kI / 2][2 * (kI & 1) + 1];
      return u32x4{mx_pair_bf16<8, 0>(d, f), mx_pair_bf16<8, 1>(d, f), mx_pair_bf16<8, 0>(e, f),
                   mx_pair_bf16<8, 1>(e, f)};
    }
  }
  // elements [4 i, 4 i + 4) as floats (4 bits)
  template <int kI>
  __device__ __forceinline__ u32x4 f32(int g) const {
    const float f = scale(0, g);
    const uint32_t d = v[0][kI / 2];
    const floatx2 a = mx_pair_f32<4, 2 * (kI & 1)>(d, f), b = mx_pair_f32<4, 2 * (kI & 1) + 1>(d, f);
    return u32x4{__float_as_uint(a[0]), __float_as_uint(a[1]), __float_as_uint(b[0]), __float_as_uint(b[1])};
  }
};

// One lane's 32 numbers of a row of x.
template <int kRows, int kBits>     // (of the weights beside it)
struct RowBlock;
template <int kBits>
struct RowBlock<kRowsMx, kBits> : MxBlock<8, kBits == 8> {
  template <int kI>
  __device__ __forceinline__ u32x4 operand(int g) const {
    return this->template bf16<kI>(g);
  }
};
// In full types (beside weights in 4 bits): the 32 numbers from 32 g on.
template <int kChunks>
struct PlainBlock {
  u32x4 v[kChunks];
  __device__ __forceinline__ void load(const uint8_t* q, const uint8_t*, int kt) {
    const u32x4* p = reinterpret_cast<const u32x4*>(q + static_cast<int64_t>(kt) * (64 * kChunks));
#pragma unroll
    for (int i = 0; i < kChunks; ++i) v[i] = p[i];
  }
  __device__ __forceinline__ void load_part(const uint8_t* q, const uint8_t* sc, int kt, int left, int g) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) v[i] = u32x4{0, 0, 0, 0};
    if (g < left) load(q, sc, kt);
  }
  template <int kI>
  __device__ __forceinline__ u32x4 operand(int) const {
    return v[kI];
  }
};
template <>
struct RowBlock<kRowsBf16, 4> : PlainBlock<4> {};
template <>
struct RowBlock<kRowsF32, 4> : PlainBlock<8> {};

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
};

// One k-tile of a wave's operands.
template <int kBits, int kRows, int kGroups, int kNT>
struct TileData {
  MxBlock<kBits> w[kGroups];
  RowBlock<kRows, kBits> x[kNT];
};

template <int kI, int kBits, int kRows, int kGroups, int kNT>
__device__ __forceinline__ void multiply(const TileData<kBits, kRows, kGroups, kNT>& t, int g,
                                         floatx4 (&acc)[kGroups][kNT]) {
  constexpr int kSteps = kRows == kRowsF32 ? 8 : 4;
  if constexpr (kI < kSteps) {
    u32x4 b[kNT];
#pragma unroll
    for (int n = 0; n < kNT; ++n) b[n] = t.x[n].template operand<kI>(g);
#pragma unroll
    for (int m = 0; m < kGroups; ++m) {
      u32x4 a;
      if constexpr (kRows == kRowsF32) a = t.w[m].template f32<kI>(g);
      else a = t.w[m].template bf16<kI>(g);
#pragma unroll
      for (int n = 0; n < kNT; ++n) acc[m][n] = mma16<kRows == kRowsF32>(a, b[n], acc[m][n]);
    }
    multiply<kI + 1>(t, g, acc);
  }
}

// The sums of a strip: part[wave][row][16 kGroups], pitch 16 kGroups + 4, as results of rows
// first .. (kRowsHere of them, those below end), outputs n0 .. . A block of kWaves waves.
template <int kRows, int kGroups, int kRowsHere, int kWaves, bool kSwiglu, bool kMxOut>
__device__ __forceinline__ void finish(const FewArgs& a, const float* part, int first, int end, int n0, int No) {
  constexpr int kOuts = kSwiglu ? 8 * kGroups : 16 * kGroups, kPitch = 16 * kGroups + 4;
  // four neighbouring outputs a thread; eight threads are a block of 32
  for (int i = threadIdx.x; i < kRowsHere * (kOuts / 4); i += kWaves * kWave) {
    const int row = i / (kOuts / 4), c = (i % (kOuts / 4)) * 4;
    auto total = [&](int col) {
      floatx4 s = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < kWaves; ++w)
        s += *reinterpret_cast<const floatx4*>(part + (w * kRowsHere + row) * kPitch + col);
      return s;
    };
    floatx4 v = total(c);
    if constexpr (kSwiglu) {
      const floatx4 u = total(c + kOuts);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = swiglu<false>(v[j], u[j]);
    }
    const int64_t out = static_cast<int64_t>(first) + row;      // (a strip may end past 2^31)
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
      if (out < end) store4<kF32>(static_cast<Out*>(a.y) + out * No, n0 + c, No, No % 4 == 0, v);
    }
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
    wq[m] = a.w + row * wbytes + 16 * g;
    wsc[m] = a.ws + row * blocks;
  }
  constexpr int kXBytes = kRows == kRowsMx ? 1 : kRows == kRowsBf16 ? 2 : 4;
  const uint8_t* xq[kNT];
  const uint8_t* xsc[kNT];
#pragma unroll
  for (int n = 0; n < kNT; ++n) {
    int64_t row = min(static_cast<int64_t>(first) + n * 16 + r, static_cast<int64_t>(end - 1));
    if (a.rows) row = a.rows[row];
    row = max(int64_t{0}, min(row, a.T - 1));
    xq[n] = a.x + row * a.K * kXBytes + (kBits == 8 ? 16 : 32 * kXBytes) * g;
    xsc[n] = a.xs + row * blocks;
  }
  floatx4 acc[kGroups][kNT];
#pragma unroll
  for (int m = 0; m < kGroups; ++m)
#pragma unroll
    for (int n = 0; n < kNT; ++n) acc[m][n] = floatx4{0, 0, 0, 0};

  const int whole = a.K / kTile;
  TileData<kBits, kRows, kGroups, kNT> t[2];
  // k-tiles wave, wave + kWaves, ..: `n` of them
  const int n = wave < whole ? (whole - 1 - wave) / kFewWaves + 1 : 0;
  auto load = [&](auto& d, int i) {
    const int kt = wave + min(i, n - 1) * kFewWaves;   // (past the last: the last again, not used)
#pragma unroll
    for (int m = 0; m < kGroups; ++m) d.w[m].load(wq[m], wsc[m], kt);
#pragma unroll
    for (int k = 0; k < kNT; ++k) d.x[k].load(xq[k], xsc[k], kt);
  };
  if (n > 0) {
    load(t[0], 0);
    int i = 0;
#pragma clang loop unroll(disable)
    for (; i + 2 <= n; i += 2) {
      load(t[1], i + 1);
      multiply<0>(t[0], g, acc);
      load(t[0], i + 2);
      multiply<0>(t[1], g, acc);
    }
    if (i < n) multiply<0>(t[0], g, acc);
  }
  if (wave == whole % kFewWaves && blocks % 4) {   // the blocks of a last, partial k-tile
#pragma unroll
    for (int m = 0; m < kGroups; ++m) t[0].w[m].load_part(wq[m], wsc[m], whole, blocks % 4, g);
#pragma unroll
    for (int k = 0; k < kNT; ++k) t[0].x[k].load_part(xq[k], xsc[k], whole, blocks % 4, g);
    multiply<0>(t[0], g, acc);
  }

  constexpr int kPitch = 16 * kGroups + 4;
  float* mine = part + wave * (16 * kNT * kPitch);
#pragma unroll
  for (int m = 0; m < kGroups; ++m)
#pragma unroll
    for (int k = 0; k < kNT; ++k)
      *reinterpret_cast<floatx4*>(mine + (k * 16 + r) * kPitch + m * 16 + 4 * g) = acc[m][k];
  __syncthreads();
  finish<kRows, kGroups, 16 * kNT, kFewWaves, kSwiglu, kMxOut>(a, part, first, end, n0, No);
  __syncthreads();
}

template <int kBits, int kRows, int kGroups, int kNT, bool kSwiglu, bool kMxOut>
__global__ __launch_bounds__(kFewWaves* kWave) void few_products(FewArgs a) {
  __shared__ float part[kFewWaves * 16 * kNT * (16 * kGroups + 4)];
  const int e = blockIdx.y;
  int begin = 0, end = a.R;
  if (a.offsets) {
    begin = max(0, min(a.offsets[e], a.R));
    end = max(begin, min(a.offsets[e + 1], a.R));
  }
  const int64_t step = static_cast<int64_t>(gridDim.z) * (16 * kNT);
  for (int64_t first = begin + static_cast<int64_t>(blockIdx.z) * (16 * kNT); first < end; first += step)
    few_strip<kBits, kRows, kGroups, kNT, kSwiglu, kMxOut>(a, e, static_cast<int>(first), end, blockIdx.x, part);
}

// --------------------------------------------------------------------------
// At most 16 rows, K >= 256
// --------------------------------------------------------------------------
// A k-tile is 128 bytes of every row of w: 128 numbers, or 256 in 4 bits. Each wave has a
// contiguous part of K and a ring of kStages k-tiles of its own in LDS, one multiplied and
// the others in flight, so no wave waits for another before the sum. Scales are put in LDS
// first, for kPhase numbers of every row.
constexpr int kPhase = 8192, kScalePitch = kPhase / kMxBlock + 16;   // (16 rows on different banks)

__device__ u32x4 few_zeros[1];     // what is loaded in place of numbers past K (never written)

#if defined(__HIP_DEVICE_COMPILE__)
// 16 scale bytes of a row from block `at` on, 0 past the last.
__device__ __forceinline__ u32x4 load_scales16(const uint8_t* row, int at, int blocks) {
  if (blocks >= 16) {
    const int from = min(at, blocks - 16), over = at - from;
    typedef uint32_t Odd __attribute__((ext_vector_type(4), aligned(1)));
    const Odd d = *reinterpret_cast<const Odd*>(row + from);
    const unsigned __int128 v = __builtin_bit_cast(unsigned __int128, (u32x4){d[0], d[1], d[2], d[3]});
    return __builtin_bit_cast(u32x4, over < 16 ? v >> (8 * over) : 0);
  }
  u32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (at + i < blocks) v[i >> 2] |= static_cast<uint32_t>(row[at + i]) << (8 * (i & 3));
  return v;
}
#endif

// kXRows: rows of x in LDS.
template <int kBits, int kRows, int kGroups, int kXRows, int kWaves, int kStages, bool kSwiglu, bool kMxOut>
__global__ __launch_bounds__(kWaves* kWave) void stream_products(FewArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr bool kMxRows = kRows == kRowsMx;
  constexpr int kUnit = kBits == 8 ? 128 : 256;                  // numbers of a k-tile
  constexpr int kPer = kUnit / 8;                                // of a chunk (16 bytes) of w
  constexpr int kXEs = kMxRows ? 1 : kRows == kRowsBf16 ? 2 : 4;
  constexpr int kXPer = kUnit * kXEs / 16;                       // chunks of a row of x
  constexpr int kWUnits = 16 * kGroups * 8;                      // chunks of a stage
  constexpr int kWLoads = 2 * kGroups, kXLoads = (kXRows * kXPer + 63) / 64, kLoads = kWLoads + kXLoads;
  constexpr int kStage = kWUnits + kXLoads * 64;
  constexpr int kSRows = 16 * kGroups + (kMxRows ? 16 : 0);      // rows of scales
  // distinct objects: an access to one stage does not wait for loads into another
  __shared__ u32x4 s0[kWaves][kStage], s1[kWaves][kStage], s2[kStages > 2 ? kWaves : 1][kStages > 2 ? kStage : 1];
  __shared__ __align__(16) uint8_t scale[kSRows * kScalePitch];
  static_assert(kStages == 2 || kStages == 3, "stages");
  static_assert(kWaves * 16 * (16 * kGroups + 4) * 4 <= kWaves * kStage * 16, "the sums fit a stage");
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r = lane & 15, g = lane >> 4;
  const int e = blockIdx.y;
  int begin = 0, end = a.R;
  if (a.offsets) {
    begin = max(0, min(a.offsets[e], a.R));
    end = max(begin, min(a.offsets[e + 1], a.R));
  }
  if (begin == end) return;
  constexpr int kOuts = kSwiglu ? 8 * kGroups : 16 * kGroups;
  constexpr int kHalf = kSwiglu ? kGroups / 2 : kGroups;
  const int No = kSwiglu ? a.N / 2 : a.N;
  const int n0 = blockIdx.x * kOuts;
  const int blocks = a.K / kMxBlock;
  const int64_t wbytes = static_cast<int64_t>(a.K) * kBits / 8;
  // row lr of the strip (those past the last are the last again: not stored)
  auto w_row = [&](int lr) {
    const int m = lr >> 4;
    return min(n0 + (m % kHalf) * 16 + (lr & 15), No - 1) + (m < kHalf ? 0 : No);
  };
  auto x_row = [&](int lr) {
    int64_t row = min(begin + lr, end - 1);
    if (a.rows) row = a.rows[row];
    return max(int64_t{0}, min(row, a.T - 1));
  };
  const uint64_t left = static_cast<uint64_t>(a.N - n0) * wbytes;
  const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(a.w + (static_cast<int64_t>(e) * a.N + n0) * wbytes), 0,
      static_cast<int>(left < 0x7fffffff ? left : 0x7fffffff), kRawBuffer);
  uint32_t w_off[kWLoads];
#pragma unroll
  for (int j = 0; j < kWLoads; ++j)
    w_off[j] = static_cast<uint32_t>((w_row(j * 8 + (lane >> 3)) - n0) * wbytes) + ((lane & 7) ^ (lane >> 3) ^ (j & 1)) * 16;
  // chunk c of row lr of x lies at c ^ swizzle(lr), so that 16 rows' reads are on different banks
  auto swizzle = [](int lr) { return kXPer == 8 ? (lr & 7) ^ ((lr >> 3) & 1) : lr & 15; };
  const uint8_t* xp[kXLoads];
  int xc[kXLoads];
#pragma unroll
  for (int j = 0; j < kXLoads; ++j) {
    const int lr = min((j * 64 + lane) / kXPer, kXRows - 1);
    xc[j] = (lane % kXPer) ^ swizzle(lr);
    xp[j] = a.x + x_row(lr) * (static_cast<int64_t>(a.K) * kXEs) + xc[j] * 16;
  }
  floatx4 acc[kGroups];
#pragma unroll
  for (int m = 0; m < kGroups; ++m) acc[m] = floatx4{0, 0, 0, 0};

  for (int p0 = 0; p0 < a.K; p0 += kPhase) {
    const int units = (min(a.K - p0, kPhase) + kUnit - 1) / kUnit;
    // this wave's k-tiles of the phase
    const int k0 = p0 / kUnit + units * wave / kWaves, k1 = p0 / kUnit + units * (wave + 1) / kWaves;
    auto load = [&](u32x4* st, int kt) {
      const int at = __builtin_amdgcn_readfirstlane(kt);
      const bool mine = at < k1;     // (past this wave's last: nothing is read)
#pragma unroll
      for (int j = 0; j < kWLoads; ++j) {
        const int c = (lane & 7) ^ (lane >> 3) ^ (j & 1);
        const uint32_t past = mine && (at * 8 + c) * kPer < a.K ? 0 : kPast;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(st + j * 64), 16, w_off[j] | past, at * 128, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < kXLoads; ++j) {
        const bool in = mine && at * kUnit + xc[j] * (16 / kXEs) < a.K;
        const uint8_t* p = in ? xp[j] + static_cast<int64_t>(at) * (kUnit * kXEs) : reinterpret_cast<const uint8_t*>(few_zeros);
        __builtin_amdgcn_global_load_lds((global_void*)p, (lds_void*)(st + kWUnits + j * 64), 16, 0, 0);
      }
    };
    // scales, sixteen bytes a thread; behind them the first k-tiles
    constexpr int kChunks = kPhase / kMxBlock / 16, kTurns = (kSRows * kChunks + kWaves * kWave - 1) / (kWaves * kWave);
    u32x4 sv[kTurns];
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
      const int at = threadIdx.x + i * kWaves * kWave, lr = min(at / kChunks, kSRows - 1), c = at % kChunks;
      const uint8_t* row = kMxRows && lr >= 16 * kGroups ? a.xs + x_row(lr - 16 * kGroups) * blocks
                                                         : a.ws + (static_cast<int64_t>(e) * a.N + w_row(lr)) * blocks;
      sv[i] = u32x4{0, 0, 0, 0};
      if (p0 / kMxBlock + c * 16 < blocks) sv[i] = load_scales16(row, p0 / kMxBlock + c * 16, blocks);
    }
    load(s0[wave], k0);
    if constexpr (kStages > 2) load(s1[wave], k0 + 1);
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
      const int at = threadIdx.x + i * kWaves * kWave;
      if (at < kSRows * kChunks)
        *reinterpret_cast<u32x4*>(scale + (at / kChunks) * kScalePitch + (at % kChunks) * 16) = sv[i];
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");

    auto multiply = [&](const u32x4* st, int kt) {
      const int swz = (r & 7) ^ (r >> 3);
      const int rx = min(r, kXRows - 1);
      const u32x4* sx = st + kWUnits + rx * kXPer;
      const int xf = swizzle(rx);
      const int b0 = kt * (kUnit / kMxBlock) - p0 / kMxBlock;     // its first block in the phase
      uint32_t below = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int c = 4 * u + g;       // this lane's chunk of w: its block's scale is
        const int b = b0 + (kBits == 8 ? c >> 1 : c);
        u32x4 w[kGroups];
        float wf[kGroups];
#pragma unroll
        for (int m = 0; m < kGroups; ++m) {
          w[m] = st[(m * 16 + r) * 8 + (c ^ swz)];
          wf[m] = mx_scale(scale[(m * 16 + r) * kScalePitch + b]);
        }
        float xfactor = 0.0f;
        if constexpr (kMxRows) xfactor = mx_scale(scale[(16 * kGroups + r) * kScalePitch + b]);
#pragma unroll
        for (int o = 0; o < kPer / 8; ++o) {      // eight numbers of the chunk
          if constexpr (kRows == kRowsF32) {
            const Split x = split_bf16(sx[(8 * c + 2 * o) ^ xf], sx[(8 * c + 2 * o + 1) ^ xf]);
#pragma unroll
            for (int m = 0; m < kGroups; ++m) {
              const u32x4 v = widen4(w[m][o], wf[m]);
              acc[m] = mma16<false>(v, x.low, acc[m]);
              acc[m] = mma16<false>(v, x.mid, acc[m]);
              acc[m] = mma16<false>(v, x.top, acc[m]);
            }
            below |= x.below;
          } else {
            u32x4 x;
            if constexpr (kRows == kRowsBf16) {
              x = sx[(4 * c + o) ^ xf];
            } else {
              const u32x4 v = kBits == 8 ? sx[c ^ xf] : sx[(2 * c + o / 2) ^ xf];
              const uint32_t d = v[2 * (o & 1)], f = v[2 * (o & 1) + 1];
              x = u32x4{mx_pair_bf16<8, 0>(d, xfactor), mx_pair_bf16<8, 1>(d, xfactor),
                        mx_pair_bf16<8, 0>(f, xfactor), mx_pair_bf16<8, 1>(f, xfactor)};
            }
#pragma unroll
            for (int m = 0; m < kGroups; ++m) {
              u32x4 v;
              if constexpr (kBits == 4) {
                v = widen4(w[m][o], wf[m]);
              } else {
                const uint32_t d = w[m][2 * o], f = w[m][2 * o + 1];
                v = u32x4{mx_pair_bf16<8, 0>(d, wf[m]), mx_pair_bf16<8, 1>(d, wf[m]), mx_pair_bf16<8, 0>(f, wf[m]),
                          mx_pair_bf16<8, 1>(f, wf[m])};
              }
              acc[m] = mma16<false>(v, x, acc[m]);
            }
          }
        }
      }
      if constexpr (kRows == kRowsF32) {
        if (any_below(below)) {
          // what the three parts could not hold (numbers below 2^-110)
#pragma clang loop unroll(disable)
          for (int i = 0; i < 8; ++i) {
            const int c = (i & 4) + g, o = i & 3;
            const Split x = split_rest(sx[(8 * c + 2 * o) ^ xf], sx[(8 * c + 2 * o + 1) ^ xf]);
#pragma unroll
            for (int m = 0; m < kGroups; ++m) {
              const uint32_t d = reinterpret_cast<const uint32_t*>(st + (m * 16 + r) * 8 + (c ^ swz))[o];
              const u32x4 v = widen4(d, scale_down(mx_scale(scale[(m * 16 + r) * kScalePitch + b0 + c])));
              acc[m] = mma16<false>(v, x.mid, acc[m]);
              acc[m] = mma16<false>(v, x.top, acc[m]);
            }
          }
        }
      }
    };
    // A k-tile: it has landed (sent since: kStages - 2 others); the next one not yet sent
    // goes where the one before lay, which this wave has read.
    auto one = [&](u32x4* st, u32x4* next, int kt) {
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(kLoads * (kStages - 2), false));
      asm volatile("" ::: "memory");
      load(next, kt + kStages - 1);
      multiply(st, kt);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    };
    int kt = k0;
#pragma clang loop unroll(disable)
    for (; kt + kStages <= k1; kt += kStages) {
      one(s0[wave], kStages == 2 ? s1[wave] : s2[wave], kt);
      one(s1[wave], s0[wave], kt + 1);
      if constexpr (kStages > 2) one(s2[wave], s1[wave], kt + 2);
    }
    // the last, fewer than kStages: all have been sent
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if (kt < k1) multiply(s0[wave], kt);
    if (kStages > 2 && kt + 1 < k1) multiply(s1[wave], kt + 1);
    __syncthreads();    // the scales, and at the end the stages, are free
  }
  float* part = reinterpret_cast<float*>(s0);
  constexpr int kPitch = 16 * kGroups + 4;
#pragma unroll
  for (int m = 0; m < kGroups; ++m)
    *reinterpret_cast<floatx4*>(part + (wave * 16 + r) * kPitch + m * 16 + 4 * g) = acc[m];
  __syncthreads();
  finish<kRows, kGroups, 16, kWaves, kSwiglu, kMxOut>(a, part, begin, end, n0, No);
#endif  // __HIP_DEVICE_COMPILE__
}

template <int kBits, int kRows, bool kSwiglu, bool kMxOut>
struct Launch {
  static constexpr int kGroups = kSwiglu && kMxOut ? 4 : 2;
  static dim3 grid(const FewArgs& a, int E) {
    const int No = kSwiglu ? a.N / 2 : a.N;
    return dim3(static_cast<uint32_t>(cdiv(No, kSwiglu ? 8 * kGroups : 16 * kGroups)), static_cast<uint32_t>(E));
  }
  template <int kNT>
  static void few(const FewArgs& a, int E, hipStream_t st) {
    // rows beside each other, too, up to some thousand blocks
    dim3 g = grid(a, E);
    const int64_t chunks = cdiv(a.R, 16 * kNT), room = cdiv(4096, static_cast<int64_t>(g.x) * g.y);
    g.z = static_cast<uint32_t>(chunks < room ? chunks : room);
    few_products<kBits, kRows, kGroups, kNT, kSwiglu, kMxOut><<<g, kFewWaves * kWave, 0, st>>>(a);
  }
  template <int kXRows, int kWaves, int kStages>
  static void stream(const FewArgs& a, int E, hipStream_t st) {
    stream_products<kBits, kRows, kGroups, kXRows, kWaves, kStages, kSwiglu, kMxOut>
        <<<grid(a, E), kWaves * kWave, 0, st>>>(a);
  }
  // waves by what a stage of each takes of LDS: 4 KiB of w (8 with four groups) and x
  static void any(const FewArgs& a, int E, hipStream_t st) {
    if (a.R > 16) few<4>(a, E, st);
    else if (a.K < 256 || (kRows == kRowsF32 && a.R > 4)) few<1>(a, E, st);   // (16 rows of fp32 are too much LDS)
    else if constexpr (kRows == kRowsF32) stream<4, 6, 3>(a, E, st);
    else if constexpr (kRows == kRowsBf16) {
      if (a.R <= 4) stream<4, 8, 3>(a, E, st);
      else stream<16, 4, 3>(a, E, st);
    } else if constexpr (kGroups == 4) {
      if constexpr (kBits == 8) stream<16, 4, 3>(a, E, st);
      else if (a.R <= 4) stream<4, 4, 3>(a, E, st);
      else stream<16, 3, 3>(a, E, st);
    } else if constexpr (kBits == 8) {
      stream<16, 8, 3>(a, E, st);
    } else {
      if (a.R <= 4) stream<4, 8, 3>(a, E, st);
      else stream<16, 6, 3>(a, E, st);
    }
  }
};

template <int kBits, int kRows, bool kSwiglu, bool kMxOut>
void launch_rows(const FewArgs& a, int E, hipStream_t st) {
  Launch<kBits, kRows, kSwiglu, kMxOut>::any(a, E, st);
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
                      const int* offsets, const int* rows, void* y, void* ys, hipStream_t st) {
  const FewArgs a{static_cast<const uint8_t*>(x), static_cast<const uint8_t*>(xs),
                  static_cast<const uint8_t*>(w), static_cast<const uint8_t*>(ws), offsets, rows, y,
                  static_cast<uint8_t*>(ys), d.T, static_cast<int>(d.R), static_cast<int>(d.K),
                  static_cast<int>(d.N)};
  if (d.bits == 4) launch_experts<4>(d, a, st);
  else launch_experts<8>(d, a, st);
  return hipGetLastError();
}

hipError_t linear4_few(const tr_linear4_desc& d, const void* x, const void* w, const void* ws, void* y,
                       hipStream_t st) {
  const FewArgs a{static_cast<const uint8_t*>(x), nullptr, static_cast<const uint8_t*>(w),
                  static_cast<const uint8_t*>(ws), nullptr, nullptr, y, nullptr, d.T,
                  static_cast<int>(d.T), static_cast<int>(d.K), static_cast<int>(d.N)};
  if (d.dtype == TR_F32) launch_rows<4, kRowsF32, false, false>(a, 1, st);
  else launch_rows<4, kRowsBf16, false, false>(a, 1, st);
  return hipGetLastError();
}

}  // namespace tr
