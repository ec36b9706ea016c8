// Products grouped by expert with rows in 8 bits and weights in 8 or 4, in blocks of 32
// with scales (tr_mx.h), for experts with many rows.
//
//   y[r][n] = sum over k of x[rows[r]][k] w[e][n][k]; with SwiGLU silu(gate) * up
//
// 256 x 256 block tiles with k-tiles of 128 on the matrix instructions that take such
// blocks (v_mfma_scale_f32_32x32x64_f8f6f4, twice the bf16 rate): four waves, each 128 x
// 128 in 256 accumulation registers, every other 32 rows by 128 neighbouring rows of w. A
// row of a k-tile is 128 bytes (64 for weights in 4 bits), so bytes, LDS reads and
// instruction times are those of bf16 tiles with k-tiles of 64, and twice the numbers. The
// instruction's operands: lane 32 h + r holds of row r the 16-byte chunks h and 2 + h of a
// step's four (in 4 bits the one chunk h of two), and the scale of the row's block h. It
// adds products in groups of eight, aligned to the largest with 13 bits kept, to fp32 sums:
// 1.5e-5 of a sum's norm as a rule, a hundredth of the rounding to bf16 of results of that size,
// for twice the rate of widened operands.
//
// Both operands go from memory to LDS without registers, into the stage of two that the
// step before has finished reading. A step (k-tile) is 32 matrix instructions a wave, 64
// cycles each, and everything else lies between them, spread so that no unit gets a burst:
//   0..7    the second half's fragments come from LDS, two reads each
//   10      the stage is free (a barrier)
//   10..25  one load to LDS each, of the k-tile after next
//   20      the next k-tile has landed (a barrier)
//   20..27  its first half's fragments come, and its scales
// so a load has 27 to 42 instructions, 1700 to 2700 cycles, to land. Scales go through
// registers to LDS, eight bytes of every row for two k-tiles.
//
// An expert's rows go over its m-tiles as evenly as units of 64 allow, and a wave leaves out
// the instructions of row blocks past its tile's rows (of 64 rows 8 of 32 a step are left).
// Against full tiles and a last one in full: 32 experts, 7168 x 2048, 2048 / 4096 / 8192
// rows 126 / 136 / 179 -> 121 / 132 / 174 us, 4 bits 7168 x 4096, 4096 rows 174 -> 163; one
// expert of 8192 rows pays 1% for the branches (425 -> 432). The rests of all experts after
// all whole tiles would even out the blocks' work more, but brings their weights in twice:
// 8192 rows 196 us.
//
// Scheduling is on the device from the offsets: groups of kGroupM m-tiles by all n-tiles,
// in contiguous runs for each of the 8 XCDs, whose L2s then hold a group's rows and
// weights. Rows past a segment and chunks past K are loads from past the buffer: zeros
// without an access.
//
// Bound by the matrix instructions and the power they take: 8192^3 in 8 bits 421-430 us (2.6
// PFLOP/s, the library's product 2.65; of zeros 3.8), 16384 rows over 32 experts with uneven
// counts 477-508 at 7168 x 4096 with SwiGLU and 265-288 at 2048 x 7168 (1.7-2.0 PFLOP/s).
#include "tr_internal.h"
#include "tr_mx.h"

namespace tr {
namespace {

constexpr int kThreads = 256;
constexpr int BM = 256, BN = 256, BK = 128;
constexpr int kGroupM = 4;
constexpr int kShare = 56;     // rows an expert from which 256-row tiles are faster than 64-row ones

struct MxArgs {
  const uint8_t* x;        // [T, K]
  const uint8_t* xs;       // [T, K / 32]
  const uint8_t* w;        // [E, N, K] of kBits
  const uint8_t* ws;       // [E, N, K / 32]
  const int* offsets;      // [E + 1]
  const int* rows;         // [R] or NULL
  void* y;                 // [R, No] bf16 or 8 bits
  uint8_t* ys;             // [R, No / 32]
  int64_t T;
  int R, K, N, E;
  int share;               // rows an expert from which mx_tiles takes a call, and below mx_mid; 0: no other is launched
};

#if defined(__HIP_DEVICE_COMPILE__)

typedef int intx8 __attribute__((ext_vector_type(8)));

// Distinct objects, so that an access to one stage does not wait for loads into the
// other.
__shared__ u32x4 g_a0[BM * 8], g_a1[BM * 8];   // 256 rows of 128 bytes
__shared__ u32x4 g_b0[BN * 8], g_b1[BN * 8];   // (4 bits: the first half)
__shared__ uint2 g_sa[2][BM], g_sb[2][BN];     // scales of a row's eight blocks

template <int S>
__device__ __forceinline__ u32x4* stage_a() { return S == 0 ? g_a0 : g_a1; }
template <int S>
__device__ __forceinline__ u32x4* stage_b() { return S == 0 ? g_b0 : g_b1; }

struct Tile {
  int e, row0, valid, n0;
};

// Where a tile's operands come from, for this wave and lane. A wave moves 64 rows of
// each operand, in pieces of 1 KiB: 8 rows of 8 chunks, or 16 rows of 4.
template <int kBits>
struct Source {
  static constexpr int kBPieces = kBits;
  __amdgpu_buffer_rsrc_t a, b;
  uint32_t a_off[8];      // of piece j, chunk of k-tile 0
  uint32_t b_off;         // of piece 0
  int b_pieces;           // pieces whose row (this lane's) is an output
  const uint8_t* sa;      // scales of this lane's row of 64 of x, and of w
  const uint8_t* sb;
};

template <int kBits>
struct Lane {
  int a_chunk, b_chunk;   // chunk of this lane in piece 0
  uint32_t b_step;        // bytes from a piece of w to the next
};

// The row of x of row wave * 64 + lane of a tile.
__device__ __forceinline__ int x_row(const MxArgs& a, const Tile& t, int wave, int lane) {
  const int lr = min(wave * 64 + lane, t.valid - 1);
  return a.rows ? a.rows[t.row0 + lr] : lr;     // (within the tile where rows are not gathered)
}

// `row`: x_row of the tile.
template <int kBits, bool kSwiglu>
__device__ __forceinline__ Source<kBits> source(const MxArgs& a, const Tile& t, int row, int wave, int lane) {
  asm volatile("" : "+v"(row));   // (waited for here, not where it is loaded)
  if (a.rows) row = max(0, min(row, static_cast<int>(a.T) - 1));
  Source<kBits> s;
  const int blocks = a.K / kMxBlock;
  const int64_t kb = static_cast<int64_t>(a.K) * kBits / 8;   // bytes of a row of w
  const int No = kSwiglu ? a.N / 2 : a.N;
  // x: piece j has rows wave * 64 + 8 j + lane / 8; row r's chunk c lies at c ^ f(r),
  // f(r) = (r & 7) ^ (r >> 3 & 1), which keeps 16 rows' reads on different banks
  const uint8_t* base = a.rows ? a.x : a.x + static_cast<int64_t>(t.row0) * a.K;
  const uint64_t a_bytes = a.rows ? static_cast<uint64_t>(a.T) * a.K : static_cast<uint64_t>(t.valid) * a.K;
  s.a = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, static_cast<int>(a_bytes), kRawBuffer);
  const int chunk = (lane & 7) ^ (lane >> 3);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int lr = wave * 64 + j * 8 + (lane >> 3);
    const uint32_t r = __shfl(row, j * 8 + (lane >> 3), kWave);
    s.a_off[j] = lr < t.valid ? r * static_cast<uint32_t>(a.K) + (chunk ^ (j & 1)) * 16 : kPast;
  }
  const int64_t srow = a.rows ? row : t.row0 + row;
  s.sa = a.xs + srow * blocks;
  // w: gate rows first, then up
  const uint8_t* wbase = a.w + static_cast<int64_t>(t.e) * a.N * kb;
  const int64_t w_bytes = a.N * kb;
  s.b = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(wbase), 0, static_cast<int>(w_bytes), kRawBuffer);
  const int first = kSwiglu ? t.n0 + (wave & 1) * 64 : t.n0 + wave * 64;   // output of this wave's row 0
  const int up = kSwiglu && wave >= 2 ? No : 0;
  constexpr int kRows = kBits == 8 ? 8 : 16;    // of a piece
  const int lr = lane / (64 / kRows);
  const int bchunk = kBits == 8 ? chunk : (lane & 3) ^ ((lane >> 4) & 3);
  s.b_off = static_cast<uint32_t>(up + first + lr) * static_cast<uint32_t>(kb) + bchunk * 16;
  const int left = No - first - lr;
  s.b_pieces = left > 0 ? (left + kRows - 1) / kRows : 0;
  s.sb = a.ws + (static_cast<int64_t>(t.e) * a.N + up + min(first + lane, No - 1)) * blocks;
  return s;
}

template <int S, int kBits>
__device__ __forceinline__ void load_a(const Source<kBits>& s, int kt, uint32_t past, int wave, int j) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(s.a, (lds_void*)(stage_a<S>() + wave * 512 + j * 64), 16,
                                           s.a_off[j] | past, kt * BK, 0, 0);
}

template <int S, int kPolicy, int kBits>
__device__ __forceinline__ void load_b(const Source<kBits>& s, int kt, uint32_t past, uint32_t step, int wave, int j) {
  uint32_t off = s.b_off;
  if constexpr (kBits == 8) {
    if (j & 1) off ^= 16;     // (f of rows 8..15; a row's start is a multiple of 32)
  }
  off = j < s.b_pieces ? off + j * step : kPast;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(s.b, (lds_void*)(stage_b<S>() + wave * (64 * kBits) + j * 64), 16,
                                           off | past, kt * (BK * kBits / 8), 0, kPolicy);
}

template <int kBits>
struct Frags {
  intx8 a[2][4], b[2][4];   // of a step's two halves: rows of x, rows of w
  uint32_t sa[2][4], sb[2][4];   // of this k-tile and the next: scales (shift_scales: from block h on)
  floatx16 acc[4][4];       // acc[i][j]: row block i, block j of rows of w
};

struct Geo {
  int a_row, b_row[4];      // first row of this wave's blocks (of rows of x: every other, 64 apart)
  int a_unit[2][2];         // per half: unit in a row block of its two chunks
  int b_unit[2][2];
};

typedef __attribute__((ext_vector_type(4))) int intx4;

// Fragment n of half P of stage S: rows of w first, whose four the first instructions need.
template <int S, int P, int kBits>
__device__ __forceinline__ void read_frag(Frags<kBits>& f, const Geo& g, int n) {
  if (n >= 4) {
    const u32x4* s = stage_a<S>() + (g.a_row + (n - 4) * 64) * 8;
    f.a[P][n - 4] = __builtin_shufflevector(__builtin_bit_cast(intx4, s[g.a_unit[P][0]]),
                                            __builtin_bit_cast(intx4, s[g.a_unit[P][1]]), 0, 1, 2, 3, 4, 5, 6, 7);
  } else if constexpr (kBits == 8) {
    const u32x4* s = stage_b<S>() + g.b_row[n] * 8;
    f.b[P][n] = __builtin_shufflevector(__builtin_bit_cast(intx4, s[g.b_unit[P][0]]),
                                        __builtin_bit_cast(intx4, s[g.b_unit[P][1]]), 0, 1, 2, 3, 4, 5, 6, 7);
  } else {
    const u32x4 v = stage_b<S>()[g.b_row[n] * 4 + g.b_unit[P][0]];
    f.b[P][n] = intx8{static_cast<int>(v[0]), static_cast<int>(v[1]), static_cast<int>(v[2]),
                      static_cast<int>(v[3]), 0, 0, 0, 0};
  }
}

// Scales of row block n of the k-tile in half S of LDS buffer `buf`.
template <int S, int kBits>
__device__ __forceinline__ void read_scale(Frags<kBits>& f, const Geo& g, int buf, int lane, int n) {
  const uint2* p = &g_sa[buf][g.a_row + n * 64 + (lane & 31)];
  f.sa[S][n] = S == 0 ? p->x : p->y;
  const uint2* q = &g_sb[buf][g.b_row[n] + (lane & 31)];
  f.sb[S][n] = S == 0 ? q->x : q->y;
}

template <int S, int kBits>
__device__ __forceinline__ void shift_scales(Frags<kBits>& f, int lane) {
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    f.sa[S][n] >>= 8 * (lane >> 5);
    f.sb[S][n] >>= 8 * (lane >> 5);
  }
}

// Matrix instruction m of half P of a step in stage S.
template <int S, int P, int kBits>
__device__ __forceinline__ void mma(Frags<kBits>& f, int m) {
  const int i = m >> 2, j = m & 3;
  f.acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(f.b[P][j], f.a[P][i], f.acc[i][j],
                                                                kBits == 4 ? 4 : 0, 0, 2 * P, f.sb[S][j], 2 * P,
                                                                f.sa[S][i]);
}

// Step of the k-tile in stage S, whose first half's fragments and scales are in
// registers. `src`, `kt`: what comes into this stage next; `buf`: the scale buffer of the
// next k-tile. kScales (the first step of a pair): the next pair's scales are loaded, and
// written to buffer `into`. `active`: row blocks with rows.
template <int S, bool kScales, int kPolicy, int kBits>
__device__ __forceinline__ void step(Frags<kBits>& f, const Geo& g, const Source<kBits>& src, int kt, int K,
                                     int a_chunk, int b_chunk, uint32_t b_step, int buf, int into, int active,
                                     int wave, int lane) {
  constexpr int kFree = 10, kLanded = 20, kLoads = 8 + Source<kBits>::kBPieces;
  const int blocks = K / kMxBlock;
  uint2 na{}, nb{};
  if constexpr (kScales) {
    na = load_scale8(src.sa, kt * 4, blocks);
    nb = load_scale8(src.sb, kt * 4, blocks);
  }
  shift_scales<S>(f, lane);
  // chunks past K (pairs of them: K is a multiple of 32)
  const uint32_t past_a = kt * 8 + a_chunk < K / 16 ? 0 : kPast;
  const uint32_t past_b = kBits == 8 ? past_a : (kt * 4 + b_chunk < K / 32 ? 0 : kPast);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int m = 0; m < 32; ++m) {
    if (m == kFree) {
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(63, true));   // this wave's reads of the stage are done
      lds_barrier();
    }
    if (m == kLanded) {
      // what the step before sent has landed
      constexpr int kSent = kLoads < kLanded - kFree ? kLoads : kLanded - kFree;
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(kSent, false));
      lds_barrier();
      if constexpr (kScales) {
        // (not shifted, and so not waited for, before this)
        asm volatile("" : "+v"(na.x), "+v"(na.y), "+v"(nb.x), "+v"(nb.y));
        g_sa[into][wave * 64 + lane] = scale8(na, kt * 4, blocks);
        g_sb[into][wave * 64 + lane] = scale8(nb, kt * 4, blocks);
      }
    }
    if (m < 8) read_frag<S, 1>(f, g, m);
    if (m >= kLanded && m < kLanded + 8) read_frag<1 - S, 0>(f, g, m - kLanded);
    if (m >= kLanded && m < kLanded + 4) read_scale<1 - S>(f, g, buf, lane, m - kLanded);
    if (((m >> 2) & 3) < active) {
      if (m < 16) mma<S, 0>(f, m);
      else mma<S, 1>(f, m - 16);
    }
    const int n = m - kFree;
    if (n >= 0 && n < 8) load_a<S>(src, kt, past_a, wave, n);
    else if (n >= 8 && n < kLoads) load_b<S, kPolicy>(src, kt, past_b, b_step, wave, n - 8);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Tile L of the order.
__device__ __forceinline__ Tile tile_of(const int* pre, const int* cnt, const int* off, int E, int total_m, int NT,
                                        int outs, int L) {
  const int group = L / (kGroupM * NT);
  const int first = group * kGroupM;
  const int size = min(total_m - first, kGroupM);
  const int within = L - group * kGroupM * NT;
  const int gm = first + within % size;
  int lo = 0, hi = E;      // pre[lo] <= gm < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= gm) lo = mid; else hi = mid;
  }
  Tile t;
  t.e = __builtin_amdgcn_readfirstlane(lo);
  // an expert's rows, in units of 64, as evenly over its m-tiles as they go
  const int mt = __builtin_amdgcn_readfirstlane(gm - pre[t.e]);
  const int count = __builtin_amdgcn_readfirstlane(cnt[t.e]);
  const int units = static_cast<int>((static_cast<uint32_t>(count) + 63) / 64), mts = (units + 3) / 4;
  const int per = units / mts, more = units - per * mts;
  const int at = 64 * (mt * per + min(mt, more));
  t.row0 = __builtin_amdgcn_readfirstlane(off[t.e]) + at;
  t.valid = min(64 * (per + (mt < more ? 1 : 0)), count - at);
  t.n0 = within / size * outs;
  return t;
}

// Eight neighbouring outputs from column `col` of a row of bf16.
__device__ __forceinline__ void store_bf16(uint16_t* row, int col, int No, const u32x4& v) {
  if (col + 8 <= No) {
    typedef uint32_t Odd __attribute__((ext_vector_type(4), aligned(2)));
    *reinterpret_cast<Odd*>(row + col) = Odd{v[0], v[1], v[2], v[3]};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < No) row[col + i] = static_cast<uint16_t>(v[i >> 1] >> (16 * (i & 1)));
  }
}

// A 32 x 32 block of results: v[4 q + c] is column col + 8 q + 4 h + c of `row` (the
// lane's; h = lane / 32), stored where the row is `in` its segment.
template <bool kMxOut>
__device__ __forceinline__ void store_block(const MxArgs& a, int64_t row, bool in, int col, int No, int h,
                                            const floatx16& v) {
  if constexpr (kMxOut) {
    float top = 0.0f;
#pragma unroll
    for (int c = 0; c < 16; ++c) top = fmaxf(top, mx_magnitude(v[c]));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    const int b = mx_scale_byte<8>(top);
    const float inv = mx_inverse(b);
    uint32_t d[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      d[q] = mx_pack8(v[4 * q] * inv, v[4 * q + 1] * inv, v[4 * q + 2] * inv, v[4 * q + 3] * inv);
    // lanes below 32: columns 0..15, the others 16..31
    const auto p0 = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
    const auto p1 = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
    if (in && col < No) {
      *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(a.y) + row * No + col + 16 * h) =
          u32x4{p0[0], p0[1], p1[0], p1[1]};
      if (h == 0) a.ys[row * (No / kMxBlock) + col / kMxBlock] = static_cast<uint8_t>(b);
    }
  } else {
    uint32_t d[4][2];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      d[q][0] = cvt_bf16x2(v[4 * q], v[4 * q + 1]);
      d[q][1] = cvt_bf16x2(v[4 * q + 2], v[4 * q + 3]);
    }
    uint16_t* out = static_cast<uint16_t*>(a.y) + row * No;
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
      // lanes below 32: columns 8 q + [0, 8), the others 8 (q + 1) + [0, 8)
      const auto p0 = __builtin_amdgcn_permlane32_swap(d[q][0], d[q + 1][0], false, false);
      const auto p1 = __builtin_amdgcn_permlane32_swap(d[q][1], d[q + 1][1], false, false);
      if (in) store_bf16(out, col + 8 * (q + h), No, u32x4{p0[0], p1[0], p0[1], p1[1]});
    }
  }
}

#endif  // __HIP_DEVICE_COMPILE__

template <int kBits, bool kSwiglu, bool kMxOut, int kPolicy>
__global__ __launch_bounds__(kThreads) void mx_tiles(MxArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int kOuts = kSwiglu ? BN / 2 : BN;   // of a tile
  __shared__ int pre[kMaxE + 1], cnt[kMaxE], off[kMaxE], tmp[kThreads / kWave];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // the experts' m-tiles
  constexpr int kPer = kMaxE / kThreads;
  int mine[kPer], sum = 0, rows = 0, some = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    mine[i] = 0;
    if (e < a.E) {
      const int begin = max(0, min(a.offsets[e], a.R)), end = max(begin, min(a.offsets[e + 1], a.R));
      off[e] = begin;
      cnt[e] = end - begin;
      mine[i] = static_cast<int>((static_cast<uint32_t>(end - begin) + BM - 1) / BM);   // (unsigned: up to 2^31 - 1 rows)
      rows += end - begin;
      some += end > begin ? 1 : 0;
    }
    sum += mine[i];
  }
  if (a.share > 0) {
    int all, experts;
    block_exclusive_scan<kThreads>(rows, tmp, &all);
    block_exclusive_scan<kThreads>(some, tmp, &experts);
    if (all < a.share * experts) return;
  }
  int total_m;
  int at = block_exclusive_scan<kThreads>(sum, tmp, &total_m);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    if (e < a.E) pre[e] = at;
    at += mine[i];
  }
  if (tid == 0) pre[a.E] = total_m;
  __syncthreads();

  const int No = kSwiglu ? a.N / 2 : a.N;
  const int NT = (No + kOuts - 1) / kOuts;
  const int total = total_m * NT;
  const int G = gridDim.x;
  int pos = blockIdx.x;
  if ((G & 7) == 0) pos = (pos & 7) * (G >> 3) + (pos >> 3);
  if (pos >= total) return;

  const int h = lane >> 5;
  Geo g;
  g.a_row = (wave >> 1) * 32;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    g.b_row[j] = kSwiglu ? (j < 2 ? (wave & 1) * 64 + j * 32 : 128 + (wave & 1) * 64 + (j - 2) * 32)
                         : (wave & 1) * 128 + j * 32;
  const int swz = (lane & 7) ^ ((lane >> 3) & 1);
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    g.a_unit[p][0] = (lane & 31) * 8 + ((4 * p + h) ^ swz);
    g.a_unit[p][1] = (lane & 31) * 8 + ((4 * p + 2 + h) ^ swz);
    if constexpr (kBits == 8) {
      g.b_unit[p][0] = g.a_unit[p][0];
      g.b_unit[p][1] = g.a_unit[p][1];
    } else {
      g.b_unit[p][0] = g.b_unit[p][1] = (lane & 31) * 4 + ((2 * p + h) ^ ((lane >> 2) & 3));
    }
  }
  const int a_chunk = (lane & 7) ^ (lane >> 3);
  const int b_chunk = kBits == 8 ? a_chunk : (lane & 3) ^ ((lane >> 4) & 3);
  const uint32_t b_step = (kBits == 8 ? 8u : 16u) * static_cast<uint32_t>(a.K) * kBits / 8;
  const int pairs = (a.K + 2 * BK - 1) / (2 * BK);

  Tile t = tile_of(pre, cnt, off, a.E, total_m, NT, kOuts, pos);
  Source<kBits> s0 = source<kBits, kSwiglu>(a, t, x_row(a, t, wave, lane), wave, lane);
  Frags<kBits> f;
  int buf = 0;     // of the current pair's scales
  {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t past_a = q * 8 + a_chunk < a.K / 16 ? 0 : kPast;
      const uint32_t past_b =
          kBits == 8 ? (q * 8 + b_chunk < a.K / 16 ? 0 : kPast) : (q * 4 + b_chunk < a.K / 32 ? 0 : kPast);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (q == 0) load_a<0>(s0, q, past_a, wave, j);
        else load_a<1>(s0, q, past_a, wave, j);
      }
#pragma unroll
      for (int j = 0; j < Source<kBits>::kBPieces; ++j) {
        if (q == 0) load_b<0, kPolicy>(s0, q, past_b, b_step, wave, j);
        else load_b<1, kPolicy>(s0, q, past_b, b_step, wave, j);
      }
    }
    g_sa[0][wave * 64 + lane] = load_scale8(s0.sa, 0, a.K / kMxBlock);
    g_sb[0][wave * 64 + lane] = load_scale8(s0.sb, 0, a.K / kMxBlock);
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0, true));
    lds_barrier();
#pragma unroll
    for (int n = 0; n < 8; ++n) read_frag<0, 0>(f, g, n);
#pragma unroll
    for (int n = 0; n < 4; ++n) read_scale<0>(f, g, 0, lane, n);
  }

#pragma clang loop unroll(disable)
  for (int L = pos; L < total; L += G) {
    {
      // accumulators start as products of zeros, in their own registers (zeros that
      // differ to the compiler: it would make one product, and 15 copies of it)
#pragma unroll
      for (int m = 0; m < 16; ++m) {
        int zero = 0;
        asm volatile("" : "+v"(zero));
        const bf16x8 zf = __builtin_bit_cast(bf16x8, (intx4){zero, zero, zero, zero});
        f.acc[m >> 2][m & 3] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(zf, zf, floatx16{}, 0, 0, 0);
      }
    }
    // past the last tile: this one again, in bounds and not used
    const Tile tn = L + G < total ? tile_of(pre, cnt, off, a.E, total_m, NT, kOuts, L + G) : t;
    const int rn = x_row(a, tn, wave, lane);   // (used in the last pair)
    const int active = (t.valid - g.a_row + 63) >> 6;
    // (one loop that runs at least once: no copy of the accumulators, one of the steps)
    int p = 1;
#pragma clang loop unroll(disable)
    do {
      int kt = 2 * p;
      if (p == pairs) {     // what comes next is the next tile's
        s0 = source<kBits, kSwiglu>(a, tn, rn, wave, lane);
        kt = 0;
      }
      step<0, true, kPolicy>(f, g, s0, kt, a.K, a_chunk, b_chunk, b_step, buf, buf ^ 1, active, wave, lane);
      step<1, false, kPolicy>(f, g, s0, kt + 1, a.K, a_chunk, b_chunk, b_step, buf ^ 1, 0, active, wave, lane);
      buf ^= 1;
    } while (p++ < pairs);

    // the accumulators stay where they are up to their block's turn
    settle(f.acc[0][0]);
#pragma unroll
    for (int m = 1; m < 16; ++m) settled(f.acc[m >> 2][m & 3]);
    // acc[i][j][4 q + c]: row lane & 31 of row block i, column 8 q + 4 h + c of block j
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int lr = g.a_row + i * 64 + (lane & 31);
      const int64_t row = static_cast<int64_t>(t.row0) + lr;
#pragma unroll
      for (int j = 0; j < (kSwiglu ? 2 : 4); ++j) {
        floatx16 v = f.acc[i][j];
        asm volatile("" : "+v"(v));
        if constexpr (kSwiglu) {
          floatx16 u = f.acc[i][j + 2];
          asm volatile("" : "+v"(u));
#pragma unroll
          for (int c = 0; c < 16; ++c) v[c] = swiglu<false>(v[c], u[c]);
        }
        const int col = t.n0 + g.b_row[j];
        store_block<kMxOut>(a, row, lr < t.valid, col, No, h, v);
        __builtin_amdgcn_sched_barrier(0);   // one block at a time
      }
    }
    t = tn;
  }
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(0, true));   // loads past the last tile
#endif  // __HIP_DEVICE_COMPILE__
}

// --------------------------------------------------------------------------
// Smaller tiles, a block each: where the experts have too few rows, or the call too few
// tiles, for the loop above.
// --------------------------------------------------------------------------
// kBM x 128 (SwiGLU: 64 gate and 64 up rows of w); a k-tile is 128 bytes of every row of
// w, 128 numbers or, in 4 bits, 256 (with 64 bytes of a row at a time, 434 MB of weights
// in 4 bits came at 3.8 TB/s). kStages stages, one being multiplied and the others in
// flight. Wave (m, n) of 2 x 2 has kBM / 2 rows by 64, for SwiGLU 32 gate and the matching
// 32 up; with 32 rows wave (p, n) has them all and half p of every k-tile, and the halves'
// sums are added in LDS.
//
// Bound by reading the weights, two blocks a CU, 64 to 80 KiB in flight on it: 8 experts of a
// row, 7168 x 4096, 8 bits 39 us (6.2 TB/s); 64 rows over 32 of them, 4 bits 76 (5.7), 2048 x
// 7168 in 8 bits 68 (6.2); 256 rows, 8 bits 143 (6.8).
#if defined(__HIP_DEVICE_COMPILE__)
constexpr int kMidN = 128;

#endif

template <int kBits, int kBM, int kStages, bool kSwiglu, bool kMxOut, int kPolicy>
__global__ __launch_bounds__(kThreads) void mx_mid(MxArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int kOuts = kSwiglu ? kMidN / 2 : kMidN;
  constexpr bool kHalves = kBM == 32;        // waves share a k-tile's halves
  constexpr int kI = kHalves ? 1 : kBM / 64; // row blocks of a wave
  constexpr int kSub = kBits == 8 ? 1 : 2;   // 128 numbers of a k-tile
  constexpr int kAPieces = kBM / 32;         // of a wave, of 128 numbers: 8 rows each
  constexpr int kBPieces = 4;
  constexpr int kLoads = kAPieces * kSub + kBPieces;
  // (distinct objects, as above)
  constexpr int kA = kBM * 8 * kSub, kB = kMidN * 8;
  static_assert(kStages == 2 || kStages == 3, "stages");
  __shared__ u32x4 a0[kA], a1[kA], a2[kStages > 2 ? kA : 1];
  __shared__ u32x4 b0[kB], b1[kB], b2[kStages > 2 ? kB : 1];
  auto sa_of = [&](auto i) -> u32x4* {
    constexpr int k = decltype(i)::value;
    if constexpr (k == 0) return a0;
    else if constexpr (k == 1) return a1;
    else return a2;
  };
  auto sb_of = [&](auto i) -> u32x4* {
    constexpr int k = decltype(i)::value;
    if constexpr (k == 0) return b0;
    else if constexpr (k == 1) return b1;
    else return b2;
  };
  using Ring = ScaleRing<kSub, kBM + kMidN, 4>;
  __shared__ __align__(16) uint32_t sc[Ring::kSize];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int No = kSwiglu ? a.N / 2 : a.N;
  const int NT = (No + kOuts - 1) / kOuts;
  // The experts' m-tiles, each wave for itself: lane l has experts l per .. l per + per - 1.
  const int per = (a.E + kWave - 1) / kWave;
  auto segment = [&](int i, int* begin, int* end) {
    const int e = lane * per + i;
    *begin = max(0, min(a.offsets[min(e, a.E)], a.R));
    *end = max(*begin, min(a.offsets[min(e + 1, a.E)], a.R));
    return (*end - *begin + kBM - 1) / kBM;
  };
  int begin, end, mine = 0, rows = 0, some = 0;
  for (int i = 0; i < per; ++i) {
    mine += segment(i, &begin, &end);
    rows += end - begin;
    some += end > begin ? 1 : 0;
  }
  if (a.share > 0) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) rows += __shfl_xor(rows, d, kWave), some += __shfl_xor(some, d, kWave);
    if (rows >= a.share * some) return;
  }
  int upto = mine;      // m-tiles of this lane's and all lower lanes' experts
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int o = __shfl_up(upto, d, kWave);
    if (lane >= d) upto += o;
  }
  const int total_m = __builtin_amdgcn_readlane(upto, kWave - 1);
  // contiguous tiles for each XCD; an expert's m-tiles of one n-tile one after another
  const int total = total_m * NT;
  const int share = (total + 7) / 8;
  const int idx = blockIdx.x >> 3;
  const int L = static_cast<int>(blockIdx.x & 7) * share + idx;
  if (idx >= share || L >= total) return;
  Tile t;
  {
    const int gm = L / NT;
    const int who = __builtin_amdgcn_readfirstlane(__popcll(__ballot(upto <= gm)));   // the lane that has it
    int first = upto - mine, mts = 1, id = 0, at = 0, last = 0;
    for (int i = 0, next = first; i < per; ++i) {
      const int m = per == 1 ? mine : segment(i, &begin, &end);
      if (next <= gm && gm < next + m) first = next, mts = m, id = lane * per + i, at = begin, last = end;
      next += m;
    }
    t.e = __builtin_amdgcn_readlane(id, who);
    first = __builtin_amdgcn_readlane(first, who);
    mts = __builtin_amdgcn_readlane(mts, who);
    at = __builtin_amdgcn_readlane(at, who);
    last = __builtin_amdgcn_readlane(last, who);
    const int within = L - first * NT;
    t.n0 = within / mts * kOuts;
    t.row0 = at + within % mts * kBM;
    t.valid = min(kBM, last - t.row0);
  }
  const int blocks = a.K / kMxBlock;
  const int64_t kb = static_cast<int64_t>(a.K) * kBits / 8;
  const int chunk = (lane & 7) ^ (lane >> 3);
  const uint8_t* abase = a.rows ? a.x : a.x + static_cast<int64_t>(t.row0) * a.K;
  const uint64_t a_bytes = a.rows ? static_cast<uint64_t>(a.T) * a.K : static_cast<uint64_t>(t.valid) * a.K;
  const __amdgpu_buffer_rsrc_t ra =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(abase), 0, static_cast<int>(a_bytes), kRawBuffer);
  const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(a.w + static_cast<int64_t>(t.e) * a.N * kb), 0, static_cast<int>(a.N * kb), kRawBuffer);
  // a row of the tile of w: outputs, for SwiGLU gate and then up
  auto w_row = [&](int lr, bool* in) {
    const int n = t.n0 + (kSwiglu ? lr & 63 : lr);
    *in = n < No;
    return min(n, No - 1) + (kSwiglu && lr >= 64 ? No : 0);
  };
  uint32_t b_off[kBPieces];
#pragma unroll
  for (int j = 0; j < kBPieces; ++j) {
    const int lr = wave * 32 + j * 8 + (lane >> 3);
    bool in;
    const uint32_t row = w_row(lr, &in);
    b_off[j] = in ? row * static_cast<uint32_t>(kb) + (chunk ^ (j & 1)) * 16 : kPast;
  }
  const int steps = (a.K + BK * kSub - 1) / (BK * kSub);
  auto load_b = [&](u32x4* sb, int kt) {
    const int b_at = __builtin_amdgcn_readfirstlane(kt * 128);
#pragma unroll
    for (int j = 0; j < kBPieces; ++j) {
      const uint32_t past = kt * 8 + (chunk ^ (j & 1)) < a.K / (kBits == 8 ? 16 : 32) ? 0 : kPast;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void*)(sb + wave * 256 + j * 64), 16, b_off[j] | past, b_at, 0,
                                               kPolicy);
    }
  };
  // x's rows: of this lane's pieces, and of its turns of scales. They are looked up while w's
  // first k-tile comes.
  int a_row_of[kAPieces], s_row_of[Ring::kTurns];
#pragma unroll
  for (int j = 0; j < kAPieces; ++j) a_row_of[j] = min(wave * (kBM / 4) + j * 8 + (lane >> 3), t.valid - 1);
#pragma unroll
  for (int i = 0; i < Ring::kTurns; ++i) s_row_of[i] = min(Ring::row_of(i, wave, lane), t.valid - 1);
  if (a.rows) {
#pragma unroll
    for (int j = 0; j < kAPieces; ++j) a_row_of[j] = a.rows[t.row0 + a_row_of[j]];
#pragma unroll
    for (int i = 0; i < Ring::kTurns; ++i)
      if (Ring::row_of(i, 0, 0) < kBM) s_row_of[i] = a.rows[t.row0 + s_row_of[i]];
  }
  asm volatile("" ::: "memory");
  load_b(b0, 0);
#pragma unroll
  for (int j = 0; j < kAPieces; ++j) asm volatile("" : "+v"(a_row_of[j]));   // (waited for from here on)
#pragma unroll
  for (int i = 0; i < Ring::kTurns; ++i) asm volatile("" : "+v"(s_row_of[i]));
  uint32_t a_off[kAPieces];
#pragma unroll
  for (int j = 0; j < kAPieces; ++j) {
    const int lr = wave * (kBM / 4) + j * 8 + (lane >> 3);
    uint32_t row = a_row_of[j];
    if (a.rows) row = max(0, min(a_row_of[j], static_cast<int>(a.T) - 1));
    a_off[j] = lr < t.valid ? row * static_cast<uint32_t>(a.K) + (chunk ^ ((lr >> 3) & 1)) * 16 : kPast;
  }
  // scales: rows of x, then of w
  Ring ring;
  ring.blocks = blocks, ring.first = wave * Ring::kPart, ring.lane = lane;
#pragma unroll
  for (int i = 0; i < Ring::kTurns; ++i) {
    const int lr = Ring::row_of(i, wave, lane);
    const int64_t xr =
        a.rows ? max(0, min(s_row_of[i], static_cast<int>(a.T) - 1)) : static_cast<int64_t>(t.row0) + s_row_of[i];
    bool in;
    const int64_t wr = static_cast<int64_t>(t.e) * a.N + w_row(max(lr - kBM, 0), &in);
    ring.row[i] = lr < kBM ? a.xs + xr * blocks : a.ws + wr * blocks;
  }
  auto load_a = [&](u32x4* sa, int kt) {
    const int a_at = __builtin_amdgcn_readfirstlane(kt * (BK * kSub));   // (the scalar offset stays scalar)
#pragma unroll
    for (int u = 0; u < kSub; ++u) {
      // (chunks c and c ^ 1 are past K together: K is a multiple of 32)
      const uint32_t past = (kt * kSub + u) * 8 + chunk < a.K / 16 ? 0 : kPast;
#pragma unroll
      for (int j = 0; j < kAPieces; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(sa + u * (kBM * 8) + wave * (kBM * 2) + j * 64), 16,
                                                 a_off[j] | past, a_at + u * BK, 0, 0);
    }
  };
  const int h = lane >> 5, l31 = lane & 31;
  const int a_row = kHalves ? 0 : (wave >> 1) * (kBM / 2), wn = wave & 1;
  const int half = kHalves ? wave >> 1 : 0;
  const int b_row[2] = {kSwiglu ? wn * 32 : wn * 64, kSwiglu ? 64 + wn * 32 : wn * 64 + 32};
  const int swz = (lane & 7) ^ ((lane >> 3) & 1);
  floatx16 acc[kI][2];
#pragma unroll
  for (int i = 0; i < kI; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int c = 0; c < 16; ++c) acc[i][j][c] = 0.0f;
  // 64 numbers at a time: q = 0 .. 2 kSub - 1, of which a wave has all, or its half
  constexpr int kQ = kHalves ? kSub : 2 * kSub;
  auto multiply = [&](const u32x4* sa, const u32x4* sb, const uint32_t* s) {
    intx8 fa[kQ][kI], fb[kQ][2];
    uint32_t fs[kQ][kI], gs[kQ][2];
#pragma unroll
    for (int i = 0; i < kQ; ++i) {
      const int q = kHalves ? half * kSub + i : i;
      const int u = q >> 1, p = q & 1;
      // (in 8 bits half p is known to the wave only: its scales are shifted by 16 p)
      const int shift = 8 * h + (kHalves && kSub == 1 ? 16 * p : 0);
#pragma unroll
      for (int m = 0; m < kI; ++m) {
        const int row = a_row + m * 32 + l31;
        const u32x4* r = sa + u * (kBM * 8) + row * 8;
        fa[i][m] = __builtin_shufflevector(__builtin_bit_cast(intx4, r[(4 * p + h) ^ swz]),
                                           __builtin_bit_cast(intx4, r[(4 * p + 2 + h) ^ swz]), 0, 1, 2, 3, 4, 5, 6, 7);
        fs[i][m] = s[row * kSub + u] >> shift;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const u32x4* r = sb + (b_row[j] + l31) * 8;
        if constexpr (kBits == 8) {
          fb[i][j] = __builtin_shufflevector(__builtin_bit_cast(intx4, r[(4 * p + h) ^ swz]),
                                             __builtin_bit_cast(intx4, r[(4 * p + 2 + h) ^ swz]), 0, 1, 2, 3, 4, 5, 6,
                                             7);
        } else {
          const u32x4 v = r[(2 * q + h) ^ swz];
          fb[i][j] = intx8{static_cast<int>(v[0]), static_cast<int>(v[1]), static_cast<int>(v[2]),
                           static_cast<int>(v[3]), 0, 0, 0, 0};
        }
        gs[i][j] = s[(kBM + b_row[j] + l31) * kSub + u] >> shift;
      }
    }
    constexpr int kFormat = kBits == 4 ? 4 : 0;
#pragma unroll
    for (int i = 0; i < kQ; ++i)
#pragma unroll
      for (int m = 0; m < kI; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (i % 2 == 0 || kQ == 1)
            acc[m][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[i][j], fa[i][m], acc[m][j], kFormat, 0, 0,
                                                                        gs[i][j], 0, fs[i][m]);
          else
            acc[m][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[i][j], fa[i][m], acc[m][j], kFormat, 0, 2,
                                                                        gs[i][j], 2, fs[i][m]);
        }
  };
  // Step kt, in stage kt % kStages: scales loaded kStages steps before go to LDS, its
  // operands have landed; then the loads of step kt + kStages - 1, into the stage that the
  // step before has read.
  typename Ring::Window v[kStages], all[Ring::kTurns];
#pragma unroll
  for (int i = 0; i < Ring::kTurns; ++i) ring.load_from(all[i], ring.row[i], 0);
  ring.load(v[0], 0);
  auto fill = [&](auto i) {
    constexpr int k = decltype(i)::value;
    if constexpr (k + 1 < kStages) {
      ring.load(v[k + 1], k + 1);
      if constexpr (k > 0) load_b(sb_of(i), k);
      load_a(sa_of(i), k);
      asm volatile("" ::: "memory");
    }
  };
  fill(Index<0>{}), fill(Index<1>{});
#pragma unroll
  for (int i = 0; i < Ring::kTurns; ++i) ring.store_to(all[i], sc, i, 0);
  auto stage = [&](auto i, int kt) {
    constexpr int k = decltype(i)::value;
    if constexpr (k < kStages) {
      ring.store(v[k], sc, kt);
      // sent since this step's operands: scales and operands of kStages - 2 steps
      __builtin_amdgcn_s_waitcnt(waitcnt_vm((kLoads + 2) * (kStages - 2), true));
      lds_barrier();
      ring.load(v[k], kt + kStages);
      constexpr int next = (k + kStages - 1) % kStages;
      load_b(sb_of(Index<next>{}), kt + kStages - 1);
      load_a(sa_of(Index<next>{}), kt + kStages - 1);
      multiply(sa_of(i), sb_of(i), Ring::slot(sc, kt));
    }
  };
  int kt = 0;
#pragma clang loop unroll(disable)
  for (; kt + kStages <= steps; kt += kStages)
    stage(Index<0>{}, kt), stage(Index<1>{}, kt + 1), stage(Index<2>{}, kt + 2);
  // The last steps, fewer than kStages: everything they need has been sent.
  auto put = [&](auto i) {
    constexpr int k = decltype(i)::value;
    if constexpr (k + 1 < kStages) ring.store(v[k], sc, kt + k);
  };
  put(Index<0>{}), put(Index<1>{});
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(0, true));   // (loads past the last k-tile, too)
  lds_barrier();
  auto rest = [&](auto i) {
    constexpr int k = decltype(i)::value;
    if constexpr (k + 1 < kStages) {
      if (kt + k < steps) multiply(sa_of(i), sb_of(i), Ring::slot(sc, kt + k));
    }
  };
  rest(Index<0>{}), rest(Index<1>{});
  settle(acc[0][0]);
#pragma unroll
  for (int m = 1; m < 2 * kI; ++m) settled(acc[m >> 1][m & 1]);
  if constexpr (kHalves) {
    float* sum = reinterpret_cast<float*>(b0);    // a block of 32 x 32 for each of two waves
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      __syncthreads();
      floatx4* mine = reinterpret_cast<floatx4*>(sum) + wn * 256 + lane;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (half == 1)
          mine[c * 64] = floatx4{acc[0][j][4 * c], acc[0][j][4 * c + 1], acc[0][j][4 * c + 2], acc[0][j][4 * c + 3]};
      __syncthreads();
      if (half == 0) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const floatx4 o = mine[c * 64];
#pragma unroll
          for (int b = 0; b < 4; ++b) acc[0][j][4 * c + b] += o[b];
        }
      }
    }
    if (half == 1) return;
  }
#pragma unroll
  for (int i = 0; i < kI; ++i) {
    const int lr = a_row + i * 32 + l31;
    if constexpr (kSwiglu) {
      floatx16 v;
#pragma unroll
      for (int c = 0; c < 16; ++c) v[c] = swiglu<false>(acc[i][0][c], acc[i][1][c]);
      store_block<kMxOut>(a, t.row0 + lr, lr < t.valid, t.n0 + b_row[0], No, h, v);
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        store_block<kMxOut>(a, t.row0 + lr, lr < t.valid, t.n0 + b_row[j], No, h, acc[i][j]);
    }
  }
#endif  // __HIP_DEVICE_COMPILE__
}

// Tiles of kBM rows of `rows` rows, at most.
int64_t mid_tiles(const tr_expert_desc& d, int64_t rows, int bm) {
  return (rows / bm + d.E) * cdiv(d.swiglu ? d.N / 2 : d.N, d.swiglu ? 64 : 128);
}
// (a block each: a launch has fewer than 2^32 threads)
constexpr int64_t kMostTiles = (int64_t{1} << 24) - 8;

template <int kBits, int kBM, int kStages, int kPolicy>
void launch_mid(const tr_expert_desc& d, const MxArgs& a, hipStream_t st) {
  const int64_t tiles = mid_tiles(d, a.share > 0 ? int64_t{a.share} * d.E : d.R, kBM);
  const uint32_t blocks = static_cast<uint32_t>(cdiv(tiles, 8) * 8);
  if (d.swiglu && d.out) mx_mid<kBits, kBM, kStages, true, true, kPolicy><<<blocks, kThreads, 0, st>>>(a);
  else if (d.swiglu) mx_mid<kBits, kBM, kStages, true, false, kPolicy><<<blocks, kThreads, 0, st>>>(a);
  else if (d.out) mx_mid<kBits, kBM, kStages, false, true, kPolicy><<<blocks, kThreads, 0, st>>>(a);
  else mx_mid<kBits, kBM, kStages, false, false, kPolicy><<<blocks, kThreads, 0, st>>>(a);
}

template <int kBits, int kPolicy>
void launch(const tr_expert_desc& d, const MxArgs& a, hipStream_t st) {
  const uint32_t blocks = static_cast<uint32_t>(device_cu_count());
  if (d.swiglu && d.out) mx_tiles<kBits, true, true, kPolicy><<<blocks, kThreads, 0, st>>>(a);
  else if (d.swiglu) mx_tiles<kBits, true, false, kPolicy><<<blocks, kThreads, 0, st>>>(a);
  else if (d.out) mx_tiles<kBits, false, true, kPolicy><<<blocks, kThreads, 0, st>>>(a);
  else mx_tiles<kBits, false, false, kPolicy><<<blocks, kThreads, 0, st>>>(a);
}

// The kernel's form by the weights' bits, and whether they are read once (kOnce). Measured,
// us a pass, read so against not: 32 experts, 7168 x 4096, 32 / 256 / 1024 rows 121 / 172 / 191
// against 128 / 183 / 201, in 4 bits 64 / 91 / 109 against 68 / 98 / 118; 2048 x 7168, 64 rows 68
// against 76. 51 MB of weights, which are there from the call before, 40 against 26.
// 256-row tiles, 2048 / 4096 / 16384 rows: 178 / 192 / 506 against 199 / 212 / 477 (more rows
// read them more than once), in 4 bits (half a line a load) 153 against 139.
template <int kBM, int k8Stages, int k4Stages>
void launch_mid(const tr_expert_desc& d, const MxArgs& a, hipStream_t st) {
  const bool once = read_once(d.E * d.N * d.K * d.bits / 8);
  if (d.bits == 4) once ? launch_mid<4, kBM, k4Stages, kOnce>(d, a, st) : launch_mid<4, kBM, k4Stages, kKept>(d, a, st);
  else once ? launch_mid<8, kBM, k8Stages, kOnce>(d, a, st) : launch_mid<8, kBM, k8Stages, kKept>(d, a, st);
}

void launch(const tr_expert_desc& d, const MxArgs& a, hipStream_t st) {
  const int64_t experts = d.R < d.E ? d.R : d.E;
  if (d.bits == 4) launch<4, kKept>(d, a, st);
  else if (read_once(d.E * d.N * d.K) && d.R <= 192 * experts) launch<8, kOnce>(d, a, st);
  else launch<8, kKept>(d, a, st);
}

}  // namespace

// Which kernel, by what is known on the host: the experts with a row are at most
// min(E, R), and have some R / min(E, R) rows each (tiles: half an m-tile of each expert is
// empty; an n-tile is 128 or 256 rows of w). Measured, us a pass:
//  - ROWS (a CU's weights in one burst, K shared by its waves) where one block a CU has all:
//    1 expert of 16 rows, 7168 x 7168: 12.7 (8 bits), 10.2 (4), against 24.8 and 16.0 with
//    32-row tiles; 8 experts of a row, 7168 x 4096: 53, against 38.
//  - 256-row tiles from 56 rows an expert, with tiles for half the CUs: 32 experts, 7168 x
//    4096, 1024 / 1536 / 2048 rows: 176 / 177 / 178 (in 4 bits 134 / 136 / 139), against 157 /
//    184 / 258 (97 / 120 / 154) with 64-row tiles; 2048 x 7168, 1536 / 2048 rows: 112 / 115,
//    against 97 / 138; 4 experts, 4096 x 4096, 1000 / 2000 rows: 54 / 58, against 46 / 70.
//  - of the others 32-row tiles for up to 20 rows an expert, or where 64-row tiles are for
//    three quarters of the CUs at most (two of them run on one): 32 experts, 7168 x 4096, 640 / 1024 rows:
//    157 / 215 (in 4 bits 94 / 130), against 151 / 157 (94 / 97) with 64-row tiles; 1 expert of
//    64 / 128 / 256 rows, 7168 x 7168: 28 / 29 / 40 (17 / 18 / 27), against 30 / 33 / 35 (28 / 28
//    / 29).
tr_expert_kernel expert_kernel(const tr_expert_desc& d, bool gather) {
  const int64_t outs = d.swiglu ? d.N / 2 : d.N;
  // (gathered rows are addressed with 31 bits, tiles are numbered with 31)
  const int64_t most = (cdiv(d.R, 32) + d.E) * cdiv(outs, d.swiglu ? 64 : 128);
  const bool tiles = d.K >= 256 && (!gather || d.T * d.K < (int64_t{1} << 31)) && most < (int64_t{1} << 30);
  const bool blocks = most < kMostTiles;
  if (d.kernel == TR_EXPERT_ROWS || (d.kernel == TR_EXPERT_AUTO && !tiles)) return TR_EXPERT_ROWS;
  if (!tiles) return TR_EXPERT_AUTO;
  if (d.kernel == TR_EXPERT_TILE256 || (d.kernel == TR_EXPERT_AUTO && !blocks)) return TR_EXPERT_TILE256;
  if (!blocks) return TR_EXPERT_AUTO;
  if (d.kernel != TR_EXPERT_AUTO) return static_cast<tr_expert_kernel>(d.kernel);
  const int64_t cus = device_cu_count(), experts = d.R < d.E ? d.R : d.E;
  if (d.R <= 16 && experts * cdiv(outs, d.swiglu && !d.out ? 16 : 32) <= cus) return TR_EXPERT_ROWS;
  auto m_tiles = [&](int64_t rows) {
    const int64_t m = d.R / rows + (experts + 1) / 2;
    return m > experts ? m : experts;
  };
  if (d.R >= kShare * experts && m_tiles(256) * cdiv(outs, d.swiglu ? 128 : 256) * 2 >= cus) return TR_EXPERT_TILE256;
  if (d.R <= 20 * experts || m_tiles(64) * cdiv(outs, d.swiglu ? 64 : 128) * 4 <= cus * 3) return TR_EXPERT_TILE32;
  return TR_EXPERT_TILE64;
}

hipError_t expert_tiles(const tr_expert_desc& d, tr_expert_kernel kernel, const void* x, const void* xs,
                        const void* w, const void* ws, const int* offsets, const int* rows, void* y, void* ys,
                        bool bound, hipStream_t st) {
  MxArgs a{static_cast<const uint8_t*>(x), static_cast<const uint8_t*>(xs),
           static_cast<const uint8_t*>(w), static_cast<const uint8_t*>(ws), offsets, rows, y,
           static_cast<uint8_t*>(ys), d.T, static_cast<int>(d.R), static_cast<int>(d.K),
           static_cast<int>(d.N), d.E, 0};
  // (stages: as many as leave room for two blocks on a CU; six and one block: one token's
  // experts 50 -> 52 us, 64 tokens' in 4 bits 90 -> 103)
  if (kernel == TR_EXPERT_TILE32) launch_mid<32, 3, 3>(d, a, st);
  else if (kernel == TR_EXPERT_TILE64) launch_mid<64, 3, 2>(d, a, st);
  else if (!bound || mid_tiles(d, int64_t{kShare} * d.E, 64) >= kMostTiles) launch(d, a, st);
  else {
    // With the rows that the segments do hold, the kernels themselves say which of the two
    // takes the call. R 8192, 32 experts, 7168 x 4096, 8 and 4 bits, 1365 rows there: 198, 138
    // -> 168, 106 us; the launch that does nothing costs 4 to 7.
    a.share = kShare;
    launch_mid<64, 3, 2>(d, a, st);
    launch(d, a, st);
  }
  return hipGetLastError();
}

}  // namespace tr
