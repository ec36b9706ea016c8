// Products grouped by expert with rows in 8 bits and weights in 8 or 4, in blocks of 32
// with scales (tr_mx.h), for experts with many rows.
//
//   y[r][n] = sum over k of x[rows[r]][k] w[e][n][k]; with SwiGLU silu(gate) * up
//
// 256 x 256 block tiles with k-tiles of 128 on the matrix instructions that take such
// blocks (v_mfma_scale_f32_32x32x64_f8f6f4, twice the bf16 rate): four waves, each a 128 x
// 128 quadrant in 256 accumulation registers. A row of a k-tile is 128 bytes (64 for
// weights in 4 bits), so bytes, LDS reads and instruction times are those of bf16 tiles
// with k-tiles of 64, and twice the numbers. The instruction's operands: lane 32 h + r
// holds of row r the 16-byte chunks h and 2 + h of a step's four (in 4 bits the one chunk
// h of two), and the scale of the row's block h.
//
// Both operands go from memory to LDS without registers, into the stage of two that the
// step before has finished reading. A step (k-tile) is 32 matrix instructions a wave, 64
// cycles each:
//   0..7    the second half's fragments come from LDS; then the stage is free (a barrier)
//   8..23   one load to LDS each, of the k-tile after next
//   24..31  the next k-tile has landed (a barrier); its first half's fragments come
// so a load has 1 to 1.5 steps, 2048 to 3072 cycles, to land. Scales go through registers
// to LDS, eight bytes of every row for two k-tiles.
//
// Scheduling is on the device from the offsets: groups of kGroupM m-tiles by all n-tiles,
// in contiguous runs for each of the 8 XCDs, whose L2s then hold a group's rows and
// weights. Rows past a segment and chunks past K are loads from past the buffer: zeros
// without an access.
#include "tr_internal.h"
#include "tr_mx.h"

namespace tr {
namespace {

constexpr int kThreads = 256;
constexpr int BM = 256, BN = 256, BK = 128;
constexpr int kGroupM = 4;

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
  int least;               // experts with fewer rows are another kernel's
};

#if defined(__HIP_DEVICE_COMPILE__)

constexpr int kBufferFlags = 0x00020000;      // raw buffer, 32-bit data format
constexpr uint32_t kPast = 0x80000000u;       // an offset past every buffer here
typedef int intx8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void;

// Distinct objects, so that an access to one stage does not wait for loads into the
// other.
__shared__ u32x4 g_a0[BM * 8], g_a1[BM * 8];   // 256 rows of 128 bytes
__shared__ u32x4 g_b0[BN * 8], g_b1[BN * 8];   // (4 bits: the first half)
__shared__ uint2 g_sa[2][BM], g_sb[2][BN];     // scales of a row's eight blocks

template <int S>
__device__ __forceinline__ u32x4* stage_a() { return S == 0 ? g_a0 : g_a1; }
template <int S>
__device__ __forceinline__ u32x4* stage_b() { return S == 0 ? g_b0 : g_b1; }

__host__ __device__ constexpr int waitcnt_vm(int n, bool lgkm0) {
  return (n & 15) | ((n >> 4) << 14) | (7 << 4) | ((lgkm0 ? 0 : 15) << 8);
}

__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

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

template <int kBits, bool kSwiglu>
__device__ __forceinline__ Source<kBits> source(const MxArgs& a, const Tile& t, int wave, int lane) {
  Source<kBits> s;
  const int blocks = a.K / kMxBlock;
  const int64_t kb = static_cast<int64_t>(a.K) * kBits / 8;   // bytes of a row of w
  const int No = kSwiglu ? a.N / 2 : a.N;
  // x: piece j has rows wave * 64 + 8 j + lane / 8; row r's chunk c lies at c ^ f(r),
  // f(r) = (r & 7) ^ (r >> 3 & 1), which keeps 16 rows' reads on different banks
  const uint8_t* base = a.rows ? a.x : a.x + static_cast<int64_t>(t.row0) * a.K;
  const uint64_t a_bytes = a.rows ? static_cast<uint64_t>(a.T) * a.K : static_cast<uint64_t>(t.valid) * a.K;
  s.a = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, static_cast<int>(a_bytes), kBufferFlags);
  const int chunk = (lane & 7) ^ (lane >> 3);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int lr = wave * 64 + j * 8 + (lane >> 3);
    uint32_t row = lr;
    if (a.rows) row = max(0, min(a.rows[min(t.row0 + lr, a.R - 1)], static_cast<int>(a.T) - 1));
    s.a_off[j] = lr < t.valid ? row * static_cast<uint32_t>(a.K) + (chunk ^ (j & 1)) * 16 : kPast;
  }
  {
    const int lr = min(wave * 64 + lane, t.valid - 1);
    int64_t row = t.row0 + lr;
    if (a.rows) row = max(0, min(a.rows[row], static_cast<int>(a.T) - 1));
    s.sa = a.xs + row * blocks;
  }
  // w: gate rows first, then up
  const uint8_t* wbase = a.w + static_cast<int64_t>(t.e) * a.N * kb;
  const int64_t w_bytes = a.N * kb;
  s.b = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(wbase), 0, static_cast<int>(w_bytes), kBufferFlags);
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

template <int S, int kBits>
__device__ __forceinline__ void load_b(const Source<kBits>& s, int kt, uint32_t past, uint32_t step, int wave, int j) {
  uint32_t off = s.b_off;
  if constexpr (kBits == 8) {
    if (j & 1) off ^= 16;     // (f of rows 8..15; a row's start is a multiple of 32)
  }
  off = j < s.b_pieces ? off + j * step : kPast;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(s.b, (lds_void*)(stage_b<S>() + wave * (64 * kBits) + j * 64), 16,
                                           off | past, kt * (BK * kBits / 8), 0, 0);
}

// Eight scale bytes of a row from block `at` on, those past the last as 0.
__device__ __forceinline__ uint2 load_scales(const uint8_t* p, int at, int blocks) {
  typedef uint32_t Odd __attribute__((ext_vector_type(2), aligned(1)));
  if (at + 8 <= blocks) {
    const Odd v = *reinterpret_cast<const Odd*>(p + at);
    return uint2{v[0], v[1]};
  }
  uint32_t v[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (at + i < blocks) v[i >> 2] |= static_cast<uint32_t>(p[at + i]) << (8 * (i & 3));
  return uint2{v[0], v[1]};
}

template <int kBits>
struct Frags {
  intx8 a[2][4], b[2][4];   // of a step's two halves: rows of x, rows of w
  uint32_t sa[2][4], sb[2][4];   // of this k-tile and the next: scales, from block h on
  floatx16 acc[4][4];       // acc[i][j]: row block i, block j of rows of w
};

struct Geo {
  int a_row, b_row[4];      // first row of this wave's blocks
  int a_unit[2][2];         // per half: unit in a row block of its two chunks
  int b_unit[2][2];
};

template <int S, int P, int kBits>
__device__ __forceinline__ void read_frags(Frags<kBits>& f, const Geo& g) {
  const u32x4* sa = stage_a<S>();
  const u32x4* sb = stage_b<S>();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const u32x4 lo = sa[(g.a_row + i * 32) * 8 + g.a_unit[P][0]], hi = sa[(g.a_row + i * 32) * 8 + g.a_unit[P][1]];
    f.a[P][i] = __builtin_shufflevector(__builtin_bit_cast(__attribute__((ext_vector_type(4))) int, lo),
                                        __builtin_bit_cast(__attribute__((ext_vector_type(4))) int, hi), 0, 1, 2, 3,
                                        4, 5, 6, 7);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (kBits == 8) {
      const u32x4 lo = sb[g.b_row[j] * 8 + g.b_unit[P][0]], hi = sb[g.b_row[j] * 8 + g.b_unit[P][1]];
      f.b[P][j] = __builtin_shufflevector(__builtin_bit_cast(__attribute__((ext_vector_type(4))) int, lo),
                                          __builtin_bit_cast(__attribute__((ext_vector_type(4))) int, hi), 0, 1, 2,
                                          3, 4, 5, 6, 7);
    } else {
      const u32x4 v = sb[g.b_row[j] * 4 + g.b_unit[P][0]];
      f.b[P][j] = intx8{static_cast<int>(v[0]), static_cast<int>(v[1]), static_cast<int>(v[2]),
                        static_cast<int>(v[3]), 0, 0, 0, 0};
    }
  }
}

// Scales of the k-tile in half S of LDS buffer `buf`.
template <int S, int kBits>
__device__ __forceinline__ void read_scales(Frags<kBits>& f, const Geo& g, int buf, int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint2* p = &g_sa[buf][g.a_row + i * 32 + (lane & 31)];
    f.sa[S][i] = (S == 0 ? p->x : p->y) >> (8 * (lane >> 5));
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint2* p = &g_sb[buf][g.b_row[j] + (lane & 31)];
    f.sb[S][j] = (S == 0 ? p->x : p->y) >> (8 * (lane >> 5));
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
// written to buffer `into`.
template <int S, bool kScales, int kBits>
__device__ __forceinline__ void step(Frags<kBits>& f, const Geo& g, const Source<kBits>& src, int kt, int K,
                                     int a_chunk, int b_chunk, uint32_t b_step, int buf, int into, int wave,
                                     int lane) {
  read_frags<S, 1>(f, g);
  uint2 na{}, nb{};
  if constexpr (kScales) {
    na = load_scales(src.sa, kt * 4, K / kMxBlock);
    nb = load_scales(src.sb, kt * 4, K / kMxBlock);
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int m = 0; m < 8; ++m) mma<S, 0>(f, m);
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(63, true));   // this wave's reads of the stage are done
  barrier();
  // chunks past K (pairs of them: K is a multiple of 32)
  const uint32_t past_a = kt * 8 + a_chunk < K / 16 ? 0 : kPast;
  const uint32_t past_b = kBits == 8 ? (kt * 8 + b_chunk < K / 16 ? 0 : kPast) : (kt * 4 + b_chunk < K / 32 ? 0 : kPast);
#pragma unroll
  for (int m = 8; m < 24; ++m) {
    if (m < 16) mma<S, 0>(f, m);
    else mma<S, 1>(f, m - 16);
    const int n = m - 8;
    if (n < 8) load_a<S>(src, kt, past_a, wave, n);
    else if (n - 8 < Source<kBits>::kBPieces) load_b<S>(src, kt, past_b, b_step, wave, n - 8);
    __builtin_amdgcn_sched_barrier(0);
  }
  // what was sent before this step's loads has landed
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(8 + Source<kBits>::kBPieces, false));
  barrier();
  if constexpr (kScales) {
    g_sa[into][wave * 64 + lane] = na;
    g_sb[into][wave * 64 + lane] = nb;
  }
  read_frags<1 - S, 0>(f, g);
  read_scales<1 - S>(f, g, buf, lane);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int m = 8; m < 16; ++m) mma<S, 1>(f, m);
  __builtin_amdgcn_sched_barrier(0);
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
  const int mt = __builtin_amdgcn_readfirstlane(gm - pre[t.e]);
  t.row0 = __builtin_amdgcn_readfirstlane(off[t.e]) + mt * BM;
  t.valid = min(BM, __builtin_amdgcn_readfirstlane(cnt[t.e]) - mt * BM);
  t.n0 = within / size * outs;
  return t;
}

// Four neighbouring outputs from column `col` of a row of bf16.
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

#endif  // __HIP_DEVICE_COMPILE__

template <int kBits, bool kSwiglu, bool kMxOut>
__global__ __launch_bounds__(kThreads) void mx_tiles(MxArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int kOuts = kSwiglu ? BN / 2 : BN;   // of a tile
  __shared__ int pre[kMaxE + 1], cnt[kMaxE], off[kMaxE], tmp[kThreads / kWave];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // the experts' m-tiles
  constexpr int kPer = kMaxE / kThreads;
  int mine[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    mine[i] = 0;
    if (e < a.E) {
      const int begin = max(0, min(a.offsets[e], a.R)), end = max(begin, min(a.offsets[e + 1], a.R));
      off[e] = begin;
      cnt[e] = end - begin;
      mine[i] = end - begin < a.least ? 0 : (end - begin + BM - 1) / BM;
    }
    sum += mine[i];
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
  g.a_row = (wave >> 1) * 128;
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
  Source<kBits> s0 = source<kBits, kSwiglu>(a, t, wave, lane);
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
        if (q == 0) load_b<0>(s0, q, past_b, b_step, wave, j);
        else load_b<1>(s0, q, past_b, b_step, wave, j);
      }
    }
    g_sa[0][wave * 64 + lane] = load_scales(s0.sa, 0, a.K / kMxBlock);
    g_sb[0][wave * 64 + lane] = load_scales(s0.sb, 0, a.K / kMxBlock);
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0, true));
    barrier();
    read_frags<0, 0>(f, g);
    read_scales<0>(f, g, 0, lane);
  }

#pragma clang loop unroll(disable)
  for (int L = pos; L < total; L += G) {
    {
      // accumulators start as a product of zeros, in their own registers
      bf16x8 zf;
      int zero = 0;
      asm volatile("" : "+v"(zero));
#pragma unroll
      for (int q = 0; q < 8; ++q) zf[q] = __builtin_bit_cast(__bf16, static_cast<uint16_t>(zero));
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          f.acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(zf, zf, floatx16{}, 0, 0, 0);
    }
    // past the last tile: this one again, in bounds and not used
    const Tile tn = L + G < total ? tile_of(pre, cnt, off, a.E, total_m, NT, kOuts, L + G) : t;
    const Source<kBits> s1 = source<kBits, kSwiglu>(a, tn, wave, lane);
#pragma clang loop unroll(disable)
    for (int p = 1; p < pairs; ++p) {
      step<0, true>(f, g, s0, 2 * p, a.K, a_chunk, b_chunk, b_step, buf, buf ^ 1, wave, lane);
      step<1, false>(f, g, s0, 2 * p + 1, a.K, a_chunk, b_chunk, b_step, buf ^ 1, 0, wave, lane);
      buf ^= 1;
    }
    step<0, true>(f, g, s1, 0, a.K, a_chunk, b_chunk, b_step, buf, buf ^ 1, wave, lane);
    step<1, false>(f, g, s1, 1, a.K, a_chunk, b_chunk, b_step, buf ^ 1, 0, wave, lane);
    buf ^= 1;

    // the accumulators stay where they are up to their block's turn
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) asm volatile("" : "+a"(f.acc[i][j]));
    // acc[i][j][4 q + c]: row lane & 31 of row block i, column 8 q + 4 h + c of block j
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int lr = g.a_row + i * 32 + (lane & 31);
      const int64_t row = t.row0 + lr;
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
          if (lr < t.valid && col < No) {
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
          if (lr < t.valid) {
            uint16_t* out = static_cast<uint16_t*>(a.y) + row * No;
#pragma unroll
            for (int q = 0; q < 4; q += 2) {
              // lanes below 32: columns 8 q + [0, 8), the others 8 (q + 1) + [0, 8)
              const auto p0 = __builtin_amdgcn_permlane32_swap(d[q][0], d[q + 1][0], false, false);
              const auto p1 = __builtin_amdgcn_permlane32_swap(d[q][1], d[q + 1][1], false, false);
              store_bf16(out, col + 8 * (q + h), No, u32x4{p0[0], p1[0], p0[1], p1[1]});
            }
          }
        }
        __builtin_amdgcn_sched_barrier(0);   // one block at a time
      }
    }
    t = tn;
    s0 = s1;
  }
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(0, true));   // loads past the last tile
#endif  // __HIP_DEVICE_COMPILE__
}

template <int kBits>
void launch(const tr_expert_desc& d, const MxArgs& a, hipStream_t st) {
  const uint32_t blocks = static_cast<uint32_t>(device_cu_count());
  if (d.swiglu && d.out) mx_tiles<kBits, true, true><<<blocks, kThreads, 0, st>>>(a);
  else if (d.swiglu) mx_tiles<kBits, true, false><<<blocks, kThreads, 0, st>>>(a);
  else if (d.out) mx_tiles<kBits, false, true><<<blocks, kThreads, 0, st>>>(a);
  else mx_tiles<kBits, false, false><<<blocks, kThreads, 0, st>>>(a);
}

}  // namespace

// Whether the tiles take experts of this call: gathered rows are addressed with 31 bits,
// tiles are numbered with 31.
bool expert_can_tile(const tr_expert_desc& d, bool gather) {
  const int64_t tiles = (cdiv(d.R, BM) + d.E) * cdiv(d.swiglu ? d.N / 2 : d.N, d.swiglu ? BN / 2 : BN);
  return (!gather || d.T * d.K < (int64_t{1} << 31)) && tiles < (int64_t{1} << 30);
}

hipError_t expert_tiles(const tr_expert_desc& d, const void* x, const void* xs, const void* w, const void* ws,
                        const int* offsets, const int* rows, void* y, void* ys, int least, hipStream_t st) {
  const MxArgs a{static_cast<const uint8_t*>(x), static_cast<const uint8_t*>(xs),
                 static_cast<const uint8_t*>(w), static_cast<const uint8_t*>(ws), offsets, rows, y,
                 static_cast<uint8_t*>(ys), d.T, static_cast<int>(d.R), static_cast<int>(d.K),
                 static_cast<int>(d.N), d.E, least};
  if (d.bits == 4) launch<4>(d, a, st);
  else launch<8>(d, a, st);
  return hipGetLastError();
}

}  // namespace tr
