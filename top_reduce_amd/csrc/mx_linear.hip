// x w^T for few rows of x in bf16 or fp32 and weights w in 4 bits, in blocks of 32 with
// scales (tr_mx.h).
//
// Elements times scales are bf16 numbers (exact): they are widened in registers, two by
// one conversion, and multiplied by bf16 matrix instructions, fp32 sums. A number of x in
// fp32 is three of bf16 (split_bf16), and so three instructions: every product still counts
// in full.
//
// kBM x 128 tiles, k-tiles of 256 numbers (128 bytes of a row of w, 512 of x) in three
// stages of LDS, filled without registers by whole lines, two in flight while one is
// multiplied. A wave has 32 rows of w, which it widens, and 32 rows of x; in fp32 all rows and
// a quarter of the k-tile, so that x is split once (by four waves: 31 us for 32 rows of 7168 x
// 7168, so 18.6; with the fp32 matrix instructions, by lanes, 107). Where the
// tiles are fewer than the CUs, K is shared among `parts` blocks, whose fp32 sums a second
// launch adds in order.
//
// Bound by what a CU loads: a line of 128 bytes takes it about four cycles, of a k-tile 128
// of w and 4 kBM of x. So a tile is as wide as LDS allows, and K is shared rather than the
// rows of w. 64 rows, 7168 x 7168: 14.6 us, of which the sums' launch 2.4, in
// fp32 28.7; 1 / 64 rows, 7168 x 131072: 100 / 158 (5.0 / 3.2 TB/s).
#include "tr_internal.h"
#include "tr_mx.h"

namespace tr {
namespace {

constexpr int kBN = 128, kBK = 256;

struct LinearArgs {
  const char* x;         // [T, K] bf16, or fp32
  const uint8_t* w;      // [N, K / 2]
  const uint8_t* ws;     // [N, K / 32]
  char* y;               // [T, N], as x
  float* part;           // [parts, T, N], with more than one
  int64_t T;
  int K, N;
};

#if defined(__HIP_DEVICE_COMPILE__)
__device__ __forceinline__ floatx16 mma32(const u32x4& w, const u32x4& x, const floatx16& acc) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), acc, 0, 0, 0);
}
#endif

// Four waves for 32 rows of x.
template <bool kF32, int kBM>
__global__ __launch_bounds__(8 * kBM) void linear_tiles(LinearArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int kWaves = kBM / 8;
  constexpr int kEs = kF32 ? 4 : 2, kChunks = kBK * kEs / 16, kPer = 64 / kChunks;   // chunks of 16 bytes of a row; rows of a load
  constexpr int kXLoads = kBM / kPer / kWaves, kWLoads = 16 / kWaves, kLoads = kXLoads + kWLoads;  // of a wave, 1 KiB each
  constexpr int kA = kBM * kChunks, kB = kBN * 8;
  // distinct objects: an access to one stage does not wait for loads into another
  __shared__ u32x4 a0[kA], a1[kA], a2[kA], b0[kB], b1[kB], b2[kB];
  __shared__ uint2 sc[3][kBN];      // scales of a row's eight blocks
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, l31 = lane & 31;
  const int n0 = blockIdx.x * kBN;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * kBM;
  const int valid = static_cast<int>(min(a.T - t0, static_cast<int64_t>(kBM)));
  const int blocks = a.K / kMxBlock, all = (a.K + kBK - 1) / kBK;
  const int parts = gridDim.z;
  const int k0 = static_cast<int>(static_cast<int64_t>(all) * blockIdx.z / parts);
  const int k1 = static_cast<int>(static_cast<int64_t>(all) * (blockIdx.z + 1) / parts);
  // this block's rows of x and of w only: offsets stay below 2^31
  const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<char*>(a.x + t0 * a.K * kEs), 0, static_cast<int>(static_cast<int64_t>(valid) * a.K * kEs), kRawBuffer);
  const int rows = min(a.N - n0, kBN);
  const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(a.w + static_cast<int64_t>(n0) * (a.K / 2)), 0,
      static_cast<int>(static_cast<int64_t>(rows) * (a.K / 2)), kRawBuffer);
  // x: a load is two rows of 32 chunks, or one of 64; chunk c of row r lies at c ^ (r & 15).
  // w: eight rows of eight, at c ^ (r & 7) ^ (r >> 3 & 1).
  uint32_t x_off[kXLoads], w_off[kWLoads];
#pragma unroll
  for (int j = 0; j < kXLoads; ++j) {
    const int r = (wave * kXLoads + j) * kPer + lane / kChunks;
    x_off[j] = r < valid ? static_cast<uint32_t>(r) * static_cast<uint32_t>(a.K) * kEs + ((lane % kChunks) ^ (r & 15)) * 16
                         : kPast;
  }
  const int wc = (lane & 7) ^ (lane >> 3);
#pragma unroll
  for (int j = 0; j < kWLoads; ++j) {
    const int r = (wave * kWLoads + j) * 8 + (lane >> 3);
    w_off[j] = r < rows ? static_cast<uint32_t>(r) * static_cast<uint32_t>(a.K / 2) + (wc ^ (r >> 3 & 1)) * 16 : kPast;
  }
  const uint8_t* sp = a.ws + (n0 + static_cast<int64_t>(min(tid, rows - 1))) * blocks;
  auto load = [&](u32x4* sx, u32x4* sw, int kt) {
    const int at = __builtin_amdgcn_readfirstlane(kt);
    const bool mine = at < k1;      // (past the part's last: nothing is read)
#pragma unroll
    for (int j = 0; j < kXLoads; ++j) {
      const int r = (wave * kXLoads + j) * kPer + lane / kChunks;
      const uint32_t past = mine && at * kChunks + ((lane % kChunks) ^ (r & 15)) < a.K * kEs / 16 ? 0 : kPast;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void*)(sx + (wave * kXLoads + j) * 64), 16,
                                               x_off[j] | past, at * (kBK * kEs), 0, 0);
    }
#pragma unroll
    for (int j = 0; j < kWLoads; ++j) {
      const uint32_t past = mine && at * 8 + (wc ^ ((wave * kWLoads + j) & 1)) < blocks ? 0 : kPast;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(sw + (wave * kWLoads + j) * 64), 16, w_off[j] | past,
                                               at * 128, 0, 0);
    }
  };
  // In bf16 a wave has 32 rows of w; in fp32 all 128, and block 2 wave + h of a k-tile, so
  // that every number of x is split once.
  constexpr int kJ = kF32 ? 4 : 1;
  floatx16 acc[kJ];
#pragma unroll
  for (int j = 0; j < kJ; ++j)
#pragma unroll
    for (int c = 0; c < 16; ++c) acc[j][c] = 0.0f;
  const int xr = (kF32 ? 0 : wave >> 2) * 32 + l31;     // this lane's row of x
  // (inlined by force: as a function of its own it has the accumulators in memory, 310 us for 18)
  auto multiply = [&](const u32x4* sx, const u32x4* sw, const uint2* s) __attribute__((always_inline)) {
    const int swz = (l31 & 7) ^ ((l31 >> 3) & 1);
    const u32x4* x = sx + xr * kChunks;
    uint32_t below = 0;
#pragma unroll
    for (int i = 0; i < (kF32 ? 1 : 4); ++i) {
      const int q = kF32 ? wave : i;
      // this lane's chunks of w: block 2 q + h
      u32x4 w[kJ];
      float f[kJ];
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        const int wr = (kF32 ? j : wave & 3) * 32 + l31;
        w[j] = sw[wr * 8 + ((2 * q + h) ^ swz)];
        f[j] = mx_scale(((q < 2 ? s[wr].x : s[wr].y) >> (16 * (q & 1) + 8 * h)) & 255);
      }
#pragma unroll
      for (int o = 0; o < 4; ++o) {
        const int c = 4 * (2 * q + h) + o;     // eight numbers
        Split p;
        if constexpr (kF32) p = split_bf16(x[(2 * c) ^ (l31 & 15)], x[(2 * c + 1) ^ (l31 & 15)]);
        else p.top = x[c ^ (l31 & 15)];
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          const u32x4 v = widen4(w[j][o], f[j]);
          if constexpr (kF32) {
            acc[j] = mma32(v, p.low, acc[j]);
            acc[j] = mma32(v, p.mid, acc[j]);
          }
          acc[j] = mma32(v, p.top, acc[j]);
        }
        if constexpr (kF32) below |= p.below;
      }
    }
    if constexpr (kF32) {
      if (any_below(below)) {
        // what the three parts could not hold (numbers below 2^-110)
        const int b = 2 * wave + h;     // this lane's block
#pragma clang loop unroll(disable)
        for (int o = 0; o < 4; ++o) {
          const int c = 4 * b + o;
          const Split r = split_rest(x[(2 * c) ^ (l31 & 15)], x[(2 * c + 1) ^ (l31 & 15)]);
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            const int wr = j * 32 + l31;
            const uint32_t d = reinterpret_cast<const uint32_t*>(sw + wr * 8 + (b ^ swz))[o];
            const u32x4 v = widen4(d, scale_down(mx_scale(reinterpret_cast<const uint8_t*>(s + wr)[b])));
            acc[j] = mma32(v, r.mid, acc[j]);
            acc[j] = mma32(v, r.top, acc[j]);
          }
        }
      }
    }
  };
  // Step kt: its scales (loaded three steps before) go to LDS, its operands have landed;
  // then the loads of the step after next, into the stage that the step before has read.
  uint2 v0 = load_scale8(sp, k0 * 8, blocks), v1 = load_scale8(sp, k0 * 8 + 8, blocks);
  load(a0, b0, k0);
  asm volatile("" ::: "memory");
  uint2 v2 = load_scale8(sp, k0 * 8 + 16, blocks);
  load(a1, b1, k0 + 1);
  auto step = [&](int kt, u32x4* sx, u32x4* sw, u32x4* nx, u32x4* nw, uint2* s, uint2& v) {
    if (tid < kBN) s[tid] = scale8(v, kt * 8, blocks);
    // sent since: the scales and operands of one step
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(kLoads + 1, true));
    lds_barrier();
    v = load_scale8(sp, (kt + 3) * 8, blocks);
    load(nx, nw, kt + 2);
    multiply(sx, sw, s);
  };
  int kt = k0;
#pragma clang loop unroll(disable)
  for (; kt + 3 <= k1; kt += 3) {
    step(kt, a0, b0, a2, b2, sc[0], v0);
    step(kt + 1, a1, b1, a0, b0, sc[1], v1);
    step(kt + 2, a2, b2, a1, b1, sc[2], v2);
  }
  // The last, at most two: all has been sent.
  if (tid < kBN) {
    sc[0][tid] = scale8(v0, kt * 8, blocks);
    sc[1][tid] = scale8(v1, kt * 8 + 8, blocks);
  }
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(0, true));
  lds_barrier();
  if (kt < k1) multiply(a0, b0, sc[0]);
  if (kt + 1 < k1) multiply(a1, b1, sc[1]);
  settle(acc[0]);
#pragma unroll
  for (int j = 1; j < kJ; ++j) settled(acc[j]);

  typedef typename Elem<kF32>::type Out;
  auto store = [&](int r, int col, const floatx4& v) {      // outputs col .. col + 3 of row r
    if (r >= valid) return;
    float* sums = a.part + (static_cast<int64_t>(blockIdx.z) * a.T + t0 + r) * a.N;
    if (parts > 1) store4<true>(sums, n0 + col, a.N, a.N % 4 == 0, v);
    else store4<kF32>(reinterpret_cast<Out*>(a.y) + (t0 + r) * a.N, n0 + col, a.N, a.N % 4 == 0, v);
  };
  // acc[j][4 q + c]: row xr of x, output 8 q + 4 h + c of 32
  if constexpr (kF32) {
    // the waves' sums, in order: outputs 4 n .. of row r lie at r 32 + (n ^ r)
    floatx4* mine = reinterpret_cast<floatx4*>(wave < 2 ? a0 : a1) + (wave & 1) * 1024;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kJ; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        mine[xr * 32 + ((8 * j + 2 * q + h) ^ xr)] =
            floatx4{acc[j][4 * q], acc[j][4 * q + 1], acc[j][4 * q + 2], acc[j][4 * q + 3]};
    __syncthreads();
    for (int i = tid; i < kBM * 32; i += 64 * kWaves) {
      const int r = i >> 5, n = i & 31, at = r * 32 + (n ^ r);
      const floatx4* p0 = reinterpret_cast<const floatx4*>(a0);
      const floatx4* p1 = reinterpret_cast<const floatx4*>(a1);
      store(r, 4 * n, p0[at] + p0[1024 + at] + p1[at] + p1[1024 + at]);
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      store(xr, (wave & 3) * 32 + 8 * q + 4 * h,
            floatx4{acc[0][4 * q], acc[0][4 * q + 1], acc[0][4 * q + 2], acc[0][4 * q + 3]});
  }
#endif  // __HIP_DEVICE_COMPILE__
}

// y = the parts' sum, four numbers a thread (kVec), or one.
template <bool kF32, bool kVec>
__global__ __launch_bounds__(256) void linear_join(const float* part, void* y, int64_t n, int parts) {
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * (kVec ? 4 : 1);
  if (at >= n) return;
  typedef typename Elem<kF32>::type Out;
  if constexpr (kVec) {
    floatx4 s = *reinterpret_cast<const floatx4*>(part + at);
    for (int p = 1; p < parts; ++p) s += *reinterpret_cast<const floatx4*>(part + p * n + at);
    if constexpr (kF32) *reinterpret_cast<floatx4*>(static_cast<Out*>(y) + at) = s;
    else *reinterpret_cast<uint2*>(static_cast<Out*>(y) + at) = uint2{cvt_bf16x2(s[0], s[1]), cvt_bf16x2(s[2], s[3])};
  } else {
    float s = part[at];
    for (int p = 1; p < parts; ++p) s += part[p * n + at];
    if constexpr (kF32) static_cast<Out*>(y)[at] = s;
    else static_cast<Out*>(y)[at] = static_cast<Out>(f32_to_bf16_bits(s));
  }
}

// k-tiles from which K is shared (one is 0.7 us or so, in fp32 1.9, and a second launch some 4
// of the host's and the GPU's).
constexpr int kSharedTiles = 12;

// Whether rows of w go over the blocks 32 at a time: up to 16 rows of x while the tiles are for
// less than half the CUs, in fp32 where they would not share K. bf16, 7168 x 7168, 1 / 16 rows:
// 8.9 / 11.8 us against 11.9 / 13.1 in tiles; x 16384: 17.1 / 23.1 against 17.2 / 18.4; x 131072:
// 125 / 188 against 100 / 121. fp32, 1440 x 1001, 1 / 5 / 16 rows: 7.3 / 7.6 / 8.4 against 12.9 /
// 13.0 / 13.4; 7168 x 7168: 18.0 / 28.7 / 33.1 against 17.2 / 17.7 / 18.7.
bool by_rows(const tr_linear4_desc& d) {
  return d.K < kBK || (d.T <= 16 && cdiv(d.N, kBN) * 2 < kPlanCus &&
                       (d.dtype == TR_BF16 || cdiv(d.K, kBK) < kSharedTiles));
}

int tile_rows(const tr_linear4_desc& d) { return d.T <= 32 || d.dtype == TR_F32 ? 32 : 64; }

// Blocks that share K: as many as keep the blocks within the CUs, with four k-tiles each at
// least.
int parts_of(const tr_linear4_desc& d) {
  const int64_t tiles = cdiv(d.N, kBN) * cdiv(d.T, tile_rows(d)), all = cdiv(d.K, kBK), most = all / 4;
  const int64_t p = kPlanCus / tiles;
  return static_cast<int>(p < 1 || all < kSharedTiles ? 1 : p < most ? p : most);
}

template <bool kF32>
void launch(const tr_linear4_desc& d, const void* x, const void* w, const void* ws, void* y, void* scratch,
            hipStream_t st) {
  constexpr int kEs = kF32 ? 4 : 2;
  const int parts = parts_of(d), rows = tile_rows(d);
  const int64_t n_tiles = cdiv(d.N, kBN);
  // (a launch has fewer than 2^16 blocks in y; more rows are further launches)
  for (int64_t t = 0; t < d.T; t += int64_t{65535} * rows) {
    const int64_t here = d.T - t < int64_t{65535} * rows ? d.T - t : int64_t{65535} * rows;
    const LinearArgs a{static_cast<const char*>(x) + t * d.K * kEs, static_cast<const uint8_t*>(w),
                       static_cast<const uint8_t*>(ws), static_cast<char*>(y) + t * d.N * kEs,
                       static_cast<float*>(scratch), here, static_cast<int>(d.K), static_cast<int>(d.N)};
    const dim3 grid(static_cast<uint32_t>(n_tiles), static_cast<uint32_t>(cdiv(here, rows)),
                    static_cast<uint32_t>(parts));
    if constexpr (kF32) linear_tiles<true, 32><<<grid, 256, 0, st>>>(a);
    else if (rows == 32) linear_tiles<false, 32><<<grid, 256, 0, st>>>(a);
    else linear_tiles<false, 64><<<grid, 512, 0, st>>>(a);
  }
  if (parts > 1) {
    const int64_t n = d.T * d.N;
    const float* part = static_cast<const float*>(scratch);
    if (n % 4 == 0) linear_join<kF32, true><<<static_cast<uint32_t>(cdiv(n, 1024)), 256, 0, st>>>(part, y, n, parts);
    else linear_join<kF32, false><<<static_cast<uint32_t>(cdiv(n, 256)), 256, 0, st>>>(part, y, n, parts);
  }
}

}  // namespace

size_t linear4_workspace(const tr_linear4_desc& d) {
  if (d.T == 0 || by_rows(d)) return 0;   // (no rows have no tiles to share K among)
  const int parts = parts_of(d);
  return parts > 1 ? static_cast<size_t>(parts) * d.T * d.N * 4 : 0;
}

hipError_t linear_mx4(const tr_linear4_desc& d, const void* x, const void* w, const void* ws, void* y, void* scratch,
                      hipStream_t st) {
  if (by_rows(d)) return linear4_few(d, x, w, ws, y, st);
  if (d.dtype == TR_F32) launch<true>(d, x, w, ws, y, scratch, st);
  else launch<false>(d, x, w, ws, y, scratch, st);
  return hipGetLastError();
}

}  // namespace tr
