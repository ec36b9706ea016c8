// x w^T for few rows of x in bf16 and weights w in 4 bits, in blocks of 32 with
// scales (tr_mx.h).
//
// Elements times scales are bf16 numbers (exact): they are widened in registers, two by
// one conversion, and multiplied by bf16 matrix instructions, fp32 sums.
//
// kBM x 128 tiles, k-tiles of 256 numbers (128 bytes of a row of w, 512 of x) in three
// stages of LDS, filled without registers by whole lines, two in flight while one is
// multiplied. A wave has 32 rows of w, which it widens, and 32 rows of x. Where the
// tiles are fewer than the CUs, K is shared among `parts` blocks, whose fp32 sums a second
// launch adds in order.
//
// Bound by what a CU loads: a line of 128 bytes takes it about four cycles, of a k-tile 128
// of w and 4 kBM of x. So a tile is as wide as LDS allows, and K is shared rather than the
// rows of w. 64 rows, 7168 x 7168: 14.6 us, of which the sums' launch 2.4 to 4.8; 1 / 64 rows,
// 7168 x 131072: 100 / 158 (5.0 / 3.2 TB/s).
#include "tr_internal.h"
#include "tr_mx.h"

namespace tr {
namespace {

constexpr int kBN = 128, kBK = 256;

struct LinearArgs {
  const uint16_t* x;     // [T, K]
  const uint8_t* w;      // [N, K / 2]
  const uint8_t* ws;     // [N, K / 32]
  uint16_t* y;           // [T, N]
  float* part;           // [parts, T, N], with more than one
  int64_t T;
  int K, N;
};

// Four waves for 32 rows of x.
template <int kBM>
__global__ __launch_bounds__(8 * kBM) void linear_tiles(LinearArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int kWaves = kBM / 8;
  constexpr int kXLoads = kBM / 2 / kWaves, kWLoads = 16 / kWaves, kLoads = kXLoads + kWLoads;  // of a wave, 1 KiB each
  constexpr int kA = kBM * 32, kB = kBN * 8;                                    // chunks of 16 bytes
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
      const_cast<uint16_t*>(a.x + t0 * a.K), 0, static_cast<int>(static_cast<int64_t>(valid) * a.K * 2), kRawBuffer);
  const int rows = min(a.N - n0, kBN);
  const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(a.w + static_cast<int64_t>(n0) * (a.K / 2)), 0,
      static_cast<int>(static_cast<int64_t>(rows) * (a.K / 2)), kRawBuffer);
  // x: a load is two rows of 32 chunks; chunk c of row r lies at c ^ (r & 15). w: eight rows
  // of eight, at c ^ (r & 7) ^ (r >> 3 & 1).
  uint32_t x_off[kXLoads], w_off[kWLoads];
#pragma unroll
  for (int j = 0; j < kXLoads; ++j) {
    const int r = (wave * kXLoads + j) * 2 + h;
    x_off[j] = r < valid ? static_cast<uint32_t>(r) * static_cast<uint32_t>(a.K) * 2 + (l31 ^ (r & 15)) * 16 : kPast;
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
      const int r = (wave * kXLoads + j) * 2 + h;
      const uint32_t past = mine && at * 32 + (l31 ^ (r & 15)) < a.K / 8 ? 0 : kPast;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_void*)(sx + (wave * kXLoads + j) * 64), 16,
                                               x_off[j] | past, at * 512, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < kWLoads; ++j) {
      const uint32_t past = mine && at * 8 + (wc ^ ((wave * kWLoads + j) & 1)) < blocks ? 0 : kPast;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_void*)(sw + (wave * kWLoads + j) * 64), 16, w_off[j] | past,
                                               at * 128, 0, 0);
    }
  };
  floatx16 acc;
#pragma unroll
  for (int c = 0; c < 16; ++c) acc[c] = 0.0f;
  const int wr = (wave & 3) * 32 + l31, xr = (wave >> 2) * 32 + l31;     // this lane's rows
  auto multiply = [&](const u32x4* sx, const u32x4* sw, const uint2* s) {
    const int swz = (l31 & 7) ^ ((l31 >> 3) & 1);
    const uint32_t s0 = s[wr].x, s1 = s[wr].y;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      // this lane's chunk of w: block 2 q + h
      const u32x4 w = sw[wr * 8 + ((2 * q + h) ^ swz)];
      const float f = mx_scale(((q < 2 ? s0 : s1) >> (16 * (q & 1) + 8 * h)) & 255);
#pragma unroll
      for (int o = 0; o < 4; ++o) {
        const u32x4 v = {mx_pair_bf16<4, 0>(w[o], f), mx_pair_bf16<4, 1>(w[o], f), mx_pair_bf16<4, 2>(w[o], f),
                         mx_pair_bf16<4, 3>(w[o], f)};
        const u32x4 x = sx[xr * 32 + ((4 * (2 * q + h) + o) ^ (l31 & 15))];
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, v), __builtin_bit_cast(bf16x8, x),
                                                      acc, 0, 0, 0);
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
  settle(acc);

  // acc[4 q + c]: row xr of x, output 8 q + 4 h + c of this wave's 32
  if (xr >= valid) return;
  const int col0 = n0 + (wave & 3) * 32;
  float* sums = a.part + (static_cast<int64_t>(blockIdx.z) * a.T + t0 + xr) * a.N;
  uint16_t* out = a.y + (t0 + xr) * a.N;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const floatx4 v = {acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
    if (parts > 1) store4<true>(sums, col0 + 8 * q + 4 * h, a.N, a.N % 4 == 0, v);
    else store4<false>(out, col0 + 8 * q + 4 * h, a.N, a.N % 4 == 0, v);
  }
#endif  // __HIP_DEVICE_COMPILE__
}

// y = the parts' sum, four numbers a thread (kVec), or one.
template <bool kVec>
__global__ __launch_bounds__(256) void linear_join(const float* part, uint16_t* y, int64_t n, int parts) {
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * (kVec ? 4 : 1);
  if (at >= n) return;
  if constexpr (kVec) {
    floatx4 s = *reinterpret_cast<const floatx4*>(part + at);
    for (int p = 1; p < parts; ++p) s += *reinterpret_cast<const floatx4*>(part + p * n + at);
    *reinterpret_cast<uint2*>(y + at) = uint2{cvt_bf16x2(s[0], s[1]), cvt_bf16x2(s[2], s[3])};
  } else {
    float s = part[at];
    for (int p = 1; p < parts; ++p) s += part[p * n + at];
    y[at] = static_cast<uint16_t>(f32_to_bf16_bits(s));
  }
}

// Few rows, or none of the sizes above.
// Whether rows of w go over the blocks 32 at a time: always with x in fp32, else up to 16
// rows of x while the tiles are for less than half the CUs. 7168 x 7168, 1 / 16 rows: 8.9 / 11.8
// us against 11.9 / 13.1 in tiles; x 16384: 17.1 / 23.1 against 17.2 / 18.4; x 131072: 125 / 188
// against 100 / 121.
bool by_rows(const tr_linear4_desc& d) {
  return d.dtype == TR_F32 || d.K < kBK || (d.T <= 16 && cdiv(d.N, kBN) * 2 < kPlanCus);
}

int tile_rows(const tr_linear4_desc& d) { return d.T <= 32 ? 32 : 64; }

// Blocks that share K: as many as keep the blocks within the CUs, with four k-tiles each at
// least (a k-tile is 0.7 us or so, and a second launch some 4 of the host's and the GPU's:
// fewer than twelve are not shared).
int parts_of(const tr_linear4_desc& d) {
  const int64_t tiles = cdiv(d.N, kBN) * cdiv(d.T, tile_rows(d)), all = cdiv(d.K, kBK), most = all / 4;
  const int64_t p = kPlanCus / tiles;
  return static_cast<int>(p < 1 || all < 12 ? 1 : p < most ? p : most);
}

}  // namespace

size_t linear4_workspace(const tr_linear4_desc& d) {
  if (by_rows(d)) return 0;
  const int parts = parts_of(d);
  return parts > 1 ? static_cast<size_t>(parts) * d.T * d.N * 4 : 0;
}

hipError_t linear_mx4(const tr_linear4_desc& d, const void* x, const void* w, const void* ws, void* y, void* scratch,
                      hipStream_t st) {
  if (by_rows(d)) return linear4_few(d, x, w, ws, y, st);
  const int parts = parts_of(d), rows = tile_rows(d);
  const int64_t n_tiles = cdiv(d.N, kBN);
  // (a launch has fewer than 2^16 blocks in y; more rows are further launches)
  for (int64_t t = 0; t < d.T; t += int64_t{65535} * rows) {
    const int64_t here = d.T - t < int64_t{65535} * rows ? d.T - t : int64_t{65535} * rows;
    const LinearArgs a{static_cast<const uint16_t*>(x) + t * d.K, static_cast<const uint8_t*>(w),
                       static_cast<const uint8_t*>(ws), static_cast<uint16_t*>(y) + t * d.N,
                       static_cast<float*>(scratch), here, static_cast<int>(d.K), static_cast<int>(d.N)};
    const dim3 grid(static_cast<uint32_t>(n_tiles), static_cast<uint32_t>(cdiv(here, rows)),
                    static_cast<uint32_t>(parts));
    if (rows == 32) linear_tiles<32><<<grid, 256, 0, st>>>(a);
    else linear_tiles<64><<<grid, 512, 0, st>>>(a);
  }
  if (parts > 1) {
    const int64_t n = d.T * d.N;
    const float* part = static_cast<const float*>(scratch);
    uint16_t* out = static_cast<uint16_t*>(y);
    if (n % 4 == 0) linear_join<true><<<static_cast<uint32_t>(cdiv(n, 1024)), 256, 0, st>>>(part, out, n, parts);
    else linear_join<false><<<static_cast<uint32_t>(cdiv(n, 256)), 256, 0, st>>>(part, out, n, parts);
  }
  return hipGetLastError();
}

}  // namespace tr
