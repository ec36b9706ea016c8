// Root-mean-square norm with the residual's addition, and rows in blocks of 32 with
// scales (tr_mx.h).
//
//   z = x + residual,  y = z / sqrt(mean(z^2) + eps) * weight
//
// z, the sum of its squares and y are fp32. y is rounded once, to the rows' type and
// from the same fp32 value to 8 bits; z is rounded once for the next residual and
// normalized as it was before that rounding.
//
// Bound by memory: every number is read once and written once. A row belongs to one wave
// or one block and stays in registers between the sum and the outputs; only rows past
// 32768 are read twice. A block of 32 is four neighbouring lanes, eight numbers each.
//
// Outputs that the L2s cannot hold (8 of 4 MiB) are written past them, and inputs that the
// 256 MiB behind those cannot hold are read past them. 16384 x 7168 bf16 with residual, y
// and 8 bits (1.06 GB): 226 us as usual, 202 with such stores, 193 (5.5 TB/s) with such
// loads, too; 4096 x 4096: 32, 26, 33.
#include "tr_internal.h"
#include "tr_mx.h"

namespace tr {
namespace {

struct NormArgs {
  const void* x;
  const void* residual;   // or NULL
  const void* weight;
  void* y;                // or NULL
  void* residual_out;     // or NULL
  uint8_t* q;             // or NULL
  uint8_t* s;
  int64_t T;
  int64_t H;
  float eps;
};

// 16 bytes, past the caches or not.
template <bool kPast, typename V>
__device__ __forceinline__ V load_v(const V* p) {
  if constexpr (kPast) return __builtin_nontemporal_load(p);
  else return *p;
}
template <bool kPast, typename V>
__device__ __forceinline__ void store_v(V* p, const V& v) {
  if constexpr (kPast) __builtin_nontemporal_store(v, p);
  else *p = v;
}

// Eight neighbouring numbers of a row.
template <bool kF32, bool kPast = false>
__device__ __forceinline__ void load8(const void* p, int64_t at, float* v) {
  if constexpr (kF32) {
    const floatx4* f = reinterpret_cast<const floatx4*>(static_cast<const float*>(p) + at);
    const floatx4 a = load_v<kPast>(f), b = load_v<kPast>(f + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  } else {
    const u32x4 a = load_v<kPast>(reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + at));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
  }
}

template <bool kF32, bool kPast>
__device__ __forceinline__ void store8(void* p, int64_t at, const float* v) {
  if constexpr (kF32) {
    floatx4* f = reinterpret_cast<floatx4*>(static_cast<float*>(p) + at);
    store_v<kPast>(f, floatx4{v[0], v[1], v[2], v[3]});
    store_v<kPast>(f + 1, floatx4{v[4], v[5], v[6], v[7]});
  } else {
    store_v<kPast>(reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + at),
                   u32x4{cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]), cvt_bf16x2(v[4], v[5]), cvt_bf16x2(v[6], v[7])});
  }
}

// Eight numbers, from number `at` of all the rows in order, as 8 or 4 bits (four lanes
// are a block; every one of the four calls it).
template <int kBits>
__device__ __forceinline__ void quantize(uint8_t* q, uint8_t* s, int64_t at, const float* v) {
  float top = 0.0f;
  bool fine = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    top = fmaxf(top, mx_magnitude(v[i]));
    if constexpr (kBits == 4) fine &= fabsf(v[i]) <= kMaxFloat;
  }
  if constexpr (kBits == 4) top = fine ? top : __uint_as_float(0x7f800000u);
  top = fmaxf(top, __shfl_xor(top, 1, 4));
  top = fmaxf(top, __shfl_xor(top, 2, 4));
  if constexpr (kBits == 8) {
    const int b = mx_scale_byte<8>(top);
    const float inv = mx_inverse(b);
    *reinterpret_cast<uint2*>(q + at) = uint2{mx_pack8(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                                              mx_pack8(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv)};
    if ((at & 31) == 0) s[at / kMxBlock] = static_cast<uint8_t>(b);
  } else {
    fine = top <= kMaxFloat;   // of all four lanes
    const int b = fine ? mx_scale_byte<4>(top) : 255;
    const float inv = fine ? mx_inverse(b) : 0.0f;
    uint32_t d = 0;
    d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[0] * inv, v[1] * inv, 1.0f, 0);
    d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[2] * inv, v[3] * inv, 1.0f, 1);
    d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[4] * inv, v[5] * inv, 1.0f, 2);
    d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[6] * inv, v[7] * inv, 1.0f, 3);
    *reinterpret_cast<uint32_t*>(q + at / 2) = fine ? d : 0;
    if ((at & 31) == 0) s[at / kMxBlock] = static_cast<uint8_t>(b);
  }
}

// The sum of v over the kPer threads of a row. tmp: kPer / 64 floats in LDS (kPer > 64).
template <int kPer>
__device__ __forceinline__ float row_sum(float v, float* tmp) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, kWave);
  if constexpr (kPer > kWave) {
    if (lane_id() == 0) tmp[threadIdx.x / kWave] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < kPer / kWave; ++w) v += tmp[w];
  }
  return v;
}

// Rows of at most 8 kPer kChunks numbers, kPer threads each.
template <bool kF32, int kPer, int kChunks, bool kLoadPast, bool kStorePast>
__global__ __launch_bounds__(kPer < 256 ? 256 : kPer) void norm_rows(NormArgs a) {
  constexpr int kThreads = kPer < 256 ? 256 : kPer;
  __shared__ float tmp[kPer / kWave];
  const int me = threadIdx.x % kPer;
  const int H = static_cast<int>(a.H);
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / kPer);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / kPer) + threadIdx.x / kPer; t < a.T; t += step) {
    const int64_t row = t * a.H;
    float z[kChunks][8], w[kChunks][8];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int at = (c * kPer + me) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) z[c][i] = 0.0f;
      if (at < H) load8<kF32, kLoadPast>(a.x, row + at, z[c]);
    }
    if (a.residual) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int at = (c * kPer + me) * 8;
        if (at < H) {
          float r[8];
          load8<kF32, kLoadPast>(a.residual, row + at, r);
#pragma unroll
          for (int i = 0; i < 8; ++i) z[c][i] += r[i];
        }
      }
    }
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int at = (c * kPer + me) * 8;
      if (at < H) load8<kF32>(a.weight, at, w[c]);
    }
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(z[c][i], z[c][i], sum);
    sum = row_sum<kPer>(sum, tmp);
    const float inv = 1.0f / sqrtf(sum / static_cast<float>(H) + a.eps);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int at = (c * kPer + me) * 8;
      if (at >= H) continue;
      if (a.residual_out) store8<kF32, kStorePast>(a.residual_out, row + at, z[c]);
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = z[c][i] * inv * w[c][i];
      if (a.y) store8<kF32, kStorePast>(a.y, row + at, y);
      if (a.q) quantize<8>(a.q, a.s, row + at, y);
    }
    if constexpr (kPer > kWave) __syncthreads();   // tmp, before the next row's sum
  }
}

// Longer rows, a block each, read twice (64 / 2048 rows of 65536, bf16 with residual, y and 8 bits:
// 20 / 303 us, where one reading takes 6 / 192). An element is read and written by one thread, so
// outputs may lie over the inputs.
template <bool kF32>
__global__ __launch_bounds__(1024) void norm_long(NormArgs a) {
  __shared__ float tmp[16];
  const int H = static_cast<int>(a.H);
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t row = t * a.H;
    float sum = 0.0f;
    for (int at = threadIdx.x * 8; at < H; at += 8192) {
      float z[8];
      load8<kF32>(a.x, row + at, z);
      if (a.residual) {
        float r[8];
        load8<kF32>(a.residual, row + at, r);
  #pragma unroll
        for (int i = 0; i < 8; ++i) z[i] += r[i];
      }
  #pragma unroll
      for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(z[i], z[i], sum);
    }
    sum = row_sum<1024>(sum, tmp);
    const float inv = 1.0f / sqrtf(sum / static_cast<float>(H) + a.eps);
    for (int at = threadIdx.x * 8; at < H; at += 8192) {
      float z[8], w[8], y[8];
      load8<kF32>(a.x, row + at, z);
      load8<kF32>(a.weight, at, w);
      if (a.residual) {
        float r[8];
        load8<kF32>(a.residual, row + at, r);
  #pragma unroll
        for (int i = 0; i < 8; ++i) z[i] += r[i];
      }
      if (a.residual_out) store8<kF32, false>(a.residual_out, row + at, z);
  #pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = z[i] * inv * w[i];
      if (a.y) store8<kF32, false>(a.y, row + at, y);
      if (a.q) quantize<8>(a.q, a.s, row + at, y);
    }
    __syncthreads();   // tmp, before the next row's sum
  }
}

// `chunks` times eight numbers, a multiple of 4, as blocks with scales. Bound by memory: bf16, 16384
// x 7168 in 8 / 4 bits 65 / 52 us (5.5 TB/s), 4096 rows 15 / 12.
template <bool kF32, int kBits>
__global__ __launch_bounds__(256) void quantize_rows(const void* x, int64_t chunks, uint8_t* q, uint8_t* s) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  // (the four lanes of a block leave the loop together)
  for (int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; c < chunks; c += step) {
    float v[8];
    load8<kF32>(x, c * 8, v);
    quantize<kBits>(q, s, c * 8, v);
  }
}

// (a launch has fewer than 2^32 threads; more rows are other turns of the blocks)
constexpr int64_t kMostBlocks = 1 << 20;

template <bool kF32, int kPer, int kChunks>
void launch_rows(const NormArgs& a, hipStream_t st) {
  constexpr int kThreads = kPer < 256 ? 256 : kPer;
  const int64_t need = cdiv(a.T, kThreads / kPer), blocks = need < kMostBlocks ? need : kMostBlocks;
  const int64_t bytes = a.T * a.H * (kF32 ? 4 : 2);
  const int64_t in = bytes * (a.residual ? 2 : 1);
  const int64_t out = bytes * ((a.y ? 1 : 0) + (a.residual_out ? 1 : 0)) + (a.q ? a.T * a.H : 0);
  if (in > (int64_t{256} << 20)) norm_rows<kF32, kPer, kChunks, true, true><<<static_cast<uint32_t>(blocks), kThreads, 0, st>>>(a);
  else if (out > (int64_t{32} << 20)) norm_rows<kF32, kPer, kChunks, false, true><<<static_cast<uint32_t>(blocks), kThreads, 0, st>>>(a);
  else norm_rows<kF32, kPer, kChunks, false, false><<<static_cast<uint32_t>(blocks), kThreads, 0, st>>>(a);
}

template <bool kF32>
void launch_norm(const NormArgs& a, hipStream_t st) {
  if (a.H <= 512) launch_rows<kF32, 64, 1>(a, st);
  else if (a.H <= 2048) launch_rows<kF32, 64, 4>(a, st);
  else if (a.H <= 8192) launch_rows<kF32, 256, 4>(a, st);
  else if (a.H <= 32768) launch_rows<kF32, 1024, 4>(a, st);
  else norm_long<kF32><<<static_cast<uint32_t>(a.T < kMostBlocks ? a.T : kMostBlocks), 1024, 0, st>>>(a);
}

}  // namespace

hipError_t rms_norm(const tr_norm_desc& d, const void* x, const void* residual, const void* weight, void* y,
                    void* residual_out, void* q, void* s, hipStream_t st) {
  const NormArgs a{x, residual, weight, y, residual_out, static_cast<uint8_t*>(q), static_cast<uint8_t*>(s),
                   d.T, d.H, d.eps};
  if (d.dtype == TR_F32) launch_norm<true>(a, st);
  else launch_norm<false>(a, st);
  return hipGetLastError();
}

hipError_t quantize_mx(int64_t rows, int64_t K, bool f32, int bits, const void* x, void* q, void* s,
                       hipStream_t st) {
  const int64_t chunks = rows * (K / 8);
  const int64_t most = static_cast<int64_t>(device_cu_count()) * 32;   // blocks
  const uint32_t blocks = static_cast<uint32_t>(cdiv(chunks, 256) < most ? cdiv(chunks, 256) : most);
  uint8_t* qb = static_cast<uint8_t*>(q);
  uint8_t* sb = static_cast<uint8_t*>(s);
  if (f32 && bits == 8) quantize_rows<true, 8><<<blocks, 256, 0, st>>>(x, chunks, qb, sb);
  else if (f32) quantize_rows<true, 4><<<blocks, 256, 0, st>>>(x, chunks, qb, sb);
  else if (bits == 8) quantize_rows<false, 8><<<blocks, 256, 0, st>>>(x, chunks, qb, sb);
  else quantize_rows<false, 4><<<blocks, 256, 0, st>>>(x, chunks, qb, sb);
  return hipGetLastError();
}

}  // namespace tr
