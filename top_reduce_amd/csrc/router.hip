// The router: logits (linear.hip), then every token's choice (tr_select.h), one
// wave a token; small routers do both in one launch (route_direct). Bound: latency
// for a few tokens, the logits' bytes and the selection's instructions for many.
#include "tr_chunk.h"
#include "tr_internal.h"
#include "tr_select.h"

namespace tr {
namespace {

constexpr int kThreads = 256;

// masks (NULL: none): the tokens that chose each of the local experts [begin,
// begin + E), zeroed before; slots: see FewRoutes.
template <int NR>
__global__ __launch_bounds__(kThreads) void route_select(SelectArgs a, FewRoutes f) {
  __shared__ SelectScratch scratch[kThreads / kWave];
  const int wave = threadIdx.x >> 6;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 6) + wave;
  if (t >= a.T) return;
  const Chosen c = choose<NR>(a, t, scratch[wave]);
  store_chosen(a, t, c);
  if (f.masks && c.rank >= 0) {
    const int64_t e = c.e - f.begin;
    if (e >= 0 && e < f.E) {
      atomicOr(f.masks + e, 1ull << t);
      f.slots[e * 64 + t] = static_cast<uint8_t>(c.rank);
    }
  }
}

template <int NR>
hipError_t launch_select(const SelectArgs& a, const FewRoutes& f, hipStream_t st) {
  // a few tokens: one wave a block, on a CU each
  const int threads = a.T <= 256 ? kWave : kThreads;
  const int64_t blocks = cdiv(a.T, threads / kWave);
  hipLaunchKernelGGL(route_select<NR>, dim3(static_cast<unsigned>(blocks)), dim3(threads), 0, st, a, f);
  return hipGetLastError();
}

// Logits and choice of 16 tokens by one block of 16 waves: every wave a share of
// the reduction against all experts (NT tiles of 16), the shares added in LDS, a
// token a wave. masks: with at most 16 tokens only. Bound by what a CU reads of
// rows (a batch of four 64-byte blocks a wave, mostly past its share, took 9 us
// where two take 6.6).
constexpr int kDirectWaves = 16;
template <bool kF32, int NT>
__global__ __launch_bounds__(kDirectWaves * kWave) void route_direct(SelectArgs a, FewRoutes f, const char* x,
                                                                     const char* w, int64_t row_bytes) {
  constexpr int kU = 2, kPitch = 68;
  __shared__ floatx4 red[kDirectWaves][NT][kWave];
  __shared__ float logit[16][kPitch];
  __shared__ uint32_t mask[kWave];
  __shared__ SelectScratch scratch;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * 16;
  if (tid < kWave) mask[tid] = 0;
  // (rows past the last token or expert: the last one's, never stored)
  const char* xp = x + min(t0 + r, a.T - 1) * row_bytes;
  const char* wp[NT];
  floatx4 acc[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    wp[i] = w + min(i * 16 + r, a.G - 1) * row_bytes;
    acc[i] = floatx4{0, 0, 0, 0};
  }
  const int nkb = static_cast<int>((row_bytes + 63) >> 6), last = static_cast<int>(row_bytes) - 16;
  const int kb0 = wave * nkb / kDirectWaves, kb1 = (wave + 1) * nkb / kDirectWaves;
  for (int kb = kb0; kb < kb1; kb += kU) {
    u32x4 xv[kU], wv[kU][NT];
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      const int at = min((kb + j) * 64 + g * 16, last);
      xv[j] = load16(xp + at);
#pragma unroll
      for (int i = 0; i < NT; ++i) wv[j][i] = load16(wp[i] + at);
    }
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      // past the share or the row: both operands zero (the row's end may hold
      // what is not a number)
      const bool in = kb + j < kb1 && (kb + j) * 64 + g * 16 <= last;
      if (!in) xv[j] = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        if (!in) wv[j][i] = u32x4{0, 0, 0, 0};
        acc[i] = mma16<kF32>(wv[j][i], xv[j], acc[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) red[wave][i][lane] = acc[i];
  __syncthreads();
  if (wave < NT) {
    floatx4 v = red[0][wave][lane];
#pragma unroll
    for (int q = 1; q < kDirectWaves; ++q) v += red[q][wave][lane];
    *reinterpret_cast<floatx4*>(&logit[r][wave * 16 + 4 * g]) = v;
  }
  __syncthreads();
  const int64_t t = t0 + wave;
  if (t < a.T) {
    SelectArgs own = a;   // this block's logits
    own.part = &logit[0][0];
    own.T = 16;
    own.S = 1;
    own.pitch = kPitch;
    const Chosen c = choose<1>(own, wave, scratch);
    store_chosen(a, t, c);
    const int64_t e = c.e - f.begin;
    if (f.masks && c.rank >= 0 && e >= 0 && e < f.E) {
      atomicOr(&mask[e], 1u << t);
      f.slots[e * 64 + t] = static_cast<uint8_t>(c.rank);
    }
  }
  if (f.masks) {   // (the same for the block)
    __syncthreads();
    if (tid < f.E) f.masks[tid] = mask[tid];
  }
}

template <bool kF32, int NT>
hipError_t launch_direct(const SelectArgs& a, const FewRoutes& f, const void* x, const void* w,
                         int64_t row_bytes, hipStream_t st) {
  hipLaunchKernelGGL((route_direct<kF32, NT>), dim3(static_cast<unsigned>(cdiv(a.T, 16))),
                     dim3(kDirectWaves * kWave), 0, st, a, f, static_cast<const char*>(x),
                     static_cast<const char*>(w), row_bytes);
  return hipGetLastError();
}
// Whether one launch takes the router: up to 32 experts, 64 KiB of weights in
// whole tiles and a block a CU. bf16, in a graph and with the host's part: 16
// tokens, 16 x 512 5.0 and 9.6 us (two launches 6.6 and 12.4), 32 x 1024 6.6 and
// 9.6 (7.0 and 12.5), but 32 x 2048 9.1 and 9.6 (7.0 and 12.5), 64 x 512 9.5 and
// 9.7 (7.5 and 12.5); 4096 tokens, 16 x 512 5.6 and 9.8 (7.4 and 12.6).
bool direct(const tr_route_desc& d, int64_t row_bytes) {
  return d.G <= 32 && d.T <= 16 * kPlanCus && cdiv(d.G, 16) * 16 * row_bytes <= 1 << 16;
}

}  // namespace

size_t route_workspace(const tr_route_desc& d) {
  return logits_layout(d.T, d.H, d.G, d.dtype == TR_F32).bytes;
}

SelectArgs select_args(const tr_route_desc& d, const float* bias, void* idx, float* w, const void* ws) {
  const LogitsLayout L = logits_layout(d.T, d.H, d.G, d.dtype == TR_F32);
  SelectArgs a{};
  a.part = static_cast<const float*>(ws);
  a.bias = bias;
  a.idx = idx;
  a.w = w;
  a.T = d.T;
  a.S = L.parts;
  a.pitch = L.pitch;
  a.G = d.G;
  a.K = d.K;
  a.idx64 = d.idx_dtype == TR_IDX_I64;
  a.sigmoid = d.score == TR_SCORE_SIGMOID;
  a.renorm = d.renorm;
  a.scale = d.scale;
  return a;
}

hipError_t route_topk(const tr_route_desc& d, const void* x, const void* w_gate, const float* bias,
                      void* idx, float* w, void* ws, hipStream_t st, const FewRoutes* few) {
  const bool f32 = d.dtype == TR_F32;
  const int64_t row_bytes = d.H * (f32 ? 4 : 2);
  const SelectArgs a = select_args(d, bias, idx, w, ws);
  const FewRoutes f = few ? *few : FewRoutes{};
  if (direct(d, row_bytes) && (!few || d.T <= 16)) {
    if (f32)
      return d.G <= 16 ? launch_direct<true, 1>(a, f, x, w_gate, row_bytes, st)
                       : launch_direct<true, 2>(a, f, x, w_gate, row_bytes, st);
    return d.G <= 16 ? launch_direct<false, 1>(a, f, x, w_gate, row_bytes, st)
                     : launch_direct<false, 2>(a, f, x, w_gate, row_bytes, st);
  }
  hipError_t e = logits(d.T, d.H, d.G, f32, x, w_gate, static_cast<float*>(ws),
                        few ? reinterpret_cast<uint32_t*>(few->masks) : nullptr,
                        few ? 2 * few->E : 0, st);
  if (e != hipSuccess) return e;
  // registers of logits for the experts there are (16384 tokens of 128 experts by 2
  // 10.7 us, by 4 12.7; 4096 of 512 by 8 10.4 us, by 16 14.2). Past 1024 experts 64 of
  // them leave one wave a SIMD: 4096 tokens, 8 of 1025 experts 63 us, 16 of 4096 55 us.
  if (d.G <= 64) return launch_select<1>(a, f, st);
  if (d.G <= 128) return launch_select<2>(a, f, st);
  if (d.G <= 256) return launch_select<4>(a, f, st);
  if (d.G <= 512) return launch_select<8>(a, f, st);
  if (d.G <= 1024) return launch_select<16>(a, f, st);
  return launch_select<64>(a, f, st);
}

}  // namespace tr
