// Router selection: scores of a token's logits, its K best experts and their
// gate weights.
//
//   p = softmax(logits) over all G experts, or sigmoid(logits)
//   key = logits (both scores keep their order), or p + bias with a balancing
//         bias, which decides the selection only
//   idx = the K largest keys, descending, ties to the lowest id
//   w   = scale * p[idx], divided by their sum with renorm
//
// One wave takes one token, its keys in registers (expert 64 i + lane in
// register i). Keys are compared as integers that order like the floats, NaN
// below everything, so that every row yields K different valid ids. Each of
// the K rounds reduces one integer over the lanes. Bound: latency of the
// rounds for one token, the logits' bytes for many.
#include "tr_chunk.h"
#include "tr_internal.h"

namespace tr {
namespace {

constexpr int kThreads = 256;

struct SelectArgs {
  const float* part;     // [S, T, pitch] parts of the logits
  const float* bias;     // [G] or NULL
  void* idx;             // [T, K] int32 or int64
  float* w;              // [T, K]
  int64_t T;
  int S, pitch, G, K;
  int idx64, sigmoid, renorm;
  float scale;
  // a few tokens' local routes (NULL: none), see layer_few.hip
  unsigned long long* masks;   // [E], zeroed before
  uint8_t* slots;              // [E, 64]
  int64_t begin;
  int E;
};

constexpr uint32_t kUsed = 0, kNan = 1;

// An integer that orders like v: kNan < -inf < ... < +inf; -0 and +0 alike.
__device__ __forceinline__ uint32_t order_key(float v) {
  v += 0.0f;
  const uint32_t u = __float_as_uint(v);
  if ((u & 0x7fffffffu) > 0x7f800000u) return kNan;
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v = max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), d, kWave)));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d, kWave);
  return v;
}

// NR registers of logits a lane: G <= 64 NR.
template <int NR>
__global__ __launch_bounds__(kThreads) void route_select(SelectArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 6) + (threadIdx.x >> 6);
  if (t >= a.T) return;
  float p[NR];
  uint32_t key[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) p[i] = 0.0f;
  for (int s = 0; s < a.S; ++s) {
    const float* row = a.part + (s * a.T + t) * a.pitch;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int e = i * kWave + lane;
      if (e < a.G) p[i] += row[e];
    }
  }
  // the logits' keys; the largest logit (of those that are numbers)
  uint32_t best = kUsed;
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    key[i] = i * kWave + lane < a.G ? order_key(p[i]) : kUsed;
    best = max(best, key[i]);
  }
  // scores
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < NR; ++i) p[i] = 1.0f / (1.0f + expf(-p[i]));
  } else {
    const uint32_t mk = wave_max(best);
    const float m = __uint_as_float((mk & 0x80000000u) ? mk & 0x7fffffffu : ~mk);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      p[i] = i * kWave + lane < a.G ? expf(p[i] - m) : 0.0f;
      sum += p[i];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < NR; ++i) p[i] /= sum;
  }
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int e = i * kWave + lane;
      if (e < a.G) key[i] = order_key(p[i] + a.bias[e]);
    }
  }

  // K rounds; lane k keeps the k-th expert and its score
  int my_e = 0;
  float my_p = 0.0f;
  for (int k = 0; k < a.K; ++k) {
    uint32_t lb = kUsed;
    int li = 0;
#pragma unroll
    for (int i = 0; i < NR; ++i)
      if (key[i] > lb) { lb = key[i]; li = i; }
    const uint32_t top = wave_max(lb);
    // the lowest id among the lanes that hold the largest key
    uint32_t cand = lb == top ? ~static_cast<uint32_t>(li * kWave + lane) : 0u;
    uint64_t hit = __ballot(lb == top);
    int e;
    if (__popcll(hit) == 1) {
      const int l = __ffsll(static_cast<unsigned long long>(hit)) - 1;
      e = __builtin_amdgcn_readlane(li, l) * kWave + l;
    } else {
      e = static_cast<int>(~wave_max(cand));
    }
    const int owner = e & 63, reg = e >> 6;
    float pe = 0.0f;
#pragma unroll
    for (int i = 0; i < NR; ++i)
      if (i == reg) {
        pe = p[i];
        if (lane == owner) key[i] = kUsed;
      }
    pe = __shfl(pe, owner, kWave);
    if (lane == k) {
      my_e = e;
      my_p = pe;
    }
  }
  float w = my_p;
  if (a.renorm) {
    const float sum = wave_sum(lane < a.K ? my_p : 0.0f);
    // a sum below the smallest normal float (all scores 0) divides by that
    // instead: weights 0, not NaN
    w = my_p / (sum < 1.17549435e-38f ? 1.17549435e-38f : sum);
  }
  w *= a.scale;
  if (lane < a.K) {
    const int64_t o = t * a.K + lane;
    if (a.idx64) static_cast<int64_t*>(a.idx)[o] = my_e;
    else static_cast<int32_t*>(a.idx)[o] = my_e;
    a.w[o] = w;
    if (a.masks) {
      const int64_t le = my_e - a.begin;
      if (le >= 0 && le < a.E) {
        atomicOr(a.masks + le, 1ull << t);
        a.slots[le * 64 + t] = static_cast<uint8_t>(lane);
      }
    }
  }
}

template <int NR>
hipError_t launch_select(const SelectArgs& a, hipStream_t st) {
  // a few tokens: one wave a block, on a CU each
  const int threads = a.T <= 256 ? kWave : kThreads;
  const int64_t blocks = cdiv(a.T, threads / kWave);
  hipLaunchKernelGGL(route_select<NR>, dim3(static_cast<unsigned>(blocks)), dim3(threads), 0, st, a);
  return hipGetLastError();
}

}  // namespace

size_t route_workspace(const tr_route_desc& d) {
  return logits_layout(d.T, d.H, d.G, d.dtype == TR_F32).bytes;
}

hipError_t route_topk(const tr_route_desc& d, const void* x, const void* w_gate, const float* bias,
                      void* idx, float* w, void* ws, hipStream_t st, const FewRoutes* few) {
  const bool f32 = d.dtype == TR_F32;
  const LogitsLayout L = logits_layout(d.T, d.H, d.G, f32);
  hipError_t e = logits(d.T, d.H, d.G, f32, x, w_gate, static_cast<float*>(ws),
                        few ? reinterpret_cast<uint32_t*>(few->masks) : nullptr,
                        few ? 2 * few->E : 0, st);
  if (e != hipSuccess) return e;
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
  if (few) {
    a.masks = few->masks;
    a.slots = few->slots;
    a.begin = few->begin;
    a.E = few->E;
  }
  if (d.G <= 64) return launch_select<1>(a, st);
  if (d.G <= 256) return launch_select<4>(a, st);
  if (d.G <= 1024) return launch_select<16>(a, st);
  return launch_select<64>(a, st);
}

}  // namespace tr
