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
#include <type_traits>

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

// Reductions over the 64 lanes by row operations: lanes swapped within rows of
// 16 by DPP, then rows 0 and 2 into 1 and 3 and row 1 into 3; lane 63 holds the
// result. A round of the selection waits for this chain.
template <typename F>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, uint32_t neutral, F op) {
  auto dpp = [&](auto ctrl, auto rows) {
    v = op(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
                  static_cast<int>(neutral), static_cast<int>(v), decltype(ctrl)::value,
                  decltype(rows)::value, 0xf, false)));
  };
  using All = std::integral_constant<int, 0xf>;
  dpp(std::integral_constant<int, 0xb1>{}, All{});    // lanes 1 0 3 2
  dpp(std::integral_constant<int, 0x4e>{}, All{});    // lanes 2 3 0 1
  dpp(std::integral_constant<int, 0x141>{}, All{});   // mirrored in 8 lanes
  dpp(std::integral_constant<int, 0x140>{}, All{});   // mirrored in 16 lanes
  dpp(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xa>{});
  dpp(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xc>{});
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  return wave_reduce(v, 0u, [](uint32_t a, uint32_t b) { return max(a, b); });
}
__device__ __forceinline__ float wave_sum(float v) {
  return __uint_as_float(wave_reduce(__float_as_uint(v), 0u, [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

// f(0), f(1), .. f(N - 1) with constants.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void each_group(F f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    each_group<N, I + 1>(f);
  }
}

// NR registers of logits a lane: G <= 64 NR.
template <int NR>
__global__ __launch_bounds__(kThreads) void route_select(SelectArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 6) + (threadIdx.x >> 6);
  if (t >= a.T) return;
  // v: the logits, and with a bias (which needs every score) the scores
  float v[NR];
  uint32_t key[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) v[i] = 0.0f;
  {
    // four parts' loads at a time, unconditional (indices clamped into the
    // row) so that all go out before the first wait
    constexpr int kB = NR <= 4 ? 4 : NR <= 16 ? 2 : 1;
    int col[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) col[i] = min(i * kWave + lane, a.G - 1);
    for (int s0 = 0; s0 < a.S; s0 += kB) {
      float ld[kB][NR];
#pragma unroll
      for (int b = 0; b < kB; ++b) {
        const float* row = a.part + (min(s0 + b, a.S - 1) * a.T + t) * a.pitch;
#pragma unroll
        for (int i = 0; i < NR; ++i) ld[b][i] = row[col[i]];
      }
#pragma unroll
      for (int b = 0; b < kB; ++b)
        if (s0 + b < a.S) {
#pragma unroll
          for (int i = 0; i < NR; ++i) v[i] += ld[b][i];
        }
    }
  }
#pragma unroll
  for (int i = 0; i < NR; ++i) key[i] = i * kWave + lane < a.G ? order_key(v[i]) : kUsed;
  float m = 0.0f, sum = 1.0f;
  if (!a.sigmoid) {
    // the largest logit (of those that are numbers), the sum of exp
    uint32_t best = kUsed;
#pragma unroll
    for (int i = 0; i < NR; ++i) best = max(best, key[i]);
    const uint32_t mk = wave_max(best);
    m = __uint_as_float((mk & 0x80000000u) ? mk & 0x7fffffffu : ~mk);
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NR; ++i) sum += i * kWave + lane < a.G ? expf(v[i] - m) : 0.0f;
    sum = wave_sum(sum);
  }
  auto score = [&](float l) { return a.sigmoid ? 1.0f / (1.0f + expf(-l)) : expf(l - m) / sum; };
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int e = i * kWave + lane;
      v[i] = score(v[i]);
      if (e < a.G) key[i] = order_key(v[i] + a.bias[e]);
    }
  }

  // K rounds; lane k keeps the k-th expert and its value. Every lane offers its
  // largest key (the lowest register among equals), the largest of the maxima
  // of its groups of registers: a round marks one register of one lane, so it
  // renews one group's maximum only (register and group are the same for the
  // whole wave).
  constexpr int kGrp = NR <= 4 ? 1 : NR <= 16 ? 4 : 8;
  constexpr int kPer = NR / kGrp;
  uint32_t gk[kGrp];   // a group's largest key, and its register
  int gi[kGrp];
  auto renew = [&](auto grp) {
    constexpr int q = decltype(grp)::value;
    gk[q] = key[q * kPer];
    gi[q] = q * kPer;
#pragma unroll
    for (int i = q * kPer + 1; i < (q + 1) * kPer; ++i)
      if (key[i] > gk[q]) {
        gk[q] = key[i];
        gi[q] = i;
      }
  };
  each_group<kGrp>(renew);
  int my_e = 0;
  float my_v = 0.0f;
  for (int k = 0; k < a.K; ++k) {
    uint32_t lb = gk[0];
    int li = gi[0];
#pragma unroll
    for (int q = 1; q < kGrp; ++q)
      if (gk[q] > lb) {
        lb = gk[q];
        li = gi[q];
      }
    const uint32_t top = wave_max(lb);
    const uint64_t hit = __ballot(lb == top);
    int owner = __ffsll(static_cast<unsigned long long>(hit)) - 1;
    if (hit & (hit - 1)) {
      // several lanes: the lowest id among them
      const uint32_t e = ~wave_max(lb == top ? ~static_cast<uint32_t>(li * kWave + lane) : 0u);
      owner = static_cast<int>(e & 63);
    }
    const int reg = __builtin_amdgcn_readlane(li, owner);
    float ev = 0.0f;
    each_group<kGrp>([&](auto grp) {
      constexpr int q = decltype(grp)::value;
      if (reg / kPer != q) return;
#pragma unroll
      for (int i = q * kPer; i < (q + 1) * kPer; ++i)
        if (i == reg) {
          ev = __uint_as_float(static_cast<uint32_t>(
              __builtin_amdgcn_readlane(static_cast<int>(__float_as_uint(v[i])), owner)));
          if (lane == owner) key[i] = kUsed;
        }
      renew(grp);
    });
    if (lane == k) {
      my_e = reg * kWave + owner;
      my_v = ev;
    }
  }
  const float my_p = a.bias ? my_v : score(my_v);
  float w = my_p;
  if (a.renorm) {
    const float all = wave_sum(lane < a.K ? my_p : 0.0f);
    // a sum below the smallest normal float (all scores 0) divides by that
    // instead: weights 0, not NaN
    w = my_p / (all < 1.17549435e-38f ? 1.17549435e-38f : all);
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
