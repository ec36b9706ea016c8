// Router selection of one token by one wave (router.hip, layer_few.hip).
//
//   p = softmax(logits) over all G experts, or sigmoid(logits)
//   key = logits (both scores keep their order), or p + bias with a balancing
//         bias, which decides the selection only
//   idx = the K largest keys, descending, ties to the lowest id
//   w   = scale * p[idx], divided by their sum with renorm
//
// Expert 64 i + lane is in register i. Keys are compared as integers that order
// like the floats, NaN below everything, so that every token gets K different
// valid ids. The K-th largest of the lanes' largest keys is a bound that at
// least K keys reach (for K up to 8 a lower one that is quicker to find serves:
// the least of eight groups' largest keys). The keys that reach it, seldom many
// more than K, are gathered into one register, lowest id first, and each one's
// place is the number of keys before it. These are counting loops of independent
// steps, not K rounds of a reduction over the wave: choosing 16 of 896 took
// 3.9 us in rounds of 0.25 us (the whole kernel 8.3 us, now 5.2). Where over 64
// keys reach the bound (many equal ones) the rounds are taken.
#pragma once

#include <type_traits>

#include "tr_device.h"

namespace tr {

struct SelectArgs {
  const float* part;     // [S, T, pitch] parts of the logits
  const float* bias;     // [G] or NULL
  void* idx;             // [T, K] int32 or int64
  float* w;              // [T, K]
  int64_t T;
  int S, pitch, G, K;
  int idx64, sigmoid, renorm;
  float scale;
};

// LDS of one wave's selection.
struct SelectScratch {
  uint32_t key[kWave];
  int id[kWave];
  float v[kWave];
};

// A lane's share of a token's choice: expert `e` at place `rank` (-1: none).
struct Chosen {
  int rank, e;
  float w;
};

constexpr uint32_t kUsed = 0, kNan = 1;

// An integer that orders like v: kNan < -inf < ... < +inf; -0 and +0 alike.
__device__ __forceinline__ uint32_t order_key(float v) {
  v += 0.0f;
  const uint32_t u = __float_as_uint(v);
  if ((u & 0x7fffffffu) > 0x7f800000u) return kNan;
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Lanes moved within rows of 16 by DPP.
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_move(uint32_t v) {
  return static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(0, static_cast<int>(v), kCtrl, 0xf, 0xf, false));
}

// Reductions over the 64 lanes by row operations: lanes swapped within rows of
// 16 by DPP, then rows 0 and 2 into 1 and 3 and row 1 into 3; lane 63 holds the
// result.
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
__device__ __forceinline__ uint32_t wave_min(uint32_t v) {
  return wave_reduce(v, ~0u, [](uint32_t a, uint32_t b) { return min(a, b); });
}
__device__ __forceinline__ float wave_sum(float v) {
  return __uint_as_float(wave_reduce(__float_as_uint(v), 0u, [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

__device__ __forceinline__ int wave_add(int v) {
  return static_cast<int>(wave_reduce(static_cast<uint32_t>(v), 0u, [](uint32_t a, uint32_t b) { return a + b; }));
}
// How many of the first n lanes' keys are larger than this lane's (lanes from n
// on hold kUsed, so that the count may go on to the next multiple of 8).
__device__ __forceinline__ int count_larger(uint32_t key, int n) {
  int c = 0;
  for (int j0 = 0; j0 < n; j0 += 8) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      c += static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(key), j0 + j)) > key;
  }
  return c;
}

// Token t's choice; NR registers of logits a lane: G <= 64 NR.
template <int NR>
__device__ __forceinline__ Chosen choose(const SelectArgs& a, int64_t t, SelectScratch& s) {
  const int lane = lane_id();
  // v: the logits, and with a bias (which needs every score) the scores
  float v[NR];
  uint32_t key[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) v[i] = 0.0f;
  {
    // several parts' loads at a time, unconditional (indices clamped into the
    // row) so that all go out before the first wait
    constexpr int kB = NR <= 1 ? 8 : NR <= 16 ? 4 : 1;
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
  uint32_t best = kUsed;   // the lane's largest key
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    key[i] = i * kWave + lane < a.G ? order_key(v[i]) : kUsed;
    best = max(best, key[i]);
  }
  float m = 0.0f, sum = 1.0f;
  if (!a.sigmoid) {
    // the largest logit (of those that are numbers), the sum of exp
    const uint32_t mk = wave_max(best);
    m = __uint_as_float((mk & 0x80000000u) ? mk & 0x7fffffffu : ~mk);
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NR; ++i) sum += i * kWave + lane < a.G ? expf(v[i] - m) : 0.0f;
    sum = wave_sum(sum);
  }
  auto score = [&](float l) { return a.sigmoid ? 1.0f / (1.0f + expf(-l)) : expf(l - m) / sum; };
  if (a.bias) {
    best = kUsed;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int e = i * kWave + lane;
      v[i] = score(v[i]);
      if (e < a.G) key[i] = order_key(v[i] + a.bias[e]);
      best = max(best, key[i]);
    }
  }

  // candidates: c_n of them, lowest id first, one a lane
  uint32_t c_key = key[0];
  int c_id = lane, c_n = a.G;
  float c_v = v[0];
  if constexpr (NR > 1) {
    uint32_t bound;
    if (a.K <= 8) {
      // the least of the maxima of 8 groups of 8 lanes: it takes about 8 (1 + 1/2
      // + .. + 1/8) = 22 of the largest keys, dealt to 8 groups, to reach them all
      uint32_t g = best;
      g = max(g, dpp_move<0xb1>(g));
      g = max(g, dpp_move<0x4e>(g));
      g = max(g, dpp_move<0x141>(g));
      bound = wave_min(g);
    } else {
      // the least of the lane maxima with fewer than K larger ones
      const int larger = count_larger(best, kWave);
      bound = wave_min(larger < a.K ? best : ~0u);
    }
    c_n = 0;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const uint64_t in = __ballot(key[i] >= bound);   // (bound > kUsed)
      const int at = c_n + popc_below(in);
      if (key[i] >= bound && at < kWave) {
        s.key[at] = key[i];
        s.id[at] = i * kWave + lane;
        s.v[at] = v[i];
      }
      c_n += __popcll(in);
    }
    wave_lds_fence();
    if (c_n <= kWave) {
      c_key = s.key[lane];
      c_id = s.id[lane];
      c_v = s.v[lane];
    } else {
      // K rounds over the wave; lane k keeps the k-th expert
      c_n = a.K;
      for (int k = 0; k < a.K; ++k) {
        uint32_t lb = key[0];
        int li = 0;
        float lv = v[0];
#pragma unroll
        for (int i = 1; i < NR; ++i)
          if (key[i] > lb) {
            lb = key[i];
            li = i;
            lv = v[i];
          }
        const uint32_t top = wave_max(lb);
        const uint32_t e = ~wave_max(lb == top ? ~static_cast<uint32_t>(li * kWave + lane) : 0u);
        const int owner = static_cast<int>(e & 63);
        const float ev = __uint_as_float(static_cast<uint32_t>(
            __builtin_amdgcn_readlane(static_cast<int>(__float_as_uint(lv)), owner)));
        if (lane == k) {
          c_key = ~0u - k;   // already in order
          c_id = static_cast<int>(e);
          c_v = ev;
        }
#pragma unroll
        for (int i = 0; i < NR; ++i)
          if (lane == owner && i == li) key[i] = kUsed;
      }
    }
  }
  // A candidate's place: the larger ones, and the equal ones of lower id. Without
  // equal keys the first are a permutation, whose sum is known.
  if (lane >= c_n) c_key = kUsed;
  Chosen c{count_larger(c_key, c_n), c_id, 0.0f};
  if (wave_add(lane < c_n ? c.rank : 0) != c_n * (c_n - 1) / 2) {
    for (int j = 0; j < c_n; ++j)
      c.rank += static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(c_key), j)) == c_key && j < lane;
  }
  if (lane >= c_n || c.rank >= a.K) c.rank = -1;
  const float p = c.rank < 0 ? 0.0f : a.bias ? c_v : score(c_v);
  c.w = p;
  if (a.renorm) {
    // a sum below the smallest normal float (all scores 0) counts as that:
    // weights 0, not NaN
    const float all = wave_sum(p);
    c.w = p / (all < 1.17549435e-38f ? 1.17549435e-38f : all);
  }
  c.w *= a.scale;
  return c;
}

// The choice to the caller's arrays.
__device__ __forceinline__ void store_chosen(const SelectArgs& a, int64_t t, const Chosen& c) {
  if (c.rank < 0) return;
  const int64_t o = t * a.K + c.rank;
  if (a.idx64) static_cast<int64_t*>(a.idx)[o] = c.e;
  else static_cast<int32_t*>(a.idx)[o] = c.e;
  a.w[o] = c.w;
}

}  // namespace tr
