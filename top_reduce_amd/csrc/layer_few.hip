// The local experts of a mixture-of-experts layer for at most 64 tokens, from
// the router's choice to the output, in two launches:
//
//   few_up:    h[t, k] = w[t, k] silu(W1g[e] x[t]) * (W1u[e] x[t])   e = idx[t, k]
//   few_down:  y[t]    = sum over the token's local experts e: W2[e] h[t, k(e)]
//
// Bound: reading the weights of the experts that some token chose, once. The
// tokens of an expert are a 64-bit mask, so there is no expanded row order and
// no route scan: in few_up the tokens ride in MFMA columns in groups of 16
// (groups without a token of the expert are skipped), and few_down adds a
// column's sum over an expert to the token's total where the token chose it,
// experts ascending, so that the weighted sum over experts stays in registers.
//
// The gate weight is folded into h. bf16: h is kept as two bf16 numbers whose
// sum has 16 significant bits, and few_down multiplies both; the MFMA units
// have time for it while the weights stream, and y is then rounded once, as
// if h had never been rounded.
#include "tr_chunk.h"
#include "tr_internal.h"

namespace tr {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kU = 8;   // 64-byte k-blocks of one batch of loads

struct FewArgs {
  const char* x;                     // [T, H]
  const void* w1;                    // [E, 2 I, H]
  const void* w2;                    // [E, H, I]
  const unsigned long long* masks;   // [E] tokens of each local expert
  const uint8_t* slots;              // [E, 64] slot of token t that names expert e
  const float* w;                    // [T, K] gate weights
  char* h;                           // [T * K][parts][Ip]
  void* y;                           // [T, H]
  int T, K, E;
  int64_t H, I, Ip;
};

// The experts with a token, in ascending order, in LDS; returns how many.
template <int kBlock>
__device__ __forceinline__ int active_experts(const FewArgs& a, int* list, uint64_t* mask_s,
                                              int* tmp) {
  constexpr int kPer = kMaxE / kBlock;
  const int per = (a.E + kBlock - 1) / kBlock;
  uint64_t m[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = static_cast<int>(threadIdx.x) * per + j;
    m[j] = j < per && e < a.E ? a.masks[e] : 0;
  }
  int n = 0, total = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) n += m[j] != 0;
  int at = block_exclusive_scan<kBlock>(n, tmp, &total);
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (m[j]) {
      list[at] = static_cast<int>(threadIdx.x) * per + j;
      mask_s[at] = m[j];
      ++at;
    }
  __syncthreads();
  return total;
}

// A unit: 16 gate rows and the matching 16 up rows of one expert, the
// reduction over the block's waves.
template <bool kF32, int NQ>
__global__ __launch_bounds__(kThreads) void few_up(FewArgs a) {
  __shared__ int list[kMaxE];
  __shared__ uint64_t mask_s[kMaxE];
  __shared__ int tmp[kWaves];
  __shared__ floatx4 red[kWaves][NQ][2][kWave];
  const int n_act = active_experts<kThreads>(a, list, mask_s, tmp);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, r = lane & 15;
  const int upe = static_cast<int>(a.Ip / 16);
  const int total = n_act * upe;
  const int64_t row_bytes = a.H * Elem<kF32>::kBytes;
  const int nkb = static_cast<int>((row_bytes + 63) >> 6), nfull = static_cast<int>(row_bytes >> 6);
  const int kb0 = wave * nkb / kWaves, kb1 = (wave + 1) * nkb / kWaves;
  const int kbf = min(kb1, nfull);
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    const int q = u / upe, c = u % upe;
    const int e = list[q];
    const uint64_t mask = mask_s[q];
    const int first = __ffsll(static_cast<unsigned long long>(mask)) - 1;
    const int64_t col = min(static_cast<int64_t>(c * 16 + r), a.I - 1);
    const char* wg = static_cast<const char*>(a.w1) + (2 * e * a.I + col) * row_bytes + g * 16;
    const char* wu = wg + a.I * row_bytes;
    const char* xp[NQ];
    bool on[NQ];
    floatx4 ag[NQ], au[NQ];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int t = i * 16 + r;
      on[i] = (mask >> (16 * i)) & 0xffff;
      xp[i] = a.x + ((mask >> t) & 1 ? t : first) * row_bytes + g * 16;
      ag[i] = au[i] = floatx4{0, 0, 0, 0};
    }
    // Batches of kU blocks. A share's last batch may be short: its loads
    // re-read the last whole block and the products are skipped.
    for (int kb = kb0; kb < kbf; kb += kU) {
      u32x4 vg[kU], vu[kU];
#pragma unroll
      for (int j = 0; j < kU; ++j) {
        vg[j] = load16(wg + min(kb + j, kbf - 1) * 64);
        vu[j] = load16(wu + min(kb + j, kbf - 1) * 64);
      }
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        if (NQ > 1 && !on[i]) continue;
        u32x4 xb[kU];
#pragma unroll
        for (int j = 0; j < kU; ++j) xb[j] = load16(xp[i] + min(kb + j, kbf - 1) * 64);
        // every load of the batch is out before the first product
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < kU; ++j)
          if (kb + j < kbf) {
            ag[i] = mma16<kF32>(vg[j], xb[j], ag[i]);
            au[i] = mma16<kF32>(vu[j], xb[j], au[i]);
          }
      }
    }
    if (kb1 > nfull) {   // the short block at the end of the rows
      const bool in = nfull * 64 + g * 16 < row_bytes;
      const u32x4 z = {0, 0, 0, 0};
      const u32x4 vg = in ? load16(wg + nfull * 64) : z, vu = in ? load16(wu + nfull * 64) : z;
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        if (!on[i]) continue;
        const u32x4 xb = in ? load16(xp[i] + nfull * 64) : z;
        ag[i] = mma16<kF32>(vg, xb, ag[i]);
        au[i] = mma16<kF32>(vu, xb, au[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      red[wave][i][0][lane] = ag[i];
      red[wave][i][1][lane] = au[i];
    }
    __syncthreads();
    for (int i = wave; i < NQ; i += kWaves) {
      const int t = i * 16 + r;
      if (!((mask >> t) & 1)) continue;
      floatx4 vg = red[0][i][0][lane], vu = red[0][i][1][lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) {
        vg += red[w][i][0][lane];
        vu += red[w][i][1][lane];
      }
      const int slot = t * a.K + a.slots[e * 64 + t];
      const float wt = a.w[slot];
      const int64_t c0 = c * 16 + 4 * g;
      floatx4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = c0 + j < a.I ? wt * swiglu<kF32>(vg[j], vu[j]) : 0.0f;
      if constexpr (kF32) {
        *reinterpret_cast<floatx4*>(a.h + (slot * a.Ip + c0) * 4) = v;
      } else {
        const uint32_t h0 = cvt_bf16x2(v[0], v[1]), h1 = cvt_bf16x2(v[2], v[3]);
        // the rest of a number past bf16's range (or of a NaN) is 0, not NaN
        const float hf[4] = {__uint_as_float(h0 << 16), __uint_as_float(h0 & 0xffff0000u),
                             __uint_as_float(h1 << 16), __uint_as_float(h1 & 0xffff0000u)};
        float lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) lo[j] = fabsf(hf[j]) <= 3.3895314e38f ? v[j] - hf[j] : 0.0f;
        const uint32_t l0 = cvt_bf16x2(lo[0], lo[1]), l1 = cvt_bf16x2(lo[2], lo[3]);
        char* row = a.h + (slot * 2 * a.Ip + c0) * 2;
        *reinterpret_cast<uint2*>(row) = uint2{h0, h1};
        *reinterpret_cast<uint2*>(row + a.Ip * 2) = uint2{l0, l1};
      }
    }
    __syncthreads();
  }
}

// A unit: 16 output columns of every token; the (expert, batch of k) pairs of
// the sum are shared by the block's waves, each a run of them. kVec: rows of w2
// start on 16 bytes.
constexpr int kDownThreads = 512;
constexpr int kDownWaves = kDownThreads / kWave;

template <bool kF32, int NQ, bool kVec>
__global__ __launch_bounds__(kDownThreads) void few_down(FewArgs a) {
  typedef typename Elem<kF32>::type E;
  constexpr int kC = Elem<kF32>::kChunk, kB = Elem<kF32>::kBytes;
  constexpr int kParts = kF32 ? 1 : 2;
  __shared__ int list[kMaxE];
  __shared__ uint64_t mask_s[kMaxE];
  __shared__ int tmp[kDownWaves];
  __shared__ floatx4 red[kDownWaves][NQ][kWave];
  const int n_act = active_experts<kDownThreads>(a, list, mask_s, tmp);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, r = lane & 15;
  const int I = static_cast<int>(a.I), Ip = static_cast<int>(a.Ip);
  const int nkb = (I * kB + 63) >> 6;             // 64-byte blocks of a row
  const int nb = (nkb + kU - 1) / kU;             // batches of an expert
  const int items = n_act * nb;
  const int i0 = static_cast<int>(static_cast<int64_t>(wave) * items / kDownWaves);
  const int i1 = static_cast<int>(static_cast<int64_t>(wave + 1) * items / kDownWaves);
  const int units = static_cast<int>((a.H + 15) / 16);
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t n = min(static_cast<int64_t>(u * 16 + r), a.H - 1);
    floatx4 acc[NQ], cur[NQ];   // over the experts; of the expert at hand
#pragma unroll
    for (int i = 0; i < NQ; ++i) acc[i] = cur[i] = floatx4{0, 0, 0, 0};
    int q = i0 / nb, b = i0 % nb;
    for (int it = i0; it < i1;) {
      // expert q: this wave's batches of it
      const int e = __builtin_amdgcn_readfirstlane(list[q]);
      const uint64_t mask = mask_s[q];
      const E* wrow = static_cast<const E*>(a.w2) + (e * a.H + n) * a.I;
      const char* hp[NQ];
      bool on[NQ];
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        const int t = i * 16 + r;
        const int at = (mask >> t) & 1 ? t : __ffsll(static_cast<unsigned long long>(mask)) - 1;
        on[i] = (mask >> (16 * i)) & 0xffff;
        hp[i] = a.h + static_cast<int64_t>(at * a.K + a.slots[e * 64 + at]) * kParts * Ip * kB;
      }
      const int b1 = min(nb, b + i1 - it);
      it += b1 - b;
      for (; b < b1; ++b) {
        u32x4 wv[kU];
        const int k0 = b * kU * 4 * kC + g * kC;
        const bool whole = (b + 1) * kU * 4 * kC <= I;   // the same in every lane
        if (kVec && whole) {
#pragma unroll
          for (int j = 0; j < kU; ++j) wv[j] = load16(reinterpret_cast<const char*>(wrow + k0 + j * 4 * kC));
        } else {
#pragma unroll
          for (int j = 0; j < kU; ++j) {
            const int k = k0 + j * 4 * kC;
            wv[j] = u32x4{0, 0, 0, 0};
            if (k < I) {
              if constexpr (kVec) wv[j] = load16(reinterpret_cast<const char*>(wrow + k));
              else wv[j] = load16_any<kF32>(wrow, k, I);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
          if (NQ > 1 && !on[i]) continue;
          // past I both operands are zero (h has zeros from I to Ip)
          u32x4 hv[kParts][kU];
#pragma unroll
          for (int part = 0; part < kParts; ++part)
#pragma unroll
            for (int j = 0; j < kU; ++j)
              hv[part][j] = load16(hp[i] + (part * Ip + min(k0 + j * 4 * kC, Ip - kC)) * kB);
          if (!whole) {
#pragma unroll
            for (int part = 0; part < kParts; ++part)
#pragma unroll
              for (int j = 0; j < kU; ++j)
                if (k0 + j * 4 * kC >= Ip) hv[part][j] = u32x4{0, 0, 0, 0};
          }
          // every load of the batch is out before the first product
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int part = 0; part < kParts; ++part)
#pragma unroll
            for (int j = 0; j < kU; ++j) cur[i] = mma16<kF32>(wv[j], hv[part][j], cur[i]);
        }
      }
      // the expert's sums go to its own tokens only: infinities in its weights
      // reach no other
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        if ((mask >> (i * 16 + r)) & 1) acc[i] += cur[i];
        cur[i] = floatx4{0, 0, 0, 0};
      }
      ++q;
      b = 0;
    }
#pragma unroll
    for (int i = 0; i < NQ; ++i) red[wave][i][lane] = acc[i];
    __syncthreads();
    for (int i = wave; i < NQ; i += kDownWaves) {
      const int t = i * 16 + r;
      if (t >= a.T) continue;
      floatx4 v = red[0][i][lane];
#pragma unroll
      for (int w = 1; w < kDownWaves; ++w) v += red[w][i][lane];
      store4<kF32>(static_cast<E*>(a.y) + t * a.H, u * 16 + 4 * g, a.H, true, v);
    }
    __syncthreads();
  }
}

template <bool kF32, int NQ>
hipError_t launch_few(const FewArgs& a, hipStream_t st) {
  const int cus = device_cu_count();
  const int64_t most = static_cast<int64_t>(a.T) * a.K < a.E ? static_cast<int64_t>(a.T) * a.K : a.E;
  const int64_t u1 = most * (a.Ip / 16), u2 = cdiv(a.H, 16);
  const unsigned g1 = static_cast<unsigned>(u1 < 4 * cus ? u1 : 4 * cus);
  const unsigned g2 = static_cast<unsigned>(u2 < 4 * cus ? u2 : 4 * cus);
  hipLaunchKernelGGL((few_up<kF32, NQ>), dim3(g1), dim3(kThreads), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.I % Elem<kF32>::kChunk == 0)
    hipLaunchKernelGGL((few_down<kF32, NQ, true>), dim3(g2), dim3(kDownThreads), 0, st, a);
  else
    hipLaunchKernelGGL((few_down<kF32, NQ, false>), dim3(g2), dim3(kDownThreads), 0, st, a);
  return hipGetLastError();
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct FewLayout {
  size_t masks, slots, h, total;
  int64_t Ip;
};
FewLayout few_layout(const tr_layer_desc& d) {
  FewLayout L{};
  L.Ip = cdiv(d.I, 32) * 32;
  size_t o = 0;
  auto take = [&](size_t n) { const size_t at = o; o = up256(o + n); return at; };
  L.masks = take(8 * static_cast<size_t>(d.E));
  L.slots = take(64 * static_cast<size_t>(d.E));
  // two bf16 or one fp32 number: 4 bytes each
  L.h = take(4 * static_cast<size_t>(d.route.T) * d.route.K * L.Ip);
  L.total = o;
  return L;
}

}  // namespace

size_t few_workspace(const tr_layer_desc& d) { return few_layout(d).total; }

FewRoutes few_routes(const tr_layer_desc& d, void* ws) {
  const FewLayout L = few_layout(d);
  char* b = static_cast<char*>(ws);
  return FewRoutes{reinterpret_cast<unsigned long long*>(b + L.masks),
                   reinterpret_cast<uint8_t*>(b + L.slots), d.expert_begin, d.E};
}

hipError_t few_experts(const tr_layer_desc& d, const void* x, const void* w1, const void* w2,
                       const float* w, void* y, void* ws, hipStream_t st) {
  const FewLayout L = few_layout(d);
  const FewRoutes f = few_routes(d, ws);
  FewArgs a{};
  a.x = static_cast<const char*>(x);
  a.w1 = w1;
  a.w2 = w2;
  a.masks = f.masks;
  a.slots = f.slots;
  a.w = w;
  a.h = static_cast<char*>(ws) + L.h;
  a.y = y;
  a.T = static_cast<int>(d.route.T);
  a.K = d.route.K;
  a.E = d.E;
  a.H = d.route.H;
  a.I = d.I;
  a.Ip = L.Ip;
  const bool f32 = d.route.dtype == TR_F32;
  if (a.T <= 16) return f32 ? launch_few<true, 1>(a, st) : launch_few<false, 1>(a, st);
  if (a.T <= 32) return f32 ? launch_few<true, 2>(a, st) : launch_few<false, 2>(a, st);
  return f32 ? launch_few<true, 4>(a, st) : launch_few<false, 4>(a, st);
}

}  // namespace tr
