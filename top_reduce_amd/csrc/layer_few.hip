// The local experts of a mixture-of-experts layer for at most 64 tokens, from
// the router's logits to the output, in two launches:
//
//   few_up:    the choice, where it is little work for every block to make it
//              (else it is there already, from a launch of its own)
//              h[t, e] = w[t, e] silu(W1g[e] x[t]) * (W1u[e] x[t])
//   few_down:  y[t]    = sum over the token's local experts e: W2[e] h[t, e]
//
// Bound: reading the weights of the experts that some token chose, once. The
// tokens of an expert are a 64-bit mask, so there is no route scan and no
// expanded copy of x: 16 of an expert's tokens (in most decode batches all of
// them) are the columns of one MFMA operand, weight rows go from memory into
// the other, and a row of h has its place by the expert's tokens before it.
// Both kernels keep two batches of loads per wave, one in flight while the
// other's products run, with a batch small enough that 16 waves fit a CU.
//
// The gate weight is folded into h. bf16: h is kept as two bf16 numbers whose
// sum has 16 significant bits, and few_down multiplies both, as different columns
// of one MFMA operand; y is then rounded once, as if h had never been rounded.
#include "tr_chunk.h"
#include "tr_internal.h"
#include "tr_select.h"

namespace tr {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kDownThreads = 256;
constexpr int kDownWaves = kDownThreads / kWave;
constexpr int kU = 4;   // 64-byte k-blocks of one batch of loads
// groups of 8 or 16 tokens of an expert: one for each expert with a token, and
// one more for every 8 routes at most
constexpr int kMaxGroups = kMaxE + kFewTokens * kMaxK / 8;

struct FewArgs {
  const char* x;                     // [T, H]
  const void* w1;                    // [E, 2 I, H]
  const void* w2;                    // [E, H, I]
  unsigned long long* masks;         // [E] tokens of each local expert
  const uint8_t* slots;              // [E, 64] slot of token t that names expert e
  const float* w;                    // [T, K] gate weights
  char* h;                           // [routes][parts][Ip]
  void* y;                           // [T, H]
  int T, K, E;
  int64_t H, I, Ip;
};

// Groups in LDS, experts ascending.
struct Groups {
  uint64_t mask[kMaxGroups];   // the expert's tokens
  int expert[kMaxGroups];
  int row[kMaxGroups];         // row of h of the group's first token
  int rank[kMaxGroups];        // that token's rank among the expert's
};

// Fills `s` from masks (E of them) with groups of up to kGroup tokens; returns
// their number. tmp: LDS of kBlock / 64 ints.
template <int kBlock, int kGroup>
__device__ __forceinline__ int find_groups(const unsigned long long* masks, int E, Groups& s, int* tmp) {
  constexpr int kPer = (kMaxE + kBlock - 1) / kBlock;
  const int per = (E + kBlock - 1) / kBlock;
  uint64_t m[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = static_cast<int>(threadIdx.x) * per + j;
    m[j] = j < per && e < E ? masks[e] : 0;
  }
  // routes and groups of the experts before: one scan of both (at most 2048
  // routes and 1280 groups)
  int n = 0, total = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int c = __popcll(m[j]);
    n += c | ((c + kGroup - 1) / kGroup) << 16;
  }
  int at = block_exclusive_scan<kBlock>(n, tmp, &total);
  int row = at & 0xffff, g = at >> 16;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int c = __popcll(m[j]);
    for (int k = 0; k < c; k += kGroup) {
      s.mask[g] = m[j];
      s.expert[g] = static_cast<int>(threadIdx.x) * per + j;
      s.row[g] = row + k;
      s.rank[g] = k;
      ++g;
    }
    row += c;
  }
  __syncthreads();
  return total >> 16;
}

// The token of rank `rank` + r in `mask` (r the lane's; r >= n: the group's first
// token). mask and rank are the same in every lane.
__device__ __forceinline__ int group_token(uint64_t mask, int rank, int n, int r) {
  const int lane = lane_id();
  // lane t of the mask sends t to the lane of its rank
  const int to = (mask >> lane) & 1 ? popc_below(mask) : 63;
  int by_rank = __builtin_amdgcn_ds_permute(to * 4, lane);
  // (64 tokens: lane 63 is its own rank; fewer: what lane 63 gets is not used)
  return __shfl(by_rank, rank + (r < n ? r : 0), kWave);
}

// Up to this many tokens (one a wave) and experts few_up makes the choice: every
// block repeats it, 2.5 us, which is less than the launch that it saves (about
// 5 us on the GPU, 3 on the host). Two tokens a wave cost as much as the launch,
// four more (16 tokens of 8 experts: 11.1 us instead of 5.6 + 3.2).
constexpr int kChooseTokens = kWaves;
constexpr int kChooseGates = 256;

// A unit: 16 gate rows and the matching 16 up rows of one group's expert, the
// reduction over the block's waves. NR > 0: every block makes the tokens'
// choice from the logits' parts (NR registers a lane); block 0 stores it.
template <bool kF32, int NR>
__global__ __launch_bounds__(kThreads, 3) void few_up(FewArgs a, SelectArgs sel, int64_t begin) {
  __shared__ Groups s;
  __shared__ int tmp[kWaves];
  __shared__ floatx4 red[kWaves][2][kWave];
  __shared__ unsigned long long mask_s[NR ? kChooseGates : 1];
  __shared__ float w_s[NR ? kChooseGates * kChooseTokens : 1];   // [local expert][token]
  __shared__ SelectScratch scratch[NR ? kWaves : 1];
  if constexpr (NR > 0) {
    for (int e = threadIdx.x; e < a.E; e += kThreads) mask_s[e] = 0;
    __syncthreads();
    const int t = threadIdx.x >> 6;
    if (t < a.T) {
      const Chosen c = choose<NR>(sel, t, scratch[t]);
      if (blockIdx.x == 0) store_chosen(sel, t, c);
      const int64_t e = c.e - begin;
      if (c.rank >= 0 && e >= 0 && e < a.E) {
        atomicOr(&mask_s[e], 1ull << t);
        w_s[e * a.T + t] = c.w;
      }
    }
    __syncthreads();
    if (blockIdx.x == 0)
      for (int e = threadIdx.x; e < a.E; e += kThreads) a.masks[e] = mask_s[e];
  }
  const int n_groups = find_groups<kThreads, 16>(NR ? mask_s : a.masks, a.E, s, tmp);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int upe = static_cast<int>(a.Ip / 16);
  const int total = n_groups * upe;
  const int64_t row_bytes = a.H * Elem<kF32>::kBytes;
  const int nkb = static_cast<int>((row_bytes + 63) >> 6), nfull = static_cast<int>(row_bytes >> 6);
  const int kb0 = wave * nkb / kWaves, kb1 = (wave + 1) * nkb / kWaves;
  const int kbf = min(kb1, nfull);
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    const int q = u / upe, c = u % upe;
    const int e = __builtin_amdgcn_readfirstlane(s.expert[q]);
    const uint64_t mask = s.mask[q];
    const int rank = s.rank[q];
    const int n = min(16, __popcll(mask) - rank);   // tokens of the group
    const int t = group_token(mask, rank, n, r);
    // addresses: a start that is the same for the wave, 32-bit offsets in it.
    // Rows past I (the last units fill h up to Ip with zeros) read the last row.
    const int64_t c0 = min(static_cast<int64_t>(c * 16), a.I - 1);
    const char* wg = static_cast<const char*>(a.w1) + (2 * e * a.I + c0) * row_bytes;
    const char* wu = wg + a.I * row_bytes;
    const uint32_t wo = static_cast<uint32_t>(min(static_cast<int64_t>(r), a.I - 1 - c0)) *
                            static_cast<uint32_t>(row_bytes) + g * 16;
    const uint32_t xo = static_cast<uint32_t>(t) * static_cast<uint32_t>(row_bytes) + g * 16;
    floatx4 ag = {0, 0, 0, 0}, au = {0, 0, 0, 0};

    struct Batch {
      u32x4 wg[kU], wu[kU], x[kU];
    } b0, b1;
    // a share's last batch starts early enough to end with it; the products of
    // blocks that it reads again are skipped
    auto start = [&](int kb) { return min(kb, max(kbf - kU, 0)); };
    auto load = [&](Batch& b, int kb) {
      const uint32_t k = static_cast<uint32_t>(start(kb)) * 64;
#pragma unroll
      for (int j = 0; j < kU; ++j) {
        b.wg[j] = load16(wg + (wo + k) + j * 64);
        b.wu[j] = load16(wu + (wo + k) + j * 64);
        b.x[j] = load16(a.x + (xo + k) + j * 64);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    auto mma = [&](const Batch& b, int kb) {
      const int k = start(kb);
#pragma unroll
      for (int j = 0; j < kU; ++j)
        if (k + j >= kb && k + j < kbf) {
          ag = mma16<kF32>(b.wg[j], b.x[j], ag);
          au = mma16<kF32>(b.wu[j], b.x[j], au);
        }
      __builtin_amdgcn_sched_barrier(0);
    };
    if (nfull >= kU) {
      // (no load below is under a condition inside the loop: a load that may not
      // have been made would turn the waits for the batch before it into waits
      // for everything)
      if (kb0 < kbf) {
        load(b0, kb0);
        int kb = kb0;
        for (; kb + 2 * kU < kbf; kb += 2 * kU) {
          load(b1, kb + kU);
          mma(b0, kb);
          load(b0, kb + 2 * kU);
          mma(b1, kb + kU);
        }
        if (kb + kU < kbf) {
          load(b1, kb + kU);
          mma(b0, kb);
          mma(b1, kb + kU);
        } else {
          mma(b0, kb);
        }
      }
    } else {   // rows of fewer blocks than a batch has
      for (int kb = kb0; kb < kbf; ++kb) {
        const u32x4 vx = load16(a.x + xo + kb * 64);
        ag = mma16<kF32>(load16(wg + wo + kb * 64), vx, ag);
        au = mma16<kF32>(load16(wu + wo + kb * 64), vx, au);
      }
    }
    if (kb1 > nfull) {   // the short block at the end of the rows
      const bool in = nfull * 64 + g * 16 < row_bytes;
      const u32x4 z = {0, 0, 0, 0};
      const u32x4 vg = in ? load16(wg + wo + nfull * 64) : z;
      const u32x4 vu = in ? load16(wu + wo + nfull * 64) : z;
      const u32x4 vx = in ? load16(a.x + xo + nfull * 64) : z;
      ag = mma16<kF32>(vg, vx, ag);
      au = mma16<kF32>(vu, vx, au);
    }
    red[wave][0][lane] = ag;
    red[wave][1][lane] = au;
    __syncthreads();
    if (wave == 0 && r < n) {
      floatx4 vg = red[0][0][lane], vu = red[0][1][lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) {
        vg += red[w][0][lane];
        vu += red[w][1][lane];
      }
      const float wt = NR ? w_s[e * a.T + t] : a.w[t * a.K + a.slots[e * 64 + t]];
      const int64_t col = c * 16 + 4 * g;
      const int64_t row = s.row[q] + r;
      floatx4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = col + j < a.I ? wt * swiglu<kF32>(vg[j], vu[j]) : 0.0f;
      if constexpr (kF32) {
        *reinterpret_cast<floatx4*>(a.h + (row * a.Ip + col) * 4) = v;
      } else {
        const uint32_t h0 = cvt_bf16x2(v[0], v[1]), h1 = cvt_bf16x2(v[2], v[3]);
        // the rest of a number past bf16's range (or of a NaN) is 0, not NaN
        const float hf[4] = {__uint_as_float(h0 << 16), __uint_as_float(h0 & 0xffff0000u),
                             __uint_as_float(h1 << 16), __uint_as_float(h1 & 0xffff0000u)};
        float lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) lo[j] = fabsf(hf[j]) <= 3.3895314e38f ? v[j] - hf[j] : 0.0f;
        char* dst = a.h + (row * 2 * a.Ip + col) * 2;
        *reinterpret_cast<uint2*>(dst) = uint2{h0, h1};
        *reinterpret_cast<uint2*>(dst + a.Ip * 2) = uint2{cvt_bf16x2(lo[0], lo[1]), cvt_bf16x2(lo[2], lo[3])};
      }
    }
    __syncthreads();
  }
}

// A wave's place in the (group, batch) pairs of few_down.
struct Item {
  int q, b;
  __device__ __forceinline__ void next(int nb) {
    if (++b == nb) {
      b = 0;
      ++q;
    }
  }
};

// A unit: 16 output columns of every token; the block's waves share the
// reduction. A wave adds a group's sums to its tokens' totals, which it keeps
// in LDS, experts ascending, so an expert's infinities reach its own tokens
// only; then the waves' totals are added.
// The second MFMA operand has 16 columns. bf16: a group is 8 tokens, whose h
// fill columns 0 to 7 with their first numbers and 8 to 15 with their second, so
// that a batch loads as much of h as of w2. (16 tokens and two operands load
// twice as much of h: OLD)
// kVec: rows of w2 start on 16 bytes.
template <bool kF32, bool kVec>
__global__ __launch_bounds__(kDownThreads, 3) void few_down(FewArgs a) {
  typedef typename Elem<kF32>::type E;
  constexpr int kC = Elem<kF32>::kChunk, kB = Elem<kF32>::kBytes;
  constexpr int kParts = kF32 ? 1 : 2, kGroup = 16 / kParts;
  __shared__ Groups s;
  __shared__ int tmp[kDownWaves];
  __shared__ floatx4 sum[kDownWaves][kFewTokens][4];
  const int n_groups = find_groups<kDownThreads, kGroup>(a.masks, a.E, s, tmp);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int tr = r % kGroup, part = r / kGroup;   // the lane's token of a group and number
  const int I = static_cast<int>(a.I), Ip = static_cast<int>(a.Ip);
  // This wave's 64-byte blocks of every row of h and w2 (the same for every
  // expert, so that a token's sums do not depend on the other tokens), in
  // batches of kU: whole blocks by wide loads, the last of which start early
  // enough to end with the share; then what is left of the row's end.
  const int nkb = (I * kB + 63) >> 6;
  const int nfull = kVec && (I * kB >> 6) >= kU ? I * kB >> 6 : 0;
  const int kb0 = wave * nkb / kDownWaves, kb1 = (wave + 1) * nkb / kDownWaves;
  const int kbf = max(min(kb1, nfull), kb0);
  const int nbf = (kbf - kb0 + kU - 1) / kU;
  const int items = n_groups * nbf;
  const int units = static_cast<int>((a.H + 15) / 16);
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    // (H is a multiple of 8: the last unit may have 8 columns)
    const uint32_t lr = static_cast<uint32_t>(min(static_cast<int64_t>(r), a.H - 1 - u * 16));
    const uint32_t wo = lr * static_cast<uint32_t>(I * kB) + g * 16;
    for (int t = lane; t < a.T * 4; t += kWave) sum[wave][t >> 2][t & 3] = floatx4{0, 0, 0, 0};
    floatx4 acc = {0, 0, 0, 0};

    struct Batch {
      u32x4 w[kU], h[kU];
    } b0, b1;
    auto start = [&](int b) { return min(kb0 + b * kU, max(kbf - kU, 0)); };
    auto w_at = [&](int q) {
      const int e = __builtin_amdgcn_readfirstlane(s.expert[q]);
      return static_cast<const char*>(a.w2) + (e * a.H + u * 16) * a.I * kB;
    };
    auto h_at = [&](int q) {
      const int row = __builtin_amdgcn_readfirstlane(s.row[q]);
      return a.h + static_cast<int64_t>(row) * kParts * Ip * kB;
    };
    // the lane's row of h; past the group's last token its first one's
    auto h_off = [&](int q) {
      const int n = __popcll(s.mask[q]) - s.rank[q];
      return static_cast<uint32_t>((tr < n ? tr * kParts : 0) + part) * Ip * kB + g * 16;
    };
    auto load = [&](Batch& v, const Item& it) {
      const char* w0 = w_at(it.q);
      const char* h0 = h_at(it.q);
      const uint32_t k = static_cast<uint32_t>(start(it.b)) * 64, ho = h_off(it.q) + k;
#pragma unroll
      for (int j = 0; j < kU; ++j) {
        v.w[j] = load16(w0 + (wo + k) + j * 64);
        v.h[j] = load16(h0 + ho + j * 64);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    // the group's sums to its tokens
    auto add = [&](int q) {
      const uint64_t mask = s.mask[q];
      const int rank = s.rank[q];
      const int n = min(kGroup, __popcll(mask) - rank);
      const int t = group_token(mask, rank, n, r);
      if constexpr (kParts == 2) {
        // lanes 0 to 7 of each 16: what the second numbers, 8 lanes on, gave
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[j] += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(acc[j]), 0x128, 15, 15, true));
      }
      if (r < n) sum[wave][t][g] += acc;
      acc = floatx4{0, 0, 0, 0};
    };
    auto mma = [&](const Batch& v, Item& it) {
      // products of blocks that a batch reads again are skipped
      const int k = start(it.b), kb = kb0 + it.b * kU;
#pragma unroll
      for (int j = 0; j < kU; ++j)
        if (k + j >= kb && k + j < kbf) acc = mma16<kF32>(v.w[j], v.h[j], acc);
      __builtin_amdgcn_sched_barrier(0);
      if (it.b + 1 == nbf) add(it.q);
      it.next(nbf);
    };
    if (items > 0) {   // as in few_up: no load under a condition
      Item at{0, 0}, ahead{0, 0};   // of the products, of the loads
      load(b0, ahead);
      int i = 0;
      for (; i + 2 < items; i += 2) {
        ahead.next(nbf);
        load(b1, ahead);
        mma(b0, at);
        ahead.next(nbf);
        load(b0, ahead);
        mma(b1, at);
      }
      if (i + 1 < items) {
        ahead.next(nbf);
        load(b1, ahead);
        mma(b0, at);
        mma(b1, at);
      } else {
        mma(b0, at);
      }
    }
    if (kbf < kb1) {
      // what is left of the rows: past I both operands are zero (h has zeros from
      // I to Ip)
      for (int q = 0; q < n_groups; ++q) {
        const E* wrow = reinterpret_cast<const E*>(w_at(q) + lr * static_cast<uint32_t>(I * kB));
        const char* hrow = h_at(q) + h_off(q);
        for (int kb = kbf; kb < kb1; kb += kU) {
          u32x4 w[kU], h[kU];
#pragma unroll
          for (int j = 0; j < kU; ++j) {
            const int k = (kb + j) * 4 * kC + g * kC;
            const bool in = kb + j < kb1;
            w[j] = u32x4{0, 0, 0, 0};
            if (in && k < I) {
              if constexpr (kVec) w[j] = load16(reinterpret_cast<const char*>(wrow + k));
              else w[j] = load16_any<kF32>(wrow, k, I);
            }
            h[j] = in && k < Ip ? load16(hrow + (kb + j) * 64) : u32x4{0, 0, 0, 0};
          }
#pragma unroll
          for (int j = 0; j < kU; ++j) acc = mma16<kF32>(w[j], h[j], acc);
        }
        add(q);
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.T * 4; i += kDownThreads) {
      const int t = i >> 2, gg = i & 3;
      floatx4 v = sum[0][t][gg];
#pragma unroll
      for (int w = 1; w < kDownWaves; ++w) v += sum[w][t][gg];
      store4<kF32>(static_cast<E*>(a.y) + t * a.H, u * 16 + 4 * gg, a.H, true, v);
    }
    __syncthreads();
  }
}

template <bool kF32>
hipError_t launch_few(const FewArgs& a, const SelectArgs* sel, int64_t begin, hipStream_t st) {
  const int cus = device_cu_count();
  const int64_t most = static_cast<int64_t>(a.T) * a.K < a.E ? static_cast<int64_t>(a.T) * a.K
                                                             : a.E + static_cast<int64_t>(a.T) * a.K / 16;
  const int64_t u1 = most * (a.Ip / 16), u2 = cdiv(a.H, 16);
  // as many blocks as fit at once
  const unsigned g1 = static_cast<unsigned>(u1 < 3 * cus ? u1 : 3 * cus);
  const unsigned g2 = static_cast<unsigned>(u2 < 2 * cus ? u2 : 2 * cus);
  if (!sel)
    hipLaunchKernelGGL((few_up<kF32, 0>), dim3(g1), dim3(kThreads), 0, st, a, SelectArgs{}, begin);
  else if (sel->G <= 64)
    hipLaunchKernelGGL((few_up<kF32, 1>), dim3(g1), dim3(kThreads), 0, st, a, *sel, begin);
  else
    hipLaunchKernelGGL((few_up<kF32, 4>), dim3(g1), dim3(kThreads), 0, st, a, *sel, begin);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.I % Elem<kF32>::kChunk == 0)
    hipLaunchKernelGGL((few_down<kF32, true>), dim3(g2), dim3(kDownThreads), 0, st, a);
  else
    hipLaunchKernelGGL((few_down<kF32, false>), dim3(g2), dim3(kDownThreads), 0, st, a);
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

hipError_t few_layer(const tr_layer_desc& d, const void* x, const void* w_gate, const float* bias,
                     const void* w1, const void* w2, void* y, void* idx, float* w, void* route_ws,
                     void* ws, hipStream_t st) {
  const FewLayout L = few_layout(d);
  const tr_route_desc& r = d.route;
  const bool f32 = r.dtype == TR_F32;
  char* b = static_cast<char*>(ws);
  const FewRoutes f{reinterpret_cast<unsigned long long*>(b + L.masks),
                    reinterpret_cast<uint8_t*>(b + L.slots), d.expert_begin, d.E};
  const bool fused = r.T <= kChooseTokens && r.G <= kChooseGates;
  hipError_t e = fused ? logits(r.T, r.H, r.G, f32, x, w_gate, static_cast<float*>(route_ws), nullptr, 0, st)
                       : route_topk(r, x, w_gate, bias, idx, w, route_ws, st, &f);
  if (e != hipSuccess) return e;
  FewArgs a{};
  a.x = static_cast<const char*>(x);
  a.w1 = w1;
  a.w2 = w2;
  a.masks = f.masks;
  a.slots = f.slots;
  a.w = w;
  a.h = b + L.h;
  a.y = y;
  a.T = static_cast<int>(r.T);
  a.K = r.K;
  a.E = d.E;
  a.H = r.H;
  a.I = d.I;
  a.Ip = L.Ip;
  const SelectArgs sel = select_args(r, bias, idx, w, route_ws);
  return f32 ? launch_few<true>(a, fused ? &sel : nullptr, d.expert_begin, st)
             : launch_few<false>(a, fused ? &sel : nullptr, d.expert_begin, st);
}

}  // namespace tr
