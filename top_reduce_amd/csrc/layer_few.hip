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
// expanded copy of x: an expert's tokens are the columns of one MFMA operand,
// weight rows go from memory into the other, and h has its place by the expert's
// tokens before. Both kernels keep two batches of loads per wave, one in flight
// while the other's products run, with a batch small enough that 12 waves fit a
// CU. What a CU reads of rows (16 rows of 64 bytes a load) is at most 34 KB/us,
// from L2 too, so operands beside the weights count: h is stored in the order in
// which few_down loads it (64 tokens of 8 experts, all chosen: 147 -> 100 us).
//
// One token, 8 of 32 experts of 7168 x 2048: 83 + 42 us for 708 MB, 5.7 TB/s; 64
// tokens, 8 of 256 experts, 32 of them here: 237 + 127 us for the 2091 MB of the
// experts chosen, 5.7 TB/s (a kernel that only reads reaches 6.3).
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
// h is kept as few_down multiplies it. An expert's tokens, ascending, in blocks of
// kGroup; of a block, for each 64 bytes of a row, the tokens' pieces with their
// second numbers beside them: 16 pieces, the columns of an MFMA operand.
template <bool kF32>
struct HPlace {
  static constexpr int kParts = kF32 ? 1 : 2, kGroup = 16 / kParts;
};
// groups of tokens of an expert, blocks of h: one for each expert with a token,
// and one more for every 8 routes at most
constexpr int kMaxGroups = kMaxE + kFewTokens * kMaxK / 8;

struct FewArgs {
  const char* x;                     // [T, H]
  const void* w1;                    // [E, 2 I, H]
  const void* w2;                    // [E, H, I]
  unsigned long long* masks;         // [E] tokens of each local expert
  const uint8_t* slots;              // [E, 64] slot of token t that names expert e
  const float* w;                    // [T, K] gate weights
  char* h;                           // [blocks][Ip * bytes / 64][16][64 bytes]
  void* y;                           // [T, H]
  int T, K, E;
  int cols, parts;                   // few_down's units: output columns, parts of the reduction
  bool by_expert;                    // its waves share the experts, not their reductions
  float* sums;                       // [parts][T][H] with more than one part
  int64_t H, I, Ip;
};

// Groups in LDS, experts ascending.
struct Groups {
  uint64_t mask[kMaxGroups];     // the expert's tokens
  uint16_t expert[kMaxGroups];
  uint16_t block[kMaxGroups];    // block of h of the group's first token
  uint16_t rank[kMaxGroups];     // that token's rank among the expert's
};

// Fills `s` from masks (E of them) with groups of up to kGroup tokens; returns
// their number. tmp: LDS of kBlock / 64 ints.
template <bool kF32, int kBlock, int kGroup>
__device__ __forceinline__ int find_groups(const unsigned long long* masks, int E, Groups& s, int* tmp) {
  constexpr int kPer = (kMaxE + kBlock - 1) / kBlock;
  const int per = (E + kBlock - 1) / kBlock;
  uint64_t m[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = static_cast<int>(threadIdx.x) * per + j;
    m[j] = j < per && e < E ? masks[e] : 0;
  }
  constexpr int kH = HPlace<kF32>::kGroup;
  static_assert(kGroup % kH == 0, "whole blocks of h");
  // blocks and groups of the experts before: one scan of both (at most 1280)
  int n = 0, total = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int c = __popcll(m[j]);
    n += (c + kH - 1) / kH | ((c + kGroup - 1) / kGroup) << 16;
  }
  int at = block_exclusive_scan<kBlock>(n, tmp, &total);
  int block = at & 0xffff, g = at >> 16;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int c = __popcll(m[j]);
    for (int k = 0; k < c; k += kGroup) {
      s.mask[g] = m[j];
      s.expert[g] = static_cast<uint16_t>(static_cast<int>(threadIdx.x) * per + j);
      s.block[g] = static_cast<uint16_t>(block + k / kH);
      s.rank[g] = static_cast<uint16_t>(k);
      ++g;
    }
    block += (c + kH - 1) / kH;
  }
  __syncthreads();
  return total >> 16;
}

// Up to this many tokens (one a wave) and experts few_up makes the choice: every
// block repeats it, 2.5 us, which is less than the launch that it saves (about
// 5 us on the GPU, 3 on the host). Two tokens a wave cost as much as the launch,
// four more (16 tokens of 8 experts: 11.1 us instead of 5.6 + 3.2).
constexpr int kChooseTokens = kWaves;
constexpr int kChooseGates = 256;

// A unit: 16 gate rows and the matching 16 up rows of one group's expert, the
// reduction over the block's waves. A group: up to 16 NQ tokens of an expert, for
// which weights are loaded once. NR > 0: every block makes the tokens'
// choice from the logits' parts (NR registers a lane); block 0 stores it.
template <bool kF32, int NR, int NQ>
__global__ __launch_bounds__(kThreads, NQ == 4 ? 2 : 3) void few_up(FewArgs a, SelectArgs sel, int64_t begin) {
  constexpr int kU = NQ == 1 ? 4 : 2;   // 64-byte k-blocks of one batch of loads
  __shared__ Groups s;
  __shared__ int tmp[kWaves];
  __shared__ floatx4 red[kWaves][NQ][2][kWave];
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
  const int n_groups = find_groups<kF32, kThreads, 16 * NQ>(NR ? mask_s : a.masks, a.E, s, tmp);
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
    const int n = min(16 * NQ, __popcll(mask) - rank);   // tokens of the group
    const int by_rank = tokens_by_rank(mask);
    // addresses: a start that is the same for the wave, 32-bit offsets in it.
    // Rows past I (the last units fill h up to Ip with zeros) read the last row.
    const int64_t c0 = min(static_cast<int64_t>(c * 16), a.I - 1);
    const char* wg = static_cast<const char*>(a.w1) + (2 * e * a.I + c0) * row_bytes;
    const char* wu = wg + a.I * row_bytes;
    const uint32_t wo = static_cast<uint32_t>(min(static_cast<int64_t>(r), a.I - 1 - c0)) *
                            static_cast<uint32_t>(row_bytes) + g * 16;
    // (a lane past the group's last token reads its first one's row)
    uint32_t xo[NQ];
    floatx4 ag[NQ], au[NQ];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int t = __shfl(by_rank, rank + (16 * i + r < n ? 16 * i + r : 0), kWave);
      xo[i] = static_cast<uint32_t>(t) * static_cast<uint32_t>(row_bytes) + g * 16;
      ag[i] = au[i] = floatx4{0, 0, 0, 0};
    }

    struct Batch {
      u32x4 wg[kU], wu[kU], x[NQ][kU];
    } b0, b1;
    auto products = [&](const u32x4& vg, const u32x4& vu, int i, const u32x4& vx) {
      ag[i] = mma16<kF32>(vg, vx, ag[i]);
      au[i] = mma16<kF32>(vu, vx, au[i]);
    };
    // a share's last batch starts early enough to end with it; the products of
    // blocks that it reads again are skipped
    auto start = [&](int kb) { return min(kb, max(kbf - kU, 0)); };
    auto load = [&](Batch& b, int kb) {
      const uint32_t k = static_cast<uint32_t>(start(kb)) * 64;
#pragma unroll
      for (int j = 0; j < kU; ++j) {
        b.wg[j] = load16(wg + (wo + k) + j * 64);
        b.wu[j] = load16(wu + (wo + k) + j * 64);
#pragma unroll
        for (int i = 0; i < NQ; ++i) b.x[i][j] = load16(a.x + (xo[i] + k) + j * 64);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    auto mma = [&](const Batch& b, int kb) {
      const int k = start(kb);
#pragma unroll
      for (int j = 0; j < kU; ++j)
        if (k + j >= kb && k + j < kbf) {
#pragma unroll
          for (int i = 0; i < NQ; ++i) products(b.wg[j], b.wu[j], i, b.x[i][j]);
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
        const u32x4 vg = load16(wg + wo + kb * 64), vu = load16(wu + wo + kb * 64);
#pragma unroll
        for (int i = 0; i < NQ; ++i) products(vg, vu, i, load16(a.x + xo[i] + kb * 64));
      }
    }
    if (kb1 > nfull) {   // the short block at the end of the rows
      const bool in = nfull * 64 + g * 16 < row_bytes;
      const u32x4 z = {0, 0, 0, 0};
      const u32x4 vg = in ? load16(wg + wo + nfull * 64) : z;
      const u32x4 vu = in ? load16(wu + wo + nfull * 64) : z;
#pragma unroll
      for (int i = 0; i < NQ; ++i) products(vg, vu, i, in ? load16(a.x + xo[i] + nfull * 64) : z);
    }
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      red[wave][i][0][lane] = ag[i];
      red[wave][i][1][lane] = au[i];
    }
    __syncthreads();
    static_assert(NQ <= kWaves, "a wave for every 16 tokens");
    const int at = 16 * wave + r;   // of the group's tokens
    const int t = __shfl(by_rank, min(rank + at, kWave - 1), kWave);
    if (wave < NQ && at < n) {
      const int i = min(wave, NQ - 1);
      floatx4 vg = red[0][i][0][lane], vu = red[0][i][1][lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) {
        vg += red[w][i][0][lane];
        vu += red[w][i][1][lane];
      }
      const float wt = NR ? w_s[e * a.T + t] : a.w[t * a.K + a.slots[e * 64 + t]];
      const int64_t col = c * 16 + 4 * g;
      typedef HPlace<kF32> P;
      char* dst = a.h + ((s.block[q] + at / P::kGroup) * (a.Ip * Elem<kF32>::kBytes >> 6) +
                         (col * Elem<kF32>::kBytes >> 6)) * 1024 +
                  at % P::kGroup * P::kParts * 64 + (col * Elem<kF32>::kBytes & 63);
      floatx4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = col + j < a.I ? wt * swiglu<kF32>(vg[j], vu[j]) : 0.0f;
      if constexpr (kF32) {
        *reinterpret_cast<floatx4*>(dst) = v;
      } else {
        uint2 hi, lo;
        split_bf16(v, hi, lo);
        *reinterpret_cast<uint2*>(dst) = hi;
        *reinterpret_cast<uint2*>(dst + 64) = lo;
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

// A unit: a.cols (at most 16) output columns of every token; the block's waves (and
// a.parts blocks) share the reduction. A wave adds a group's sums to its tokens' totals, which it keeps
// in LDS, experts ascending, so an expert's infinities reach its own tokens
// only; then the waves' totals are added.
// A group: ND blocks of h, for which weights are loaded once. bf16: a block is 8
// tokens with both numbers of each, so that a batch loads as much of h as of w2
// (16 tokens in two operands, with half of their columns empty in most decode
// batches, took 50 us for one token where this took 43).
template <bool kF32, int ND>
__global__ __launch_bounds__(kThreads, 3) void few_down(FewArgs a) {
  constexpr int kU = ND <= 2 ? 4 : 2;   // 64-byte k-blocks of one batch of loads
  typedef typename Elem<kF32>::type E;
  constexpr int kC = Elem<kF32>::kChunk, kB = Elem<kF32>::kBytes;
  constexpr int kParts = HPlace<kF32>::kParts, kGroup = HPlace<kF32>::kGroup;
  __shared__ Groups s;
  __shared__ uint16_t mine[kWaves][kMaxGroups];
  __shared__ int tmp[kWaves];
  __shared__ floatx4 sum[kWaves][kFewTokens][4];
  const int n_groups = find_groups<kF32, kThreads, kGroup * ND>(a.masks, a.E, s, tmp);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int tr = r / kParts, part = r % kParts;   // the lane's token of a block and number
  const int I = static_cast<int>(a.I);
  const uint32_t h_bytes = static_cast<uint32_t>(a.Ip * kB) * 16;   // of a block of h
  // The waves share every expert's reduction, or the experts (either way a token's
  // sums do not depend on the other tokens).
  // This wave's 64-byte blocks of rows of h and w2, in batches of kU: whole blocks
  // by wide loads, the last of which start early enough to end with the share;
  // then what is left of the row's end.
  const int nkb = (I * kB + 63) >> 6;
  const int nfull = (I * kB >> 6) >= kU ? I * kB >> 6 : 0;
  const bool by_expert = a.by_expert;
  const int share = by_expert ? 0 : blockIdx.y * kWaves + wave, shares = by_expert ? 1 : a.parts * kWaves;
  const int kb0 = static_cast<int>(static_cast<int64_t>(share) * nkb / shares);
  const int kb1 = static_cast<int>(static_cast<int64_t>(share + 1) * nkb / shares);
  const int kbf = max(min(kb1, nfull), kb0);
  const int nbf = (kbf - kb0 + kU - 1) / kU;
  // this wave's groups
  int n_mine = 0;
  for (int q0 = 0; q0 < n_groups; q0 += kWave) {
    const int q = q0 + lane;
    const bool in = q < n_groups && (!by_expert || s.expert[min(q, n_groups - 1)] % kWaves == wave);
    const uint64_t all = __ballot(in);
    if (in) mine[wave][n_mine + popc_below(all)] = static_cast<uint16_t>(q);
    n_mine += __popcll(all);
  }
  wave_lds_fence();
  const int items = n_mine * nbf;
  const int units = static_cast<int>((a.H + a.cols - 1) / a.cols);
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    // (a lane past the unit's last column reads that one's row)
    const int64_t col0 = static_cast<int64_t>(u) * a.cols;
    const uint32_t lr = static_cast<uint32_t>(min(static_cast<int64_t>(min(r, a.cols - 1)), a.H - 1 - col0));
    const uint32_t wo = lr * static_cast<uint32_t>(I * kB) + g * 16;
    for (int t = lane; t < a.T * 4; t += kWave) sum[wave][t >> 2][t & 3] = floatx4{0, 0, 0, 0};
    floatx4 acc[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) acc[d] = floatx4{0, 0, 0, 0};

    struct Batch {
      u32x4 w[kU], h[ND][kU];
    } b0, b1;
    auto start = [&](int b) { return min(kb0 + b * kU, max(kbf - kU, 0)); };
    auto w_at = [&](int q) {
      const int e = __builtin_amdgcn_readfirstlane(s.expert[q]);
      return static_cast<const char*>(a.w2) + (e * a.H + col0) * a.I * kB;
    };
    auto h_at = [&](int q) {
      const int block = __builtin_amdgcn_readfirstlane(s.block[q]);
      return a.h + static_cast<int64_t>(block) * h_bytes;
    };
    // the lane's column of h; past the group's last token its first one's
    auto h_off = [&](int q, int d) {
      const int n = __popcll(s.mask[q]) - s.rank[q], at = d * kGroup + tr;
      return (at < n ? d * h_bytes + r * 64 : part * 64) + g * 16;
    };
    auto load = [&](Batch& v, const Item& it) {
      const int group = mine[wave][it.q];
      const char* w0 = w_at(group);
      const char* h0 = h_at(group);
      const uint32_t k = static_cast<uint32_t>(start(it.b));
      uint32_t ho[ND];
#pragma unroll
      for (int d = 0; d < ND; ++d) ho[d] = h_off(group, d) + k * 1024;
#pragma unroll
      for (int j = 0; j < kU; ++j) {
        v.w[j] = load16_odd(w0 + (wo + k * 64) + j * 64);
#pragma unroll
        for (int d = 0; d < ND; ++d) v.h[d][j] = load16(h0 + ho[d] + j * 1024);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    // the group's sums to its tokens
    auto add = [&](int q) {
      const uint64_t mask = s.mask[q];
      const int rank = s.rank[q];
      const int n = __popcll(mask) - rank, by_rank = tokens_by_rank(mask);
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        const int at = d * kGroup + tr;
        const int t = __shfl(by_rank, min(rank + at, kWave - 1), kWave);
        if constexpr (kParts == 2) {
          // even lanes: what the second numbers, a lane on, gave. With a weight that
          // is not a number or infinite that says nothing (0 or another sign times
          // infinity), and the first numbers have given the result.
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float lo = __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(acc[d][j]), 0xf5, 15, 15, true));
            acc[d][j] += fabsf(lo) <= kMaxFloat ? lo : 0.0f;
          }
        }
        // (the token's sum so far is another lane's, of another group or the zero)
        wave_lds_fence();
        if (part == 0 && at < n) sum[wave][t][g] += acc[d];
        acc[d] = floatx4{0, 0, 0, 0};
      }
    };
    auto mma = [&](const Batch& v, Item& it) {
      // products of blocks that a batch reads again are skipped
      const int k = start(it.b), kb = kb0 + it.b * kU;
#pragma unroll
      for (int j = 0; j < kU; ++j)
        if (k + j >= kb && k + j < kbf) {
#pragma unroll
          for (int d = 0; d < ND; ++d) acc[d] = mma16<kF32>(v.w[j], v.h[d][j], acc[d]);
        }
      __builtin_amdgcn_sched_barrier(0);
      if (it.b + 1 == nbf) add(mine[wave][it.q]);
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
      for (int i = 0; i < n_mine; ++i) {
        const int q = mine[wave][i];
        const E* wrow = reinterpret_cast<const E*>(w_at(q) + lr * static_cast<uint32_t>(I * kB));
        const char* h0 = h_at(q);
        for (int kb = kbf; kb < kb1; kb += kU) {
          u32x4 w[kU];
#pragma unroll
          for (int j = 0; j < kU; ++j) {
            const int k = (kb + j) * 4 * kC + g * kC;
            const bool in = kb + j < kb1;
            w[j] = u32x4{0, 0, 0, 0};
            if (in && k < I) w[j] = load16_any<kF32>(wrow, k, I);
          }
#pragma unroll
          for (int d = 0; d < ND; ++d) {
            u32x4 h[kU];
#pragma unroll
            for (int j = 0; j < kU; ++j)
              h[j] = kb + j < kb1 ? load16(h0 + h_off(q, d) + (kb + j) * 1024) : u32x4{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < kU; ++j) acc[d] = mma16<kF32>(w[j], h[j], acc[d]);
          }
        }
        add(q);
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.T * 4; i += kThreads) {
      const int t = i >> 2, gg = i & 3;
      if (4 * gg >= a.cols) continue;
      floatx4 v = sum[0][t][gg];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v += sum[w][t][gg];
      const int64_t col = col0 + 4 * gg;
      if (a.parts == 1) {
        store4<kF32>(static_cast<E*>(a.y) + t * a.H, col, min(a.H, col0 + a.cols), (a.cols & 3) == 0, v);
      } else if (col < a.H) {   // (H is a multiple of 8)
        *reinterpret_cast<floatx4*>(a.sums + (static_cast<int64_t>(blockIdx.y) * a.T + t) * a.H + col) = v;
      }
    }
    __syncthreads();
  }
}

// y = the sum of few_down's parts, four elements a thread.
template <bool kF32>
__global__ __launch_bounds__(kThreads) void few_join(FewArgs a) {
  const int64_t n = a.T * a.H, i = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * 4;
  if (i >= n) return;
  floatx4 v = *reinterpret_cast<const floatx4*>(a.sums + i);
  for (int s = 1; s < a.parts; ++s) v += *reinterpret_cast<const floatx4*>(a.sums + s * n + i);
  store4<kF32>(static_cast<typename Elem<kF32>::type*>(a.y), i, n, true, v);
}

template <bool kF32, int ND>
hipError_t launch_down(const FewArgs& a, unsigned grid, hipStream_t st) {
  hipLaunchKernelGGL((few_down<kF32, ND>), dim3(grid, a.parts), dim3(kThreads), 0, st, a);
  return hipGetLastError();
}
template <bool kF32>
hipError_t launch_down(const FewArgs& a, double per_expert, unsigned grid, hipStream_t st) {
  constexpr int kGroup = kF32 ? 16 : 8;
  if (per_expert <= kGroup)
    return launch_down<kF32, 1>(a, grid, st);
  if (per_expert <= 2 * kGroup)
    return launch_down<kF32, 2>(a, grid, st);
  return launch_down<kF32, 4>(a, grid, st);
}

template <bool kF32>
hipError_t launch_few(const FewArgs& a, const SelectArgs* sel, double per_expert, int64_t begin, hipStream_t st) {
  const int cus = device_cu_count();
  const int64_t most = static_cast<int64_t>(a.T) * a.K < a.E ? static_cast<int64_t>(a.T) * a.K
                                                             : a.E + static_cast<int64_t>(a.T) * a.K / 16;
  const int64_t u1 = most * (a.Ip / 16), u2 = cdiv(a.H, a.cols);
  // Tokens for which weights are loaded once, by those that an expert gets on
  // average (4096 x 2048; up by 16, 32 and 64, down by 8, 16 and 32 tokens: 64
  // tokens, 8 of 8 experts 178, 122 and 98 us, 176, 124 and 100 us; 2 of 8 71, 58 and
  // 70, 61, 47 and 48; 48 tokens, 2 of 16 92, 97 and 122, 55, 60 and 81)
  // As many blocks as fit at once.
  const int nq = a.T <= 16 || per_expert <= 8 ? 1 : a.T <= 32 || per_expert <= 32 ? 2 : 4;
  const int b1 = (nq == 4 ? 2 : 3) * cus;
  const unsigned g1 = static_cast<unsigned>(u1 < b1 ? u1 : b1);
  const unsigned g2 = static_cast<unsigned>(u2 < 2 * cus ? u2 : 2 * cus);
  if (sel && sel->G <= 64)
    hipLaunchKernelGGL((few_up<kF32, 1, 1>), dim3(g1), dim3(kThreads), 0, st, a, *sel, begin);
  else if (sel)
    hipLaunchKernelGGL((few_up<kF32, 4, 1>), dim3(g1), dim3(kThreads), 0, st, a, *sel, begin);
  else if (nq == 1)
    hipLaunchKernelGGL((few_up<kF32, 0, 1>), dim3(g1), dim3(kThreads), 0, st, a, SelectArgs{}, begin);
  else if (nq == 2)
    hipLaunchKernelGGL((few_up<kF32, 0, 2>), dim3(g1), dim3(kThreads), 0, st, a, SelectArgs{}, begin);
  else
    hipLaunchKernelGGL((few_up<kF32, 0, 4>), dim3(g1), dim3(kThreads), 0, st, a, SelectArgs{}, begin);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if ((e = launch_down<kF32>(a, per_expert, g2, st)) != hipSuccess || a.parts == 1) return e;
  hipLaunchKernelGGL(few_join<kF32>, dim3(static_cast<unsigned>(cdiv(a.T * a.H, 4 * kThreads))), dim3(kThreads), 0,
                     st, a);
  return hipGetLastError();
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// few_down's units. Columns: those that leave the fullest CU the fewest (2880
// columns by 12 and not 16: 33 us instead of 35; 7168 by 14: 40 instead of 44). Parts:
// where not even half of the CUs get a unit of 16 and the split takes 192 KiB of
// weights and more from each, 8 us at what a CU reads, which pays for the launch
// that adds the parts (1024 x 2048, 8 tokens that choose 4 of 16 experts: 31 us
// whole, 13 + 4 in four parts; two experts, 128 KiB a unit: 6 whole, 5 + 2).
// Experts to the waves: rows of less than a batch of loads for each wave (64 tokens
// that choose 4 of 32, I = 128: 10 us, by shares of rows 28), or of less than two
// with experts enough to be even (8 tokens, 4 of 16, I = 800: 16 us, 19; but one
// token, 8 of 64, I = 768: 12 us, by shares 11).
struct DownShape {
  int cols, parts;
  bool by_expert;
};
DownShape down_shape(const tr_layer_desc& d) {
  const int64_t H = d.route.H, row = d.I * (d.route.dtype == TR_F32 ? 4 : 2);
  const int64_t units = cdiv(H, 16);
  DownShape s{16, 1, false};
  int64_t parts = kPlanCus / units;
  if (parts > row / 1024) parts = row / 1024;   // a batch of loads for a wave
  if (parts > 8) parts = 8;
  // bytes of weights of a unit, for the experts that the rows would choose at most,
  // were the routes uniform
  const double routes = static_cast<double>(d.route.T) * d.route.K * d.E / d.route.G;
  const double experts = routes < 1 ? 1 : routes < d.E ? routes : d.E;
  const double bytes = 16.0 * row * experts;
  if (parts > 1 && bytes * (1.0 - 1.0 / parts) >= 3 << 16) {
    s.parts = static_cast<int>(parts);
    return s;
  }
  s.by_expert = row <= 64 * 15 || (row <= 64 * 31 && experts >= 16);
  auto fullest = [&](int cols) { return cdiv(cdiv(H, cols), kPlanCus) * cols; };
  for (int cols = 14; cols >= 8; cols -= 2)
    if (fullest(cols) < fullest(s.cols)) s.cols = cols;
  return s;
}

struct FewLayout {
  size_t masks, slots, h, sums, total;
  int64_t Ip;
  DownShape down;
};
FewLayout few_layout(const tr_layer_desc& d) {
  FewLayout L{};
  L.Ip = cdiv(d.I, 32) * 32;
  size_t o = 0;
  auto take = [&](size_t n) { const size_t at = o; o = up256(o + n); return at; };
  L.masks = take(8 * static_cast<size_t>(d.E));
  L.slots = take(64 * static_cast<size_t>(d.E));
  const size_t routes = static_cast<size_t>(d.route.T) * d.route.K, E = d.E;
  const bool f32 = d.route.dtype == TR_F32;
  const size_t blocks = (routes < E ? routes : E) + routes / (f32 ? HPlace<true>::kGroup : HPlace<false>::kGroup);
  L.down = down_shape(d);
  L.sums = take(L.down.parts > 1 ? 4 * static_cast<size_t>(L.down.parts) * d.route.T * d.route.H : 0);
  L.h = take(blocks * 16 * L.Ip * (f32 ? 4 : 2));
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
  a.sums = reinterpret_cast<float*>(b + L.sums);
  a.cols = L.down.cols;
  a.parts = L.down.parts;
  a.by_expert = L.down.by_expert;
  a.y = y;
  a.T = static_cast<int>(r.T);
  a.K = r.K;
  a.E = d.E;
  a.H = r.H;
  a.I = d.I;
  a.Ip = L.Ip;
  const SelectArgs sel = select_args(r, bias, idx, w, route_ws);
  const double per_expert = static_cast<double>(r.T) * r.K / r.G;
  return f32 ? launch_few<true>(a, fused ? &sel : nullptr, per_expert, d.expert_begin, st)
             : launch_few<false>(a, fused ? &sel : nullptr, per_expert, d.expert_begin, st);
}

}  // namespace tr
