// Projections y = x W^T of rows of x: the router's logits and the projection
// that all requests share, with each token's low-rank adapter beside it.
//
//   logits[t, g] = x[t] . Wg[g]
//   y[t, n] = x[t] . W[n] + s[a] sum_j (x[t] . A[a][j]) B[a][n, j],  a = ids[t]
//
// The same code serves bf16 and fp32 (tr_chunk.h). Forms, by the number of
// tokens T:
//  - stream_partial (T <= 16): bound by reading W. Weight rows go from memory
//    straight into MFMA operands, the tokens ride in the other operand, and
//    the reduction dimension is split over the waves of a block and over
//    blocks, so that a few hundred rows still occupy every compute unit.
//  - few_linear (more, as long as tiles of 64 x 128 leave CUs without one): the
//    same split of the reduction over blocks, W and x staged through LDS, so that
//    a weight row is read for 64 tokens.
//    The sums of a block's part go to fp32 partials; the kernel that follows
//    (router selection, adapter_few) adds them in a fixed order. The adapters'
//    low-rank products x A^T are units of the same launch, and one wave of it
//    writes the table of units (a unit: up to 16 tokens of one adapter) that
//    adapter_few goes by.
//  - adapter_order, adapter_shrink, then linear_tile or adapter_tiled
//    (grouped_gemm.hip) with the adapters on top, for many tokens; the router's
//    logits of many tokens are linear_tile alone.
#include "tr_chunk.h"
#include "tr_internal.h"

namespace tr {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kU = 8;   // 64-byte k-blocks of one batch of loads

// --------------------------------------------------------------------------
// A few tokens
// --------------------------------------------------------------------------
// Up to 16 of a chunk's 64 tokens that have one adapter, or none (aid -1);
// n = 0: no unit.
struct AdapterUnit {
  int aid, n;
  int tok[16];   // in the chunk
};

struct StreamArgs {
  const char* x;         // [T, H]
  const char* w;         // [N, H]
  float* part;           // [S, T, Np] sums of each part of the reduction
  int64_t row_bytes;     // bytes of a row of x and of w
  int64_t T;
  int N, Np;
  int tiles;             // ceil(N / 16), of stream_wide ceil(N / 32)
  // adapters (NULL ids: none)
  const int32_t* ids;    // [T]
  const char* a;         // [A, R, H]
  float* vpart;          // [S, T, Rp]
  int A, R, Rp, rank_tiles;
  AdapterUnit* units;    // [chunks, n_units], for the kernel that follows
  int n_units, chunks;
  // memory that the next kernel wants zeroed
  uint32_t* zero;
  int n_zero;
};

// Lane t: the lanes with the same id as t (lanes without a token have an id
// that no token has; n: the lanes that count, rounded up to 8).
__device__ __forceinline__ uint64_t same_id(int id, int n) {
  uint64_t same = 0;
  for (int j0 = 0; j0 < n; j0 += 8) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m |= (id == __builtin_amdgcn_readlane(id, j0 + j) ? 1u : 0u) << j;
    same |= static_cast<uint64_t>(m) << j0;
  }
  return same;
}
// Lane `from`'s v, in every lane.
__device__ __forceinline__ uint64_t lane_u64(uint64_t v, int from) {
  return static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v >> 32), from))) << 32 |
         static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), from));
}
// The u-th set bit of m (the same in every lane), or -1.
__device__ __forceinline__ int nth_bit(uint64_t m, int u) {
  const uint64_t hit = __ballot(((m >> lane_id()) & 1) && popc_below(m) == u);
  return __ffsll(static_cast<unsigned long long>(hit)) - 1;
}

// One wave: the units of a chunk's tokens, one for each adapter (tokens without
// one are alike) and for every further 16 of its tokens.
__device__ __forceinline__ void make_units(const StreamArgs& p, int chunk) {
  const int lane = lane_id();
  const int64_t t0 = static_cast<int64_t>(chunk) * kFewTokens;
  const int n_tok = static_cast<int>(min(static_cast<int64_t>(kFewTokens), p.T - t0));
  int id = lane < n_tok ? p.ids[t0 + lane] : -2;
  if (lane < n_tok && (id < 0 || id >= p.A)) id = -1;
  AdapterUnit* out = p.units + static_cast<int64_t>(chunk) * p.n_units;
  const uint64_t same = same_id(id, n_tok);
  const int rank = __popcll(same & ((1ull << lane) - 1));
  uint64_t leads = __ballot(lane < n_tok && rank % 16 == 0);
  int u = 0;
  for (; leads; leads &= leads - 1, ++u) {
    const int lead = __ffsll(static_cast<unsigned long long>(leads)) - 1;
    const int first = __builtin_amdgcn_readlane(rank, lead);
    const uint64_t tokens = lane_u64(same, lead);
    const int at = popc_below(tokens) - first;
    if (((tokens >> lane) & 1) && at >= 0 && at < 16) out[u].tok[at] = lane;
    if (lane == lead) {
      out[u].aid = id;
      out[u].n = min(16, __popcll(tokens) - first);
    }
  }
  for (u += lane; u < p.n_units; u += kWave) out[u].n = 0;
}

// Unit (chunk, tile, s): 16 weight rows against the chunk's tokens (64, the last
// chunk the rest) over part s of the reduction, which its waves share. Tiles past
// the weight's are adapter tiles: unit (slot, rank tile) takes 16 rows of the
// slot-th different adapter among the tokens' ids, and keeps the sums of that
// adapter's tokens. red: LDS of kWaves * NQ * kWave floatx4.
template <bool kF32, int NQ>
__device__ __forceinline__ void stream_unit(const StreamArgs& p, int chunk, int tile, int s, int S,
                                            floatx4* red) {
  const int64_t t0 = static_cast<int64_t>(chunk) * kFewTokens;
  const int n_tok = static_cast<int>(min(static_cast<int64_t>(kFewTokens), p.T - t0));
  const char* x0 = p.x + t0 * p.row_bytes;
  const int tid = threadIdx.x;
  const int lane = tid & 63, wave = tid >> 6;
  const int g = lane >> 4, r = lane & 15;

  const bool is_w = tile < p.tiles;
  uint64_t mask = n_tok == 64 ? ~0ull : (1ull << n_tok) - 1;   // tokens of this tile
  const char* wp;
  int rt = 0;
  if (is_w) {
    wp = p.w + static_cast<int64_t>(min(tile * 16 + r, p.N - 1)) * p.row_bytes;
  } else {
    const int u = tile - p.tiles, slot = u / p.rank_tiles;
    rt = u % p.rank_tiles;
    const int id = lane < n_tok ? p.ids[t0 + lane] : -2;
    // the first tokens of the different adapters
    const uint64_t same = same_id(id, n_tok);
    const int lead = nth_bit(__ballot(id >= 0 && id < p.A && (same & ((1ull << lane) - 1)) == 0), slot);
    if (lead < 0) return;   // fewer different adapters (the same in every wave)
    const int aid = __builtin_amdgcn_readlane(id, lead);
    mask = lane_u64(same, lead);
    wp = p.a + (static_cast<int64_t>(aid) * p.R + min(rt * 16 + r, p.R - 1)) * p.row_bytes;
  }

  // The tile's tokens are its first columns. A lane past the last one reads the
  // first one's row: its sums are never stored, and the columns of an MFMA do not
  // mix.
  const int n = __popcll(mask), by_rank = tokens_by_rank(mask);
  const char* xp[NQ];
#pragma unroll
  for (int q = 0; q < NQ; ++q)
    xp[q] = x0 + __shfl(by_rank, q * 16 + r < n ? q * 16 + r : 0, kWave) * p.row_bytes + g * 16;
  wp += g * 16;

  // this wave's 64-byte blocks; the last one of a row may be short
  const int nkb = static_cast<int>((p.row_bytes + 63) >> 6);
  const int nfull = static_cast<int>(p.row_bytes >> 6);
  const int part = s * kWaves + wave, parts = S * kWaves;
  int kb = static_cast<int>(static_cast<int64_t>(part) * nkb / parts);
  const int kb1 = static_cast<int>(static_cast<int64_t>(part + 1) * nkb / parts);
  const int kbf = min(kb1, nfull);
  floatx4 acc[NQ];
#pragma unroll
  for (int q = 0; q < NQ; ++q) acc[q] = floatx4{0, 0, 0, 0};
  // Batches of kU blocks. A part's last batch may be short: its loads re-read
  // the last whole block and the products are skipped, so that it costs one
  // wait like the others and not one a block.
  for (; kb < kbf; kb += kU) {
    u32x4 wa[kU];
#pragma unroll
    for (int j = 0; j < kU; ++j) wa[j] = load16(wp + min(kb + j, kbf - 1) * 64);
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      if (q * 16 >= n) continue;
      u32x4 xb[kU];
#pragma unroll
      for (int j = 0; j < kU; ++j) xb[j] = load16(xp[q] + min(kb + j, kbf - 1) * 64);
#pragma unroll
      for (int j = 0; j < kU; ++j)
        if (kb + j < kbf) acc[q] = mma16<kF32>(wa[j], xb[j], acc[q]);
    }
  }
  if (kb1 > nfull) {   // the short block at the end of the rows
    const bool in = nfull * 64 + g * 16 < p.row_bytes;
    const u32x4 wa = in ? load16(wp + nfull * 64) : u32x4{0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      if (q * 16 >= n) continue;
      const u32x4 xb = in ? load16(xp[q] + nfull * 64) : u32x4{0, 0, 0, 0};
      acc[q] = mma16<kF32>(wa, xb, acc[q]);
    }
  }
#pragma unroll
  for (int q = 0; q < NQ; ++q) red[(wave * NQ + q) * kWave + lane] = acc[q];
  __syncthreads();
  for (int q = wave; q < NQ; q += kWaves) {
    const int t = __shfl(by_rank, q * 16 + r, kWave);
    if (q * 16 + r >= n) continue;
    floatx4 v = red[q * kWave + lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += red[(w * NQ + q) * kWave + lane];
    const int64_t row = s * p.T + t0 + t;
    float* dst = is_w ? p.part + row * p.Np + tile * 16 + 4 * g
                      : p.vpart + row * p.Rp + rt * 16 + 4 * g;
    *reinterpret_cast<floatx4*>(dst) = v;
  }
}

// Unit (tile, s) with 32 weight rows, for at most 16 tokens and long weights: x is
// loaded once for both halves, and a batch of loads is in flight while the other's
// products run. red: LDS of 2 * kWaves * kWave floatx4.
template <bool kF32>
__device__ __forceinline__ void stream_wide(const StreamArgs& p, int tile, int s, int S, floatx4* red) {
  constexpr int kW = 4;   // 64-byte blocks of a batch
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int n = static_cast<int>(p.T);
  // addresses: starts that are the same for the wave, 32-bit offsets. A lane past
  // the last row or token reads the last one's.
  const uint32_t row_bytes = static_cast<uint32_t>(p.row_bytes);
  const int row0 = tile * 32;
  const char* w0 = p.w + static_cast<int64_t>(row0) * p.row_bytes;
  uint32_t wo[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) wo[c] = static_cast<uint32_t>(min(c * 16 + r, p.N - 1 - row0)) * row_bytes + g * 16;
  const uint32_t xo = static_cast<uint32_t>(min(r, n - 1)) * row_bytes + g * 16;
  const int nkb = static_cast<int>((row_bytes + 63) >> 6), nfull = static_cast<int>(row_bytes >> 6);
  const int part = s * kWaves + wave, parts = S * kWaves;
  const int kb0 = static_cast<int>(static_cast<int64_t>(part) * nkb / parts);
  const int kb1 = static_cast<int>(static_cast<int64_t>(part + 1) * nkb / parts);
  const int kbf = min(kb1, nfull);
  floatx4 acc[2] = {floatx4{0, 0, 0, 0}, floatx4{0, 0, 0, 0}};
  struct Batch {
    u32x4 w[2][kW], x[kW];
  } b0, b1;
  // a share's last batch starts early enough to end with it; the products of
  // blocks that it reads again are skipped
  auto start = [&](int kb) { return min(kb, kbf - kW); };
  auto load = [&](Batch& b, int kb) {
    const uint32_t k = static_cast<uint32_t>(start(kb)) * 64;
#pragma unroll
    for (int j = 0; j < kW; ++j) {
#pragma unroll
      for (int c = 0; c < 2; ++c) b.w[c][j] = load16(w0 + (wo[c] + k) + j * 64);
      b.x[j] = load16(p.x + (xo + k) + j * 64);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto mma = [&](const Batch& b, int kb) {
    const int k = start(kb);
#pragma unroll
    for (int j = 0; j < kW; ++j)
      if (k + j >= kb && k + j < kbf) {
#pragma unroll
        for (int c = 0; c < 2; ++c) acc[c] = mma16<kF32>(b.w[c][j], b.x[j], acc[c]);
      }
    __builtin_amdgcn_sched_barrier(0);
  };
  // (a share has 16 whole blocks: stream_rows)
  load(b0, kb0);
  int kb = kb0;
  for (; kb + 2 * kW < kbf; kb += 2 * kW) {
    load(b1, kb + kW);
    mma(b0, kb);
    load(b0, kb + 2 * kW);
    mma(b1, kb + kW);
  }
  if (kb + kW < kbf) {
    load(b1, kb + kW);
    mma(b0, kb);
    mma(b1, kb + kW);
  } else {
    mma(b0, kb);
  }
  if (kb1 > nfull) {   // the short block at the end of the rows
    const bool in = nfull * 64u + g * 16 < row_bytes;
    const u32x4 z = {0, 0, 0, 0};
    const u32x4 xv = in ? load16(p.x + xo + nfull * 64) : z;
#pragma unroll
    for (int c = 0; c < 2; ++c) acc[c] = mma16<kF32>(in ? load16(w0 + wo[c] + nfull * 64) : z, xv, acc[c]);
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) red[(wave * 2 + c) * kWave + lane] = acc[c];
  __syncthreads();
  const int col = row0 + wave * 16 + 4 * g;   // wave c: half c
  if (wave < 2 && r < n && col < p.Np) {
    floatx4 v = red[wave * kWave + lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += red[(w * 2 + wave) * kWave + lane];
    *reinterpret_cast<floatx4*>(p.part + (static_cast<int64_t>(s) * p.T + r) * p.Np + col) = v;
  }
}

struct ExpandArgs {
  const float* part;     // [S, T, Np]
  const float* vpart;    // [S, T, Rp]
  const AdapterUnit* units;   // [chunks, n_units]
  const float* scales;   // [A] or NULL
  const void* b;         // [A, N, R]
  void* y;               // [T, N]
  int64_t T;
  int S, N, Np, A, R, Rp, n_units;
};

// y[t, n] = the sum of the parts + s[a] sum_j v[t, j] B[a][n, j]. One block:
// 128 columns of one unit's tokens, 32 columns a wave. Rows of B are one MFMA
// operand, read whole and once for all of the unit's tokens, the low-rank sums
// the other: for bf16 as two bf16 numbers each (16 significant bits), so that y
// is rounded once. Bound by latency: the loads of B (kKb blocks of it at a time),
// of the parts (kParts at a time) and of the low-rank sums go out together.
// (Sums with the second numbers in accumulators of their own, dropped where they
// are not finite, took 1.7 us more than finite_bf16's 0.3 us for 64 x 7168 x 7168
// with 24 adapters of rank 64.)
template <bool kF32, int kKb, int kParts>
__global__ __launch_bounds__(kThreads) void adapter_few(ExpandArgs p) {
  typedef typename Elem<kF32>::type E;
  constexpr int kC = Elem<kF32>::kChunk;
  constexpr int kV = kF32 ? 1 : 2;       // numbers that make up a low-rank sum
  constexpr int kTok = 16, kNs = 2;
  constexpr int kPitch = kMaxRank + kC;  // (a pad: rows in other banks)
  __shared__ E v_s[kV][kTok][kPitch];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, r = lane & 15;
  const int64_t t0 = static_cast<int64_t>(blockIdx.z) * kFewTokens;
  const AdapterUnit* unit = p.units + static_cast<int64_t>(blockIdx.z) * p.n_units + blockIdx.y;
  const int aid = unit->aid, n = unit->n;
  if (n == 0) return;   // fewer units
  const int64_t t = t0 + unit->tok[min(r, n - 1)];   // this lane's token
  const bool has = aid >= 0;   // the same for the whole block
  const int col0 = (blockIdx.x * kWaves + wave) * 16 * kNs;

  // rows of B: lane r's column of each 16, chunk g of a k-block
  const E* row[kNs];
#pragma unroll
  for (int j = 0; j < kNs; ++j)
    row[j] = static_cast<const E*>(p.b) +
             (static_cast<int64_t>(max(aid, 0)) * p.N + min(col0 + j * 16 + r, p.N - 1)) * p.R;
  const bool vec = (p.R % kC) == 0;
  auto b_chunk = [&](int j, int kb) -> u32x4 {
    const int k = kb * 4 * kC + g * kC;
    if (k >= p.R) return u32x4{0, 0, 0, 0};
    return vec ? load16(reinterpret_cast<const char*>(row[j] + k)) : load16_any<kF32>(row[j], k, p.R);
  };
  u32x4 bv[kKb][kNs];
  if (has) {
#pragma unroll
    for (int kb = 0; kb < kKb; ++kb)
#pragma unroll
      for (int j = 0; j < kNs; ++j) bv[kb][j] = b_chunk(j, kb);
  }
  // The parts' sums, eight parts' loads at a time (the last is read again), and
  // this thread's first low-rank sum: all of these loads go out together.
  const int Rk = (p.R + 4 * kC - 1) / (4 * kC) * (4 * kC);   // v_s: zero from R to Rk
  const float sc = has && p.scales ? p.scales[aid] : 1.0f;
  const int n_v = has ? n * Rk : 0;
  auto v_at = [&](int i) {
    const int k = i / Rk, j = i - k * Rk;
    return p.vpart + (t0 + unit->tok[min(k, n - 1)]) * p.Rp + min(j, p.R - 1);
  };
  floatx4 acc[kNs];
#pragma unroll
  for (int j = 0; j < kNs; ++j) acc[j] = floatx4{0, 0, 0, 0};
  floatx4 f[kParts][kNs];
  auto load_parts = [&](int s0) {
#pragma unroll
    for (int i = 0; i < kParts; ++i)
#pragma unroll
      for (int j = 0; j < kNs; ++j)
        f[i][j] = *reinterpret_cast<const floatx4*>(
            p.part + (min(s0 + i, p.S - 1) * p.T + t) * p.Np + min(col0 + j * 16, p.Np - 16) + 4 * g);
  };
  auto add_parts = [&](int s0) {
#pragma unroll
    for (int i = 0; i < kParts; ++i)
      if (s0 + i < p.S) {
#pragma unroll
        for (int j = 0; j < kNs; ++j) acc[j] += f[i][j];
      }
  };
  float fv[kParts];
  auto load_v = [&](const float* v, int s0) {
#pragma unroll
    for (int q = 0; q < kParts; ++q) fv[q] = v[min(s0 + q, p.S - 1) * p.T * p.Rp];
  };
  const float* v0 = p.vpart;
  load_parts(0);
  if (has) {
    v0 = v_at(min(static_cast<int>(threadIdx.x), n_v - 1));
    load_v(v0, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
  add_parts(0);
  for (int s0 = kParts; s0 < p.S; s0 += kParts) {
    load_parts(s0);
    add_parts(s0);
  }
  if (has) {
    for (int i = threadIdx.x; i < n_v; i += kThreads) {
      if (i >= kThreads) {
        v0 = v_at(i);
        load_v(v0, 0);
      }
      float total = 0.0f;
      for (int s0 = 0; s0 < p.S; s0 += kParts) {
        if (s0 > 0) load_v(v0, s0);
#pragma unroll
        for (int q = 0; q < kParts; ++q)
          if (s0 + q < p.S) total += fv[q];
      }
      const int k = i / Rk, j = i - k * Rk;
      total = j < p.R ? total * sc : 0.0f;
      if constexpr (kF32) {
        v_s[0][k][j] = total;
      } else {
        const uint32_t hi = cvt_bf16x2(first_bf16(total), 0.0f) & 0xffffu;
        v_s[0][k][j] = static_cast<uint16_t>(hi);
        v_s[1][k][j] =
            static_cast<uint16_t>(cvt_bf16x2(second_bf16(total, bf16_bits_to_f32(hi)), 0.0f) & 0xffffu);
      }
    }
    __syncthreads();
    for (int kb0 = 0; kb0 < Rk / (4 * kC); kb0 += kKb) {
#pragma unroll
      for (int kb = 0; kb < kKb; ++kb) {
        if ((kb0 + kb) * 4 * kC >= Rk) continue;
#pragma unroll
        for (int q = 0; q < kV; ++q) {
          const u32x4 vv = *reinterpret_cast<const u32x4*>(&v_s[q][r][(kb0 + kb) * 4 * kC + g * kC]);
#pragma unroll
          for (int j = 0; j < kNs; ++j)
            acc[j] = mma16<kF32>(q == 0 ? bv[kb][j] : finite_bf16(bv[kb][j]), vv, acc[j]);
        }
      }
      if ((kb0 + kKb) * 4 * kC < Rk) {
#pragma unroll
        for (int kb = 0; kb < kKb; ++kb)
#pragma unroll
          for (int j = 0; j < kNs; ++j) bv[kb][j] = b_chunk(j, kb0 + kKb + kb);
      }
    }
  }
  if (r >= n) return;
#pragma unroll
  for (int j = 0; j < kNs; ++j) {
    const int col = col0 + j * 16 + 4 * g;
    if (col < p.N) store4<kF32>(static_cast<E*>(p.y) + t * p.N, col, p.N, (p.N & 3) == 0, acc[j]);
  }
}

// --------------------------------------------------------------------------
// Many tokens: their order by adapter
// --------------------------------------------------------------------------
// Positions of each window of 2048 tokens in the order of their adapters, tokens
// without one last: perm[pos] is the token, sid[pos] its adapter (or -1). The
// kernels that follow work on positions, so that a group of 16 or 32 has one
// adapter or two however the requests' tokens are mixed (8192 x 7168 x 7168 with
// 32 adapters of rank 64 dealt at random take 826 + 2277 us in the tokens' order,
// and 5 + 106 + 870 to 910 us so). A window whose tokens already come in runs keeps
// its order.
// Counting in LDS: a thread's token takes its place among its adapter's by an
// atomic add, whose order varies and does not matter, as a row's sums do not
// depend on its place. More than kBins adapters share bins with their neighbours.
// (A bitonic sort of the same window took 15 us.)
constexpr int kWindow = 2048;
constexpr int kOrderThreads = kWindow / 2;
constexpr int kBins = kOrderThreads - 1;   // and one for tokens without an adapter

__global__ __launch_bounds__(kOrderThreads) void adapter_order(const int32_t* __restrict__ ids,
                                                               int64_t T, int A, int32_t* perm,
                                                               int32_t* sid) {
  __shared__ int bins[kOrderThreads];
  __shared__ int tmp[kOrderThreads / kWave];
  const int tid = threadIdx.x;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kWindow;
  const int n = static_cast<int>(min(static_cast<int64_t>(kWindow), T - t0));
  int id[2], bin[2], at[2];
  int ends = 0, all = 0;   // tokens whose adapter differs from the one's before
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int i = tid + q * kOrderThreads;
    id[q] = -1;
    bin[q] = kBins;
    if (i < n) {
      id[q] = ids[t0 + i];
      ends += id[q] != ids[t0 + max(i - 1, 0)];
      if (id[q] < 0 || id[q] >= A) id[q] = -1;
      else bin[q] = A <= kBins ? id[q] : static_cast<int>(static_cast<int64_t>(id[q]) * kBins / A);
    }
    at[q] = i;
  }
  bins[tid] = 0;
  block_exclusive_scan<kOrderThreads>(ends, tmp, &all);   // (with a barrier)
  // runs of fewer than 32 tokens on average (the same in every thread)
  if (all * 32 > n) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (tid + q * kOrderThreads < n) at[q] = atomicAdd(&bins[bin[q]], 1);
    __syncthreads();
    const int count = bins[tid];
    bins[tid] = block_exclusive_scan<kOrderThreads>(count, tmp, &all);
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q) at[q] += bins[bin[q]];
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int i = tid + q * kOrderThreads;
    if (i >= n) continue;
    perm[t0 + at[q]] = static_cast<int32_t>(t0 + i);
    sid[t0 + at[q]] = id[q];
  }
}

// --------------------------------------------------------------------------
// Many tokens: the adapters' low-rank products
// --------------------------------------------------------------------------
struct ShrinkArgs {
  const char* x;
  const char* a;
  const int32_t* ids;    // by position
  const int32_t* perm;   // the positions' tokens, or NULL: the same
  const float* scales;
  void* v;               // [T, parts, Rq], zero past R: fp32, or two bf16 numbers
  int64_t row_bytes;
  int64_t T;
  int A, R, Rq;
};

// v[t, j] = s[a] x[t] . A[a][j] for a group of 16 kNG tokens: 16 kRT rows of A at
// a time, the waves sharing the reduction, two batches of loads in flight.
// Bound by x from memory and A from L2: 39 us for 8192 x 7168 and rank 32 with x
// in the last-level cache, 63 us with x from memory (16 tokens a group, which read A
// twice as often, took 58 us where this takes 39, of which 41 us were A's loads
// alone; x alone takes 25 us). The different adapters among the tokens
// (one where tokens of a request are neighbours) are dealt to kSlots blocks, so
// that a group at the border of two requests takes no longer than the others. v
// is kept as the tiles multiply it: fp32, or two bf16 numbers with 16 significant
// bits, so that a row is the same however many rows share its call.
template <bool kF32>
constexpr int kVParts = kF32 ? 1 : 2;   // numbers that make up an element of v
constexpr int kSlots = 2;
constexpr int kShrinkThreads = 384;   // two blocks a CU
constexpr int kShrinkWaves = kShrinkThreads / kWave;

template <bool kF32, int kRT, int kNG>
__global__ __launch_bounds__(kShrinkThreads, 3) void adapter_shrink(ShrinkArgs p) {
  typedef typename Elem<kF32>::type E;
  // 64-byte blocks of a batch (kRT = kNG = 2: by 4, which spill, 42 us; by 2 50 us;
  // by 3 39 us, with one register spilled, three in fp32)
  constexpr int kB = kRT + kNG == 4 ? 3 : 4;
  __shared__ floatx4 red[kShrinkWaves][kRT][kNG][kWave];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * 16 * kNG;
  const bool in = lane < 16 * kNG && t0 + lane < p.T;
  const int id = in ? p.ids[t0 + lane] : -1;
  uint32_t todo = static_cast<uint32_t>(__ballot(id >= 0 && id < p.A));
  // rows of x by 32-bit offsets: from the group's first token, or with perm from
  // the first of all (x is below 2 GiB then)
  const char* x0 = p.perm ? p.x : p.x + t0 * p.row_bytes;
  const int row = p.perm ? (in ? p.perm[t0 + lane] : 0) : lane;
  const uint32_t row_bytes = static_cast<uint32_t>(p.row_bytes);
  const int nkb = static_cast<int>((row_bytes + 63) >> 6);
  const int nfull = static_cast<int>(row_bytes >> 6);
  const int kb0 = wave * nkb / kShrinkWaves, kb1 = (wave + 1) * nkb / kShrinkWaves;
  const int kbf = min(kb1, nfull);
  for (int slot = 0; todo; ++slot) {
    const int first = __ffs(todo) - 1;
    const int aid = __builtin_amdgcn_readlane(id, first);
    const uint32_t mask = static_cast<uint32_t>(__ballot(id == aid));
    todo &= ~mask;
    if (slot % kSlots != static_cast<int>(blockIdx.y)) continue;
    // a token of another adapter reads the first one's row: not stored
    uint32_t xo[kNG];
#pragma unroll
    for (int q = 0; q < kNG; ++q)
      xo[q] = __shfl(row, (mask >> (16 * q + r)) & 1 ? 16 * q + r : first, kWave) * row_bytes + g * 16;
    const float sc = p.scales ? p.scales[aid] : 1.0f;
    for (int j0 = blockIdx.z * 16 * kRT; j0 < p.R; j0 += gridDim.z * 16 * kRT) {
      // rows past R read the last one: zeros are stored for them
      const int base = min(j0, p.R - 1);
      const char* a0 = p.a + (static_cast<int64_t>(aid) * p.R + base) * p.row_bytes;
      uint32_t ao[kRT];
#pragma unroll
      for (int c = 0; c < kRT; ++c) ao[c] = min(c * 16 + r, p.R - 1 - base) * row_bytes + g * 16;
      floatx4 acc[kRT][kNG];
#pragma unroll
      for (int c = 0; c < kRT; ++c)
#pragma unroll
        for (int q = 0; q < kNG; ++q) acc[c][q] = floatx4{0, 0, 0, 0};
      struct Batch {
        u32x4 x[kNG][kB], a[kRT][kB];
      } b0, b1;
      // a share's last batch starts early enough to end with it; the products of
      // blocks that it reads again are skipped
      auto start = [&](int kb) { return min(kb, max(kbf - kB, 0)); };
      auto load = [&](Batch& b, int kb) {
        const uint32_t k = static_cast<uint32_t>(start(kb)) * 64;
#pragma unroll
        for (int j = 0; j < kB; ++j) {
#pragma unroll
          for (int q = 0; q < kNG; ++q) b.x[q][j] = load16(x0 + (xo[q] + k) + j * 64);
#pragma unroll
          for (int c = 0; c < kRT; ++c) b.a[c][j] = load16(a0 + (ao[c] + k) + j * 64);
        }
        __builtin_amdgcn_sched_barrier(0);
      };
      auto mma = [&](const Batch& b, int kb) {
        const int k = start(kb);
#pragma unroll
        for (int j = 0; j < kB; ++j)
          if (k + j >= kb && k + j < kbf) {
#pragma unroll
            for (int c = 0; c < kRT; ++c)
#pragma unroll
              for (int q = 0; q < kNG; ++q) acc[c][q] = mma16<kF32>(b.a[c][j], b.x[q][j], acc[c][q]);
          }
        __builtin_amdgcn_sched_barrier(0);
      };
      if (nfull >= kB) {
        if (kb0 < kbf) {
          load(b0, kb0);
          int kb = kb0;
          for (; kb + 2 * kB < kbf; kb += 2 * kB) {
            load(b1, kb + kB);
            mma(b0, kb);
            load(b0, kb + 2 * kB);
            mma(b1, kb + kB);
          }
          if (kb + kB < kbf) {
            load(b1, kb + kB);
            mma(b0, kb);
            mma(b1, kb + kB);
          } else {
            mma(b0, kb);
          }
        }
      } else {   // rows of fewer blocks than a batch has
        for (int kb = kb0; kb < kbf; ++kb)
#pragma unroll
          for (int q = 0; q < kNG; ++q) {
            const u32x4 xv = load16(x0 + xo[q] + kb * 64);
#pragma unroll
            for (int c = 0; c < kRT; ++c)
              acc[c][q] = mma16<kF32>(load16(a0 + ao[c] + kb * 64), xv, acc[c][q]);
          }
      }
      if (kb1 > nfull) {   // the short block at the end of the rows
        const bool in = nfull * 64u + g * 16 < row_bytes;
#pragma unroll
        for (int q = 0; q < kNG; ++q) {
          const u32x4 xv = in ? load16(x0 + xo[q] + nfull * 64) : u32x4{0, 0, 0, 0};
#pragma unroll
          for (int c = 0; c < kRT; ++c)
            acc[c][q] = mma16<kF32>(in ? load16(a0 + ao[c] + nfull * 64) : u32x4{0, 0, 0, 0}, xv, acc[c][q]);
        }
      }
#pragma unroll
      for (int c = 0; c < kRT; ++c)
#pragma unroll
        for (int q = 0; q < kNG; ++q) red[wave][c][q][lane] = acc[c][q];
      __syncthreads();
      // wave c + kRT q: rank tile c of token group q
      const int c = wave % kRT, q = wave / kRT;
      const int col = j0 + c * 16 + 4 * g;
      if (q < kNG && ((mask >> (16 * q + r)) & 1) && col < p.Rq) {
        floatx4 v = red[0][c][q][lane];
#pragma unroll
        for (int w = 1; w < kShrinkWaves; ++w) v += red[w][c][q][lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = col + i < p.R ? v[i] * sc : 0.0f;
        E* out = static_cast<E*>(p.v) + (t0 + 16 * q + r) * kVParts<kF32> * p.Rq + col;
        if constexpr (kF32) {
          *reinterpret_cast<floatx4*>(out) = v;
        } else {
          uint2 hi, lo;
          split_bf16(v, hi, lo);
          *reinterpret_cast<uint2*>(out) = hi;
          *reinterpret_cast<uint2*>(out + p.Rq) = lo;
          // (one tile of two that an MFMA takes: zeros in the other's place)
          if (kRT == 1 && col + 16 < p.Rq)
            *reinterpret_cast<uint2*>(out + 16) = *reinterpret_cast<uint2*>(out + p.Rq + 16) = uint2{0, 0};
        }
      }
      __syncthreads();
    }
  }
}

template <bool kF32, int kRT, int kNG>
hipError_t launch_shrink(const ShrinkArgs& s, int64_t passes, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(cdiv(s.T, 16 * kNG)), kSlots, static_cast<unsigned>(passes));
  hipLaunchKernelGGL((adapter_shrink<kF32, kRT, kNG>), grid, dim3(kShrinkThreads), 0, st, s);
  return hipGetLastError();
}
// Groups of 16 tokens where their blocks fit the CUs once (1000 x 4096, rank 16: 10 us
// and not 14; 3500 x 7168, rank 32, one request: 25 and not 33, but with eleven borders
// of requests, whose second blocks share CUs, 41 and not 33; 4000 x 4096, rank 16: 20
// and not 17). Ranks past 32: a block for every 32 (2048 x 7168, rank 64: 33 us; one
// block for both 58).
template <bool kF32>
hipError_t launch_shrink(const ShrinkArgs& s, hipStream_t st) {
  const int64_t passes = cdiv(s.R, 32);
  const bool few = cdiv(s.T, 16) * passes * 8 <= kPlanCus * 7;
  if (s.R <= 16) return few ? launch_shrink<kF32, 1, 1>(s, 1, st) : launch_shrink<kF32, 1, 2>(s, 1, st);
  return few ? launch_shrink<kF32, 2, 1>(s, passes, st) : launch_shrink<kF32, 2, 2>(s, passes, st);
}

// --------------------------------------------------------------------------
// Tiles staged through LDS
// --------------------------------------------------------------------------
constexpr int kLine = 8;                      // 16-byte chunks of a k-tile's row
constexpr int kBufferFlags = 0x00020000;      // raw buffer, 32-bit data format
constexpr uint32_t kPast = 0x80000000u;       // an offset past every buffer here

struct TileArgs {
  const char* x;         // [T, H]
  const char* w;         // [N, H]
  int64_t row_bytes;
  int64_t T;
  int N;
  int m_tiles, n_tiles, parts;
  float* part;           // [parts, T, Np] fp32 sums, or NULL: y
  int Np;
  void* y;               // [T, N]
  const int32_t* ids;    // adapters by position (NULL: none)
  const int32_t* perm;   // the positions' tokens, or NULL: the same
  const void* v;         // [T, parts, Rq], by position (ShrinkArgs)
  const void* b;         // [A, N, R]
  int A, R, Rq;
};

// A tile's shape: WM x WN waves of MS x NS blocks of 16 x 16, kStages k-tiles
// of 128 bytes a row in LDS.
template <int WM, int WN, int MS, int NS, int kStages_>
struct Shape {
  static constexpr int kWm = WM, kWn = WN, kMs = MS, kNs = NS, kStages = kStages_;
  static constexpr int kM = 16 * WM * MS, kN = 16 * WN * NS;
  static constexpr int kBlock = WM * WN * kWave;
  // 1 KiB pieces (8 rows) of a stage that a wave loads
  static constexpr int kXp = kM / 8 / (WM * WN), kWp = kN / 8 / (WM * WN);
  static_assert(kXp * 8 * WM * WN == kM && kWp * 8 * WM * WN == kN, "whole pieces a wave");
  static_assert((kStages - 1) * (kXp + kWp) <= 63, "vmcnt range");
};

typedef __attribute__((address_space(3))) void lds_ptr;

#if defined(__HIP_DEVICE_COMPILE__)
// Stage S's token half and weight half: distinct objects, so that reads of one
// are not taken to wait for DMA into another.
template <typename C, int S>
__device__ __forceinline__ u32x4* stage_x() {
  __shared__ u32x4 lds[C::kM * kLine];
  return lds;
}
template <typename C, int S>
__device__ __forceinline__ u32x4* stage_w() {
  __shared__ u32x4 lds[C::kN * kLine];
  return lds;
}

template <typename C>
struct TileLoad {
  __amdgpu_buffer_rsrc_t xr, wr;
  uint32_t xo[C::kXp], wo[C::kWp];   // this lane's byte offsets in its pieces; kPast: zeros
  uint32_t xc[C::kXp], wc[C::kWp];   // its byte in the k-tile's row
  uint32_t row_bytes;
};

// k-tile kt into stage S. Row i of a stage keeps its chunk c at c ^ ((i >> 1) & 7):
// the 16 lanes that LDS serves at a time, rows 0-3 and 12-15 of one chunk and 4-11
// of the next, lie in different banks (no conflict counted; c ^ (i & 7) ^ ((i >> 3)
// & 1) had two lanes in each, and twice the LDS cycles). Rows past T or N, bytes
// past the row and k-tiles from k1 on are given an offset past the buffer, whose
// DMA writes zeros.
template <typename C, int S>
__device__ __forceinline__ void tile_dma(const TileLoad<C>& l, int wave, int kt, int k1) {
  const uint32_t k = kt < k1 ? static_cast<uint32_t>(kt) * 128 : l.row_bytes;
#pragma unroll
  for (int j = 0; j < C::kXp; ++j)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        l.xr, (lds_ptr*)(stage_x<C, S>() + (wave * C::kXp + j) * 8 * kLine), 16,
        k + l.xc[j] < l.row_bytes ? l.xo[j] + k : kPast, 0, 0, 0);
#pragma unroll
  for (int j = 0; j < C::kWp; ++j)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        l.wr, (lds_ptr*)(stage_w<C, S>() + (wave * C::kWp + j) * 8 * kLine), 16,
        k + l.wc[j] < l.row_bytes ? l.wo[j] + k : kPast, 0, 0, 0);
}

// A wave's fragments of half of a k-tile (64 bytes of every row).
template <typename C>
struct Frags {
  u32x4 x[C::kMs], w[C::kNs];
};
template <typename C, int S>
__device__ __forceinline__ void tile_read(Frags<C>& f, int wm, int wn, int frag) {
#pragma unroll
  for (int i = 0; i < C::kMs; ++i) f.x[i] = stage_x<C, S>()[(wm * C::kMs + i) * 16 * kLine + frag];
#pragma unroll
  for (int j = 0; j < C::kNs; ++j) f.w[j] = stage_w<C, S>()[(wn * C::kNs + j) * 16 * kLine + frag];
  __builtin_amdgcn_sched_barrier(0);
}
template <bool kF32, typename C>
__device__ __forceinline__ void tile_mma(const Frags<C>& f, floatx4 (&acc)[C::kMs][C::kNs]) {
#pragma unroll
  for (int i = 0; i < C::kMs; ++i)
#pragma unroll
    for (int j = 0; j < C::kNs; ++j) acc[i][j] = mma16<kF32>(f.w[j], f.x[i], acc[i][j]);
  __builtin_amdgcn_sched_barrier(0);
}
// At most n DMA of this wave in flight, its LDS reads done; then every wave.
template <int n>
__device__ __forceinline__ void tile_wait() {
  // s_waitcnt: vmcnt(n), lgkmcnt(0), no wait for exports
  __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | 0x70);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Step kt of the ring (stage S), its first half's fragments in f0. Fragments
// are read half a k-tile ahead of their products, so that the LDS reads of all
// waves run beside products and not before them. After the barrier in the
// middle k-tile kt + 1 has landed (the DMA of the kStages - 2 after it may be in
// flight) and every wave has read all of k-tile kt, whose stage takes k-tile
// kt + kStages.
template <bool kF32, typename C, int S>
__device__ __forceinline__ void tile_step(const TileLoad<C>& l, int wave, int wm, int wn, int kt,
                                          int k1, const int (&frag)[2], Frags<C>& f0,
                                          floatx4 (&acc)[C::kMs][C::kNs]) {
  Frags<C> f1;
  tile_read<C, S>(f1, wm, wn, frag[1]);
  tile_mma<kF32, C>(f0, acc);
  tile_wait<(C::kStages - 2) * (C::kXp + C::kWp)>();
  tile_read<C, (S + 1) % C::kStages>(f0, wm, wn, frag[0]);
  tile_dma<C, S>(l, wave, kt + C::kStages, k1);
  __builtin_amdgcn_sched_barrier(0);
  tile_mma<kF32, C>(f1, acc);
}

// Block `block` of m_tiles x n_tiles x parts: a tile over one part of the
// reduction.
template <bool kF32, typename C, bool kAdapt>
__device__ __forceinline__ void tile_unit(const TileArgs& p, int block) {
  typedef typename Elem<kF32>::type E;
  constexpr int kC = Elem<kF32>::kChunk;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::kWn, wn = wave % C::kWn;
  const int g = lane >> 4, r = lane & 15;

  const int total = p.m_tiles * p.n_tiles;
  const int s = block / total, pos = block % total;
  // groups of 1024 tokens, token tiles fastest: the tiles that an XCD runs at a
  // time share rows of both operands in its L2
  constexpr int kGroup = 1024 / C::kM;
  const int group = pos / (kGroup * p.n_tiles), in = pos - group * kGroup * p.n_tiles;
  const int gm = min(kGroup, p.m_tiles - group * kGroup);
  const int mt = group * kGroup + in % gm, nt = in / gm;
  const int64_t t0 = static_cast<int64_t>(mt) * C::kM;
  const int n0 = nt * C::kN;
  const int rows = static_cast<int>(min(static_cast<int64_t>(C::kM), p.T - t0));
  const int cols = min(C::kN, p.N - n0);

  const int nkt = static_cast<int>((p.row_bytes + 127) >> 7);
  const int k0 = static_cast<int>(static_cast<int64_t>(s) * nkt / p.parts);
  const int k1 = static_cast<int>(static_cast<int64_t>(s + 1) * nkt / p.parts);

  TileLoad<C> l;
  l.row_bytes = static_cast<uint32_t>(p.row_bytes);
  // at most 128 (256) rows of 2^24 (2^23) bytes: within the 2^31 that an offset
  // reaches
  const bool moved = kAdapt && p.perm != nullptr;   // (x is below 2 GiB then)
  l.xr = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<char*>(moved ? p.x : p.x + t0 * p.row_bytes), 0,
      static_cast<int>((moved ? static_cast<uint32_t>(p.T) : rows) * l.row_bytes), kBufferFlags);
  l.wr = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<char*>(p.w + static_cast<int64_t>(n0) * p.row_bytes), 0,
      static_cast<int>(cols * l.row_bytes), kBufferFlags);
#pragma unroll
  for (int j = 0; j < C::kXp; ++j) {
    const int pc = wave * C::kXp + j, row = pc * 8 + (lane >> 3);
    l.xc[j] = ((lane & 7) ^ ((pc & 1) * 4 + (lane >> 4))) * 16;
    l.xo[j] = kPast;
    if (row < rows) l.xo[j] = (moved ? p.perm[t0 + row] : row) * l.row_bytes + l.xc[j];
  }
#pragma unroll
  for (int j = 0; j < C::kWp; ++j) {
    const int pc = wave * C::kWp + j, row = pc * 8 + (lane >> 3);
    l.wc[j] = ((lane & 7) ^ ((pc & 1) * 4 + (lane >> 4))) * 16;
    l.wo[j] = row < cols ? row * l.row_bytes + l.wc[j] : kPast;
  }
  int frag[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) frag[q] = r * kLine + ((4 * q + g) ^ (r >> 1));

  floatx4 acc[C::kMs][C::kNs];
#pragma unroll
  for (int i = 0; i < C::kMs; ++i)
#pragma unroll
    for (int j = 0; j < C::kNs; ++j) acc[i][j] = floatx4{0, 0, 0, 0};

  tile_dma<C, 0>(l, wave, k0, k1);
  tile_dma<C, 1>(l, wave, k0 + 1, k1);
  if constexpr (C::kStages > 2) tile_dma<C, 2>(l, wave, k0 + 2, k1);
  if constexpr (C::kStages > 3) tile_dma<C, 3>(l, wave, k0 + 3, k1);
  tile_wait<(C::kStages - 1) * (C::kXp + C::kWp)>();
  Frags<C> f0;
  tile_read<C, 0>(f0, wm, wn, frag[0]);
  // (whole turns of the ring in a loop without conditions, then the rest: a
  // step that may not have run would make the compiler wait for every DMA)
  int kt = k0;
  for (; kt + C::kStages <= k1; kt += C::kStages) {
    tile_step<kF32, C, 0>(l, wave, wm, wn, kt, k1, frag, f0, acc);
    tile_step<kF32, C, 1>(l, wave, wm, wn, kt + 1, k1, frag, f0, acc);
    if constexpr (C::kStages > 2) tile_step<kF32, C, 2>(l, wave, wm, wn, kt + 2, k1, frag, f0, acc);
    if constexpr (C::kStages > 3) tile_step<kF32, C, 3>(l, wave, wm, wn, kt + 3, k1, frag, f0, acc);
  }
  if (kt < k1) {
    tile_step<kF32, C, 0>(l, wave, wm, wn, kt, k1, frag, f0, acc);
    if constexpr (C::kStages > 2)
      if (kt + 1 < k1) {
        tile_step<kF32, C, 1>(l, wave, wm, wn, kt + 1, k1, frag, f0, acc);
        if constexpr (C::kStages > 3)
          if (kt + 2 < k1) tile_step<kF32, C, 2>(l, wave, wm, wn, kt + 2, k1, frag, f0, acc);
      }
  }
  __builtin_amdgcn_s_waitcnt(0x0070);   // the DMA past the last k-tile

  // lane (g, r): columns n0 + 16 (wn NS + j) + 4 g .. + 3 of token 16 (wm MS + i) + r
#pragma unroll
  for (int i = 0; i < C::kMs; ++i) {
    const int lt0 = (wm * C::kMs + i) * 16;
    const int64_t t = t0 + lt0 + r;
    if constexpr (kAdapt) {
      const int id = lt0 + r < rows ? p.ids[t] : -1;
      uint32_t todo = static_cast<uint32_t>(__ballot(id >= 0 && id < p.A)) & 0xffffu;
      const bool vec = (p.R % kC) == 0;
      while (todo) {
        const int lead = __ffs(todo) - 1;
        const int aid = __builtin_amdgcn_readlane(id, lead);
        const bool mine = id == aid;
        todo &= ~static_cast<uint32_t>(__ballot(mine));
        const E* vrow = static_cast<const E*>(p.v) + (mine ? t : t0 + lt0 + lead) * kVParts<kF32> * p.Rq;
        floatx4 d[C::kNs];
#pragma unroll
        for (int j = 0; j < C::kNs; ++j) d[j] = floatx4{0, 0, 0, 0};
        for (int j0 = 0; j0 < p.R; j0 += 4 * kC) {
          const int k = j0 + g * kC;
          const u32x4 fv = load16(reinterpret_cast<const char*>(vrow + k));
          u32x4 fl = {0, 0, 0, 0};
          if constexpr (!kF32) fl = load16(reinterpret_cast<const char*>(vrow + p.Rq + k));
#pragma unroll
          for (int j = 0; j < C::kNs; ++j) {
            const int n = min(n0 + (wn * C::kNs + j) * 16 + r, p.N - 1);
            const E* row = static_cast<const E*>(p.b) + (static_cast<int64_t>(aid) * p.N + n) * p.R;
            u32x4 fb = {0, 0, 0, 0};
            if (k < p.R)
              fb = vec ? load16(reinterpret_cast<const char*>(row + k)) : load16_any<kF32>(row, k, p.R);
            d[j] = mma16<kF32>(fb, fv, d[j]);
            if constexpr (!kF32) d[j] = mma16<kF32>(finite_bf16(fb), fl, d[j]);
          }
        }
        // added to its own tokens only: an adapter's infinities reach no other
        if (mine) {
#pragma unroll
          for (int j = 0; j < C::kNs; ++j) acc[i][j] += d[j];
        }
      }
    }
    if (lt0 + r >= rows) continue;
    const int64_t out = moved ? p.perm[t] : t;
#pragma unroll
    for (int j = 0; j < C::kNs; ++j) {
      const int n = n0 + (wn * C::kNs + j) * 16 + 4 * g;
      if (n >= p.N) continue;
      if constexpr (kAdapt)
        store4<kF32>(static_cast<E*>(p.y) + out * p.N, n, p.N, (p.N & 3) == 0, acc[i][j]);
      else
        *reinterpret_cast<floatx4*>(p.part + (s * p.T + out) * p.Np + n) = acc[i][j];
    }
  }
}
#endif  // __HIP_DEVICE_COMPILE__

// Bound by the loop's loads, LDS reads and products together, and with one tile a
// CU by what nothing covers, its first loads and its stores. bf16: 16384 x 7168 x
// 256 in two parts 69 us, 0.87 PFLOP/s; 8192 x 7160 x 7000 with adapters 1040 us,
// 0.79; 1000 x 4096 x 4096 60 us, 0.56. fp32: 1000 x 4096 x 4096 305 us, 110
// TFLOP/s of the 155 that a large product reaches; 16384 x 7168 x 256 480 us, 125.
// kAdapt: the epilogue adds each token's adapter, v B^T, one different adapter
// of a 16-token group after another, and writes y; otherwise fp32 parts.
template <bool kF32, typename C, bool kAdapt>
__global__ __launch_bounds__(C::kBlock) void linear_tile(TileArgs p) {
#if defined(__HIP_DEVICE_COMPILE__)
  // blocks are dealt round-robin to the 8 XCDs: each XCD gets a run of the
  // order; the grid is a multiple of 8
  const int per = gridDim.x >> 3;
  const int block = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if (block < p.m_tiles * p.n_tiles * p.parts) tile_unit<kF32, C, kAdapt>(p, block);
#endif
}

// At most 16 tokens: block (tile, s) of the weight's and then the adapters'
// tiles. Bound by latency for small weights (3584 x 3584: 10 us, a burst of loads),
// by reading W for large ones (7168 x 7168: 21 us, 4.9 TB/s).
template <bool kF32, bool kWide>
__global__ __launch_bounds__(kThreads, 3) void stream_partial(StreamArgs p) {
  const int64_t z = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * kThreads + threadIdx.x;
  if (z < p.n_zero) p.zero[z] = 0;
  __shared__ floatx4 red[(kWide ? 2 : 1) * kWaves * kWave];
  if (p.units && blockIdx.x + 1 == gridDim.x) {   // the last blocks: the tokens' units
    if (blockIdx.y == 0 && threadIdx.x < kWave) make_units(p, 0);
    return;
  }
  if (kWide && static_cast<int>(blockIdx.x) < p.tiles)
    stream_wide<kF32>(p, blockIdx.x, blockIdx.y, gridDim.y, red);
  else
    stream_unit<kF32, 1>(p, 0, blockIdx.x, blockIdx.y, gridDim.y, red);
}

// More tokens: the first `tiles` blocks are weight tiles of 64 tokens x 128 rows
// (every token beside each weight byte, so that x is read once a tile and not
// once for 16 rows), the others units of the adapters' low-rank products,
// `units` for each 64 tokens (first they would fill the CUs' LDS: 44 us and not 26
// for 64 tokens, a 7168 x 7168 weight and 24 adapters of rank 64).
typedef Shape<1, 4, 4, 2, 3> FewShape;
template <bool kF32>
__global__ __launch_bounds__(kThreads) void few_linear(TileArgs p, StreamArgs q, int tiles, int units) {
#if defined(__HIP_DEVICE_COMPILE__)
  int b = blockIdx.x;
  const int64_t z = static_cast<int64_t>(b) * kThreads + threadIdx.x;
  if (z < q.n_zero) q.zero[z] = 0;
  // (the units' sums meet in the tiles' LDS: two blocks fit a CU)
  static_assert(sizeof(u32x4) * FewShape::kN * kLine >= sizeof(floatx4) * kWaves * 4 * kWave, "");
  if (b < tiles) {
    tile_unit<kF32, FewShape, false>(p, b);
  } else if (b + q.chunks >= static_cast<int>(gridDim.x)) {   // the last blocks: the tokens' units
    if (threadIdx.x < kWave) make_units(q, static_cast<int>(gridDim.x) - 1 - b);
  } else {
    b -= tiles;
    const int u = b / p.parts;
    stream_unit<kF32, 4>(q, u / units, u % units, b % p.parts, p.parts,
                         reinterpret_cast<floatx4*>(stage_w<FewShape, 0>()));
  }
#endif
}

typedef Shape<2, 2, 2, 2, 4> SmallShape;   // 64 x 64
typedef Shape<2, 2, 4, 4, 2> MidShape;     // 128 x 128
typedef Shape<2, 4, 4, 4, 3> WideShape;    // 128 x 256, eight waves

template <bool kF32, typename C, bool kAdapt>
hipError_t launch_tile(TileArgs a, hipStream_t st) {
  a.m_tiles = static_cast<int>(cdiv(a.T, C::kM));
  a.n_tiles = static_cast<int>(cdiv(a.N, C::kN));
  const int64_t total = static_cast<int64_t>(a.m_tiles) * a.n_tiles * a.parts;
  hipLaunchKernelGGL((linear_tile<kF32, C, kAdapt>), dim3(static_cast<unsigned>(cdiv(total, 8) * 8)),
                     dim3(C::kBlock), 0, st, a);
  return hipGetLastError();
}

// Parts of the reduction for n tiles of `ksteps` steps: enough for `per_cu`
// blocks a CU, at least `least` steps each.
int parts_for(int per_cu, int64_t n, int64_t ksteps, int64_t least, int64_t most) {
  int64_t want = cdiv(static_cast<int64_t>(per_cu) * kPlanCus, n);
  if (want > ksteps / least) want = ksteps / least;
  if (want > most) want = most;
  return static_cast<int>(want < 1 ? 1 : want);
}

// For n 64 x 128 tiles. bf16: at most one block a CU (64 x 4096 x 11008 in two
// parts 24 us, in three 29; 216 x 1088 x 2816 in two 12.5, in three 14.9, in five
// 16.6). fp32, bound by its products and not by reading: the least work for the
// fullest CU (200 x 3000 x 4500, 144 tiles: in five parts 78 us, in two 108; 211 x
// 1840 x 5392, 172 tiles: in four 61, in two 70, in one 79).
int few_parts(int64_t n, int64_t row_bytes, bool f32) {
  int64_t most = cdiv(row_bytes, 128) / 3;
  if (most < 1) most = 1;
  if (most > 8) most = 8;
  int64_t parts = kPlanCus / n;
  if (f32) {
    parts = 1;
    for (int64_t p = 2; p <= most; ++p)   // a block more must be worth 3% of its work
      if (cdiv(n * p, kPlanCus) * (100 + 3 * p) * parts < cdiv(n * parts, kPlanCus) * (100 + 3 * parts) * p) parts = p;
  }
  if (parts > most) parts = most;
  return static_cast<int>(parts < 1 ? 1 : parts);
}

// At most 16 tokens. Parts of units of 32 rows (stream_wide): three blocks a CU at
// most.
int wide_parts(int64_t N) {
  const int64_t parts = 3 * kPlanCus / cdiv(N, 32);
  return static_cast<int>(parts < 1 ? 1 : parts);
}
// Rows of a unit: 32 where that leaves a wave four batches of loads, else 16 (one
// and eight tokens of 7168 x 7168: 21 and 25 us, by 16 28 and 33; 16 of 4096 x
// 4096, with two batches: 15.7 us, by 16 14.1).
int stream_rows(int64_t N, int64_t row_bytes) {
  return row_bytes / 64 >= 16 * kWaves * wide_parts(N) ? 32 : 16;
}
// Parts of units of 16: one batch of loads for each of a part's waves, or a few
// where that already gives four blocks a CU.
int stream_parts(int64_t N, int64_t row_bytes) {
  if (stream_rows(N, row_bytes) == 32) return wide_parts(N);
  const int64_t tiles = cdiv(N, 16), batches = cdiv(cdiv(row_bytes, 64), kU * kWaves);
  int64_t each = 1;
  while (each < batches && tiles * cdiv(batches, each + 1) >= 4 * kPlanCus) ++each;
  return static_cast<int>(cdiv(batches, each));
}
template <bool kF32, bool kWide>
hipError_t launch_stream(const StreamArgs& a, int x, int parts, hipStream_t st) {
  hipLaunchKernelGGL((stream_partial<kF32, kWide>), dim3(x, parts), dim3(kThreads), 0, st, a);
  return hipGetLastError();
}
hipError_t launch_stream(const StreamArgs& a, bool f32, int x, int parts, hipStream_t st) {
  if (stream_rows(a.N, a.row_bytes) == 32)
    return f32 ? launch_stream<true, true>(a, x, parts, st) : launch_stream<false, true>(a, x, parts, st);
  return f32 ? launch_stream<true, false>(a, x, parts, st) : launch_stream<false, false>(a, x, parts, st);
}

int64_t up16(int64_t v) { return cdiv(v, 16) * 16; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

// ---- the router's logits --------------------------------------------------
namespace {
// Shapes of the logits' tiles: 128 x 256 where that leaves a tile for every
// fourth CU or more, so that four parts fill them all; else 64 x 64 (7168 x 256:
// 16384 tokens 69 us, by 64 x 64 126; 8192 tokens 39 and 64; 4096 tokens 31 and 27;
// 2048 tokens 28 and 17.5).
bool wide_logits(int64_t T, int64_t row_bytes, int N) {
  return N > 128 && row_bytes <= (int64_t{1} << 23) &&
         cdiv(T, WideShape::kM) * cdiv(N, WideShape::kN) >= kPlanCus / 4;
}
}  // namespace

LogitsLayout logits_layout(int64_t T, int64_t H, int N, bool f32) {
  LogitsLayout L{};
  const int64_t row_bytes = H * (f32 ? 4 : 2), ktiles = cdiv(row_bytes, 128);
  L.pitch = static_cast<int>(up16(N));
  if (T <= 16)
    L.parts = stream_parts(N, row_bytes);
  else if (T <= kFewTokens)
    L.parts = parts_for(1, cdiv(N, FewShape::kN), ktiles, 3, 16);
  else if (wide_logits(T, row_bytes, N))
    L.parts = parts_for(1, cdiv(T, WideShape::kM) * cdiv(N, WideShape::kN), ktiles, 6, 4);
  else
    L.parts = parts_for(2, cdiv(T, SmallShape::kM) * cdiv(N, SmallShape::kN), ktiles, 4, 16);
  L.bytes = up256(sizeof(float) * static_cast<size_t>(L.parts) * T * L.pitch);
  return L;
}

hipError_t logits(int64_t T, int64_t H, int N, bool f32, const void* x, const void* w, float* part,
                  uint32_t* zero, int n_zero, hipStream_t st) {
  const LogitsLayout L = logits_layout(T, H, N, f32);
  const int64_t row_bytes = H * (f32 ? 4 : 2);
  StreamArgs a{};
  a.x = static_cast<const char*>(x);
  a.w = static_cast<const char*>(w);
  a.part = part;
  a.row_bytes = row_bytes;
  a.T = T;
  a.N = N;
  a.Np = L.pitch;
  a.tiles = static_cast<int>(cdiv(N, stream_rows(N, row_bytes)));
  a.zero = zero;
  a.n_zero = n_zero;
  if (T <= 16) {
    return launch_stream(a, f32, a.tiles, L.parts, st);
  }
  TileArgs t{};
  t.x = a.x;
  t.w = a.w;
  t.row_bytes = row_bytes;
  t.T = T;
  t.N = N;
  t.part = part;
  t.Np = L.pitch;
  t.parts = L.parts;
  if (T <= kFewTokens) {
    t.m_tiles = 1;
    t.n_tiles = static_cast<int>(cdiv(N, FewShape::kN));
    const int tiles = t.n_tiles * t.parts;
    if (f32) hipLaunchKernelGGL(few_linear<true>, dim3(tiles), dim3(kThreads), 0, st, t, a, tiles, 0);
    else hipLaunchKernelGGL(few_linear<false>, dim3(tiles), dim3(kThreads), 0, st, t, a, tiles, 0);
    return hipGetLastError();
  }
  if (wide_logits(T, row_bytes, N))
    return f32 ? launch_tile<true, WideShape, false>(t, st) : launch_tile<false, WideShape, false>(t, st);
  return f32 ? launch_tile<true, SmallShape, false>(t, st) : launch_tile<false, SmallShape, false>(t, st);
}

// ---- the shared projection with adapters ------------------------------------
namespace {
// Whether the projection goes through fp32 parts: a few tokens, or too few
// 64 x 128 tiles to occupy the CUs without dividing the reduction.
bool adapter_in_parts(const tr_adapter_desc& d) {
  return cdiv(d.T, FewShape::kM) * cdiv(d.N, FewShape::kN) < kPlanCus;
}
template <bool kF32, int kKb, int kParts>
hipError_t launch_expand(const ExpandArgs& p, dim3 grid, hipStream_t st) {
  hipLaunchKernelGGL((adapter_few<kF32, kKb, kParts>), grid, dim3(kThreads), 0, st, p);
  return hipGetLastError();
}
struct AdapterLayout {
  int parts, Np, Rp, Rq, n_units;
  size_t vpart, units, perm, sid, total;
};
AdapterLayout adapter_layout(const tr_adapter_desc& d) {
  AdapterLayout L{};
  const bool f32 = d.dtype == TR_F32;
  const int64_t row_bytes = d.H * (f32 ? 4 : 2);
  L.Np = static_cast<int>(up16(d.N));
  L.Rp = static_cast<int>(up16(d.R));
  L.Rq = static_cast<int>(f32 ? up16(d.R) : cdiv(d.R, 32) * 32);
  if (adapter_in_parts(d)) {
    L.parts = d.T <= 16 ? stream_parts(d.N, row_bytes)
                        : few_parts(cdiv(d.T, FewShape::kM) * cdiv(d.N, FewShape::kN), row_bytes, f32);
    L.vpart = up256(sizeof(float) * static_cast<size_t>(L.parts) * d.T * L.Np);
    L.units = L.vpart + up256(sizeof(float) * static_cast<size_t>(L.parts) * d.T * L.Rp);
    // units of 64 tokens: one for each adapter (and for none), one more for every
    // 16 tokens
    const int64_t chunk = d.T < kFewTokens ? d.T : kFewTokens, most = d.A + 1 + chunk / 16;
    L.n_units = static_cast<int>(most < chunk ? most : chunk);
    L.total = L.units + up256(sizeof(AdapterUnit) * L.n_units * cdiv(d.T, kFewTokens));
  } else {
    L.perm = up256(static_cast<size_t>(d.T) * L.Rq * 4);   // fp32, or two bf16 numbers
    L.sid = L.perm + up256(4 * static_cast<size_t>(d.T));
    L.total = L.sid + up256(4 * static_cast<size_t>(d.T));
  }
  if (L.total == 0) L.total = 256;
  return L;
}
}  // namespace

size_t adapter_workspace(const tr_adapter_desc& d) { return adapter_layout(d).total; }

hipError_t adapter_linear(const tr_adapter_desc& d, const void* x, const void* w, const void* a,
                          const void* b, const int32_t* ids, const float* scales, void* y, void* ws,
                          hipStream_t st) {
  const AdapterLayout L = adapter_layout(d);
  const bool f32 = d.dtype == TR_F32;
  const int64_t row_bytes = d.H * (f32 ? 4 : 2);
  hipError_t e;
  if (adapter_in_parts(d)) {
    StreamArgs s{};
    s.x = static_cast<const char*>(x);
    s.w = static_cast<const char*>(w);
    s.part = static_cast<float*>(ws);
    s.row_bytes = row_bytes;
    s.T = d.T;
    s.N = static_cast<int>(d.N);
    s.Np = L.Np;
    s.ids = ids;
    s.a = static_cast<const char*>(a);
    s.vpart = reinterpret_cast<float*>(static_cast<char*>(ws) + L.vpart);
    s.A = d.A;
    s.R = d.R;
    s.Rp = L.Rp;
    s.rank_tiles = L.Rp / 16;
    s.units = reinterpret_cast<AdapterUnit*>(static_cast<char*>(ws) + L.units);
    s.n_units = L.n_units;
    const int64_t chunk = d.T < kFewTokens ? d.T : kFewTokens;
    const int slots = static_cast<int>(chunk < d.A ? chunk : d.A);   // adapters among 64 tokens
    const int chunks = static_cast<int>(cdiv(d.T, kFewTokens));
    s.chunks = chunks;
    if (d.T <= 16) {
      s.tiles = static_cast<int>(cdiv(d.N, stream_rows(d.N, row_bytes)));
      if ((e = launch_stream(s, f32, s.tiles + slots * s.rank_tiles + 1, L.parts, st)) != hipSuccess) return e;
    } else {
      TileArgs t{};
      t.x = s.x;
      t.w = s.w;
      t.row_bytes = row_bytes;
      t.T = d.T;
      t.N = s.N;
      t.part = s.part;
      t.Np = L.Np;
      t.parts = L.parts;
      t.m_tiles = chunks;
      t.n_tiles = static_cast<int>(cdiv(d.N, FewShape::kN));
      const int tiles = t.m_tiles * t.n_tiles * t.parts;
      const int units = slots * s.rank_tiles;   // (s.tiles is 0: the adapters' only)
      const dim3 grid(tiles + chunks * units * t.parts + chunks);
      if (f32) hipLaunchKernelGGL(few_linear<true>, grid, dim3(kThreads), 0, st, t, s, tiles, units);
      else hipLaunchKernelGGL(few_linear<false>, grid, dim3(kThreads), 0, st, t, s, tiles, units);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
    ExpandArgs p{};
    p.part = s.part;
    p.vpart = s.vpart;
    p.units = s.units;
    p.n_units = L.n_units;
    p.scales = scales;
    p.b = b;
    p.y = y;
    p.S = L.parts;
    p.T = s.T;
    p.N = s.N;
    p.Np = L.Np;
    p.A = d.A;
    p.R = d.R;
    p.Rp = L.Rp;
    const dim3 grid(static_cast<unsigned>(cdiv(d.N, 32 * kWaves)), static_cast<unsigned>(L.n_units),
                    static_cast<unsigned>(chunks));
    // few parts and ranks: 86 registers a lane, five waves a SIMD, and not 139 and
    // three (64 x 7168 x 7168, 24 adapters of rank 64: 12.8 us and not 15.6); more
    // parts in steps of four take longer (100 x 7168 x 1024: 6.8 us, by eight 6.0)
    const bool small = L.parts <= 4 && d.R <= (f32 ? 32 : 64);
    if (f32) return small ? launch_expand<true, 2, 4>(p, grid, st) : launch_expand<true, 4, 8>(p, grid, st);
    return small ? launch_expand<false, 2, 4>(p, grid, st) : launch_expand<false, 4, 8>(p, grid, st);
  }
  // the positions' order: the tokens' own where x is past the 32-bit offsets that
  // gather its rows
  int32_t *perm = nullptr, *sid = nullptr;
  if (d.T * row_bytes < (int64_t{1} << 31)) {
    perm = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + L.perm);
    sid = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + L.sid);
    hipLaunchKernelGGL(adapter_order, dim3(static_cast<unsigned>(cdiv(d.T, kWindow))), dim3(kOrderThreads),
                       0, st, ids, d.T, d.A, perm, sid);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    ids = sid;
  }
  ShrinkArgs s{};
  s.x = static_cast<const char*>(x);
  s.a = static_cast<const char*>(a);
  s.ids = ids;
  s.perm = perm;
  s.scales = scales;
  s.v = ws;
  s.row_bytes = row_bytes;
  s.T = d.T;
  s.A = d.A;
  s.R = d.R;
  s.Rq = L.Rq;
  if ((e = f32 ? launch_shrink<true>(s, st) : launch_shrink<false>(s, st)) != hipSuccess) return e;
  if (adapter_can_tile(d)) return adapter_tiles(d, x, w, b, ids, perm, ws, L.Rq, y, st);
  TileArgs t{};
  t.x = s.x;
  t.w = static_cast<const char*>(w);
  t.row_bytes = row_bytes;
  t.T = d.T;
  t.N = static_cast<int>(d.N);
  t.parts = 1;
  t.y = y;
  t.ids = ids;
  t.perm = perm;
  t.v = ws;
  t.b = b;
  t.A = d.A;
  t.R = d.R;
  t.Rq = L.Rq;
  // the largest tiles of which there is one for each CU: 8192 x 7160 x 7000 takes
  // 1040 us on the wide ones and 1090 us on the middle ones, 1000 x 5000 x 6001
  // (376 middle tiles) 111 us on the middle and 165 us on the small ones
  if (cdiv(d.T, WideShape::kM) * cdiv(d.N, WideShape::kN) >= kPlanCus && row_bytes <= (int64_t{1} << 23))
    return f32 ? launch_tile<true, WideShape, true>(t, st) : launch_tile<false, WideShape, true>(t, st);
  if (cdiv(d.T, MidShape::kM) * cdiv(d.N, MidShape::kN) >= kPlanCus)
    return f32 ? launch_tile<true, MidShape, true>(t, st) : launch_tile<false, MidShape, true>(t, st);
  return f32 ? launch_tile<true, SmallShape, true>(t, st) : launch_tile<false, SmallShape, true>(t, st);
}

}  // namespace tr
