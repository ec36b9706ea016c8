// The router: logits (linear.hip), then every token's choice (tr_select.h), one
// wave a token. Bound: latency for a few tokens, the logits' bytes and the
// selection's instructions for many.
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
  hipError_t e = logits(d.T, d.H, d.G, d.dtype == TR_F32, x, w_gate, static_cast<float*>(ws),
                        few ? reinterpret_cast<uint32_t*>(few->masks) : nullptr,
                        few ? 2 * few->E : 0, st);
  if (e != hipSuccess) return e;
  const SelectArgs a = select_args(d, bias, idx, w, ws);
  const FewRoutes f = few ? *few : FewRoutes{};
  if (d.G <= 64) return launch_select<1>(a, f, st);
  if (d.G <= 256) return launch_select<4>(a, f, st);
  if (d.G <= 1024) return launch_select<16>(a, f, st);
  return launch_select<64>(a, f, st);
}

}  // namespace tr
