// Internal launchers of libtopreduce (host side). Not part of the C ABI.
#pragma once

#include <hip/hip_runtime.h>

#include "topreduce.h"

namespace tr {

constexpr int kMaxScanBlocks = 256;
constexpr int kMaxK = 32;
constexpr int kMaxE = 1024;
// Experts with at most this many routes go to the weight-streaming GEMM.
constexpr int kStreamMaxRows = 32;
// A batch of at most this many expanded rows (T * K) sends every expert to the
// weight-streaming GEMM in the automatic mode: such experts rarely fill a
// tile, and the tiled kernels' launches would mostly find nothing to do.
constexpr int kSmallBatchRows = 128;
// The fewest routes of an expert the tiled GEMM takes under d's flags (the
// route scan marks the rows of such experts for the reduce folded into GEMM2).
inline int min_tiled_routes(const tr_moe_desc& d) {
  if (d.flags & TR_FLAG_GEMM_FORCE_STREAM) return 0x7fffffff;
  if (d.flags & TR_FLAG_GEMM_FORCE_TILED) return 1;
  return d.T * d.K <= kSmallBatchRows ? 0x7fffffff : kStreamMaxRows + 1;
}
// Spare rows after R_cap in the expanded (Xe) and intermediate (h) buffers,
// so GEMM tiles may read a full tile of rows from any segment start.
constexpr int kRowPad = 256;
// bf16 shapes of the tiled and streaming GEMM kernels: H a multiple of
// kColMultiple, I of kColMultiple / 2 (other shapes: the any-shape kernel).
constexpr int kColMultiple = 256;
// Most worker blocks of a DP-padded buffer (their counts' prefix sits in LDS).
constexpr int kMaxPadBlocks = 4096;

hipError_t route_scan(const tr_moe_plan& p, const void* idx, hipStream_t st);
void route_scan_geometry(int64_t T, int K, int* blocks, int* rows_per_block);
hipError_t expand(const tr_moe_plan& p, const void* x, hipStream_t st);
enum { kGemmUp = 1, kGemmDown = 2 };
// parts: kGemmUp (Xe -> h, SwiGLU), kGemmDown (h -> O), or both. With
// x_gather (bf16 only), GEMM1 reads the received rows x through the plan's
// route table instead of Xe, so no expand pass is needed.
// With y_fused (bf16 only), GEMM2 writes the rows of received rows with one
// local slot straight to y, weighted (w_fused, NULL for 1) and rounded as the
// reduce would; combine_reduce with skip_single then completes y. With
// y_done as well, a decode batch may run the whole reduce inside GEMM2: then
// *y_done is set and y is complete (no combine_reduce needed).
hipError_t grouped_gemm(const tr_moe_plan& p, const void* w1, const void* w2, int parts,
                        hipStream_t st, const void* x_gather = nullptr,
                        const float* w_fused = nullptr, void* y_fused = nullptr,
                        bool* y_done = nullptr);
// Whether GEMM1 may gather from x of this shape (32-bit buffer offsets).
bool gemm_can_gather(const tr_moe_desc& d);
hipError_t combine_reduce(const tr_moe_plan& p, const void* expert_out, const float* w, void* y,
                          hipStream_t st, bool skip_single = false);
// y[t] = sum over j of recv[src[t][j]] (src >= 0 and < n_recv), unit weights.
hipError_t combine_epilogue(int64_t T, int J, int64_t H, bool bf16, const int* src,
                            const void* recv, int64_t n_recv, void* y, hipStream_t st);

// Rows of a DP-padded buffer that carry data (block j of B rows: its first
// counts[j], clamped) copied to compact order, or back (to_padded).
hipError_t compact_rows(int64_t T, int B, const int* counts, int64_t row_bytes, const void* src,
                        void* dst, bool to_padded, int* n_out, hipStream_t st);

// Compute units of the current device (cached per device).
int device_cu_count();
// Compute units that a workspace's layout is planned for (a layout must not
// depend on the device that is current).
constexpr int kPlanCus = 256;

// --- router, few-token layer, shared projection with adapters ---------------
// Batches of at most this many tokens take the weight-streaming kernels (their
// tokens are the bits of one 64-bit mask).
constexpr int kFewTokens = 64;
constexpr int kMaxGates = 4096;   // experts a router chooses from
constexpr int kMaxRank = 256;     // of an adapter

// Logits x w^T as fp32 parts [parts, T, pitch]; their sum is the logits.
struct LogitsLayout {
  int parts, pitch;
  size_t bytes;
};
LogitsLayout logits_layout(int64_t T, int64_t H, int N, bool f32);
// Few tokens only: also zeroes n_zero words at `zero` (n_zero at most 2048).
hipError_t logits(int64_t T, int64_t H, int N, bool f32, const void* x, const void* w, float* part,
                  uint32_t* zero, int n_zero, hipStream_t st);

// Local routes of at most kFewTokens tokens, written by the router's selection.
struct FewRoutes {
  unsigned long long* masks;   // [E] the tokens that chose each local expert
  uint8_t* slots;              // [E, 64] the token's slot that names it
  int64_t begin;
  int E;
};
size_t route_workspace(const tr_route_desc& d);
hipError_t route_topk(const tr_route_desc& d, const void* x, const void* w_gate, const float* bias,
                      void* idx, float* w, void* ws, hipStream_t st, const FewRoutes* few = nullptr);

struct SelectArgs;   // tr_select.h
SelectArgs select_args(const tr_route_desc& d, const float* bias, void* idx, float* w, const void* ws);

// A whole layer of at most kFewTokens rows. route_ws: route_workspace bytes; ws:
// few_workspace bytes.
size_t few_workspace(const tr_layer_desc& d);
hipError_t few_layer(const tr_layer_desc& d, const void* x, const void* w_gate, const float* bias,
                     const void* w1, const void* w2, void* y, void* idx, float* w, void* route_ws,
                     void* ws, hipStream_t st);

// The shared projection on the grouped GEMM's 256 x 256 tiles: whether its shape
// allows that and gives at least two tiles a CU (bf16; ids and v, low-rank
// products as adapter_linear makes them, [T, 2, Rq], by position; perm: the
// positions' tokens, x being below 2 GiB, or NULL: the same).
bool adapter_can_tile(const tr_adapter_desc& d);
hipError_t adapter_tiles(const tr_adapter_desc& d, const void* x, const void* w, const void* b,
                         const int32_t* ids, const int32_t* perm, const void* v, int Rq, void* y,
                         hipStream_t st);
size_t adapter_workspace(const tr_adapter_desc& d);
hipError_t adapter_linear(const tr_adapter_desc& d, const void* x, const void* w, const void* a,
                          const void* b, const int32_t* ids, const float* scales, void* y, void* ws,
                          hipStream_t st);

}  // namespace tr
