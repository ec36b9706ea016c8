"""top_reduce_amd: one GPU's share of an expert-parallel MoE FFN on MI355X.

Route scan -> expand -> grouped SwiGLU GEMM -> weighted top-k reduce, as
hand-written gfx950 HIP kernels behind the C ABI of ``libtopreduce.so``
(``include/topreduce.h``). This package is the thin Python binding: it checks
and marshals PyTorch tensors (device memory and streams only) and calls the
library; every step of the path runs in the library's kernels. There is no
fallback: if the library is not built, importing the binding's entry points
raises.

Entry points: ``plan`` (route scan; with ``block_rows``/``block_counts`` over
a DP-padded buffer), ``forward`` (the whole layer), the stages ``expand``,
``grouped_gemm`` (``grouped_gemm_up``/``_down``, ``grouped_gemm_up_x``
gathering x, ``grouped_gemm_down_y`` writing single-slot rows to y),
``combine_reduce`` / ``combine_reduce_multi``, the cross-rank
``combine_epilogue``, ``compact_rows`` (effective rows of a padded buffer)
and ``plan_stats``. ``FLAG_NO_XE`` plans without the expanded-row buffer.
``forward_noalloc`` is plan + forward in the library's own static workspace,
for callers that cannot allocate device memory.

Before and beside the expert path: ``route_topk`` (the router: logits, top-k,
gate weights), ``layer`` (the whole layer from hidden rows, router included)
and ``adapter_linear`` (a projection all rows share, with a low-rank adapter
of each row's request), each with its ``*_workspace_size``.

In 8 and 4 bits (blocks of 32 numbers with a power of two as scale): ``rms_norm`` (the
residual's addition and the norm, its result in the rows' type, in 8 bits, or both),
``quantize_mx``, ``expert_linear`` (products grouped by expert over ragged segments),
``forward_mx`` (the plan's whole layer) and ``linear_mx4`` (few rows, weights in 4 bits).
"""

from ._binding import (  # noqa: F401
    ABI_VERSION,
    BF16,
    F32,
    FLAG_GEMM_FORCE_STREAM,
    FLAG_GEMM_FORCE_TILED,
    FLAG_NO_XE,
    NOALLOC_SCRATCH_BYTES,
    MoePlan,
    TopReduceError,
    adapter_linear,
    adapter_workspace_size,
    combine_epilogue,
    compact_rows,
    combine_reduce,
    combine_reduce_multi,
    expand,
    forward,
    forward_noalloc,
    grouped_gemm,
    grouped_gemm_down,
    grouped_gemm_down_y,
    grouped_gemm_up,
    grouped_gemm_up_x,
    layer,
    layer_workspace_size,
    lib_path,
    load_library,
    make_desc,
    plan,
    plan_stats,
    route_topk,
    route_workspace_size,
    workspace_size,
)

from ._mx import (  # noqa: F401
    Normed,
    expert_linear,
    forward_mx,
    linear_mx4,
    linear_mx4_workspace_size,
    quantize_mx,
    rms_norm,
)
