"""KDA (Kimi Delta Attention) gated-delta recurrence for GB300 (sm_103a).

Per sequence and head, S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1}
+ beta_t k_t v_t^T and o_t = S_t^T q_t (the web page
"研究KimiK3，我发现大模型正在学会“管理自己的计算”", pwwt.cn, §四 and §二.1).

Entry points (thin ctypes binding over the C ABI in include/kda.h):
``prefill`` (per-channel, scalar or no gate), ``prefill_fp8`` (MX-style FP8
q, k, v), ``prefill_segmented`` (one long sequence cut into segments that run
at once), ``varlen_prefill``,
``decode_step``; host (CPU) tensors given to ``prefill`` or ``prefill_fp8``
go through the native host-buffer pipeline (kda_prefill_host,
kda_prefill_fp8_host); and for serving with a pool of states indexed by slot:
``varlen_prefill_slots``, ``decode_step_slots``; for training,
``prefill_backward`` (the gradients of ``prefill``). Linear attention with a
decay (the update without its erase step): ``linear_prefill``,
``linear_varlen_prefill``, their gradients ``linear_prefill_backward`` and
``linear_varlen_prefill_backward``, ``linear_decode_step`` and
``linear_decode_step_slots``; the norm of query and key heads with the rotary
positions: ``qk_norm_rope``, ``qk_norm_rope_backward``, ``rope_table``. Build the CUDA library with
``kda_gated_delta_chunkwise_gb300.build.build()`` first.
"""
from ._binding import (ALGOS, EXPORTS, GATES, KDA_DEV_BAD_CU_SEQLENS, KDA_DEV_BAD_SLOT, KDA_DEV_BAD_POSITION,  # noqa: F401
                       KDA_DEV_OK, KdaError, decode_step, decode_step_slots, device_errors, lib_path, load,
                       prefill, prefill_backward, prefill_fp8, prefill_segmented, prefill_segmented_workspace_bytes,
                       prefill_workspace_bytes, segment_plan, selftest_bounded_wait, varlen_prefill,
                       varlen_prefill_backward,
                       varlen_prefill_slots, varlen_workspace_bytes)
from ._linear import (DECAYS, NORMS, ROPE_LAYOUTS, linear_decode_step, linear_decode_step_slots,  # noqa: F401
                      linear_prefill, linear_prefill_backward, linear_prefill_backward_workspace_bytes,
                      linear_prefill_workspace_bytes, linear_varlen_prefill, linear_varlen_prefill_backward,
                      linear_varlen_prefill_backward_workspace_bytes, linear_varlen_prefill_workspace_bytes,
                      qk_norm_rope, qk_norm_rope_backward, rope_table)
