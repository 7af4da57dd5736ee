"""GB300-native global attention with decomposed relative-position bias.

The computation lives in ``libdera_relpos.so`` (hand-written sm_103a CUDA
behind a C ABI, declared in ``include/dera_relpos.h`` and ``include/dera_train.h``);
this package is its thin Python binding.  Entry points: :func:`project`,
:func:`attention`, :func:`fused`; for training, :func:`fused_lse` and
:func:`fused_backward`, or step by step :func:`qk_norm_rope`, :func:`project`,
:func:`attention_lse` and the backward of each.
"""
from .api import (DERA_BF16, DERA_F16, DERA_F32, DeraError, attention, backward_workspace_size, declared_entry_points,
                  device_status, fused, fused_backward, fused_lse, load_library, project, selftest_wait_timeout,
                  workspace_size)
from .train import (attention_backward, attention_backward_workspace_size, attention_lse, project_backward,
                    project_backward_workspace_size, qk_norm_rope, qk_norm_rope_backward,
                    qk_norm_rope_backward_workspace_size)

__all__ = ["DERA_BF16", "DERA_F16", "DERA_F32", "DeraError", "attention", "attention_backward",
           "attention_backward_workspace_size", "attention_lse", "backward_workspace_size", "declared_entry_points",
           "device_status", "fused", "fused_backward", "fused_lse", "load_library", "project", "project_backward",
           "project_backward_workspace_size", "qk_norm_rope", "qk_norm_rope_backward",
           "qk_norm_rope_backward_workspace_size", "selftest_wait_timeout", "workspace_size"]
