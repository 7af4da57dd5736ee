"""CPU float64 oracle (test infrastructure; never part of the product path)."""
from .relpos_oracle import (attention, attention_backward, attention_rows, dense_bias, fused, fused_backward,
                            fused_rows, lse2, project, project_rows, rel_index)
from .train_oracle import (attention_backward_from, masked_attention, project_backward, qk_norm_rope,
                           qk_norm_rope_backward, rotate)

__all__ = ["attention", "attention_backward", "attention_backward_from", "attention_rows", "dense_bias", "fused",
           "fused_backward", "fused_rows", "lse2", "masked_attention", "project", "project_backward", "project_rows",
           "qk_norm_rope", "qk_norm_rope_backward", "rel_index", "rotate"]
