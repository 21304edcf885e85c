"""Frozen-NF4-base + LoRA linear layer for AMD Instinct MI355X (gfx950).

The compute path is the HIP library ``libqlora_nf4.so`` behind the C ABI in
``include/qlora_nf4.h``; this package only loads it and marshals torch
tensors into its calls (see :mod:`quantized_base_lora_nf4_amd.ops`).
"""

from ._lib import LIB_PATH, EXPORTS, QloraError, lib  # noqa: F401
from .ops import (LqResult, NF4Weight, QLoRALinear, QLoRALinearFunction,  # noqa: F401
                  alloc_nf4, code_table, ilp_plan, lq_init, lq_workspace_size, nf4_dequantize,
                  nf4_quantize, qlora_linear_bwd, qlora_linear_fwd, qlora_linear_fwd_noalloc,
                  quant_error, storage_bytes, user_table, workspace_size, USER_CODES)
from .multi_ops import (QLoRAMultiLinear, multi_workspace_size,  # noqa: F401
                        qlora_linear_multi_fwd)
from .optim import AdamW, AdamWState, adamw_init, adamw_step, adamw_values  # noqa: F401
from .train_ops import (LayerNorm, RMSNorm, attention, attention_bwd, attention_fwd,  # noqa: F401
                        clip_grad_norm, grad_norm, norm, norm_bwd, norm_fwd, rope, rope_bwd,
                        rope_fwd, rope_frequencies)
