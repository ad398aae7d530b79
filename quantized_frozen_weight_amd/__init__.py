"""libqlora: frozen int8 / 4-bit weight + trainable LoRA linear on MI355X.

The computation lives in the HIP library libqlora.so (C ABI in
include/qlora.h); ``binding`` is its ctypes wrapper and ``workloads`` the
seeded synthetic inputs. Importing the package loads nothing; the first
library call does, and raises if the library has not been built.
"""

from .binding import (  # noqa: F401
    AdamW, Checkpoint, QLinear, QloraError, qlora_act_bwd, qlora_adamw, qlora_bwd, qlora_bwd_epi,
    qlora_bwd_epi_partial, qlora_bwd_workspace, qlora_ckpt_read,
    qlora_ckpt_write, qlora_embed, qlora_embed_bwd, qlora_fwd, qlora_fwd_acc, qlora_fwd_ckpt, qlora_fwd_epi,
    qlora_fwd_workspace, qlora_moment_read, qlora_moment_write, qlora_quantize, qlora_quantize_rows,
    qlora_status_str, qlora_weight_bytes, qlora_xent_bwd, qlora_xent_fwd,
)
