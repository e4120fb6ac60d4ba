"""MI355X (gfx950) GPTQ layer quantizer: Hessian accumulation, damped
Cholesky factor of the inverse, blocked column sweep with error feedback and
lazy-batch trailing updates, and code packing, in hand-written HIP kernels
behind a C ABI (include/gptq.h); for inference, the dequantising product of a
packed layer; and for mixtures of experts the order of tokens by expert and
back, the packed products of the experts and their gradients, and activations
kept in 8 bits for the weight gradient. This package is its Python binding."""
from .gptq import (BF16, F32, Checkpoint, GPTQError, NOALLOC_SCRATCH_BYTES, QuantResult, Route, accumulate_hessian,
                   checkpoint_restore, checkpoint_save, checkpoint_weight_grad, combine, combine_grad, dequant_matmul,
                   dequant_matmul_noalloc, dispatch, eora, eora_workspace_bytes, expert_matmul, expert_matmul_grad, refine_lowrank,
                   refine_workspace_bytes, quantize_rtn, route,
                   dequant_matmul_workspace_bytes, factor_hinv, hessian_workspace_bytes, load, make_params, pack_codes, profile_collect,
                   profile_enable, quantize_layer, repack_act_order, unpack_codes, workspace_bytes, LIB_PATH,
                   PROF_CLASSES)

__all__ = ["BF16", "F32", "Checkpoint", "GPTQError", "NOALLOC_SCRATCH_BYTES", "QuantResult", "Route",
           "accumulate_hessian", "checkpoint_restore", "checkpoint_save", "checkpoint_weight_grad", "combine",
           "combine_grad", "dispatch", "expert_matmul", "expert_matmul_grad", "route",
           "dequant_matmul", "dequant_matmul_noalloc", "eora", "eora_workspace_bytes", "refine_lowrank",
           "refine_workspace_bytes", "quantize_rtn",
           "dequant_matmul_workspace_bytes", "factor_hinv",
           "hessian_workspace_bytes", "load", "make_params", "pack_codes", "profile_collect",
           "profile_enable", "quantize_layer", "repack_act_order", "unpack_codes", "workspace_bytes", "LIB_PATH",
           "PROF_CLASSES"]
