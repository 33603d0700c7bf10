"""MI355X (gfx950) sparse Mixture-of-Experts layer forward.

Thin Python binding over libmoe.so's C ABI (include/moe.h, and include/moe_ext.h
for the operators around the layer): the functions below carry the C names and only marshal arguments (torch tensors are device
buffers; their data pointers and torch's current HIP stream go to the
library). Every step of the layer runs in the library's HIP kernels; there is
no CPU or PyTorch fallback, and importing fails when the library is missing.
"""

from ._lib import (  # noqa: F401
    MOE_DTYPE_BF16,
    MOE_DTYPE_F32,
    MOE_STAGE_FORWARD,
    MOE_STAGE_GROUPED_FFN,
    MOE_STAGE_PERMUTE,
    MOE_STAGE_ROUTE,
    MOE_STAGE_TRAIN,
    MoEError,
    Problem,
    lib_path,
    make_problem,
    moe_combine,
    moe_backward,
    moe_forward,
    moe_forward_train,
    moe_grouped_ffn,
    moe_grouped_ffn_gather,
    moe_permute,
    moe_permute_index,
    moe_permute_index_noalloc,
    moe_plan,
    moe_route,
    moe_route_ws,
    moe_status_str,
    moe_workspace_size,
)
from ._ext import (  # noqa: F401
    MOEX_STAGE_BALANCE,
    MOEX_STAGE_FFN_FP8,
    MOEX_STAGE_FORWARD_FP8,
    MOEX_STAGE_NORM_BACKWARD,
    MOEX_STAGE_TRAIN_BALANCED,
    code_pitch,
    expert_shapes,
    moex_add_rmsnorm,
    moex_add_rmsnorm_backward,
    moex_backward_balanced,
    moex_balance_loss,
    moex_forward_fp8,
    moex_grouped_ffn_fp8,
    moex_quantize_experts,
    moex_quantize_rows,
    moex_workspace_size,
    scale_pitch,
)
from .layer import MoEBlockFP8, MoEForward  # noqa: F401
