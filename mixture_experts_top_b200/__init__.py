"""B200-native forward pass of a sparsely-gated Mixture-of-Experts layer.

The compute lives in ``libmoe_b200.so`` (CUDA for sm_100a, C ABI in
``include/moe.h``); :mod:`.api` is its Python binding and :mod:`.layer` a
small helper that allocates a call's buffers with torch.  Importing this
package does not load the library; the first call does, and fails loudly if
the library has not been built.
"""
from .api import (  # noqa: F401
    MoeConfig,
    MoeError,
    alloc_adapter_plan,
    alloc_adapter_workspace,
    alloc_balance_workspace,
    alloc_workspace,
    make_config,
    moe_adapter,
    moe_adapter_backward,
    moe_adapter_plan,
    moe_balance_loss,
    moe_balance_loss_backward,
    moe_combine,
    moe_combine_dropout,
    moe_combine_dropout_backward,
    moe_device_status,
    moe_dispatch,
    moe_dropout,
    moe_expert_ffn,
    moe_forward,
    moe_route,
    moe_route_backward_add,
    moe_workspace_init,
    moe_workspace_size,
)
