"""Python binding of ``libmoe_b200.so`` (the C ABI in ``include/moe.h`` and
``include/moe_packed.h``).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  torch tensors supply device pointers and torch supplies the current
CUDA stream; nothing here computes any part of the layer, and there is no
fallback: if the library is missing or a call fails, an exception is raised.

Function names match the C entry points.  Each takes a :class:`MoeConfig`
and torch tensors (``None`` where the C side accepts NULL) and raises
:class:`MoeError` on a non-OK status.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

LIB_NAME = "libmoe_b200.so"
LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), LIB_NAME)

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_CUDA, \
    MOE_ERR_DEVICE_CHECK = range(6)
EXPERT_KINDS = {"linear": 0, "relu": 1, "swiglu": 2}
DTYPES = {"f32": 0, "bf16": 1}

# Every symbol include/moe.h declares, with its ctypes signature.
_c_p = ctypes.c_void_p
_SIGNATURES = {
    "moe_workspace_size": (ctypes.c_size_t, [_c_p]),
    "moe_workspace_init": (ctypes.c_int, [_c_p, ctypes.c_size_t, _c_p]),
    "moe_device_status": (ctypes.c_int, [_c_p, ctypes.c_size_t, _c_p, _c_p]),
    "moe_route": (ctypes.c_int, [_c_p] * 10 + [ctypes.c_size_t, _c_p]),
    "moe_route_noalloc": (ctypes.c_int, [_c_p] * 10),
    "moe_route_noisy": (ctypes.c_int, [_c_p] * 5 + [ctypes.c_uint64, ctypes.c_uint64,
                                                    ctypes.c_int64] + [_c_p] * 6
                        + [ctypes.c_size_t, _c_p]),
    "moe_check_wait_timeout": (ctypes.c_int, [_c_p, ctypes.c_size_t, ctypes.c_uint32, _c_p]),
    "moe_expert_backward_workspace_size": (ctypes.c_size_t, [_c_p]),
    "moe_expert_ffn_backward": (ctypes.c_int, [_c_p] * 12 + [ctypes.c_size_t, _c_p]),
    "moe_expert_ffn_backward_saved": (ctypes.c_int, [_c_p] * 12 + [ctypes.c_size_t, _c_p]),
    "moe_expert_ffn_train": (ctypes.c_int, [_c_p] * 8 + [ctypes.c_size_t, _c_p, ctypes.c_size_t,
                                                          _c_p]),
    "moe_permute_backward": (ctypes.c_int, [_c_p] * 6),
    "moe_combine_backward": (ctypes.c_int, [_c_p] * 8),
    "moe_route_backward": (ctypes.c_int, [_c_p] * 9 + [ctypes.c_int32] + [_c_p] * 5 +
                           [ctypes.c_size_t, _c_p]),
    "moe_gate_noise": (ctypes.c_int, [_c_p] * 3 + [ctypes.c_uint64, ctypes.c_uint64,
                                                   ctypes.c_int64, _c_p, _c_p, ctypes.c_size_t,
                                                   _c_p]),
    "moe_dispatch": (ctypes.c_int, [_c_p] * 13 + [ctypes.c_size_t, _c_p]),
    "moe_dispatch_count": (ctypes.c_int, [_c_p] * 4 + [ctypes.c_size_t, _c_p]),
    "moe_shard_record": (ctypes.c_int, [_c_p] * 5 + [ctypes.c_size_t, _c_p]),
    "moe_dispatch_shard": (ctypes.c_int, [_c_p] * 14 + [ctypes.c_size_t, _c_p]),
    "moe_expert_ffn": (ctypes.c_int, [_c_p] * 8 + [ctypes.c_size_t, _c_p]),
    "moe_expert_ffn_gather": (ctypes.c_int, [_c_p] * 9 + [ctypes.c_size_t, _c_p]),
    "moe_combine": (ctypes.c_int, [_c_p] * 6),
    "moe_expert_ffn_combine": (ctypes.c_int, [_c_p] * 11 + [ctypes.c_size_t, _c_p]),
    "moe_forward_combine_fused": (ctypes.c_int, [_c_p, _c_p]),
    "moe_forward": (ctypes.c_int, [_c_p] * 15 + [ctypes.c_size_t, _c_p]),
    "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_last_error_message": (ctypes.c_char_p, []),
}

# Every symbol include/moe_packed.h declares.
_PACKED_SIGNATURES = {
    "moe_balance_workspace_size": (ctypes.c_size_t, [_c_p, ctypes.c_int32]),
    "moe_balance_loss": (ctypes.c_int, [_c_p, ctypes.c_int32] + [_c_p] * 9
                         + [ctypes.c_size_t, _c_p]),
    "moe_balance_loss_backward": (ctypes.c_int, [_c_p, ctypes.c_int32] + [_c_p] * 8
                                  + [ctypes.c_size_t, _c_p]),
    "moe_route_backward_add": (ctypes.c_int, [_c_p] * 9 + [ctypes.c_int32] + [_c_p] * 6 +
                               [ctypes.c_size_t, _c_p]),
    "moe_dropout": (ctypes.c_int, [_c_p] * 2 + [ctypes.c_int32] * 2 + [_c_p] * 4),
    "moe_combine_dropout": (ctypes.c_int, [_c_p] * 8),
    "moe_combine_dropout_backward": (ctypes.c_int, [_c_p] * 9),
    "moe_adapter_plan_size": (ctypes.c_size_t, [_c_p, ctypes.c_int32]),
    "moe_adapter_plan": (ctypes.c_int, [_c_p, ctypes.c_int32, _c_p, _c_p, ctypes.c_size_t, _c_p]),
    "moe_adapter": (ctypes.c_int, [_c_p] + [ctypes.c_int32] * 2 + [_c_p, ctypes.c_size_t]
                    + [_c_p] * 8),
    "moe_adapter_workspace_size": (ctypes.c_size_t, [_c_p] + [ctypes.c_int32] * 2),
    "moe_adapter_backward": (ctypes.c_int, [_c_p] + [ctypes.c_int32] * 2
                             + [_c_p, ctypes.c_size_t] + [_c_p] * 11 + [ctypes.c_size_t, _c_p]),
}


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        super().__init__(f"{where}: status {status} ({message})")
        self.status = status


class MoeConfig(ctypes.Structure):
    """Mirror of ``moe_config_t``."""
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("d_hidden", ctypes.c_int32),
                ("d_out", ctypes.c_int32), ("E", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("expert_kind", ctypes.c_int32), ("act_dtype", ctypes.c_int32),
                ("capacity_factor", ctypes.c_float)]


class MoeShard(ctypes.Structure):
    """Mirror of ``moe_shard_t``: this rank of a batch split over ranks and
    every rank's exchange record (world, 2E+1) int32."""
    _fields_ = [("rank", ctypes.c_int32), ("world", ctypes.c_int32), ("T_global", ctypes.c_int32),
                ("records", ctypes.c_void_p)]


class MoeDropout(ctypes.Structure):
    """Mirror of ``moe_dropout_t``."""
    _fields_ = [("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("offset_dev", ctypes.c_void_p), ("token_base", ctypes.c_int64)]


def make_config(T: int, d: int, d_hidden: int, d_out: int, E: int, top_k: int, kind: str,
                dtype: str, capacity_factor: float = 0.0) -> MoeConfig:
    return MoeConfig(T, d, d_hidden, d_out, E, top_k, EXPERT_KINDS[kind], DTYPES[dtype],
                     float(capacity_factor))


def router_tc_width_supported(cfg: "MoeConfig") -> bool:
    """Whether the tensor-core router (and moe_gate_noise) serves `cfg`:
    bf16 activations and at most 64 experts."""
    return cfg.act_dtype == DTYPES["bf16"] and cfg.E <= 64


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the library once; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"{LIB_NAME} not found at {path}: build it with "
                               "`python -m mixture_experts_top_b200.build` (needs nvcc)")
        lib = ctypes.CDLL(path)
        for name, (res, args) in {**_SIGNATURES, **_PACKED_SIGNATURES}.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def exported_symbols() -> list:
    """The entry points of include/moe.h."""
    return list(_SIGNATURES)


def packed_symbols() -> list:
    """The entry points of include/moe_packed.h."""
    return list(_PACKED_SIGNATURES)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor arguments must be CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    import torch
    if stream is None:   # the handle alone: a Stream object costs 3 us a call
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _check(status: int, where: str) -> None:
    if status != MOE_OK:
        lib = load_library()
        msg = lib.moe_last_error_message().decode() or lib.moe_status_string(status).decode()
        raise MoeError(status, where, msg)


def moe_workspace_size(cfg: MoeConfig) -> int:
    n = load_library().moe_workspace_size(ctypes.byref(cfg))
    if n == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, "moe_workspace_size",
                       load_library().moe_last_error_message().decode())
    return n


def moe_workspace_init(ws, stream=None) -> None:
    _check(load_library().moe_workspace_init(_ptr(ws), ws.numel(), _stream(stream)),
           "moe_workspace_init")


def moe_device_status(ws, stream=None) -> int:
    code = ctypes.c_int32(0)
    st = load_library().moe_device_status(_ptr(ws), ws.numel(), ctypes.byref(code), _stream(stream))
    if st not in (MOE_OK, MOE_ERR_DEVICE_CHECK):
        _check(st, "moe_device_status")
    return int(code.value)


def alloc_workspace(cfg: MoeConfig, device="cuda", stream=None):
    """Caller-owned workspace as a torch uint8 tensor, error word cleared."""
    import torch
    ws = torch.empty(moe_workspace_size(cfg), dtype=torch.uint8, device=device)
    moe_workspace_init(ws, stream)
    return ws


def moe_route(cfg, x, W_router, logit_bias, noise, expert_indices, gates, prob_mean, logits_out,
              ws, stream=None) -> None:
    _check(load_library().moe_route(
        ctypes.byref(cfg), _ptr(x), _ptr(W_router), _ptr(logit_bias), _ptr(noise),
        _ptr(expert_indices), _ptr(gates), _ptr(prob_mean), _ptr(logits_out), _ptr(ws),
        ws.numel(), _stream(stream)), "moe_route")


def moe_route_noisy(cfg, x, W_router, logit_bias, W_noise, seed, offset, token_base,
                    expert_indices, gates, prob_mean, logits_out, noise_out, ws,
                    stream=None) -> None:
    _check(load_library().moe_route_noisy(
        ctypes.byref(cfg), _ptr(x), _ptr(W_router), _ptr(logit_bias), _ptr(W_noise), int(seed),
        int(offset), int(token_base), _ptr(expert_indices), _ptr(gates), _ptr(prob_mean),
        _ptr(logits_out), _ptr(noise_out), _ptr(ws), ws.numel(), _stream(stream)),
        "moe_route_noisy")


def moe_route_noalloc(cfg, x, W_router, logit_bias, noise, expert_indices, gates, prob_mean,
                      logits_out, stream=None) -> None:
    """moe_route for callers that cannot allocate: no workspace argument;
    the library's fixed scratch array is used (see include/moe.h)."""
    _check(load_library().moe_route_noalloc(
        ctypes.byref(cfg), _ptr(x), _ptr(W_router), _ptr(logit_bias), _ptr(noise),
        _ptr(expert_indices), _ptr(gates), _ptr(prob_mean), _ptr(logits_out), _stream(stream)),
        "moe_route_noalloc")


def moe_combine_backward(cfg, dy, y_perm, dest, gates, dy_perm, dgates, stream=None) -> None:
    _check(load_library().moe_combine_backward(
        ctypes.byref(cfg), _ptr(dy), _ptr(y_perm), _ptr(dest), _ptr(gates), _ptr(dy_perm),
        _ptr(dgates), _stream(stream)), "moe_combine_backward")


def moe_route_backward(cfg, x, W_router, logits, expert_indices, gates, f, dgates, daux, T_batch,
                       dx, dW_router, dbias, dlogits, ws, stream=None) -> None:
    _check(load_library().moe_route_backward(
        ctypes.byref(cfg), _ptr(x), _ptr(W_router), _ptr(logits), _ptr(expert_indices),
        _ptr(gates), _ptr(f), _ptr(dgates), _ptr(daux), int(T_batch), _ptr(dx), _ptr(dW_router),
        _ptr(dbias), _ptr(dlogits), _ptr(ws), ws.numel(), _stream(stream)), "moe_route_backward")


def moe_expert_backward_workspace_size(cfg: MoeConfig) -> int:
    n = load_library().moe_expert_backward_workspace_size(ctypes.byref(cfg))
    if n == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, "moe_expert_backward_workspace_size",
                       load_library().moe_last_error_message().decode())
    return n


def alloc_backward_workspace(cfg: MoeConfig, device="cuda", stream=None):
    """Caller-owned workspace of moe_expert_ffn_backward, error word cleared."""
    import torch
    ws = torch.empty(moe_expert_backward_workspace_size(cfg), dtype=torch.uint8, device=device)
    moe_workspace_init(ws, stream)
    return ws


def moe_expert_ffn_backward(cfg, x_perm, offsets, W_in, W_up, W_out, dy_perm, dx_perm, dW_in,
                            dW_up, dW_out, ws, stream=None) -> None:
    _check(load_library().moe_expert_ffn_backward(
        ctypes.byref(cfg), _ptr(x_perm), _ptr(offsets), _ptr(W_in), _ptr(W_up), _ptr(W_out),
        _ptr(dy_perm), _ptr(dx_perm), _ptr(dW_in), _ptr(dW_up), _ptr(dW_out), _ptr(ws),
        ws.numel(), _stream(stream)), "moe_expert_ffn_backward")


def moe_permute_backward(cfg, dx_perm, dest, dx_add, dx, stream=None) -> None:
    _check(load_library().moe_permute_backward(
        ctypes.byref(cfg), _ptr(dx_perm), _ptr(dest), _ptr(dx_add), _ptr(dx), _stream(stream)),
        "moe_permute_backward")


def moe_check_wait_timeout(ws, limit_us: int, stream=None) -> None:
    _check(load_library().moe_check_wait_timeout(_ptr(ws), ws.numel(), int(limit_us),
                                                  _stream(stream)), "moe_check_wait_timeout")


def moe_gate_noise(cfg, x, W_noise, seed, offset, token_base, noise_out, ws, stream=None) -> None:
    _check(load_library().moe_gate_noise(
        ctypes.byref(cfg), _ptr(x), _ptr(W_noise), int(seed), int(offset), int(token_base),
        _ptr(noise_out), _ptr(ws), ws.numel(), _stream(stream)), "moe_gate_noise")


def moe_dispatch(cfg, x, expert_indices, prob_mean, counts, offsets, dest, perm_token, drop_mask,
                 f, aux_loss, x_perm, ws, stream=None) -> None:
    _check(load_library().moe_dispatch(
        ctypes.byref(cfg), _ptr(x), _ptr(expert_indices), _ptr(prob_mean), _ptr(counts),
        _ptr(offsets), _ptr(dest), _ptr(perm_token), _ptr(drop_mask), _ptr(f), _ptr(aux_loss),
        _ptr(x_perm), _ptr(ws), ws.numel(), _stream(stream)), "moe_dispatch")


def moe_dispatch_count(cfg, expert_indices, counts, ws, stream=None) -> None:
    _check(load_library().moe_dispatch_count(
        ctypes.byref(cfg), _ptr(expert_indices), _ptr(counts), _ptr(ws), ws.numel(),
        _stream(stream)), "moe_dispatch_count")


def moe_shard_record(cfg, expert_indices, prob_mean, record, ws, stream=None) -> None:
    _check(load_library().moe_shard_record(
        ctypes.byref(cfg), _ptr(expert_indices), _ptr(prob_mean), _ptr(record), _ptr(ws),
        ws.numel(), _stream(stream)), "moe_shard_record")


def moe_dispatch_shard(cfg, rank, world, T_global, records, x, expert_indices, prob_mean,
                       counts, offsets, dest, perm_token, drop_mask, f, aux_loss, x_perm, ws,
                       stream=None) -> None:
    shard = MoeShard(rank, world, T_global, _ptr(records))
    _check(load_library().moe_dispatch_shard(
        ctypes.byref(cfg), ctypes.byref(shard), _ptr(x), _ptr(expert_indices), _ptr(prob_mean),
        _ptr(counts), _ptr(offsets), _ptr(dest), _ptr(perm_token), _ptr(drop_mask), _ptr(f),
        _ptr(aux_loss), _ptr(x_perm), _ptr(ws), ws.numel(), _stream(stream)),
        "moe_dispatch_shard")


def moe_expert_ffn_backward_saved(cfg, x_perm, offsets, W_in, W_up, W_out, dy_perm, dx_perm,
                                  dW_in, dW_up, dW_out, ws, stream=None) -> None:
    """moe_expert_ffn_backward with the pre-activations that
    moe_expert_ffn_train left in `ws`."""
    _check(load_library().moe_expert_ffn_backward_saved(
        ctypes.byref(cfg), _ptr(x_perm), _ptr(offsets), _ptr(W_in), _ptr(W_up), _ptr(W_out),
        _ptr(dy_perm), _ptr(dx_perm), _ptr(dW_in), _ptr(dW_up), _ptr(dW_out), _ptr(ws),
        ws.numel(), _stream(stream)), "moe_expert_ffn_backward_saved")


def moe_expert_ffn_train(cfg, x_perm, offsets, W_in, W_up, W_out, y_perm, ws, bwd_ws,
                         stream=None) -> None:
    """moe_expert_ffn that also keeps the pre-activations in bwd_ws (the
    experts' backward workspace)."""
    _check(load_library().moe_expert_ffn_train(
        ctypes.byref(cfg), _ptr(x_perm), _ptr(offsets), _ptr(W_in), _ptr(W_up), _ptr(W_out),
        _ptr(y_perm), _ptr(ws), ws.numel(), _ptr(bwd_ws), bwd_ws.numel(), _stream(stream)),
        "moe_expert_ffn_train")


def moe_expert_ffn(cfg, x_perm, offsets, W_in, W_up, W_out, y_perm, ws, stream=None) -> None:
    _check(load_library().moe_expert_ffn(
        ctypes.byref(cfg), _ptr(x_perm), _ptr(offsets), _ptr(W_in), _ptr(W_up), _ptr(W_out),
        _ptr(y_perm), _ptr(ws), ws.numel(), _stream(stream)), "moe_expert_ffn")


def moe_expert_ffn_gather(cfg, x, perm_token, offsets, W_in, W_up, W_out, y_perm, ws,
                          stream=None) -> None:
    _check(load_library().moe_expert_ffn_gather(
        ctypes.byref(cfg), _ptr(x), _ptr(perm_token), _ptr(offsets), _ptr(W_in), _ptr(W_up),
        _ptr(W_out), _ptr(y_perm), _ptr(ws), ws.numel(), _stream(stream)), "moe_expert_ffn_gather")


def moe_expert_ffn_combine(cfg, x_perm, offsets, perm_token, dest, gates, W_in, W_up, W_out,
                           output, ws, stream=None) -> None:
    _check(load_library().moe_expert_ffn_combine(
        ctypes.byref(cfg), _ptr(x_perm), _ptr(offsets), _ptr(perm_token), _ptr(dest), _ptr(gates),
        _ptr(W_in), _ptr(W_up), _ptr(W_out), _ptr(output), _ptr(ws), ws.numel(), _stream(stream)),
        "moe_expert_ffn_combine")


def moe_forward_combine_fused(cfg) -> bool:
    """Whether moe_forward runs the combine in the down projection's epilogue
    (moe_expert_ffn_combine) for cfg, rather than moe_expert_ffn then
    moe_combine.  Host-only."""
    out = ctypes.c_int32(0)
    _check(load_library().moe_forward_combine_fused(ctypes.byref(cfg), ctypes.byref(out)),
           "moe_forward_combine_fused")
    return bool(out.value)


def moe_combine(cfg, y_perm, dest, gates, output, stream=None) -> None:
    _check(load_library().moe_combine(
        ctypes.byref(cfg), _ptr(y_perm), _ptr(dest), _ptr(gates), _ptr(output), _stream(stream)),
        "moe_combine")


def moe_forward(cfg, x, W_router, logit_bias, noise, W_in, W_up, W_out, output, expert_indices,
                gates, aux_loss, counts, drop_mask, ws, stream=None) -> None:
    _check(load_library().moe_forward(
        ctypes.byref(cfg), _ptr(x), _ptr(W_router), _ptr(logit_bias), _ptr(noise), _ptr(W_in),
        _ptr(W_up), _ptr(W_out), _ptr(output), _ptr(expert_indices), _ptr(gates), _ptr(aux_loss),
        _ptr(counts), _ptr(drop_mask), _ptr(ws), ws.numel(), _stream(stream)), "moe_forward")


# ---- packed batches: balance loss per sequence, dropout, low-rank adapters ----
#
# These calls take many tensors of related shapes, so the binding checks each
# one's type, shape and device before the library sees its pointer.

def _arg(t, name: str, dtype, shape, dev: int) -> Optional[int]:
    """Pointer of a contiguous tensor of this type and shape (None: any) on
    CUDA device `dev`, the current one.  No tensor is NULL, which the library
    takes for an optional argument and refuses by name for another."""
    if t is None:
        return None
    if (t.dtype is dtype and (shape is None or t.shape == shape) and t.get_device() == dev
            and t.is_contiguous()):
        return t.data_ptr()
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{name} must be on the current CUDA device")
    raise ValueError(f"{name} must be contiguous")


def _buf(t, name: str, u8, dev: int):
    """Pointer and bytes of a workspace or plan."""
    return _arg(t, name, u8, None, dev), 0 if t is None else t.numel()


def _mask(t, T: int, dev: int) -> Optional[int]:
    """A token mask: uint8, or bool (bytes of 0 and 1)."""
    if t is None:
        return None
    import torch
    return _arg(t, "token_mask", torch.bool if t.dtype is torch.bool else torch.uint8, (T,), dev)


def _not_null(t, name: str, where: str) -> None:
    """The library's refusal, for a tensor whose type or shape is read before the call."""
    if t is None:
        raise MoeError(MOE_ERR_INVALID_ARG, where, f"{name} is NULL")


def _where(stream):
    """The current device, which the call's tensors must be on (-2, no tensor's
    device, before CUDA is initialised), and the stream's handle."""
    import torch
    if not torch.cuda.is_initialized():
        return -2, None
    dev = torch.cuda.current_device()
    return dev, (torch._C._cuda_getCurrentRawStream(dev) if stream is None
                 else stream.cuda_stream)


def _act(cfg):
    import torch
    return torch.bfloat16 if cfg.act_dtype == DTYPES["bf16"] else torch.float32


def _seqs(seq_offsets, i32, dev):
    """Number of sequences and the offsets' pointer (None: one sequence)."""
    if seq_offsets is None:
        return 1, None
    if seq_offsets.dim() != 1:
        raise ValueError("seq_offsets must have one dimension")
    return seq_offsets.numel() - 1, _arg(seq_offsets, "seq_offsets", i32, None, dev)


def _sized(n: int, where: str) -> int:
    if n == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, where,
                       load_library().moe_last_error_message().decode())
    return n


def _alloc(n: int, device, stream):
    import torch
    buf = torch.empty(n, dtype=torch.uint8, device=device)
    moe_workspace_init(buf, stream)
    return buf


def moe_balance_workspace_size(cfg: MoeConfig, n_seqs: int) -> int:
    return _sized(load_library().moe_balance_workspace_size(ctypes.byref(cfg), int(n_seqs)),
                  "moe_balance_workspace_size")


def alloc_balance_workspace(cfg: MoeConfig, n_seqs: int, device="cuda", stream=None):
    """Workspace of moe_balance_loss for n_seqs sequences, error word cleared."""
    return _alloc(moe_balance_workspace_size(cfg, n_seqs), device, stream)


def moe_balance_loss(cfg, seq_offsets, token_mask, logits, expert_indices, counts, prob_mean,
                     tokens, losses, ws, stream=None) -> None:
    """seq_offsets (n_seqs+1) int32 or None (one sequence: all tokens);
    token_mask (T) uint8 or bool, or None; see include/moe_packed.h for the outputs."""
    import torch
    f32, i32 = torch.float32, torch.int32
    dev, st = _where(stream)
    n, off = _seqs(seq_offsets, i32, dev)
    T, E = cfg.T, cfg.E
    wp, wn = _buf(ws, "ws", torch.uint8, dev)
    _check(load_library().moe_balance_loss(
        ctypes.byref(cfg), n, off, _mask(token_mask, T, dev),
        _arg(logits, "logits", f32, (T, E), dev),
        _arg(expert_indices, "expert_indices", i32, (T, cfg.top_k), dev),
        _arg(counts, "counts", i32, (n, E), dev), _arg(prob_mean, "prob_mean", f32, (n, E), dev),
        _arg(tokens, "tokens", i32, (n + 2,), dev), _arg(losses, "losses", f32, (2,), dev), wp, wn,
        st), "moe_balance_loss")


def moe_balance_loss_backward(cfg, seq_offsets, token_mask, logits, counts, tokens, dlosses,
                              dlogits, ws, stream=None) -> None:
    import torch
    f32, i32 = torch.float32, torch.int32
    dev, st = _where(stream)
    n, off = _seqs(seq_offsets, i32, dev)
    T, E = cfg.T, cfg.E
    wp, wn = _buf(ws, "ws", torch.uint8, dev)
    _check(load_library().moe_balance_loss_backward(
        ctypes.byref(cfg), n, off, _mask(token_mask, T, dev),
        _arg(logits, "logits", f32, (T, E), dev), _arg(counts, "counts", i32, (n, E), dev),
        _arg(tokens, "tokens", i32, (n + 2,), dev), _arg(dlosses, "dlosses", f32, (2,), dev),
        _arg(dlogits, "dlogits", f32, (T, E), dev), wp, wn, st),
        "moe_balance_loss_backward")


def moe_route_backward_add(cfg, x, W_router, logits, expert_indices, gates, f, dgates, daux,
                           T_batch, dlogits_add, dx, dW_router, dbias, dlogits, ws,
                           stream=None) -> None:
    """moe_route_backward with dlogits_add (T, E) fp32 added to the logits' gradient."""
    import torch
    dev, st = _where(stream)
    add = _arg(dlogits_add, "dlogits_add", torch.float32, (cfg.T, cfg.E), dev)
    _check(load_library().moe_route_backward_add(
        ctypes.byref(cfg), _ptr(x), _ptr(W_router), _ptr(logits), _ptr(expert_indices),
        _ptr(gates), _ptr(f), _ptr(dgates), _ptr(daux), int(T_batch), add, _ptr(dx),
        _ptr(dW_router), _ptr(dbias), _ptr(dlogits), _ptr(ws), 0 if ws is None else ws.numel(), st),
        "moe_route_backward_add")


def _drop(p, seed, offset, token_base, dev):
    """moe_dropout_t; offset is an int, or a one-element int64 CUDA tensor that
    the kernel reads when it runs (fresh masks from one captured graph)."""
    if isinstance(offset, int):
        return MoeDropout(p, seed, offset, None, token_base)
    import torch
    return MoeDropout(p, seed, 0, _arg(offset, "offset", torch.int64, (1,), dev), token_base)


def moe_dropout(cfg, p, seed, offset, token_base, x, add, out, stream=None) -> None:
    """out = add + dropout(x) over (T, width) rows, bf16 or fp32; add may be
    None, out may be x or add."""
    import torch
    _not_null(x, "x", "moe_dropout")
    dt, shape = x.dtype, x.shape
    if dt is not torch.bfloat16 and dt is not torch.float32:
        raise ValueError(f"x must be bfloat16 or float32, got {dt}")
    if len(shape) != 2 or shape[0] != cfg.T:
        raise ValueError(f"x must have shape ({cfg.T}, width), got {tuple(shape)}")
    dev, st = _where(stream)
    d = _drop(p, seed, offset, token_base, dev)
    _check(load_library().moe_dropout(
        ctypes.byref(cfg), ctypes.byref(d), shape[1],
        DTYPES["bf16"] if dt is torch.bfloat16 else DTYPES["f32"], _arg(x, "x", dt, None, dev),
        _arg(add, "add", dt, shape, dev), _arg(out, "out", dt, shape, dev), st),
        "moe_dropout")


def moe_combine_dropout(cfg, p, seed, offset, token_base, y_perm, dest, gates, residual, output,
                        stream=None) -> None:
    """moe_combine with dropout, plus residual (or None) added after it."""
    import torch
    f32, act, T, k, w = torch.float32, _act(cfg), cfg.T, cfg.top_k, cfg.d_out
    dev, st = _where(stream)
    d = _drop(p, seed, offset, token_base, dev)
    _check(load_library().moe_combine_dropout(
        ctypes.byref(cfg), ctypes.byref(d), _arg(y_perm, "y_perm", f32, (T * k, w), dev),
        _arg(dest, "dest", torch.int32, (T, k), dev), _arg(gates, "gates", f32, (T, k), dev),
        _arg(residual, "residual", act, (T, w), dev), _arg(output, "output", act, (T, w), dev),
        st), "moe_combine_dropout")


def moe_combine_dropout_backward(cfg, p, seed, offset, token_base, dy, y_perm, dest, gates,
                                 dy_perm, dgates, stream=None) -> None:
    import torch
    f32, act, T, k, w = torch.float32, _act(cfg), cfg.T, cfg.top_k, cfg.d_out
    dev, st = _where(stream)
    d = _drop(p, seed, offset, token_base, dev)
    _check(load_library().moe_combine_dropout_backward(
        ctypes.byref(cfg), ctypes.byref(d), _arg(dy, "dy", act, (T, w), dev),
        _arg(y_perm, "y_perm", f32, (T * k, w), dev), _arg(dest, "dest", torch.int32, (T, k), dev),
        _arg(gates, "gates", f32, (T, k), dev), _arg(dy_perm, "dy_perm", f32, (T * k, w), dev),
        _arg(dgates, "dgates", f32, (T, k), dev), st), "moe_combine_dropout_backward")


def moe_adapter_plan_size(cfg: MoeConfig, n_adapters: int) -> int:
    return _sized(load_library().moe_adapter_plan_size(ctypes.byref(cfg), int(n_adapters)),
                  "moe_adapter_plan_size")


def moe_adapter_workspace_size(cfg: MoeConfig, n_adapters: int, rank: int) -> int:
    return _sized(load_library().moe_adapter_workspace_size(ctypes.byref(cfg), int(n_adapters),
                                                            int(rank)),
                  "moe_adapter_workspace_size")


def alloc_adapter_plan(cfg: MoeConfig, n_adapters: int, device="cuda", stream=None):
    """Buffer of moe_adapter_plan, error word cleared."""
    return _alloc(moe_adapter_plan_size(cfg, n_adapters), device, stream)


def alloc_adapter_workspace(cfg: MoeConfig, n_adapters: int, rank: int, device="cuda"):
    """Workspace of moe_adapter_backward."""
    import torch
    return torch.empty(moe_adapter_workspace_size(cfg, n_adapters, rank), dtype=torch.uint8,
                       device=device)


def moe_adapter_plan(cfg, n_adapters, token_adapter, plan, stream=None) -> None:
    """Groups the tokens by adapter: token_adapter (T) int32, negative for none."""
    import torch
    dev, st = _where(stream)
    pp, pn = _buf(plan, "plan", torch.uint8, dev)
    _check(load_library().moe_adapter_plan(
        ctypes.byref(cfg), int(n_adapters),
        _arg(token_adapter, "token_adapter", torch.int32, (cfg.T,), dev), pp, pn, st),
        "moe_adapter_plan")


def _adapter_shape(cfg, A, where):
    _not_null(A, "A", where)
    if A.dim() != 3 or A.shape[1] != cfg.d:
        raise ValueError(f"A must have shape (n_adapters, {cfg.d}, rank), got {tuple(A.shape)}")
    return A.shape[0], A.shape[2]


def moe_adapter(cfg, plan, x, A, B, scale, base, output, u, stream=None) -> None:
    """output = base + scale x A B by each token's adapter; base and u may be None."""
    import torch
    bf, f32, T, w = torch.bfloat16, torch.float32, cfg.T, cfg.d_out
    n, r = _adapter_shape(cfg, A, "moe_adapter")
    dev, st = _where(stream)
    pp, pn = _buf(plan, "plan", torch.uint8, dev)
    _check(load_library().moe_adapter(
        ctypes.byref(cfg), n, r, pp, pn, _arg(x, "x", bf, (T, cfg.d), dev),
        _arg(A, "A", bf, None, dev),
        _arg(B, "B", bf, (n, r, w), dev), _arg(scale, "scale", f32, (n,), dev),
        _arg(base, "base", bf, (T, w), dev), _arg(output, "output", bf, (T, w), dev),
        _arg(u, "u", f32, (T, r), dev), st), "moe_adapter")


def moe_adapter_backward(cfg, plan, x, u, dy, A, B, scale, dx_add, dx, dA, dB, ws,
                         stream=None) -> None:
    import torch
    bf, f32, T, w = torch.bfloat16, torch.float32, cfg.T, cfg.d_out
    n, r = _adapter_shape(cfg, A, "moe_adapter_backward")
    dev, st = _where(stream)
    pp, pn = _buf(plan, "plan", torch.uint8, dev)
    wp, wn = _buf(ws, "ws", torch.uint8, dev)
    _check(load_library().moe_adapter_backward(
        ctypes.byref(cfg), n, r, pp, pn, _arg(x, "x", bf, (T, cfg.d), dev),
        _arg(u, "u", f32, (T, r), dev),
        _arg(dy, "dy", bf, (T, w), dev), _arg(A, "A", bf, None, dev),
        _arg(B, "B", bf, (n, r, w), dev),
        _arg(scale, "scale", f32, (n,), dev), _arg(dx_add, "dx_add", f32, (T, cfg.d), dev),
        _arg(dx, "dx", f32, (T, cfg.d), dev), _arg(dA, "dA", f32, A.shape, dev),
        _arg(dB, "dB", f32, (n, r, w), dev), wp, wn, st), "moe_adapter_backward")
