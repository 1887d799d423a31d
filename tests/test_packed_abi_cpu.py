"""Argument checks of the packed-batch calls: every refusal comes from the
host, before any CUDA call, so this file needs no GPU.  Pointers are host
addresses that are never followed."""
import ctypes
import os
import re

import pytest
import torch

from mixture_experts_top_b200 import api

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = 1 << 20            # a 256-byte aligned address, never dereferenced
ODD = P + 8            # not on a 16-byte boundary


def _cfg(T=64, d=64, d_out=64, E=8, k=2, dtype="bf16"):
    return api.make_config(T, d, 64, d_out, E, k, "swiglu" if dtype == "bf16" else "linear", dtype)


def _drop(p=0.1, token_base=0, offset_dev=None):
    return api.MoeDropout(p, 1, 2, offset_dev, token_base)


def _call(lib, name, cfg, *args):
    return getattr(lib, name)(ctypes.byref(cfg) if cfg is not None else None, *args)


def test_every_declared_symbol_is_exported(moe_lib):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "moe_packed.h")).read(),
                  flags=re.S)
    names = sorted(set(re.findall(r"\b(moe_[a-z_]+)\s*\(", text)))
    assert names == sorted(api.packed_symbols()) and len(names) == 12
    for n in names:
        assert hasattr(moe_lib, n), n


def test_balance_refusals(moe_lib):
    f = lambda cfg=_cfg(), n=3, off=P, mask=None, logits=P, idx=P, counts=P, pm=P, tok=P, loss=P, \
        ws=P, nb=1 << 40: _call(moe_lib, "moe_balance_loss", cfg, n, off, mask, logits, idx,
                                counts, pm, tok, loss, ws, nb, None)
    for name in ("logits", "idx", "counts", "pm", "tok", "loss"):
        assert f(**{name: None}) == INVALID, name
    assert f(cfg=None) == INVALID
    assert f(n=0) == INVALID and f(n=-1) == INVALID
    assert f(off=None) == INVALID                       # several sequences need offsets
    assert f(ws=None) == WORKSPACE and f(ws=P + 16) == WORKSPACE
    need = api.moe_balance_workspace_size(_cfg(), 3)
    assert f(nb=need - 1) == WORKSPACE
    assert f(cfg=_cfg(T=(1 << 29) + 1), logits=P) == UNSUPPORTED
    assert f(n=(1 << 30) + 1) == UNSUPPORTED
    b = lambda cfg=_cfg(), n=3, off=P, logits=P, counts=P, tok=P, dl=P, out=P, ws=P, nb=1 << 40: \
        _call(moe_lib, "moe_balance_loss_backward", cfg, n, off, None, logits, counts, tok, dl, out,
              ws, nb, None)
    for name in ("logits", "counts", "tok", "dl", "out"):
        assert b(**{name: None}) == INVALID, name
    assert b(n=0) == INVALID and b(off=None) == INVALID
    assert b(nb=need - 1) == WORKSPACE and b(ws=None) == WORKSPACE


def test_balance_workspace_size(moe_lib):
    assert moe_lib.moe_balance_workspace_size(None, 1) == 0
    assert moe_lib.moe_balance_workspace_size(ctypes.byref(_cfg()), 0) == 0
    sizes = [api.moe_balance_workspace_size(_cfg(T=t), 4) for t in (0, 64, 4096, 1 << 20)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    assert api.moe_balance_workspace_size(_cfg(), 1000) > api.moe_balance_workspace_size(_cfg(), 1)
    with pytest.raises(api.MoeError):
        api.moe_balance_workspace_size(_cfg(), 0)


@pytest.mark.parametrize("p", [-0.1, 1.0, 1.5, float("nan"), float("inf"), 1 - 2.0 ** -18])
def test_dropout_probability_refused(moe_lib, p):
    d = _drop(p)
    assert _call(moe_lib, "moe_dropout", _cfg(), ctypes.byref(d), 64, 1, P, None, P, None) == INVALID
    assert _call(moe_lib, "moe_combine_dropout", _cfg(), ctypes.byref(d), P, P, P, None, P,
                 None) == INVALID
    assert _call(moe_lib, "moe_combine_dropout_backward", _cfg(), ctypes.byref(d), P, P, P, P, P, P,
                 None) == INVALID


def test_dropout_refusals(moe_lib):
    d, neg, mis = _drop(), _drop(token_base=-1), _drop(offset_dev=P + 4)
    f = lambda cfg=_cfg(), drop=d, width=64, dtype=1, x=P, add=P, out=P: _call(
        moe_lib, "moe_dropout", cfg, ctypes.byref(drop) if drop is not None else None, width, dtype,
        x, add, out, None)
    assert f(cfg=None) == INVALID and f(drop=None) == INVALID
    assert f(drop=neg) == INVALID and f(drop=mis) == INVALID
    assert f(width=0) == UNSUPPORTED and f(width=12) == UNSUPPORTED and f(width=-8) == UNSUPPORTED
    assert f(dtype=2) == INVALID
    assert f(x=None) == INVALID and f(out=None) == INVALID
    assert f(x=ODD) == INVALID and f(add=ODD) == INVALID and f(out=ODD) == INVALID
    c = lambda y=P, dest=P, gates=P, res=P, out=P, drop=d: _call(
        moe_lib, "moe_combine_dropout", _cfg(), ctypes.byref(drop), y, dest, gates, res, out, None)
    for name in ("y", "dest", "gates", "out"):
        assert c(**{name: None}) == INVALID, name
    assert c(res=ODD) == INVALID and c(drop=neg) == INVALID
    b = lambda dy=P, y=P, dest=P, gates=P, dyp=P, dg=P: _call(
        moe_lib, "moe_combine_dropout_backward", _cfg(), ctypes.byref(d), dy, y, dest, gates, dyp,
        dg, None)
    for name in ("dy", "y", "dest", "gates", "dyp", "dg"):
        assert b(**{name: None}) == INVALID, name
    assert b(dy=ODD) == INVALID


def test_adapter_refusals(moe_lib):
    f = lambda cfg=_cfg(), n=4, r=16, plan=P, nb=1 << 40, x=P, A=P, B=P, s=P, base=P, out=P, u=P: \
        _call(moe_lib, "moe_adapter", cfg, n, r, plan, nb, x, A, B, s, base, out, u, None)
    assert f(cfg=None) == INVALID
    assert f(cfg=_cfg(dtype="f32")) == UNSUPPORTED
    assert f(n=0) == INVALID and f(n=1025) == UNSUPPORTED
    assert f(r=0) == INVALID and f(r=12) == UNSUPPORTED and f(r=136) == UNSUPPORTED
    assert f(plan=None) == WORKSPACE and f(plan=P + 16) == WORKSPACE
    assert f(nb=api.moe_adapter_plan_size(_cfg(), 4) - 1) == WORKSPACE
    for name in ("x", "A", "B", "s", "out"):
        assert f(**{name: None}) == INVALID, name
    for name in ("x", "A", "B", "base", "out", "u"):
        assert f(**{name: ODD}) == INVALID, name
    g = lambda cfg=_cfg(), ids=P, plan=P, nb=1 << 40, n=4: _call(
        moe_lib, "moe_adapter_plan", cfg, n, ids, plan, nb, None)
    assert g(ids=None) == INVALID and g(plan=None) == WORKSPACE and g(nb=8) == WORKSPACE
    assert g(n=0) == INVALID and g(cfg=_cfg(T=(1 << 30) + 8, k=1)) == UNSUPPORTED
    b = lambda plan=P, nb=1 << 40, x=P, u=P, dy=P, A=P, B=P, s=P, add=P, dx=P, dA=P, dB=P, ws=P, \
        wb=1 << 40, r=16: _call(moe_lib, "moe_adapter_backward", _cfg(), 4, r, plan, nb, x, u, dy, A,
                                B, s, add, dx, dA, dB, ws, wb, None)
    for name in ("x", "u", "dy", "A", "B", "s", "dx", "dA", "dB"):
        assert b(**{name: None}) == INVALID, name
    for name in ("x", "u", "dy", "A", "B", "add", "dx", "dA", "dB"):
        assert b(**{name: ODD}) == INVALID, name
    assert b(ws=None) == WORKSPACE
    assert b(wb=api.moe_adapter_workspace_size(_cfg(), 4, 16) - 1) == WORKSPACE
    assert b(plan=None) == WORKSPACE and b(r=20) == UNSUPPORTED


def test_adapter_sizes(moe_lib):
    assert moe_lib.moe_adapter_plan_size(None, 4) == 0
    assert moe_lib.moe_adapter_plan_size(ctypes.byref(_cfg(dtype="f32")), 4) == 0
    assert moe_lib.moe_adapter_workspace_size(ctypes.byref(_cfg()), 4, 12) == 0
    assert api.moe_adapter_plan_size(_cfg(T=4096), 4) > api.moe_adapter_plan_size(_cfg(), 4)


def test_route_backward_add_needs_its_gradient(moe_lib):
    args = [P] * 8
    assert _call(moe_lib, "moe_route_backward_add", _cfg(), *args, 0, None, P, P, P, P, P, 1 << 40,
                 None) == INVALID


def test_binding_refuses_wrong_tensors(moe_lib):
    """The binding names the argument; none of these reaches the library."""
    cfg = _cfg(T=4, d=8, d_out=8)
    bf = torch.zeros(4, 8, dtype=torch.bfloat16)
    buf = torch.zeros(1024, dtype=torch.uint8)
    with pytest.raises(ValueError, match="x must have shape"):
        api.moe_dropout(cfg, 0.1, 0, 0, 0, torch.zeros(3, 8), None, bf)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        api.moe_dropout(cfg, 0.1, 0, 0, 0, torch.zeros(4, 8, dtype=torch.float16), None, bf)
    with pytest.raises(ValueError, match="CUDA device"):
        api.moe_dropout(cfg, 0.1, 0, 0, 0, bf, None, bf)
    with pytest.raises(ValueError, match="offset must be"):
        api.moe_dropout(cfg, 0.1, 0, torch.zeros(1), 0, bf, None, bf)
    with pytest.raises(ValueError, match="A must have shape"):
        api.moe_adapter(cfg, buf, bf, torch.zeros(2, 7, 8), None, None, None, None, None)
    with pytest.raises(ValueError, match="plan must be"):
        api.moe_adapter(cfg, torch.zeros(9), bf, torch.zeros(2, 8, 8), None, None, None, None, None)
    with pytest.raises(ValueError, match="seq_offsets"):
        api.moe_balance_loss(cfg, torch.zeros(3), None, bf, bf, bf, bf, bf, bf, buf)
