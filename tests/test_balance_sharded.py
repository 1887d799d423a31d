"""The balance loss of a batch split over ranks in whole sequences: every rank's
losses weighted by its share of the sequences and of the tokens give the whole
batch's, and its gradient for dlosses scaled by the same shares is its rows of the
whole batch's."""
import numpy as np
import pytest
import torch

from mixture_experts_top_b200 import api
from oracle import packed_oracle as Q

U = 2.0 ** -24
T, E, K = 700, 16, 2
OFF = np.array([0, 90, 90, 300, 301, 480, 640, 690], np.int32)   # the last tokens: none's
CUTS = [0, 2, 3, 7]                                              # ranks by sequences


def _case():
    rng = np.random.default_rng(4)
    L = np.clip(rng.standard_normal((T, E)) * 2, -5, 5).astype(np.float32)
    idx = np.argsort(-L, axis=1, kind="stable")[:, :K].astype(np.int32)
    mask = (rng.random(T) < 0.8).astype(np.uint8)
    mask[300] = 0                                                # a sequence without a counted token
    return L, idx, mask


def _ranks():
    """Rows and local offsets of each rank; the last one also has the rows of no sequence."""
    for a, b in zip(CUTS[:-1], CUTS[1:]):
        lo, hi = int(OFF[a]), int(OFF[b]) if b < len(OFF) - 1 else T
        yield lo, hi, OFF[a:b + 1] - lo


def test_oracle():
    L, idx, mask = _case()
    whole = Q.balance_loss(L, idx, E, OFF, mask)
    N, live = whole["tokens"][-2:]
    dl = (0.7, 0.3)
    grad = Q.balance_loss_backward(L, idx, E, OFF, mask, *dl)
    balance = z = 0.0
    for lo, hi, off in _ranks():
        r = Q.balance_loss(L[lo:hi], idx[lo:hi], E, off, mask[lo:hi])
        n, s = r["tokens"][-2:]
        balance, z = balance + s / live * r["balance"], z + n / N * r["z"]
        g = Q.balance_loss_backward(L[lo:hi], idx[lo:hi], E, off, mask[lo:hi], dl[0] * s / live,
                                    dl[1] * n / N)
        assert np.allclose(g, grad[lo:hi], rtol=1e-12, atol=1e-18)
    assert abs(balance - whole["balance"]) < 1e-12 and abs(z - whole["z"]) < 1e-12


@pytest.mark.gpu
def test_device():
    """tokens is on the device on every rank: its last two entries, added over the
    ranks, give the shares without a copy to the host."""
    L, idx, mask = _case()
    i32 = dict(dtype=torch.int32, device="cuda")

    def run(lo, hi, off, scale=None):
        n, S = hi - lo, len(off) - 1
        cfg = api.make_config(n, 8, 8, 8, E, K, "swiglu", "bf16")
        ws = api.alloc_balance_workspace(cfg, S)
        o, m, l, ix = (torch.from_numpy(np.ascontiguousarray(v)).cuda()
                       for v in (off, mask[lo:hi], L[lo:hi], idx[lo:hi]))
        c, P = torch.empty((S, E), **i32), torch.empty((S, E), device="cuda")
        tok, loss, g = torch.empty(S + 2, **i32), torch.empty(2, device="cuda"), torch.empty_like(l)
        api.moe_balance_loss(cfg, o, m, l, ix, c, P, tok, loss, ws)
        dl = torch.tensor([0.7, 0.3], device="cuda")
        if scale is not None:
            dl *= tok[-2:].flip(0) / scale                       # (S+, N) shares
        api.moe_balance_loss_backward(cfg, o, m, l, c, tok, dl, g, ws)
        assert api.moe_device_status(ws) == 0
        return loss.double(), tok[-2:].flip(0), g.double()

    loss, total, grad = run(0, T, OFF)
    shards = [run(lo, hi, off, total) for lo, hi, off in _ranks()]
    assert torch.equal(sum(s[1] for s in shards), total)
    got = sum(s[0] * (s[1].double() / total) for s in shards)
    # each side within 200 units of exact (test_gpu_balance_layouts.py), the share's and
    # the scaled dlosses' roundings 4
    assert torch.all((got - loss).abs() <= 404 * U * loss.clamp(min=1.0))
    g = torch.cat([s[2] for s in shards])
    assert torch.all((g - grad).abs() <= 404 * U * grad.abs().amax(dim=1, keepdim=True) + 1e-37)
