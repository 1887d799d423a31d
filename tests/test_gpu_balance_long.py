"""The balance loss on long batches: a chain of fp32 additions covers at most 64
tokens, however long the batch and its sequences are.

Tolerances, in units of 2^-24 (half a step of fp32).  A softmax term 2^((l - m)
log2 e): the subtraction's rounding and the product's (with its constant's) cost
2.3 |l - m| units, the hardware's 2^x 4.  A token's sum of at most 256 terms (16 a
lane, a butterfly of 5): 21; the reciprocal and the product 2; twice the term's
for p.  With |l - m| <= 12 p is within 87 units, P (at most 64
additions in a warp, 3 over a CTA's warps in pairs, two roundings) within 160; the log-sum-exp within 65 units of
max(1, |lse|), z within 200 units of its scale's square.
"""
import numpy as np
import pytest
import torch

from mixture_experts_top_b200 import api

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _run(L, idx, off):
    T, E = L.shape
    k = idx.shape[1]
    cfg = api.make_config(T, 8, 8, 8, E, k, "swiglu", "bf16")
    S = 1 if off is None else off.numel() - 1
    ws = api.alloc_balance_workspace(cfg, S)
    i32 = dict(dtype=torch.int32, device="cuda")
    c, P = torch.empty((S, E), **i32), torch.full((S, E), float("nan"), device="cuda")
    n, loss = torch.empty(S + 2, **i32), torch.full((2,), float("nan"), device="cuda")
    api.moe_balance_loss(cfg, off, None, L, idx, c, P, n, loss, ws)
    assert api.moe_device_status(ws) == 0
    return c, P, n, loss


def _reference(L, idx, off):
    """counts, P, balance, z in fp64 on the device, by sequence."""
    T, E = L.shape
    k = idx.shape[1]
    cuts = [0, T] if off is None else off.tolist()
    counts, P, z = [], [], 0.0
    for lo, hi in zip(cuts[:-1], cuts[1:]):
        rows = L[lo:hi].double()
        lse = torch.logsumexp(rows, 1)
        P.append(torch.exp(rows - lse[:, None]).mean(0))
        z += float((lse ** 2).sum())
        counts.append(torch.bincount(idx[lo:hi].reshape(-1).long(), minlength=E))
    counts, P = torch.stack(counts), torch.stack(P)
    n = torch.tensor([hi - lo for lo, hi in zip(cuts[:-1], cuts[1:])], device="cuda").double()
    balance = float(E * (counts.double() / (n * k)[:, None] * P).sum() / len(n))
    return counts, P, balance, z / float(n.sum())


def _check(L, idx, off):
    c, P, n, loss = _run(L, idx, off)
    counts, Pr, balance, z = _reference(L, idx, off)
    assert torch.equal(c.long(), counts)
    worst = float(((P.double() - Pr).abs() / Pr.clamp(min=1e-30)).max()) / U
    assert worst <= 160, worst
    assert abs(float(loss[0]) - balance) <= 200 * U * balance
    assert abs(float(loss[1]) - z) <= 200 * U * z, abs(float(loss[1]) - z) / z / U


@pytest.mark.parametrize("step", [0, 3000])
@pytest.mark.parametrize("E", [17, 256])
def test_small_terms_behind_a_large_one(E, step):
    """Every 512th token has lse^2 = 2^24 and p = 1 on expert 0, the others lse^2 = 1
    and p = 0.77 2^-24 there: in fp32 each of these is lost behind the large one.
    Of 64 tokens that loses 63 units, of 512 tokens 511.  One sequence, and
    sequences of 3000 tokens (no CTA's tokens are one sequence's).  E = 17: a warp
    walks its tokens one by one."""
    T = 4736 * 256   # a warp owns 512 tokens
    L = torch.full((T, E), float("-inf"), device="cuda")
    L[:, 0], L[:, 1] = -15.9, 1.0
    L[::512] = 0.0
    L[::512, 0] = 4096.0
    idx = torch.ones((T, 1), dtype=torch.int32, device="cuda")
    idx[::512] = 0
    off = None
    if step:
        off = torch.arange(0, T - step, step, dtype=torch.int32, device="cuda")
    _check(L, idx, off)


@pytest.mark.parametrize("T,E", [(40000, 256), (151552, 64), (303104, 256), (303104, 64),
                                 (700001, 17), (1300003, 8), (5000011, 4)])
def test_long_sequences(T, E):
    """One sequence, and three of which the last tokens belong to none."""
    g = torch.Generator(device="cuda").manual_seed(T + E)
    L = torch.randn((T, E), generator=g, device="cuda").clamp(-5, 5)
    idx = torch.topk(L, 2, dim=1).indices.to(torch.int32)
    L += 1.0
    _check(L, idx, None)
    off = torch.tensor([0, T // 3 + 5, T // 2, T - 77], dtype=torch.int32, device="cuda")
    _check(L, idx, off)


def test_repeats_bit_exact():
    T, E = 700001, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    L = torch.randn((T, E), generator=g, device="cuda")
    idx = torch.topk(L, 2, dim=1).indices.to(torch.int32)
    off = torch.tensor([0, 100, 5000, T], dtype=torch.int32, device="cuda")
    for a, b in zip(_run(L, idx, off), _run(L, idx, off)):
        assert torch.equal(a, b)
