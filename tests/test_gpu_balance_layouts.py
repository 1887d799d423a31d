"""The balance loss for expert counts and alignments of every lane layout: rows
read by 16-byte vectors (E a multiple of 4, rows 16-byte aligned) or one value at
a time, 1 to 32 lanes a token; against the fp64 oracle.

Tolerances in units of 2^-24: for logits within 12 of a token's largest a
probability is within 87 units, P within 160, the log-sum-exp within 65 units of
max(1, |lse|) (the 2^x form: 2.3 |l - m| + 4 a term; 21 for a sum of 256 terms).  z: 200 units
of that scale's square.  A logit gradient p (a - p.a + dz lse): p and each of the
terms within 87 + 87 + 20 units of their magnitudes: 200.
"""
import numpy as np
import pytest
import torch

from gpu_util import dev, host
from mixture_experts_top_b200 import api
from oracle import packed_oracle as Q

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _logits(L, skew):
    """On the device, `skew` floats behind a 16-byte boundary."""
    buf = torch.empty(L.size + 8, device="cuda")
    v = buf[skew:skew + L.size].view(L.shape)
    v.copy_(torch.from_numpy(L))
    assert v.data_ptr() % 16 == 4 * (skew % 4)
    return v


def _run(L, idx, E, off, mask, dl, skew=0, out_skew=0):
    T, k = idx.shape
    cfg = api.make_config(T, 8, 8, 8, E, k, "swiglu", "bf16")
    S = 1 if off is None else len(off) - 1
    ws = api.alloc_balance_workspace(cfg, S)
    i32 = dict(dtype=torch.int32, device="cuda")
    c, P = torch.empty((S, E), **i32), torch.empty((S, E), device="cuda")
    n, loss = torch.empty(S + 2, **i32), torch.empty(2, device="cuda")
    g = torch.full((T * E + 8,), float("nan"), device="cuda")
    g = g[out_skew:out_skew + T * E].view(T, E)
    o, m, ix, d = (dev(v) for v in (off, mask, idx, dl))
    Ld = _logits(L, skew)
    api.moe_balance_loss(cfg, o, m, Ld, ix, c, P, n, loss, ws)
    api.moe_balance_loss_backward(cfg, o, m, Ld, c, n, d, g, ws)
    assert api.moe_device_status(ws) == 0
    return [host(v) for v in (c, P, n, loss, g)]


def _case(T, E, k, seed):
    rng = np.random.default_rng(seed)
    L = np.clip(rng.standard_normal((T, E)) * 2, -5, 5).astype(np.float32) + 1
    idx = np.argsort(-L, axis=1, kind="stable")[:, :k].astype(np.int32)
    cuts = np.sort(rng.integers(0, T + 1, 5)).astype(np.int32)
    return L, idx, cuts, (rng.random(T) < 0.8).astype(np.uint8)


def _check(L, idx, E, off, mask, got, dl):
    c, P, n, loss, g = got
    r = Q.balance_loss(L, idx, E, off, mask)
    assert np.array_equal(c, r["counts"]) and np.array_equal(n, r["tokens"])
    assert np.all(np.abs(P - r["prob_mean"]) <= 160 * U * r["prob_mean"])
    assert abs(loss[0] - r["balance"]) <= 200 * U * r["balance"]
    M = L.astype(np.float64)
    lse = M.max(axis=1) + np.log(np.exp(M - M.max(axis=1, keepdims=True)).sum(axis=1))
    scale = np.maximum(1.0, np.abs(lse))
    seqs = Q.counted_tokens(len(L), off, mask)
    counted = np.concatenate(seqs)
    if len(counted):
        assert abs(loss[1] - r["z"]) <= 200 * U * (scale[counted] ** 2).mean()
    ref = Q.balance_loss_backward(L, idx, E, off, mask, float(dl[0]), float(dl[1]))
    mag, k = np.zeros_like(ref), idx.shape[1]
    for s, m in enumerate(seqs):
        if len(m) == 0:
            continue
        p = np.exp(M[m] - lse[m, None])
        a = float(dl[0]) * E / (r["tokens"][-1] * len(m)) * r["counts"][s] / (len(m) * k)
        mag[m] = p * (a + (p @ a)[:, None] + float(dl[1]) * 2 * scale[m, None] / len(counted))
    assert np.all(np.abs(g - ref) <= 200 * U * mag + 1e-37)


@pytest.mark.parametrize("T", [9, 530, 2500])
@pytest.mark.parametrize("E", [2, 4, 5, 6, 13, 15, 17, 20, 28, 32, 36, 63, 65, 130, 132, 255])
def test_expert_counts(E, T):
    """T = 530: the sums in the first launch's last CTA; 2500: in one of their own."""
    k = min(2, E)
    L, idx, cuts, mask = _case(T, E, k, T + E)
    dl = np.array([0.7, 0.03], np.float32)
    for o, m in ((None, None), (cuts, mask)):
        _check(L, idx, E, o, m, _run(L, idx, E, o, m, dl), dl)


@pytest.mark.parametrize("E", [4, 8, 16, 64, 128, 256])
@pytest.mark.parametrize("skew,out_skew", [(1, 0), (2, 3), (0, 1)])
def test_rows_off_16_byte_boundaries(E, skew, out_skew):
    L, idx, cuts, mask = _case(300, E, 2, E)
    dl = np.array([0.7, 0.03], np.float32)
    _check(L, idx, E, cuts, mask, _run(L, idx, E, cuts, mask, dl, skew, out_skew), dl)
