"""The fp64 fine-tuning step that the GPU step is held against: its composed
gradients against central differences of the loss written out from the formulas,
so that a term left out of one of them shows."""
import numpy as np
import pytest

import packed_step as S
from oracle import moe_oracle as O


def _case(T, d, h, E, k, n, r, seed):
    rng = np.random.default_rng(seed)
    f = lambda *s: rng.standard_normal(s)
    p = dict(x=f(T, d), W_router=f(d, E) / d ** 0.5, W_in=f(E, d, h) / d ** 0.5,
             W_up=f(E, d, h) / d ** 0.5, W_out=f(E, h, d) / h ** 0.5, A=f(n, d, r) / d ** 0.5,
             B=f(n, r, d) / r ** 0.5)
    t = dict(dy=f(T, d), ids=rng.integers(-1, n, T), scale=f(n) + 2, p=0.25, seed=3, offset=5,
             seqs=np.array([0, T // 3, T // 3, T - 4, T - 2]),
             mask=(rng.random(T) < 0.8).astype(np.uint8), dlosses=(0.5, 0.05))
    idx = O.top_k((p["x"] @ p["W_router"]).astype(np.float32), k)
    return p, t, idx, rng


@pytest.mark.parametrize("capacity_factor", [0.0, 0.7])
def test_gradients_are_the_loss_differences(capacity_factor):
    p, t, idx, rng = _case(T=20, d=16, h=24, E=4, k=2, n=3, r=8, seed=1)
    _, _, g, _ = S.gradients(p, t, idx, capacity_factor)
    h = 1e-5
    for q in S.PARAMS:
        for _ in range(3):
            v = rng.standard_normal(p[q].shape)
            ends = [S.loss({**p, q: p[q] + s * h * v}, t, idx, capacity_factor) for s in (1, -1)]
            slope, want = (ends[0] - ends[1]) / (2 * h), float((g[q] * v).sum())
            # the oracle's gates are rounded to fp32 (2^-24 relative); the slope's own
            # error is h^2 and 2^-52 |loss| / h, below 1e-8 here
            assert abs(slope - want) <= 1e-6 * np.linalg.norm(g[q]), (q, slope, want)


def test_the_residual_carries_its_gradient():
    """Without experts' and adapters' weights and the balance loss, dx is dy."""
    p, t, idx, _ = _case(T=12, d=16, h=8, E=4, k=2, n=2, r=8, seed=2)
    for q in ("W_out", "B"):
        p[q] = np.zeros_like(p[q])
    t["dlosses"] = (0.0, 0.0)
    out, _, g, _ = S.gradients(p, t, idx, 0.0)
    assert np.array_equal(out, p["x"]) and np.array_equal(g["x"], t["dy"])
