"""One fine-tuning step of the layer on a packed, padded batch with all of its
input's gradient, the residual's dy among it, against the fp64 step of
packed_step.py (whose gradients are pinned by differences of its loss).

Limits, normwise: bf16 weights and rows are exact inputs of both sides.  The
experts' hidden values and the adapters' dropped-out input are rounded to bf16 on
the way (2^-8 relative an element): 1e-2 for the output and the weights'
gradients, 4e-2 for what depends on the gates' gradients (dx without the
residual's part, dW_router), as in the layer's own backward test.
"""
import numpy as np
import pytest
import torch

import packed_step as S
from gpu_util import dev, host
from mixture_experts_top_b200 import api
from oracle import moe_oracle as O
from test_gpu_packed_training import P, SEED, Step, _extra, _norm
from workloads import WORKLOADS, make_inputs

pytestmark = pytest.mark.gpu


class WholeStep(Step):
    """dx = the inner gradient + the residual's dy."""

    def __call__(self):
        super().__call__()
        self.inner = self.dx.clone()
        self.dx.add_(self.dy)


def _f64(v):
    return v.detach().double().cpu().numpy()


@pytest.mark.parametrize("T,capacity_factor", [(300, 0.0), (257, 0.75)])
def test_step_with_the_residual(T, capacity_factor):
    w = WORKLOADS["mixtral"].replace(T=T, d=256, d_hidden=384, d_out=256,
                                     capacity_factor=capacity_factor)
    inp, t = make_inputs(w, seed=15), _extra(w, 16)
    s = WholeStep(w, inp, t)
    s()
    assert s.status() == [0, 0, 0, 0]
    p = {q: O.widen(inp[q], "bf16") for q in ("x", "W_in", "W_up", "W_out")}
    p.update(W_router=inp["W_router"].astype(np.float64), A=_f64(s.A), B=_f64(s.B))
    batch = dict(dy=_f64(s.dy), ids=t["ids"], scale=t["scale"].astype(np.float64), p=P, seed=SEED,
                 offset=1, seqs=t["seqs"], mask=t["mask"],
                 dlosses=tuple(float(v) for v in t["dlosses"]))
    out, losses, g, counts = S.gradients(p, batch, host(s.idx), capacity_factor)
    got = s.results()
    assert np.array_equal(got["bcounts"].cpu().numpy(), counts)
    assert _norm(got["losses"], losses) < 1e-5
    inner = g["x"] - batch["dy"]
    for name, a, b, lim in (("out", got["out"], out, 1e-2), ("dA", got["dA"], g["A"], 1e-2),
                            ("dB", got["dB"], g["B"], 1e-2), ("dW_in", got["dWi"], g["W_in"], 1e-2),
                            ("dW_up", got["dWu"], g["W_up"], 1e-2),
                            ("dW_out", got["dWo"], g["W_out"], 1e-2),
                            ("dW_router", got["dWr"], g["W_router"], 4e-2),
                            ("dx inside", s.inner, inner, 4e-2), ("dx", got["dx"], g["x"], 4e-2)):
        assert _norm(a, b) < lim, (name, _norm(a, b))
    # dy is a part of dx that the limit would not let pass if it were missing
    assert np.linalg.norm(batch["dy"]) > 0.2 * np.linalg.norm(g["x"])
