"""One fine-tuning step of the layer on a packed, padded batch, as a program
would run it: route, dispatch, experts, the combine with dropout and residual,
adapters on the dropped-out input beside the layer's output, the balance loss
per sequence -- and the backward of all of it, eager and as one captured graph.

loss = <dy, output> + <dlosses, (balance, z)>.  The reference composes the
fp64 oracles on the same inputs and masks.  The bf16 experts' rounding carries
over: expert weights within 1e-2 normwise, and what depends on the gates'
gradients (dx, dW_router) within 4e-2, as in the layer's own backward test;
the adapters see x rounded to bf16 once after dropout (2^-8 relative an
element): within 1e-2 normwise.
"""
import numpy as np
import pytest
import torch

from gpu_util import cfg_of, dev, host
from mixture_experts_top_b200 import api
from oracle import moe_oracle as O
from oracle import packed_oracle as Q
from workloads import WORKLOADS, make_inputs

pytestmark = pytest.mark.gpu

P, SEED = 0.1, 77
N, R = 3, 16


class Step:
    def __init__(self, w, inp, extra):
        self.w, self.cfg = w, cfg_of(w)
        T, k, E, d = w.T, w.top_k, w.E, w.d
        f32 = dict(dtype=torch.float32, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.W = {q: dev(inp[q]) for q in ("W_router", "W_in", "W_up", "W_out")}
        self.x = dev(inp["x"])
        self.t = {q: dev(v) for q, v in extra.items()}
        self.A, self.B = self.t["A"].bfloat16(), self.t["B"].bfloat16()
        self.dy = self.t["dy"].bfloat16()
        self.offset = torch.tensor([1], dtype=torch.int64, device="cuda")
        e = torch.empty
        self.idx, self.gates = e((T, k), **i32), e((T, k), **f32)
        self.prob, self.L = e(E, **f32), e((T, E), **f32)
        self.counts, self.offsets = e(E, **i32), e(E + 1, **i32)
        self.dest, self.perm = e((T, k), **i32), e(T * k, **i32)
        self.dropped = e((T, k), dtype=torch.uint8, device="cuda")
        self.f, self.aux = e(E, **f32), e(1, **f32)
        self.x_perm, self.y_perm = e((T * k, d), **bf), e((T * k, d), **f32)
        self.xa, self.out, self.u = e((T, d), **bf), e((T, d), **bf), e((T, R), **f32)
        S = len(extra["seqs"]) - 1
        self.bcounts, self.bprob = e((S, E), **i32), e((S, E), **f32)
        self.tokens, self.losses = e(S + 2, **i32), e(2, **f32)
        self.dlogits = e((T, E), **f32)
        self.dy_perm, self.dgates = torch.zeros((T * k, d), **f32), e((T, k), **f32)
        self.dxa, self.dx_perm, self.dx = e((T, d), **f32), e((T * k, d), **f32), e((T, d), **f32)
        self.dWr, self.db = e((d, E), **f32), e(E, **f32)
        self.dWi, self.dWu = (e((E, d, w.d_hidden), **f32) for _ in range(2))
        self.dWo = e((E, w.d_hidden, d), **f32)
        self.dA, self.dB = e((N, d, R), **f32), e((N, R, d), **f32)
        self.zero = torch.zeros(1, **f32)
        self.ws, self.bws = api.alloc_workspace(self.cfg), api.alloc_backward_workspace(self.cfg)
        self.lws = api.alloc_balance_workspace(self.cfg, S)
        self.plan = api.alloc_adapter_plan(self.cfg, N)
        self.aws = api.alloc_adapter_workspace(self.cfg, N, R)

    def __call__(self):
        s, t, W, cfg, ws = self, self.t, self.W, self.cfg, self.ws
        api.moe_route(cfg, s.x, W["W_router"], None, None, s.idx, s.gates, s.prob, s.L, ws)
        api.moe_dispatch(cfg, s.x, s.idx, s.prob, s.counts, s.offsets, s.dest, s.perm, s.dropped,
                         s.f, s.aux, s.x_perm, ws)
        api.moe_expert_ffn_train(cfg, s.x_perm, s.offsets, W["W_in"], W["W_up"], W["W_out"],
                                 s.y_perm, ws, s.bws)
        api.moe_combine_dropout(cfg, P, SEED, s.offset, 0, s.y_perm, s.dest, s.gates, s.x, s.out)
        api.moe_adapter_plan(cfg, N, t["ids"], s.plan)
        api.moe_dropout(cfg, P, SEED + 1, s.offset, 0, s.x, None, s.xa)
        api.moe_adapter(cfg, s.plan, s.xa, s.A, s.B, t["scale"], s.out, s.out, s.u)
        api.moe_balance_loss(cfg, t["seqs"], t["mask"], s.L, s.idx, s.bcounts, s.bprob, s.tokens,
                             s.losses, s.lws)
        # backward
        api.moe_balance_loss_backward(cfg, t["seqs"], t["mask"], s.L, s.bcounts, s.tokens,
                                      t["dlosses"], s.dlogits, s.lws)
        api.moe_adapter_backward(cfg, s.plan, s.xa, s.u, s.dy, s.A, s.B, t["scale"], None, s.dxa,
                                 s.dA, s.dB, s.aws)
        api.moe_combine_dropout_backward(cfg, P, SEED, s.offset, 0, s.dy, s.y_perm, s.dest,
                                         s.gates, s.dy_perm, s.dgates)
        api.moe_route_backward_add(cfg, s.x, W["W_router"], s.L, s.idx, s.gates, s.f, s.dgates,
                                   s.zero, 0, s.dlogits, s.dx, s.dWr, s.db, None, ws)
        api.moe_expert_ffn_backward_saved(cfg, s.x_perm, s.offsets, W["W_in"], W["W_up"],
                                          W["W_out"], s.dy_perm, s.dx_perm, s.dWi, s.dWu, s.dWo,
                                          s.bws)
        api.moe_permute_backward(cfg, s.dx_perm, s.dest, s.dx, s.dx)
        api.moe_dropout(cfg, P, SEED + 1, s.offset, 0, s.dxa, s.dx, s.dx)   # + the residual's dy

    def results(self):
        keys = ("out", "losses", "dx", "dWr", "db", "dWi", "dWu", "dWo", "dA", "dB", "bcounts")
        return {q: getattr(self, q).clone() for q in keys}

    def status(self):
        return [api.moe_device_status(b) for b in (self.ws, self.bws, self.lws, self.plan)]


def _extra(w, seed):
    rng = np.random.default_rng(seed)
    f = lambda *s: rng.standard_normal(s).astype(np.float32)
    T = w.T
    return dict(A=f(N, w.d, R) / 16, B=f(N, R, w.d) / 4, scale=f(N) + 2, dy=f(T, w.d),
                ids=np.repeat([0, 2, -1, 1], [T // 4, T // 4, T // 4, T - 3 * (T // 4)])
                .astype(np.int32),
                seqs=np.array([0, T // 3, T // 3, T - 20, T - 5], np.int32),
                mask=(rng.random(T) < 0.9).astype(np.uint8),
                dlosses=np.array([0.5, 0.05], np.float32))


def _reference(w, inp, t, step, offset):
    """The same step in fp64 with the GPU's routing choice."""
    T, E, k, d = w.T, w.E, w.top_k, w.d
    x = O.widen(inp["x"], "bf16")
    bf = lambda a: dev(a).bfloat16().double().cpu().numpy()
    A, B, dy = bf(t["A"]), bf(t["B"]), bf(t["dy"])
    idx = host(step.idx)
    L = O.router_logits(inp["x"], inp["W_router"], "bf16")
    gates = O.renormalised_gates(L, idx)
    disp = O.dispatch(idx, E, w.capacity_factor)
    weights = {q: inp[q] for q in ("W_in", "W_up", "W_out")}
    Y = O.run_experts(w.kind, inp["x"], "bf16", disp, weights, d)
    y = Q.dropout(O.combine(Y, disp["dest"], gates), P, SEED, offset, 0, x)
    xa = Q.dropout(x, P, SEED + 1, offset)
    y, _ = Q.adapter(xa, A, B, t["scale"], t["ids"], y)
    bal = Q.balance_loss(L, idx, E, t["seqs"], t["mask"])
    wb, wz = (float(v) for v in t["dlosses"])
    add = Q.balance_loss_backward(L, idx, E, t["seqs"], t["mask"], wb, wz)
    dxa, dA, dB = Q.adapter_backward(xa, A, B, t["scale"], t["ids"], dy)
    dY, dg = O.combine_backward(Y, disp["dest"], gates, Q.dropout(dy, P, SEED, offset))
    r = O.route_backward(inp["x"], inp["W_router"], "bf16", L, idx, gates,
                         np.zeros(E), dg, 0.0)
    dL = r["dlogits"] + add
    dx = dL @ inp["W_router"].astype(np.float64).T + Q.dropout(dxa, P, SEED + 1, offset)
    g = dict(dWi=[], dWu=[], dWo=[])
    offs = disp["offsets"]
    tok = np.zeros(int(offs[-1]), int)
    for i in range(T):
        for j in range(k):
            if disp["dest"][i, j] >= 0:
                tok[disp["dest"][i, j]] = i
    for e in range(E):
        rows = slice(int(offs[e]), int(offs[e + 1]))
        b = O.expert_backward(w.kind, x[tok[rows]], *O.expert_weights(weights, e, "bf16"), dY[rows])
        np.add.at(dx, tok[rows], b["dx"])
        for q, name in (("dWi", "dW_in"), ("dWu", "dW_up"), ("dWo", "dW_out")):
            g[q].append(b[name])
    out = dict(out=y, losses=np.array([bal["balance"], bal["z"]]), dx=dx, dWr=x.T @ dL,
               db=dL.sum(0), dA=dA, dB=dB, bcounts=bal["counts"])
    out.update({q: np.stack(v) for q, v in g.items()})
    return out


def _norm(got, ref):
    got = got.double().cpu().numpy()
    return np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-30)


W = WORKLOADS["mixtral"].replace(T=300, d=256, d_hidden=384, d_out=256)


def test_step_against_the_oracles():
    inp, t = make_inputs(W, seed=5), _extra(W, 6)
    s = Step(W, inp, t)
    s()
    torch.cuda.synchronize()
    assert s.status() == [0, 0, 0, 0]
    ref, got = _reference(W, inp, t, s, 1), s.results()
    assert np.array_equal(got["bcounts"].cpu().numpy(), ref["bcounts"])
    assert _norm(got["losses"], ref["losses"]) < 1e-5
    for q, lim in dict(out=1e-2, dA=1e-2, dB=1e-2, dWi=1e-2, dWu=1e-2, dWo=1e-2, dx=4e-2, dWr=4e-2,
                       db=4e-2).items():
        assert _norm(got[q], ref[q]) < lim, (q, _norm(got[q], ref[q]))


def test_captured_step_equals_eager_steps():
    """Three replays, the offset raised by the graph itself (a fresh mask each)
    and the requests changed in between; eager steps on a second set of
    buffers give the same bits."""
    inp, t, t2 = make_inputs(W, seed=7), _extra(W, 8), _extra(W, 9)
    a, b = Step(W, inp, t), Step(W, inp, t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        a()
        a.offset.add_(1)
    seen = []
    for step in range(3):
        if step == 2:
            for q in ("ids", "seqs", "mask", "dy"):
                for st in (a, b):
                    st.t[q].copy_(dev(t2[q]))
            a.dy.copy_(a.t["dy"])
            b.dy.copy_(b.t["dy"])
        graph.replay()
        torch.cuda.synchronize()
        b()
        b.offset.add_(1)
        torch.cuda.synchronize()
        ra, rb = a.results(), b.results()
        for q in ra:
            assert torch.equal(ra[q], rb[q]), (step, q)
        seen.append(ra["out"])
    assert not torch.equal(seen[0], seen[1])
    assert a.status() == [0] * 4 and b.status() == [0] * 4
