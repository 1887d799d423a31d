"""One fine-tuning step of the layer on a packed batch in fp64: its loss, written
out from the formulas, and its gradients, composed of the oracles.

  out  = x + drop_0(sum_j g_j expert_j(x)) + s_a (drop_1(x) A_a) B_a
  loss = <dy, out> + <dlosses, (balance, z)>

with the routing choice held fixed.  dx has four parts: dy itself (the residual),
the experts' and the router's inputs, and the adapters' through drop_1."""
import numpy as np

from oracle import moe_oracle as O
from oracle import packed_oracle as Q

PARAMS = ("x", "W_router", "W_in", "W_up", "W_out", "A", "B")


def loss(p, t, idx, capacity_factor):
    """The step's loss as a number; p: PARAMS in fp64, t: the batch."""
    x, T, k = p["x"], len(p["x"]), idx.shape[1]
    L = x @ p["W_router"]
    E = L.shape[1]
    kept = O.dispatch(idx, E, capacity_factor)["dest"] >= 0
    chosen = np.take_along_axis(L, idx.astype(np.int64), axis=1)
    g = np.exp(chosen - chosen.max(axis=1, keepdims=True))
    g /= g.sum(axis=1, keepdims=True)
    y = np.zeros_like(t["dy"])
    for e in range(E):
        a, b = x @ p["W_in"][e], x @ p["W_up"][e]
        ffn = (a / (1.0 + np.exp(-a)) * b) @ p["W_out"][e]
        y += ((g * kept * (idx == e)).sum(axis=1))[:, None] * ffn
    keep = [Q.keep_mask(T, x.shape[1], t["p"], t["seed"] + i, t["offset"]) for i in (0, 1)]
    scale = 65536.0 / (65536.0 - Q.threshold(t["p"]))
    out = x + keep[0] * scale * y
    xa = keep[1] * scale * x
    for i in range(T):
        a = t["ids"][i]
        if a >= 0:
            out[i] += t["scale"][a] * (xa[i] @ p["A"][a]) @ p["B"][a]
    m = L.max(axis=1, keepdims=True)
    lse = (m + np.log(np.exp(L - m).sum(axis=1, keepdims=True)))[:, 0]
    P = np.exp(L - lse[:, None])
    balance, z, live, N = 0.0, 0.0, 0, 0
    for lo, hi in zip(t["seqs"][:-1], t["seqs"][1:]):
        rows = [i for i in range(lo, hi) if t["mask"][i]]
        if not rows:
            continue
        f = np.bincount(idx[rows].reshape(-1), minlength=E) / (len(rows) * k)
        balance += E * (f @ P[rows].mean(axis=0))
        z += (lse[rows] ** 2).sum()
        live, N = live + 1, N + len(rows)
    wb, wz = t["dlosses"]
    return (t["dy"] * out).sum() + wb * balance / live + wz * z / N


def gradients(p, t, idx, capacity_factor):
    """(out, losses, gradients by PARAMS, slot counts), from the oracles."""
    x, T, E = p["x"], len(p["x"]), p["W_router"].shape[1]
    weights = {q: p[q] for q in ("W_in", "W_up", "W_out")}
    L = x @ p["W_router"]
    gates = O.renormalised_gates(L, idx)
    disp = O.dispatch(idx, E, capacity_factor)
    Y = O.run_experts("swiglu", x, "f64", disp, weights, x.shape[1])
    drop = lambda v, i, add=None: Q.dropout(v, t["p"], t["seed"] + i, t["offset"], 0, add)
    y = drop(O.combine(Y, disp["dest"], gates), 0, x)
    xa = drop(x, 1)
    out, _ = Q.adapter(xa, p["A"], p["B"], t["scale"], t["ids"], y)
    bal = Q.balance_loss(L, idx, E, t["seqs"], t["mask"])
    wb, wz = t["dlosses"]
    dxa, dA, dB = Q.adapter_backward(xa, p["A"], p["B"], t["scale"], t["ids"], t["dy"])
    dY, dg = O.combine_backward(Y, disp["dest"], gates, drop(t["dy"], 0))
    r = O.route_backward(x, p["W_router"], "f64", L, idx, gates, np.zeros(E), dg, 0.0)
    dL = r["dlogits"] + Q.balance_loss_backward(L, idx, E, t["seqs"], t["mask"], wb, wz)
    g = {q: np.zeros_like(p[q]) for q in PARAMS}
    g["A"], g["B"], g["W_router"] = dA, dB, x.T @ dL
    g["x"] = t["dy"] + dL @ p["W_router"].T + drop(dxa, 1)
    offs, perm = disp["offsets"], disp["perm_token"]
    for e in range(E):
        rows = perm[offs[e]:offs[e + 1]]
        b = O.expert_backward("swiglu", x[rows], *(p[q][e] for q in ("W_in", "W_up", "W_out")),
                              dY[offs[e]:offs[e + 1]])
        np.add.at(g["x"], rows, b["dx"])
        for q in ("W_in", "W_up", "W_out"):
            g[q][e] = b["d" + q]
    return out, np.array([bal["balance"], bal["z"]]), g, bal["counts"]
