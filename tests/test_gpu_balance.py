"""The balance loss per sequence on the GPU against the fp64 oracle.

Counts and token numbers are exact.  Tolerances, in units of 2^-24 (half a
step of fp32): a softmax term exp(l - max) carries the subtraction's rounding
times |l - max| (at most 40 here: 40 units), expf's own error (2 ulp: 4), the
sum's chain over 8 experts a lane and a butterfly (13), a reciprocal and a
product (3): p is within 64 units, P (a chain of at most 64 tokens and 8 warps
on top) within 160, the log-sum-exp within 64 units of max(1, |lse|), and z
within 160 units of its scale; a logit gradient within 160 units of the sum of
its terms' magnitudes.
"""
import numpy as np
import pytest
import torch

from gpu_util import dev, host
from mixture_experts_top_b200 import api
from oracle import packed_oracle as Q

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _cfg(T, E, k):
    return api.make_config(T, 8, 8, 8, E, k, "swiglu", "bf16")


def _buffers(T, E, S):
    i32 = dict(dtype=torch.int32, device="cuda")
    return (torch.full((S, E), -7, **i32), torch.full((S, E), float("nan"), device="cuda"),
            torch.full((S + 2,), -7, **i32), torch.full((2,), float("nan"), device="cuda"),
            torch.full((T, E), float("nan"), device="cuda"))


def _run(L, idx, E, off, mask, dl, ws=None, stream=None):
    T, k = idx.shape
    cfg = _cfg(T, E, k)
    S = 1 if off is None else len(off) - 1
    ws = api.alloc_balance_workspace(cfg, S) if ws is None else ws
    c, P, n, loss, g = _buffers(T, E, S)
    a = [dev(v) for v in (off, mask, L, idx, dl)]
    api.moe_balance_loss(cfg, a[0], a[1], a[2], a[3], c, P, n, loss, ws, stream)
    api.moe_balance_loss_backward(cfg, a[0], a[1], a[2], c, n, a[4], g, ws, stream)
    torch.cuda.synchronize()
    return [host(v) for v in (c, P, n, loss, g)] + [ws]


def _case(T, E, k, seed, hot=0.0):
    rng = np.random.default_rng(seed)
    L = (rng.standard_normal((T, E)) * 2).astype(np.float32)
    L[:, : max(1, E // 8)] += hot
    idx = np.argsort(-L, axis=1, kind="stable")[:, :k].astype(np.int32)
    return rng, L, idx


def _check(L, idx, E, off, mask, dl=(0.7, 0.03)):
    dl = np.array(dl, np.float32)
    c, P, n, loss, g, ws = _run(L, idx, E, off, mask, dl)
    assert api.moe_device_status(ws) == 0
    r = Q.balance_loss(L, idx, E, off, mask)
    assert np.array_equal(c, r["counts"]) and np.array_equal(n, r["tokens"])
    assert np.all(np.abs(P - r["prob_mean"]) <= 160 * U * r["prob_mean"])
    assert abs(loss[0] - r["balance"]) <= 200 * U * r["balance"]
    seqs = Q.counted_tokens(len(L), off, mask)
    counted = np.concatenate([np.zeros(0, int)] + seqs)
    with np.errstate(over="ignore"):
        M = L[counted].astype(np.float64)
    lse = M.max(axis=1) + np.log(np.exp(M - M.max(axis=1, keepdims=True)).sum(axis=1)) if len(M) \
        else np.zeros(0)
    scale = np.maximum(1.0, np.abs(lse))
    assert abs(loss[1] - r["z"]) <= 160 * U * (scale ** 2).mean() if len(M) else loss[1] == 0
    ref = Q.balance_loss_backward(L, idx, E, off, mask, float(dl[0]), float(dl[1]))
    live, N = int(r["tokens"][-1]), max(1, int(r["tokens"][-2]))
    mag = np.zeros_like(ref)
    k = idx.shape[1]
    for s, m in enumerate(seqs):
        if len(m) == 0:
            continue
        rows = L[m].astype(np.float64)
        p = np.exp(rows - rows.max(axis=1, keepdims=True))
        p /= p.sum(axis=1, keepdims=True)
        a = abs(float(dl[0])) * E / (live * len(m)) * r["counts"][s] / (len(m) * k)
        where = np.searchsorted(counted, m)
        mag[m] = p * (a + (p @ a)[:, None] + abs(float(dl[1])) * 2 * scale[where, None] / N)
    assert np.all(np.abs(g - ref) <= 160 * U * mag + 1e-37)
    untouched = np.setdiff1d(np.arange(len(L)), counted)
    assert (g[untouched] == 0).all()
    return c, P, n, loss, g


@pytest.mark.parametrize("T", [1, 7, 8, 64, 65, 300, 2049])
@pytest.mark.parametrize("E,k", [(1, 1), (3, 2), (8, 2), (16, 1), (33, 4), (64, 6), (128, 8),
                                 (256, 8)])
def test_sizes(T, E, k):
    rng, L, idx = _case(T, E, k, 100 * T + E, hot=2.0)
    _check(L, idx, E, None, None)
    cuts = np.sort(rng.integers(0, T + 1, 6)).astype(np.int32)
    mask = (rng.random(T) < 0.8).astype(np.uint8)
    _check(L, idx, E, cuts, mask)


@pytest.mark.parametrize("T,S", [(40000, 1), (40000, 3), (9000, 700), (600, 2000), (70000, 5)])
def test_long_and_many_sequences(T, S):
    rng, L, idx = _case(T, 8, 2, T + S)
    cuts = np.sort(rng.integers(0, T + 1, S + 1)).astype(np.int32)
    if S == 1:
        cuts[:] = 0, T
    _check(L, idx, 8, cuts, (rng.random(T) < 0.9).astype(np.uint8))


def test_sequences_on_chunk_borders():
    """Sequences that start and end where a warp's or a CTA's tokens do."""
    T = 1024
    for step in (8, 64, 128):
        _, L, idx = _case(T, 16, 2, step)
        _check(L, idx, 16, np.arange(0, T + 1, step, dtype=np.int32), None)


@pytest.mark.parametrize("off", [[0, 0, 0], [5, 5, 5], [20, 20, 20], [0, 0, 20], [0, 20, 20],
                                 [3, 4, 17], [0, 10, 20]])
def test_empty_sequences_and_padded_ends(off):
    _, L, idx = _case(20, 8, 2, 5)
    off = np.array(off, np.int32)
    _check(L, idx, 8, off, None)
    _check(L, idx, 8, off, np.zeros(20, np.uint8))   # nothing is counted
    L[:off[0]] = np.nan
    L[off[-1]:] = np.inf
    _check(L, idx, 8, off, None)


def test_uncounted_rows_may_hold_anything():
    rng, L, idx = _case(500, 8, 2, 6)
    mask = (rng.random(500) < 0.5).astype(np.uint8)
    mask[100:140] *= 37                               # any non-zero byte counts
    off = np.array([0, 130, 410, 500], np.int32)
    want = _check(L, idx, 8, off, mask)
    L2, idx2 = L.copy(), idx.copy()
    L2[mask == 0] = np.where(rng.random((int((mask == 0).sum()), 8)) < 0.5, np.nan, np.inf)
    idx2[mask == 0] = -123456
    got = _run(L2, idx2, 8, off, mask, np.array([0.7, 0.03], np.float32))
    assert api.moe_device_status(got[5]) == 0
    for a, b in zip(want, got):
        assert np.array_equal(a, b)


def test_experts_switched_off():
    _, L, idx = _case(100, 8, 1, 7)
    L[:, 5] = -np.inf
    L[3, :] = -np.inf
    L[3, 2] = 1.5                                     # one expert left
    L[4, 0] = -3.4e38                                 # the type's lowest range
    idx = np.argsort(-L, axis=1, kind="stable")[:, :1].astype(np.int32)
    _, P, _, _, g = _check(L, idx, 8, None, None)
    assert (P[:, 5] == 0).all() and (g[:, 5] == 0).all()


@pytest.mark.parametrize("E", [8, 64, 100, 256])
def test_logits_at_the_lowest_value(E):
    """Experts switched off by the type's lowest value instead of -inf, up to all
    of a token's: P stays a distribution, and without the z-loss's weight the
    gradient is finite."""
    T, k, low = 70, 2, np.finfo(np.float32).min
    rng, L, idx = _case(T, E, k, 12)
    L[rng.random((T, E)) < 0.5] = low
    L[[3, 40]] = low
    c, P, n, loss, g, ws = _run(L, idx, E, None, None, np.array([0.7, 0.0], np.float32))
    r = Q.balance_loss(L, idx, E, None, None)
    assert np.array_equal(c, r["counts"]) and np.array_equal(n, r["tokens"])
    assert np.all(np.abs(P - r["prob_mean"]) <= 160 * U * r["prob_mean"])
    assert abs(loss[0] - r["balance"]) <= 200 * U * r["balance"]
    ref = Q.balance_loss_backward(L, idx, E, None, None, float(np.float32(0.7)), 0.0)
    a = 0.7 * E / T * r["counts"][0] / (T * k)
    assert np.all(np.abs(g - ref) <= 160 * U * 2 * a.max() + 1e-37)


def test_no_tokens():
    cfg = _cfg(0, 4, 2)
    ws = api.alloc_balance_workspace(cfg, 2)
    c, P, n, loss, g = _buffers(0, 4, 2)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    L = torch.empty((0, 4), device="cuda")
    idx = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    api.moe_balance_loss(cfg, off, None, L, idx, c, P, n, loss, ws)
    api.moe_balance_loss_backward(cfg, off, None, L, c, n, torch.ones(2, device="cuda"), g, ws)
    torch.cuda.synchronize()
    assert api.moe_device_status(ws) == 0
    for t in (c, P, n, loss):
        assert (host(t) == 0).all()


def test_whole_batch_equals_dispatch_loss():
    """One sequence: moe_dispatch's aux_loss and counts, and moe_route_backward's
    part of the gradient."""
    from workloads import WORKLOADS, make_inputs
    w = WORKLOADS["fine_grained"].replace(T=777, d=256, d_hidden=64, d_out=64)
    inp = make_inputs(w, seed=9, with_experts=False)
    cfg = api.make_config(w.T, w.d, w.d_hidden, w.d_out, w.E, w.top_k, w.kind, w.dtype, 0.0)
    ws = api.alloc_workspace(cfg)
    T, k, E = w.T, w.top_k, w.E
    i32 = dict(dtype=torch.int32, device="cuda")
    x, Wr = dev(inp["x"]), dev(inp["W_router"])
    idx, gates = torch.empty((T, k), **i32), torch.empty((T, k), device="cuda")
    P, L = torch.empty(E, device="cuda"), torch.empty((T, E), device="cuda")
    api.moe_route(cfg, x, Wr, dev(inp["logit_bias"]), None, idx, gates, P, L, ws)
    counts, f, aux = torch.empty(E, **i32), torch.empty(E, device="cuda"), torch.empty(1, device="cuda")
    api.moe_dispatch(cfg, x, idx, P, counts, torch.empty(E + 1, **i32), torch.empty((T, k), **i32),
                     torch.empty(T * k, **i32), torch.empty((T, k), dtype=torch.uint8, device="cuda"),
                     f, aux, None, ws)
    bws = api.alloc_balance_workspace(cfg, 1)
    c, Pm, n, loss, g = _buffers(T, E, 1)
    api.moe_balance_loss(cfg, None, None, L, idx, c, Pm, n, loss, bws)
    dl = torch.tensor([0.9, 0.0], device="cuda")
    api.moe_balance_loss_backward(cfg, None, None, L, c, n, dl, g, bws)
    zero = torch.zeros((T, k), device="cuda")
    f32 = dict(dtype=torch.float32, device="cuda")
    outs = [[torch.empty((T, w.d), **f32), torch.empty((w.d, E), **f32), torch.empty(E, **f32),
             torch.empty((T, E), **f32)] for _ in range(2)]
    api.moe_route_backward(cfg, x, Wr, L, idx, gates, f, zero, dl[:1], 0, *outs[0], ws)
    api.moe_route_backward_add(cfg, x, Wr, L, idx, gates, f, zero, torch.zeros(1, device="cuda"),
                               0, g, *outs[1], ws)
    torch.cuda.synchronize()
    assert np.array_equal(host(c)[0], host(counts))
    assert abs(float(loss[0]) - float(aux)) <= 1e-5 * float(aux)
    for a, b in zip(*outs):
        a, b = host(a).astype(np.float64), host(b).astype(np.float64)
        # p (a_e - p.a) cancels: normwise, both within 160 units of p (|a| + p.|a|) <= 2 max |a| p
        assert np.linalg.norm(a - b) <= 1e-4 * np.linalg.norm(a)


def test_route_backward_add_adds():
    """Zeros change nothing, and dlogits = moe_route_backward's + the addend,
    also in place."""
    T, d, E, k = 130, 64, 24, 3
    rng, L, idx = _case(T, E, k, 11)
    cfg = api.make_config(T, d, 64, 64, E, k, "swiglu", "bf16")
    ws = api.alloc_workspace(cfg)
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, W = rnd(T, d).bfloat16(), rnd(d, E)
    gates, dg = torch.softmax(rnd(T, k), 1), rnd(T, k)
    f, daux, add = torch.rand(E, generator=g, device="cuda"), rnd(1), rnd(T, E)
    Ld, ix = dev(L), dev(idx)
    new = lambda: [torch.empty((T, d), device="cuda"), torch.empty((d, E), device="cuda"),
                   torch.empty(E, device="cuda"), torch.empty((T, E), device="cuda")]
    base, zero, some, place = new(), new(), new(), new()
    args = (cfg, x, W, Ld, ix, gates, f, dg, daux, 0)
    api.moe_route_backward(*args, *base, ws)
    api.moe_route_backward_add(*args, torch.zeros(T, E, device="cuda"), *zero, ws)
    api.moe_route_backward_add(*args, add, *some, ws)
    place[3].copy_(add)
    api.moe_route_backward_add(*args, place[3], *place, ws)
    torch.cuda.synchronize()
    for a, b in zip(base, zero):
        assert torch.equal(a, b)
    assert torch.equal(some[3], base[3] + add)
    for a, b in zip(some, place):
        assert torch.equal(a, b)
    dL = some[3].double()
    assert torch.all((some[0].double() - dL @ W.double().T).abs()
                     <= 2 * E * U * (dL.abs() @ W.double().abs().T) + 1e-30)
    assert torch.all((some[1].double() - x.double().T @ dL).abs()
                     <= 2 * T * U * (x.double().abs().T @ dL.abs()) + 1e-30)


def test_bad_index_and_bad_offsets_are_reported():
    _, L, idx = _case(50, 8, 2, 8)
    idx[17, 1] = 8
    c, _, n, _, _, ws = _run(L, idx, 8, None, None, np.ones(2, np.float32))
    assert api.moe_device_status(ws) == 1
    assert c.sum() == 99 and n[0] == 50
    idx[17, 1] = 0
    for off in ([0, 30, 20, 50], [0, 20, 51], [-1, 20, 50]):
        ws = _run(L, idx, 8, np.array(off, np.int32), None, np.ones(2, np.float32), ws=None)[5]
        assert api.moe_device_status(ws) == 2
    _check(L, idx, 8, np.array([0, 20, 50], np.int32), None)   # nothing lingers


def test_repeats_bit_exact_and_reuses_the_workspace():
    rng, L, idx = _case(5000, 64, 6, 12)
    off = np.sort(rng.integers(0, 5001, 30)).astype(np.int32)
    dl = np.array([0.5, 0.1], np.float32)
    a = _run(L, idx, 64, off, None, dl)
    a[5][256:].fill_(0xFF)                            # stale partial sums must not be read
    b = _run(L, idx, 64, off, None, dl, ws=a[5])
    for u, v in zip(a[:5], b[:5]):
        assert np.array_equal(u, v)


def test_captured_on_another_stream_with_new_inputs():
    rng, L, idx = _case(900, 16, 2, 13)
    _, L2, idx2 = _case(900, 16, 2, 14)
    off, off2 = (np.array(v, np.int32) for v in ([0, 100, 900], [10, 700, 800]))
    cfg = _cfg(900, 16, 2)
    ws = api.alloc_balance_workspace(cfg, 2)
    ins = [dev(v) for v in (off, L, idx)]
    dl = torch.tensor([0.5, 0.25], device="cuda")
    c, P, n, loss, g = _buffers(900, 16, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def step():
        api.moe_balance_loss(cfg, ins[0], None, ins[1], ins[2], c, P, n, loss, ws)
        api.moe_balance_loss_backward(cfg, ins[0], None, ins[1], c, n, dl, g, ws)

    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for o, l, i in ((off2, L2, idx2), (off, L, idx), (off2, L2, idx2)):
        for dst, src in zip(ins, (o, l, i)):
            dst.copy_(dev(src))
        graph.replay()
        torch.cuda.synchronize()
        want = _run(l, i, 16, o, None, np.array([0.5, 0.25], np.float32))
        for a, b in zip((c, P, n, loss, g), want):
            assert np.array_equal(host(a), b)
