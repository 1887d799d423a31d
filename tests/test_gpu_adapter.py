"""Low-rank adapters on the GPU against the fp64 oracle on the same bf16 inputs.

Tolerances.  u and v are fp32 sums of K = d or d_out exact products: within
K 2^-24 of the sum of the products' magnitudes (the tensor core's adds
included: it truncates, so 2 K 2^-24), times a rounded scale.  As operands
they keep 16 bits (two bf16 terms, forward: 2^-16 relative) or 24 (three,
backward: 2^-24).  So, with |.| the same expression on magnitudes:
  output: (2^-16 + 2 (d + r + 2) 2^-24) |u| |B|, plus bf16's 2^-8 of the result
  dx:     2 (d_out + r + 4) 2^-24 |v| |A|, plus 2^-24 of the result
  dA, dB: 2 (K + rows + 4) 2^-24 of the magnitudes' product
"""
import numpy as np
import pytest
import torch

from mixture_experts_top_b200 import api
from oracle import packed_oracle as Q

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _cfg(T, d, d_out):
    return api.make_config(T, d, 8, d_out, 8, 2, "swiglu", "bf16")


def _f64(t):
    return t.detach().double().cpu().numpy()


def _inputs(T, d, d_out, n, r, seed, none=0.2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    ids = rng.integers(0, n, T)
    ids = np.where(rng.random(T) < none, -1 - rng.integers(0, 3, T), ids).astype(np.int32)
    bf = torch.bfloat16
    return dict(x=rnd(T, d).to(bf), A=(rnd(n, d, r) / d ** 0.5).to(bf),
                B=(rnd(n, r, d_out) / r ** 0.5).to(bf), scale=rnd(n), base=rnd(T, d_out).to(bf),
                dy=rnd(T, d_out).to(bf), dx_add=rnd(T, d), ids=ids)


def _plan(cfg, n, ids):
    plan = api.alloc_adapter_plan(cfg, n)
    api.moe_adapter_plan(cfg, n, torch.from_numpy(ids).cuda(), plan)
    return plan


def _run(i, T, d, d_out, n, r, base=True, dx_add=True):
    cfg = _cfg(T, d, d_out)
    plan = _plan(cfg, n, i["ids"])
    nan = lambda *s: torch.full(s, float("nan"), device="cuda")
    out, u = nan(T, d_out).bfloat16(), nan(T, r)
    dx, dA, dB = nan(T, d), nan(n, d, r), nan(n, r, d_out)
    ws = api.alloc_adapter_workspace(cfg, n, r).fill_(0xFF)
    api.moe_adapter(cfg, plan, i["x"], i["A"], i["B"], i["scale"], i["base"] if base else None, out,
                    u)
    api.moe_adapter_backward(cfg, plan, i["x"], u, i["dy"], i["A"], i["B"], i["scale"],
                             i["dx_add"] if dx_add else None, dx, dA, dB, ws)
    torch.cuda.synchronize()
    assert api.moe_device_status(plan) == 0
    return out, u, dx, dA, dB


def _check(i, got, base=True, dx_add=True):
    out, u, dx, dA, dB = (_f64(t) for t in got)
    x, A, B, s, dy = (_f64(i[k]) for k in ("x", "A", "B", "scale", "dy"))
    ids = i["ids"]
    (T, d), d_out, r = x.shape, B.shape[2], A.shape[2]
    b = _f64(i["base"]) if base else None
    add = _f64(i["dx_add"]) if dx_add else None
    ref, uref = Q.adapter(x, A, B, s, ids, b)
    rx, rA, rB = Q.adapter_backward(x, A, B, s, ids, dy, add)
    mag, umag = Q.adapter(np.abs(x), np.abs(A), np.abs(B), np.abs(s), ids)
    mx, mA, mB = Q.adapter_backward(np.abs(x), np.abs(A), np.abs(B), np.abs(s), ids, np.abs(dy))
    has = (ids >= 0)
    assert np.isnan(u[~has]).all()                    # rows without an adapter: untouched
    assert np.all(np.abs(u - uref)[has] <= 2 * (d + 2) * U * umag[has] + 1e-30)
    lim = (2.0 ** -16 + 2 * (d + r + 2) * U) * mag + 2.0 ** -8 * np.abs(ref)
    assert np.all(np.abs(out - ref) <= lim + 1e-30)
    assert np.all(np.abs(dx - rx) <= 2 * (d_out + r + 4) * U * mx + U * np.abs(rx) + 1e-30)
    rows = np.bincount(ids[has], minlength=A.shape[0])[:, None, None]
    assert np.all(np.abs(dA - rA) <= 2 * (d_out + rows + 4) * U * mA + 1e-30)
    assert np.all(np.abs(dB - rB) <= 2 * (d + rows + 4) * U * mB + 1e-30)
    assert np.array_equal(out[~has], b[~has] if base else np.zeros_like(out[~has]))
    assert np.array_equal(dx[~has], add[~has] if dx_add else np.zeros_like(dx[~has]))


@pytest.mark.parametrize("T,d,d_out,n,r", [
    (1, 8, 8, 1, 8), (1, 2048, 264, 3, 16), (2, 64, 128, 2, 16), (16, 128, 64, 1, 16),
    (17, 136, 72, 2, 24), (64, 1024, 512, 64, 16), (100, 72, 1032, 5, 40), (333, 776, 1032, 5, 24),
    (70, 200, 88, 4, 128), (1025, 256, 320, 3, 64), (2500, 520, 264, 7, 32), (2049, 64, 64, 2, 72),
    (1300, 1032, 136, 5, 128), (4000, 128, 64, 1, 8), (1100, 96, 40, 1000, 8),
    # many rows: the tcgen05 products
    (4800, 64, 64, 1, 16), (4801, 72, 40, 40, 8), (4900, 776, 1032, 5, 24), (5000, 520, 264, 7, 32),
    (5200, 1032, 200, 3, 64), (6000, 136, 648, 3, 128), (4999, 2056, 72, 2, 72),
    (8192, 200, 136, 6, 88), (20000, 40, 24, 2, 8), (3000, 264, 136, 2, 96),
    (6600, 776, 264, 5, 16), (4000, 136, 72, 100, 64)])
def test_sizes(T, d, d_out, n, r):
    i = _inputs(T, d, d_out, n, r, seed=T + r)
    _check(i, _run(i, T, d, d_out, n, r))


@pytest.mark.parametrize("T", [40, 1500, 4800, 6600])
@pytest.mark.parametrize("base,dx_add", [(False, True), (True, False), (False, False)])
def test_without_addends(T, base, dx_add):
    i = _inputs(T, 136, 264, 3, 16, seed=1)
    _check(i, _run(i, T, 136, 264, 3, 16, base, dx_add), base, dx_add)


@pytest.mark.parametrize("T,n,d,w", [
    (50, 6, 72, 136), (3, 8, 136, 328), (4, 18, 72, 136), (1500, 6, 72, 136), (4900, 6, 72, 136),
    (6600, 6, 72, 136)])
@pytest.mark.parametrize("ids", ["none", "one", "last"])
def test_extreme_groups(T, n, d, w, ids):
    """No token with an adapter; all on one; only the last token on the last."""
    i = _inputs(T, d, w, n, 16, seed=2)
    i["ids"][:] = {"none": -1, "one": 2, "last": -5}[ids]
    if ids == "last":
        i["ids"][-1] = n - 1
    got = _run(i, T, d, w, n, 16)
    _check(i, got)
    idle = [a for a in range(n) if not (i["ids"] == a).any()]
    assert (got[3][idle] == 0).all() and (got[4][idle] == 0).all()


@pytest.mark.parametrize("T", [300, 4800, 6600])
def test_in_place(T):
    d, w, n, r = 136, 264, 4, 16
    i = _inputs(T, d, w, n, r, seed=3)
    out, u, dx, dA, dB = _run(i, T, d, w, n, r)
    cfg = _cfg(T, d, w)
    plan = _plan(cfg, n, i["ids"])
    y, g = i["base"].clone(), i["dx_add"].clone()
    api.moe_adapter(cfg, plan, i["x"], i["A"], i["B"], i["scale"], y, y, None)
    ws = api.alloc_adapter_workspace(cfg, n, r)
    api.moe_adapter_backward(cfg, plan, i["x"], u, i["dy"], i["A"], i["B"], i["scale"], g, g,
                             torch.empty_like(dA), torch.empty_like(dB), ws)
    assert torch.equal(y, out) and torch.equal(g, dx)


@pytest.mark.parametrize("T", [200, 1400, 4900, 6600])
def test_rows_do_not_leak_into_one_another(T):
    """NaN in the rows of one adapter and of tokens without one stays there."""
    d, w, n, r = 72, 136, 3, 16
    i = _inputs(T, d, w, n, r, seed=4)
    good = _run(i, T, d, w, n, r)
    bad = torch.from_numpy((i["ids"] < 0) | (i["ids"] == 1)).cuda()
    for key in ("x", "dy"):
        i[key] = torch.where(bad[:, None], torch.full_like(i[key], float("nan")), i[key])
    i["A"][1] = float("inf")
    out, u, dx, dA, dB = _run(i, T, d, w, n, r)
    for a, b in zip((out, u, dx), (good[0], good[1], good[2])):
        assert torch.equal(a[~bad], b[~bad])
    for a, b in zip((dA, dB), (good[3], good[4])):
        assert torch.equal(a[[0, 2]], b[[0, 2]])
    none = torch.from_numpy(i["ids"] < 0).cuda()
    assert torch.equal(out[none], i["base"][none]) and torch.equal(dx[none], i["dx_add"][none])


@pytest.mark.parametrize("T,n", [(1, 1), (64, 64), (1000, 1), (5000, 37), (3000, 1024), (0, 4)])
def test_plan_is_a_stable_grouping(T, n):
    """Read back through an identity adapter: u = scale_a * x_a marks each row."""
    rng = np.random.default_rng(T + n)
    ids = rng.integers(-1, n, T).astype(np.int32)
    cfg = _cfg(T, 8, 8)
    plan = _plan(cfg, n, ids)
    x = torch.from_numpy(rng.integers(1, 100, (T, 8)).astype(np.float32)).cuda().bfloat16()
    A = torch.eye(8, device="cuda").bfloat16().repeat(n, 1, 1)
    scale = torch.arange(n, device="cuda", dtype=torch.float32) + 1
    u = torch.full((T, 8), -1.0, device="cuda")
    out = torch.empty((T, 8), device="cuda", dtype=torch.bfloat16)
    api.moe_adapter(cfg, plan, x, A, A, scale, None, out, u)
    torch.cuda.synchronize()
    assert api.moe_device_status(plan) == 0
    want = np.where((ids >= 0)[:, None], (ids[:, None] + 1.0) * _f64(x), -1.0)
    assert np.array_equal(_f64(u), want)


def test_bad_adapter_index_is_reported_and_treated_as_none():
    T, d, w, n, r = 90, 64, 64, 3, 8
    i = _inputs(T, d, w, n, r, seed=5)
    cfg = _cfg(T, d, w)
    outs = []
    for bad in (-1, n, 2 ** 31 - 1):
        i["ids"][40] = bad
        plan = _plan(cfg, n, i["ids"])
        out = torch.empty_like(i["base"])
        api.moe_adapter(cfg, plan, i["x"], i["A"], i["B"], i["scale"], i["base"], out, None)
        assert api.moe_device_status(plan) == (0 if bad < 0 else 1)
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_foreign_plan_is_reported_and_nothing_is_written():
    T, d, w, n, r = 90, 64, 64, 3, 8
    i = _inputs(T, d, w, n, r, seed=6)
    cfg, other = _cfg(T, d, w), _cfg(T - 1, d, w)
    blank = api.alloc_adapter_plan(cfg, n)
    wrong_t = _plan(other, n, i["ids"][:-1])
    wrong_t = torch.cat([wrong_t, torch.zeros(4096, dtype=torch.uint8, device="cuda")])
    wrong_n = _plan(cfg, n + 1, i["ids"])
    for plan in (blank, wrong_t, wrong_n):
        out = torch.full((T, w), 5.0, device="cuda", dtype=torch.bfloat16)
        api.moe_adapter(cfg, plan, i["x"], i["A"], i["B"], i["scale"], i["base"], out, None)
        assert api.moe_device_status(plan) == 5
        assert (out == 5.0).all()
        dx, dA = torch.full((T, d), 5.0, device="cuda"), torch.full((n, d, r), 5.0, device="cuda")
        dB = torch.full((n, r, w), 5.0, device="cuda")
        api.moe_adapter_backward(cfg, plan, i["x"], torch.zeros(T, r, device="cuda"), i["dy"],
                                 i["A"], i["B"], i["scale"], None, dx, dA, dB,
                                 api.alloc_adapter_workspace(cfg, n, r))
        assert api.moe_device_status(plan) == 5
        assert (dx == 5.0).all() and (dA == 5.0).all() and (dB == 5.0).all()


def test_no_tokens():
    d, w, n, r = 64, 72, 2, 8
    cfg = _cfg(0, d, w)
    plan = _plan(cfg, n, np.zeros(0, np.int32))
    i = _inputs(1, d, w, n, r, seed=7)
    e = lambda *s, dt=torch.float32: torch.empty(s, device="cuda", dtype=dt)
    bf = torch.bfloat16
    out, u = e(0, w, dt=bf), e(0, r)
    api.moe_adapter(cfg, plan, e(0, d, dt=bf), i["A"], i["B"], i["scale"], None, out, u)
    dA, dB = torch.full((n, d, r), 5.0, device="cuda"), torch.full((n, r, w), 5.0, device="cuda")
    api.moe_adapter_backward(cfg, plan, e(0, d, dt=bf), u, e(0, w, dt=bf), i["A"], i["B"],
                             i["scale"], None, e(0, d), dA, dB,
                             api.alloc_adapter_workspace(cfg, n, r))
    torch.cuda.synchronize()
    assert (dA == 0).all() and (dB == 0).all()


@pytest.mark.parametrize("T", [64, 3000, 5000])
def test_repeats_bit_exact(T):
    i = _inputs(T, 264, 136, 2, 32, seed=8)
    for a, b in zip(_run(i, T, 264, 136, 2, 32), _run(i, T, 264, 136, 2, 32)):
        assert torch.equal(a.nan_to_num(7), b.nan_to_num(7))


def test_captured_step_with_new_requests_on_another_stream():
    """The plan, the adapters and their backward in one graph; a replay after
    the requests' adapters and tokens changed gives the eager call's bits."""
    T, d, w, n, r = 130, 136, 200, 5, 16
    i, j = (_inputs(T, d, w, n, r, seed=s) for s in (9, 10))
    cfg = _cfg(T, d, w)
    plan, ws = api.alloc_adapter_plan(cfg, n), api.alloc_adapter_workspace(cfg, n, r)
    keys = ("x", "A", "B", "scale", "base", "dy", "dx_add")
    t = {k: i[k].clone() for k in keys}
    ids = torch.from_numpy(i["ids"]).cuda()
    out, u = torch.empty_like(t["base"]), torch.full((T, r), float("nan"), device="cuda")
    dx, dA, dB = torch.empty_like(t["dx_add"]), torch.empty(n, d, r, device="cuda"), \
        torch.empty(n, r, w, device="cuda")

    def step():
        api.moe_adapter_plan(cfg, n, ids, plan)
        api.moe_adapter(cfg, plan, t["x"], t["A"], t["B"], t["scale"], t["base"], out, u)
        api.moe_adapter_backward(cfg, plan, t["x"], u, t["dy"], t["A"], t["B"], t["scale"],
                                 t["dx_add"], dx, dA, dB, ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for q in (j, i, j):
        for k in keys:
            t[k].copy_(q[k])
        ids.copy_(torch.from_numpy(q["ids"]))
        u.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want = _run(q, T, d, w, n, r)
        for a, b in zip((out, u, dx, dA, dB), want):
            assert torch.equal(a.nan_to_num(7), b.nan_to_num(7))


def test_two_layers_share_a_plan():
    T, n = 77, 3
    i, j = _inputs(T, 64, 136, n, 8, seed=11), _inputs(T, 64, 136, n, 16, seed=12)
    cfg = _cfg(T, 64, 136)
    plan = _plan(cfg, n, i["ids"])
    for q in (i, j, i):
        out = torch.empty_like(q["base"])
        api.moe_adapter(cfg, plan, q["x"], q["A"], q["B"], q["scale"], q["base"], out, None)
        ref = _run({**q, "ids": i["ids"]}, T, 64, 136, n, q["A"].shape[2])[0]
        assert torch.equal(out, ref)


def test_two_streams_share_a_plan():
    """Two layers' backwards at once, each with its own workspace."""
    T, d, w, n, r = 5000, 264, 136, 3, 32
    ins = [_inputs(T, d, w, n, r, seed=s) for s in (13, 14)]
    ins[1]["ids"] = ins[0]["ids"]
    cfg = _cfg(T, d, w)
    plan = _plan(cfg, n, ins[0]["ids"])
    want = [_run(i, T, d, w, n, r) for i in ins]
    streams = [torch.cuda.Stream() for _ in ins]
    e = lambda *s: torch.empty(s, device="cuda")
    bufs = [(torch.empty_like(i["base"]), torch.full((T, r), float("nan"), device="cuda"), e(T, d),
             e(n, d, r), e(n, r, w), api.alloc_adapter_workspace(cfg, n, r)) for i in ins]
    torch.cuda.synchronize()
    for _ in range(3):
        for i, s, (out, u, dx, dA, dB, ws) in zip(ins, streams, bufs):
            with torch.cuda.stream(s):
                api.moe_adapter(cfg, plan, i["x"], i["A"], i["B"], i["scale"], i["base"], out, u)
                api.moe_adapter_backward(cfg, plan, i["x"], u, i["dy"], i["A"], i["B"],
                                         i["scale"], i["dx_add"], dx, dA, dB, ws)
    torch.cuda.synchronize()
    assert api.moe_device_status(plan) == 0
    for b, q in zip(bufs, want):
        for x, y in zip(b[:5], q):
            assert torch.equal(x.nan_to_num(7), y.nan_to_num(7))
