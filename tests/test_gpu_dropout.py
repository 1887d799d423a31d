"""Dropout, alone and in the combine, against the fp64 oracle.

The mask is exact: an element that the oracle drops equals the addend.  fp32
elements: one product by a scale rounded to fp32 and one add, each at most
half a step: 2 * 2^-24 |x scale| + 2^-24 |out|; bf16 adds 2^-8 |out| for the
output's rounding.  The combine's sum is a chain of k fused multiply-adds:
k * 2^-24 sum_j |g y| before the scale.
"""
import numpy as np
import pytest
import torch

from gpu_util import dev, host
from mixture_experts_top_b200 import api
from oracle import moe_oracle as O
from oracle import packed_oracle as Q

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SEED, OFFSET = 0xDEADBEEF12345678, (9 << 32) + 5


def _cfg(T, d_out=64, E=8, k=2, dtype="bf16", cf=0.0):
    return api.make_config(T, 8, 8, d_out, E, k, "swiglu" if dtype == "bf16" else "linear", dtype,
                           cf)


def _f64(t):
    return t.detach().double().cpu().numpy()


def _rand(g, *shape, dtype):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("T,width", [(1, 8), (3, 24), (64, 768), (257, 1000), (5, 4104)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1 - 2.0 ** -16])
def test_dropout(T, width, dtype, p):
    g = _gen(T + width)
    x, add = _rand(g, T, width, dtype=dtype), _rand(g, T, width, dtype=dtype)
    cfg = _cfg(T)
    keep = Q.keep_mask(T, width, p, SEED, OFFSET, 11)
    scale = 65536.0 / (65536.0 - Q.threshold(p))
    for a in (None, add):
        out = torch.full_like(x, float("nan"))
        api.moe_dropout(cfg, p, SEED, OFFSET, 11, x, a, out)
        ref = Q.dropout(_f64(x), p, SEED, OFFSET, 11, None if a is None else _f64(a))
        got = _f64(out)
        half = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
        lim = 2 * U * np.abs(_f64(x) * scale) + (U + half) * np.abs(ref) + 1e-38
        assert np.all(np.abs(got - ref) <= lim)
        want = np.zeros_like(got) if a is None else _f64(a)
        assert np.array_equal(got[~keep], want[~keep])
    if p == 0.0:
        assert torch.equal(out, (x.float() + add.float()).to(dtype))


@pytest.mark.parametrize("token_base", [0, 1, 2 ** 31 + 5, 2 ** 40])
def test_counters_past_32_bits(token_base):
    T, width = 9, 40
    x = torch.ones(T, width, device="cuda")
    out = torch.empty_like(x)
    api.moe_dropout(_cfg(T), 0.5, SEED, 2 ** 64 - 1, token_base, x, None, out)
    keep = Q.keep_mask(T, width, 0.5, SEED, 2 ** 64 - 1, token_base)
    assert np.array_equal(host(out) == 2.0, keep)


def test_rows_of_a_sharded_batch_draw_the_batch_mask():
    T, width = 30, 64
    x = torch.ones(T, width, device="cuda", dtype=torch.bfloat16)
    whole, part = torch.empty_like(x), torch.empty_like(x)
    api.moe_dropout(_cfg(T), 0.3, 7, 8, 0, x, None, whole)
    for lo, hi in ((0, 11), (11, 12), (12, 30)):
        rows = part[lo:hi]
        api.moe_dropout(_cfg(hi - lo), 0.3, 7, 8, lo, x[lo:hi], None, rows)
    assert torch.equal(whole, part)


def test_seed_and_offset_change_the_mask():
    x = torch.ones(64, 64, device="cuda")
    outs = []
    for seed, offset in ((1, 1), (2, 1), (1, 2), (1 + 2 ** 32, 1), (1, 1 + 2 ** 32)):
        out = torch.empty_like(x)
        api.moe_dropout(_cfg(64), 0.5, seed, offset, 0, x, None, out)
        outs.append(host(out))
    for i in range(5):
        for j in range(i):
            assert 0.3 < (outs[i] == outs[j]).mean() < 0.7


def test_in_place_and_the_gradient():
    """out may be x or add; the gradient is the same call on the gradient."""
    g = _gen(3)
    x, add = _rand(g, 50, 72, dtype=torch.float32), _rand(g, 50, 72, dtype=torch.float32)
    cfg, out = _cfg(50), torch.empty_like(x)
    api.moe_dropout(cfg, 0.2, 5, 6, 0, x, add, out)
    a, b = x.clone(), add.clone()
    api.moe_dropout(cfg, 0.2, 5, 6, 0, a, add, a)
    api.moe_dropout(cfg, 0.2, 5, 6, 0, x, b, b)
    assert torch.equal(a, out) and torch.equal(b, out)
    # d/dx <w, dropout(x)> = dropout(w): the map is linear and symmetric
    w, dx = _rand(g, 50, 72, dtype=torch.float32), torch.empty_like(x)
    y = torch.empty_like(x)
    api.moe_dropout(cfg, 0.2, 5, 6, 0, w, None, dx)
    api.moe_dropout(cfg, 0.2, 5, 6, 0, x, None, y)
    lhs, rhs = (w.double() * y.double()).sum(), (dx.double() * x.double()).sum()
    scale = (w.double() * y.double()).abs().sum()
    assert abs(lhs - rhs) <= 8 * U * scale


def test_dropped_infinities_and_nan_have_no_effect():
    T, width = 40, 64
    keep = torch.from_numpy(Q.keep_mask(T, width, 0.5, 3, 4)).cuda()
    x = torch.ones(T, width, device="cuda", dtype=torch.bfloat16)
    bad = torch.where(keep, x, torch.full_like(x, float("nan")))
    bad[:, ::3] = torch.where(keep, x, torch.full_like(x, float("inf")))[:, ::3]
    out = torch.empty_like(x)
    api.moe_dropout(_cfg(T), 0.5, 3, 4, 0, bad, x, out)
    assert torch.equal(out, x + 2.0 * keep.to(x.dtype))


def test_no_rows():
    x = torch.empty((0, 64), device="cuda")
    api.moe_dropout(_cfg(0), 0.5, 3, 4, 0, x, None, x)
    torch.cuda.synchronize()


def _combine_case(T, d_out, E, k, dtype, cf, seed):
    rng = np.random.default_rng(seed)
    idx = np.argsort(rng.random((T, E)) + (np.arange(E) >= E // 2) * 0.3, axis=1)[:, :k]
    d = O.dispatch(idx.astype(np.int32), E, cf)
    act = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = _gen(seed)
    t = dict(y=_rand(g, T * k, d_out, dtype=torch.float32), dest=dev(d["dest"].astype(np.int32)),
             gates=torch.softmax(_rand(g, T, k, dtype=torch.float32), 1),
             res=_rand(g, T, d_out, dtype=act), dy=_rand(g, T, d_out, dtype=act))
    return _cfg(T, d_out, E, k, dtype, cf), t, d["dest"], act


@pytest.mark.parametrize("T,d_out,E,k,dtype,cf", [
    (1, 8, 2, 1, "bf16", 0.0), (65, 264, 8, 2, "bf16", 0.0), (200, 768, 16, 1, "bf16", 0.5),
    (77, 1032, 16, 6, "bf16", 0.4), (64, 32, 8, 2, "f32", 0.0), (130, 520, 8, 8, "f32", 0.7),
    (33, 2056, 64, 6, "bf16", 0.3), (17, 4104, 16, 8, "f32", 0.0), (9, 8200, 8, 5, "bf16", 0.2),
    (50, 1536, 8, 4, "bf16", 0.5)])
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_combine(T, d_out, E, k, dtype, cf, p):
    cfg, t, dest, act = _combine_case(T, d_out, E, k, dtype, cf, T + k)
    drop = (p, SEED, OFFSET, 4)
    keep = Q.keep_mask(T, d_out, *drop)
    scale = 65536.0 / (65536.0 - Q.threshold(p))
    Y, gates = _f64(t["y"]), _f64(t["gates"])
    s = O.combine(Y, dest, gates)
    mag = O.combine(np.abs(Y), dest, gates)
    half = 2.0 ** -8 if dtype == "bf16" else 0.0
    for res in (None, t["res"]):
        out = torch.full((T, d_out), float("nan"), dtype=act, device="cuda")
        api.moe_combine_dropout(cfg, *drop, t["y"], t["dest"], t["gates"], res, out)
        r = 0.0 if res is None else _f64(res)
        ref = r + np.where(keep, s * scale, 0.0)
        lim = (k + 2) * U * scale * mag + (U + half) * np.abs(ref) + 1e-38
        assert np.all(np.abs(_f64(out) - ref) <= lim)
    place = t["res"].clone()
    api.moe_combine_dropout(cfg, *drop, t["y"], t["dest"], t["gates"], place, place)
    assert torch.equal(place, out)
    # backward: rows of dropped slots stay as they were
    dyp = torch.full((T * k, d_out), 9.0, device="cuda")
    dg = torch.full((T, k), float("nan"), device="cuda")
    api.moe_combine_dropout_backward(cfg, *drop, t["dy"], t["y"], t["dest"], t["gates"], dyp, dg)
    D = np.where(keep, _f64(t["dy"]) * scale, 0.0)
    dY, dG = O.combine_backward(Y, dest, gates, D)
    kept = dest[dest >= 0]
    got = _f64(dyp)
    assert np.all(np.abs(got[kept] - dY[kept]) <= 4 * U * np.abs(dY[kept]) + 1e-38)
    assert (got[np.setdiff1d(np.arange(T * k), kept)] == 9.0).all()
    lim = np.zeros((T, k))
    for i in range(T):
        for j in range(k):
            if dest[i, j] >= 0:
                lim[i, j] = np.abs(D[i]) @ np.abs(Y[dest[i, j]])
    assert np.all(np.abs(_f64(dg) - dG) <= (d_out + 4) * U * lim)
    assert (_f64(dg)[dest < 0] == 0).all()


@pytest.mark.parametrize("k", [3, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_dropout_it_is_the_combine(dtype, k):
    cfg, t, dest, act = _combine_case(300, 136, 8, k, dtype, 0.6, 5)
    a, b = (torch.empty((300, 136), dtype=act, device="cuda") for _ in range(2))
    api.moe_combine(cfg, t["y"], t["dest"], t["gates"], a)
    api.moe_combine_dropout(cfg, 0.0, 1, 2, 0, t["y"], t["dest"], t["gates"], None, b)
    assert torch.equal(a, b)
    da, db = (torch.zeros_like(t["y"]) for _ in range(2))
    ga, gb = (torch.empty((300, k), device="cuda") for _ in range(2))
    api.moe_combine_backward(cfg, t["dy"], t["y"], t["dest"], t["gates"], da, ga)
    api.moe_combine_dropout_backward(cfg, 0.0, 1, 2, 0, t["dy"], t["y"], t["dest"], t["gates"], db,
                                     gb)
    assert torch.equal(da, db)
    # the dot products' order is the kernel's own: d_out terms each
    lim = 2 * 140 * U * (t["dy"].double().abs().max() * t["y"].double().abs().max() * 136)
    assert torch.all((ga - gb).abs() <= lim)


def test_combine_drops_the_same_elements_as_dropout():
    """One generator: the combine's mask is moe_dropout's on (T, d_out) rows."""
    cfg, t, _, act = _combine_case(90, 256, 8, 2, "bf16", 0.0, 6)
    plain, both = (torch.empty((90, 256), device="cuda", dtype=act) for _ in range(2))
    api.moe_combine(cfg, t["y"], t["dest"], t["gates"], plain)
    api.moe_dropout(cfg, 0.4, 5, 5, 3, plain, None, both)
    fused = torch.empty_like(both)
    api.moe_combine_dropout(cfg, 0.4, 5, 5, 3, t["y"], t["dest"], t["gates"], None, fused)
    assert torch.equal(fused == 0, both == 0)


@pytest.mark.parametrize("k", [2, 8])
def test_combine_backward_ignores_dropped_infinities(k):
    cfg, t, dest, act = _combine_case(40, 64, 8, k, "bf16", 0.0, 7)
    keep = torch.from_numpy(Q.keep_mask(40, 64, 0.5, 1, 1)).cuda()
    args = (cfg, 0.5, 1, 1, 0)

    def run(dy, y):
        dyp, dg = torch.zeros_like(y), torch.empty((40, k), device="cuda")
        api.moe_combine_dropout_backward(*args, dy, y, t["dest"], t["gates"], dyp, dg)
        return dyp, dg

    dy = torch.where(keep, t["dy"], torch.full_like(t["dy"], float("nan")))
    row = torch.zeros(40 * k, dtype=torch.int64, device="cuda")
    row[t["dest"].long().reshape(-1)] = torch.arange(40, device="cuda").repeat_interleave(k)
    y = torch.where(keep[row], t["y"], torch.full_like(t["y"], float("inf")))
    for a, b in zip(run(t["dy"], t["y"]), run(dy, y)):
        assert torch.equal(a, b)


def test_captured_graph_draws_a_fresh_mask_from_the_device_offset():
    T, width = 33, 80
    x = torch.ones(T, width, device="cuda")
    out = torch.empty_like(x)
    off = torch.tensor([100], dtype=torch.int64, device="cuda")
    cfg = _cfg(T)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        api.moe_dropout(cfg, 0.5, 3, off, 0, x, None, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        api.moe_dropout(cfg, 0.5, 3, off, 0, x, None, out)
        off.add_(1)
    for step in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(out) == 2.0, Q.keep_mask(T, width, 0.5, 3, 100 + step))


def test_binding_checks_devices_and_shapes():
    cfg, t, _, act = _combine_case(10, 64, 8, 2, "bf16", 0.0, 8)
    x = torch.ones(10, 64, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        api.moe_dropout(cfg, 0.1, 0, 0, 0, x.t().contiguous().t(), None, torch.empty_like(x))
    with pytest.raises(ValueError, match="add must be"):
        api.moe_dropout(cfg, 0.1, 0, 0, 0, x, x.bfloat16(), torch.empty_like(x))
    with pytest.raises(api.MoeError, match="multiple of 8"):
        y = torch.ones(10, 12, device="cuda")
        api.moe_dropout(cfg, 0.1, 0, 0, 0, y, None, torch.empty_like(y))
    with pytest.raises(api.MoeError, match="p must be"):
        api.moe_dropout(cfg, 1.0, 0, 0, 0, x, None, torch.empty_like(x))
    with pytest.raises(ValueError, match="residual must be"):
        api.moe_combine_dropout(cfg, 0.1, 0, 0, 0, t["y"], t["dest"], t["gates"], x, t["res"])
