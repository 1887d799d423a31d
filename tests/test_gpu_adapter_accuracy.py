"""What the adapters' products keep of u and v, where the elementwise bounds of
random inputs are too wide to tell: sums by blocks of 256 input columns, three
bf16 terms (24 bits) for the gradients, and outputs that do not depend on
whether u is kept.

The exact cases have one non-zero product in every sum that a lost bit could
hide in, so that nothing but the operand's own representation is rounded.  With s = 1 + 2^-9 +
2^-17 - 2^-23, s - bf16(s) = 2^-9 + (2^-17 - 2^-23) and the third bf16 term is
2^-17 - 2^-23 = 126 units of 2^-24: without it every gradient is 126 units off.

Normwise limits of random inputs, in units u = 2^-24.  The tensor core truncates
its running sum once every 16 products, by 0.7 u of it on average, and the sum
of n steps of independent products grows with sqrt(n).  u, v: 16 steps a block
give 0.7 * 0.8 * sum_j sqrt(j) / 4 <= 7 u of a block's root mean square, and the
blocks' signs are independent: 7, 16 with a margin of two and the fp32 sum of the
blocks.  dx: v's, and 3 r / 16 <= 24 steps more, the three terms' alike: at most
0.7 * 16 u more: 32.  dA, dB: v's (u's), and 64 steps a chunk of rows: 0.7 * 0.8 *
343 / 8 = 24: 40.
"""
import numpy as np
import pytest
import torch

from mixture_experts_top_b200 import api

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
S = 1 + 2.0 ** -9 + 2.0 ** -17 - 2.0 ** -23
BF = torch.bfloat16


def _cfg(T, d, d_out):
    return api.make_config(T, d, 8, d_out, 8, 2, "swiglu", "bf16")


def _step(x, dy, A, B, scale, ids, dx_add=None):
    """u, dx, dA, dB of an adapter step."""
    (T, d), w, (n, _, r) = x.shape, dy.shape[1], A.shape
    cfg = _cfg(T, d, w)
    plan = api.alloc_adapter_plan(cfg, n)
    api.moe_adapter_plan(cfg, n, ids, plan)
    e = lambda *s: torch.full(s, float("nan"), device="cuda")
    out, u, dx, dA, dB = e(T, w).to(BF), e(T, r), e(T, d), e(n, d, r), e(n, r, w)
    ws = api.alloc_adapter_workspace(cfg, n, r)
    api.moe_adapter(cfg, plan, x, A, B, scale, None, out, u)
    api.moe_adapter_backward(cfg, plan, x, u, dy, A, B, scale, dx_add, dx, dA, dB, ws)
    assert api.moe_device_status(plan) == 0
    return u, dx, dA, dB


# few rows, clusters; 64-row clusters; tcgen05 at each of its shapes
SHAPES = [(60, 136, 72, 3, 16), (100, 264, 136, 2, 128), (1500, 136, 264, 4, 40),
          (2000, 72, 136, 2, 64), (4900, 136, 264, 5, 64), (6700, 72, 136, 3, 16),
          (6700, 264, 72, 3, 8), (5000, 136, 520, 2, 88), (6000, 520, 136, 4, 128),
          (20000, 136, 136, 2, 32)]


@pytest.mark.parametrize("T,d,w,n,r", SHAPES)
def test_gradients_keep_24_bits(T, d, w, n, r):
    """Row i of an adapter is one-hot in x at column i mod d and in dy at i mod w;
    A and B have one 1 in each row of A and column of B.  Then u = v = s (at the
    column's rank index), dx = s at A's column's ones, and an adapter's gradients
    are whole multiples of s: a sum of identical values, each of whose terms'
    sums is exact; the three terms' sum, and one fp32 addition for each of
    the parts that an adapter's rows are cut into, are rounded."""
    ids = (torch.arange(T, device="cuda") * 7919 % T * n // T).to(torch.int32)
    pos = torch.zeros(T, dtype=torch.int64, device="cuda")
    for a in range(n):
        m = ids == a
        pos[m] = torch.arange(int(m.sum()), device="cuda")
    t = torch.arange(T, device="cuda")
    x, dy = torch.zeros(T, d, device="cuda"), torch.zeros(T, w, device="cuda")
    x[t, pos % d], dy[t, pos % w] = 1, 1
    A, B = torch.zeros(n, d, r, device="cuda"), torch.zeros(n, r, w, device="cuda")
    A[:, torch.arange(d), torch.arange(d) % r] = 1
    B[:, torch.arange(w) % r, torch.arange(w)] = 1
    sign = torch.tensor([1.0, -2.0, 0.5, 4.0, -0.25], device="cuda")[:n]
    scale = (sign.double() * S).float()
    assert torch.equal(scale.double(), sign.double() * S)
    u, dx, dA, dB = _step(x.to(BF), dy.to(BF), A.to(BF), B.to(BF), scale, ids)
    sc = scale.double()[ids.long()][:, None]
    ur, vr = torch.zeros(T, r, device="cuda").double(), torch.zeros(T, r, device="cuda").double()
    ur[t, pos % d % r], vr[t, pos % w % r] = 1, 1
    assert torch.equal(u.double(), ur * sc)
    A, B, x, dy = A.double(), B.double(), x.double(), dy.double()
    dxr = torch.zeros(T, d, device="cuda").double()
    dAr, dBr = torch.zeros_like(A), torch.zeros_like(B)
    for a in range(n):
        m = ids == a
        dxr[m] = sc[m] * (vr[m] @ A[a].T)
        dAr[a], dBr[a] = x[m].T @ (sc[m] * vr[m]), (sc[m] * ur[m]).T @ dy[m]
    assert torch.equal(dx.double(), dxr)
    parts = T // 256 + 2
    for got, ref in ((dA, dAr), (dB, dBr)):
        assert torch.all((got.double() - ref).abs() <= (2 + parts) * U * ref.abs())
        assert parts + 2 < 126


@pytest.mark.parametrize("T,n,r", [(60, 3, 16), (1500, 3, 64), (5000, 3, 64), (6700, 3, 16),
                                   (6000, 3, 128)])
def test_small_products_behind_a_large_one(T, n, r):
    """u's and v's columns are summed by blocks of at most 256: products of 2^-27
    behind one of 1, each lost to a truncated fp32 sum, are lost in the first block
    alone (255 of them: 32 units), not in all (2047: 256 units)."""
    d = w = 2048
    x, dy = torch.full((T, d), 2.0 ** -27, device="cuda"), torch.full((T, w), 2.0 ** -27,
                                                                    device="cuda")
    x[:, 0], dy[:, 0] = 1, 1
    A, B = torch.ones(n, d, r, device="cuda", dtype=BF), torch.ones(n, r, w, device="cuda",
                                                                   dtype=BF)
    ids = (torch.arange(T, device="cuda") % n).to(torch.int32)
    u, dx, _, _ = _step(x.to(BF), dy.to(BF), A, B, torch.ones(n, device="cuda"), ids)
    want = 1 + 2047 * 2.0 ** -27
    assert float((u.double() - want).abs().max()) <= 36 * U
    # dx = r v, each of at most 3 r / 16 truncated additions within 2 units
    assert float((dx.double() / (r * want) - 1).abs().max()) <= (36 + 2 * 24 + 2) * U


@pytest.mark.parametrize("T,d,w,n,r", [(5200, 1032, 520, 3, 64), (8192, 2048, 2048, 8, 64),
                                       (5000, 776, 1032, 2, 88), (6000, 1544, 520, 3, 128),
                                       (8192, 1032, 776, 6, 16)])
def test_normwise(T, d, w, n, r):
    g = torch.Generator(device="cuda").manual_seed(T + r)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, dy = rnd(T, d).to(BF), rnd(T, w).to(BF)
    A, B, scale = (rnd(n, d, r) / d ** 0.5).to(BF), (rnd(n, r, w) / r ** 0.5).to(BF), rnd(n)
    ids = torch.randint(-1, n, (T,), generator=g, device="cuda").to(torch.int32)
    u, dx, dA, dB = _step(x, dy, A, B, scale, ids)
    x, dy, A, B, scale = (v.double() for v in (x, dy, A, B, scale))

    def off(got, ref):
        return float((got.double() - ref).norm() / ref.norm()) / U

    worst = dict(u=0.0, dx=0.0, dA=0.0, dB=0.0)
    for a in range(n):
        m = ids == a
        ur, vr = scale[a] * (x[m] @ A[a]), scale[a] * (dy[m] @ B[a].T)
        for q, got, ref in (("u", u[m], ur), ("dx", dx[m], vr @ A[a].T), ("dA", dA[a], x[m].T @ vr),
                            ("dB", dB[a], ur.T @ dy[m])):
            worst[q] = max(worst[q], off(got, ref))
    assert worst["u"] <= 16 and worst["dx"] <= 32 and worst["dA"] <= 40 and worst["dB"] <= 40, worst


@pytest.mark.parametrize("T,d,r", [(60, 2048, 16), (1500, 2048, 64), (5000, 776, 32),
                                   (6700, 2048, 16), (8192, 2056, 64), (6000, 4104, 128)])
def test_output_is_the_same_with_and_without_u(T, d, r):
    """Serving (no u) and training give the same bits."""
    n, w = 3, 520
    g = torch.Generator(device="cuda").manual_seed(T + d)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, base = rnd(T, d).to(BF), rnd(T, w).to(BF)
    A, B, scale = (rnd(n, d, r) / d ** 0.5).to(BF), (rnd(n, r, w) / r ** 0.5).to(BF), rnd(n)
    ids = torch.randint(-1, n, (T,), generator=g, device="cuda").to(torch.int32)
    cfg = _cfg(T, d, w)
    plan = api.alloc_adapter_plan(cfg, n)
    api.moe_adapter_plan(cfg, n, ids, plan)
    outs = []
    for u in (torch.empty(T, r, device="cuda"), None):
        outs.append(torch.empty(T, w, device="cuda", dtype=BF))
        api.moe_adapter(cfg, plan, x, A, B, scale, base, outs[-1], u)
    assert api.moe_device_status(plan) == 0
    assert torch.equal(*outs)
    uref = torch.zeros(T, r, device="cuda").double()
    ref = base.double()
    for a in range(n):
        m = ids == a
        uref[m] = scale[a].double() * (x[m].double() @ A[a].double())
        ref[m] += uref[m] @ B[a].double()
    mag = torch.zeros_like(ref)
    for a in range(n):
        m = ids == a
        mag[m] = uref[m].abs() @ B[a].double().abs()
    # bf16's half step, u's 16 bits, the second product's truncated sums; u's own
    # error (16 units normwise, 2^-20) in a margin of 16 for single elements
    lim = 2.0 ** -8 * ref.abs() + (2.0 ** -16 + 4 * r * U) * mag + 2.0 ** -16 * mag.mean()
    assert torch.all((outs[1].double() - ref).abs() <= lim)
