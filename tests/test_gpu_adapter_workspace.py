"""The adapters' backward keeps to its workspace, whose parts are as many as the
chunks that the rows are cut into and the adapters that a chunk's end can cut, not
as many as the adapters."""
import pytest
import torch

from mixture_experts_top_b200 import api

U = 2.0 ** -24


def _cfg(T, d, d_out):
    return api.make_config(T, d, 8, d_out, 8, 2, "swiglu", "bf16")


def test_size_does_not_follow_the_gradients(moe_lib):
    """A decode-sized batch on many adapters: rows by tile slot are T + 16 (n + 1) at
    most, in chunks of 960 at least; a chunk's part is r (d + d_out) fp32."""
    T, d, r = 64, 4096, 128
    for n in (256, 1024):
        rows = T + 16 * (n + 1)
        chunks = max(rows // 960 + 1, 2 * 200 // 64)
        part = r * 2 * d * 4
        size = api.moe_adapter_workspace_size(_cfg(T, d, d), n, r)
        assert size <= 2 * chunks * part + 2 * (rows * r * 6 + 256) + 256
        assert size < n * part // 4                   # the gradients are n parts
    # few adapters: a part for each chunk and each adapter
    few = api.moe_adapter_workspace_size(_cfg(8192, 2048, 2048), 1, 64)
    assert few <= api.moe_adapter_workspace_size(_cfg(8192, 2048, 2048), 8, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,w,n,r", [
    (64, 264, 136, 300, 16), (3000, 72, 136, 1000, 8), (9000, 40, 72, 3, 8), (9000, 40, 72, 200, 8),
    (40000, 24, 16, 1, 8), (40000, 24, 16, 37, 16), (6144, 136, 72, 64, 24), (2048, 2048, 512, 8, 96),
    (3000, 72, 136, 200, 128), (9000, 136, 72, 130, 128)])
@pytest.mark.parametrize("spread", ["even", "random", "one"])
def test_parts_stay_inside(T, d, w, n, r, spread):
    g = torch.Generator(device="cuda").manual_seed(T + n)
    bf = torch.bfloat16
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    ids = {"even": torch.arange(T, device="cuda") * n // T,
           "random": torch.randint(-1, n, (T,), generator=g, device="cuda"),
           "one": torch.full((T,), n // 2, device="cuda")}[spread].to(torch.int32)
    x, dy = rnd(T, d).to(bf), rnd(T, w).to(bf)
    A, B, scale = (rnd(n, d, r) / d ** 0.5).to(bf), (rnd(n, r, w) / r ** 0.5).to(bf), rnd(n)
    cfg = _cfg(T, d, w)
    plan = api.alloc_adapter_plan(cfg, n)
    api.moe_adapter_plan(cfg, n, ids, plan)
    out, u = torch.empty(T, w, device="cuda", dtype=bf), torch.zeros(T, r, device="cuda")
    api.moe_adapter(cfg, plan, x, A, B, scale, None, out, u)
    e = lambda *s: torch.full(s, float("nan"), device="cuda")
    dx, dA, dB = e(T, d), e(n, d, r), e(n, r, w)
    size = api.moe_adapter_workspace_size(cfg, n, r)
    room = torch.full((size + (64 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    api.moe_adapter_backward(cfg, plan, x, u, dy, A, B, scale, None, dx, dA, dB, room[:size])
    assert api.moe_device_status(plan) == 0
    assert bool((room[size:] == 0xA5).all())
    for a in (range(n) if n < 100 else list(range(0, n, 37)) + [n // 2, n - 1]):
        m = ids == a
        xa, ya = x[m].double(), dy[m].double()
        s, Aa, Ba = scale[a].double(), A[a].double(), B[a].double()
        v, ua = s * (ya @ Ba.T), s * (xa @ Aa)
        mv, mu = s.abs() * (ya.abs() @ Ba.abs().T), s.abs() * (xa.abs() @ Aa.abs())
        # the operands' sums and the rows', each truncated: 2 units an addition
        lim = 2 * (max(d, w) + int(m.sum()) + 4) * U
        for got, p, q, mp, mq in ((dA[a], xa.T, v, xa.abs().T, mv),
                                  (dB[a], ua.T, ya, mu.T, ya.abs())):
            assert torch.all((got.double() - p @ q).abs() <= lim * (mp @ mq) + 1e-30), a
