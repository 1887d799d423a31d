"""The packed-batch calls of the binding: a required tensor that is None is the
library's refusal by name, as in the other calls, and a mask may be torch.bool."""
import pytest
import torch

from mixture_experts_top_b200 import api

CFG = dict(T=4, d=8, d_hidden=8, d_out=16, E=4, top_k=2, kind="swiglu", dtype="bf16")


def _cfg():
    return api.make_config(**CFG)


def _refused(name, f, *args):
    with pytest.raises(api.MoeError) as e:
        f(*args)
    assert e.value.status == api.MOE_ERR_INVALID_ARG and f"{name} is NULL" in str(e.value)


def test_none_is_refused_by_name(moe_lib):
    c, no = _cfg(), None
    _refused("logits", api.moe_balance_loss, c, no, no, no, no, no, no, no, no, no)
    _refused("logits", api.moe_balance_loss_backward, c, no, no, no, no, no, no, no, no)
    _refused("x", api.moe_dropout, c, 0.1, 0, 0, 0, no, no, no)
    _refused("y_perm", api.moe_combine_dropout, c, 0.1, 0, 0, 0, no, no, no, no, no)
    _refused("dy", api.moe_combine_dropout_backward, c, 0.1, 0, 0, 0, no, no, no, no, no, no)
    _refused("A", api.moe_adapter, c, no, no, no, no, no, no, no, no)
    _refused("A", api.moe_adapter_backward, c, no, no, no, no, no, no, no, no, no, no, no, no)
    _refused("token_adapter", api.moe_adapter_plan, c, 3, no, no)
    _refused("dlogits_add", api.moe_route_backward_add, c, no, no, no, no, no, no, no, no, 0, no,
             no, no, no, no, no)


def test_none_workspace_is_refused(moe_lib):
    c = api.make_config(**{**CFG, "T": 0})
    with pytest.raises(api.MoeError, match="plan is NULL"):
        api.moe_adapter_plan(c, 3, None, None)


def _tensors():
    """Arguments of the calls below, by name, all valid."""
    T, d, w, E, k, n, r, S = 4, 8, 16, 4, 2, 3, 8, 2
    e = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device="cuda")
    i, bf = torch.int32, torch.bfloat16
    c = _cfg()
    off = torch.tensor([0, 2, 4], dtype=i, device="cuda")
    ids = e(T, dt=i)
    plan = api.alloc_adapter_plan(c, n)
    api.moe_adapter_plan(c, n, ids, plan)
    return c, dict(
        moe_balance_loss=[("seq_offsets", off), ("token_mask", None), ("logits", e(T, E)),
                          ("expert_indices", e(T, k, dt=i)), ("counts", e(S, E, dt=i)),
                          ("prob_mean", e(S, E)), ("tokens", e(S + 2, dt=i)), ("losses", e(2)),
                          ("workspace", api.alloc_balance_workspace(c, S))],
        moe_balance_loss_backward=[("seq_offsets", off), ("token_mask", None), ("logits", e(T, E)),
                                   ("counts", e(S, E, dt=i)), ("tokens", e(S + 2, dt=i)),
                                   ("dlosses", e(2)), ("dlogits", e(T, E)),
                                   ("workspace", api.alloc_balance_workspace(c, S))],
        moe_dropout=[("p", 0.1), ("seed", 1), ("offset", 2), ("base", 0), ("x", e(T, 8)),
                     ("add", None), ("out", e(T, 8))],
        moe_combine_dropout=[("p", 0.1), ("seed", 1), ("offset", 2), ("base", 0),
                             ("y_perm", e(T * k, w)), ("dest", e(T, k, dt=i)), ("gates", e(T, k)),
                             ("residual", None), ("output", e(T, w, dt=bf))],
        moe_combine_dropout_backward=[("p", 0.1), ("seed", 1), ("offset", 2), ("base", 0),
                                      ("dy", e(T, w, dt=bf)), ("y_perm", e(T * k, w)),
                                      ("dest", e(T, k, dt=i)), ("gates", e(T, k)),
                                      ("dy_perm", e(T * k, w)), ("dgates", e(T, k))],
        moe_adapter=[("plan", plan), ("x", e(T, d, dt=bf)), ("A", e(n, d, r, dt=bf)),
                     ("B", e(n, r, w, dt=bf)), ("scale", e(n)), ("base", None),
                     ("output", e(T, w, dt=bf)), ("u", None)],
        moe_adapter_backward=[("plan", plan), ("x", e(T, d, dt=bf)), ("u", e(T, r)),
                              ("dy", e(T, w, dt=bf)), ("A", e(n, d, r, dt=bf)),
                              ("B", e(n, r, w, dt=bf)), ("scale", e(n)), ("dx_add", None),
                              ("dx", e(T, d)), ("dA", e(n, d, r)), ("dB", e(n, r, w)),
                              ("workspace", api.alloc_adapter_workspace(c, n, r))])


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["moe_balance_loss", "moe_balance_loss_backward", "moe_dropout",
                                  "moe_combine_dropout", "moe_combine_dropout_backward",
                                  "moe_adapter", "moe_adapter_backward"])
def test_each_required_tensor(call):
    c, args = _tensors()
    args = args[call]
    getattr(api, call)(c, *[v for _, v in args])      # valid as it stands
    for at, (name, v) in enumerate(args):
        if not isinstance(v, torch.Tensor):
            continue
        values = [None if i == at else q for i, (_, q) in enumerate(args)]
        if name == "seq_offsets":                     # one sequence: the outputs' shapes differ
            with pytest.raises(ValueError, match="must have shape"):
                getattr(api, call)(c, *values)
            continue
        with pytest.raises(api.MoeError, match=f"{name} is NULL"):
            getattr(api, call)(c, *values)
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_bool_mask():
    c, args = _tensors()
    g = torch.Generator(device="cuda").manual_seed(3)
    L = torch.randn(4, 4, generator=g, device="cuda")
    got = []
    for mask in (torch.tensor([1, 0, 1, 1], dtype=torch.uint8, device="cuda"),
                 torch.tensor([True, False, True, True], device="cuda")):
        a = [v.clone() if isinstance(v, torch.Tensor) else v for _, v in args["moe_balance_loss"]]
        a[1], a[2] = mask, L
        api.moe_balance_loss(c, *a)
        b = [v.clone() if isinstance(v, torch.Tensor) else v
             for _, v in args["moe_balance_loss_backward"]]
        b[1], b[2], b[3], b[4] = mask, L, a[4], a[6]
        b[5] = torch.ones(2, device="cuda")
        api.moe_balance_loss_backward(c, *b)
        got.append([a[4], a[5], a[6], a[7], b[6]])
    for x, y in zip(*got):
        assert torch.equal(x, y)
    assert got[0][2].tolist() == [1, 2, 3, 2]
    with pytest.raises(ValueError, match="token_mask must be"):
        a[1] = torch.ones(4, device="cuda")
        api.moe_balance_loss(c, *a)
