"""Cases of the layer's training and serving operators on packed batches: what is
measured, in plain torch (`own = False`) and through the library (`own = True`).

Operators
* ``balance``: the balance loss and z-loss of packed, padded sequences with their
  per-expert counts, then the gradient with respect to the router's logits.
* ``dropout``: dropout of (T, width) rows whose mask comes from a counter-based
  generator and is never stored, added to another tensor.
* ``combine``: the gate-weighted combine with dropout and a residual, then its
  backward, which draws the same mask again.
* ``adapter``: low-rank adapters of many requests beside the output all requests
  share; with ``train`` also the gradients of x, A and B.

The generator is Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random
numbers: as easy as 1, 2, 3", SC 2011): block b of 8 consecutive elements of the
row-major tensor takes the counter (b low, b high, offset low, offset high) under
the key (seed low, seed high); element i of the block takes 16 bits, the low half
of word i / 2 for even i and the high half for odd i, and is kept where they are
at least round(65536 p).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one short request being tuned: latency only
        dict(name="balance_small", op="balance", T=64, E=8, k=2, S=1, mask=False, ragged=False),
        # the fine-grained layer's batch, packed from 23 sequences with padding
        dict(name="balance_packed", op="balance", T=16384, E=64, k=6, S=23, mask=True, ragged=True),
        # many experts, a large global batch of short documents
        dict(name="balance_large", op="balance", T=131072, E=256, k=8, S=311, mask=True,
             ragged=True),
        # a decode-sized batch of a narrow model
        dict(name="dropout_small", op="dropout", T=64, width=768, dtype="bf16", p=0.1, add=True),
        # the fp32 input gradient of the large layer on its way through dropout
        dict(name="dropout_grad", op="dropout", T=8192, width=4096, dtype="f32", p=0.1, add=True),
        # top-1 layer with capacity: dropped slots, residual
        dict(name="combine_top1", op="combine", T=4096, E=64, k=1, width=768, cf=1.25, p=0.1,
             dtype="bf16"),
        # the large top-2 layer's residual branch
        dict(name="combine_top2", op="combine", T=8192, E=8, k=2, width=4096, cf=0.0, p=0.1,
             dtype="bf16"),
        # fine-grained routing, odd token count and width
        dict(name="combine_top6_odd", op="combine", T=5003, E=64, k=6, width=2056, cf=1.0, p=0.3,
             dtype="bf16"),
        # decoding: 64 requests, each with an adapter of its own
        dict(name="adapter_decode", op="adapter", T=64, d=4096, d_out=4096, n=64, r=16,
             train=False, none=0.0),
        # a prompt batch over 8 adapters, some tokens without one
        dict(name="adapter_prompt", op="adapter", T=8192, d=4096, d_out=4096, n=8, r=16,
             train=False, none=0.1),
        # odd sizes: few tokens, odd widths, an odd rank
        dict(name="adapter_odd", op="adapter", T=333, d=776, d_out=1032, n=5, r=24, train=True,
             none=0.2),
        # fine-tuning 8 adapters at once on a packed batch
        dict(name="adapter_train", op="adapter", T=8192, d=2048, d_out=2048, n=8, r=64,
             train=True, none=0.05),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "dropout", "combine", "combine", "adapter", "adapter"])
    if op == "balance":
        T, E = _log(rng, 1, 60000), rng.choice([3, 8, 16, 40, 64, 100, 128, 256])
        S = _log(rng, 1, max(2, min(2000, T)))
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), S=S, mask=rng.random() < 0.7,
                    ragged=True)
    if op == "dropout":
        return dict(op=op, T=_log(rng, 1, 9000), width=8 * _log(rng, 1, 500),
                    dtype=rng.choice(["bf16", "f32"]), p=rng.choice([0.0, 0.05, 0.1, 0.5, 0.9]),
                    add=rng.random() < 0.7)
    if op == "combine":
        E = rng.choice([4, 8, 64])
        k = rng.randint(1, min(8, E))
        return dict(op=op, T=_log(rng, 1, 32000 // k), E=E, k=k, width=8 * _log(rng, 4, 300),
                    cf=rng.choice([0.0, 0.5, 1.0]), p=rng.choice([0.0, 0.1, 0.4]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
    train = rng.random() < 0.5
    return dict(op=op, T=_log(rng, 1, 8192), d=8 * _log(rng, 8, 250), d_out=8 * _log(rng, 8, 250),
                n=_log(rng, 1, 64), r=8 * rng.choice([1, 1, 2, 2, 3, 4, 5, 8]), train=train,
                none=rng.choice([0.0, 0.1, 0.5]))


# ------------------------------------------------------------------ inputs --

def _act(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    cpu = np.random.default_rng(seed)

    def randn(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)

    s = {"case": case}
    T = case["T"]
    if case["op"] == "balance":
        E, k, S = case["E"], case["k"], case["S"]
        logits = randn(T, E, scale=1.5)
        logits[:, : max(1, E // 16)] += 2.0          # hot experts
        s["logits"] = logits
        s["idx"] = torch.topk(logits, k, dim=1).indices.to(torch.int32)
        s["dlosses"] = torch.tensor([0.01, 0.001], device=DEV)
        s["offsets"] = s["mask"] = None
        if case["ragged"]:                            # some empty, a padded tail behind the last
            cuts = np.sort(cpu.integers(0, T + 1, size=S + 1)).astype(np.int32)
            cuts[0] = 0
            s["offsets"] = torch.from_numpy(cuts).to(DEV)
        if case["mask"]:
            s["mask"] = (torch.rand(T, generator=g, device=DEV) >= 0.1).to(torch.uint8)
        return s
    if case["op"] == "adapter":
        d, n, r, do = case["d"], case["n"], case["r"], case["d_out"]
        bf = torch.bfloat16
        s["x"] = randn(T, d, dtype=bf)
        s["base"] = randn(T, do, dtype=bf)
        s["A"] = randn(n, d, r, dtype=bf, scale=d ** -0.5)
        s["B"] = randn(n, r, do, dtype=bf, scale=r ** -0.5)
        s["scale"] = torch.rand(n, generator=g, device=DEV) + 0.5
        # requests follow one another in the batch; each has one adapter, or none
        starts = np.unique(np.concatenate([[0], cpu.integers(0, T, size=4 * n)]))
        if T <= 4 * n:
            starts = np.arange(T)                     # decoding: a request is one token
        ids = cpu.integers(0, n, size=len(starts))
        if T == n:
            ids = cpu.permutation(n)
        ids = np.where(cpu.random(len(starts)) < case["none"], -1, ids).astype(np.int32)
        row = np.repeat(ids, np.diff(np.concatenate([starts, [T]])))
        s["ids"] = torch.from_numpy(row).to(DEV)
        if case["train"]:
            s["dy"] = randn(T, do, dtype=bf)
            s["dx_add"] = randn(T, d)
        return s
    w, act = case["width"], _act(case)
    s["seed"], s["offset"], s["token_base"] = 0x1234567800000000 + seed, (7 + (seed << 33)) % 2 ** 63, 0
    if case["op"] == "dropout":
        s["x"] = randn(T, w, dtype=act)
        s["add"] = randn(T, w, dtype=act) if case["add"] else None
        return s
    E, k = case["E"], case["k"]
    score = torch.rand(T, E, generator=g, device=DEV)
    score[:, : E // 4] += 0.3
    idx = torch.topk(score, k, dim=1).indices.reshape(-1)
    order = torch.sort(idx, stable=True).indices
    counts = torch.zeros(E, dtype=torch.int64, device=DEV)
    counts.index_add_(0, idx, torch.ones_like(idx))
    first = torch.cumsum(counts, 0) - counts
    pos = torch.empty_like(idx)
    pos[order] = torch.arange(T * k, device=DEV)
    pos -= first[idx]
    cap = math.ceil(case["cf"] * T * k / E) if case["cf"] > 0 else T * k
    kept = torch.clamp(counts, max=cap)
    base = torch.cumsum(kept, 0) - kept
    dest = torch.where(pos < cap, base[idx] + pos, torch.full_like(pos, -1))
    s["dest"] = dest.reshape(T, k).to(torch.int32)
    s["gates"] = torch.softmax(randn(T, k), dim=1)
    s["y_perm"] = randn(T * k, w)
    s["residual"] = randn(T, w, dtype=act)
    s["dy"] = randn(T, w, dtype=act)
    return s


# -------------------------------------------------------------- plain form --

def _mulhilo(a, b):
    """High and low 32 bits of the product of two 32-bit values held in int64."""
    p = a * b                                         # exact modulo 2^64
    return (p >> 32) & 0xFFFFFFFF, p & 0xFFFFFFFF


def _keep(rows, width, p, seed, offset, token_base):
    """The keep mask (rows, width) of the generator described at the top."""
    nblk = width // 8
    b = torch.arange(rows * nblk, device=DEV, dtype=torch.int64) + token_base * nblk
    c0, c1 = b & 0xFFFFFFFF, b >> 32
    c2 = torch.full_like(b, offset & 0xFFFFFFFF)
    c3 = torch.full_like(b, (offset >> 32) & 0xFFFFFFFF)
    k0, k1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    for _ in range(10):                               # the generator's rounds
        h0, l0 = _mulhilo(c0, 0xD2511F53)
        h1, l1 = _mulhilo(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    words = torch.stack([c0, c1, c2, c3], dim=1)
    u16 = torch.stack([words & 0xFFFF, words >> 16], dim=2)
    return (u16 >= _threshold(p)).reshape(rows, width)


def _threshold(p):
    return math.floor(p * 65536.0 + 0.5)


def _scale(p):
    return 65536.0 / (65536.0 - _threshold(p))


def _mask(s):
    c = s["case"]
    return _keep(c["T"], c["width"], c["p"], s["seed"], s["offset"], s["token_base"])


def _plain_balance(s):
    c = s["case"]
    T, E, k, S = c["T"], c["E"], c["k"], c["S"] if c["ragged"] else 1
    logits = s["logits"]
    t = torch.arange(T, device=DEV)
    seq, valid = torch.zeros_like(t), torch.ones_like(t, dtype=torch.bool)
    if s["offsets"] is not None:
        off = s["offsets"].long()
        seq = torch.searchsorted(off[1:].contiguous(), t, right=True)
        valid = (t >= off[0]) & (t < off[-1])
    if s["mask"] is not None:
        valid = valid & (s["mask"] != 0)
    seq = torch.where(valid, seq, S)                  # row S collects what is not counted
    m = logits.amax(dim=1, keepdim=True)
    e = torch.exp(logits - m)
    z = e.sum(dim=1, keepdim=True)
    p, lse = e / z, (m + torch.log(z))[:, 0]
    counts = torch.zeros((S + 1) * E, dtype=torch.int32, device=DEV)
    slot = (seq[:, None] * E + s["idx"].long()).reshape(-1)
    counts.index_add_(0, slot, torch.ones_like(slot, dtype=torch.int32))
    counts = counts.reshape(S + 1, E)
    n = torch.zeros(S + 1, dtype=torch.int32, device=DEV)
    n.index_add_(0, seq, torch.ones_like(seq, dtype=torch.int32))
    psum = torch.zeros(S + 1, E, dtype=torch.float64, device=DEV).index_add_(0, seq, p.double())
    counts, n, psum = counts[:S], n[:S], psum[:S]
    nd = n.clamp(min=1).double()
    P, f = psum / nd[:, None], counts.double() / (nd * k)[:, None]
    live = (n > 0).sum().clamp(min=1).double()
    N = n.sum().clamp(min=1).double()
    balance = E * (f * P).sum() / live
    zloss = (torch.where(valid, lse, torch.zeros_like(lse)).double() ** 2).sum() / N
    a = (s["dlosses"][0].double() * E / (live * nd))[:, None] * f       # (S, E)
    a = torch.cat([a, torch.zeros(1, E, dtype=torch.float64, device=DEV)]).float()[seq]
    pa = (p * a).sum(dim=1, keepdim=True)
    dz = (s["dlosses"][1].double() * 2 / N).float() * lse
    dl = torch.where(valid[:, None], p * (a - pa + dz[:, None]), torch.zeros_like(p))
    tokens = torch.cat([n, n.sum().reshape(1), (n > 0).sum().reshape(1)]).to(torch.int32)
    return {"counts": counts, "prob_mean": P.float(), "tokens": tokens,
            "losses": torch.stack([balance, zloss]).float(), "dlogits": dl}


def _plain_dropout(s):
    c = s["case"]
    x = s["x"].float()
    y = torch.where(_mask(s), x * _scale(c["p"]), torch.zeros_like(x))
    if s["add"] is not None:
        y = y + s["add"].float()
    return {"out": y.to(s["x"].dtype)}


def _plain_combine(s):
    c = s["case"]
    keep, scale = _mask(s), _scale(c["p"])
    dest = s["dest"].long()
    kept = (dest >= 0)[:, :, None]
    rows = torch.where(kept, s["y_perm"][dest.clamp(min=0)], torch.zeros((), device=DEV))
    y = (rows * s["gates"][:, :, None]).sum(dim=1)
    y = torch.where(keep, y * scale, torch.zeros_like(y)) + s["residual"].float()
    dy = s["dy"].float()
    dy = torch.where(keep, dy * scale, torch.zeros_like(dy))
    dgates = (rows * dy[:, None, :]).sum(dim=2)
    dy_perm = torch.zeros_like(s["y_perm"])
    dy_perm[dest[kept[:, :, 0]]] = (s["gates"][:, :, None] * dy[:, None, :])[kept[:, :, 0]]
    return {"output": y.to(s["residual"].dtype), "dy_perm": dy_perm, "dgates": dgates}


def _plain_adapter(s):
    """Every token against every adapter's columns at once, the others' masked out."""
    c = s["case"]
    T, n, r = c["T"], c["n"], c["r"]
    d, do = c["d"], c["d_out"]
    ids = s["ids"].long()
    w = (ids[:, None] == torch.arange(n, device=DEV)) * s["scale"]       # (T, n), 0 elsewhere
    w = w.repeat_interleave(r, dim=1)
    A = s["A"].float().permute(1, 0, 2).reshape(d, n * r)
    B = s["B"].float().reshape(n * r, do)
    x = s["x"].float()
    u = (x @ A) * w
    out = {"output": (s["base"].float() + u @ B).to(torch.bfloat16)}
    if c["train"]:
        dy = s["dy"].float()
        v = (dy @ B.T) * w
        out["dx"] = s["dx_add"] + v @ A.T
        out["dA"] = (x.T @ v).reshape(d, n, r).permute(1, 0, 2).contiguous()
        out["dB"] = (u.T @ dy).reshape(n, r, do)
    return out


# ------------------------------------------------------- the library's call --

def _config(case):
    from mixture_experts_top_b200 import api
    T, k, E = case["T"], case.get("k", 1), case.get("E", 8)
    w = case.get("width", case.get("d", 8))
    f32 = case.get("dtype") == "f32"
    return api.make_config(T, w, 8, case.get("d_out", w), E, k, "linear" if f32 else "swiglu",
                           "f32" if f32 else "bf16", case.get("cf", 0.0))


def _handles(s):
    """What a program allocates once for its shapes: the configuration, workspaces, outputs."""
    from mixture_experts_top_b200 import api
    c = s["case"]
    h = {"cfg": _config(c), "api": api}
    T = c["T"]
    f32 = dict(dtype=torch.float32, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    if c["op"] == "balance":
        S, E = c["S"] if c["ragged"] else 1, c["E"]
        h["ws"] = api.alloc_balance_workspace(h["cfg"], S)
        h["out"] = {"counts": torch.empty(S, E, **i32), "prob_mean": torch.empty(S, E, **f32),
                    "tokens": torch.empty(S + 2, **i32), "losses": torch.empty(2, **f32),
                    "dlogits": torch.empty(T, E, **f32)}
    elif c["op"] == "dropout":
        h["out"] = {"out": torch.empty_like(s["x"])}
    elif c["op"] == "combine":
        h["out"] = {"output": torch.empty_like(s["residual"]),
                    "dy_perm": torch.zeros_like(s["y_perm"]),
                    "dgates": torch.empty_like(s["gates"])}
    else:
        h["plan"] = api.alloc_adapter_plan(h["cfg"], c["n"])
        h["out"] = {"output": torch.empty_like(s["base"])}
        h["u"] = None
        if c["train"]:
            h["u"] = torch.empty(T, c["r"], **f32)
            h["ws"] = api.alloc_adapter_workspace(h["cfg"], c["n"], c["r"])
            h["out"].update(dx=torch.empty(T, c["d"], **f32),
                            dA=torch.empty(c["n"], c["d"], c["r"], **f32),
                            dB=torch.empty(c["n"], c["r"], c["d_out"], **f32))
    return h


def _own(s):
    if "own" not in s:
        s["own"] = _handles(s)
    c, h = s["case"], s["own"]
    api, cfg, o = h["api"], h["cfg"], h["out"]
    if c["op"] == "balance":
        api.moe_balance_loss(cfg, s["offsets"], s["mask"], s["logits"], s["idx"], o["counts"],
                             o["prob_mean"], o["tokens"], o["losses"], h["ws"])
        api.moe_balance_loss_backward(cfg, s["offsets"], s["mask"], s["logits"], o["counts"],
                                      o["tokens"], s["dlosses"], o["dlogits"], h["ws"])
    elif c["op"] == "dropout":
        api.moe_dropout(cfg, c["p"], s["seed"], s["offset"], s["token_base"], s["x"], s["add"],
                        o["out"])
    elif c["op"] == "combine":
        draws = (c["p"], s["seed"], s["offset"], s["token_base"])
        api.moe_combine_dropout(cfg, *draws, s["y_perm"], s["dest"], s["gates"], s["residual"],
                                o["output"])
        api.moe_combine_dropout_backward(cfg, *draws, s["dy"], s["y_perm"], s["dest"], s["gates"],
                                         o["dy_perm"], o["dgates"])
    else:
        api.moe_adapter_plan(cfg, c["n"], s["ids"], h["plan"])
        api.moe_adapter(cfg, h["plan"], s["x"], s["A"], s["B"], s["scale"], s["base"],
                        o["output"], h["u"])
        if c["train"]:
            api.moe_adapter_backward(cfg, h["plan"], s["x"], h["u"], s["dy"], s["A"], s["B"],
                                     s["scale"], s["dx_add"], o["dx"], o["dA"], o["dB"], h["ws"])
    return o


def run(state):
    if own:
        return _own(state)
    return {"balance": _plain_balance, "dropout": _plain_dropout, "combine": _plain_combine,
            "adapter": _plain_adapter}[state["case"]["op"]](state)


# -------------------------------------------------------------------- work --

def work(case):
    """One pass's inputs read once and outputs written once, and its products."""
    T = case["T"]
    if case["op"] == "balance":
        E, k, S = case["E"], case["k"], case["S"]
        # the forward has to see every logit before the backward can start
        return {"bytes": T * (8 * E + 4 * k + 4 * E + 2 * case["mask"]) + 8 * S * E,
                "flops": 12 * T * E}
    if case["op"] == "dropout":
        b = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": T * case["width"] * b * (3 if case["add"] else 2),
                "flops": 2 * T * case["width"]}
    if case["op"] == "combine":
        b, k, w = 2 if case["dtype"] == "bf16" else 4, case["k"], case["width"]
        # forward: expert rows and residual in, output out; backward: the rows
        # and dy in, the rows' gradients out (capacity may drop some)
        kept = min(1.0, case["cf"]) if case["cf"] > 0 else 1.0
        return {"bytes": T * w * (3 * b + 12 * k * kept) + 16 * T * k, "flops": 6 * T * k * w}
    d, do, n, r = case["d"], case["d_out"], case["n"], case["r"]
    rows = T * (1 - case["none"])
    used = min(n, T)
    by = 2 * rows * d + 4 * T * do + 2 * used * r * (d + do) + 4 * T
    fl = 2 * rows * r * (d + do)
    if case["train"]:
        by += 2 * rows * (d + do) + 8 * T * d + 2 * used * r * (d + do) + 4 * n * r * (d + do)
        fl *= 3
    return {"bytes": by, "flops": fl}


# ------------------------------------------- the definition in 64-bit floats --

def _philox_numpy(blocks, seed, offset):
    """The generator's four words per block, in unsigned 64-bit arithmetic."""
    u, m32 = np.uint64, np.uint64(0xFFFFFFFF)
    c = [blocks & m32, blocks >> u(32), np.full_like(blocks, u(offset) & m32),
         np.full_like(blocks, (u(offset) >> u(32)) & m32)]
    key = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        a, b = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(b >> u(32)) ^ c[1] ^ u(key[0]), b & m32, (a >> u(32)) ^ c[3] ^ u(key[1]), a & m32]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    return np.stack(c, axis=1).astype(np.uint32)


def _exact_drop(s):
    """Per element 0 or 1 / (1 - p), p rounded to a multiple of 2^-16; (T, width) fp64."""
    c = s["case"]
    per_row = c["width"] // 8
    first = s["token_base"] * per_row
    words = _philox_numpy(np.arange(first, first + c["T"] * per_row, dtype=np.uint64), s["seed"],
                          s["offset"])
    halves = words.astype("<u4").view("<u2").reshape(c["T"], c["width"])
    cut = int(c["p"] * 65536 + 0.5)
    return torch.from_numpy(np.where(halves < cut, 0.0, 1.0 / (1.0 - cut / 65536.0))).to(DEV)


def exact(case, seed):
    s = prepare(case, seed)
    T = case["T"]
    if case["op"] == "dropout":
        y = s["x"].double() * _exact_drop(s)
        return {"out": y if s["add"] is None else y + s["add"].double()}
    if case["op"] == "combine":
        drop = _exact_drop(s)
        dy = s["dy"].double() * drop
        gates, out = s["gates"].double(), torch.zeros_like(drop)
        dy_perm = torch.zeros(s["y_perm"].shape, dtype=torch.float64, device=DEV)
        dgates = torch.zeros_like(gates)
        for j in range(case["k"]):
            t = torch.nonzero(s["dest"][:, j] >= 0)[:, 0]
            row = s["dest"][t, j].long()
            y = s["y_perm"][row].double()
            out[t] += gates[t, j, None] * y
            dgates[t, j] = torch.einsum("tc,tc->t", dy[t], y)
            dy_perm[row] = gates[t, j, None] * dy[t]
        return {"output": s["residual"].double() + drop * out, "dy_perm": dy_perm,
                "dgates": dgates}
    if case["op"] == "adapter":
        out = s["base"].double()
        train = case["train"]
        dA = torch.zeros(s["A"].shape, dtype=torch.float64, device=DEV)
        dB = torch.zeros(s["B"].shape, dtype=torch.float64, device=DEV)
        dx = s["dx_add"].double() if train else None
        for a in range(case["n"]):
            t = torch.nonzero(s["ids"] == a)[:, 0]
            if t.numel() == 0:
                continue
            x, A, B = s["x"][t].double(), s["A"][a].double(), s["B"][a].double()
            sc = s["scale"][a].double()
            out[t] += sc * ((x @ A) @ B)
            if train:
                dy = s["dy"][t].double()
                dx[t] += sc * (dy @ B.T) @ A.T
                dA[a] = sc * (x.T @ (dy @ B.T))
                dB[a] = sc * ((x @ A).T @ dy)
        return {"output": out, "dx": dx, "dA": dA, "dB": dB} if train else {"output": out}
    E, k, S = case["E"], case["k"], case["S"] if case["ragged"] else 1
    L = s["logits"].double()
    off = [0, T] if s["offsets"] is None else s["offsets"].tolist()
    ok = torch.ones(T, dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"].bool()
    lse = torch.logsumexp(L, 1)
    p = torch.exp(L - lse[:, None])
    members = [off[i] + torch.nonzero(ok[off[i]:off[i + 1]])[:, 0] for i in range(S)]
    sizes = [m.numel() for m in members]
    N, live = max(1, sum(sizes)), max(1, sum(1 for m in sizes if m))
    P = torch.zeros(S, E, dtype=torch.float64, device=DEV)
    dl, balance, z = torch.zeros_like(L), 0.0, 0.0
    wb, wz = (float(v) for v in s["dlosses"])
    for i, m in enumerate(members):
        if not sizes[i]:
            continue
        f = torch.bincount(s["idx"][m].reshape(-1).long(), minlength=E).double() / (sizes[i] * k)
        P[i] = p[m].mean(0)
        balance += float(E * torch.dot(f, P[i])) / live
        z += float((lse[m] ** 2).sum()) / N
        dl[m] = wb * E / (live * sizes[i]) * p[m] * (f - (p[m] @ f)[:, None])
        dl[m] += wz * 2 / N * lse[m, None] * p[m]
    return {"counts": None, "prob_mean": P, "tokens": None,
            "losses": torch.tensor([balance, z], dtype=torch.float64), "dlogits": dl}
