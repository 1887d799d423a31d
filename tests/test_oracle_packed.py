"""Pins of the packed-batch oracle: closed forms, the whole-batch loss, the
generator's published test vectors, and central finite differences."""
import numpy as np
import pytest

from oracle import moe_oracle as O
from oracle import packed_oracle as Q


def _routing(T, E, k, seed):
    rng = np.random.default_rng(seed)
    L = rng.standard_normal((T, E))
    return rng, L, O.top_k(L.astype(np.float32), k)


def test_one_sequence_is_the_whole_batch_loss():
    _, L, idx = _routing(37, 6, 2, 0)
    r = Q.balance_loss(L, idx, 6)
    d = O.dispatch(idx, 6, 0.0)
    aux = O.aux_loss(d["f"].astype(np.float64), O.softmax_rows(L).mean(axis=0))
    assert abs(r["balance"] - aux) <= 1e-6 * aux
    assert np.array_equal(r["counts"][0], d["counts"])
    assert list(r["tokens"]) == [37, 37, 1]


def test_uniform_logits_give_one_and_log_e_squared():
    idx = np.tile(np.arange(2), (10, 1))
    r = Q.balance_loss(np.zeros((10, 4)), idx, 4, [0, 3, 3, 10])
    assert abs(r["balance"] - 1.0) < 1e-14 and abs(r["z"] - np.log(4.0) ** 2) < 1e-14
    assert list(r["tokens"]) == [3, 0, 7, 10, 2]


def test_uncounted_tokens_do_not_matter():
    _, L, idx = _routing(20, 5, 2, 1)
    mask = np.ones(20, np.uint8)
    mask[[2, 9, 10]] = 0
    off = [1, 8, 8, 15]
    r = Q.balance_loss(L, idx, 5, off, mask)
    L2 = L.copy()
    L2[[0, 2, 9, 10, 15, 16, 17, 18, 19]] = np.nan
    q = Q.balance_loss(L2, idx, 5, off, mask)
    assert r["balance"] == q["balance"] and r["z"] == q["z"]
    assert list(r["tokens"]) == [6, 0, 5, 11, 2]
    g = Q.balance_loss_backward(L2, idx, 5, off, mask, 1.0, 1.0)
    assert np.isfinite(g).all() and (g[[0, 2, 9, 10, 15, 19]] == 0).all()


@pytest.mark.parametrize("off", [None, [0, 4, 4, 5, 11]])
def test_balance_gradient_matches_differences(off):
    _, L, idx = _routing(12, 5, 2, 2)
    mask = np.ones(12, np.uint8)
    mask[3] = 0
    g = Q.balance_loss_backward(L, idx, 5, off, mask, 0.7, 0.3)
    h = 1e-6
    for t in range(12):
        for e in range(5):
            v = []
            for s in (h, -h):
                M = L.copy()
                M[t, e] += s
                r = Q.balance_loss(M, idx, 5, off, mask)   # the choice is held fixed
                v.append(0.7 * r["balance"] + 0.3 * r["z"])
            assert abs((v[0] - v[1]) / (2 * h) - g[t, e]) < 1e-8


def test_generator_published_vectors():
    """Known answers of Philox4x32-10 (Salmon et al., the authors' test vectors)."""
    f = 0xFFFFFFFF
    assert Q.philox4x32([0] * 4, [0] * 2) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    assert Q.philox4x32([f] * 4, [f] * 2) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]
    assert Q.philox4x32([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344],
                        [0xa4093822, 0x299f31d0]) == [0xd16cfe09, 0x94fdcceb, 0x5001e420,
                                                      0x24126ea1]


def test_mask_is_the_scalar_generator_and_shards():
    p, seed, offset, base = 0.37, 0x1122334455667788, (5 << 33) + 3, 3
    m = Q.keep_mask(4, 24, p, seed, offset, base)
    for t in range(4):
        for c in range(24):
            b = (base + t) * 3 + c // 8
            w = Q.philox4x32([b, b >> 32, offset, offset >> 32], [seed, seed >> 32])[c % 8 // 2]
            assert m[t, c] == (((w >> 16) if c % 2 else (w & 0xFFFF)) >= Q.threshold(p))
    whole = Q.keep_mask(7, 24, p, seed, offset)
    assert np.array_equal(whole[3:], m)


def test_mask_fraction_and_extremes():
    m = Q.keep_mask(500, 400, 0.25, 1, 2)
    # 200000 draws: standard deviation 0.00097
    assert abs(m.mean() - 0.75) < 0.005
    assert Q.keep_mask(3, 8, 0.0, 1, 2).all()
    x = np.arange(24.0).reshape(3, 8)
    assert np.array_equal(Q.dropout(x, 0.0, 1, 2), x)


def test_adapter_gradient_matches_differences():
    rng = np.random.default_rng(3)
    T, d, r, do, n = 6, 5, 3, 4, 3
    x, A = rng.standard_normal((T, d)), rng.standard_normal((n, d, r))
    B, scale = rng.standard_normal((n, r, do)), rng.random(n) + 0.5
    base, dy = rng.standard_normal((T, do)), rng.standard_normal((T, do))
    ids = np.array([0, -1, 2, 0, 0, -1])
    dx, dA, dB = Q.adapter_backward(x, A, B, scale, ids, dy)
    assert (dA[1] == 0).all() and (dB[1] == 0).all() and (dx[1] == 0).all()
    h = 1e-6
    args = dict(x=x, A=A, B=B)
    for name, grad in dict(x=dx, A=dA, B=dB).items():
        for i in np.ndindex(args[name].shape):
            v = []
            for s in (h, -h):
                a = {k: q.copy() for k, q in args.items()}
                a[name][i] += s
                v.append((Q.adapter(a["x"], a["A"], a["B"], scale, ids, base)[0] * dy).sum())
            assert abs((v[0] - v[1]) / (2 * h) - grad[i]) < 1e-7
