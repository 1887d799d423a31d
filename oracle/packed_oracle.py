"""Plain NumPy fp64 oracle of the packed-batch operators: the balance loss per
sequence, the counter-based dropout, the low-rank adapters, and their
gradients.  Nothing here is shared with the CUDA side."""
from __future__ import annotations

import numpy as np


# ------------------------------------------------------------ balance loss --

def counted_tokens(T, offsets, mask):
    """Per sequence, the indices of its counted tokens."""
    offsets = [0, T] if offsets is None else [int(v) for v in offsets]
    ok = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    return [lo + np.flatnonzero(ok[lo:hi]) for lo, hi in zip(offsets[:-1], offsets[1:])]


def balance_loss(logits, idx, E, offsets=None, mask=None):
    """counts (S, E), prob_mean (S, E), tokens (S+2), balance, z."""
    L = np.asarray(logits, np.float64)
    T, k = idx.shape
    seqs = counted_tokens(T, offsets, mask)
    S = len(seqs)
    counts = np.zeros((S, E), np.int64)
    P = np.zeros((S, E))
    N, live, total, z = 0, 0, 0.0, 0.0
    for s, members in enumerate(seqs):
        n = len(members)
        if n == 0:
            continue
        N, live = N + n, live + 1
        rows = L[members]
        m = rows.max(axis=1, keepdims=True)
        ex = np.exp(rows - m)
        P[s] = (ex / ex.sum(axis=1, keepdims=True)).mean(axis=0)
        z += float(((m[:, 0] + np.log(ex.sum(axis=1))) ** 2).sum())
        counts[s] = np.bincount(idx[members].reshape(-1), minlength=E)
        total += E * float((counts[s] / (n * k)) @ P[s])
    tokens = np.array([len(m) for m in seqs] + [N, live], np.int64)
    return dict(counts=counts, prob_mean=P, tokens=tokens, balance=total / live if live else 0.0,
                z=z / N if N else 0.0)


def balance_loss_backward(logits, idx, E, offsets, mask, dbalance, dz):
    """dlogits (T, E), 0 for tokens not counted."""
    L = np.asarray(logits, np.float64)
    T, k = idx.shape
    seqs = counted_tokens(T, offsets, mask)
    N, live = sum(map(len, seqs)), sum(1 for m in seqs if len(m))
    out = np.zeros((T, E))
    for members in seqs:
        n = len(members)
        if n == 0:
            continue
        rows = L[members]
        m = rows.max(axis=1, keepdims=True)
        ex = np.exp(rows - m)
        p = ex / ex.sum(axis=1, keepdims=True)
        lse = m + np.log(ex.sum(axis=1, keepdims=True))
        a = dbalance * E / (live * n) * np.bincount(idx[members].reshape(-1), minlength=E) / (n * k)
        out[members] = p * (a - (p @ a)[:, None] + dz * 2.0 * lse / N)
    return out


# ----------------------------------------------------------------- dropout --

def philox4x32(counter, key, rounds=10):
    """Philox4x32 of one 4-word counter under a 2-word key, in Python ints."""
    c = [int(v) & 0xFFFFFFFF for v in counter]
    k = [int(v) & 0xFFFFFFFF for v in key]
    for _ in range(rounds):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def threshold(p):
    return int(np.floor(p * 65536.0 + 0.5))


def keep_mask(rows, width, p, seed, offset, token_base=0):
    """(rows, width) bool."""
    nblk = width // 8
    cut = threshold(p)
    b = np.arange(rows * nblk, dtype=np.uint64) + np.uint64(token_base * nblk)
    lo = np.uint64(0xFFFFFFFF)
    c = [b & lo, b >> np.uint64(32), np.full_like(b, offset & 0xFFFFFFFF),
         np.full_like(b, (offset >> 32) & 0xFFFFFFFF)]
    k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        x, y = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(y >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), y & lo,
             (x >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), x & lo]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    halves = np.stack([h for w in c for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))], axis=1)
    return (halves >= np.uint64(cut)).reshape(rows, width)


def dropout(x, p, seed, offset, token_base=0, add=None):
    """add + keep * x / (1 - p) with p in steps of 2^-16; fp64."""
    x = np.asarray(x, np.float64)
    keep = keep_mask(x.shape[0], x.shape[1], p, seed, offset, token_base)
    y = np.where(keep, x * (65536.0 / (65536.0 - threshold(p))), 0.0)
    return y if add is None else y + np.asarray(add, np.float64)


# ---------------------------------------------------------------- adapters --

def adapter(x, A, B, scale, ids, base=None):
    """output (T, d_out) and u (T, r), fp64."""
    x, A, B = (np.asarray(v, np.float64) for v in (x, A, B))
    out = np.zeros((x.shape[0], B.shape[2])) if base is None else np.array(base, np.float64)
    u = np.zeros((x.shape[0], A.shape[2]))
    for a in range(A.shape[0]):
        t = np.flatnonzero(ids == a)
        u[t] = float(scale[a]) * (x[t] @ A[a])
        out[t] += u[t] @ B[a]
    return out, u


def adapter_backward(x, A, B, scale, ids, dy, dx_add=None):
    x, A, B, dy = (np.asarray(v, np.float64) for v in (x, A, B, dy))
    dx = np.zeros_like(x) if dx_add is None else np.array(dx_add, np.float64)
    dA, dB = np.zeros_like(A), np.zeros_like(B)
    for a in range(A.shape[0]):
        t = np.flatnonzero(ids == a)
        v = float(scale[a]) * (dy[t] @ B[a].T)
        dx[t] += v @ A[a].T
        dA[a] = x[t].T @ v
        dB[a] = float(scale[a]) * (x[t] @ A[a]).T @ dy[t]
    return dx, dA, dB
