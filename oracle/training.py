"""float64 oracle of the training operators: load-balance loss and gradient, the 8-bit checkpoint
format, the routing's slot gradients and the router's linear backward.  Plain numpy loops over the
definitions; shares no code with the CUDA library."""
from __future__ import annotations

import math

import numpy as np

BLOCK = 32


def softmax(x):
    x = np.asarray(x, np.float64)
    p = np.zeros_like(x)
    for t, row in enumerate(x):
        m = row.max() if row.size else 0.0
        if m == -np.inf:
            continue                      # no expert is open: no probability
        e = np.exp(row - m)
        p[t] = e / e.sum()
    return p


def groups(T, cu=None, valid=None):
    """The token lists of the loss's groups."""
    ok = np.ones(T, bool) if valid is None else np.asarray(valid) != 0
    cu = [0, T] if cu is None else [int(c) for c in cu]
    return [[t for t in range(a, b) if ok[t]] for a, b in zip(cu[:-1], cu[1:])]


def balance(logits, topk, E, K, cu=None, valid=None):
    gs = groups(len(logits), cu, valid)
    prob, counts = np.zeros((len(gs), E)), np.zeros((len(gs), E), np.int64)
    tokens = np.array([len(g) for g in gs])
    terms = []
    for i, g in enumerate(gs):
        if not g:
            continue
        prob[i] = softmax(logits[g]).sum(0) / len(g)
        for e in np.asarray(topk)[g].reshape(-1):
            if 0 <= e < E:
                counts[i, e] += 1
        terms.append((counts[i] * E / (K * len(g)) * prob[i]).sum())
    return dict(loss=float(np.mean(terms)) if terms else 0.0, prob=prob, counts=counts, tokens=tokens)


def balance_grad(logits, topk, E, K, scale, cu=None, valid=None, counts=None):
    """dL/dlogits with the counts held fixed (the caller's, or those of the inputs)."""
    gs = groups(len(logits), cu, valid)
    b = balance(logits, topk, E, K, cu, valid)
    counts = b["counts"] if counts is None else np.asarray(counts)
    active = sum(1 for g in gs if g)
    d = np.zeros((len(logits), E))
    for i, g in enumerate(gs):
        if not g:
            continue
        f = counts[i] * E / (K * len(g))
        p = softmax(logits[g])
        d[g] = scale / (active * len(g)) * p * (f - (p @ f)[:, None])
    return d


def encode(x):
    """(q, scale byte) of float rows, block by block."""
    x = np.asarray(x, np.float64)
    N, D = x.shape
    nb = -(-D // BLOCK)
    q, byte = np.zeros((N, nb * BLOCK), np.int8), np.zeros((N, nb), np.uint8)
    for r in range(N):
        for b in range(nb):
            v = x[r, b * BLOCK:(b + 1) * BLOCK]
            if not np.isfinite(v).all():
                byte[r, b] = 255
                continue
            a = np.abs(v).max()
            k = -120
            if a > 0:
                k = max(k, math.frexp(a)[1] - 8)
                while a > 127 * 2.0 ** k:
                    k += 1
            lim = 63 if k == 122 else 127
            byte[r, b] = k + 127
            q[r, b * BLOCK:b * BLOCK + v.size] = np.clip(np.rint(v / 2.0 ** k), -lim, lim)
    return q, byte


def decode(q, byte, D):
    step = np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))
    return (q.astype(np.float64) * np.repeat(step, BLOCK, 1))[:, :D]


def route_grad(y, gate, mlogit, dy, reg_scale, S=1):
    """Slot gradients: y [T][K][D] expert outputs."""
    T, K = gate.shape
    s = np.einsum("tkd,td->tk", y, dy)
    dr, dl = np.zeros((T, K)), np.zeros((T, K))
    reg = reg_scale / (T * K) if T else 0.0
    for t in range(0, T, S):
        run = s[t:t + S].sum(0)
        g, l = gate[t], mlogit[t]
        dg = np.where(l >= 0, run, 0.0)
        sig = 1 / (1 + np.exp(-l))
        dr[t] = g * (dg - (g * dg).sum())
        dl[t] = (run * g + len(s[t:t + S]) * reg) * sig * (1 - sig)
    return s, dr, dl
