"""Float64 oracle of the scored router, its balance loss and gradients, and of the expert FFN
with an 8-bit activation checkpoint (numpy, by the formulas of include/moe.h).  Test
infrastructure: the library never loads it."""
from __future__ import annotations

import numpy as np

SIGMOID, SOFTMAX = 0, 1


def scores(x, score):
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore"):
        if score == SIGMOID:
            return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))),
                            np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))
    e = np.exp(x - x.max(axis=1, keepdims=True))
    return e / e.sum(axis=1, keepdims=True)


def _first(key, k):
    """Places of the k largest, the lower place first among equals."""
    return np.argsort(-key, axis=-1, kind="stable")[..., :k]


def keys(x, b, score):
    """f32(score) + b in float32 (b None: the rounded score)."""
    s = scores(x, score).astype(np.float32)
    return s if b is None else s + np.asarray(b, np.float32)


def select(key, K, n_groups=1, topk_groups=1, group_top=1):
    """Selected experts [T, K] of float32 keys [T, N]."""
    T, N = key.shape
    key = key.astype(np.float32)
    if topk_groups < n_groups:
        by = key.reshape(T, n_groups, N // n_groups)
        top = -np.sort(-by, axis=2)[:, :, :group_top]
        gscore = top[:, :, 0] if group_top == 1 else top[:, :, 0] + top[:, :, 1]
        kept = np.zeros((T, n_groups), bool)
        np.put_along_axis(kept, _first(gscore, topk_groups), True, axis=1)
        key = np.where(kept[:, :, None], by, -np.inf).reshape(T, N)
    return _first(key, K).astype(np.int32)


def gates(x, idx, score, renorm, scale):
    s = np.take_along_axis(scores(x, score), idx.astype(np.int64), axis=1)
    if renorm:
        # relative to the largest selected score (log domain: nothing underflows)
        xs = np.take_along_axis(np.asarray(x, np.float64), idx.astype(np.int64), axis=1)
        lg = xs if score == SOFTMAX else np.minimum(xs, 0) - np.log1p(np.exp(-np.abs(xs)))
        w = np.exp(lg - lg.max(axis=1, keepdims=True))
        return scale * w / w.sum(axis=1, keepdims=True)
    return scale * s


def balance(x, idx, offsets, alpha, score):
    """(loss [n_seq], coef [n_seq, N]) of sequences [offsets[q], offsets[q+1])."""
    T, N = x.shape
    K = idx.shape[1]
    s = scores(x, score)
    s = s / s.sum(axis=1, keepdims=True)
    loss, coef = [], []
    for a, b in zip(offsets[:-1], offsets[1:]):
        n = b - a
        if n <= 0:
            loss.append(0.0)
            coef.append(np.zeros(N))
            continue
        ids = idx[a:b].reshape(-1)
        ids = ids[(ids >= 0) & (ids < N)]
        f = N / (K * n) * np.bincount(ids, minlength=N)
        coef.append(alpha * f / n)
        loss.append(alpha * (f * s[a:b].mean(axis=0)).sum())
    return np.array(loss), np.array(coef)


def backward(x, idx, d_gate, offsets, coef, d_loss, score, renorm, scale):
    """d_logit [T, N] by the chain rule, slot by slot (ids outside [0, N) left out)."""
    T, N = x.shape
    s = scores(x, score)
    ds = np.zeros((T, N))                      # gradient of the scores
    if d_gate is not None:
        ok = (idx >= 0) & (idx < N)
        at = np.where(ok, idx, 0).astype(np.int64)
        c = np.where(ok, np.take_along_axis(s, at, axis=1), 0.0)
        dg = np.where(ok, np.asarray(d_gate, np.float64), 0.0) * scale
        if renorm:
            tot = c.sum(axis=1, keepdims=True)
            tot = np.where(tot > 0, tot, 1.0)
            dc = (dg - (dg * c).sum(axis=1, keepdims=True) / tot) / tot
        else:
            dc = dg
        for k in range(idx.shape[1]):
            np.add.at(ds, (np.arange(T), at[:, k]), np.where(ok[:, k], dc[:, k], 0.0))
    if coef is not None:
        tot = s.sum(axis=1, keepdims=True)
        for q, (a, b) in enumerate(zip(offsets[:-1], offsets[1:])):
            g = coef[q] * (1.0 if d_loss is None else d_loss[q])
            sn = s[a:b] / tot[a:b]
            ds[a:b] += (g - (sn * g).sum(axis=1, keepdims=True)) / tot[a:b]
    if score == SIGMOID:
        return ds * s * (1 - s)
    return s * (ds - (ds * s).sum(axis=1, keepdims=True))


def e4m3(v):
    """Nearest E4M3 value (ties to even, saturated at 448) of float values."""
    v = np.asarray(v, np.float64)
    m = np.minimum(np.abs(v), 448.0)
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.where(m > 0, m, 1.0)))
    step = 2.0 ** (np.maximum(e, -6) - 3)
    return np.sign(v) * np.minimum(np.rint(m / step) * step, 448.0)


def checkpoint(a):
    """(values, scales) of pre-activations [rows, 2I] kept as E4M3 per row and 128 columns."""
    t = np.asarray(a, np.float32).reshape(a.shape[0], -1, 128)
    top = np.abs(t).max(axis=2)
    sc = np.where(top == 0, np.float32(1), top / np.float32(448)).astype(np.float32)
    return e4m3((t / sc[:, :, None]).astype(np.float32)).reshape(a.shape), sc


def from_checkpoint(q, sc):
    return (np.asarray(q, np.float64).reshape(q.shape[0], -1, 128)
            * np.asarray(sc, np.float64)[:, :, None]).reshape(q.shape)


def ffn_backward(x, Wgu, Wdn, a, dy):
    """(dx, dWgu, dWdn) of one expert from pre-activations a [rows, 2I]."""
    I = a.shape[1] // 2
    g, up = a[:, :I], a[:, I:]
    sig = scores(g, SIGMOID)
    dh = dy @ Wdn
    dA = np.concatenate([dh * up * sig * (1 + g * (1 - sig)), dh * g * sig], axis=1)
    return dA @ Wgu, dA.T @ x, dy.T @ (g * sig * up)
