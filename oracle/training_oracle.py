"""CPU oracle for the training operators beside the layer: the balance and z losses with their
gradient, the gradient norm and the AdamW step with states in 32 or 8 bits.

TEST INFRASTRUCTURE ONLY, like the layer's oracle: NumPy in float64, plain and slow, one
sequence, tensor or block at a time, sharing no code with the HIP library.

The balance loss is the auxiliary loss of "Sparse Mixture-of-Experts" (bigdataschool.ru wiki,
section "Маршрутизация токена и auxiliary loss") taken sequence by sequence; for one sequence
it is ``aux_load_balancing_loss``.
"""
from __future__ import annotations

import numpy as np

__all__ = ["balance_loss", "grad_norm", "adamw_step", "held_m", "held_v", "read_m", "read_v", "ADAMW_BLOCK"]

ADAMW_BLOCK = 256


def balance_loss(logits, ids, num_experts, alpha, z_coeff, mask=None, seq_offsets=None, dloss=(1.0, 1.0)):
    """Counts, counted tokens, mean probabilities, the two losses and their gradient on the
    logits (weighted by dloss).  A counted token without a finite logit has no probabilities."""
    l = np.asarray(logits, dtype=np.float64)
    ids = np.asarray(ids)
    T, E, k = l.shape[0], num_experts, ids.shape[1]
    off = [0, T] if seq_offsets is None else [int(o) for o in seq_offsets]
    S = len(off) - 1
    counts, tokens = np.zeros((S, E), dtype=np.int64), np.zeros(S, dtype=np.int64)
    probs, grad = np.zeros((S, E)), np.zeros((T, E))
    rows = [[t for t in range(off[s], off[s + 1]) if mask is None or mask[t]] for s in range(S)]
    tokens[:] = [len(r) for r in rows]
    live, total = int((tokens > 0).sum()), int(tokens.sum())
    balance = z2 = 0.0
    for s in range(S):
        if not rows[s]:
            continue
        n = len(rows[s])
        for t in rows[s]:
            for e in ids[t]:
                if 0 <= e < E:
                    counts[s, e] += 1
        f = counts[s] / (k * n)
        for t in rows[s]:
            if np.all(l[t] == -np.inf):
                continue
            top = l[t].max()
            e = np.exp(l[t] - top)
            p, z = e / e.sum(), top + np.log(e.sum())
            probs[s] += p / n
            z2 += z * z
            grad[t] = p * (dloss[0] * alpha * E / (live * n) * (f - (f * p).sum())
                           + dloss[1] * 2 * z_coeff / total * z)
        balance += float((f * probs[s]).sum())
    losses = np.array([alpha * E * balance / max(live, 1), z_coeff * z2 / max(total, 1)])
    return {"counts": counts, "seq_tokens": tokens, "mean_probs": probs, "losses": losses, "dlogits": grad}


def grad_norm(grads, max_norm):
    """The norm over every tensor and the factor that clips it (NaN if the norm is not finite)."""
    norm = float(np.sqrt(sum(float((np.asarray(g, dtype=np.float64) ** 2).sum()) for g in grads)))
    return norm, (min(1.0, max_norm / (norm + 1e-6)) if np.isfinite(norm) else float("nan"))


def adamw_step(w, g, m, v, t, lr, beta1, beta2, eps, weight_decay, scale=1.0):
    """New (w, m, v) in float64."""
    w, g, m, v = (np.asarray(a, dtype=np.float64) for a in (w, g, m, v))
    g = g * scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * (g * g)
    u = (m / (1 - beta1 ** t)) / (np.sqrt(v) / np.sqrt(1 - beta2 ** t) + eps)
    return w * (1 - lr * weight_decay) - lr * u, m, v


def _blocks(n):
    return [(b, min(n, b + ADAMW_BLOCK)) for b in range(0, n, ADAMW_BLOCK)]


def _held(x, top, root):
    """Codes and float32 block scales: the code c >= 0 of the level scale (c / top)^(2 root) whose
    root-th root is nearest to the value's, found by trying every level."""
    x = np.asarray(x, dtype=np.float64).ravel()
    codes, scales = np.zeros(x.size, dtype=np.int64), np.zeros(len(_blocks(x.size)), dtype=np.float32)
    levels = (np.arange(top + 1) / top) ** 2
    for i, (a, b) in enumerate(_blocks(x.size)):
        scale = np.float32(np.abs(x[a:b]).max())
        if not np.isfinite(scale):
            scales[i] = np.nan
            continue
        if scale < np.finfo(np.float32).tiny:
            continue
        scales[i] = scale
        share = (np.abs(x[a:b]) / np.float64(scale)) ** (1.0 / root)
        codes[a:b] = np.abs(share[:, None] - levels[None, :]).argmin(axis=1)
        if root == 2:
            codes[a:b] = np.where(x[a:b] > 0, np.maximum(codes[a:b], 1), codes[a:b])
    return np.where(x < 0, -codes, codes), scales


def held_m(m):
    return _held(m, 127, 1)


def held_v(v):
    return _held(v, 255, 2)


def read_m(codes, scales):
    c = np.asarray(codes, dtype=np.float64).ravel()
    return c * np.abs(c) * np.repeat(np.asarray(scales, dtype=np.float64) * (1.0 / 127.0 ** 2), ADAMW_BLOCK)[:c.size]


def read_v(codes, scales):
    c = np.asarray(codes, dtype=np.float64).ravel()
    return (c * c) * (c * c) * np.repeat(np.asarray(scales, dtype=np.float64) * (1.0 / 255.0 ** 4), ADAMW_BLOCK)[:c.size]
