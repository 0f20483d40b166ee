"""The two ends of a compressed training step in fp64: softmax cross entropy from
hidden states and output weights, and the orthogonalised optimiser step.  Plain
numpy, straight from the definitions, one token and one matrix at a time."""
from __future__ import annotations

import numpy as np

COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def cross_entropy(x, w, targets, bias=None, weights=None, scale=1.0, mean=False, ignore_index=-100):
    """(loss, lse, dx, dw, dbias) of scale * sum_t weights_t loss_t, divided by the
    number of tokens that count for mean."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    tokens, vocab = x.shape[0], w.shape[0]
    counts = [int(y) >= 0 and int(y) != ignore_index for y in targets]
    s = scale / max(1, sum(counts)) if mean else scale
    loss, lse = np.zeros(tokens), np.zeros(tokens)
    dx, dw, db = np.zeros_like(x), np.zeros_like(w), np.zeros(vocab)
    for t in range(tokens):
        with np.errstate(invalid="ignore"):
            l = w @ x[t] + (0.0 if bias is None else np.asarray(bias, np.float64))
            top = l.max()
            lse[t] = top + np.log(np.exp(l - top).sum())
        if not counts[t]:
            continue
        y = int(targets[t])
        loss[t] = lse[t] - l[y] if y < vocab else np.nan
        if y >= vocab:
            continue
        g = np.exp(l - lse[t])
        g[y] -= 1.0
        g *= s * (1.0 if weights is None else float(weights[t]))
        dx[t] = g @ w
        dw += np.outer(g, x[t])
        db += g
    return loss, lse, dx, dw, db


def newton_schulz(u, steps=5, coefficients=COEFFICIENTS, eps=1e-7):
    a, b, c = coefficients
    x = np.asarray(u, np.float64)
    x = x / (np.sqrt((x * x).sum()) + eps)
    tall = x.shape[0] > x.shape[1]
    for _ in range(steps):
        g = x.T @ x if tall else x @ x.T
        p = b * g + c * (g @ g)
        x = a * x + (x @ p if tall else p @ x)
    return x


def muon_step(param, grad, momentum, lr, mu, nesterov, weight_decay, lr_scale, **kw):
    """(new param, new momentum); momentum None: none."""
    g = np.asarray(grad, np.float64)
    m = None if momentum is None else mu * np.asarray(momentum, np.float64) + g
    u = g if m is None else g + mu * m if nesterov else m
    return (1.0 - lr * weight_decay) * np.asarray(param, np.float64) - lr * lr_scale * newton_schulz(u, **kw), m


def fp16_pieces(x, power):
    """x as the sum of `hi` and `lo`, fp16 values times 2^-power."""
    s = 2.0 ** power
    hi = (np.asarray(x, np.float64) * s).astype(np.float16).astype(np.float64)
    lo = (np.asarray(x, np.float64) * s - hi).astype(np.float16).astype(np.float64)
    return hi / s, lo / s


def newton_schulz_rounded(u, pieces, steps=5, coefficients=COEFFICIENTS, eps=1e-7):
    """The steps with X, A and B rounded as the library documents: X as two fp16
    pieces, of which the products take the upper one (pieces = 1) or both; A and
    B as one or two.  Everything else exact: what these roundings alone do."""
    a, b, c = coefficients
    take = (lambda v: fp16_pieces(v, 14)[0]) if pieces == 1 else (lambda v: sum(fp16_pieces(v, 14)))
    x = np.asarray(u, np.float64)
    x = sum(fp16_pieces(x / (np.sqrt((x * x).sum()) + eps), 14))
    tall = x.shape[0] > x.shape[1]
    for s in range(steps):
        h = take(x)
        g = take(h.T @ h if tall else h @ h.T)
        p = take(b * g + c * (g @ g))
        x = a * x + (h @ p if tall else p @ h)
        if s + 1 < steps:
            x = sum(fp16_pieces(x, 14))
    return x
