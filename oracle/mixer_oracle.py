"""CPU float64 oracle of the operators around the layer (plain numpy loops over
the formulas of include/ittt.h), with running bounds of what fp32 arithmetic
may add to each value.

Every function returns (value, bound) pairs: ``bound`` is the largest distance
an fp32 computation of that value may have from it by its number of roundings,
before the one rounding of the store.
"""

from __future__ import annotations

import math
from typing import Optional, Tuple

import numpy as np

U = 2.0 ** -24  # half a step of fp32 at 1


def _erf(x: np.ndarray) -> np.ndarray:
    return np.vectorize(math.erf, otypes=[np.float64])(x)


def sigmoid(x: np.ndarray) -> np.ndarray:
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def activate(x: np.ndarray, act: str) -> np.ndarray:
    if act == "none":
        return x
    if act == "relu":
        return np.where(x < 0, 0.0, x)
    if act == "silu":
        return x * sigmoid(x)
    if act == "gelu":
        return 0.5 * x * (1.0 + _erf(x / math.sqrt(2.0)))
    if act == "gelu_tanh":
        return 0.5 * x * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3)))
    raise ValueError(act)


def _after_act(y, bound, act):
    """Every activation has a slope below 1.2; its own evaluation in fp32 costs
    up to 16 roundings of its argument's size (tanh and erf of a rounded
    argument, a product with the sum 1 + tanh, which cancels below zero)."""
    out = activate(y, act)
    return out, (bound if act == "none" else 1.2 * bound + 16 * U * (np.abs(y) + np.abs(out)))


def linear(X, W, bias=None, residual=None, act: str = "none") -> Tuple[np.ndarray, np.ndarray]:
    X, W = np.asarray(X, np.float64), np.asarray(W, np.float64)
    K = X.shape[1]
    y = X @ W.T
    # K products and sums; the tensor cores may truncate where CUDA cores round (2 U each)
    bound = 2 * (K + 2) * U * (np.abs(X) @ np.abs(W).T)
    if bias is not None:
        y = y + bias
        bound = bound + U * np.abs(y)
    y, bound = _after_act(y, bound, act)
    if residual is not None:
        y = y + residual
        bound = bound + U * np.abs(y)
    return y, bound


def causal_conv(X, w, bias=None, act: str = "none", state=None, lengths=None, base=None):
    """(Y, bound, state_out); rows behind a sequence's end are those of ``base``."""
    X, w = np.asarray(X, np.float64), np.asarray(w, np.float64)
    B, T, d = X.shape
    k = w.shape[1]
    Y = np.zeros_like(X) if base is None else np.array(base, np.float64)
    bound = np.zeros_like(X)
    last = np.zeros((B, k - 1, d))
    for b in range(B):
        n = T if lengths is None else int(min(max(lengths[b], 0), T))
        rows = np.zeros((k - 1 + n, d))
        if state is not None:
            rows[:k - 1] = state[b]
        rows[k - 1:] = X[b, :n]
        for t in range(n):
            win = rows[t:t + k]                                  # [k, d]
            y = (win * w.T).sum(0)
            e = (k + 2) * U * np.abs(win * w.T).sum(0)
            if bias is not None:
                y = y + bias
                e = e + (k + 2) * U * (np.abs(np.asarray(bias)) + np.abs(y))
            Y[b, t], bound[b, t] = _after_act(y, e, act)
        last[b] = rows[n:]
    return Y, bound, last


def softplus(x: np.ndarray) -> np.ndarray:
    return np.maximum(x, 0.0) + np.log1p(np.exp(-np.abs(x)))


def selective_scan(U_, delta, A, Bm, Cm, D=None, Z=None, dt_bias=None, dt_softplus=False, state=None,
                   lengths=None, base=None):
    """(Y, Y's bound, h, h's bound), token after token.

    A step multiplies h by exp(s A).  In fp32 the exponent x = s A carries a few
    relative roundings (the softplus, the products, the sums of steps when
    several tokens are joined: 32 in all cover them), so the factor is off by
    32 |x| U plus the exponential's own error and the roundings of the
    multiply-add and of the new term: 16 U.  The bound E follows the recurrence
    of the absolute values H: E = a E + (16 + 32 |x|) U H.
    """
    f8 = np.float64
    U_, delta, A = np.asarray(U_, f8), np.asarray(delta, f8), np.asarray(A, f8)
    Bm, Cm = np.asarray(Bm, f8), np.asarray(Cm, f8)
    B, T, d = U_.shape
    N = A.shape[1]
    if Bm.ndim == 3:
        Bm, Cm = Bm[:, :, None], Cm[:, :, None]
    rep = d // Bm.shape[2]
    Y = np.zeros((B, T, d)) if base is None else np.array(base, f8)
    Yb = np.zeros((B, T, d))
    h = np.zeros((B, d, N)) if state is None else np.array(state, f8)
    E = np.zeros((B, d, N))
    H = np.abs(h)
    for b in range(B):
        n = T if lengths is None else int(min(max(lengths[b], 0), T))
        for t in range(n):
            s = delta[b, t] + (0.0 if dt_bias is None else dt_bias)
            ds = U * np.abs(s)
            if dt_softplus:
                s = softplus(s)
            u = U_[b, t]
            x = s[:, None] * A
            a = np.exp(x)
            Bt, Ct = np.repeat(Bm[b, t], rep, axis=0), np.repeat(Cm[b, t], rep, axis=0)
            term = (s * u)[:, None] * Bt
            h[b] = a * h[b] + term
            Hn = a * H[b] + np.abs(term)
            # the step size's own rounding before a softplus is absolute (its slope is below 1)
            E[b] = a * E[b] + (16 + 32 * np.abs(x)) * U * Hn + ds[:, None] * (
                np.abs(A) * a * H[b] + np.abs(u[:, None] * Bt))
            H[b] = Hn
            y = (h[b] * Ct).sum(1)
            e = ((E[b] + (N + 4) * U * H[b]) * np.abs(Ct)).sum(1)
            if D is not None:
                y = y + D * u
                e = e + 2 * U * (np.abs(D * u) + np.abs(y))
            if Z is not None:
                z = np.asarray(Z[b, t], f8)
                g = z * sigmoid(z)
                y, e = y * g, e * np.abs(g) + 16 * U * np.abs(y) * (np.abs(g) + np.abs(z))
            Y[b, t], Yb[b, t] = y, e
    return Y, Yb, h, E
