"""Plain float64 references of the decoder-layer operators around the products.

TEST INFRASTRUCTURE ONLY, as oracle.core.  Definitions:

* gated block: C = act(g) * u with g = A . Wg + bg, u = A . Wu + bu, and its gradients
  dU = dC act(g), dG = dC u act'(g), dA = dG . Wg^T + dU . Wu^T, dW = d^T . A,
  db = column sums;
* append: the pairs (a, b) of a head turn to (a c - b s, b c + a s);
* attention: softmax over the prefix and the own tokens j <= len - n + i of query i.

The error bounds next to them state what each rounding of the library can do (half-ulp
2**-11 of an fp16 value; fp32 sums and elementary functions at 2**-20 of the sum of
magnitudes); independent roundings of the terms of a long sum are taken at six times the
root of their sum of squares.
"""
from __future__ import annotations

import numpy as np

U16 = 2.0**-11      # half an ulp of fp16, relative
TINY16 = 2.0**-25   # half the smallest fp16 subnormal
F32 = 2.0**-20      # fp32 sums and functions, relative to the sum of magnitudes
GELU_C = np.sqrt(2.0 / np.pi)


def activation(x, act):
    """act(x) and act'(x) in float64."""
    x = np.asarray(x, dtype=np.float64)
    if act == "silu":
        s = 0.5 * (1 + np.tanh(0.5 * x))
        return x * s, s * (1 + x * (1 - s))
    t = np.tanh(GELU_C * (x + 0.044715 * x**3))
    return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * GELU_C * (1 + 3 * 0.044715 * x * x)


def gated_ref(A, Wg, Wu, act, bg=None, bu=None, rs=None, csg=None, csu=None):
    """(C, g, u) for weights [K, N] in float64."""
    A = np.asarray(A, dtype=np.float64)
    g, u = A @ Wg, A @ Wu
    if rs is not None:
        rs = np.asarray(rs, dtype=np.float64)[:, None]
        g, u = g * rs * np.asarray(csg, dtype=np.float64), u * rs * np.asarray(csu, dtype=np.float64)
    if bg is not None:
        g = g + np.asarray(bg, dtype=np.float64)
    if bu is not None:
        u = u + np.asarray(bu, dtype=np.float64)
    return activation(g, act)[0] * u, g, u


def sum_bound(A, W, rounded):
    """Error of the library's A . W: fp32 sums; with `rounded`, weights rounded to fp16 first."""
    A = np.abs(np.asarray(A, dtype=np.float64))
    e = F32 * (A @ np.abs(W))
    return e + 6 * U16 * np.sqrt(A**2 @ W**2) if rounded else e


def gated_bound(C, g, u, eg, eu, act):
    """Error of C from errors eg, eu of the pre-activations (|act'| < 1.2) and its own rounding."""
    h = np.abs(activation(g, act)[0])
    return 1.2 * eg * (np.abs(u) + eu) + h * eu + (U16 + F32) * np.abs(C) + TINY16


def gated_grads_ref(A, Wg, Wu, g, u, dC, act):
    """{dA, dw_gate, dw_up ([N, K]), dbias_gate, dbias_up, dG, dU} in float64."""
    A, dC = np.asarray(A, dtype=np.float64), np.asarray(dC, dtype=np.float64)
    h, dh = activation(g, act)
    dG, dU = dC * u * dh, dC * h
    return {"dA": dG @ Wg.T + dU @ Wu.T, "dw_gate": dG.T @ A, "dw_up": dU.T @ A, "dbias_gate": dG.sum(0),
            "dbias_up": dU.sum(0), "dG": dG, "dU": dU}


def gated_grads_bound(A, Wg, Wu, g, u, dC, act, eg, eu, rounded):
    """Error bounds of the same outputs: pre-activations kept in fp16, their gradients and
    (rounded) weights as fp16 operands (|act'| < 1.2, |act''| < 1.2)."""
    A, dC = np.abs(np.asarray(A, dtype=np.float64)), np.abs(np.asarray(dC, dtype=np.float64))
    r = gated_grads_ref(A * 0, Wg, Wu, g, u, dC, act)
    dg = eg + U16 * np.abs(g) + TINY16
    du = eu + U16 * np.abs(u) + TINY16
    dG, dU = np.abs(r["dG"]), np.abs(r["dU"])
    eG = dC * (1.2 * dg * (np.abs(u) + du) + 1.2 * du) + (U16 + F32) * dG + TINY16
    eU = dC * 1.2 * dg + (U16 + F32) * dU + TINY16

    def total(ex, x, w):  # sums over the shared axis of x . w, with errors ex of x
        e = 6 * np.sqrt(ex**2 @ w**2) + F32 * (x @ np.abs(w))
        return e + 6 * U16 * np.sqrt(x**2 @ w**2) if rounded else e

    out = {"dA": total(eG, dG, Wg.T) + total(eU, dU, Wu.T)}
    rounded = False
    out["dw_gate"], out["dw_up"] = total(eG.T, dG.T, A), total(eU.T, dU.T, A)
    ones = np.ones((A.shape[0], 1))
    out["dbias_gate"], out["dbias_up"] = total(eG.T, dG.T, ones)[:, 0], total(eU.T, dU.T, ones)[:, 0]
    return out


def rotate_ref(x, cos, sin, interleaved):
    """x [T, H, D] with its first 2 * cos.shape[1] places turned, and the error bound of the library's result."""
    x = np.asarray(x, dtype=np.float64)
    c, s = np.asarray(cos, dtype=np.float64)[:, None], np.asarray(sin, dtype=np.float64)[:, None]
    half = c.shape[-1]
    ia, ib = (np.arange(half) * 2, np.arange(half) * 2 + 1) if interleaved else (np.arange(half), np.arange(half) + half)
    y, e = x.copy(), np.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    e[..., ia] = e[..., ib] = 2.0**-22 * (np.abs(a) + np.abs(b)) + TINY16
    e += U16 * np.abs(y) * (e > 0)
    return y, e


def attention_ref(q, k, v, visible, scale):
    """One head: q [n, D], k and v [L, D], visible [n, L] -> (out, lse, bound of out), float64.

    The bound: probabilities rounded to fp16 (relative 2**-11, absolute 2**-25 where the
    largest is at least 1), scores to fp32 sums, the output's own rounding.
    """
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    n = q.shape[0]
    s = np.where(visible, (q @ k.T) * scale, -np.inf) if k.shape[0] else np.full((n, 0), -np.inf)
    m = s.max(1, initial=-np.inf)
    p = np.exp(s - np.where(np.isfinite(m), m, 0)[:, None])
    p = np.where(visible, p, 0.0)
    total = p.sum(1)
    live = total > 0
    safe = np.where(live, total, 1)[:, None]
    out = np.where(live[:, None], p @ v / safe, 0.0)
    lse = np.where(live, np.where(live, m, 0) + np.log(safe[:, 0]), -np.inf)
    es = F32 * scale * (np.abs(q) @ np.abs(k.T)).max(1, initial=0)[:, None] + 2.0**-18
    weighted = p @ np.abs(v) / safe
    vmax = np.abs(v).max(initial=0)
    bound = (U16 + 2 * es) * (weighted + np.abs(out)) + visible.sum(1)[:, None] * TINY16 * vmax / safe + U16 * np.abs(out) + TINY16
    return out, lse, bound
