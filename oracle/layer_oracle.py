"""CPU oracle of the router, the few-token layer and the grouped MXFP4
products: the definitions in float64, with bounds on how far a kernel that
sums in fp32 may be off.  Test infrastructure only."""
from __future__ import annotations

import numpy as np

from oracle.moe_oracle import bf16_to_f64, f64_to_bf16

HALF_BF16 = 2.0 ** -8       # half a bf16 step, relative
HALF_FP32 = 2.0 ** -24


def route(logits: np.ndarray, topk: int, scoring: str, bias=None, renormalize: bool = True, scale: float = 1.0):
    """logits float64 [T, E] -> ids int32 [T, topk], weights float64, and a
    bound on the fp32 error of each weight.  -inf and NaN mask an expert, +inf
    is the largest finite fp32."""
    T, E = logits.shape
    l = np.minimum(logits, float(np.finfo(np.float32).max))
    live = ~np.isnan(logits) & (logits != -np.inf)
    with np.errstate(over="ignore", invalid="ignore"):
        sig = 1.0 / (1.0 + np.exp(-l))
    key = l.copy()
    if scoring == "sigmoid" and bias is not None:
        b = np.asarray(bias, np.float64)
        live &= ~np.isnan(b)[None] & (b != -np.inf)[None]
        key = np.minimum(sig + b, np.finfo(np.float64).max)
    ids = np.full((T, topk), -1, np.int32)
    w = np.zeros((T, topk))
    tol = np.zeros((T, topk))
    for t in range(T):
        order = sorted(np.nonzero(live[t])[0], key=lambda e: (-key[t, e], e))
        pick = np.array(order[:topk], np.int64)
        n = len(pick)
        if n == 0:
            continue
        ids[t, :n] = pick
        if scoring == "softmax":
            top = l[t, pick[0]]
            ex = np.exp(l[t, live[t]] - top)
            v = np.exp(l[t, pick] - top)
            v = v / (v.sum() if renormalize else ex.sum())
            # the difference from the maximum is rounded to fp32, then exp within one unit, in weight and sum
            spread = np.abs(l[t, live[t]] - top)
            rel = 2 * (np.minimum(spread, 104.0).max() + 4) * HALF_FP32
        else:
            v = sig[t, pick]
            rel = 10 * HALF_FP32
            if renormalize:
                v = v / (v.sum() + 1e-20)
                rel *= 2
        w[t, :n] = v * scale
        tol[t, :n] = np.abs(w[t, :n]) * (rel + 2 * HALF_FP32) + abs(scale) * 2.0 ** -126
    return ids, w, tol


def few_tokens(x_bits, w1, w2, topk_ids, topk_weights, first: int):
    """x bf16 bits [T, H]; w1 float64 [E, 2I, H] (gate rows, then up rows),
    w2 float64 [E, H, I] -> y float64 [T, H] and a bound per element.

    The bound: a kernel rounds each h once to bf16 (at most half a step of
    it), after gate and up sums in fp32.  Each h is off by at most c_i, its
    roundings are independent, so the weighted sum over i is off by more than
    7 sqrt(sum (w W2 c)^2) with probability below 2 exp(-49 / 2) (Hoeffding);
    the output is rounded once more."""
    T, H = x_bits.shape
    I = w2.shape[2]
    x = bf16_to_f64(x_bits)
    y = np.zeros((T, H))
    var = np.zeros((T, H))
    sums = np.zeros((T, H))
    for t in range(T):
        for j, e in enumerate(np.asarray(topk_ids)[t]):
            if not first <= e < first + len(w1):
                continue
            W1, W2 = w1[e - first], w2[e - first]
            gu = W1 @ x[t]
            dg = (H / 8) * 2 * HALF_FP32 * (np.abs(W1) @ np.abs(x[t]))    # a rounding for every 8 terms at most
            g, u = gu[:I], gu[I:]
            with np.errstate(over="ignore"):
                h = g / (1.0 + np.exp(-g)) * u
            c = HALF_BF16 * np.abs(h) + 1.1 * np.abs(u) * dg[:I] + np.abs(g) * dg[I:] + 8 * HALF_FP32 * np.abs(h)
            wt = float(topk_weights[t, j])
            y[t] += wt * (W2 @ h)
            # one expert listed twice: the same roundings, so the deviations add
            twice = int((np.asarray(topk_ids)[t] == e).sum())
            var[t] += twice * wt * wt * ((W2 * W2) @ (c * c))
            sums[t] += abs(wt) * (np.abs(W2) @ np.abs(h))
    tol = 7 * np.sqrt(var) + HALF_BF16 * np.abs(y) + (I / 8) * 2 * HALF_FP32 * sums
    return y, tol


def product(a: np.ndarray, w: np.ndarray):
    """a float64 [M, K] . w float64 [N, K]^T -> values and a bound: exact
    products, an fp32 rounding for every 16 terms at most (two half steps
    where it truncates), one rounding to bf16."""
    y = a @ w.T
    K = a.shape[1]
    return y, HALF_BF16 * np.abs(y) + (K / 16) * 2 * HALF_FP32 * (np.abs(a) @ np.abs(w).T)


def assert_within(got_bits: np.ndarray, ref: np.ndarray, tol: np.ndarray, what: str = "") -> float:
    """bf16 bits against float64 values; returns the largest share of the bound."""
    got = bf16_to_f64(got_bits)
    err = np.abs(got - ref)
    bad = ~(err <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} out of bound; first at {i}: got {got[i]}, "
                             f"ref {ref[i]}, bound {tol[i]}")
    return float((err / np.maximum(tol, 1e-300)).max()) if err.size else 0.0


__all__ = ["route", "few_tokens", "product", "assert_within", "f64_to_bf16"]
