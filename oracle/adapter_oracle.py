"""Oracle of the group-limited router and of the INT4 products with low-rank
adapters: the definitions in float64 torch (on any device), with bounds on how
far a kernel that sums in fp32 may be off.  Test infrastructure only."""
from __future__ import annotations

import numpy as np
import torch

from oracle import layer_oracle as LO

HALF_BF16 = 2.0 ** -8       # half a bf16 step, relative
HALF_FP32 = 2.0 ** -24


def route_grouped(logits: np.ndarray, topk: int, groups: int, keep: int, scoring: str, bias=None,
                  renormalize: bool = True, scale: float = 1.0):
    """As layer_oracle.route on the experts of each row's `keep` best groups."""
    T, E = logits.shape
    size = E // groups
    l = np.minimum(logits, float(np.finfo(np.float32).max))
    live = ~np.isnan(logits) & (logits != -np.inf)
    key = l.copy()
    if scoring == "sigmoid":
        with np.errstate(over="ignore", invalid="ignore"):
            key = 1.0 / (1.0 + np.exp(-l))
        if bias is not None:
            b = np.asarray(bias, np.float64)
            live &= ~np.isnan(b)[None] & (b != -np.inf)[None]
            key = np.minimum(key + b, np.finfo(np.float64).max)
    limited = np.array(logits, np.float64)
    for t in range(T):
        score = []
        for g in range(groups):
            own = sorted((key[t, e] for e in range(g * size, (g + 1) * size) if live[t, e]), reverse=True)
            with np.errstate(over="ignore"):
                score.append(-np.inf if not own else own[0] if scoring == "softmax" or len(own) == 1 else own[0] + own[1])
        order = sorted(range(groups), key=lambda g: (-score[g], g))
        for g in order[keep:]:
            limited[t, g * size:(g + 1) * size] = -np.inf
    ids, w, tol = LO.route(limited, topk, scoring, bias, renormalize, scale)
    if scoring == "softmax" and not renormalize:
        # the sum is over every live expert, of the groups left out as well
        for t in range(T):
            n = int((ids[t] >= 0).sum())
            if n:
                top = l[t, live[t]].max()
                total = np.exp(l[t, live[t]] - top).sum()
                w[t, :n] = scale * np.exp(l[t, ids[t, :n]] - top) / total
                spread = np.minimum(np.abs(l[t, live[t]] - top), 104.0).max()
                tol[t, :n] = np.abs(w[t, :n]) * (2 * (spread + 4) + 2) * HALF_FP32 + abs(scale) * 2.0 ** -126
    return ids, w, tol


def int4_values(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """codes uint8 [.., N, K], scales bf16 [.., N, K/32] -> the weights they stand for, float64."""
    v = (codes.double() - 8.0) * scales.double().repeat_interleave(32, dim=-1)
    return v.to(torch.bfloat16).double()


def product(x: torch.Tensor, w: torch.Tensor, a=None, b=None, scale: float = 1.0, slices: int = 1):
    """Rows x bf16 [M, K] of one adapter: w float64 [N, K], a bf16 [slices r, K],
    b bf16 [N, r] (None: no adapter) -> y float64 [M, N] and a bound of what
    fp32 sums leave before the output's rounding.

    Products of bf16 numbers are exact in fp32.  A sum over K adds at most K / 8
    rounded terms (two half steps where a step truncates), and as many more for
    its partial sums of at most 64 waves or slices; h = scale A x is such a sum,
    rounded twice more; its two bf16 parts stand for it within 2^-16 (half a
    step of half a step)."""
    x = x.double()
    N, K = w.shape
    y = x @ w.t()
    steps = (K / 8 + 64) * 2 * HALF_FP32
    err = steps * (x.abs() @ w.abs().t())
    if a is None:
        return y, err
    a, b = a.double(), b.double()
    r = b.shape[1]
    h = scale * (x @ a.t())
    he = (steps + 4 * HALF_FP32) * abs(scale) * (x.abs() @ a.abs().t()) + HALF_BF16 ** 2 * h.abs()
    for s in range(slices):
        cols = slice(s * N // slices, (s + 1) * N // slices)
        part = slice(s * r, (s + 1) * r)
        y[:, cols] += h[:, part] @ b[cols].t()
        size = h[:, part].abs() @ b[cols].abs().t()
        err[:, cols] += he[:, part] @ b[cols].abs().t() + (r / 8 + 8) * 2 * HALF_FP32 * size
    err += steps * y.abs()
    return y, err


def linear(x, w, ids, adapters, slices: int = 1, silu: bool = False):
    """x bf16 [M, K], w float64 [N, K], ids [M] of adapters (a [L, slices r, K],
    b [L, N, r], scale [L] or None) -> y float64 and the bound of the bf16 output."""
    M = x.shape[0]
    y = torch.zeros(M, w.shape[0], dtype=torch.float64, device=x.device)
    err = torch.zeros_like(y)
    L = 0 if adapters is None else adapters[1].shape[0]
    ids = torch.full((M,), -1, device=x.device) if L == 0 else torch.where((ids >= 0) & (ids < L), ids, -1)
    for l in torch.unique(ids).tolist():
        rows = (ids == l).nonzero().squeeze(1)
        if l < 0:
            y[rows], err[rows] = product(x[rows], w)
        else:
            a, b, s = adapters
            y[rows], err[rows] = product(x[rows], w, a[l], b[l], 1.0 if s is None else float(s[l]), slices)
    return activate(y, err) if silu else (y, err + HALF_BF16 * y.abs() + 2.0 ** -133)


def activate(y, err):
    """silu(g) * u of the halves, each off by err, and the bound of its bf16 value."""
    (g, u), (eg, eu) = y.chunk(2, dim=1), err.chunk(2, dim=1)
    sg = g * torch.sigmoid(g)
    out = sg * u
    # |silu'| <= 1.1; its value within 8 + 2 |g| half units (the exponent's own rounding grows with |g|)
    bound = 1.1 * eg * (u.abs() + eu) + sg.abs() * eu + (8 + 2 * g.abs()) * HALF_FP32 * out.abs()
    return out, bound + HALF_BF16 * out.abs() + 2.0 ** -120


def assert_within(got: torch.Tensor, ref: torch.Tensor, bound: torch.Tensor, what: str = "") -> float:
    """bf16 values against float64 ones; returns the largest share of the bound."""
    share = (got.double() - ref).abs() / bound
    bad = ~(share <= 1.0)
    if bool(bad.any()):
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of bound; first at {i}: got {float(got[i])}, "
                             f"ref {float(ref[i])}, bound {float(bound[i])}")
    return float(share.max()) if share.numel() else 0.0
