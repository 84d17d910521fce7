"""GPU parity of the group-limited router and of the INT4 products with
low-rank adapters (one shared weight; the routed experts') against their
definitions in float64."""
import os
import re
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from gpu_util import bits, dev, log  # noqa: E402

from oracle import adapter_oracle as AO  # noqa: E402

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU visible")]

import w4a16_int4_mixture_moe_amd as M  # noqa: E402


# ------------------------------------------------------------------ router

def _check_route(logits, k, groups, keep, scoring, bias=None, renorm=True, scale=1.0, what=""):
    ids, w = M.moe_route_grouped(logits, k, groups, keep, scoring=scoring, bias=bias, renormalize=renorm, scale=scale)
    ref_ids, ref_w, tol = AO.route_grouped(logits.double().cpu().numpy(), k, groups, keep, scoring,
                                           None if bias is None else bias.double().cpu().numpy(), renorm, scale)
    np.testing.assert_array_equal(ids.cpu().numpy(), ref_ids, err_msg=what)
    err = np.abs(w.double().cpu().numpy() - ref_w)
    assert (err <= tol).all(), (what, float((err / np.maximum(tol, 1e-300)).max()))
    return ids, w


KINDS = [("softmax", False, True), ("softmax", False, False), ("sigmoid", False, True), ("sigmoid", True, True),
         ("sigmoid", True, False)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,E,groups,keep,k", [
    (1, 1, 1, 1, 1), (3, 6, 3, 1, 2), (5, 64, 64, 3, 3), (4, 64, 8, 2, 9), (9, 160, 8, 3, 6), (17, 256, 8, 4, 8),
    (33, 384, 8, 4, 8), (6, 896, 14, 5, 16), (7, 1024, 64, 7, 32), (5, 1023, 33, 2, 20), (8, 130, 65 // 5, 13, 7),
    (11, 1000, 2, 1, 32)])
def test_route_grouped_shapes(T, E, groups, keep, k, dtype):
    g = torch.Generator().manual_seed(T * 131 + E)
    l = torch.randn(T, E, generator=g).to(dtype).to(dev())
    b = (0.1 * torch.randn(E, generator=g)).to(dev())
    for scoring, biased, renorm in KINDS:
        _check_route(l, k, groups, keep, scoring, b if biased else None, renorm, 2.5, f"{scoring} {biased} {renorm}")


@pytest.mark.parametrize("E,groups,keep,k", [(384, 8, 4, 8), (500, 10, 3, 10), (96, 16, 2, 3), (128, 32, 5, 8),
                                             (700, 7, 2, 8)])
def test_route_grouped_many_tokens(E, groups, keep, k):
    """Enough tokens for the 16-lane form, where it is built (at most 512 experts in 16 groups)."""
    g = torch.Generator().manual_seed(E + k)
    T = 6147
    l = torch.randn(T, E, generator=g)
    l[torch.rand(T, E, generator=g) < 0.05] = float("-inf")
    l[3] = float("nan")
    l[4] = float("-inf")
    l[4, E - 1] = float("inf")
    l[6146] = 0.0
    b = (0.1 * torch.randn(E, generator=g)).to(dev())
    pick = torch.cat([torch.arange(40), torch.arange(3000, 3040), torch.arange(T - 40, T)])
    wide = torch.full((T, E + 7), float("inf"), device=dev())       # what lies between the rows is never chosen
    wide[:, 4:4 + E] = l.to(dev())
    for scoring, biased, renorm in KINDS:
        kw = dict(scoring=scoring, bias=b if biased else None, renormalize=renorm, scale=1.5)
        ids, w = M.moe_route_grouped(wide[:, 4:4 + E], k, groups, keep, **kw)
        ref = AO.route_grouped(l[pick].double().numpy(), k, groups, keep, scoring,
                               b.double().cpu().numpy() if biased else None, renorm, 1.5)
        np.testing.assert_array_equal(ids.cpu().numpy()[pick], ref[0])
        assert (np.abs(w.double().cpu().numpy()[pick] - ref[1]) <= ref[2]).all()
        # every row of the long batch as in a short one, which takes 64 lanes a token
        for t in (0, 2048, 5000):
            i2, w2 = M.moe_route_grouped(wide[t:t + 64, 4:4 + E], k, groups, keep, **kw)
            assert torch.equal(ids[t:t + 64], i2)
            torch.testing.assert_close(w[t:t + 64], w2, rtol=1e-5, atol=0)


@pytest.mark.parametrize("scoring,biased", [("softmax", False), ("sigmoid", False), ("sigmoid", True)])
def test_route_grouped_masks_infinities_and_ties(scoring, biased):
    n, inf, big = float("nan"), float("inf"), 3e38
    E, groups, keep, k = 72, 9, 2, 5
    rows = torch.zeros(11, E)
    rows[0] = -inf                                        # nothing left
    rows[1] = n
    rows[2] = -inf
    rows[2, 69] = -3.0                                    # one live expert in a group
    rows[2, 1] = 1.0
    rows[2, 2] = -30.0
    rows[3, 5] = inf
    rows[3, 66] = inf
    rows[3, 7] = n
    rows[4] = -0.0
    rows[4, 3] = 0.0                                      # equal to -0
    rows[5] = -200.0                                      # scores below fp32's range
    rows[6, ::2] = -big
    rows[7, 68] = big
    rows[8] = torch.arange(E) % 3                         # every group alike
    rows[9, 8:] = -inf                                    # one group
    rows[10, :64] = n                                     # the last one
    b = None
    if biased:
        b = torch.zeros(E)
        b[0], b[1], b[2], b[9], b[17], b[33], b[34] = -inf, n, inf, 2.0, inf, -1e30, 1e30
        b = b.to(dev())
    for renorm in (True, False):
        _check_route(rows.to(dev()), k, groups, keep, scoring, b, renorm, 1.0, f"{scoring} {renorm}")


def test_route_grouped_orders_near_ties_in_64_bits():
    """Group scores that 32 bits cannot order: sums equal to about 2^-30, hidden under large biases that cancel."""
    g = torch.Generator().manual_seed(11)
    E, groups, size = 384, 8, 48
    l = torch.randn(40, E, generator=g)
    b = (0.5 - torch.sigmoid(l[0].double())).float()
    l[20:] = l[0]
    l[20:30] += 1e-6 * torch.randn(10, E, generator=g)
    _check_route(l.to(dev()), 8, groups, 4, "sigmoid", b.to(dev()), True, 1.0, "near ties")
    _check_route(torch.zeros(5, E, device=dev()), 8, groups, 3, "sigmoid", None, True, 1.0, "all equal")
    c = torch.full((E,), -500.0)                          # two experts of each group, +1000 and -1000 but for the score
    for j in range(groups):
        c[j * size + 5], c[j * size + 11] = 1000.0, -400.0
    l = torch.zeros(6, E)
    l[:, 5::size] = 1e-6 * torch.randn(6, groups, generator=g)
    _check_route(l.to(dev()), 8, groups, 4, "sigmoid", c.to(dev()), True, 1.0, "cancelling biases")
    same = torch.full((3, E), 20.0)                       # saturated scores: equal in 32 bits, not in 64
    same[:, ::7] = 21.0
    same[1, 100:] = 20.5
    _check_route(same.to(dev()), 8, groups, 2, "sigmoid", None, True, 1.0, "saturated")


@pytest.mark.parametrize("T", [5, 6151])
@pytest.mark.parametrize("E,groups,keep,k,stride,lanes", [(384, 8, 4, 8, 16, 1), (512, 16, 9, 10, 16, 3),
                                                          (1024, 32, 20, 32, 64, 31)])
def test_route_grouped_crowded_residues(T, E, groups, keep, k, stride, lanes):
    """Far more than k experts above any bound by residue, many of them equal: the list's overflow."""
    g = torch.Generator().manual_seed(T + E + k)
    l = 0.1 * torch.randn(T, E, generator=g)
    l[:, torch.arange(E) % stride < lanes] += 3.0
    l[1::3] = l[1::3].round(decimals=1)
    l[2] = 0.0
    b = (0.05 * torch.randn(E, generator=g)).to(dev())
    rows = slice(None) if T < 100 else slice(0, 60)
    d = l.to(dev())
    for scoring, bias in (("softmax", None), ("sigmoid", b), ("sigmoid", None)):
        ids, _ = M.moe_route_grouped(d, k, groups, keep, scoring=scoring, bias=bias)
        ref = AO.route_grouped(l[rows].double().numpy(), k, groups, keep, scoring,
                               None if bias is None else bias.double().cpu().numpy())
        np.testing.assert_array_equal(ids[rows].cpu().numpy(), ref[0])


def test_route_grouped_of_every_group_is_the_plain_router():
    g = torch.Generator().manual_seed(1)
    for T in (7, 6500):
        l = torch.randn(T, 384, generator=g).to(dev())
        b = (0.1 * torch.randn(384, generator=g)).to(dev())
        for kw in (dict(scoring="sigmoid", bias=b), dict(scoring="softmax", renormalize=False)):
            for groups, keep in ((1, 1), (8, 8)):
                a, c = M.moe_route_grouped(l, 8, groups, keep, **kw), M.moe_route(l, 8, **kw)
                assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])


# ----------------------------------------------------- one shared projection

class Shared:
    """Seeded weight, adapters and rows of one projection."""

    def __init__(self, T, K, N, La, r, slices=1, gate_up=False, seed=0, scaled=True, ids=None):
        g = torch.Generator(device=dev()).manual_seed(seed + 31 * T + K + N + r)
        self.x = torch.randn(T, K, generator=g, device=dev()).to(torch.bfloat16)
        codes = torch.randint(0, 16, (1, N, K), generator=g, device=dev(), dtype=torch.uint8)
        sc = (0.005 + 0.015 * torch.rand(1, N, K // 32, generator=g, device=dev())).to(torch.bfloat16)
        self.p = M.pack_w4(codes, sc, gate_up=gate_up)
        self.w = AO.int4_values(codes[0], sc[0])
        self.a = (torch.randn(La, slices * r, K, generator=g, device=dev()) / K ** 0.5).to(torch.bfloat16)
        self.b = torch.randn(La, N, r, generator=g, device=dev()).to(torch.bfloat16)
        self.s = 0.5 + torch.rand(La, generator=g, device=dev()) if scaled else None
        self.ids = torch.randint(-1, La, (T,), generator=g, device=dev(), dtype=torch.int32) if ids is None else ids
        self.slices = slices

    def ad(self):
        return M.adapters(self.a, self.b, self.s)

    def run(self, silu=False, **kw):
        return M.w4a16_linear(self.x, self.p, self.ad(), self.ids, silu=silu, **kw)

    def check(self, silu=False, what=""):
        y = self.run(silu)
        ref, bound = AO.linear(self.x, self.w, self.ids, (self.a, self.b, self.s), self.slices, silu)
        return AO.assert_within(y, ref, bound, what)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 33, 48, 64, 65, 127, 129, 300])
@pytest.mark.parametrize("K,N,r,slices", [(256, 64, 16, 1), (1120, 1040, 8, 1), (32, 32, 24, 2), (2016, 96, 40, 2)])
def test_linear_shapes(T, K, N, r, slices):
    worst = Shared(T, K, N, 5, r, slices).check(what=f"T {T} K {K} N {N} r {r}")
    if N % 32 == 0:
        worst = max(worst, Shared(T, K, N, 5, r, slices, gate_up=True).check(silu=True, what="silu"))
        Shared(T, K, N, 5, r, slices, gate_up=True, scaled=False).check(what="gate/up packed, plain store")
    log("share of the bound", T, K, N, r, slices, round(worst, 3))


@pytest.mark.parametrize("K,N,T,La", [(7168, 4096, 64, 32), (7168, 512, 1, 16), (2048, 7168, 301, 64), (1152, 2048, 700, 3)])
def test_linear_at_real_widths(K, N, T, La):
    P = Shared(T, K, N, La, 16, 2, gate_up=True)
    P.check(silu=True)
    P.check()


@pytest.mark.parametrize("T,K,N,r", [(4100, 128, 4096, 16), (2050, 384, 4096, 8), (1100, 160, 4096, 64),
                                     (4097, 288, 2080, 8)])
@pytest.mark.parametrize("runs", [1, 12, 0])
def test_linear_prefill_tiles(T, K, N, r, runs):
    """The 256-, 128- and 64-row tiles: long runs of an adapter, and every row another one."""
    ids = None
    if runs:
        g = torch.Generator().manual_seed(runs)
        ids = torch.randint(-1, 5, (runs,), generator=g).repeat_interleave(-(-T // runs))[:T].to(torch.int32).to(dev())
    P = Shared(T, K, N, 5, r, 2, gate_up=True, ids=ids)
    P.check(silu=True, what="silu")
    P.check(what="store")


def test_linear_more_rows_than_one_order():
    """Above 16384 rows the rows keep their places."""
    T = 16500
    for ids in (None, torch.arange(T, device=dev()).div(5000, rounding_mode="floor").to(torch.int32)):
        Shared(T, 128, 512, 4, 8, ids=ids).check()


@pytest.mark.parametrize("rank", [8, 16, 32, 72, 128, 256])
@pytest.mark.parametrize("T", [3, 70])
def test_linear_ranks(T, rank):
    Shared(T, 640, 160, 3, rank, 2).check()
    Shared(T, 640, 160, 3, rank, 1).check()


@pytest.mark.parametrize("T,K,N,rank,slices", [(2100, 256, 512, 128, 2), (1100, 384, 1024, 72, 1), (8200, 128, 64, 24, 1),
                                                 (2300, 160, 256, 104, 2), (17000, 128, 64, 16, 2)])
@pytest.mark.parametrize("runs", [7, 0])
def test_linear_many_rows(T, K, N, rank, slices, runs):
    """Inner values packed once, A in parts of 128 rows, the staged first half; K that it does not take; no order of
    the rows."""
    ids = None
    if runs:
        ids = torch.arange(T, device=dev()).mul(runs).div(T, rounding_mode="floor").to(torch.int32) - 1
    P = Shared(T, K, N, 6, rank, slices, ids=ids)
    P.check()
    assert torch.equal(bits_t(P.run()), bits_t(P.run()))


# whole tiles over a packed h: at least 512 rows and four planes (K of 1024 with A's rows in four waves, 4096 in one)
PACKED = [(520, 1120, 2560, 128, 2), (700, 1024, 2080, 72, 2), (1100, 1056, 4096, 256, 1), (2100, 1024, 1024, 72, 2),
          (600, 4096, 2560, 8, 2), (17000, 1024, 64, 40, 2)]


@pytest.mark.parametrize("T,K,N,rank,slices", PACKED)
@pytest.mark.parametrize("runs", [7, 0])
def test_linear_packed_inner_values(T, K, N, rank, slices, runs):
    ids = None
    if runs:
        ids = torch.arange(T, device=dev()).mul(runs).div(T, rounding_mode="floor").to(torch.int32) - 1
    P = Shared(T, K, N, 6, rank, slices, gate_up=slices == 2, ids=ids)
    P.check()
    if slices == 2:
        P.check(silu=True, what="silu")


def test_linear_packed_rows_do_not_see_other_requests():
    P = Shared(700, 1024, 2080, 6, 72, 2)
    y = P.run()
    P.a[2].fill_(float("nan"))
    P.b[4].fill_(float("inf"))
    z = P.run()
    rest = (P.ids != 2) & (P.ids != 4)
    assert torch.equal(bits_t(y)[rest], bits_t(z)[rest])
    assert z[P.ids == 2].isnan().all()


@pytest.mark.parametrize("T", [1, 17, 64, 65])
@pytest.mark.parametrize("K,rank,slices", [(3232, 64, 2), (6400, 32, 2), (3328, 256, 1)])
def test_linear_long_rows_of_a(T, K, rank, slices):
    """Few rows and wide adapters: eight planes of inner values."""
    Shared(T, K, 96, 5, rank, slices).check()


@pytest.mark.parametrize("T", [5, 40, 400])
def test_linear_one_slice_for_gate_and_up(T):
    P = Shared(T, 384, 160, 4, 16, 1, gate_up=True)
    P.check(silu=True)
    P.check()


@pytest.mark.parametrize("T,La", [(64, 1024), (300, 1024), (16, 64), (64, 64), (640, 1)])
def test_linear_adapter_counts(T, La):
    Shared(T, 256, 128, La, 8).check()
    ids = torch.randperm(max(T, La), device=dev())[:T].to(torch.int32)      # every row another adapter, some past the last
    Shared(T, 256, 128, La, 8, ids=ids).check()


def test_linear_ids_outside_the_table_are_no_adapter():
    T = 40
    ids = torch.tensor([-1, -7, 2**31 - 1, -2**31, 5, 4, 0, 1000] * 5, dtype=torch.int32, device=dev())
    P = Shared(T, 256, 128, 5, 16, ids=ids)
    P.check()
    y, bare = P.run(), M.w4a16_linear(P.x, P.p)
    none = (ids < 0) | (ids >= 5)
    assert torch.equal(bits_t(y)[none], bits_t(bare)[none])
    AO.assert_within(bare, *AO.linear(P.x, P.w, ids, None))
    P.ids = torch.full((T,), -1, dtype=torch.int32, device=dev())
    assert torch.equal(bits_t(P.run()), bits_t(bare))


def bits_t(t):
    return t.view(torch.int16)


@pytest.mark.parametrize("T", [9, 30, 64, 300])
def test_linear_rows_do_not_see_other_requests(T):
    """An adapter of infinities and NaN, and rows of them, reach their own rows only; a row's bits do not depend on
    where it stands."""
    P = Shared(T, 512, 256, 6, 16, 2, gate_up=True)
    clean = P.run(silu=True)
    perm = torch.randperm(T, device=dev())
    kept = P.x, P.ids
    P.x, P.ids = P.x[perm].contiguous(), P.ids[perm].contiguous()
    assert torch.equal(bits_t(P.run(silu=True)), bits_t(clean)[perm])
    P.x, P.ids = kept
    for bad in (float("inf"), float("nan")):
        P.a[2, 3, 5::7] = bad
        P.b[2, ::5, 1] = bad
        other = P.ids != 2
        y = P.run(silu=True)
        assert torch.equal(bits_t(y)[other], bits_t(clean)[other])
        if bool((~other).any()):
            assert not torch.isfinite(y[~other].float()).all()
    P.x = P.x.clone()
    P.x[T // 2] = float("nan")
    P.ids = torch.where(P.ids == 2, 1, P.ids)
    z, ref = P.run(silu=True), M.w4a16_linear(kept[0], P.p, P.ad(), P.ids, silu=True)
    rest = torch.arange(T, device=dev()) != T // 2
    assert torch.equal(bits_t(z)[rest], bits_t(ref)[rest])


def test_linear_large_inner_values():
    """h past fp16, far above the product, and subnormal: two bf16 parts keep its bits."""
    P = Shared(20, 256, 64, 3, 8)
    P.x *= 200.0
    P.b *= 2.0 ** -12
    P.s = torch.tensor([1e5, 3.0, 2.0 ** -100], device=dev())
    P.check()


def test_linear_writes_its_rows_only_and_takes_its_workspace():
    P = Shared(37, 256, 96, 4, 8)
    need = M.linear_workspace_bytes(P.p, 37, P.ad())
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device=dev())     # NaN everywhere: nothing is read before it is written
    out = torch.full((50, 96), -3.0, dtype=torch.bfloat16, device=dev())
    P.run(out=out, workspace=ws[:need])
    assert torch.equal(bits_t(out[:37]), bits_t(P.run()))
    assert bool((out[37:] == -3.0).all()) and bool((ws[need:] == 255).all())
    with pytest.raises(M.W4A16Error):
        P.run(workspace=ws[:need - 16])
    for bad in (dict(out=out[:30]), dict(out=out.float()), dict(out=out.t()), dict(workspace=ws.float())):
        with pytest.raises((ValueError, TypeError)):
            P.run(**bad)
    with pytest.raises(ValueError):
        M.w4a16_linear(P.x, P.p, P.ad())
    with pytest.raises(ValueError):
        M.w4a16_linear(P.x, P.p, P.ad(), P.ids[:-1])
    with pytest.raises(ValueError):
        M.w4a16_linear(P.x[:, :64], P.p)
    with pytest.raises(TypeError):
        M.w4a16_linear(P.x, P.p, P.ad(), P.ids.long())
    with pytest.raises(ValueError):
        M.adapters(P.a, P.b[:, :, :4].contiguous())
    with pytest.raises(ValueError):
        M.adapters(P.a, P.b[:2])
    with pytest.raises(ValueError):
        M.adapters(P.a, P.b, P.s[:2])
    with pytest.raises(M.W4A16Error):
        M.w4a16_linear(P.x, P.p, M.adapters(P.a, P.b[:, :64].contiguous()), P.ids)     # another width
    empty = M.w4a16_linear(P.x[:0], P.p, P.ad(), P.ids[:0])
    assert empty.shape == (0, 96)


# ------------------------------------------------------- the routed experts

class Routed:
    def __init__(self, T, k, E, first, El, K, N, La, r, slices=1, gate_up=False, seed=0):
        g = torch.Generator(device=dev()).manual_seed(seed + 17 * T + K + N + r)
        self.T, self.k, self.E, self.first, self.El, self.slices = T, k, E, first, El, slices
        self.ids = torch.rand(T, E, generator=g, device=dev()).topk(k, dim=1).indices.to(torch.int32).contiguous()
        self.wt = torch.softmax(torch.randn(T, k, generator=g, device=dev()), dim=1)
        self.x = torch.randn(T, K, generator=g, device=dev()).to(torch.bfloat16)
        self.xs = torch.randn(T * k, K, generator=g, device=dev()).to(torch.bfloat16)
        codes = torch.randint(0, 16, (El, N, K), generator=g, device=dev(), dtype=torch.uint8)
        sc = (0.005 + 0.015 * torch.rand(El, N, K // 32, generator=g, device=dev())).to(torch.bfloat16)
        self.p = M.pack_w4(codes, sc, gate_up=gate_up)
        self.w = AO.int4_values(codes, sc)
        self.a = (torch.randn(La, El, slices * r, K, generator=g, device=dev()) / K ** 0.5).to(torch.bfloat16)
        self.b = torch.randn(La, El, N, r, generator=g, device=dev()).to(torch.bfloat16)
        self.s = 0.5 + torch.rand(La, generator=g, device=dev())
        self.token = torch.randint(-1, La, (T,), generator=g, device=dev(), dtype=torch.int32)

    def ad(self):
        return M.adapters(self.a, self.b, self.s)

    def align(self, block_m):
        return M.moe_align(self.ids, self.E, self.first, self.El, block_m)

    def slots(self, rows):
        """y float64 [T k, N] of the local slots (rows [T k, K]), its fp32 bound, and which are local."""
        T, k = self.T, self.k
        y = torch.zeros(T * k, self.w.shape[1], dtype=torch.float64, device=dev())
        err = torch.zeros_like(y)
        flat = self.ids.view(-1) - self.first
        local = (flat >= 0) & (flat < self.El)
        for e in range(self.El):
            s = (flat == e).nonzero().squeeze(1)
            t = self.token[s // k]
            for l in torch.unique(t).tolist():
                m = s[t == l]
                if l < 0:
                    y[m], err[m] = AO.product(rows[m], self.w[e])
                else:
                    y[m], err[m] = AO.product(rows[m], self.w[e], self.a[l, e], self.b[l, e], float(self.s[l]), self.slices)
        return y, err, local


def _positions(r, T, k):
    """sorted position of every local slot"""
    s = r.sorted_ids.long()
    at = (s < T * k).nonzero().squeeze(1)
    return s[at], at


SHAPES = [dict(T=1, k=8, E=16, first=0, El=16, K=256, N=64, La=2, r=16),
          dict(T=37, k=3, E=12, first=2, El=7, K=1120, N=96, La=5, r=24),
          dict(T=130, k=4, E=10, first=4, El=5, K=384, N=160, La=7, r=8),
          dict(T=600, k=2, E=3, first=0, El=2, K=128, N=288, La=3, r=40),
          dict(T=900, k=2, E=4, first=1, El=3, K=256, N=64, La=4, r=72)]      # enough slots for packed inner values


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("block_m", [16, 32, 64, 128, 256])
def test_routed_gemm_and_silu(shape, block_m):
    T, k, N = shape["T"], shape["k"], shape["N"]
    P = Routed(**shape, slices=2, gate_up=True)
    r = P.align(block_m)
    rows = P.x.repeat_interleave(k, dim=0)
    y, err, local = P.slots(rows)
    out = torch.full((T * k, N), 5.0, dtype=torch.bfloat16, device=dev())
    M.moe_adapter_gemm(P.x, P.p, r, P.ad(), P.token, out=out)
    AO.assert_within(out[local], y[local], (err + AO.HALF_BF16 * y.abs())[local], "per slot")
    assert bool((out[~local] == 5.0).all())
    inter = torch.full((r.capacity, N // 2), 7.0, dtype=torch.bfloat16, device=dev())
    M.moe_adapter_gate_up_silu(P.x, P.p, r, P.ad(), P.token, out=inter)
    s, at = _positions(r, T, k)
    z, bound = AO.activate(y[s], err[s])
    AO.assert_within(inter[at], z, bound, "silu")
    rest = torch.ones(r.capacity, dtype=torch.bool, device=dev())
    rest[at] = False
    assert bool((inter[rest] == 7.0).all())


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("block_m", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("slices", [1, 2])
def test_routed_combine(shape, block_m, slices):
    T, k = shape["T"], shape["k"]
    P = Routed(**shape, slices=slices)
    r = P.align(block_m)
    y, err, local = P.slots(P.xs)
    w = (P.wt.double().view(-1, 1) * local.view(-1, 1)).double()
    ref = (w * y).view(T, k, -1).sum(1)
    size = (w * y).abs().view(T, k, -1).sum(1)
    bound = (w * err).view(T, k, -1).sum(1) + AO.HALF_BF16 * ref.abs() + (k + 2) * 2 * AO.HALF_FP32 * size + 2.0 ** -133
    out = M.moe_adapter_gemm(P.xs, P.p, r, P.ad(), P.token, topk_weights=P.wt)
    AO.assert_within(out, ref, bound, "combine")
    s, at = _positions(r, T, k)
    rows = torch.full((r.capacity, P.xs.shape[1]), float("nan"), dtype=torch.bfloat16, device=dev())
    rows[at] = P.xs[s]
    again = M.moe_adapter_gemm(rows, P.p, r, P.ad(), P.token, topk_weights=P.wt, a_layout="sorted")
    assert torch.equal(bits_t(out), bits_t(again))
    # passes over columns give the same bits
    c = M.indexed_config(r, P.p)
    c.split_k, c.combine_cols = 1, 32
    assert torch.equal(bits_t(out), bits_t(M.moe_adapter_gemm(P.xs, P.p, r, P.ad(), P.token, topk_weights=P.wt, cfg=c)))


@pytest.mark.parametrize("cfg", [(16, 1, 8), (16, 2, 4), (16, 4, 4), (32, 2, 4), (64, 2, 4), (128, 2, 4), (128, 4, 4),
                                 (256, 2, 8)])
def test_routed_every_tile(cfg):
    """Each built tile, K a multiple of 128, blocks that mix adapters and blocks of one."""
    for mixed in (True, False):
        P = Routed(300, 2, 4, 1, 3, 640, 352, 6, 16, slices=2, gate_up=True)
        if not mixed:
            P.token = torch.arange(300, device=dev()).div(130, rounding_mode="floor").to(torch.int32) - 1
        r = P.align(cfg[0])
        y, err, local = P.slots(P.x.repeat_interleave(2, dim=0))
        c = M.config(*cfg)
        out = M.moe_adapter_gemm(P.x, P.p, r, P.ad(), P.token, cfg=c)
        AO.assert_within(out[local], y[local], (err + AO.HALF_BF16 * y.abs())[local], "per slot")
        inter = M.moe_adapter_gate_up_silu(P.x, P.p, r, P.ad(), P.token, cfg=c)
        s, at = _positions(r, 300, 2)
        AO.assert_within(inter[at], *AO.activate(y[s], err[s]), "silu")
        D = Routed(300, 2, 4, 1, 3, 640, 352, 6, 16, seed=9)
        D.ids, D.token = P.ids, P.token
        yd, ed, _ = D.slots(D.xs)
        w = P.wt.double().view(-1, 1) * local.view(-1, 1)
        ref = (w * yd).view(300, 2, -1).sum(1)
        bound = ((w * ed).view(300, 2, -1).sum(1) + AO.HALF_BF16 * ref.abs() +
                 8 * AO.HALF_FP32 * (w * yd).abs().view(300, 2, -1).sum(1) + 2.0 ** -133)
        AO.assert_within(M.moe_adapter_gemm(D.xs, D.p, r, D.ad(), D.token, topk_weights=P.wt, cfg=c), ref, bound, "combine")


def test_routed_without_adapters_is_the_plain_product():
    """Rows without an adapter give what moe_w4a16_gemm gives, to the bit, whatever the tables hold."""
    P = Routed(50, 4, 8, 0, 8, 512, 128, 3, 16)
    P.token.fill_(-1)
    P.a.fill_(float("nan"))
    P.b.fill_(float("inf"))
    for bm, nr, waves in ((16, 2, 4), (32, 2, 4), (64, 2, 4)):
        r, c = P.align(bm), M.config(bm, nr, waves)
        assert torch.equal(bits_t(M.moe_adapter_gemm(P.x, P.p, r, P.ad(), P.token, cfg=c)),
                           bits_t(M.moe_w4a16_gemm(P.x, P.p, r, cfg=c)))


def test_routed_other_experts_and_requests_do_not_matter():
    P = Routed(60, 3, 9, 2, 4, 256, 64, 4, 8, slices=2, gate_up=True)
    r = P.align(16)
    clean = M.moe_adapter_gemm(P.x, P.p, r, P.ad(), P.token)
    P.a[1, 2] = float("nan")
    P.b[3, 0] = float("inf")
    y = M.moe_adapter_gemm(P.x, P.p, r, P.ad(), P.token)
    e = P.ids.view(-1) - P.first
    t = P.token.repeat_interleave(3)
    hit = ((e == 2) & (t == 1)) | ((e == 0) & (t == 3))
    assert torch.equal(bits_t(y)[~hit], bits_t(clean)[~hit])
    same = torch.zeros_like(P.ids)                        # one expert chosen by every slot, another never
    P.ids = same + P.first + 1
    r = P.align(16)
    z, err, local = P.slots(P.x.repeat_interleave(3, dim=0))
    out = M.moe_adapter_gemm(P.x, P.p, r, P.ad(), P.token)
    AO.assert_within(out, z, err + AO.HALF_BF16 * z.abs())


# --------------------------------------------------- streams, graphs, a layer

def _layer():
    """router -> routed experts with adapters + the shared expert with its own, as a step of a serving loop"""
    T, k, E, H, I = 24, 4, 32, 512, 256
    up = Routed(T, k, E, 0, E, H, 2 * I, 4, 16, slices=2, gate_up=True)
    down = Routed(T, k, E, 0, E, I, H, 4, 16)
    s_up = Shared(T, H, 2 * I, 4, 8, 2, gate_up=True)
    s_down = Shared(T, I, H, 4, 8)
    g = torch.Generator(device=dev()).manual_seed(2)
    gate = torch.randn(E, H, generator=g, device=dev()).to(torch.bfloat16)
    return T, k, E, up, down, s_up, s_down, gate


def _step(x, token, k, E, up, down, s_up, s_down, gate):
    ids, w = M.moe_route_grouped((x @ gate.t()).float(), k, 8, 4, scoring="sigmoid", scale=2.0)
    r = M.moe_align(ids, E, 0, E, 16)
    h = M.moe_adapter_gate_up_silu(x, up.p, r, up.ad(), token)
    y = M.moe_adapter_gemm(h, down.p, r, down.ad(), token, topk_weights=w, a_layout="sorted")
    hs = M.w4a16_linear(x, s_up.p, s_up.ad(), token, silu=True)
    return ids, w, r, h, y, hs, M.w4a16_linear(hs, s_down.p, s_down.ad(), token)


def test_layer_end_to_end():
    T, k, E, up, down, s_up, s_down, gate = _layer()
    token = up.token
    ids, w, r, h, y, hs, ys = _step(up.x, token, k, E, up, down, s_up, s_down, gate)
    l = (up.x @ gate.t()).float()
    np.testing.assert_array_equal(ids.cpu().numpy(), AO.route_grouped(l.double().cpu().numpy(), k, 8, 4, "sigmoid")[0])
    up.ids = down.ids = ids
    down.token = token
    a, ea, _ = up.slots(up.x.repeat_interleave(k, dim=0))
    s, at = _positions(r, T, k)
    AO.assert_within(h[at], *AO.activate(a[s], ea[s]), "gate/up")
    rows = torch.empty(T * k, h.shape[1], dtype=torch.bfloat16, device=dev())
    rows[s] = h[at]                                       # each step against its own rounded input
    d, ed, _ = down.slots(rows)
    wd = w.double().view(-1, 1)
    ref = (wd * d).view(T, k, -1).sum(1)
    bound = ((wd * ed).view(T, k, -1).sum(1) + AO.HALF_BF16 * ref.abs() +
             (k + 2) * 2 * AO.HALF_FP32 * (wd * d).abs().view(T, k, -1).sum(1))
    AO.assert_within(y, ref, bound, "down")
    AO.assert_within(hs, *AO.linear(up.x, s_up.w, token, (s_up.a, s_up.b, s_up.s), 2, True), "shared gate/up")
    AO.assert_within(ys, *AO.linear(hs, s_down.w, token, (s_down.a, s_down.b, s_down.s)), "shared down")


def test_layer_captured_and_replayed():
    """New rows, routing and adapters through one captured step, replayed between eager work on the same memory."""
    T, k, E, up, down, s_up, s_down, gate = _layer()
    x, token = up.x.clone(), up.token.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(x, token, k, E, up, down, s_up, s_down, gate)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _step(x, token, k, E, up, down, s_up, s_down, gate)
    g = torch.Generator(device=dev()).manual_seed(5)
    for i in range(4):
        x.copy_(torch.randn(x.shape, generator=g, device=dev()))
        token.copy_(torch.randint(-1, 4, (T,), generator=g, device=dev()))
        graph.replay()
        torch.cuda.synchronize()
        replayed = [got[j].clone() for j in (0, 1, 4, 5, 6)]
        eager = _step(x, token, k, E, up, down, s_up, s_down, gate)
        for a, b in zip(replayed, [eager[j] for j in (0, 1, 4, 5, 6)]):
            assert torch.equal(a, b), i


def test_two_streams_at_once():
    P, Q = Shared(64, 2048, 1024, 8, 16, seed=1), Shared(300, 1024, 2048, 8, 16, seed=2)
    ref = P.run(), Q.run()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        with torch.cuda.stream(s1):
            outs.append((0, P.run()))
        with torch.cuda.stream(s2):
            outs.append((1, Q.run()))
    torch.cuda.synchronize()
    for i, y in outs:
        assert torch.equal(bits_t(y), bits_t(ref[i]))


def test_repeated_calls_give_the_same_bits():
    P = Shared(301, 2048, 1024, 64, 32)
    first = P.run()
    for _ in range(5):
        assert torch.equal(bits_t(P.run()), bits_t(first))
