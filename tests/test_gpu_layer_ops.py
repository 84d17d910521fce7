"""GPU parity of the router, the few-token layer, the MXFP4 weight quantiser
and the grouped MXFP4 products against the float64 oracle."""
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from gpu_util import bits, dev, log, to_dev, to_dev_bf16  # noqa: E402

from oracle import layer_oracle as LO  # noqa: E402
from oracle import moe_oracle as O  # noqa: E402
from oracle import mx_oracle as X  # noqa: E402
from synth import workloads as W  # noqa: E402

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU visible")]

import w4a16_int4_mixture_moe_amd as M  # noqa: E402


# ------------------------------------------------------------------ router

def _check_route(logits: torch.Tensor, k, scoring, bias=None, renorm=True, scale=1.0, what=""):
    ids, w = M.moe_route(logits, k, scoring=scoring, bias=bias, renormalize=renorm, scale=scale)
    ref_ids, ref_w, tol = LO.route(logits.double().cpu().numpy(), k, scoring,
                                   None if bias is None else bias.double().cpu().numpy(), renorm, scale)
    np.testing.assert_array_equal(ids.cpu().numpy(), ref_ids, err_msg=what)
    err = np.abs(w.double().cpu().numpy() - ref_w)
    assert (err <= tol).all(), (what, float((err / np.maximum(tol, 1e-300)).max()))
    return ids, w


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 5, 5), (5, 63, 2), (4, 64, 32), (7, 65, 8), (257, 384, 8),
                                   (33, 448, 9), (9, 768, 6), (66, 896, 16), (6, 1024, 32)])
def test_route_shapes(T, E, k, dtype):
    g = torch.Generator().manual_seed(T * 131 + E)
    l = torch.randn(T, E, generator=g).to(dtype).to(dev())
    b = (0.1 * torch.randn(E, generator=g)).to(dev())
    for renorm in (True, False):
        _check_route(l, k, "softmax", None, renorm, 1.0, "softmax")
        _check_route(l, k, "sigmoid", None, renorm, 2.5, "sigmoid")
        _check_route(l, k, "sigmoid", b, renorm, 2.5, "sigmoid + bias")


@pytest.mark.parametrize("scoring,biased", [("softmax", False), ("sigmoid", False), ("sigmoid", True)])
def test_route_masks_infinities_and_ties(scoring, biased):
    n, inf, big = float("nan"), float("inf"), 3e38
    E, k = 70, 4
    rows = torch.zeros(9, E)
    rows[0] = -inf                                        # nothing left
    rows[1] = n
    rows[2] = -inf
    rows[2, 69] = -3.0                                    # fewer than k
    rows[2, 1] = 1.0
    rows[3, 5] = inf
    rows[3, 66] = inf                                     # two infinities share
    rows[3, 7] = n
    rows[4] = -0.0
    rows[4, 3] = 0.0                                      # equal to -0
    rows[5] = -200.0                                      # scores below fp32's range
    rows[6, ::2] = -big
    rows[7, 68] = big
    rows[8] = torch.arange(E) % 3                         # many ties
    b = torch.zeros(E) if biased else None
    if biased:
        b[0], b[1], b[2], b[9] = -inf, n, inf, 2.0
    l = rows.to(dev())
    b = None if b is None else b.to(dev())
    for renorm in (True, False):
        _check_route(l, k, scoring, b, renorm, 1.0, f"{scoring} {renorm}")


def test_route_orders_near_ties_in_64_bits():
    """Biases that bring every sum to about one half: 32-bit keys cannot order them."""
    g = torch.Generator().manual_seed(11)
    E = 384
    l = torch.randn(40, E, generator=g)
    l[20:] = l[0]
    l[20:30] += 1e-6 * torch.randn(10, E, generator=g)
    b = (0.5 - torch.sigmoid(l[0].double())).float()
    _check_route(l.to(dev()), 8, "sigmoid", b.to(dev()), True, 1.0, "near ties")
    _check_route(torch.zeros(5, E, device=dev()), 8, "sigmoid", torch.zeros(E, device=dev()), True, 1.0, "all equal")
    huge = torch.linspace(1e4, 1e4 + 0.4, E).to(dev())    # the bias swallows the score's low bits in 32 bits
    _check_route(l.to(dev()), 8, "sigmoid", huge, True, 1.0, "large bias")


@pytest.mark.parametrize("T", [5, 6151])
@pytest.mark.parametrize("E,k,stride,lanes", [(384, 8, 16, 1), (1024, 9, 16, 3), (1024, 32, 64, 31), (896, 10, 64, 9)])
def test_route_crowded_residues(T, E, k, stride, lanes):
    """The largest logits at experts of a few residues: far more than k experts lie above any bound by residue."""
    g = torch.Generator().manual_seed(T + E + k)
    l = 0.1 * torch.randn(T, E, generator=g)
    l[:, torch.arange(E) % stride < lanes] += 3.0
    l[1::3] = l[1::3].round(decimals=1)                   # and many equal ones
    b = (0.05 * torch.randn(E, generator=g)).to(dev())
    for dtype in (torch.float32, torch.bfloat16):
        d = l.to(dtype).to(dev())
        _check_route(d, k, "softmax", None, True, 1.0, "softmax")
        _check_route(d, k, "sigmoid", b, True, 1.5, "sigmoid + bias")


@pytest.mark.parametrize("E,k", [(384, 8), (9, 9), (100, 10), (1000, 3)])
def test_route_many_tokens(E, k):
    g = torch.Generator().manual_seed(E + k)
    l = torch.randn(6147, E, generator=g)
    l[torch.rand(6147, E, generator=g) < 0.05] = float("-inf")
    l[3] = float("nan")
    l[4] = float("-inf")
    l[4, E - 1] = float("inf")
    l[6146] = 0.0
    b = (0.1 * torch.randn(E, generator=g)).to(dev())
    _check_route(l.to(dev()), k, "softmax", None, False, 1.0, "softmax")
    _check_route(l.to(dev()), k, "sigmoid", b, True, 1.0, "sigmoid + bias")
    wide = torch.full((6147, E + 7), float("inf"), device=dev())   # what lies between the rows is never chosen
    wide[:, 4:4 + E] = l.to(dev())
    _check_route(wide[:, 4:4 + E], k, "sigmoid", None, True, 1.0, "strided")


def _route_constant(name):
    """A launch rule's constant, from the kernel's source."""
    import re
    src = os.path.join(os.path.dirname(M.__file__), "csrc", "route.hip")
    return int(re.search(rf"constexpr int {name} = (\d+);", open(src).read()).group(1))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("E", [100, 200, 384, 500, 700, 1000])
@pytest.mark.parametrize("T,k", [(41, 8), (6149, 8), (6149, 12)])
def test_route_every_built_width(T, k, E, dtype):
    """16 lanes a token hold 8, 16, 24 or 32 keys each, 64 lanes 2, 4, 6, 8, 14 or 16; every logit type.
    Against the definition in 64 bits, all rows at once."""
    narrow = (T >= _route_constant("kNarrowMinTokens") and k <= _route_constant("kNarrowMaxTopk") and
              E <= _route_constant("kNarrowMaxExperts"))
    assert narrow == ((T, k) == (6149, 8) and E <= 500)
    g = torch.Generator().manual_seed(T + E + k)
    l = torch.randn(T, E, generator=g)
    l[torch.rand(T, E, generator=g) < 0.03] = float("-inf")
    l[5] = float("-inf")
    l[6, 9:] = float("nan")                                # nine experts left
    l[7, E - 1], l[7, 0] = float("inf"), float("inf")
    l = l.to(dtype)
    b = 0.1 * torch.randn(E, generator=g)
    x = l.double().clamp(max=float(np.finfo(np.float32).max))
    live = ~(l.isnan() | (l == float("-inf")))
    for scoring, bias, renorm in (("softmax", None, True), ("softmax", None, False), ("sigmoid", None, False),
                                  ("sigmoid", b, True)):
        ids, w = M.moe_route(l.to(dev()), k, scoring=scoring, bias=None if bias is None else b.to(dev()),
                             renormalize=renorm, scale=1.5)
        sig = 1.0 / (1.0 + torch.exp(-x))
        key = torch.where(live, x if bias is None else sig + b.double(), float("-inf"))
        order = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
        ok = live.gather(1, order)
        assert torch.equal(ids.cpu(), torch.where(ok, order, -1).int()), (scoring, renorm)
        top = torch.where(live, x, float("-inf")).amax(1, keepdim=True)
        score = torch.where(live, sig if scoring == "sigmoid" else torch.exp(x - top), 0.0)
        ref = score.gather(1, order)
        if scoring == "softmax":
            ref = ref / (ref if renorm else score).sum(1, keepdim=True).clamp(min=1e-300)
        elif renorm:
            ref = ref / (ref.sum(1, keepdim=True) + 1e-20)
        ref = torch.where(ok, ref, 0.0) * 1.5
        # differences from the maximum up to 16 rounded once, exp and division a few units, in weight and sum
        # (row 7's other differences are past fp32's exp, and 0 in both)
        tol = 2 * (16 + 8) * 2.0 ** -24 * ref + 2.0 ** -126
        assert ((w.double().cpu() - ref).abs() <= tol).all(), (scoring, renorm)


def test_route_strided_rows_other_stream_and_refusals():
    wide = torch.randn(50, 512, device=dev())
    _check_route(wide[::2, 64:64 + 96], 5, "softmax", what="strided")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ids, w = M.moe_route(wide, 4)
    s.synchronize()
    ref = M.moe_route(wide, 4)
    assert torch.equal(ids, ref[0]) and torch.equal(w, ref[1])
    e = M.moe_route(wide[:0], 4)
    assert e[0].shape == (0, 4) and e[1].shape == (0, 4)
    with pytest.raises(ValueError):
        M.moe_route(wide.t(), 4)
    with pytest.raises(ValueError):
        M.moe_route(wide, 4, scoring="max")
    with pytest.raises(TypeError):
        M.moe_route(wide.double(), 4)
    with pytest.raises(ValueError):
        M.moe_route(wide, 4, scoring="sigmoid", bias=torch.zeros(4, device=dev()))
    for k in (33, 0, -1, 513, 2**32 + 4):
        with pytest.raises(M.W4A16Error):
            M.moe_route(wide, k)


@pytest.mark.parametrize("T", [3, 6147])
def test_route_scores_below_the_normal_range(T):
    """Scores that fp32 holds in a few bits or not at all, brought back into range by the sum or the scale."""
    lows = torch.linspace(-78.0, -130.0, 53)
    l = torch.full((T, 64), float("-inf"))
    l[0, :53] = lows
    l[1, :53] = lows.flip(0)
    l[2, 7:11] = -100.0
    l[3:, 3], l[3:, 60] = -95.0, -103.0
    d = l.to(dev())
    v = l.double().numpy()
    bias = torch.zeros(64, device=dev())
    for scoring, renorm, b, scale in (("sigmoid", True, None, 1.0), ("sigmoid", True, bias, 2.5),
                                      ("sigmoid", False, None, 2.0**70), ("softmax", True, None, 2.0**100),
                                      ("softmax", False, None, 2.0**100)):
        ids, w = M.moe_route(d, 4, scoring=scoring, bias=b, renormalize=renorm, scale=scale)
        ref_ids, ref_w, _ = LO.route(v, 4, scoring, None if b is None else np.zeros(64), renorm, scale)
        np.testing.assert_array_equal(ids.cpu().numpy(), ref_ids)
        got = w.double().cpu().numpy()
        # a score within 5 units of 2^-24 (difference, exp, sum and division round once each, exp twice), the
        # chosen scores' sum as far, one rounding of the weight, which may be a subnormal; a difference from the
        # maximum is exact here (all are whole numbers)
        tol = 11 * 2.0 ** -24 * np.abs(ref_w) + 2.0 ** -150
        assert (np.abs(got - ref_w) <= tol).all(), (scoring, renorm, float((np.abs(got - ref_w) / tol).max()))


@pytest.mark.parametrize("T,E,k", [(2**26 + 5, 11, 11), (2**28 + 5, 2, 1)])
def test_route_more_tokens_than_one_grid_holds(T, E, k):
    """Past 2^26 (64 lanes a token) or 2^28 tokens (16 lanes) the threads of one launch do not fit 32 bits."""
    n = 2**20
    g = torch.Generator().manual_seed(k)
    block = torch.randn(n, E, generator=g).half().to(dev())
    logits = block.repeat(T // n + 1, 1)[:T]
    ref_ids, ref_w = M.moe_route(block, k)
    _check_route(block[:500].contiguous(), k, "softmax")
    ids, w = M.moe_route(logits, k)
    for got, ref in ((ids, ref_ids), (w, ref_w)):
        whole = got[:T // n * n].view(T // n, n, k)
        assert all(torch.equal(part, ref) for part in whole)
        assert torch.equal(got[T // n * n:], ref[:T % n])


def test_sizes_past_32_bits_are_refused(layers):
    """Cut to 32 bits each of these would be a small call; nothing is written, so nothing is launched."""
    big = 2**32
    for T, E in ((big + 4, 1), (1, big + 8), (2**31, 1)):
        with pytest.raises(ValueError, match="32-bit"):
            M.moe_route(torch.empty(T, E, dtype=torch.float16, device=dev()), 1)
    lay = layers["int4"]
    x = torch.zeros(1, lay.H, dtype=torch.bfloat16, device=dev())
    ids = torch.empty(1, big + 1, dtype=torch.int32, device=dev())
    with pytest.raises(ValueError, match="32-bit"):
        M.moe_few_tokens(x, lay.p1, lay.p2, ids, ids.view(torch.float32))
    del ids
    packed, _ = _mx_weight(1, 16, 128, 2)
    rows = M.MXRows(torch.zeros(8, 64, dtype=torch.uint8, device=dev()), torch.zeros(8, 4, dtype=torch.uint8, device=dev()))
    with pytest.raises(ValueError, match="32-bit"):
        M.grouped_mxfp4_masked(rows, packed, torch.zeros(1, dtype=torch.int32, device=dev()), big + 8)
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ few-token layer

class Layer:
    """Seeded weights of one layer share, on the device and as float64."""

    def __init__(self, kind, E, H, I, seed=0):
        rng = np.random.default_rng(seed)
        self.kind, self.E, self.H, self.I = kind, E, H, I
        if kind == "int4":
            c1, c2 = (rng.integers(0, 16, s, dtype=np.uint8) for s in ((E, 2 * I, H), (E, H, I)))
            s1, s2 = (W.to_bf16_bits(rng.uniform(0.005, 0.02, s).astype(np.float32))
                      for s in ((E, 2 * I, H // 32), (E, H, I // 32)))
            self.p1 = M.pack_w4(to_dev(c1), to_dev_bf16(s1), gate_up=True)
            self.p2 = M.pack_w4(to_dev(c2), to_dev_bf16(s2))
            self.w1, self.w2 = O.dequant(c1, s1), O.dequant(c2, s2)
        else:
            c1, c2 = (rng.integers(0, 256, s, dtype=np.uint8) for s in ((E, 2 * I, H // 2), (E, H, I // 2)))
            s1, s2 = (rng.integers(119, 123, s, dtype=np.uint8) for s in ((E, 2 * I, H // 32), (E, H, I // 32)))
            self.p1 = M.pack_mxfp4(to_dev(c1), to_dev(s1), gate_up=True)
            self.p2 = M.pack_mxfp4(to_dev(c2), to_dev(s2))
            self.w1 = X.mx_dequant(X.unpack_nibbles(c1), s1)
            self.w2 = X.mx_dequant(X.unpack_nibbles(c2), s2)

    def check(self, x_bits, ids, wt, first, what):
        T, k = ids.shape
        n = M.few_tokens_workspace_bytes(self.p1, T, k)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=dev())     # not initialised: any contents do
        out = torch.full((T + 1, self.H), 7.0, dtype=torch.bfloat16, device=dev())
        M.moe_few_tokens(to_dev_bf16(x_bits), self.p1, self.p2, to_dev(ids), to_dev(wt), first, out=out, workspace=ws)
        torch.cuda.synchronize()
        assert (out[T] == 7.0).all(), f"{what}: wrote behind the last token"
        ref, tol = LO.few_tokens(x_bits, self.w1, self.w2, ids, wt, first)
        share = LO.assert_within(bits(out[:T]), ref, tol, what)
        log(f"few {self.kind} {what}: {share:.2f} of the bound")
        return bits(out[:T])


def _tokens(T, k, E_glob, H, seed):
    rng = np.random.default_rng(seed)
    x = W.to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32))
    ids = np.stack([rng.permutation(E_glob)[:k] for _ in range(T)]).astype(np.int32) if T else np.zeros((0, k), np.int32)
    wt = rng.uniform(0.05, 1.0, (T, k)).astype(np.float32)
    return x, ids, wt


@pytest.fixture(scope="module")
def layers():
    return {"int4": Layer("int4", 6, 288, 160), "mxfp4": Layer("mxfp4", 6, 384, 128),
            "int4_wide": Layer("int4", 3, 1280, 640, 1)}


@pytest.mark.parametrize("kind", ["int4", "mxfp4"])
@pytest.mark.parametrize("T,k", [(1, 1), (1, 6), (2, 3), (7, 4), (16, 2), (17, 3), (32, 6), (33, 2), (64, 4), (64, 16)])
def test_few_tokens_shapes(layers, kind, T, k):
    lay = layers[kind]
    x, ids, wt = _tokens(T, k, 20, lay.H, T * 17 + k)      # experts 3..8 of 20 are held here
    lay.check(x, ids, wt, 3, f"T={T} k={k}")


@pytest.mark.parametrize("kind", ["int4", "mxfp4"])
def test_few_tokens_routing_corners(layers, kind):
    lay = layers[kind]
    x, ids, wt = _tokens(40, 3, 6, lay.H, 5)
    hot = ids.copy()
    hot[:, 0] = 2                                          # one expert holds every token: blocks of 16, 16, 8
    hot[:, 1] = np.where(ids[:, 1] == 2, 0, ids[:, 1])
    lay.check(x, hot, wt, 0, "hot expert")
    twice = ids.copy()
    twice[::3, 2] = twice[::3, 0]                          # a token names an expert twice
    twice[4] = 5
    lay.check(x, twice, wt, 0, "twice")
    away = ids.copy()
    away[::2] = -1                                         # rows without any expert
    away[1, 1] = 99
    away[3] = np.iinfo(np.int32).min
    y = lay.check(x, away, wt, 0, "held elsewhere")
    assert not y[::2].any()
    lay.check(x, np.full_like(ids, 9), wt, 0, "none held")
    wt[:, 1] = 0.0
    wt[5] = -wt[5]
    lay.check(x, ids, wt, 0, "zero and negative weights")


def test_few_tokens_wide_layer_and_nan_rows(layers):
    lay = layers["int4_wide"]
    x, ids, wt = _tokens(20, 2, 3, lay.H, 8)
    y = lay.check(x, ids, wt, 0, "wide")
    x2 = x.copy()
    x2[3] = 0x7FC0                                         # one token's NaN stays with it
    x2[17, 0] = 0x7F80
    out = M.moe_few_tokens(to_dev_bf16(x2), lay.p1, lay.p2, to_dev(ids), to_dev(wt))
    got = bits(out)
    keep = [t for t in range(20) if t not in (3, 17)]
    np.testing.assert_array_equal(got[keep], y[keep])
    assert torch.isnan(out[3].float()).all()


def test_few_tokens_empty_and_refusals(layers):
    lay = layers["int4"]
    x, ids, wt = _tokens(4, 2, 6, lay.H, 1)
    dx, di, dw = to_dev_bf16(x), to_dev(ids), to_dev(wt)
    assert M.moe_few_tokens(dx[:0], lay.p1, lay.p2, di[:0], dw[:0]).shape == (0, lay.H)
    with pytest.raises(ValueError):
        M.moe_few_tokens(dx, lay.p1, lay.p2, di[:3], dw)
    with pytest.raises(ValueError):
        M.moe_few_tokens(dx[:, :256].contiguous(), lay.p1, lay.p2, di, dw)
    with pytest.raises(ValueError):
        M.moe_few_tokens(dx.t().contiguous().t(), lay.p1, lay.p2, di, dw)
    with pytest.raises(TypeError):
        M.moe_few_tokens(dx, lay.p1, lay.p2, di.long(), dw)
    with pytest.raises(M.W4A16Error):
        M.moe_few_tokens(dx, lay.p2, lay.p1, di, dw) if lay.p2.K == lay.H else M.moe_few_tokens(
            dx, lay.p1, lay.p1, di, dw)
    with pytest.raises(M.W4A16Error):
        M.moe_few_tokens(dx, lay.p1, lay.p2, di, dw, workspace=torch.empty(64, dtype=torch.uint8, device=dev()))
    ws = torch.empty(4 * M.few_tokens_workspace_bytes(lay.p1, 4, 2), dtype=torch.uint8, device=dev())
    with pytest.raises(ValueError):                       # bytes between a strided view's are not the call's
        M.moe_few_tokens(dx, lay.p1, lay.p2, di, dw, workspace=ws[::2])
    with pytest.raises(TypeError):
        M.moe_few_tokens(dx, lay.p1, lay.p2, di, dw, workspace=ws.view(torch.int32))
    for first in (-1, 2**32):
        with pytest.raises(ValueError):
            M.moe_few_tokens(dx, lay.p1, lay.p2, di, dw, first_expert=first)


def _few_constant(name):
    """A launch rule's constant, from the kernel's source."""
    import re
    src = os.path.join(os.path.dirname(M.__file__), "csrc", "few.hip")
    return int(re.search(rf"constexpr int {name} = (\d+);", open(src).read()).group(1))


def _blocks(ids, first, E):
    """Blocks of 16 rows of the local experts (a token counts once an expert)."""
    return sum(-(-int((ids == first + e).any(1).sum()) // 16) for e in range(E))


@pytest.mark.parametrize("kind,H,I", [("int4", 416, 2048), ("mxfp4", 384, 2048), ("int4", 1280, 1696)])
def test_few_tokens_several_items_a_workgroup(kind, H, I):
    """More than two rounds of gate/up items, of blocks with unequal row counts: items follow each other in a
    workgroup with loads in flight, and both buffers of partial sums are used again."""
    lay = Layer(kind, 4, H, I, H)
    x, ids, wt = _tokens(64, 4, 6, H, I)                     # experts 1..4 of 6
    ids[:, 3] = np.where(ids[:, 3] == 2, -1, ids[:, 3])
    ids[40:][ids[40:] == 4] = 0
    blocks = _blocks(ids, 1, 4)
    counts = {int((ids == e).any(1).sum()) % 16 for e in range(1, 5)}
    assert blocks * (I // 16) > 2 * _few_constant("kFewGroups") and len(counts) > 1
    lay.check(x, ids, wt, 1, f"{blocks * (I // 16)} items")


@pytest.mark.parametrize("kind,I", [("int4", 480), ("mxfp4", 512)])
def test_few_tokens_two_column_tiles(kind, I):
    """The down kernel of wide layers, in each of its token counts; INT4's I ends inside a chunk."""
    H = 7168
    lay = Layer(kind, 2, H, I, 3)
    for T, k in ((16, 8), (13, 10), (32, 6), (17, 8), (64, 4), (33, 4)):
        assert H // 16 >= 2 * _few_constant("kFewWideDown")
        assert T * k * -(-I // 128) >= _few_constant("kFewWideUnits")
        x, ids, wt = _tokens(T, k, 12, H, T)                 # experts 4, 5 of 12
        lay.check(x, ids, wt, 4, f"wide T={T}")


@pytest.mark.parametrize("kind,E,H,I", [("int4", 200, 96, 160), ("mxfp4", 300, 128, 256), ("int4", 600, 96, 64)])
def test_few_tokens_many_blocks(kind, E, H, I):
    """More blocks than the down kernel's waves stage at a time; experts past the 512th."""
    lay = Layer(kind, E, H, I, E)
    x, ids, wt = _tokens(64, 16, E, H, E)
    waves, stage = _few_constant("kFewWaves"), _few_constant("kStage")
    assert _blocks(ids, 0, E) > (waves + 1) * stage           # some wave has more than kStage blocks
    lay.check(x, ids, wt, 0, f"{E} experts")


@pytest.mark.parametrize("kind,H,I", [("int4", 64, 32), ("mxfp4", 128, 128)])
def test_few_tokens_as_many_blocks_as_slots(kind, H, I):
    """The largest call in blocks: 1024 slots, an expert each."""
    E = _few_constant("kFewWaves") * 64 * 2                  # W4A16_FEW_MAX_EXPERTS
    lay = Layer(kind, E, H, I, 9)
    x, _, wt = _tokens(64, 16, 16, H, 9)
    ids = np.random.default_rng(9).permutation(E).astype(np.int32).reshape(64, 16)
    assert _blocks(ids, 0, E) == 1024
    lay.check(x, ids, wt, 0, "a block a slot")
    ids[:, 1:] = E - 1                                       # and the last expert for everyone, many times
    lay.check(x, ids, wt, 0, "one expert listed 15 times")


@pytest.mark.parametrize("kind", ["int4", "mxfp4"])
def test_few_tokens_repeats_its_bits(kind):
    """Sums meet in a fixed order: every run of a call gives the same bits."""
    lay = Layer(kind, 4, 1280, 2048, 5)
    x, ids, wt = _tokens(64, 4, 4, 1280, 6)
    dx, di, dw = to_dev_bf16(x), to_dev(ids), to_dev(wt)
    ref = M.moe_few_tokens(dx, lay.p1, lay.p2, di, dw).clone()
    for _ in range(20):
        assert torch.equal(M.moe_few_tokens(dx, lay.p1, lay.p2, di, dw), ref)


def test_few_tokens_first_expert_limit(layers):
    lay = layers["int4"]
    x, ids, wt = _tokens(5, 3, 6, lay.H, 12)
    top = 2**30
    lay.check(x, ids + np.int32(top), wt, top, "last first expert")
    for low in (np.iinfo(np.int32).min, np.iinfo(np.int32).min + 5, -1, 0, top - 1):      # below the range, however far
        assert not lay.check(x, np.full_like(ids, low), wt, top, "below").any()
    dx, di, dw = to_dev_bf16(x), to_dev(ids), to_dev(wt)
    for first in (top + 1, 2**31 - 1):
        with pytest.raises(ValueError, match="first_expert"):
            M.moe_few_tokens(dx, lay.p1, lay.p2, di, dw, first_expert=first)


def test_few_tokens_agrees_with_the_routed_path(layers):
    """align + fused gate/up + down on the same inputs: the same h up to its
    extra bf16 roundings of gate and up, the same sums."""
    lay = layers["int4_wide"]
    x, ids, wt = _tokens(24, 2, 3, lay.H, 21)
    dx, di, dw = to_dev_bf16(x), to_dev(ids), to_dev(wt)
    y = M.moe_few_tokens(dx, lay.p1, lay.p2, di, dw).float()
    r = M.moe_align(di, 3, 0, 3, 16)
    z = M.moe_w4a16_gemm(M.moe_gate_up_silu(dx, lay.p1, r), lay.p2, r, dw, a_layout="sorted").float()
    # gate, up and their product rounded to bf16: three half steps an h instead of one, independent,
    # against sums whose root mean square is that of the outputs
    rms = y.pow(2).mean().sqrt()
    assert ((y - z).abs() <= 7 * 4 * 2.0 ** -8 * rms + 2.0 ** -7 * y.abs()).all()


def test_routed_path_skips_slots_without_an_expert(layers):
    """The router's -1 ids through moe_align and the combine."""
    lay = layers["int4_wide"]
    x, _, _ = _tokens(20, 2, 3, lay.H, 31)
    dx = to_dev_bf16(x)
    l = torch.randn(20, 3, device=dev())
    l[::4] = float("-inf")
    l[1, 1:] = float("nan")                                # one expert left for two slots
    di, dw = M.moe_route(l, 2)
    assert (di[::4] == -1).all() and di[1].tolist() == [0, -1] and dw[1].tolist() == [1.0, 0.0]
    y = M.moe_few_tokens(dx, lay.p1, lay.p2, di, dw).float()
    r = M.moe_align(di, 3, 0, 3, 16)
    z = M.moe_w4a16_gemm(M.moe_gate_up_silu(dx, lay.p1, r), lay.p2, r, dw, a_layout="sorted").float()
    assert not y[::4].any() and not z[::4].any()
    rms = y.pow(2).mean().sqrt()                           # bounds as in the test above
    assert ((y - z).abs() <= 7 * 4 * 2.0 ** -8 * rms + 2.0 ** -7 * y.abs()).all()


# ------------------------------------------------------------------ chain, graph, streams

def test_route_then_layer_captured_and_replayed(layers):
    """Router and layer in one HIP graph on new inputs each replay, eager work
    between, against the eager calls; two graphs alive at once."""
    for kind in ("int4", "mxfp4"):
        lay = layers[kind]
        T, k = 18, 3
        x = torch.empty(T, lay.H, dtype=torch.bfloat16, device=dev())
        l = torch.empty(T, lay.E, device=dev())

        def step():
            ids, w = M.moe_route(l, k, scoring="sigmoid")
            return M.moe_few_tokens(x, lay.p1, lay.p2, ids, w)

        x.normal_()
        l.normal_()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graphs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                y = step()
            graphs.append((g, y))
        for rep in range(4):
            x.normal_()
            l.normal_()
            l[rep] = float("-inf")                          # a padded token: no expert
            torch.cuda.synchronize()
            for g, y in graphs:
                g.replay()
            torch.cuda.synchronize()
            ref = step()
            for g, y in graphs:
                assert torch.equal(y, ref), (kind, rep)
            assert not ref[rep].any()
            _ = (x.float() @ x.float().t()).sum().item()


def test_few_tokens_on_two_streams_at_once(layers):
    lay = layers["int4_wide"]
    x, ids, wt = _tokens(30, 2, 3, lay.H, 77)
    dx, di, dw = to_dev_bf16(x), to_dev(ids), to_dev(wt)
    ref = M.moe_few_tokens(dx, lay.p1, lay.p2, di, dw)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(5):
        for s, o in zip(streams, outs):
            with torch.cuda.stream(s):
                o.append(M.moe_few_tokens(dx, lay.p1, lay.p2, di, dw))
    torch.cuda.synchronize()
    for o in outs:
        for y in o:
            assert torch.equal(y, ref)


# ------------------------------------------------------------------ MXFP4 weights

def _special(N, K, rng):
    v = rng.standard_normal((N, K)) * np.repeat(2.0 ** rng.integers(-20, 20, (N, K // 32)), 32, axis=1)
    v[0, :32] = 0.0
    v[1, :32] = -0.0
    v[2, :12] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -2.5, 5.01, 0.24]     # every tie, at scale 1
    v[2, 12:32] = 0.0
    v[3, :32] = 2.0 ** -130
    v[4, :4] = [7.5, -7.9, 7.0, 0.1]
    v[5, :2] = [2.0 ** 127, -(2.0 ** 126)]
    return v


@pytest.mark.parametrize("gate_up", [False, True])
@pytest.mark.parametrize("E,N,K", [(1, 64, 128), (3, 192, 384), (2, 64, 1280)])
def test_quant_pack_bf16_equals_quantise_then_pack(E, N, K, gate_up):
    rng = np.random.default_rng(N + K)
    w = W.to_bf16_bits(np.stack([_special(N, K, rng) for _ in range(E)]).astype(np.float32))
    d = to_dev_bf16(w)
    p = M.quant_pack_mxfp4(d, gate_up=gate_up)
    q = M.mxfp4_quant(d.view(E * N, K))
    ref = M.pack_mxfp4(q.codes.view(E, N, K // 2), q.scales.view(E, N, K // 32), gate_up=gate_up)
    assert torch.equal(p.w, ref.w) and torch.equal(p.s, ref.s)
    oc, os_ = X.mx_quantize(w.reshape(E * N, K))
    val = X.mx_dequant(oc, os_).reshape(E, N, K)
    got = O.bf16_to_f64(bits(M.dequant_mxfp4(p)))
    np.testing.assert_array_equal(got, val)
    assert (np.signbit(got) == np.signbit(val)).all()


def test_quant_pack_fp32_rounds_once():
    rng = np.random.default_rng(4)
    E, N, K = 2, 96, 256
    v = np.stack([_special(N, K, rng) for _ in range(E)]).astype(np.float32)
    # just beside ties that a bf16 copy would land on
    v[0, 6, :32] = np.float32(2.5) * np.where(np.arange(32) % 2, 1 + 2.0 ** -20, 1 - 2.0 ** -20)
    v[0, 6, 0] = 6.0
    v[0, 7, :32] = np.float32(1.0)
    v[0, 7, 0] = np.nextafter(np.float32(8.0), np.float32(0))        # the exponent from all 24 bits
    got = O.bf16_to_f64(bits(M.dequant_mxfp4(M.quant_pack_mxfp4(to_dev(v)))))
    f = v.astype(np.float64).reshape(E, N, K // 32, 32)
    amax = np.abs(f).max(-1)
    code = np.where(amax > 0, np.clip(np.frexp(amax)[1].astype(np.int64) - 3, -127, 127) + 127, 0)
    y = f / X.e8m0_to_f64(code)[..., None]
    ref = X.e2m1_to_f64(X.f64_to_e2m1(y, np.signbit(f))) * X.e8m0_to_f64(code)[..., None]
    np.testing.assert_array_equal(got, ref.reshape(E, N, K))


def test_dequant_covers_every_scale_code():
    codes = np.tile(np.arange(256, dtype=np.uint8), (1, 16, 256 * 16 // 256))[:, :, :256 * 16]     # K = 8192
    scales = np.tile(np.arange(256, dtype=np.uint8), (1, 16, 1))
    got = M.dequant_mxfp4(M.pack_mxfp4(to_dev(codes), to_dev(scales))).float().cpu().numpy()
    with np.errstate(over="ignore", invalid="ignore"):
        ref = X.mx_dequant(X.unpack_nibbles(codes), scales)
        ref = np.where(np.abs(ref) >= 2.0 ** 128, np.sign(ref) * np.inf, ref)
    np.testing.assert_array_equal(got.astype(np.float64)[..., :255 * 32], ref[..., :255 * 32])
    assert np.isnan(got[..., 255 * 32:]).all()


def test_quant_pack_refusals():
    with pytest.raises(TypeError):
        M.quant_pack_mxfp4(torch.zeros(1, 16, 128, dtype=torch.float16, device=dev()))
    with pytest.raises(ValueError):
        M.quant_pack_mxfp4(torch.zeros(16, 128, device=dev()))
    with pytest.raises(ValueError):
        M.quant_pack_mxfp4(torch.zeros(1, 128, 16, device=dev()).transpose(1, 2))
    with pytest.raises(M.W4A16Error):
        M.quant_pack_mxfp4(torch.zeros(1, 16, 96, device=dev()))         # K % 128
    with pytest.raises(ValueError):
        M.dequant_mxfp4(M.pack_w4(torch.zeros(1, 16, 128, dtype=torch.uint8, device=dev()),
                                  torch.zeros(1, 16, 4, dtype=torch.bfloat16, device=dev())))


@pytest.mark.parametrize("kind,E,N,K", [("int4", 9, 65536, 65536), ("mxfp4", 33, 65536, 65536)])
def test_packing_past_one_grid(kind, E, N, K):
    """More words than the threads of one launch can be (2^32): every expert is packed as it is by itself."""
    if torch.cuda.mem_get_info()[0] < 200 * 2**30:
        pytest.skip("needs 200 GiB of free GPU memory")
    g = torch.Generator(device=dev()).manual_seed(E)
    codes = torch.randint(0, 256, (1, N, K // 2), generator=g, dtype=torch.uint8, device=dev())
    if kind == "int4":
        one = torch.cat((codes & 15, codes >> 4), dim=2)
        scales = torch.randn(1, N, K // 32, generator=g, device=dev()).to(torch.bfloat16)
        pack = M.pack_w4
    else:
        one, pack = codes, M.pack_mxfp4
        scales = torch.randint(100, 140, (1, N, K // 32), generator=g, dtype=torch.uint8, device=dev())
    ref = pack(one, scales)
    many = one.new_empty(E, *one.shape[1:])
    many[:] = one
    p = pack(many, scales.expand(E, -1, -1).contiguous())
    del many
    for e in range(E):
        assert torch.equal(p.w.view(E, -1)[e], ref.w), e
        assert torch.equal(p.s.view(E, -1)[e], ref.s), e
    del p, ref, one, codes, scales
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ grouped MXFP4

def _mx_weight(E, N, K, seed, gate_up=False):
    rng = np.random.default_rng(seed)
    c = rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
    s = rng.integers(119, 124, (E, N, K // 32), dtype=np.uint8)
    return M.pack_mxfp4(to_dev(c), to_dev(s), gate_up=gate_up), X.mx_dequant(X.unpack_nibbles(c), s)


def _mx_rows(m, K, seed):
    rng = np.random.default_rng(seed)
    c = rng.integers(0, 256, (m, K // 2), dtype=np.uint8)
    s = rng.integers(124, 129, (m, K // 32), dtype=np.uint8)
    return c, s, X.mx_dequant(X.unpack_nibbles(c), s)


def _grouped_check(got, rows, experts, a, w, what):
    """Rows of `rows` against a . w[expert]; every other row still holds the sentinel."""
    touched = np.zeros(len(got), bool)
    worst = 0.0
    for e in sorted(set(experts)):
        r = np.array([i for i, x in zip(rows, experts) if x == e])
        touched[r] = True
        ref, tol = LO.product(a[r], w[e])
        worst = max(worst, LO.assert_within(got[r], ref, tol, f"{what} expert {e}"))
    assert (got[~touched] == 0x4000).all(), f"{what}: wrote rows that hold nothing"
    log(f"grouped {what}: {worst:.2f} of the bound")


CONTIGUOUS = [((1,), 1, 16, 128), ((128, 0, 5), 4, 208, 256), ((129, 300, 0, 17, 64), 5, 1040, 640),
              ((40, 256, 384), 3, 512, 384), ((1000,), 1, 768, 1152),
              # 256-row blocks: odd and even numbers of 128-row blocks, halves that end early
              ((700, 130, 257, 128), 4, 272, 512), ((1500,), 1, 96, 1024), ((256, 0, 385, 640, 1, 900), 6, 528, 512)]


@pytest.mark.parametrize("counts,E,N,K", CONTIGUOUS)
@pytest.mark.parametrize("gate_up", [False, True])
def test_grouped_contiguous(counts, E, N, K, gate_up):
    if gate_up and N % 64:
        N = (N + 63) // 64 * 64
    packed, w = _mx_weight(E, N, K, N + K, gate_up)
    idx = []
    for e, n in enumerate(counts):
        idx += [e] * n + [-1] * (-n % 128)
    idx += [-1] * 128                                     # an over-allocated tail
    c, s, a = _mx_rows(len(idx), K, 3)
    pad = np.array(idx) < 0
    s[pad] = 255                                          # NaN rows in the padding
    out = torch.full((len(idx) + 2, N), 2.0, dtype=torch.bfloat16, device=dev())
    M.grouped_mxfp4_contiguous(M.MXRows(to_dev(c), to_dev(s)), packed, to_dev(np.array(idx, np.int32)), out=out)
    live = [i for i, e in enumerate(idx) if e >= 0]
    _grouped_check(bits(out), live, [idx[i] for i in live], a, w, f"contiguous {counts} N={N} K={K}")


def test_grouped_contiguous_experts_out_of_order_and_foreign_ids():
    packed, w = _mx_weight(4, 96, 256, 9)
    idx = [3] * 100 + [-1] * 28 + [0] * 128 + [0] * 2 + [-1] * 126 + [7] * 128 + [-5] * 128 + [1] * 1 + [-1] * 127
    c, s, a = _mx_rows(len(idx), 256, 4)
    out = torch.full((len(idx), 96), 2.0, dtype=torch.bfloat16, device=dev())
    M.grouped_mxfp4_contiguous(M.MXRows(to_dev(c), to_dev(s)), packed, to_dev(np.array(idx, np.int32)), out=out)
    live = [i for i, e in enumerate(idx) if 0 <= e < 4]
    _grouped_check(bits(out), live, [idx[i] for i in live], a, w, "out of order")


MASKED = [((1,), 1, 1, 1, 16, 128), ((0, 3, 16), 16, 5, 3, 208, 256), ((17, 0, 40, 33), 40, 20, 4, 1040, 640),
          ((128, 1, 70), 130, 60, 3, 512, 384), ((500, 130, 0), 512, 200, 3, 272, 1152), ((9, 200, 1), 200, 4, 3, 64, 256)]


@pytest.mark.parametrize("counts,max_m,expected,E,N,K", MASKED)
def test_grouped_masked(counts, max_m, expected, E, N, K):
    packed, w = _mx_weight(E, N, K, N + K + 1)
    c, s, a = _mx_rows(E * max_m, K, 6)
    live = [(g * max_m + r, g) for g, n in enumerate(counts) for r in range(n)]
    dead = np.ones(E * max_m, bool)
    dead[[i for i, _ in live]] = False
    s[dead] = 255
    out = torch.full((E * max_m + 1, N), 2.0, dtype=torch.bfloat16, device=dev())
    M.grouped_mxfp4_masked(M.MXRows(to_dev(c), to_dev(s)), packed, to_dev(np.array(counts, np.int32)), expected, out=out)
    _grouped_check(bits(out), [i for i, _ in live], [g for _, g in live], a, w, f"masked {counts} N={N} K={K}")


def test_grouped_contiguous_long_runs_and_split_segments():
    """More than 512 blocks of one expert in a row, then two segments of one
    expert next to each other, the first ending inside a block."""
    packed, w = _mx_weight(2, 32, 512, 12)
    idx = [0] * (128 * 515 + 5) + [-1] * 123 + [1] * 130 + [-1] * 126 + [1] * 200 + [-1] * 56 + [1] * 3 + [-1] * 125
    c, s, a = _mx_rows(len(idx), 512, 4)
    out = torch.full((len(idx), 32), 2.0, dtype=torch.bfloat16, device=dev())
    M.grouped_mxfp4_contiguous(M.MXRows(to_dev(c), to_dev(s)), packed, to_dev(np.array(idx, np.int32)), out=out)
    live = [i for i, e in enumerate(idx) if e >= 0]
    touched = np.array(idx) >= 0
    got = bits(out)
    assert (got[~touched] == 0x4000).all()
    for e in (0, 1):
        r = np.nonzero(np.array(idx) == e)[0]
        ref, tol = LO.product(a[r], w[e])
        LO.assert_within(got[r], ref, tol, f"expert {e}")
    assert len(live) == int(touched.sum())


@pytest.mark.parametrize("K", [128, 256, 384, 512, 640, 1024])
@pytest.mark.parametrize("N", [272, 512])
def test_grouped_every_tile_count_and_pipeline_length(K, N):
    """One to eight token tiles a block (built: 1, 2, 4, 6, 8), both ends of each; one to eight K chunks, row scales
    fetched a chunk or four chunks at a time; a column tile that ends inside a workgroup's."""
    packed, w = _mx_weight(4, N, K, N + K)
    counts = [n for t in range(1, 9) for n in (16 * t - 15, 16 * t)]
    idx = []
    for i, n in enumerate(counts):
        idx += [i % 4] * n + [-1] * (128 - n)
    c, s, a = _mx_rows(len(idx), K, 3)
    s[np.array(idx) < 0] = 255
    live = [i for i, e in enumerate(idx) if e >= 0]
    codes = to_dev(c)
    for at in (0, 4):                                      # K = 512, 1024: scales on 16 bytes or not
        buf = torch.empty(s.size + at, dtype=torch.uint8, device=dev())
        rows = M.MXRows(codes, buf[at:].view(s.shape).copy_(to_dev(s)))
        out = torch.full((len(idx), N), 2.0, dtype=torch.bfloat16, device=dev())
        M.grouped_mxfp4_contiguous(rows, packed, to_dev(np.array(idx, np.int32)), out=out)
        _grouped_check(bits(out), live, [idx[i] for i in live], a, w, f"contiguous tiles N={N} K={K} at {at}")
        # the same rows as groups of 512: whole blocks, then one that ends early
        for first in range(0, 4):
            cnt = [(128 * (g + first)) % 512 + counts[4 * g + first] for g in range(4)]
            out.fill_(2.0)
            M.grouped_mxfp4_masked(rows, packed, to_dev(np.array(cnt, np.int32)), 100, out=out)
            sel = [(g * 512 + r, g) for g in range(4) for r in range(cnt[g])]
            good = [(r, g) for r, g in sel if idx[r] >= 0]  # the others are NaN rows here, and come out as NaN
            got = bits(out)
            bad = np.array([r for r, _ in sel if idx[r] < 0], np.int64)
            assert np.isnan(O.bf16_to_f64(got[bad])).all()
            got[bad] = 0x4000
            _grouped_check(got, [r for r, _ in good], [g for _, g in good], a, w, f"masked tiles N={N} K={K} at {at}")


def test_grouped_masked_clamps_counts():
    packed, w = _mx_weight(3, 64, 128, 2)
    c, s, a = _mx_rows(3 * 20, 128, 6)
    out = torch.full((60, 64), 2.0, dtype=torch.bfloat16, device=dev())
    M.grouped_mxfp4_masked(M.MXRows(to_dev(c), to_dev(s)), packed, to_dev(np.array([-4, 99, 2], np.int32)), 8, out=out)
    rows = list(range(20, 40)) + [40, 41]
    _grouped_check(bits(out), rows, [1] * 20 + [2] * 2, a, w, "clamped")


def test_grouped_mxfp4_scales_on_four_bytes():
    """K a multiple of 512 with scales that lie on 4 bytes but not on 16: the same bits."""
    packed, _ = _mx_weight(2, 64, 1024, 2)
    c, s, _ = _mx_rows(256, 1024, 6)
    codes, idx = to_dev(c), to_dev(np.repeat(np.array([0, 1], np.int32), 128))
    buf = torch.empty(s.size + 4, dtype=torch.uint8, device=dev())
    moved = buf[4:].view(256, 32).copy_(to_dev(s))
    assert moved.data_ptr() % 16 == 4
    ref = M.grouped_mxfp4_contiguous(M.MXRows(codes, to_dev(s)), packed, idx)
    assert torch.equal(M.grouped_mxfp4_contiguous(M.MXRows(codes, moved), packed, idx), ref)
    counts = torch.tensor([128, 77], dtype=torch.int32, device=dev())
    ref = M.grouped_mxfp4_masked(M.MXRows(codes, to_dev(s)), packed, counts, 100)
    assert torch.equal(M.grouped_mxfp4_masked(M.MXRows(codes, moved), packed, counts, 100), ref)


def test_grouped_mxfp4_refusals_and_empty():
    packed, _ = _mx_weight(2, 64, 128, 2)
    c, s, _ = _mx_rows(256, 128, 6)
    rows = M.MXRows(to_dev(c), to_dev(s))
    idx = torch.zeros(256, dtype=torch.int32, device=dev())
    with pytest.raises(ValueError):
        M.grouped_mxfp4_contiguous(rows, packed, idx[:128])
    with pytest.raises(ValueError):
        M.grouped_mxfp4_contiguous(M.MXRows(rows.codes, rows.scales[:, :2].contiguous()), packed, idx)
    with pytest.raises(ValueError):
        M.grouped_mxfp4_masked(rows, packed, idx[:3], 8)
    with pytest.raises(ValueError):
        M.grouped_mxfp4_masked(M.MXRows(rows.codes[:255], rows.scales[:255]), packed, idx[:2], 8)
    with pytest.raises(M.W4A16Error):
        M.grouped_mxfp4_masked(rows, packed, idx[:2], 0)
    with pytest.raises(M.W4A16Error):
        M.grouped_mxfp4_contiguous(M.MXRows(rows.codes[:64], rows.scales[:64]), packed, idx[:64])
    e = M.grouped_mxfp4_contiguous(M.MXRows(rows.codes[:0], rows.scales[:0]), packed, idx[:0])
    assert e.shape == (0, 64)


def test_quantised_layer_over_the_contiguous_layout_matches_the_indexed_calls():
    """A layer as a user runs it: weights quantised and packed from bf16,
    logits routed, rows laid out by expert, both projections grouped; against
    the indexed A4W4 calls on the same routing."""
    T, k, E, H, I = 150, 2, 4, 256, 128
    g = torch.Generator().manual_seed(2)
    w1 = (0.05 * torch.randn(E, 2 * I, H, generator=g)).to(torch.bfloat16).to(dev())
    w2 = (0.05 * torch.randn(E, H, I, generator=g)).to(torch.bfloat16).to(dev())
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).to(dev())
    p1, p2 = M.quant_pack_mxfp4(w1), M.quant_pack_mxfp4(w2)
    ids, wt = M.moe_route(torch.randn(T, E, generator=g).to(dev()), k)
    flat = ids.cpu().numpy().reshape(-1)
    rows, idx = [], []
    for e in range(E):
        sl = np.nonzero(flat == e)[0]
        rows += sl.tolist() + [0] * (-len(sl) % 128)
        idx += [e] * len(sl) + [-1] * (-len(sl) % 128)
    rows_d, idx_d = to_dev(np.array(rows)), to_dev(np.array(idx, np.int32))
    h = M.grouped_mxfp4_contiguous(M.mxfp4_quant(x[rows_d // k]), p1, idx_d)
    r = M.moe_align(ids, E, 0, E, 64)
    hi = M.moe_mxfp4_gemm(M.mxfp4_quant(x), p1, r)
    live = idx_d >= 0
    assert torch.equal(h[live], hi[rows_d[live]])          # one summation order whatever the tile
    act = (torch.nn.functional.silu(h[:, :I].float()) * h[:, I:].float()).to(torch.bfloat16)
    z = M.grouped_mxfp4_contiguous(M.mxfp4_quant(act.contiguous()), p2, idx_d)
    slot = torch.zeros(T * k, H, device=dev())
    slot[rows_d[live]] = z[live].float()
    y = (slot.view(T, k, H) * wt[..., None]).sum(1)
    acti = torch.zeros(T * k, I, dtype=torch.bfloat16, device=dev())
    acti[rows_d[live]] = act[live]
    ref = M.moe_mxfp4_gemm(M.mxfp4_quant(acti), p2, r, wt).float()
    # here each expert's row is rounded to bf16 before the sum, there the sum is rounded once
    tol = 2.0 ** -8 * ((slot.abs().view(T, k, H) * wt[..., None]).sum(1) + 2 * ref.abs())
    assert ((y - ref).abs() <= tol).all()


def test_grouped_mxfp4_captured_and_replayed():
    packed, _ = _mx_weight(3, 320, 512, 5)
    c, s, _ = _mx_rows(384, 512, 6)
    rows = M.MXRows(to_dev(c), to_dev(s))
    idx = to_dev(np.array([1] * 100 + [-1] * 28 + [0] * 128 + [2] * 3 + [-1] * 125, np.int32))
    cnt = to_dev(np.array([5, 128, 0], np.int32))
    x = torch.randn(384, 512, dtype=torch.bfloat16, device=dev())

    def step():
        M.mxfp4_quant(x, out=rows)
        return M.grouped_mxfp4_contiguous(rows, packed, idx), M.grouped_mxfp4_masked(rows, packed, cnt, 40)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for rep in range(4):
        x.normal_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        ref = step()
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1]), rep
        _ = (x.float() @ x.float().t()).sum().item()
