"""Host-side checks (no GPU needed) of the router, the few-token layer, the
MXFP4 weight quantiser and the grouped MXFP4 products: their oracle against
independent evaluations, and the refusal of bad arguments before anything is
enqueued."""
import ctypes

import numpy as np
import pytest
import torch

import w4a16_int4_mixture_moe_amd as W
from oracle import layer_oracle as LO
from w4a16_int4_mixture_moe_amd import _lib

P = 4096          # a pointer that is never followed: every call below is refused, or has nothing to do


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(W.lib_path()):
        pytest.skip("library not built")
    return W.load()


# ------------------------------------------------------------------ oracle

@pytest.mark.parametrize("renorm", [True, False])
def test_route_oracle_against_torch_float64(renorm):
    g = torch.Generator().manual_seed(3)
    l = torch.randn(37, 50, generator=g, dtype=torch.float64)
    ids, w, _ = LO.route(l.numpy(), 6, "softmax", renormalize=renorm, scale=1.5)
    p = torch.softmax(l, 1)
    v, i = p.topk(6, 1)
    if renorm:
        v = v / v.sum(1, keepdim=True)
    np.testing.assert_array_equal(ids, i.numpy())
    np.testing.assert_allclose(w, 1.5 * v.numpy(), rtol=1e-12)
    b = torch.randn(50, generator=g, dtype=torch.float64) * 0.2
    ids, w, _ = LO.route(l.numpy(), 6, "sigmoid", b.numpy(), renorm)
    s = torch.sigmoid(l)
    i = (s + b).topk(6, 1).indices
    v = s.gather(1, i)
    if renorm:
        v = v / v.sum(1, keepdim=True)
    np.testing.assert_array_equal(ids, i.numpy())
    np.testing.assert_allclose(w, v.numpy(), rtol=1e-12)


def test_route_oracle_masks_and_ties():
    n, inf = np.nan, np.inf
    l = np.array([[1.0, 2.0, 2.0, -inf], [-inf, n, -inf, -inf], [inf, 0.0, inf, n], [-0.0, 0.0, -inf, 0.0]])
    ids, w, _ = LO.route(l, 3, "softmax")
    assert ids.tolist() == [[1, 2, 0], [-1, -1, -1], [0, 2, 1], [0, 1, 3]]
    assert (w[1] == 0).all() and w[2].tolist() == [0.5, 0.5, 0.0] and np.allclose(w[3], 1 / 3)
    ids, _, _ = LO.route(np.zeros((1, 4)), 2, "sigmoid", np.array([-inf, 0.0, n, 0.5]))
    assert ids.tolist() == [[3, 1]]


def test_few_tokens_oracle_against_torch_float64():
    g = torch.Generator().manual_seed(5)
    T, k, E, H, I = 4, 3, 5, 32, 64
    x = torch.randn(T, H, generator=g).to(torch.bfloat16)
    w1 = torch.randn(E, 2 * I, H, generator=g, dtype=torch.float64)
    w2 = torch.randn(E, H, I, generator=g, dtype=torch.float64)
    ids = torch.tensor([[0, 3, 4], [7, 2, -1], [1, 1, 2], [9, 8, 0]], dtype=torch.int32)      # first = 1: 1..5 are local
    wt = torch.rand(T, k, generator=g)
    y, _ = LO.few_tokens(x.view(torch.int16).numpy().view(np.uint16), w1.numpy(), w2.numpy(), ids.numpy(), wt.numpy(), 1)
    ref = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j]) - 1
            if 0 <= e < E:
                gate, up = (w1[e] @ x[t].double()).chunk(2)
                ref[t] += wt[t, j].double() * (w2[e] @ (torch.nn.functional.silu(gate) * up))
    np.testing.assert_allclose(y, ref.numpy(), rtol=1e-11, atol=1e-11)
    assert not y[3].any()


# ---------------------------------------------------------------- refusals

def test_route_refusals(L):
    def call(logits=P, dtype=0, T=4, E=64, stride=64, bias=None, k=8, scoring=0, renorm=1, scale=1.0, ids=P, w=P):
        return L.w4a16_moe_route(logits, dtype, T, E, stride, bias, k, scoring, renorm, scale, ids, w, None)
    assert call(T=0, logits=None, ids=None, w=None) == 0                 # nothing to do
    assert call(T=-1) == -1 and call(E=0) == -1 and call(k=0) == -1
    assert call(k=65) == -1                                              # more than E
    assert call(k=33) == -2 and call(E=1025, stride=1025) == -2          # past the built sizes
    assert call(dtype=3) == -4 and call(scoring=2) == -4
    assert call(bias=P) == -4                                            # a bias with softmax
    assert call(scale=float("nan")) == -1 and call(scale=float("inf")) == -1
    assert call(stride=63) == -1 and call(stride=(1 << 26) + 1) == -2
    assert call(logits=None) == -1 and call(ids=None) == -1 and call(w=None) == -1
    assert call(logits=P + 2) == -1 and call(ids=P + 1) == -1            # not aligned to the element
    assert call(logits=P + 1, dtype=1) == -1
    assert b"aligned" in L.w4a16_last_error()


def _pair(E=4, H=256, I=128, mx=False):
    if mx:
        return W.mxfp4_weight_desc(E, 2 * I, H, gate_up=True), W.mxfp4_weight_desc(E, H, I)
    return W.weight_desc(E, 2 * I, H, gate_up=True), W.weight_desc(E, H, I)


@pytest.mark.parametrize("mx", [False, True])
def test_few_tokens_refusals(L, mx):
    g, d = _pair(mx=mx)
    need = L.w4a16_moe_few_tokens_workspace_bytes(ctypes.byref(g), 4, 8)
    assert need >= 4 * 8 * (128 * 2 + 16 * 8 + 4) and need % 256 == 0

    def call(g=g, d=d, w1=P, x=P, T=4, k=8, ids=P, w=P, first=0, out=P, ws=P, wsb=need):
        return L.w4a16_moe_few_tokens(ctypes.byref(g), w1, P, ctypes.byref(d), P, P, x, T, k, ids, w, first, out, ws,
                                      wsb, None)
    assert call(T=0, x=None, ids=None, w=None, out=None, ws=None, wsb=0) == 0
    assert call(wsb=need - 1) == -8 and call(ws=None) == -8 and call(ws=P + 8) == -8
    assert call(T=-1) == -1 and call(k=0) == -1 and call(first=-1) == -1 and call(first=2 ** 30 + 1) == -1
    assert call(T=65, k=1) == -2 and call(T=64, k=17) == -2 and call(T=1, k=1025) == -2
    assert call(x=None) == -1 and call(ids=None) == -1 and call(w=None) == -1 and call(out=None) == -1
    assert call(w1=None) == -1 and call(x=P + 8) == -1 and call(ids=P + 2) == -1
    plain = W.mxfp4_weight_desc(4, 256, 256) if mx else W.weight_desc(4, 256, 256)
    assert call(g=plain) == -3                                           # not gate/up packed
    assert call(d=g) == -3                                               # down packed as gate/up
    assert call(d=_pair(mx=not mx)[1]) == -3                             # two formats
    assert call(d=_pair(E=5, mx=mx)[1]) == -2                            # another expert count
    assert call(d=_pair(H=128, mx=mx)[1]) == -2 and call(d=_pair(I=256, mx=mx)[1]) == -2
    bad = W.weight_desc(4, 256, 256)
    bad.N = 128
    assert call(g=bad) == -3
    f = L.w4a16_moe_few_tokens_workspace_bytes
    assert f(ctypes.byref(g), 0, 8) == 0 and f(ctypes.byref(g), 65, 1) == 0 and f(ctypes.byref(g), 64, 17) == 0


def test_quant_pack_and_dequant_refusals(L):
    d = W.mxfp4_weight_desc(2, 32, 128)
    q = lambda w=P, dt=1, d=d, pw=P, ps=P: L.w4a16_mxfp4_quant_pack(w, dt, ctypes.byref(d), pw, ps, None)
    assert q(dt=2) == -4                                                 # fp16 weights are not taken
    assert q(w=None) == -1 and q(pw=None) == -1 and q(w=P + 2) == -1 and q(ps=P + 4) == -1
    assert q(d=W.weight_desc(2, 32, 128)) == -3
    u = lambda d=d, pw=P, out=P: L.w4a16_mxfp4_dequant(ctypes.byref(d), pw, P, out, None)
    assert u(d=W.weight_desc(2, 32, 128)) == -3 and u(out=None) == -1 and u(out=P + 2) == -1 and u(pw=None) == -1


def test_grouped_mxfp4_refusals(L):
    d = W.mxfp4_weight_desc(4, 64, 256)
    c = lambda d=d, a=P, s=P, m=256, idx=P, out=P: L.w4a16_mxfp4_grouped_contiguous(
        ctypes.byref(d), P, P, a, s, m, idx, out, None)
    assert c(m=0, a=None, s=None, idx=None, out=None) == 0
    assert c(m=-128) == -1 and c(m=64) == -2                             # segments start at multiples of 128
    assert c(a=None) == -1 and c(s=None) == -1 and c(idx=None) == -1 and c(out=None) == -1
    assert c(a=P + 8) == -1 and c(out=P + 8) == -1 and c(s=P + 2) == -1
    assert c(d=W.weight_desc(4, 64, 256)) == -3
    assert c(m=1 << 25) == -2                                            # 4 GiB of codes
    m = lambda d=d, a=P, mm=P, max_m=32, exp=8, out=P: L.w4a16_mxfp4_grouped_masked(
        ctypes.byref(d), P, P, a, P, max_m, mm, exp, out, None)
    assert m(max_m=0) == -1 and m(exp=0) == -1 and m(a=None) == -1 and m(mm=None) == -1 and m(out=None) == -1
    assert m(d=W.weight_desc(4, 64, 256)) == -3
    assert m(max_m=1 << 23) == -2 and m(max_m=1 << 29) == -2


def test_grouped_mxfp4_refuses_grids_past_32_bits(L):
    """2^24 tiles are 2^32 threads, a launch that would wrap to no workgroup at all."""
    for E, N in ((1 << 24, 16), (1 << 22, 1024), ((1 << 23) + 1, 272)):
        d = W.mxfp4_weight_desc(E, N, 128)
        assert L.w4a16_mxfp4_grouped_masked(ctypes.byref(d), P, P, P, P, 1, P, 1, P, None) == -2
    d = W.mxfp4_weight_desc(1, 1 << 18, 128)                             # 2^10 tiles a block
    assert L.w4a16_mxfp4_grouped_contiguous(ctypes.byref(d), P, P, P, P, 128 << 14, P, P, None) == -2


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="GPU"):
        W.moe_route(x, 2)
    with pytest.raises(ValueError, match="GPU"):
        W.quant_pack_mxfp4(torch.zeros(1, 16, 128))
    with pytest.raises(TypeError):
        W.moe_route(x.numpy(), 2)


def test_few_tokens_first_expert_limit(L):
    """The header's limit, the library's and the binding's are one number."""
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "w4a16_moe.h")).read()
    shift = int(re.search(r"#define W4A16_FEW_MAX_FIRST_EXPERT \(1 << (\d+)\)", src).group(1))
    assert _lib.FEW_MAX_FIRST_EXPERT == 1 << shift
    g, d = _pair()
    for first, status in ((1 << shift, 0), ((1 << shift) + 1, -1), (2**31 - 1, -1)):
        assert L.w4a16_moe_few_tokens(ctypes.byref(g), P, P, ctypes.byref(d), P, P, None, 0, 8, None, None, first, None,
                                      None, 0, None) == status


@pytest.mark.parametrize("make", [W.weight_desc, W.mxfp4_weight_desc])
def test_binding_refuses_sizes_past_32_bits(L, make):
    """Cut to 32 bits these would be the small weight [1, 64, 128]."""
    big = 2**32
    for E, N, K in ((big + 1, 64, 128), (1, big + 64, 128), (1, 64, big + 128), (1 - big, 64, 128)):
        with pytest.raises(ValueError, match="32-bit"):
            make(E, N, K)
    g = make(1, 128, 128, gate_up=True)
    p = W.PackedW4(g, None, None)
    assert W.few_tokens_workspace_bytes(p, 4, 2) > 0
    for T, k in ((big + 4, 2), (4, big + 2), (4 - big, 2), (-1, 2), (4, -1)):
        assert W.few_tokens_workspace_bytes(p, T, k) == 0


def test_header_constants_match_the_binding(tmp_path):
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "w4a16_moe.h")).read()
    for name, val in (("DTYPE_F32", _lib.DTYPE_F32), ("DTYPE_BF16", _lib.DTYPE_BF16), ("DTYPE_F16", _lib.DTYPE_F16),
                      ("SCORE_SOFTMAX", _lib.SCORE_SOFTMAX), ("SCORE_SIGMOID", _lib.SCORE_SIGMOID)):
        assert int(re.search(rf"#define W4A16_{name} (\d+)", src).group(1)) == val


@pytest.mark.parametrize("mx", [False, True])
def test_layer_widths_are_whole_pairs_of_tiles(L, mx):
    """The down kernel of wide layers takes two 16-column tiles a workgroup: H, the gate/up weight's K, is a multiple of 32."""
    make = W.mxfp4_weight_desc if mx else W.weight_desc
    for H in (16, 48, 6160, 7184):
        with pytest.raises(W.W4A16Error):
            make(1, 128, H, gate_up=True)
