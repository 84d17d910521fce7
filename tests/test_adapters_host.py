"""Host-side checks (no GPU needed) of the group-limited router and of the
INT4 products with low-rank adapters: their oracle against independent
evaluations, and the refusal of bad arguments before anything is enqueued."""
import ctypes

import numpy as np
import pytest
import torch

import w4a16_int4_mixture_moe_amd as W
from oracle import adapter_oracle as AO
from w4a16_int4_mixture_moe_amd import _lib

P = 4096          # a pointer that is never followed: every call below is refused, or has nothing to do


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(W.lib_path()):
        pytest.skip("library not built")
    return W.load()


# ------------------------------------------------------------------ oracle

@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_grouped_oracle_against_torch_float64(scoring, renorm):
    g = torch.Generator().manual_seed(3)
    T, E, G, keep, k = 29, 60, 6, 2, 5
    l = torch.randn(T, E, generator=g, dtype=torch.float64)
    b = 0.2 * torch.randn(E, generator=g, dtype=torch.float64) if scoring == "sigmoid" else None
    ids, w, _ = AO.route_grouped(l.numpy(), k, G, keep, scoring, None if b is None else b.numpy(), renorm, 1.5)
    s = torch.softmax(l, 1) if scoring == "softmax" else torch.sigmoid(l)
    c = (s if b is None else s + b).view(T, G, E // G)
    score = c.amax(2) if scoring == "softmax" else c.topk(2, 2).values.sum(2)
    mask = torch.zeros(T, G, dtype=torch.bool).scatter_(1, score.topk(keep, 1).indices, True)
    i = c.masked_fill(~mask.unsqueeze(2), -9.0).view(T, E).topk(k, 1).indices
    v = s.gather(1, i)
    if renorm:
        v = v / v.sum(1, keepdim=True)
    np.testing.assert_array_equal(ids, i.numpy())
    np.testing.assert_allclose(w, 1.5 * v.numpy(), rtol=1e-12)


def test_route_grouped_oracle_masks_and_ties():
    n, inf = np.nan, np.inf
    l = np.array([[0.0, 0.0, 0.0, 0.0, 0.0, 0.0],              # all groups equal: the lower ones
                  [-inf, n, -inf, 5.0, 1.0, 1.0],              # a dead group, one with a single live expert
                  [-inf, -inf, -inf, n, -inf, -inf],           # nothing
                  [-inf, -inf, -inf, -inf, -inf, 1.0]])        # one expert in all
    ids, w, _ = AO.route_grouped(l, 3, 3, 2, "sigmoid")
    # row 1: sigmoid(5) alone against 2 sigmoid(1): both groups stay
    assert ids.tolist() == [[0, 1, 2], [3, 4, 5], [-1, -1, -1], [5, -1, -1]]
    assert (w[2] == 0).all()
    ids, _, _ = AO.route_grouped(l, 2, 3, 1, "sigmoid")
    assert ids.tolist() == [[0, 1], [4, 5], [-1, -1], [5, -1]]
    ids, _, _ = AO.route_grouped(l, 2, 3, 1, "softmax")
    assert ids.tolist() == [[0, 1], [3, -1], [-1, -1], [5, -1]]


def test_adapter_oracle_against_torch_float64():
    g = torch.Generator().manual_seed(5)
    M, K, N, r, La = 7, 64, 32, 8, 3
    x = torch.randn(M, K, generator=g).to(torch.bfloat16)
    codes = torch.randint(0, 16, (N, K), generator=g, dtype=torch.uint8)
    sc = (0.01 * torch.rand(N, K // 32, generator=g)).to(torch.bfloat16)
    w = AO.int4_values(codes, sc)
    assert float(w[3, 40]) == float(((codes[3, 40].float() - 8) * sc[3, 1].float()).to(torch.bfloat16))
    a = torch.randn(La, 2 * r, K, generator=g).to(torch.bfloat16)
    b = torch.randn(La, N, r, generator=g).to(torch.bfloat16)
    s = torch.rand(La, generator=g)
    ids = torch.tensor([0, -1, 2, 7, 1, 1, 0])
    y, _ = AO.linear(x, w, ids, (a, b, s), slices=2)
    for t in range(M):
        l = int(ids[t])
        ref = w @ x[t].double()
        if 0 <= l < La:
            low = torch.zeros(N, K, dtype=torch.float64)
            low[:N // 2] = b[l, :N // 2].double() @ a[l, :r].double()
            low[N // 2:] = b[l, N // 2:].double() @ a[l, r:].double()
            ref = ref + float(s[l]) * (low @ x[t].double())
        torch.testing.assert_close(y[t], ref, rtol=1e-12, atol=1e-12)
    z, _ = AO.linear(x, w, ids, (a, b, s), slices=2, silu=True)
    torch.testing.assert_close(z, torch.nn.functional.silu(y[:, :N // 2]) * y[:, N // 2:], rtol=1e-12, atol=1e-12)


# ---------------------------------------------------------------- refusals

def _route(L, logits=P, dtype=_lib.DTYPE_F32, T=2, E=64, stride=64, bias=None, groups=8, keep=4, k=8, scoring=0, renorm=1,
           scale=1.0, ids=P, w=P):
    return L.w4a16_moe_route_grouped(logits, dtype, T, E, stride, bias, groups, keep, k, scoring, renorm, scale, ids, w,
                                     None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -1), (dict(E=0), -1), (dict(groups=0), -1), (dict(groups=-8), -1), (dict(groups=7), -1),
    (dict(groups=128, E=128, stride=128), -2), (dict(keep=0), -1), (dict(keep=9), -1), (dict(keep=-1), -1),
    (dict(k=0), -1), (dict(k=33), -1), (dict(keep=1, k=9), -1), (dict(E=2048, stride=2048), -2),
    (dict(E=1024, stride=1024, k=33), -2), (dict(dtype=3), -4), (dict(scoring=2), -4), (dict(bias=P), -4),
    (dict(scale=float("nan")), -1), (dict(stride=63), -1), (dict(stride=(1 << 26) + 1), -2), (dict(logits=None), -1),
    (dict(ids=None), -1), (dict(w=None), -1), (dict(logits=P + 2), -1), (dict(ids=P + 2), -1), (dict(w=P + 1), -1),
])
def test_route_grouped_refuses(L, kw, code):
    assert _route(L, **kw) == code
    assert L.w4a16_last_error()
    assert _route(L, T=0) == 0


def _adapters(La=4, E=1, N=64, K=256, rank=16, slices=1, a=P, b=P, scale=P, ids=P):
    return _lib.AdaptersC(a, b, scale, ids, La, E, N, K, rank, slices)


BAD_ADAPTERS = [
    (dict(La=0), -1), (dict(La=1025), -2), (dict(rank=0), -1), (dict(rank=12), -2), (dict(rank=264), -2),
    (dict(slices=0), -1), (dict(slices=3), -1), (dict(N=80), -2), (dict(K=128), -2), (dict(E=2), -2), (dict(a=None), -1),
    (dict(b=None), -1), (dict(ids=None), -1), (dict(a=P + 8), -1), (dict(b=P + 8), -1), (dict(scale=P + 2), -1),
    (dict(ids=P + 1), -1),
]


def _linear(L, desc=None, pw=P, ps=P, x=P, T=3, ad=None, silu=0, out=P, ws=P, wb=1 << 40):
    d = W.weight_desc(1, 64, 256) if desc is None else desc
    return L.w4a16_linear(ctypes.byref(d), pw, ps, x, T, None if ad is None else ctypes.byref(ad), silu, out, ws, wb, None)


@pytest.mark.parametrize("kw,code", BAD_ADAPTERS)
def test_linear_refuses_bad_adapters(L, kw, code):
    assert _linear(L, ad=_adapters(**kw)) == code
    assert L.w4a16_last_error()
    d = W.weight_desc(1, 64, 256)
    assert L.w4a16_linear_workspace_bytes(ctypes.byref(d), 3, ctypes.byref(_adapters(**kw))) == 0


def test_linear_refuses(L):
    assert _linear(L, T=-1) == -1
    assert _linear(L, desc=W.weight_desc(2, 64, 256)) == -3
    assert _linear(L, desc=W.mxfp4_weight_desc(1, 64, 256)) == -3
    assert _linear(L, silu=1) == -3                                       # not gate/up packed
    for kw in (dict(pw=None), dict(ps=None), dict(x=None), dict(out=None), dict(pw=P + 8), dict(x=P + 4), dict(out=P + 2)):
        assert _linear(L, **kw) == -1, kw
    assert _linear(L, desc=W.weight_desc(1, 64, 1 << 20), T=1 << 12) == -2     # 8 GiB of rows
    d = W.weight_desc(1, 80, 256)                                         # 80 columns have no two halves of 16-column tiles
    assert _linear(L, desc=d, ad=_adapters(N=80, slices=2)) == -2
    ad = _adapters()
    d = W.weight_desc(1, 64, 256)
    need = L.w4a16_linear_workspace_bytes(ctypes.byref(d), 3, ctypes.byref(ad))
    assert need >= 3 * 16 * 4
    assert _linear(L, ad=ad, ws=None) == -8 and _linear(L, ad=ad, wb=need - 1) == -8
    assert _linear(L, ad=ad, ws=P + 8) == -8
    assert _linear(L, ws=None) == -8 and _linear(L, wb=3 * 64 * 4 - 1) == -8
    assert _linear(L, T=0, x=None, out=None, ws=None, wb=0) == 0
    assert _linear(L, ad=ad, T=0, x=None, out=None, ws=None, wb=0) == 0
    assert L.w4a16_linear_workspace_bytes(ctypes.byref(d), 3, None) >= 3 * 64 * 4         # slices of K


@pytest.mark.parametrize("T,K,N,rank,planes,packed", [
    (520, 1120, 2560, 128, 4, True), (511, 1120, 2560, 128, 4, False), (520, 992, 2560, 128, 4, True),
    (520, 896, 2560, 128, 3, False),                                      # 7 chunks of 128, two a plane at least
    (64, 3232, 96, 64, 8, None), (65, 3232, 96, 64, 4, None), (64, 3200 // 4, 96, 64, 3, None)])
def test_linear_workspace_holds_the_planes_and_a_packed_copy(L, T, K, N, rank, planes, packed):
    d = W.weight_desc(1, N, K)
    al = lambda n: (n + 255) // 256 * 256
    need = L.w4a16_linear_workspace_bytes(ctypes.byref(d), T, ctypes.byref(_adapters(N=N, K=K, rank=rank, slices=2)))
    bare = L.w4a16_linear_workspace_bytes(ctypes.byref(d), T, None)       # slices of K
    want = al(planes * T * 2 * rank * 4) + al(4 * T) + (al(T * 2 * -(-rank // 16) * 64) if packed else 0)
    assert need - bare == want
    assert (bare == 0) == (packed is not None)


def _routing(T=3, topk=2, E=4, block_m=16, **kw):
    f = dict(sorted_ids=P, expert_ids=P, num_tokens_padded=P, capacity=W.align_capacity(T, topk, E, block_m),
             block_m=block_m, T=T, topk=topk, topk_ids=P, first_expert=0, E_loc=E, E_glob=E)
    f.update(kw)
    return _lib.IndexedRouting(**f)


def _gemm(L, desc=None, a=P, a_rows=1 << 20, layout=0, r=None, ad=None, w=None, out=P, cfg=None, ws=P, wb=1 << 40):
    d = W.weight_desc(4, 64, 256) if desc is None else desc
    r = _routing() if r is None else r
    return L.w4a16_moe_adapter_gemm(ctypes.byref(d), P, P, a, a_rows, layout, ctypes.byref(r),
                                    ctypes.byref(_adapters(E=4) if ad is None else ad), w, out,
                                    None if cfg is None else ctypes.byref(cfg), ws, wb, None)


def _silu(L, desc=None, x=P, x_rows=1 << 20, r=None, ad=None, out=P, cfg=None, ws=P, wb=1 << 40):
    d = W.weight_desc(4, 64, 256, gate_up=True) if desc is None else desc
    r = _routing() if r is None else r
    return L.w4a16_moe_adapter_gate_up_silu(ctypes.byref(d), P, P, x, x_rows, ctypes.byref(r),
                                            ctypes.byref(_adapters(E=4) if ad is None else ad), out,
                                            None if cfg is None else ctypes.byref(cfg), ws, wb, None)


@pytest.mark.parametrize("kw,code", BAD_ADAPTERS)
def test_routed_calls_refuse_bad_adapters(L, kw, code):
    kw = dict(dict(E=4), **kw)
    assert _gemm(L, ad=_adapters(**kw)) == code
    assert _silu(L, ad=_adapters(**kw)) == code
    d = W.weight_desc(4, 64, 256)
    assert L.w4a16_moe_adapter_workspace_bytes(ctypes.byref(d), ctypes.byref(_routing()), ctypes.byref(_adapters(**kw)), 0,
                                               None) == 0


def test_routed_calls_refuse(L):
    assert _gemm(L, a=None) == -1 and _gemm(L, out=P + 8) == -1 and _gemm(L, layout=3) == -1
    assert _gemm(L, a_rows=2) == -2 and _silu(L, x_rows=2) == -2
    assert _gemm(L, r=_routing(E_loc=3)) == -3 and _silu(L, r=_routing(E_loc=3)) == -3
    assert _silu(L, desc=W.weight_desc(4, 64, 256)) == -3                 # not gate/up packed
    assert _gemm(L, desc=W.weight_desc(4, 64, 256, gate_up=True), w=P) == -3
    assert _gemm(L, desc=W.mxfp4_weight_desc(4, 64, 256)) == -3
    assert _gemm(L, w=P, r=_routing(topk_ids=None)) == -1
    for call in (_gemm, _silu):
        assert call(L, cfg=W.config(16, 2, split_k=2)) == -4
        assert call(L, cfg=W.config(16, 2, split_k=0)) == -4
        assert call(L, cfg=W.config(16, 2, stages=4)) == -4              # built without adapters only
        assert call(L, cfg=W.config(32, 2)) == -3                        # not a divisor of the routing's rows
        assert call(L, cfg=W.config(16, 2, kind="masked")) == -1
        assert call(L, ws=None) == -8 and call(L, wb=15) == -8
        assert call(L, r=_routing(T=0, topk_ids=None), ws=None, wb=0) == 0
    d = W.weight_desc(4, 64, 256)
    need = [L.w4a16_moe_adapter_workspace_bytes(ctypes.byref(d), ctypes.byref(_routing()), ctypes.byref(_adapters(E=4)), c,
                                                None) for c in (0, 1)]
    assert need[0] >= 6 * 16 * 4 and need[1] >= need[0] + 6 * 64 * 4
    assert _gemm(L, w=P, wb=need[1] - 1) == -8


def test_structs_match_the_header(tmp_path):
    import os
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    fields = [f for f, _ in _lib.AdaptersC._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "w4a16_moe.h"\nint main(void) {\n'
                   + "".join(f'printf("%zu\\n", offsetof(w4a16_adapters, {f}));\n' for f in fields)
                   + 'printf("%zu\\n", sizeof(w4a16_adapters));\nreturn 0;\n}\n')
    exe = tmp_path / "layout"
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)],
                   check=True, capture_output=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [getattr(_lib.AdaptersC, f).offset for f in fields] + [ctypes.sizeof(_lib.AdaptersC)]


def test_binding_refuses_on_the_host():
    x = torch.zeros(3, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        W.adapters(x, x)                                                  # not on a GPU
    with pytest.raises(TypeError):
        W.adapters([1], x)
    with pytest.raises(ValueError):
        W.moe_route_grouped(torch.zeros(2, 8), 2, 2, 1)
