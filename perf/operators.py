"""Measured cases of the router, the few-token MoE layer, the MXFP4 weight
quantiser and the grouped MXFP4 products.

Each operator has a plain form (elementary torch operations in 32 bits; 64
bits where an order between values decides) and the framework's call; `exact`
evaluates the definition in 64 bits.

  route    logits [T, E] -> expert ids and weights of the top k
  few      x [T, H] through the experts its tokens chose: gate/up, SiLU * up,
           down, weighted sum; INT4 weights with bf16 group-32 scales, or MXFP4
  quant    weight [E, N, K] -> MXFP4 and back to the values it stands for
  grouped  MXFP4 rows x MXFP4 weights, experts' rows back to back
           ("contiguous", segments start at multiples of 128 rows) or a fixed
           row budget per expert ("masked")
"""
import math
import random

import torch

own = False

GROUP = 32
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding user: 384 experts, top 8, sigmoid scores with a selection bias
        dict(name="route_one_token", op="route", T=1, E=384, k=8, scoring="sigmoid", bias=True, renorm=True,
             dtype="float32", masked=False),
        # an odd prefill chunk of the 16-of-896 routing, bf16 logits, some experts masked and some rows empty
        dict(name="route_wide_masked", op="route", T=4097, E=896, k=16, scoring="softmax", bias=False, renorm=True,
             dtype="bfloat16", masked=True),
        # a long prefill of the 8-of-384 routing
        dict(name="route_prefill", op="route", T=16384, E=384, k=8, scoring="sigmoid", bias=True, renorm=True,
             dtype="float32", masked=False),
        # one token on a tensor-parallel eighth of the layer (latency counts)
        dict(name="few_int4_slice_one", op="few", kind="int4", T=1, k=8, E=384, first=0, El=384, H=7168, I=256),
        # a decode batch on one expert-parallel eighth
        dict(name="few_int4_share", op="few", kind="int4", T=16, k=8, E=384, first=0, El=48, H=7168, I=2048),
        # an odd batch on a share of the 16-of-896 routing, MXFP4 weights
        dict(name="few_mxfp4_share", op="few", kind="mxfp4", T=37, k=16, E=896, first=112, El=112, H=7168, I=2048),
        # a small layer whose widths end inside a 128-wide chunk
        dict(name="few_int4_odd", op="few", kind="int4", T=7, k=3, E=12, first=0, El=12, H=1120, I=352),
        # one projection of a tensor-parallel slice, fp32 master weights
        dict(name="quant_slice", op="quant", E=3, N=512, K=7168, dtype="float32"),
        # a whole expert-parallel gate/up weight, bf16
        dict(name="quant_share", op="quant", E=48, N=4096, K=7168, dtype="bfloat16"),
        # decode on the masked layout: about 12 rows an expert, two experts idle
        dict(name="grouped_masked_decode", op="grouped", layout="masked", E=48, N=4096, K=7168, rows=576,
             max_m=64, empty=2),
        # prefill on the contiguous layout, gate/up of an expert-parallel eighth, uneven experts
        dict(name="grouped_contiguous_prefill", op="grouped", layout="contiguous", E=48, N=4096, K=7168, rows=16384,
             max_m=0, empty=4),
        # a few ragged segments on a narrow weight
        dict(name="grouped_contiguous_odd", op="grouped", layout="contiguous", E=5, N=1040, K=640, rows=301,
             max_m=0, empty=1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("route", "few", "quant", "grouped"))
    if op == "route":
        E = rng.randint(8, 1024)
        sig = rng.random() < 0.5
        return dict(op=op, T=_log_int(rng, 1, 16384), E=E, k=rng.randint(1, min(E, 32)),
                    scoring="sigmoid" if sig else "softmax", bias=sig and rng.random() < 0.7,
                    renorm=rng.random() < 0.7, dtype=rng.choice(("float32", "bfloat16", "float16")),
                    masked=rng.random() < 0.5)
    if op == "few":
        kind = rng.choice(("int4", "mxfp4"))
        unit = 32 if kind == "int4" else 128
        E = rng.randint(8, 448)
        El = rng.randint(1, min(E, 48))
        k = rng.randint(1, min(E, 16))
        return dict(op=op, kind=kind, T=_log_int(rng, 1, 64), k=k, E=E, first=rng.randint(0, E - El), El=El,
                    H=unit * _log_int(rng, 512 // unit, 7168 // unit),
                    I=unit * _log_int(rng, 128 // unit, 2048 // unit))
    if op == "quant":
        return dict(op=op, E=_log_int(rng, 1, 48), N=16 * _log_int(rng, 1, 256), K=128 * _log_int(rng, 1, 56),
                    dtype=rng.choice(("bfloat16", "float32")))
    E = _log_int(rng, 1, 48)
    layout = rng.choice(("contiguous", "masked"))
    max_m = _log_int(rng, 1, 512) if layout == "masked" else 0
    empty = rng.randint(0, E // 4)
    cap = max_m * (E - empty) if layout == "masked" else 16384
    return dict(op=op, layout=layout, E=E, N=16 * _log_int(rng, 4, 256), K=128 * _log_int(rng, 2, 56),
                rows=_log_int(rng, 1, min(cap, 16384)), max_m=max_m, empty=empty)


def work(case):
    op = case["op"]
    if op == "route":
        size = 4 if case["dtype"] == "float32" else 2
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * size + (4 * E if case["bias"] else 0) + 8 * T * k, "flops": 4 * T * E}
    if op == "few":
        T, k, E, El, H, I = (case[n] for n in ("T", "k", "E", "El", "H", "I"))
        touched = El * (1.0 - (1.0 - k / E) ** T)            # experts expected to hold a slot
        slots = T * k * El / E
        per = 0.5 + (2.0 if case["kind"] == "int4" else 1.0) / GROUP
        return {"bytes": touched * 3 * H * I * per + 4 * T * H + 8 * T * k, "flops": 6 * slots * H * I}
    if op == "quant":
        n = case["E"] * case["N"] * case["K"]
        return {"bytes": n * ((4 if case["dtype"] == "float32" else 2) + 2), "flops": 2 * n}
    E, N, K, rows = (case[n] for n in ("E", "N", "K", "rows"))
    live = min(E - case["empty"], rows)
    per = 0.5 + 1.0 / GROUP
    return {"bytes": (live * N + rows) * K * per + 2 * rows * N, "flops": 2 * rows * N * K}


# ------------------------------------------------------------------ inputs

def _counts(case, seed):
    """Rows of each expert: `rows` in all, `empty` experts without any, no more than max_m each."""
    rnd = random.Random(seed * 7919 + case["rows"])
    live = rnd.sample(range(case["E"]), case["E"] - case["empty"])
    cap = case["max_m"] or case["rows"]
    counts = [0] * case["E"]
    for e in live[:case["rows"]]:
        counts[e] = 1
    share = {e: rnd.uniform(0.3, 1.7) for e in live}
    left = case["rows"] - sum(counts)
    while left:
        free = [e for e in live if counts[e] < cap]
        for e in rnd.choices(free, [share[e] for e in free], k=left):
            if counts[e] < cap:
                counts[e] += 1
                left -= 1
    return counts


def prepare(case, seed):
    return _inputs(case, seed, own)


def _inputs(case, seed, packed):
    """What the program holds: with `packed` its weights are laid out by the framework, else as given."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    op = case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def bytes_(high, *shape, low=0):
        return torch.randint(low, high, shape, generator=gen, device=dev, dtype=torch.uint8)

    st = dict(case)
    if op == "route":
        T, E = case["T"], case["E"]
        logits = normal(T, E)
        if case["masked"]:
            logits[torch.rand(T, E, generator=gen, device=dev) < 0.02] = -math.inf
            logits[torch.rand(T, generator=gen, device=dev) < 0.06] = -math.inf
        st["logits"] = logits.to(getattr(torch, case["dtype"]))
        st["b"] = 0.1 * normal(E) if case["bias"] else None
        st["scale"] = 2.5
        return st
    if op == "few":
        T, k, E, El, H, I = (case[n] for n in ("T", "k", "E", "El", "H", "I"))
        st["x"] = normal(T, H).to(torch.bfloat16)
        st["ids"] = torch.rand(T, E, generator=gen, device=dev).topk(k, dim=1).indices.to(torch.int32).contiguous()
        st["w"] = torch.softmax(normal(T, k), dim=1)
        if case["kind"] == "int4":
            raw = [bytes_(16, El, n, kk) for n, kk in ((2 * I, H), (H, I))]
            scl = [(0.005 + 0.015 * torch.rand(El, n, kk // GROUP, generator=gen, device=dev)).to(torch.bfloat16)
                   for n, kk in ((2 * I, H), (H, I))]
        else:
            raw = [bytes_(256, El, n, kk // 2) for n, kk in ((2 * I, H), (H, I))]
            scl = [bytes_(123, El, n, kk // GROUP, low=120) for n, kk in ((2 * I, H), (H, I))]
        if packed:
            import w4a16_int4_mixture_moe_amd as M
            pack = M.pack_w4 if case["kind"] == "int4" else M.pack_mxfp4
            st["p1"], st["p2"] = pack(raw[0], scl[0], gate_up=True), pack(raw[1], scl[1])
        else:
            st["raw"], st["scl"] = raw, scl
        return st
    if op == "quant":
        shape = (case["E"], case["N"], case["K"])
        w = torch.empty(shape, device=dev, dtype=getattr(torch, case["dtype"]))
        for e in range(case["E"]):                       # trained weights: near normal, blocks of unequal size
            w[e] = 0.02 * normal(*shape[1:]) * torch.exp(normal(shape[1], 1))
        st["weight"] = w
        return st
    E, N, K = case["E"], case["N"], case["K"]
    counts = _counts(case, seed)
    if case["layout"] == "contiguous":
        starts, ids = [], []
        for e, c in enumerate(counts):
            starts.append(len(ids))
            ids += [e] * c + [-1] * (-c % 128)
        # the buffer is as long as any split of the rows over the experts needs
        m = 128 * (case["rows"] // 128 + E - case["empty"])
        ids += [-1] * (m - len(ids))
        st["index"] = torch.tensor(ids, dtype=torch.int32, device=dev)
    else:
        m = E * case["max_m"]
        starts = [e * case["max_m"] for e in range(E)]
        st["index"] = torch.tensor(counts, dtype=torch.int32, device=dev)
    st["counts"], st["starts"] = counts, starts
    # activations as the row quantiser leaves them: N(0, 1) rows, codes of the block's scale
    codes, scales = _quantise(normal(m, K).to(torch.bfloat16).float())
    st["a"] = (codes[:, 0::2] | (codes[:, 1::2] << 4), scales)
    weight = bytes_(256, E, N, K // 2)
    wscale = bytes_(123, E, N, K // GROUP, low=120)
    if packed:
        import w4a16_int4_mixture_moe_amd as M
        st["packed"] = M.pack_mxfp4(weight, wscale)
        st["rows_mx"] = M.MXRows(*(t.contiguous() for t in st["a"]))
        st["expected"] = max(1, -(-case["rows"] // E))
    else:
        st["weight"], st["wscale"] = weight, wscale
    st["out"] = torch.zeros(m, N, dtype=torch.bfloat16, device=dev)
    return st


# ------------------------------------------------------------- plain forms

def _pow2(n):
    """2^n in fp32 for whole n of -149..127."""
    table = torch.tensor([2.0 ** i for i in range(-149, 128)], device=n.device)
    return table[n.long() + 149]


def _quantise(v):
    """fp32 [.., K] -> E2M1 codes (one a byte) and E8M0 scale codes of the blocks of 32."""
    blocks = v.unflatten(-1, (-1, GROUP))
    exponent = torch.frexp(blocks.abs().amax(-1)).exponent.to(torch.int32) - 1
    code = torch.where(blocks.abs().amax(-1) > 0, (exponent + 125).clamp(0, 254), 0)
    y = blocks * _pow2(127 - code).unsqueeze(-1)
    a = y.abs()
    q = torch.zeros_like(a, dtype=torch.uint8)
    for t in (0.25, 1.25, 2.5, 5.0):
        q += (a > t).to(torch.uint8)                     # a tie goes to the even code below
    for t in (0.75, 1.75, 3.5):
        q += (a >= t).to(torch.uint8)                    # ... or above
    q |= (torch.signbit(y).to(torch.uint8) << 3)
    return q.flatten(-2), code.to(torch.uint8)


def _fp4_values(codes, scales):
    """Byte pairs [.., K/2] and scale codes [.., K/32] -> values [.., K]."""
    table = torch.tensor(E2M1, device=codes.device)
    v = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), dim=-1).flatten(-2)
    return (v.unflatten(-1, (-1, GROUP)) * _pow2(scales.to(torch.int32) - 127).unsqueeze(-1)).flatten(-2)


def _int4_values(codes, scales):
    """Codes [.., K] and bf16 scales [.., K/32] -> the bf16 weights they stand for, in fp32."""
    v = (codes.float() - 8.0).unflatten(-1, (-1, GROUP)) * scales.float().unsqueeze(-1)
    return v.flatten(-2).to(torch.bfloat16).float()


def _plain_route(st):
    x = st["logits"].double()
    live = ~(torch.isnan(x) | (x == -math.inf))
    if st["scoring"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-x))
    else:
        score = torch.exp(x - torch.where(live, x, -math.inf).amax(1, keepdim=True).clamp_min(-3e38))
        score = torch.where(live, score, 0.0)
    key = (score + st["b"].double() if st["b"] is not None else score) if st["scoring"] == "sigmoid" else x
    key = torch.where(live, key, -math.inf)
    order = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :st["k"]]
    ok = live.gather(1, order)
    w = torch.where(ok, score.gather(1, order), 0.0)
    if st["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    elif st["scoring"] == "softmax":
        w = w / (score.sum(1, keepdim=True) + 1e-20)
    return torch.where(ok, order, -1).to(torch.int32), (w * st["scale"]).float()


def _plain_few(st):
    values = _int4_values if st["kind"] == "int4" else _fp4_values
    x = st["x"].float()
    T, I = x.shape[0], st["I"]
    y = torch.zeros_like(x)
    for e in range(st["El"]):
        w = torch.where(st["ids"] == st["first"] + e, st["w"], 0.0).sum(1, keepdim=True)
        gu = x @ values(st["raw"][0][e], st["scl"][0][e]).t()
        g, u = gu[:, :I], gu[:, I:]
        h = g / (1.0 + torch.exp(-g)) * u
        y += w * (h @ values(st["raw"][1][e], st["scl"][1][e]).t())
    return y.to(torch.bfloat16)


def _plain_quant(st):
    out = torch.empty(st["weight"].shape, dtype=torch.bfloat16, device=st["weight"].device)
    for e in range(st["E"]):
        codes, scales = _quantise(st["weight"][e].float())
        out[e] = _fp4_values(codes[:, 0::2] | (codes[:, 1::2] << 4), scales).to(torch.bfloat16)
    return out


def _plain_grouped(st):
    out = st["out"]
    a = _fp4_values(*st["a"])
    for e, (n, r) in enumerate(zip(st["counts"], st["starts"])):
        if n:
            out[r:r + n] = (a[r:r + n] @ _fp4_values(st["weight"][e], st["wscale"][e]).t()).to(torch.bfloat16)
    return out


# --------------------------------------------------------------- operators

def run(state):
    op = state["op"]
    if not own:
        return {"route": _plain_route, "few": _plain_few, "quant": _plain_quant, "grouped": _plain_grouped}[op](state)
    import w4a16_int4_mixture_moe_amd as M
    if op == "route":
        return M.moe_route(state["logits"], state["k"], scoring=state["scoring"], bias=state["b"],
                           renormalize=state["renorm"], scale=state["scale"])
    if op == "few":
        return M.moe_few_tokens(state["x"], state["p1"], state["p2"], state["ids"], state["w"],
                                first_expert=state["first"])
    if op == "quant":
        return M.dequant_mxfp4(M.quant_pack_mxfp4(state["weight"]))
    if state["layout"] == "contiguous":
        return M.grouped_mxfp4_contiguous(state["rows_mx"], state["packed"], state["index"], out=state["out"])
    return M.grouped_mxfp4_masked(state["rows_mx"], state["packed"], state["index"], state["expected"],
                                  out=state["out"])


# ------------------------------------------------------------------- exact

def exact(case, seed):
    st = _inputs(case, seed, False)
    f64 = torch.float64

    def two(n):                                          # 2^n, put together from its bits
        return ((n.to(torch.int64) + 1023) << 52).view(f64)

    def fp4(codes, scales):                              # sign, exponent and mantissa of each nibble
        n = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).to(f64)
        sign = 1.0 - 2.0 * (n >= 8)
        n = n % 8
        ex, man = torch.floor(n / 2), n % 2
        mag = torch.where(ex == 0, 0.5 * man, (1.0 + 0.5 * man) * two(ex - 1))
        return sign * mag * two(scales.to(torch.int64) - 127).repeat_interleave(GROUP, dim=-1)

    op = case["op"]
    if op == "route":
        rows = st["logits"].to(f64)
        masked = (rows == -math.inf) | rows.isnan()
        score = torch.sigmoid(rows) if case["scoring"] == "sigmoid" else torch.softmax(rows, dim=1)
        key = rows if case["scoring"] == "softmax" else score + (st["b"].to(f64) if case["bias"] else 0.0)
        key = key.masked_fill(masked, -math.inf)
        # the k largest one after another, the lowest index of equals
        picks, weights = [], []
        cols = torch.arange(case["E"], device=rows.device)
        for _ in range(case["k"]):
            top = key.amax(1, keepdim=True)
            i = torch.where(key == top, cols, case["E"]).amin(1)
            gone = top.squeeze(1) == -math.inf
            picks.append(torch.where(gone, -1, i))
            weights.append(score.gather(1, i.unsqueeze(1)).squeeze(1).masked_fill(gone, 0.0))
            key.scatter_(1, i.unsqueeze(1), -math.inf)
        w = torch.stack(weights, 1)
        if case["renorm"]:
            w = w / (w.sum(1, keepdim=True) + 1e-20)
        return torch.stack(picks, 1).to(torch.int32), w * st["scale"]
    if op == "few":
        y = torch.zeros(case["T"], case["H"], dtype=f64, device=st["x"].device)
        for e in range(case["El"]):
            hit = (st["ids"] == case["first"] + e)
            if not bool(hit.any()):
                continue
            t, j = hit.nonzero(as_tuple=True)
            if case["kind"] == "int4":
                w1, w2 = (((c[e].to(f64) - 8.0) * s[e].to(f64).repeat_interleave(GROUP, dim=-1))
                          .to(torch.bfloat16).to(f64) for c, s in zip(st["raw"], st["scl"]))
            else:
                w1, w2 = (fp4(c[e], s[e]) for c, s in zip(st["raw"], st["scl"]))
            g, u = (st["x"][t].to(f64) @ w1.t()).chunk(2, dim=1)
            y.index_add_(0, t, st["w"][t, j].to(f64).unsqueeze(1) * ((g * torch.sigmoid(g) * u) @ w2.t()))
        return y
    if op == "quant":
        out = torch.empty(st["weight"].shape, dtype=f64, device=st["weight"].device)
        for e in range(case["E"]):
            v = st["weight"][e].to(f64).view(case["N"], -1, GROUP)
            top = v.abs().amax(-1, keepdim=True)
            ex = ((top.view(torch.int64) >> 52) - 1025).clamp_min(-127)   # floor(log2 top) - 2
            y = v * two(-ex)
            step = torch.where(y.abs() < 2.0, 0.5, torch.where(y.abs() < 4.0, 1.0, 2.0))
            out[e] = ((torch.round(y / step) * step).clamp(-6.0, 6.0) * two(ex)).view(case["N"], case["K"])
        return out
    out = torch.zeros(st["out"].shape, dtype=f64, device=st["out"].device)
    rows = fp4(*st["a"])
    for e in range(case["E"]):
        n, r = st["counts"][e], st["starts"][e]
        if n:
            out[r:r + n] = rows[r:r + n] @ fp4(st["weight"][e], st["wscale"][e]).t()
    return out
