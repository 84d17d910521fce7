"""Measured cases of the group-limited router and of low-rank adapters beside
INT4 projections: a shared one and the routed experts'.

Each operator has a plain form (elementary torch operations in 32 bits; 64
bits where an order between values decides) and the framework's call; `exact`
evaluates the definition in 64 bits.

  route    logits [T, E] -> the best groups of consecutive experts, then expert
           ids and weights of the top k inside them
  shared   x [T, K] times one INT4 weight [N, K], plus s_a B_a (A_a x_t) of the
           adapter a that the token's request uses (none where a is -1);
           optionally SiLU(gate) * up of the two halves
  experts  x [T, H] through the INT4 experts its tokens chose, the request's
           adapter of that expert beside both projections: gate/up, SiLU * up,
           down, weighted sum
"""
import math

import torch

own = False

GROUP = 32


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding user: 384 experts in 8 groups, the best 4 kept, sigmoid scores with a selection bias
        dict(name="route_one_token", op="route", T=1, E=384, k=8, groups=8, keep=4, scoring="sigmoid", bias=True,
             renorm=True, dtype="float32", masked=False),
        # an odd prefill chunk, 16 of 896 bf16 logits, groups scored by their maximum, experts masked, rows empty
        dict(name="route_wide_masked", op="route", T=4097, E=896, k=16, groups=14, keep=5, scoring="softmax",
             bias=False, renorm=False, dtype="bfloat16", masked=True),
        # a long prefill of the first routing
        dict(name="route_prefill", op="route", T=16384, E=384, k=8, groups=8, keep=4, scoring="sigmoid", bias=True,
             renorm=True, dtype="float32", masked=False),
        # one token through a tensor-parallel eighth of the shared gate/up (latency counts)
        dict(name="shared_slice_one", op="shared", T=1, K=7168, N=512, silu=True, L=16, r=16, requests=1),
        # a decode batch, every token another request, on the whole shared gate/up
        dict(name="shared_decode", op="shared", T=64, K=7168, N=4096, silu=True, L=32, r=16, requests=64),
        # a large decode batch through the shared down projection
        dict(name="shared_down_batch", op="shared", T=301, K=2048, N=7168, silu=False, L=64, r=32, requests=301),
        # widths that end inside a 128-wide chunk, a rank below the matrix instruction's depth
        dict(name="shared_odd", op="shared", T=37, K=1120, N=1040, silu=False, L=3, r=8, requests=5),
        # prefill of a few dozen requests on the whole shared gate/up, a large rank
        dict(name="shared_prefill", op="shared", T=8192, K=7168, N=4096, silu=True, L=16, r=64, requests=24),
        # one token on a tensor-parallel eighth of the layer
        dict(name="experts_slice_one", op="experts", T=1, k=8, E=384, first=0, El=384, H=7168, I=256, L=2, r=16,
             requests=1),
        # a decode batch on one expert-parallel eighth
        dict(name="experts_decode_share", op="experts", T=32, k=8, E=384, first=48, El=48, H=7168, I=2048, L=8, r=16,
             requests=32),
        # a small layer with ragged widths and a rank that is no power of two
        dict(name="experts_odd", op="experts", T=61, k=3, E=12, first=2, El=7, H=1120, I=352, L=5, r=24, requests=9),
        # prefill of a few requests on one expert-parallel eighth
        dict(name="experts_prefill_share", op="experts", T=4096, k=8, E=384, first=0, El=48, H=7168, I=2048, L=4,
             r=16, requests=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("route", "shared", "experts"))
    if op == "route":
        groups = rng.randint(1, 32)
        size = rng.randint(1, 1024 // groups)
        keep = rng.randint(1, groups)
        sig = rng.random() < 0.5
        return dict(op=op, T=_log_int(rng, 1, 16384), E=groups * size, k=rng.randint(1, min(keep * size, 32)),
                    groups=groups, keep=keep, scoring="sigmoid" if sig else "softmax",
                    bias=sig and rng.random() < 0.7, renorm=rng.random() < 0.7,
                    dtype=rng.choice(("float32", "bfloat16", "float16")), masked=rng.random() < 0.5)
    if op == "shared":
        T = _log_int(rng, 1, 8192)
        silu = rng.random() < 0.5
        return dict(op=op, T=T, K=32 * _log_int(rng, 4, 224), N=32 * _log_int(rng, 2, 128), silu=silu,
                    L=_log_int(rng, 1, 64), r=8 * _log_int(rng, 1, 8), requests=rng.choice((T, _log_int(rng, 1, T))))
    T = _log_int(rng, 1, 4096)
    E = rng.randint(4, 384)
    El = rng.randint(1, min(E, 48))
    return dict(op=op, T=T, k=rng.randint(1, min(E, 8)), E=E, first=rng.randint(0, E - El), El=El,
                H=32 * _log_int(rng, 8, 224), I=32 * _log_int(rng, 2, 64), L=_log_int(rng, 1, 4),
                r=8 * _log_int(rng, 1, 2), requests=rng.choice((T, _log_int(rng, 1, T))))


def work(case):
    op, T = case["op"], case["T"]
    if op == "route":
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": T * case["E"] * size + (4 * case["E"] if case["bias"] else 0) + 8 * T * case["k"],
                "flops": 4 * T * case["E"]}
    L, r = case["L"], case["r"]
    per = 0.5 + 2.0 / GROUP
    used = L * (1.0 - (1.0 - 1.0 / (L + 1)) ** case["requests"])          # adapters expected in use, of L + 1 choices
    adapted = T * L / (L + 1.0)
    if op == "shared":
        N, K, halves = case["N"], case["K"], 2 if case["silu"] else 1
        return {"bytes": N * K * per + 2 * used * r * (halves * K + N) + 2 * T * (K + N // halves) + 4 * T,
                "flops": 2 * T * N * K + 2 * adapted * r * (halves * K + N)}
    k, E, El, H, I = (case[n] for n in ("k", "E", "El", "H", "I"))
    slots = T * k * El / E
    touched = El * (1.0 - (1.0 - k / E) ** T)
    pairs = El * used * (1.0 - (1.0 - k / E) ** (T / (L + 1.0)))          # (expert, adapter) with a token
    return {"bytes": touched * 3 * H * I * per + 2 * pairs * r * (3 * H + 3 * I) + 4 * T * H + 8 * T * k + 4 * T,
            "flops": 6 * slots * H * I + 2 * slots * L / (L + 1.0) * r * (3 * H + 3 * I)}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    return _inputs(case, seed, own)


def _inputs(case, seed, packed):
    """What the program holds: with `packed` its weights are laid out by the framework, else as given."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    op, T = case["op"], case["T"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=dev)

    def int4(e, n, k):
        return (torch.randint(0, 16, (e, n, k), generator=gen, device=dev, dtype=torch.uint8),
                (0.005 + 0.015 * uniform(e, n, k // GROUP)).to(torch.bfloat16))

    def adapter(lead, halves, r, k, n):
        # A as it is initialised (its product with a normal row is near normal), B as training leaves it: the
        # adapter moves a projection by about a fifth
        a = torch.empty(*lead, halves * r, k, device=dev, dtype=torch.bfloat16)
        b = torch.empty(*lead, n, r, device=dev, dtype=torch.bfloat16)
        for i in range(lead[0]):
            a[i] = normal(*a.shape[1:]) / math.sqrt(k)
            b[i] = normal(*b.shape[1:]) / math.sqrt(r)
        return a, b, 0.5 + uniform(lead[0])

    st = dict(case)
    if op == "route":
        E = case["E"]
        logits = normal(T, E)
        if case["masked"]:
            logits[uniform(T, E) < 0.02] = -math.inf
            logits[uniform(T) < 0.06] = -math.inf
        st["logits"] = logits.to(getattr(torch, case["dtype"]))
        st["b"] = 0.1 * normal(E) if case["bias"] else None
        st["scale"] = 2.5
        return st
    L, r, R = case["L"], case["r"], case["requests"]
    # consecutive tokens of a request share its adapter; one request in L + 1 has none
    of_request = torch.randint(-1, L, (R,), generator=gen, device=dev, dtype=torch.int32)
    if R == T:
        st["adapter_ids"] = of_request
    else:
        starts = torch.zeros(T, device=dev, dtype=torch.int64)
        starts[uniform(T).topk(R - 1).indices if R > 1 else torch.zeros(0, device=dev, dtype=torch.int64)] = 1
        starts[0] = 0
        st["adapter_ids"] = of_request[starts.cumsum(0)]
    if op == "shared":
        K, N = case["K"], case["N"]
        st["x"] = normal(T, K).to(torch.bfloat16)
        codes, scales = int4(1, N, K)
        a, b, s = adapter((L,), 2 if case["silu"] else 1, r, K, N)
        if packed:
            import w4a16_int4_mixture_moe_amd as M
            st["packed"] = M.pack_w4(codes, scales, gate_up=case["silu"])
            st["adapters"] = M.adapters(a, b, s)
        else:
            st["weight"], st["low"] = (codes, scales), (a, b, s)
        return st
    k, E, El, H, I = (case[n] for n in ("k", "E", "El", "H", "I"))
    st["x"] = normal(T, H).to(torch.bfloat16)
    st["ids"] = uniform(T, E).topk(k, dim=1).indices.to(torch.int32).contiguous()
    st["w"] = torch.softmax(normal(T, k), dim=1)
    up, down = int4(El, 2 * I, H), int4(El, H, I)
    low1, low2 = adapter((L, El), 2, r, H, 2 * I), adapter((L, El), 1, r, I, H)
    if packed:
        import w4a16_int4_mixture_moe_amd as M
        st["p1"], st["p2"] = M.pack_w4(*up, gate_up=True), M.pack_w4(*down)
        st["a1"], st["a2"] = M.adapters(*low1), M.adapters(*low2)
        st["block_m"] = M.select(T, k, E, El, 2 * I, H).block_m
    else:
        st["weight"], st["low"] = (up, down), (low1, low2)
    return st


# ------------------------------------------------------------- plain forms

def _int4_values(codes, scales):
    """Codes [.., K] and bf16 scales [.., K/32] -> the bf16 weights they stand for, in fp32."""
    v = (codes.float() - 8.0).unflatten(-1, (-1, GROUP)) * scales.float().unsqueeze(-1)
    return v.flatten(-2).to(torch.bfloat16).float()


def _plain_route(st):
    T, E, G = st["T"], st["E"], st["groups"]
    x = st["logits"].double()
    live = ~(torch.isnan(x) | (x == -math.inf))
    if st["scoring"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-x))
        key = score + st["b"].double() if st["b"] is not None else score
    else:
        score = torch.exp(x - torch.where(live, x, -math.inf).amax(1, keepdim=True).clamp_min(-3e38))
        score = torch.where(live, score, 0.0)
        key = x
    key = torch.where(live, key, -math.inf)
    best = torch.sort(key.view(T, G, E // G), dim=2, descending=True).values
    of_group = best[:, :, 0]
    if st["scoring"] == "sigmoid" and E // G > 1:
        of_group = of_group + torch.where(best[:, :, 1] > -math.inf, best[:, :, 1], 0.0)
    groups = torch.sort(of_group, dim=1, descending=True, stable=True).indices[:, :st["keep"]]
    kept = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, groups, True)
    live_in = live & kept.repeat_interleave(E // G, dim=1)
    key = torch.where(live_in, key, -math.inf)
    order = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :st["k"]]
    ok = live_in.gather(1, order)
    w = torch.where(ok, score.gather(1, order), 0.0)
    if st["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    elif st["scoring"] == "softmax":
        w = w / (score.sum(1, keepdim=True) + 1e-20)
    return torch.where(ok, order, -1).to(torch.int32), (w * st["scale"]).float()


def _low_rank(x, ids, low, expert, halves):
    """s_a B_a (A_a x) of every row's adapter: all adapters' A at once, a row keeps its own adapter's part."""
    a, b, s = low
    if expert is not None:
        a, b = a[:, expert], b[:, expert]
    L, n, r = b.shape
    mine = torch.where(ids.unsqueeze(1) == torch.arange(L, device=x.device), s, 0.0)
    h = (x @ a.reshape(-1, a.shape[-1]).float().t()).view(-1, L, halves, r) * mine.view(-1, L, 1, 1)
    b = b.float().view(L, halves, n // halves, r)
    return torch.cat([h[:, :, i].flatten(1) @ b[:, i].permute(0, 2, 1).reshape(L * r, -1) for i in range(halves)], 1)


def _plain_shared(st):
    x = st["x"].float()
    y = x @ _int4_values(st["weight"][0][0], st["weight"][1][0]).t()
    y = y + _low_rank(x, st["adapter_ids"], st["low"], None, 2 if st["silu"] else 1)
    if st["silu"]:
        g, u = y.chunk(2, dim=1)
        y = g / (1.0 + torch.exp(-g)) * u
    return y.to(torch.bfloat16)


def _plain_experts(st):
    x = st["x"].float()
    y = torch.zeros_like(x)
    (up, down), (low1, low2) = st["weight"], st["low"]
    for e in range(st["El"]):
        t, j = (st["ids"] == st["first"] + e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        rows, ids = x[t], st["adapter_ids"][t]
        gu = rows @ _int4_values(up[0][e], up[1][e]).t() + _low_rank(rows, ids, low1, e, 2)
        g, u = gu.chunk(2, dim=1)
        h = g / (1.0 + torch.exp(-g)) * u
        d = h @ _int4_values(down[0][e], down[1][e]).t() + _low_rank(h, ids, low2, e, 1)
        y.index_add_(0, t, st["w"][t, j].unsqueeze(1) * d)
    return y.to(torch.bfloat16)


# --------------------------------------------------------------- operators

def run(state):
    op = state["op"]
    if not own:
        return {"route": _plain_route, "shared": _plain_shared, "experts": _plain_experts}[op](state)
    import w4a16_int4_mixture_moe_amd as M
    if op == "route":
        return M.moe_route_grouped(state["logits"], state["k"], state["groups"], state["keep"],
                                   scoring=state["scoring"], bias=state["b"], renormalize=state["renorm"],
                                   scale=state["scale"])
    if op == "shared":
        return M.w4a16_linear(state["x"], state["packed"], state["adapters"], state["adapter_ids"],
                              silu=state["silu"])
    r = M.moe_align(state["ids"], state["E"], state["first"], state["El"], state["block_m"])
    h = M.moe_adapter_gate_up_silu(state["x"], state["p1"], r, state["a1"], state["adapter_ids"])
    return M.moe_adapter_gemm(h, state["p2"], r, state["a2"], state["adapter_ids"], topk_weights=state["w"],
                              a_layout="sorted")


# ------------------------------------------------------------------- exact

def exact(case, seed):
    st = _inputs(case, seed, False)
    f64 = torch.float64
    op, T = case["op"], case["T"]
    if op == "route":
        E, G, size = case["E"], case["groups"], case["E"] // case["groups"]
        rows = st["logits"].to(f64)
        masked = (rows == -math.inf) | rows.isnan()
        score = torch.sigmoid(rows) if case["scoring"] == "sigmoid" else torch.softmax(rows, dim=1)
        key = rows if case["scoring"] == "softmax" else score + (st["b"].to(f64) if case["bias"] else 0.0)
        key = key.masked_fill(masked, -math.inf)

        def take(values):
            """The largest of each row, the lowest index of equals, taken out; -inf and an index past the end: none."""
            top = values.amax(-1, keepdim=True)
            cols = torch.arange(values.shape[-1], device=values.device)
            i = torch.where(values == top, cols, values.shape[-1]).amin(-1, keepdim=True)
            values.scatter_(-1, i, -math.inf)
            return top.squeeze(-1), i.squeeze(-1)

        by_group = key.view(T, G, size).clone()
        value = take(by_group)[0]
        if case["scoring"] == "sigmoid":
            second = take(by_group)[0]
            value = value + second.masked_fill(second == -math.inf, 0.0)
        kept = torch.zeros(T, G, dtype=torch.bool, device=rows.device)
        # a group without a live expert has nothing to give, chosen or not
        value = value.masked_fill(value == -math.inf, -1e300)
        for _ in range(case["keep"]):
            kept.scatter_(1, take(value)[1].unsqueeze(1), True)
        key = key.view(T, G, size).masked_fill(~kept.unsqueeze(2), -math.inf).view(T, E)
        picks, weights = [], []
        for _ in range(case["k"]):
            top, i = take(key)
            gone = top == -math.inf
            picks.append(torch.where(gone, -1, i))
            weights.append(score.gather(1, i.unsqueeze(1)).squeeze(1).masked_fill(gone, 0.0))
        w = torch.stack(weights, 1)
        if case["renorm"]:
            w = w / (w.sum(1, keepdim=True) + 1e-20)
        return torch.stack(picks, 1).to(torch.int32), w * st["scale"]

    def weights_of(codes, scales):
        return ((codes.to(f64) - 8.0) * scales.to(f64).repeat_interleave(GROUP, dim=-1)).to(torch.bfloat16).to(f64)

    def project(rows, ids, weight, low, e, halves):
        """W x + s_a B_a A_a x, one adapter's rows after another's."""
        y = rows @ weights_of(*(t[e or 0] for t in weight)).t()
        a, b, s = low
        for i in range(case["L"]):
            mine = (ids == i).nonzero().squeeze(1)
            if mine.numel() == 0:
                continue
            ai, bi = (a[i], b[i]) if e is None else (a[i, e], b[i, e])
            h = s[i].to(f64) * (rows[mine] @ ai.to(f64).t())
            n, r = bi.shape
            for q in range(halves):
                cols = slice(q * n // halves, (q + 1) * n // halves)
                y[mine, cols] += h[:, q * r:(q + 1) * r] @ bi[cols].to(f64).t()
        return y

    x = st["x"].to(f64)
    if op == "shared":
        y = project(x, st["adapter_ids"], st["weight"], st["low"], None, 2 if case["silu"] else 1)
        if case["silu"]:
            g, u = y.chunk(2, dim=1)
            y = g * torch.sigmoid(g) * u
        return y
    out = torch.zeros(T, case["H"], dtype=f64, device=x.device)
    for e in range(case["El"]):
        t, j = (st["ids"] == case["first"] + e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        ids = st["adapter_ids"][t]
        g, u = project(x[t], ids, st["weight"][0], st["low"][0], e, 2).chunk(2, dim=1)
        d = project(g * torch.sigmoid(g) * u, ids, st["weight"][1], st["low"][1], e, 1)
        out.index_add_(0, t, st["w"][t, j].to(f64).unsqueeze(1) * d)
    return out
