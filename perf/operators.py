"""Cases of the epilogue and expert operators: what is measured, in plain form and through the package.

Four operators of a served transformer layer, each in an elementary torch form (32-bit, rounded once) and as the
package's call:

* ``linear``  the multi-LoRA layer with bias, activation, gate and residual (``linear_epilogue``)
* ``route``   top-k expert choice of a batch and its segments (``route``)
* ``experts`` the product of each routed row with its expert's weight, activation and gate included (``experts_linear``)
* ``combine`` the product back, each token's rows weighted and added to the residual (``experts_combine``)

Sizes: 4096 -> 14336 and 4096 -> 4096 are the layer shapes of this repository's workloads, 256 -> 256 its tiny fp32 one,
64 and 4096 tokens its decode and prefill batches; expert counts are generic.
"""
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8w": torch.bfloat16}


def _linear(name, dtype, T, d_in, d_out, segs, rank, act, gated, bias, residual):
    return {"name": name, "op": "linear", "dtype": dtype, "T": T, "d_in": d_in, "d_out": d_out, "segs": segs, "rank": rank,
            "act": act, "gated": gated, "bias": bias, "residual": residual}


def _route(name, dtype, T, E, k, pad, renorm):
    return {"name": name, "op": "route", "dtype": dtype, "T": T, "E": E, "k": k, "pad": pad, "renorm": renorm}


def _experts(name, dtype, T, E, k, pad, d_in, d_out, act, gated, bias):
    return {"name": name, "op": "experts", "dtype": dtype, "T": T, "E": E, "k": k, "pad": pad, "d_in": d_in, "d_out": d_out,
            "act": act, "gated": gated, "bias": bias}


def _combine(name, dtype, T, E, k, pad, d_in, d_out, bias, residual):
    return {"name": name, "op": "combine", "dtype": dtype, "T": T, "E": E, "k": k, "pad": pad, "d_in": d_in, "d_out": d_out,
            "bias": bias, "residual": residual}


def listed():
    return [
        # output projection of a decode batch: one token per request, 32 adapters, added to the residual stream
        _linear("linear_decode_residual", "bf16", 64, 4096, 4096, 32, 16, "none", False, True, True),
        # gate|up of a single request with the base weight in FP8
        _linear("linear_one_token_fp8w", "fp8w", 1, 4096, 2 * 14336, 1, 32, "silu", True, False, False),
        # gate|up of a prefill batch of 64 prompts, each with its adapter
        _linear("linear_prefill_gated", "bf16", 4096, 4096, 2 * 14336, 64, 64, "silu", True, False, False),
        # the smallest fp32 layer, where latency is all
        _linear("linear_tiny_f32", "f32", 16, 256, 256, 4, 8, "gelu", False, True, True),
        # router of a decode batch over many small experts
        _route("route_decode", "bf16", 64, 128, 8, 0, True),
        # router of a prefill batch whose last rows are padding
        _route("route_prefill", "f32", 4096, 64, 8, 77, True),
        # one token through two of eight large experts
        _experts("experts_one_token", "bf16", 1, 8, 2, 0, 4096, 2 * 14336, "silu", True, False),
        # a decode batch over many small experts stored in FP8, ragged: about eight rows each
        _experts("experts_decode_fp8w", "fp8w", 64, 64, 8, 0, 4096, 2 * 1024, "silu", True, False),
        # a prefill batch through eight large experts
        _experts("experts_prefill", "bf16", 4096, 8, 2, 0, 4096, 2 * 14336, "silu", True, False),
        # a tiny fp32 layer of experts with odd sizes and padding
        _experts("experts_tiny_f32", "f32", 37, 5, 2, 4, 256, 2 * 172, "gelu_tanh", True, True),
        # the way back of a decode batch over many small experts
        _combine("combine_decode", "bf16", 64, 64, 8, 0, 1024, 4096, False, True),
        # the way back of a prefill batch through eight large experts
        _combine("combine_prefill", "bf16", 4096, 8, 2, 0, 14336, 4096, False, True),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _mult(rng, lo, hi, m):
    return max(m, _log(rng, lo, hi) // m * m)


def draw(rng):
    op = rng.choice(["linear", "linear", "route", "experts", "experts", "combine"])
    while True:
        dtype = rng.choice(["bf16", "bf16", "fp8w", "f32"])
        T = _log(rng, 1, 4096)
        if op == "route":
            E = _log(rng, 2, 256)
            k = min(E, _log(rng, 1, 8))
            return {"op": op, "dtype": rng.choice(["bf16", "f32"]), "T": T, "E": E, "k": k,
                    "pad": rng.choice([0, 0, T // 7]), "renorm": rng.choice([True, False])}
        act = rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"])
        if dtype == "f32":
            T, d_in, d_out = _log(rng, 1, 256), _mult(rng, 128, 1024, 8), _log(rng, 64, 1024)
        else:
            d_in, d_out = _mult(rng, 512, 14336, 16), _log(rng, 256, 14336)
        if op == "linear":
            if dtype == "fp8w":
                T = _log(rng, 1, 64)
            gated = rng.choice([True, False])
            segs = min(T, _log(rng, 1, 64))
            if T * d_out * (2 if gated else 1) * d_in > 8192 * 28672 * 4096:
                continue
            return {"op": op, "dtype": dtype, "T": T, "d_in": d_in, "d_out": 2 * d_out if gated else d_out, "segs": segs,
                    "rank": rng.choice([8, 16, 32, 64]), "act": act, "gated": gated, "bias": rng.choice([True, False]),
                    "residual": rng.choice([True, False])}
        if dtype == "fp8w":
            T = _log(rng, 1, 128)
        E = _log(rng, 4, 128)
        k = min(E, _log(rng, 1, 8))
        gated = op == "experts" and rng.choice([True, False])
        rows = 2 * d_out if gated else d_out
        if E * rows * d_in > 8 * 28672 * 4096 or T * k * rows * d_in > 8192 * 28672 * 4096:
            continue
        if dtype == "fp8w" and T * k > 1024:
            continue
        c = {"op": op, "dtype": dtype, "T": T, "E": E, "k": k, "pad": rng.choice([0, 0, T // 7]), "d_in": d_in, "d_out": rows,
             "bias": rng.choice([True, False])}
        if op == "experts":
            return dict(c, act=act, gated=gated)
        return dict(c, residual=rng.choice([True, False]))


# ---------------------------------------------------------------- inputs


def _normal(g, shape, sigma, dtype):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32 if dtype == torch.float32 else torch.bfloat16)
            * sigma).to(dtype)


def _e4m3(W):
    """Codes and float32 row scales of a weight whose last axis is d_in."""
    scale = W.abs().amax(dim=-1).float() / 448.0
    return (W / scale[..., None].to(W.dtype)).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _weight(g, shape, case):
    W = _normal(g, shape, 0.02, DT[case["dtype"]])
    return _e4m3(W) if case["dtype"] == "fp8w" else (W, None)


def _logits(g, case, dtype):
    """Router logits: normal, some experts more popular than others; padded rows are -inf."""
    T, E = case["T"], case["E"]
    x = torch.randn((T, E), generator=g, device="cuda") + 0.5 * torch.randn((1, E), generator=g, device="cuda")
    x[T - case["pad"]:] = float("-inf")
    return x.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, T = case["op"], case["T"]
    s = {"case": case}
    if op == "route":
        s["logits"] = _logits(g, case, DT[case["dtype"]])
        if own:
            import rank_adapter_gemm_segmented_amd as ml
            s["ml"], s["workspace"] = ml, ml.route_workspace(T, case["E"], case["k"])
        return s
    dt, d_in, d_out = DT[case["dtype"]], case["d_in"], case["d_out"]
    if op == "linear":
        s["x"] = _normal(g, (T, d_in), 1.0, dt)
        s["W"], s["w_scale"] = _weight(g, (d_out, d_in), case)
        n, r = case["segs"], case["rank"]
        s["A"], s["B"] = _normal(g, (n, r, d_in), 0.02, dt), _normal(g, (n, d_out, r), 0.01, dt)
        cut = torch.sort(torch.randperm(T - 1, generator=g, device="cuda")[: n - 1] + 1).values if n > 1 else torch.zeros(0, device="cuda")
        s["seg_start"] = torch.cat([torch.tensor([0.0], device="cuda"), cut.float(), torch.tensor([float(T)], device="cuda")]).int()
        s["seg_adapter"] = torch.randperm(n, generator=g, device="cuda").int()
        s["seg_rank"] = torch.full((n,), r, dtype=torch.int32, device="cuda")
        s["seg_scale"] = torch.full((n,), 2.0, device="cuda")
        s["bias"] = _normal(g, (d_out,), 0.1, dt) if case["bias"] else None
        s["residual"] = _normal(g, (T, d_out // 2 if case["gated"] else d_out), 1.0, dt) if case["residual"] else None
        if own:
            import rank_adapter_gemm_segmented_amd as ml
            s["ml"], s["pool"] = ml, ml.Pool(d_in, d_out, dt, r, n)
            for a in range(n):
                s["pool"].register(a, s["A"][a], s["B"][a])
            s["workspace"] = s["pool"].workspace(T)
        return s
    _, s["weight"], s["token_index"], s["seg_start"], s["position"] = _route_plain(_logits(g, case, torch.float32), case["k"], True)
    s["W"], s["w_scale"] = _weight(g, (case["E"], d_out, d_in), case)
    s["bias"] = _normal(g, (case["E"], d_out), 0.1, dt) if case["bias"] else None
    P = T * case["k"]
    if op == "experts":
        s["x"] = _normal(g, (T, d_in), 1.0, dt)
        s["out"] = torch.zeros((P, d_out // 2 if case["gated"] else d_out), dtype=dt, device="cuda")  # rows of no expert stay
    else:
        s["x"] = _normal(g, (P, d_in), 1.0, dt)
        s["residual"] = _normal(g, (T, d_out), 1.0, dt) if case["residual"] else None
    if own:
        import rank_adapter_gemm_segmented_amd as ml
        s["ml"] = ml
        s["workspace"] = ml.experts_workspace(T, case["k"], case["E"], d_out, dt) if op == "combine" else None
    return s


# ---------------------------------------------------------------- plain forms


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.7071067811865476))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z)))
    return z


def _finish(z, act, gated):
    if not gated:
        return _act(z, act)
    half = z.shape[-1] // 2
    return _act(z[..., :half], act) * z[..., half:]


def _weight32(W, scale):
    return W.float() if scale is None else W.view(torch.float8_e4m3fn).float() * scale[..., None]


def _linear_plain(s, c):
    x = s["x"].float()
    z = x @ _weight32(s["W"], s["w_scale"]).T
    # all adapters' low-rank products, those of other segments' adapters masked out
    n, r = c["segs"], c["rank"]
    p = torch.arange(c["T"], device="cuda")
    seg = torch.searchsorted(s["seg_start"][1:].contiguous(), p, right=True)
    mask = (s["seg_adapter"][seg][:, None] == torch.arange(n, device="cuda")) * s["seg_scale"][seg][:, None]
    v = (x @ s["A"].float().reshape(n * r, -1).T).reshape(-1, n, r) * mask[:, :, None]
    z = z + v.reshape(-1, n * r) @ s["B"].float().permute(0, 2, 1).reshape(n * r, -1)
    if c["bias"]:
        z = z + s["bias"].float()
    z = _finish(z, c["act"], c["gated"])
    if c["residual"]:
        z = z + s["residual"].float()
    return z.to(DT[c["dtype"]])


def _route_plain(logits, k, renorm):
    T, E = logits.shape
    l = logits.float()
    l = torch.where(torch.isnan(l), float("-inf"), l)
    top, idx = torch.sort(l, dim=-1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    m = top[:, :1]
    chosen = top > float("-inf")
    p = torch.where(l == m, 1.0, torch.exp(l - m))
    w = torch.where(top == m, 1.0, torch.exp(top - m))
    w = torch.where(chosen, w, 0.0)
    w = w / torch.where(chosen[:, :1], w.sum(-1, keepdim=True) if renorm else p.sum(-1, keepdim=True), 1.0)
    ids = torch.where(chosen, idx, E).reshape(-1)
    ids_sorted, order = torch.sort(ids, stable=True)
    there = ids_sorted < E
    token_index = torch.where(there, order // k, -1).int()
    seg_start = torch.searchsorted(ids_sorted, torch.arange(E + 1, device=ids.device)).int()
    position = torch.empty_like(order)
    position[order] = torch.where(there, torch.arange(T * k, device=ids.device), -1)
    return torch.where(chosen, idx, -1).int(), w, token_index, seg_start, position.reshape(T, k).int()


def _products(s, c, rows):
    """W_e x + b_e of each sorted position in 32 bits: the experts that have rows, padded to the longest segment."""
    start = s["seg_start"].long()
    count = start[1:] - start[:-1]
    e = torch.nonzero(count)[:, 0]
    P = rows.shape[0]
    z = torch.zeros((P, c["d_out"]), device="cuda")
    if e.numel() == 0:
        return z
    at = start[e][:, None] + torch.arange(int(count.max()), device="cuda")
    inside = at < start[e + 1][:, None]
    x = s["x"].float()[rows.clamp(min=0).long()[at.clamp(max=P - 1)]]
    y = torch.bmm(x, _weight32(s["W"][e], None if s["w_scale"] is None else s["w_scale"][e]).transpose(1, 2).contiguous())
    if c["bias"]:
        y = y + s["bias"][e].float()[:, None]
    z[at[inside]] = y[inside]
    return z


def _experts_plain(s, c):
    z = _finish(_products(s, c, s["token_index"]), c["act"], c["gated"])
    return z.to(DT[c["dtype"]])


def _combine_plain(s, c):
    z = _products(s, c, torch.arange(c["T"] * c["k"], device="cuda"))
    p = s["position"]
    y = (z[p.clamp(min=0).long()] * torch.where(p >= 0, s["weight"], 0.0)[:, :, None]).sum(1)
    if c["residual"]:
        y = y + s["residual"].float()
    return y.to(DT[c["dtype"]])


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        if op == "linear":
            return _linear_plain(s, c)
        if op == "route":
            return _route_plain(s["logits"], c["k"], c["renorm"])
        return _experts_plain(s, c) if op == "experts" else _combine_plain(s, c)
    ml = s["ml"]
    if op == "linear":
        return ml.linear_epilogue(s["x"], s["W"], s["pool"], s["seg_start"], s["seg_adapter"], s["seg_rank"], s["seg_scale"],
                                  bias=s["bias"], act=c["act"], gated=c["gated"], residual=s["residual"], w_scale=s["w_scale"],
                                  workspace=s["workspace"])
    if op == "route":
        return ml.route(s["logits"], c["k"], renormalize=c["renorm"], workspace=s["workspace"])
    if op == "experts":
        return ml.experts_linear(s["x"], s["W"], s["seg_start"], s["token_index"], bias=s["bias"], act=c["act"],
                                 gated=c["gated"], w_scale=s["w_scale"], out=s["out"])
    return ml.experts_combine(s["x"], s["W"], s["seg_start"], s["position"], s["weight"], bias=s["bias"],
                              residual=s["residual"], w_scale=s["w_scale"], workspace=s["workspace"])


# ---------------------------------------------------------------- work and exact values


def _bytes_of(dtype):
    return 4 if dtype == "f32" else 2


def work(case):
    c, el, op, T = case, _bytes_of(case["dtype"]), case["op"], case["T"]
    if op == "route":
        P = T * c["k"]
        return {"bytes": T * c["E"] * el + 16 * P + 4 * (c["E"] + 1), "flops": T * c["E"] * 4}
    d_in, d_out = c["d_in"], c["d_out"]
    wb = d_in + 4 if c["dtype"] == "fp8w" else d_in * el  # bytes of a weight row
    if op == "linear":
        y = d_out // 2 if c["gated"] else d_out
        n = d_out * wb + (T * d_in + T * y) * el + c["segs"] * c["rank"] * (d_in + d_out) * el
        n += (d_out * el if c["bias"] else 0) + (T * y * el if c["residual"] else 0)
        return {"bytes": n, "flops": 2 * T * d_in * d_out + 2 * T * c["rank"] * (d_in + d_out)}
    live = T - c["pad"]
    P = live * c["k"]
    active = c["E"] * (1 - (1 - c["k"] / c["E"]) ** live)  # experts that some row takes, expected
    n = active * d_out * wb + (active * d_out * el if c["bias"] else 0)
    if op == "experts":
        n += live * d_in * el + P * (d_out // 2 if c["gated"] else d_out) * el + 4 * P
    else:
        n += P * d_in * el + T * d_out * el * (2 if c["residual"] else 1) + 8 * P
    return {"bytes": n, "flops": 2 * P * d_in * d_out}


def _act64(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z**3))
    return z


def _pair64(z, c):
    if not c["gated"]:
        return _act64(z, c["act"])
    gate, up = z.chunk(2, dim=-1)
    return _act64(gate, c["act"]) * up


def _weight64(s, e=None):
    W, scale = (s["W"], s["w_scale"]) if e is None else (s["W"][e], None if s["w_scale"] is None else s["w_scale"][e])
    return W.double() if scale is None else W.view(torch.float8_e4m3fn).double() * scale.double().unsqueeze(-1)


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    c, op, T = case, case["op"], case["T"]
    if op == "route":
        l = s["logits"].double()
        left = l.nan_to_num(nan=float("-inf"), posinf=float("inf"), neginf=float("-inf")).clone()
        at, total = torch.arange(T, device="cuda"), torch.exp(left - left.max(-1, keepdim=True).values).sum(-1)
        first, got = left.max(-1).values, []
        for _ in range(c["k"]):
            m = left.max(-1, keepdim=True).values
            i = torch.where(left == m, torch.arange(c["E"], device="cuda"), c["E"]).min(-1).values
            got.append(torch.where(m[:, 0] > float("-inf"), torch.exp(m[:, 0] - first), torch.zeros_like(first)))
            left[at, i] = float("-inf")
        w = torch.stack(got, -1)
        w = w / (w.sum(-1, keepdim=True) if c["renorm"] else total[:, None])
        return None, torch.where(torch.isfinite(first)[:, None], w, torch.zeros_like(w)), None, None, None
    if op == "linear":
        z = s["x"].double() @ _weight64(s).T
        start = s["seg_start"].tolist()
        for i, a in enumerate(s["seg_adapter"].tolist()):
            rows = s["x"][start[i]:start[i + 1]].double()
            z[start[i]:start[i + 1]] += float(s["seg_scale"][i]) * ((rows @ s["A"][a].double().T) @ s["B"][a].double().T)
        if c["bias"]:
            z += s["bias"].double()
        z = _pair64(z, c)
        return z + s["residual"].double() if c["residual"] else z
    start = s["seg_start"].tolist()
    if op == "experts":
        y = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    else:
        y = torch.zeros((T, c["d_out"]), dtype=torch.float64, device="cuda")
        if c["residual"]:
            y += s["residual"].double()
        # the token and the weight of each sorted position
        token, weight = torch.zeros(T * c["k"], dtype=torch.long, device="cuda"), torch.zeros(T * c["k"], dtype=torch.float64, device="cuda")
        t, j = torch.nonzero(s["position"] >= 0, as_tuple=True)
        token[s["position"][t, j].long()], weight[s["position"][t, j].long()] = t, s["weight"][t, j].double()
    for e in range(c["E"]):
        a, b = start[e], start[e + 1]
        if a == b:
            continue
        rows = s["x"][s["token_index"][a:b].long()] if op == "experts" else s["x"][a:b]
        z = rows.double() @ _weight64(s, e).T
        if c["bias"]:
            z = z + s["bias"][e].double()
        if op == "experts":
            y[a:b] = _pair64(z, c)
        else:
            y.index_add_(0, token[a:b], z * weight[a:b, None])  # one row of a token per expert
    return y
