"""Cases of the operators on microscaled 4-bit weights, in plain form and through the package.

MXFP4: a row is cut into blocks of 32 columns; a block holds 32 E2M1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives,
two to a byte, the even column in the low half) and one scale 2^(s - 127), s a byte (255: NaN). Five operators of a served
model whose base weights are stored so:

* ``quantize``  a matrix to codes and scales, and back to the values they stand for (``quantize_mxfp4``, ``dequantize_mxfp4``)
* ``linear``    the multi-LoRA layer over such a base weight, with bias, activation, gate and residual (``linear_mxfp4``)
* ``route``     expert choice by biased softmax or sigmoid scores among the best groups of experts (``route``)
* ``experts``   the product of each routed row with its expert's weight, activation and gate included (``experts_linear``)
* ``combine``   the product back, each token's rows weighted and added to the residual (``experts_combine``)

The activations of a product stay in bf16 ("x": "bf16") or are quantised to MXFP4 themselves first ("x": "mxfp4").

Sizes: 4096 -> 14336 and 4096 -> 4096 are the layer shapes of this repository's workloads, 64 and 4096 tokens its decode and
prefill batches; expert and group counts are generic.
"""
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 32  # columns per scale


def _quantize(name, dtype, rows, d):
    return {"name": name, "op": "quantize", "dtype": dtype, "rows": rows, "d": d}


def _linear(name, x, T, d_in, d_out, segs, rank, act, gated, bias, residual):
    return {"name": name, "op": "linear", "x": x, "T": T, "d_in": d_in, "d_out": d_out, "segs": segs, "rank": rank, "act": act,
            "gated": gated, "bias": bias, "residual": residual}


def _route(name, dtype, T, E, k, scores, bias, groups, top_groups, pad, renorm, scale):
    return {"name": name, "op": "route", "dtype": dtype, "T": T, "E": E, "k": k, "scores": scores, "bias": bias,
            "groups": groups, "top_groups": top_groups, "pad": pad, "renorm": renorm, "scale": scale}


def _experts(name, x, T, E, k, pad, d_in, d_out, act, gated, bias):
    return {"name": name, "op": "experts", "x": x, "T": T, "E": E, "k": k, "pad": pad, "d_in": d_in, "d_out": d_out, "act": act,
            "gated": gated, "bias": bias}


def _combine(name, x, T, E, k, pad, d_in, d_out, bias, residual):
    return {"name": name, "op": "combine", "x": x, "T": T, "E": E, "k": k, "pad": pad, "d_in": d_in, "d_out": d_out,
            "bias": bias, "residual": residual}


def listed():
    return [
        # activations of a decode batch
        _quantize("quantize_decode", "bf16", 64, 4096),
        # an fp32 weight as a checkpoint holds it, before it is served
        _quantize("quantize_weight_f32", "f32", 14336, 4096),
        # gate|up of a single request
        _linear("linear_one_token", "bf16", 1, 4096, 2 * 14336, 1, 32, "silu", True, False, False),
        # output projection of a decode batch: one token per request, 32 adapters, added to the residual stream
        _linear("linear_decode_residual", "bf16", 64, 4096, 4096, 32, 16, "none", False, True, True),
        # gate|up of a prefill batch of 64 prompts, each with its adapter
        _linear("linear_prefill_gated", "bf16", 4096, 4096, 2 * 14336, 64, 64, "silu", True, False, False),
        # the same with the activations in 4 bits too
        _linear("linear_prefill_gated_mx", "mxfp4", 4096, 4096, 2 * 14336, 64, 64, "silu", True, False, False),
        # router of a decode batch: the best 4 of 8 groups of 32 experts by biased sigmoid scores
        _route("route_decode", "bf16", 64, 256, 8, "sigmoid", True, 8, 4, 0, True, 2.5),
        # router of a prefill batch whose last rows are padding
        _route("route_prefill", "f32", 4096, 160, 6, "softmax", False, 8, 3, 77, False, 16.0),
        # one token through two of eight large experts
        _experts("experts_one_token", "bf16", 1, 8, 2, 0, 4096, 2 * 14336, "silu", True, True),
        # a prefill batch through eight large experts, activations in 4 bits
        _experts("experts_prefill_mx", "mxfp4", 4096, 8, 2, 0, 4096, 2 * 14336, "silu", True, False),
        # the way back of a decode batch over many small experts
        _combine("combine_decode", "bf16", 64, 64, 8, 0, 1024, 4096, False, True),
        # the way back of a prefill batch through eight large experts
        _combine("combine_prefill", "bf16", 4096, 8, 2, 0, 14336, 4096, False, True),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _blocks(rng, lo, hi):
    return _log(rng, lo // BLOCK, hi // BLOCK) * BLOCK


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "route", "experts", "experts", "combine"])
    while True:
        if op == "quantize":
            c = {"op": op, "dtype": rng.choice(["bf16", "f32"]), "rows": _log(rng, 1, 14336), "d": _blocks(rng, 128, 14336)}
            if c["rows"] * c["d"] <= 14336 * 4096:
                return c
            continue
        T = _log(rng, 1, 4096)
        if op == "route":
            groups = rng.choice([1, 2, 4, 8, 16])
            E = groups * _log(rng, 2, 256 // groups)
            top_groups = rng.randint(1, groups)
            k = min(top_groups * (E // groups), _log(rng, 1, 10))
            scores = rng.choice(["softmax", "sigmoid"])
            bias = rng.choice([True, False]) or (scores == "softmax" and groups == 1)
            return {"op": op, "dtype": rng.choice(["bf16", "f32"]), "T": T, "E": E, "k": k, "scores": scores, "bias": bias, "groups": groups,
                    "top_groups": top_groups, "pad": rng.choice([0, 0, T // 7]), "renorm": rng.choice([True, False]),
                    "scale": rng.choice([1.0, 2.5])}
        act = rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"])
        x = rng.choice(["bf16", "bf16", "mxfp4"])
        d_in, d_out = _blocks(rng, 512, 14336), _log(rng, 256, 14336)
        if op == "linear":
            gated = rng.choice([True, False])
            segs = min(T, _log(rng, 1, 64))
            if T * d_out * (2 if gated else 1) * d_in > 4096 * 28672 * 4096:
                continue
            return {"op": op, "x": x, "T": T, "d_in": d_in, "d_out": 2 * d_out if gated else d_out, "segs": segs,
                    "rank": rng.choice([8, 16, 32, 64]), "act": act, "gated": gated, "bias": rng.choice([True, False]),
                    "residual": rng.choice([True, False])}
        E = _log(rng, 4, 128)
        k = min(E, _log(rng, 1, 8))
        gated = op == "experts" and rng.choice([True, False])
        rows = 2 * d_out if gated else d_out
        if E * rows * d_in > 8 * 28672 * 4096 or T * k * rows * d_in > 4096 * 28672 * 4096:
            continue
        c = {"op": op, "x": x, "T": T, "E": E, "k": k, "pad": rng.choice([0, 0, T // 7]), "d_in": d_in, "d_out": rows,
             "bias": rng.choice([True, False])}
        if op == "experts":
            return dict(c, act=act, gated=gated)
        return dict(c, residual=rng.choice([True, False]))


# ---------------------------------------------------------------- inputs


def _normal(g, shape, sigma, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda", dtype=dtype) * sigma).to(dtype)


def _activations(g, rows, d):
    """Normal rows with a few columns much larger than the others, as a residual stream has them."""
    x = _normal(g, (rows, d), 1.0)
    x[:, torch.randperm(d, generator=g, device="cuda")[: d // 256]] *= 12
    return x


def _tiled(scale):
    """Scales [.., rows, d / 32] in the package's layout [.., ceil(d / 128), rows, 4]."""
    lead, n = scale.shape[:-1], scale.shape[-1]
    padded = torch.full((*lead, (n + 3) // 4 * 4), 127, dtype=torch.uint8, device=scale.device)
    padded[..., :n] = scale
    return padded.reshape(*lead, -1, 4).transpose(-2, -3).contiguous()


def _pow2(n):
    """2^n in 32 bits, n an int32 tensor from -127 (0 in its place) to 127."""
    return ((n + 127) << 23).view(torch.float32)


def _encode(W):
    """Codes [rows, d / 2] and scales [rows, d / 32] of a finite matrix."""
    b = W.float().reshape(W.shape[0], -1, BLOCK)
    top = b.abs().amax(-1)
    s = ((top.view(torch.int32) >> 23) - 2).clamp(min=0)  # the exponent of the largest, less E2M1's own
    v = b * _pow2(127 - s)[..., None]
    a = v.abs()
    code = torch.bucketize(a, torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=W.device))  # ties below ..
    for tie, up in ((0.75, 2), (1.75, 4), (3.5, 6)):  # .. but these have their even code above
        code = torch.where(a == tie, up, code)
    code = torch.where(v < 0, code + 8, code).to(torch.uint8).reshape(W.shape[0], -1)
    return code[:, ::2] | (code[:, 1::2] << 4), s.to(torch.uint8)


def _weight(g, shape):
    """Codes and row-major scales of a normal weight [.., rows, d], a slice of it at a time."""
    *lead, rows, d = shape
    W = [_encode(_normal(g, (rows, d), 0.02)) for _ in range(lead[0] if lead else 1)]
    codes, scale = torch.stack([c for c, _ in W]), torch.stack([s for _, s in W])
    return (codes, scale) if lead else (codes[0], scale[0])


def _logits(g, case, dtype):
    """Router logits: normal, some experts more popular than others; padded rows are -inf."""
    T, E = case["T"], case["E"]
    x = torch.randn((T, E), generator=g, device="cuda") + 0.5 * torch.randn((1, E), generator=g, device="cuda")
    x[T - case["pad"]:] = float("-inf")
    return x.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, s = case["op"], {"case": case}
    if own:
        import rank_adapter_gemm_segmented_amd as ml
        s["ml"] = ml
    if op == "quantize":
        s["x"] = _activations(g, case["rows"], case["d"]).to(DT[case["dtype"]])
        if case["dtype"] == "f32":
            s["x"] *= 1 + 0.01 * torch.rand(s["x"].shape, generator=g, device="cuda")
        return s
    T = case["T"]
    if op == "route":
        s["logits"] = _logits(g, case, DT[case["dtype"]])
        s["bias"] = 0.1 * torch.randn(case["E"], generator=g, device="cuda") if case["bias"] else None
        if own:
            s["workspace"] = ml.route_workspace(T, case["E"], case["k"])
        return s
    d_in, d_out = case["d_in"], case["d_out"]
    if op == "linear":
        s["x"] = _activations(g, T, d_in)
        s["W"], s["w_scale"] = _weight(g, (d_out, d_in))
        n, r = case["segs"], case["rank"]
        s["A"], s["B"] = _normal(g, (n, r, d_in), 0.02), _normal(g, (n, d_out, r), 0.01)
        cut = torch.sort(torch.randperm(T - 1, generator=g, device="cuda")[: n - 1] + 1).values if n > 1 else torch.zeros(0, device="cuda")
        s["seg_start"] = torch.cat([torch.tensor([0.0], device="cuda"), cut.float(), torch.tensor([float(T)], device="cuda")]).int()
        s["seg_adapter"] = torch.randperm(n, generator=g, device="cuda").int()
        s["seg_rank"] = torch.full((n,), r, dtype=torch.int32, device="cuda")
        s["seg_scale"] = torch.full((n,), 2.0, device="cuda")
        s["bias"] = _normal(g, (d_out,), 0.1) if case["bias"] else None
        s["residual"] = _normal(g, (T, d_out // 2 if case["gated"] else d_out), 1.0) if case["residual"] else None
        if own:
            s["pool"] = ml.Pool(d_in, d_out, torch.bfloat16, r, n)
            for a in range(n):
                s["pool"].register(a, s["A"][a], s["B"][a])
            s["workspace"] = s["pool"].workspace(T)
    else:
        plain = {"scores": "softmax", "groups": 1, "top_groups": 1, "renorm": True, "scale": 1.0, "k": case["k"]}
        _, s["weight"], s["token_index"], s["seg_start"], s["position"] = _route_plain(_logits(g, case, torch.float32), None, plain)
        s["W"], s["w_scale"] = _weight(g, (case["E"], d_out, d_in))
        s["bias"] = _normal(g, (case["E"], d_out), 0.1) if case["bias"] else None
        P = T * case["k"]
        s["x"] = _activations(g, T if op == "experts" else P, d_in)
        if op == "experts":
            s["out"] = torch.zeros((P, d_out // 2 if case["gated"] else d_out), dtype=torch.bfloat16, device="cuda")  # rows of no expert stay
        else:
            s["residual"] = _normal(g, (T, d_out), 1.0) if case["residual"] else None
            if own:
                s["workspace"] = ml.experts_workspace(T, case["k"], case["E"], d_out, torch.bfloat16)
    if own:
        s["w_scale"] = _tiled(s["w_scale"])  # laid out once, as a program that serves the weight does
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


def _nearest(x):
    """The MXFP4 values nearest to x's in 32 bits (every step is exact): steps of 0.5, 1 and 2 below 2, 4 and 6."""
    b = x.float().reshape(x.shape[0], -1, BLOCK)
    top = b.abs().amax(-1, keepdim=True)
    e = ((top.view(torch.int32) >> 23) - 2).clamp(min=0) - 127
    v = b * _pow2(-e)
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.clamp(torch.round(a / step) * step, max=6.0)
    return (torch.where(v < 0, -q, q) * _pow2(e)).reshape(x.shape)


def _values(codes, scale):
    """What codes [.., d / 2] and row-major scales [.., d / 32] stand for, in 32 bits."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=codes.device)
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).reshape(*scale.shape, BLOCK)
    return (v * _pow2(scale.int() - 127)[..., None]).reshape(*codes.shape[:-1], -1)


def _x32(s, c):
    return _nearest(s["x"]) if c["x"] == "mxfp4" else s["x"].float()


def _linear_plain(s, c):
    z = _x32(s, c) @ _values(s["W"], s["w_scale"]).T
    # all adapters' low-rank products, those of other segments' adapters masked out
    n, r, x = c["segs"], c["rank"], s["x"].float()
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
    return z.to(torch.bfloat16)


def _route_plain(logits, bias, c):
    """Scores in 64 bits (choices lie next to each other), rounded to 32, where the bias is added and choices are made."""
    T, E = logits.shape
    l = logits.double()
    l = torch.where(torch.isnan(l), float("-inf"), l)
    if c["scores"] == "sigmoid":
        s = (1 / (1 + torch.exp(-l))).float()
    else:
        top = l.amax(-1, keepdim=True)
        p = torch.where(l > float("-inf"), torch.where(l == top, 1.0, torch.exp(l - top)), 0.0)
        s = (p / p.sum(-1, keepdim=True)).float()
    biased = s if bias is None else s + bias
    biased = torch.where((l > float("-inf")) & ~torch.isnan(biased), biased, float("-inf"))
    # the groups whose two best add up to the most
    G, k = c["groups"], c["k"]
    if G > 1:
        two = torch.sort(biased.reshape(T, G, -1), dim=-1, descending=True, stable=True).values[:, :, :2]
        two = torch.where(two > float("-inf"), two, torch.where(two[:, :, :1] > float("-inf"), 0.0, float("-inf")))
        at = torch.sort(two.sum(-1) if two.shape[-1] > 1 else two[:, :, 0], dim=-1, descending=True, stable=True).indices[:, :c["top_groups"]]
        kept = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, at, True)
        biased = torch.where(kept.repeat_interleave(E // G, dim=1), biased, float("-inf"))
    top, idx = torch.sort(biased, dim=-1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    chosen = top > float("-inf")
    w = torch.where(chosen, torch.gather(s, 1, idx), 0.0)
    if c["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    w = c["scale"] * w
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
    x = _x32(s, c)[rows.clamp(min=0).long()[at.clamp(max=P - 1)]]
    y = torch.bmm(x, _values(s["W"][e], s["w_scale"][e]).transpose(1, 2).contiguous())
    if c["bias"]:
        y = y + s["bias"][e].float()[:, None]
    z[at[inside]] = y[inside]
    return z


def _experts_plain(s, c):
    return _finish(_products(s, c, s["token_index"]), c["act"], c["gated"]).to(torch.bfloat16)


def _combine_plain(s, c):
    z = _products(s, c, torch.arange(c["T"] * c["k"], device="cuda"))
    p = s["position"]
    y = (z[p.clamp(min=0).long()] * torch.where(p >= 0, s["weight"], 0.0)[:, :, None]).sum(1)
    if c["residual"]:
        y = y + s["residual"].float()
    return y.to(torch.bfloat16)


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        if op == "quantize":
            return _nearest(s["x"]).to(s["x"].dtype)
        if op == "linear":
            return _linear_plain(s, c)
        if op == "route":
            return _route_plain(s["logits"], s["bias"], c)
        return _experts_plain(s, c) if op == "experts" else _combine_plain(s, c)
    ml = s["ml"]
    if op == "quantize":
        codes, scale = ml.quantize_mxfp4(s["x"])
        return ml.dequantize_mxfp4(codes, scale, s["x"].dtype)
    if op == "route":
        return ml.route(s["logits"], c["k"], renormalize=c["renorm"], workspace=s["workspace"], scores=c["scores"],
                        bias=s["bias"], n_groups=c["groups"], top_groups=c["top_groups"], scale=c["scale"])
    codes, scale = ml.quantize_mxfp4(s["x"]) if c["x"] == "mxfp4" else (None, None)
    if op == "linear":
        return ml.linear_mxfp4(s["x"], s["W"], s["w_scale"], s["pool"], s["seg_start"], s["seg_adapter"], s["seg_rank"],
                               s["seg_scale"], x_codes=codes, x_scale=scale, bias=s["bias"], act=c["act"], gated=c["gated"],
                               residual=s["residual"], workspace=s["workspace"])
    x = s["x"] if codes is None else codes
    if op == "experts":
        return ml.experts_linear(x, s["W"], s["seg_start"], s["token_index"], bias=s["bias"], act=c["act"], gated=c["gated"],
                                 w_scale=s["w_scale"], x_scale=scale, out=s["out"])
    return ml.experts_combine(x, s["W"], s["seg_start"], s["position"], s["weight"], bias=s["bias"], residual=s["residual"],
                              w_scale=s["w_scale"], x_scale=scale, workspace=s["workspace"])


# ---------------------------------------------------------------- work and exact values


def work(case):
    c, op = case, case["op"]
    if op == "quantize":
        n = c["rows"] * c["d"]
        return {"bytes": n * (4 if c["dtype"] == "f32" else 2) * 2 + n // 2 + n // BLOCK, "flops": 2 * n}
    T = c["T"]
    if op == "route":
        P = T * c["k"]
        el = 4 if c["dtype"] == "f32" else 2
        return {"bytes": T * c["E"] * el + 16 * P + 4 * (c["E"] + 1) + (4 * c["E"] if c["bias"] else 0), "flops": T * c["E"] * 6}
    d_in, d_out = c["d_in"], c["d_out"]
    wb = d_in // 2 + d_in // BLOCK  # bytes of a weight row
    if op == "linear":
        y = d_out // 2 if c["gated"] else d_out
        n = d_out * wb + (T * d_in + T * y) * 2 + c["segs"] * c["rank"] * (d_in + d_out) * 2
        n += (d_out * 2 if c["bias"] else 0) + (T * y * 2 if c["residual"] else 0)
        return {"bytes": n, "flops": 2 * T * d_in * d_out + 2 * T * c["rank"] * (d_in + d_out)}
    live = T - c["pad"]
    P = live * c["k"]
    active = c["E"] * (1 - (1 - c["k"] / c["E"]) ** live)  # experts that some row takes, expected
    n = active * d_out * wb + (active * d_out * 2 if c["bias"] else 0)
    if op == "experts":
        n += live * d_in * 2 + P * (d_out // 2 if c["gated"] else d_out) * 2 + 4 * P
    else:
        n += P * d_in * 2 + T * d_out * 2 * (2 if c["residual"] else 1) + 8 * P
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


def _exp2_64(n):
    return ((n.long() + 1023) << 52).view(torch.float64)


def _mx64(x):
    """The nearest of the format's values in 64 bits: each value's distance to all of them, the even code where two tie."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    step = max(1, (1 << 24) // x.shape[1])
    for r in range(0, x.shape[0], step):
        b = x[r:r + step].double().unflatten(-1, (-1, BLOCK))
        top = b.abs().amax(-1, keepdim=True)
        e = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(min=-127)  # top = m 2^exponent, m in [0.5, 1)
        a = b.abs() * _exp2_64(-e)
        lo = (torch.searchsorted(grid, a, right=True) - 1).clamp(max=6)
        below, above = a - grid[lo], grid[lo + 1] - a
        code = torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, lo + 1)
        out[r:r + step] = (grid[code] * torch.sign(b) * _exp2_64(e)).flatten(-2)
    return out


def _w64(codes, scale):
    low, high = codes & 15, codes >> 4
    c = torch.stack([low, high], -1).flatten(-2).unflatten(-1, (-1, BLOCK)).int()
    m, e = c & 1, (c >> 1) & 3
    v = torch.where(e > 0, (1 + 0.5 * m.double()) * _exp2_64(e - 1), 0.5 * m.double()) * (1 - 2.0 * (c >> 3))
    return (v * _exp2_64(scale.long() - 127)[..., None]).flatten(-2)


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    c, op = case, case["op"]
    if op == "quantize":
        return _mx64(s["x"])
    T = c["T"]
    if op == "route":
        l = s["logits"].double()
        if c["scores"] == "sigmoid":
            score = torch.sigmoid(l)
        else:
            score = torch.nan_to_num(torch.softmax(l, -1), nan=0.0)
        key = score.float() + (s["bias"] if c["bias"] else 0.0)  # choices are made in 32 bits
        key = torch.where(torch.isinf(l), float("-inf"), key)
        per = c["E"] // c["groups"]
        best = torch.topk(key.unflatten(-1, (-1, per)), min(2, per), dim=-1).values.sum(-1)
        at = torch.arange(T, device="cuda")

        def highest(left):  # the lowest index of the largest
            m = left.max(-1, keepdim=True).values
            return torch.where(left == m, torch.arange(left.shape[1], device="cuda"), left.shape[1]).min(-1).values

        kept_groups = torch.zeros_like(best, dtype=torch.bool)
        for _ in range(c["top_groups"]):
            i = highest(best)
            kept_groups[at, i] = True
            best[at, i] = float("-inf")
        left = torch.where(kept_groups.repeat_interleave(per, 1), key, float("-inf"))
        got = []
        for _ in range(c["k"]):
            i = highest(left)
            there = left[at, i] > float("-inf")
            got.append(torch.where(there, score[at, i], torch.zeros_like(score[:, 0])))
            left[at, i] = float("-inf")
        w = torch.stack(got, -1)
        if c["renorm"]:
            w = torch.nan_to_num(w / w.sum(-1, keepdim=True), nan=0.0)
        return None, c["scale"] * w, None, None, None
    x = _mx64(s["x"]) if c["x"] == "mxfp4" else s["x"].double()
    if op == "linear":
        z = x @ _w64(s["W"], s["w_scale"]).T
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
        rows = x[s["token_index"][a:b].long()] if op == "experts" else x[a:b]
        z = rows @ _w64(s["W"][e], s["w_scale"][e]).T
        if c["bias"]:
            z = z + s["bias"][e].double()
        if op == "experts":
            y[a:b] = _pair64(z, c)
        else:
            y.index_add_(0, token[a:b], z * weight[a:b, None])  # one row of a token per expert
    return y
