"""References in 64 bits for MXFP4 and for routing by scores.

The format's values are enumerated here and a value is quantised by its distance to each of them, apart from the
library's conversion. Products: the bound of op_util.product64 counts a rounding per product in fp32; MXFP4 values are
exact in bf16 and in the matrix units, so nothing is added to it.
"""
import torch

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def pow2(n):
    """2^n in 64 bits, exact, n an integer tensor of the format's range."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def decode(codes, scale, d):
    """[..., rows, d] in 64 bits of codes [..., rows, d / 2] and scale [..., planes, rows, 4]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=codes.device)
    low, high = table[(codes & 15).long()], table[(codes >> 4).long()]
    v = torch.stack([low, high], -1).flatten(-2)
    s = scale.transpose(-2, -3).flatten(-2)[..., : d // 32].long()
    f = torch.where(s == 255, float("nan"), pow2(s - 127))
    return v * f.repeat_interleave(32, -1)


def encode(x):
    """(values in 64 bits, scales [rows, d / 32] as int) of x [rows, d]: the nearest value of the format, the one of even
    code where two are as near; blocks of a NaN or an infinity have scale 255 and NaN values."""
    b = x.double().cpu().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    e = torch.where(top > 0, torch.frexp(torch.where(bad, 1.0, top)).exponent - 3, -127).clamp(min=-127)
    grid = torch.tensor(E2M1, dtype=torch.float64)
    a = (b.abs() * pow2(-e)[..., None]).nan_to_num(nan=0.0, posinf=0.0)
    dist = (a[..., None] - grid).abs()
    near = dist == dist.amin(-1, keepdim=True)
    code = torch.arange(8)
    pick = torch.where(near, code - 100 * (code % 2 == 0), 1000).argmin(-1)   # (even codes first)
    v = grid[pick] * torch.where(b < 0, -1.0, 1.0) * pow2(e)[..., None]
    v = torch.where(bad[..., None], float("nan"), v)
    return v.flatten(-2), torch.where(bad, 255, e + 127)


def tiled(scale):
    """Scales [..., rows, d / 32] in the library's layout, 127 behind the last block."""
    n = scale.shape[-1]
    at = torch.full((*scale.shape[:-1], (n + 3) // 4 * 4), 127, dtype=scale.dtype)
    at[..., :n] = scale
    return at.unflatten(-1, (-1, 4)).transpose(-2, -3).contiguous()


def random_mx(shape, seed, low=118, high=126, device="cuda"):
    """Codes, scales and 64-bit values of a random matrix [..., rows, d]: all codes, scales 2^(low - 127) .. 2^(high - 127)."""
    g = torch.Generator().manual_seed(seed)
    *lead, rows, d = shape
    codes = torch.randint(0, 256, (*lead, rows, d // 2), generator=g, dtype=torch.uint8).to(device)
    scale = tiled(torch.randint(low, high + 1, (*lead, rows, d // 32), generator=g, dtype=torch.uint8)).to(device)
    return codes, scale, decode(codes, scale, d)


def scored64(logits, k, scores, bias, groups, top_groups, renorm, scale):
    """mlora_route_scored one token at a time on the host: (expert, weight in 64 bits, token_index, seg_start, position)."""
    T, E = logits.shape
    l = logits.detach().double().cpu()
    l = torch.where(torch.isnan(l), -float("inf"), l)
    if scores == "sigmoid":
        s64 = 1 / (1 + torch.exp(-l))
    else:
        m = l.amax(-1, keepdim=True)
        p = torch.where(l > -float("inf"), torch.where(l == m, 1.0, torch.exp(l - m)), 0.0)
        s64 = p / p.sum(-1, keepdim=True)
    s32 = s64.float()
    c = s32 if bias is None else s32 + bias.float().cpu()
    there = (l > -float("inf")) & ~torch.isnan(c) & (c > -float("inf"))
    per = E // groups
    expert = torch.full((T, k), -1, dtype=torch.int32)
    weight = torch.zeros((T, k), dtype=torch.float64)
    for t in range(T):
        ct, ok = c[t].tolist(), there[t].tolist()
        ranked = []
        for g in range(groups):
            best = sorted((ct[e] for e in range(g * per, (g + 1) * per) if ok[e]), reverse=True)[:2]
            if best:
                total = best[0] if len(best) == 1 else float(torch.tensor(best[0]) + torch.tensor(best[1]))   # (fp32)
                ranked.append((-total, g))
        kept = {g for _, g in sorted(ranked)[:top_groups]}
        among = [e for e in range(E) if ok[e] and (groups == 1 or e // per in kept)]
        chosen = sorted(among, key=lambda e: (-ct[e], e))[:k]
        total = float(s64[t, chosen].sum()) if chosen else 0.0
        for j, e in enumerate(chosen):
            expert[t, j] = e
            w = float(s64[t, e])
            weight[t, j] = scale * ((w / total if float(s32[t, chosen].sum()) > 0 else 0.0) if renorm else w)
    return (expert, weight, *grouped(expert, E))


def grouped(expert, E):
    """(token_index, seg_start, position) of a choice [T, k]."""
    T, k = expert.shape
    flat = expert.reshape(-1).tolist()
    token_index = torch.full((T * k,), -1, dtype=torch.int32)
    position = torch.full((T * k,), -1, dtype=torch.int32)
    by = {}
    for s, e in enumerate(flat):
        by.setdefault(e, []).append(s)
    seg_start, at = [], 0
    for e in range(E):
        seg_start.append(at)
        for s in by.get(e, []):
            token_index[at], position[s] = s // k, at
            at += 1
    seg_start.append(at)
    return token_index, torch.tensor(seg_start, dtype=torch.int32), position.reshape(T, k)
