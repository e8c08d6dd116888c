"""References in 64 bits, with error bounds, for the epilogue, routing and expert operators.

Bounds count roundings. A sum of K products in fp32, in any order, is off by at
most K u S with u = 2^-24 and S the sum of the products' absolute values; twice
that is allowed (a result is accumulated in partial sums that are themselves
added). An activation of this library has slope at most 1.13 and its own error
is below 2^-20 of its argument. The result is rounded once, by at most half a
step: eps / 2 relative to it.
"""
import torch

U = 2.0 ** -24
SLOPE = 1.2          # > the steepest slope of relu, silu, gelu (1.13)
ACT_ERR = 2.0 ** -20


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def normal(shape, seed, sigma=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g) * sigma).to(dtype).cuda()


def act64(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z / 2 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    return z


def product64(x, W):
    """x W^T in 64 bits and the bound of its fp32 error."""
    x, W = x.double(), W.double()
    return x @ W.T, 2 * x.shape[1] * U * (x.abs() @ W.abs().T)


def epilogue64(z, dz, act, gated, bias, residual):
    """y and its bound before the rounding, from z and z's bound."""
    if bias is not None:
        z = z + bias.double()
        dz = dz + U * z.abs()

    def activated(z, dz):
        return act64(z, act), (SLOPE * dz + ACT_ERR * z.abs() if act != "none" else dz)

    if gated:
        half = z.shape[-1] // 2
        g, dg = activated(z[..., :half], dz[..., :half])
        u, du = z[..., half:], dz[..., half:]
        z, dz = g * u, dg * u.abs() + g.abs() * du + dg * du + U * (g * u).abs()
    else:
        z, dz = activated(z, dz)
    if residual is not None:
        z = z + residual.double()
        dz = dz + U * (z.abs() + residual.double().abs())
    return z, dz


def check(y, ref, bound, what):
    """Every element of y within bound + half a step of its type of ref."""
    assert torch.isfinite(y).all(), f"{what}: not finite"
    err = (y.double() - ref).abs()
    lim = bound + half_step(y.dtype) * (ref.abs() + bound) + 1e-30
    worst = float((err / lim).max()) if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: error / bound {worst:.3f}"
    return worst


def e4m3(W):
    """Codes and row scales of a weight [..., d_in]; and the weight they stand for."""
    scale = (W.abs().amax(-1).float() / 448).clamp(min=1e-12)
    codes = (W.float() / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, scale, codes.view(torch.float8_e4m3fn).double() * scale.double()[..., None]


def route64(logits, k, renorm):
    """The routing of a batch, one token at a time on the host: (expert, weight, token_index, seg_start, position)."""
    T, E = logits.shape
    rows = logits.detach().double().cpu().tolist()
    expert = torch.full((T, k), -1, dtype=torch.int32)
    weight = torch.zeros((T, k), dtype=torch.float64)
    inf = float("inf")
    for t, row in enumerate(rows):
        there = [e for e in range(E) if row[e] > -inf]
        chosen = sorted(there, key=lambda e: (-row[e], e))[:k]
        if not chosen:
            continue
        m = row[chosen[0]]
        p = {e: 1.0 if row[e] == m else float(torch.exp(torch.tensor(row[e] - m, dtype=torch.float64))) for e in there}
        total = sum(p[e] for e in (chosen if renorm else there))
        for j, e in enumerate(chosen):
            expert[t, j] = e
            weight[t, j] = p[e] / total
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
    return expert, weight, token_index, torch.tensor(seg_start, dtype=torch.int32), position.reshape(T, k)
