"""Activations where they fade: relative to their value, against 64 bits, on every form that applies an epilogue.

The product is zero (x = 0) and z comes in through the bias, so the only errors are the activation's own. Bounds, with u =
2^-24: an exponential or complementary error function of an argument a that is rounded n times is off by n u |a a'|
relative, a' its logarithmic slope; 40 u more are allowed for the functions themselves (a few units in the last place each,
11 u for the fit that the bf16 forms take), the products and the division. silu: exp(-z), its argument scaled once for the base-2 exponential, n = 2 and |z|. gelu_tanh:
exp(-2 u), u of six roundings and that scaling, n = 8 and |2 u|. gelu: erfc(-z / sqrt 2), n = 2 (the constant, the product)
and a a' <= z^2 + 2. Then one rounding to the output's type.
"""
import pytest
import torch

from gpu_util import log
from op_util import U, half_step, normal

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _ml():
    import rank_adapter_gemm_segmented_amd as ml
    return ml


def _exact(z, act):
    """The activation in 64 bits, without cancellation, and its relative bound."""
    if act == "silu":
        return z / (1 + torch.exp(-z)), (2 * z.abs() + 40) * U
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z / 2 ** 0.5), (2 * (z * z + 2) + 40) * U
    t = 2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3)
    return z / (1 + torch.exp(-t)), (8 * t.abs() + 40) * U


def _values(n, dtype):
    """n values of z from -9 up to 3, in dtype."""
    return torch.linspace(-9, 3, n).to(dtype).cuda()


def _check(y, z, act, gated, what):
    """Every row of y is the activation of z."""
    want, rel = _exact(z.double(), act)
    if gated:      # an up row of 1: one more rounding of nothing
        rel = rel + U
    off = (y.double() - want).abs() / want.abs().clamp(min=1e-300)
    lim = rel + half_step(y.dtype) * (1 + rel)
    bad = (off > lim) & (want != 0)
    assert not bad.any(), f"{what} {act}: relative error {float(off[bad].max()):.3g} at z = {float(z.expand_as(y)[bad][0]):.4f}"
    assert torch.all(y[..., want == 0] == 0)


# rows of the layer, its type: the decode pair, the wide stream, tiles of 64x128, 128x128, 64x256 and 256x256 (the last by
# width and tokens), and fp32 fused and not
LAYERS = [("decode", BF16, 3, 264, 250, 0), ("decode 64", BF16, 64, 264, 250, 0), ("wide", BF16, 2, 72, 16450, 0),
          ("64x128", BF16, 130, 72, 250, 0), ("128x128", BF16, 100, 72, 24640, 0), ("64x256", BF16, 257, 72, 6402, 0),
          ("256x256", BF16, 1100, 72, 12290, 0), ("f32 fused", F32, 5, 64, 250, 1), ("f32", F32, 70, 260, 1026, 0),
          ("FP8", BF16, 20, 64, 250, 2)]


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("i", range(len(LAYERS)), ids=[l[0].replace(" ", "_") for l in LAYERS])
def test_layer(i, gated, act):
    name, dtype, T, d_in, n, kind = LAYERS[i]
    log(f"[tails] layer {name} {act} gated={gated}")
    ml = _ml()
    z = _values(n, dtype)
    d_out = 2 * n if gated else n
    bias = torch.cat([z, torch.ones_like(z)]) if gated else z
    pool = ml.Pool(d_in, d_out, dtype, 8, 1)
    x, scale = torch.zeros((T, d_in), dtype=dtype, device="cuda"), None
    W = torch.zeros((d_out, d_in), dtype=dtype, device="cuda")
    if kind == 2:
        W, scale = W.to(torch.uint8), torch.ones(d_out, device="cuda")
    seg = {}
    if kind == 1:      # (the fused form needs an adapter; its term is zero)
        pool.register(0, normal((8, d_in), 1, 1.0, dtype), torch.zeros((d_out, 8), dtype=dtype, device="cuda"))
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        seg = dict(seg_start=i32([0, T]), seg_adapter=i32([0]), seg_rank=i32([8]), seg_scale=torch.ones(1, device="cuda"))
    y = ml.linear_epilogue(x, W, pool, lora_on=int(kind == 1), bias=bias, act=act, gated=gated, w_scale=scale, **seg)
    torch.cuda.synchronize()
    _check(y, z, act, gated, name)


# streamed, in tiles of 32, 64, 128 and 256 positions, fp32, FP8 streamed and tiled
EXPERTS = [("stream", BF16, [2, 0, 1], 72, 250, False), ("32", BF16, [5] * 16, 72, 2056, False), ("64", BF16, [30] * 16, 72, 2056, False),
           ("128", BF16, [100] * 16, 72, 2056, False), ("256", BF16, [200] * 16, 72, 2056, False), ("f32", F32, [3, 0, 20], 64, 250, False),
           ("FP8 stream", BF16, [3, 9], 64, 250, True), ("FP8 64", BF16, [30] * 16, 64, 2056, True)]


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("i", range(len(EXPERTS)), ids=[e[0].replace(" ", "_") for e in EXPERTS])
def test_experts(i, gated, act):
    name, dtype, counts, d_in, n, fp8 = EXPERTS[i]
    log(f"[tails] experts {name} {act} gated={gated}")
    ml = _ml()
    E, P, d_out = len(counts), sum(counts), 2 * n if gated else n
    z = _values(n, dtype)
    bias = (torch.cat([z, torch.ones_like(z)]) if gated else z).expand(E, d_out).contiguous()
    start = torch.tensor([sum(counts[:e]) for e in range(E + 1)], dtype=torch.int32, device="cuda")
    x = torch.zeros((P, d_in), dtype=dtype, device="cuda")
    W = torch.zeros((E, d_out, d_in), dtype=torch.uint8 if fp8 else dtype, device="cuda")
    y = ml.experts_linear(x, W, start, bias=bias, act=act, gated=gated, w_scale=torch.ones((E, d_out), device="cuda") if fp8 else None)
    torch.cuda.synchronize()
    _check(y, z, act, gated, name)
