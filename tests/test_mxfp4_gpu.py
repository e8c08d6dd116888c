"""mlora_quantize_mxfp4 and mlora_dequantize_mxfp4: every code, scale and value, exactly."""
import pytest
import torch

from gpu_util import log
from mx_util import decode, encode, random_mx, tiled

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _ml():
    import rank_adapter_gemm_segmented_amd as ml
    return ml


def _same(a, b):
    a, b = a.double().cpu(), b.double().cpu()
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(nan=7.0), b.nan_to_num(nan=7.0))


def _check(x):
    ml = _ml()
    codes, scale = ml.quantize_mxfp4(x)
    back = ml.dequantize_mxfp4(codes, scale, x.dtype)
    wide = ml.dequantize_mxfp4(codes, scale, torch.float32)
    torch.cuda.synchronize()
    v, s = encode(x.reshape(-1, x.shape[-1]))
    s = s.reshape(*x.shape[:-1], -1).to(torch.uint8)
    v = v.reshape(x.shape)
    assert torch.equal(scale.cpu(), tiled(s)), "scales"
    assert _same(decode(codes, scale, x.shape[-1]), v), "codes"
    assert _same(wide, v), "values in fp32"
    assert _same(back, v), "values in the type of x"
    bad = (s == 255).repeat_interleave(16, -1)
    assert torch.all(codes.cpu()[bad] == 0)


SHAPES = [(1, 32), (1, 4096), (3, 96), (16, 128), (17, 160), (33, 544), (130, 1056), (257, 32), (1000, 416)]


@pytest.mark.parametrize("kind", DT)
@pytest.mark.parametrize("rows,d", SHAPES)
def test_shapes(kind, rows, d):
    log(f"[mxfp4] {kind} {rows}x{d}")
    g = torch.Generator().manual_seed(rows + d)
    x = torch.randn((rows, d), generator=g) * torch.exp(2 * torch.randn((rows, 1), generator=g))
    _check(x.to(DT[kind]).cuda())


@pytest.mark.parametrize("kind", DT)
def test_batches(kind):
    log(f"[mxfp4] batches {kind}")
    g = torch.Generator().manual_seed(5)
    _check(torch.randn((3, 2, 21, 192), generator=g).to(DT[kind]).cuda())


@pytest.mark.parametrize("kind", DT)
def test_ties_and_borders(kind):
    """Every midpoint of two values, its neighbours on both sides, and what lies past the largest, at many exponents."""
    log(f"[mxfp4] ties {kind}")
    dt = DT[kind]
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    step = torch.finfo(dt).eps * 2
    v = torch.cat([torch.tensor([0.0, 6.0, 7.0, 7.9, 4.0]), mid, mid * (1 + step), mid * (1 - step)])
    v = torch.cat([v, torch.zeros(32 - v.numel())])            # 26 values and zeros; the largest lies in [4, 8)
    rows = torch.stack([torch.cat([v, -v, v.flip(0), -v]) * 2.0 ** e for e in range(-100, 101, 5)])
    _check(rows.to(dt).cuda())


def test_smallest_and_largest():
    log("[mxfp4] subnormals and the largest")
    x = torch.zeros((6, 128))
    x[0, 5] = 2.0 ** -149                                      # subnormal: far below half of the smallest value
    x[1, :40] = 2.0 ** -128                                    # a subnormal that is a value: 0.5 2^-127
    x[2, 3], x[2, 4] = 2.0 ** -126, 1.5 * 2.0 ** -127
    x[3, :] = torch.finfo(torch.float32).max
    x[4, 64:] = -torch.finfo(torch.float32).max
    x[4, 65] = 2.0 ** 100
    x[5, ::2] = 2.0 ** -125
    _check(x.cuda())


@pytest.mark.parametrize("kind", DT)
def test_nan_and_infinity(kind):
    log(f"[mxfp4] NaN and infinity {kind}")
    g = torch.Generator().manual_seed(9)
    x = torch.randn((20, 224), generator=g)
    x[0, 0], x[1, 33], x[2, 223], x[3, 100], x[3, 101] = float("nan"), float("inf"), -float("inf"), float("inf"), float("nan")
    x[4] = float("nan")
    _check(x.to(DT[kind]).cuda())


def test_every_scale_and_code_back():
    """All 256 scales by all 16 codes; bf16 has no values from 2^128 on."""
    log("[mxfp4] every scale")
    ml = _ml()
    codes = torch.arange(256, dtype=torch.uint8).reshape(1, 256).repeat(256, 1)        # 512 columns: every pair of codes
    scale = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 16)
    c, s = codes.cuda(), tiled(scale).cuda()
    want = decode(c, s, 512).cpu()
    wide, half = ml.dequantize_mxfp4(c, s, torch.float32), ml.dequantize_mxfp4(c, s)
    torch.cuda.synchronize()
    past = want.abs() >= 2.0 ** 128
    want = torch.where(past, torch.sign(want) * float("inf"), want)
    assert _same(wide, want) and _same(half, want)


def test_scales_in_rows():
    log("[mxfp4] layout of row-major scales")
    ml = _ml()
    s = torch.randint(0, 255, (3, 7, 9), dtype=torch.uint8)
    assert torch.equal(ml.mxfp4_scale_layout(s.cuda()).cpu(), tiled(s))


def test_outputs_stay_inside():
    """Guards around both outputs; empty matrices do nothing."""
    log("[mxfp4] guards")
    ml = _ml()
    x = torch.randn((19, 160), device="cuda")
    cb, sb = torch.full((19 * 80 + 512,), 9, dtype=torch.uint8, device="cuda"), torch.full((2 * 19 * 4 + 512,), 9, dtype=torch.uint8, device="cuda")
    ml.quantize_mxfp4(x, out=(cb[256:256 + 19 * 80].view(19, 80), sb[256:256 + 152].view(2, 19, 4)))
    torch.cuda.synchronize()
    for b, n in ((cb, 19 * 80), (sb, 152)):
        assert torch.all(b[:256] == 9) and torch.all(b[256 + n:] == 9)
    codes, scale = ml.quantize_mxfp4(torch.empty((0, 64), device="cuda"))
    assert codes.shape == (0, 32) and scale.shape == (1, 0, 4) and ml.dequantize_mxfp4(codes, scale).shape == (0, 64)


def test_refusals():
    log("[mxfp4] refusals")
    ml = _ml()
    x = torch.zeros((4, 64), device="cuda")
    codes, scale, _ = random_mx((4, 64), 0)
    with pytest.raises(ml.MloraError) as e:
        ml.quantize_mxfp4(torch.zeros((4, 48), device="cuda"))
    assert e.value.name == "MLORA_ERR_SHAPE"
    for bad in (lambda: ml.quantize_mxfp4(x.half()), lambda: ml.quantize_mxfp4(x[0]), lambda: ml.quantize_mxfp4(x.t()),
                lambda: ml.quantize_mxfp4(x, out=(codes[:3], scale)), lambda: ml.dequantize_mxfp4(codes, scale[:, :3]),
                lambda: ml.dequantize_mxfp4(codes, scale, torch.float16), lambda: ml.dequantize_mxfp4(codes.int(), scale),
                lambda: ml.quantize_mxfp4(x.cpu()), lambda: ml.mxfp4_scale_layout(scale.int())):
        with pytest.raises((TypeError, ValueError)):
            bad()
