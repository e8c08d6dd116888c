"""Every streamed form of the expert products, and the tiled FP8 way back, against 64 bits.

The form goes by the rows per expert and by how many items fill the card: 16, 32 or 64 positions an item; 64 rows and 4
waves, or 32 rows and 8 waves where items are few. The sizes here are picked for the forms, each named.
"""
import pytest
import torch

from gpu_util import log
from op_util import U, check, epilogue64, normal, product64
from test_experts_gpu import DT, _ml, _product, _segments, _weight

pytestmark = pytest.mark.gpu


def _spread(E, mean, seed=1):
    """E counts around the mean, of that sum, none of them 0."""
    g = torch.Generator().manual_seed(seed)
    c = [max(1, mean + int(torch.randint(-mean // 2, mean // 2 + 1, (1,), generator=g))) for _ in range(E - 1)]
    return c + [max(1, E * mean - sum(c))]


ONE_OR_TWO = [1 + e % 2 for e in range(130)]
FORMS = {
    # 4 waves
    "bf16 4x1": ("bf16", ONE_OR_TWO, 72, 1032), "bf16 4x2": ("bf16", _spread(16, 6), 136, 1264),
    "bf16 4x4": ("bf16", [252], 136, 5504),
    "FP8 4x1": ("fp8w", _spread(16, 8), 272, 2064), "FP8 4x2": ("fp8w", _spread(16, 15), 272, 2064), "FP8 4x4": ("fp8w", [252], 144, 5504),
    "f32 4x1": ("f32", ONE_OR_TWO, 68, 1032), "f32 4x2": ("f32", _spread(16, 15), 264, 1040), "f32 4x4": ("f32", _spread(8, 60), 264, 2056),
    # 8 waves
    "bf16 8x1": ("bf16", [2, 0, 1, 4], 1096, 250), "bf16 8x2": ("bf16", _spread(4, 15), 1096, 250), "bf16 8x4": ("bf16", _spread(4, 60), 1096, 250),
    "FP8 8x1": ("fp8w", _spread(4, 6), 1104, 250), "FP8 8x2": ("fp8w", _spread(4, 15), 1104, 250), "FP8 8x4": ("fp8w", _spread(4, 60), 1104, 250),
    "f32 8x1": ("f32", [2, 0, 1, 4], 1092, 250), "f32 8x2": ("f32", _spread(4, 15), 1092, 250), "f32 8x4": ("f32", _spread(4, 60), 1092, 250),
}
IDS = [f.replace(" ", "_") for f in FORMS]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("form", FORMS, ids=IDS)
def test_streamed(form, gated):
    log(f"[experts] streamed {form} gated={gated}")
    kind, counts, d_in, d_out = FORMS[form]
    _product(kind, counts, d_in, d_out, "silu" if gated else "gelu", gated, bias=True, seed=len(counts))


def _way_back(kind, counts, d_in, d_out):
    """One expert per token: token t's row sits at position t."""
    ml, T, E = _ml(), sum(counts), len(counts)
    W, scale, W64 = _weight(E, d_out, d_in, kind, 1)
    h, b, res = normal((T, d_in), 2, 1.0, DT[kind]), normal((E, d_out), 3, 0.5, DT[kind]), normal((T, d_out), 4, 1.0, DT[kind])
    w = torch.rand((T, 1), generator=torch.Generator().manual_seed(5)).cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda").reshape(T, 1)
    y = ml.experts_combine(h, W, _segments(counts), pos, w, bias=b, residual=res, w_scale=scale)
    torch.cuda.synchronize()
    at = 0
    for e, c in enumerate(counts):
        p = slice(at, at + c)
        z, dz = epilogue64(*product64(h[p], W64[e]), "none", False, b[e], None)
        wz = w[p].double() * z
        bound = w[p].double() * dz + 3 * U * (wz.abs() + res[p].double().abs())
        check(y[p], wz + res[p].double(), bound, f"{kind} way back, expert {e} ({c} rows)")
        at += c


@pytest.mark.parametrize("form", FORMS, ids=IDS)
def test_way_back(form):
    log(f"[experts] way back, streamed {form}")
    _way_back(*FORMS[form])


@pytest.mark.parametrize("mean,d_out", [(30, 2056), (30, 2062), (100, 2056)])
def test_way_back_of_fp8_tiles(mean, d_out):
    log(f"[experts] way back, FP8 tiles, {mean} rows per expert, {d_out} columns")
    _way_back("fp8w", _spread(16, mean), 272, d_out)
