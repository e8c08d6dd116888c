"""Tiled expert products with more experts than a wave scans at a time, and rows of odd width."""
import pytest
import torch

from gpu_util import log
from test_experts_forms_gpu import _spread, _way_back
from test_experts_gpu import _product

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kind,E,mean", [("bf16", 100, 6), ("bf16", 70, 30), ("bf16", 70, 100), ("bf16", 70, 200), ("fp8w", 70, 30)])
def test_more_than_64_experts(kind, E, mean, gated):
    log(f"[experts] {E} experts of about {mean} rows, {kind} gated={gated}")
    counts = _spread(E, mean)
    counts[3], counts[63], counts[64], counts[65] = 0, 1, 0, counts[63] + counts[64]
    _product(kind, counts, 80, 520, "silu", gated, bias=True, seed=E)


@pytest.mark.parametrize("kind,E,mean,d_out", [("bf16", 16, 5, 2055), ("bf16", 16, 30, 2055), ("bf16", 16, 100, 2053),
                                               ("bf16", 16, 201, 4101), ("fp8w", 16, 30, 2055), ("fp8w", 16, 100, 2053)])
def test_odd_widths(kind, E, mean, d_out):
    log(f"[experts] about {mean} rows per expert, {kind}, {d_out} columns")
    counts = _spread(E, mean)
    _product(kind, counts, 272, d_out, "gelu", False, bias=True, seed=1)
    _product(kind, counts, 272, 2 * d_out, "silu", True, bias=True, seed=2)
    _way_back(kind, counts, 272, d_out)
