"""Forms of the layer with an epilogue that take particular sizes: W marked as read once (33 to 64 tokens, d_in above 8192),
and the dense adapter term in tiles of 64x256."""
import pytest
import torch

from gpu_util import log
from test_epilogue_gpu import Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_long_rows(fp8, gated):
    log(f"[epilogue] 40 tokens, d_in 8208, fp8={fp8} gated={gated}")
    layer = Layer(torch.bfloat16, 40, 8208, 130, gated, seed=1, fp8=fp8, shuffled=True)
    layer.check("silu")
    layer.check("gelu", lora_on=0)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("form", ["dense", "mfma"])
def test_adapter_term_in_64x256_tiles(form, gated, monkeypatch):
    log(f"[epilogue] 257 tokens, 264 -> 6400, adapter term {form}, gated={gated}")
    monkeypatch.setenv("MLORA_EXPAND", form)
    Layer(torch.bfloat16, 257, 264, 6400, gated, seed=2, shuffled=True).check("silu")
