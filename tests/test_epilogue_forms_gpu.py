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


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,fp8,d_out", [(20, False, 192), (5, True, 192), (20, True, 192), (64, True, 192), (3, False, 16448), (3, True, 16448)])
def test_fused_pools_of_a_few_tokens(T, fp8, d_out, gated):
    log(f"[epilogue] fused pool, {T} tokens, 264 -> {d_out}, fp8={fp8} gated={gated}")
    layer = Layer(torch.bfloat16, T, 272, d_out, gated, seed=3, ranks=(16, 16), fused=True, fp8=fp8, max_run=3)
    layer.check("silu")
