"""A forced path that has no form with an epilogue leaves the choice as it is."""
import pytest
import torch

from gpu_util import log
from test_epilogue_gpu import Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,path", [(16, "path=decode "), (200, "path=gemm")])
def test_gemv_with_an_epilogue(T, path, monkeypatch, capfd):
    log(f"[epilogue] MLORA_FORCE_PATH=gemv, T={T}")
    layer = Layer(torch.bfloat16, T, 256, 192, False, seed=1)
    y = layer.run("silu")
    monkeypatch.setenv("MLORA_FORCE_PATH", "gemv")
    monkeypatch.setenv("MLORA_LOG", "1")
    capfd.readouterr()
    forced = layer.run("silu")
    err = capfd.readouterr().err
    assert path in err, err
    assert torch.equal(forced, y)
