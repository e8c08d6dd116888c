"""mlora_route where its launches are largest or change form."""
import pytest
import torch

from gpu_util import log
from test_route_gpu import _check

pytestmark = pytest.mark.gpu


# the largest launch of one workgroup (102 KB of LDS), both sides of its limit of 128 tokens, more than 256 experts or 16
# choices in it, and 65 to 256 experts, and 17 choices, in two launches
@pytest.mark.parametrize("T,E,k", [(1, 1024, 64), (128, 1024, 64), (129, 1024, 64), (128, 256, 16), (129, 256, 16), (100, 257, 3),
                                   (100, 200, 17), (500, 128, 8), (500, 256, 16), (300, 100, 17)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_largest_forms(T, E, k, dtype):
    log(f"[route] T={T} E={E} k={k} {dtype}")
    g = torch.Generator().manual_seed(T + E)
    _check(torch.randn((T, E), generator=g).to(dtype).cuda(), k, renorm=(T + E) % 2 == 0)
