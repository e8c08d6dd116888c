"""mlora_route takes a workspace of what its own launches use, 4 bytes per expert and block of 32 tokens, also where
mlora_route_workspace_bytes, which covers mlora_route_scored too, gives more."""
import pytest
import torch

from gpu_util import log

pytestmark = pytest.mark.gpu


def _own_bytes(T, E):
    blocks = min((T + 31) // 32, 256)
    return (max(blocks * E * 4, 1) + 255) // 256 * 256


@pytest.mark.parametrize("T,E,k", [(1, 3, 1), (64, 256, 8), (128, 1024, 4), (129, 64, 8), (4096, 256, 8), (8193, 100, 2)])
def test_a_workspace_of_its_own_size(T, E, k):
    log(f"[route] own workspace T={T} E={E} k={k}")
    import rank_adapter_gemm_segmented_amd as ml
    logits = torch.randn((T, E), generator=torch.Generator().manual_seed(T)).cuda()
    n = _own_bytes(T, E)
    assert n <= ml.route_workspace(T, E, k).numel()
    want = ml.route(logits, k)
    buf = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    got = ml.route(logits, k, workspace=buf[:n])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.all(buf[n:] == 0xA5), "written behind the workspace"
    with pytest.raises(ml.MloraError) as e:
        ml.route(logits, k, workspace=buf[:n - 1])
    assert e.value.name == "MLORA_ERR_WORKSPACE"


def test_by_scores_it_takes_what_the_query_gives():
    log("[route] workspace by scores")
    import rank_adapter_gemm_segmented_amd as ml
    logits = torch.randn((64, 256), device="cuda")
    n = ml.library().mlora_route_workspace_bytes(64, 256, 8)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    want = ml.route(logits, 8, scores="sigmoid")
    got = ml.route(logits, 8, scores="sigmoid", workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(ml.MloraError) as e:
        ml.route(logits, 8, scores="sigmoid", workspace=ws[:n - 1])
    assert e.value.name == "MLORA_ERR_WORKSPACE"
