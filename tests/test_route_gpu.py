"""mlora_route: top-k choice, weights and segments against a token-by-token reference in 64 bits."""
import pytest
import torch

from gpu_util import log
from op_util import U, route64

pytestmark = pytest.mark.gpu


def _ml():
    import rank_adapter_gemm_segmented_amd as ml
    return ml


def _check(logits, k, renorm):
    got = _ml().route(logits, k, renormalize=renorm)
    torch.cuda.synchronize()
    want = route64(logits, k, renorm)
    for name, g, w in zip(("expert", "weight", "token_index", "seg_start", "position"), got, want):
        if name == "weight":
            # exp of a difference d is off by about (|d| + 2) u relative (d is rounded once), the sum of E terms by
            # E u, the division by u; |d| counts only while exp(d) matters, up to 104
            err = (g.double().cpu() - w).abs()
            assert torch.all(err <= (2 * (104 + logits.shape[1]) + 8) * U * w + 1e-37), name
        else:
            assert torch.equal(g.cpu(), w), name


SIZES = [(1, 1, 1), (1, 8, 2), (3, 5, 5), (16, 64, 8), (64, 128, 8), (65, 129, 7), (100, 3, 1), (63, 64, 64),
         (1000, 60, 6), (257, 1024, 32), (4096, 64, 8), (4500, 17, 3)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sizes(T, E, k, dtype):
    log(f"[route] T={T} E={E} k={k} {dtype}")
    g = torch.Generator().manual_seed(T * 131 + E)
    logits = torch.randn((T, E), generator=g).to(dtype).cuda()   # (bf16: many ties)
    _check(logits, k, renorm=(T + k) % 2 == 0)


@pytest.mark.parametrize("T", [5, 64, 200])
@pytest.mark.parametrize("renorm", [True, False])
def test_masked_tied_and_infinite(T, renorm):
    log(f"[route] special values T={T}")
    E, k, inf = 12, 4, float("inf")
    g = torch.Generator().manual_seed(T)
    l = torch.randn((T, E), generator=g)
    l[0] = -inf                                     # a padded token
    l[1] = 0.0                                      # all equal: the first k experts
    l[1, 3] = -0.0                                  # ... -0 among them
    l[2] = float("nan")
    l[2, 7] = 1.0                                   # one logit that counts
    l[3, ::2] = inf                                 # infinite logits share the weight
    l[4] = torch.finfo(torch.float32).min           # a mask of the lowest value: still a choice
    l[4, 5] = 0.0
    if T > 64:
        l[T - 70:] = -inf                           # a padded end over several blocks
    _check(l.cuda(), k, renorm)


def test_everything_masked():
    log("[route] nothing to choose")
    for T in (7, 300):
        _check(torch.full((T, 6), float("-inf")).cuda(), 2, True)


def test_one_expert_takes_all():
    log("[route] one expert")
    l = torch.zeros((700, 9))
    l[:, 4] = 5.0
    _check(l.cuda(), 1, True)


def test_no_tokens():
    log("[route] no tokens")
    ml = _ml()
    expert, weight, token_index, seg_start, position = ml.route(torch.empty((0, 5), device="cuda"), 2)
    torch.cuda.synchronize()
    assert seg_start.tolist() == [0] * 6 and expert.numel() == weight.numel() == token_index.numel() == position.numel() == 0


def test_graph_and_streams():
    log("[route] captured and replayed, on another stream")
    ml = _ml()
    logits = torch.randn((300, 32), device="cuda")
    ws, out = ml.route_workspace(300, 32, 4), ml.route(logits, 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        ml.route(logits, 4, out=out, workspace=ws)
    for i in range(3):
        logits.copy_(torch.randn((300, 32), generator=torch.Generator().manual_seed(i)))
        graph.replay()
        torch.cuda.synchronize()
        eager = ml.route(logits, 4)
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert torch.equal(a, b)


def test_refusals():
    log("[route] refusals")
    ml = _ml()
    l = torch.zeros((4, 8), device="cuda")
    for bad in (lambda: ml.route(l, 0), lambda: ml.route(l, 9), lambda: ml.route(torch.zeros((1, 1025), device="cuda"), 2),
                lambda: ml.route(torch.zeros((100, 8), device="cuda"), 2, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ml.MloraError):
            bad()
    with pytest.raises(TypeError):
        ml.route(l.half(), 2)
    for bad in (lambda: ml.route(l[0], 1), lambda: ml.route(l.T, 2), lambda: ml.route(l.cpu(), 2)):
        with pytest.raises(ValueError):
            bad()
