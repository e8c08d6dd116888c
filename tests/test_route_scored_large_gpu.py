"""mlora_route_scored at its largest batches: all of MLORA_MAX_POSITIONS, and the most experts, groups and choices."""
import pytest
import torch

from gpu_util import log
from op_util import U

pytestmark = pytest.mark.gpu


def _expected(logits, k, scores, bias, groups, top_groups, scale):
    """(expert, weight in 64 bits) of mlora_route_scored without renormalising, a batch at a time in 64 bits."""
    T, E = logits.shape
    l = logits.double()
    s64 = 1 / (1 + torch.exp(-l)) if scores == "sigmoid" else torch.softmax(l, -1)
    c = s64.float() + bias
    if groups > 1:
        two = torch.topk(c.view(T, groups, -1), min(2, E // groups), dim=-1).values
        rank = two.sum(-1) if two.shape[-1] == 2 else two[..., 0]
        kept = torch.sort(rank, dim=-1, descending=True, stable=True).indices[:, :top_groups]
        mask = torch.zeros((T, groups), dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        c = torch.where(mask.repeat_interleave(E // groups, 1), c, -float("inf"))
    expert = torch.sort(c, dim=-1, descending=True, stable=True).indices[:, :k]
    return expert.int(), scale * torch.gather(s64, 1, expert)


@pytest.mark.parametrize("T,E,k,groups,top,scores", [(1 << 17, 1024, 64, 64, 16, "sigmoid"), (1 << 17, 1024, 64, 1, 1, "softmax"),
                                                     (1 << 20, 8, 8, 4, 4, "sigmoid"), (1 << 20, 12, 2, 2, 1, "softmax")])
def test_largest(T, E, k, groups, top, scores):
    log(f"[route scored] largest T={T} E={E} k={k} groups={groups}/{top} {scores}")
    import rank_adapter_gemm_segmented_amd as ml
    g = torch.Generator(device="cuda")
    g.manual_seed(E)
    # (the two sides' 64-bit scores differ in their last places, which round to other fp32 values for one in 2^28 or so,
    # and change a choice only next to a sum within a step of it: none for these seeds)
    logits = torch.randn((T, E), generator=g, device="cuda").bfloat16()
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    expert, weight, token_index, seg_start, position = ml.route(logits, k, renormalize=False, scores=scores, bias=bias, n_groups=groups,
                                                                top_groups=top, scale=2.5)
    torch.cuda.synchronize()
    step = 1 << 14
    for t in range(0, T, step):
        e, w = _expected(logits[t:t + step], k, scores, bias, groups, top, 2.5)
        assert torch.equal(expert[t:t + step], e), t
        assert torch.all((weight[t:t + step].double() - w).abs() <= 4 * U * w), t   # (a rounding each of score and factor)
    flat = expert.view(-1).long()
    order = torch.sort(flat, stable=True).indices
    assert torch.equal(token_index, (order // k).int())
    want = torch.empty_like(order)
    want[order] = torch.arange(T * k, device="cuda")
    assert torch.equal(position.view(-1), want.int())
    assert torch.equal(seg_start[1:], torch.cumsum(torch.bincount(flat, minlength=E), 0).int()) and int(seg_start[0]) == 0
