"""Softmax scores with no bias and one group choose by the logits themselves, as mlora_route: a factor of the weights
alone does not change which experts a token gets, also where scores round to the same fp32 value or to 0."""
import pytest
import torch

from gpu_util import log
from mx_util import grouped
from op_util import U

pytestmark = pytest.mark.gpu


def _logits(T, E):
    g = torch.Generator().manual_seed(T + E)
    l = torch.randn((T, E), generator=g)
    l[0::4] *= 200                                                              # scores that round to 0
    l[1::4] = 0.25 + 2.0 ** -25 * torch.randint(0, 9, l[1::4].shape, generator=g)   # scores 2^-25 apart, relative
    l[2::4] = -0.0
    l[2::4, ::3] = 0.0                                                          # equal logits: the lowest experts
    l[3::4, 1::2] = -float("inf")
    l[3::4, 0] = float("nan")
    l[T // 2] = -float("inf")
    return l


@pytest.mark.parametrize("T,E,k", [(12, 16, 6), (40, 96, 8), (130, 300, 12), (513, 1024, 5)])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("how", [dict(scale=2.5), dict(scores="softmax"), dict(scores="softmax", scale=0.5)])
def test_choices_of_the_logits(T, E, k, renorm, how):
    log(f"[route] T={T} E={E} k={k} renorm={renorm} {how}")
    import rank_adapter_gemm_segmented_amd as ml
    l = _logits(T, E)
    scale = how.get("scale", 1.0)
    got = ml.route(l.cuda(), k, renormalize=renorm, **how)
    plain = ml.route(l.cuda(), k, renormalize=renorm)
    torch.cuda.synchronize()
    key = torch.where(torch.isnan(l), -float("inf"), l)
    top, order = torch.sort(key, dim=-1, descending=True, stable=True)
    top, order = top[:, :k], order[:, :k]
    expert = torch.where(top > -float("inf"), order, -1).int()
    want = (expert, None, *grouped(expert, E))
    for name, g, w, p in zip(("expert", "weight", "token_index", "seg_start", "position"), got, want, plain):
        if name != "weight":
            assert torch.equal(g.cpu(), w) and torch.equal(g, p), name
    p64 = torch.where(key > -float("inf"), torch.exp(key.double() - key.amax(-1, keepdim=True)), 0.0)
    p64 = torch.where(expert >= 0, torch.gather(p64, 1, order), 0.0), p64.sum(-1, keepdim=True)
    w = scale * torch.nan_to_num(p64[0] / (p64[0].sum(-1, keepdim=True) if renorm else p64[1]), nan=0.0)
    # each score rounded once, a sum of k, the division and the factor; below the normal range a step of fp32's smallest
    # (of a score, divided by a sum of at least 1 / E where weights are renormalised)
    assert torch.all((got[1].double().cpu() - w).abs() <= 2 * (k + 4) * U * w + 2.0 ** -126)
