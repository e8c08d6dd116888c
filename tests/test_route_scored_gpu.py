"""mlora_route_scored: choices by biased scores among the best groups, against a token-by-token reference in 64 bits."""
import pytest
import torch

from gpu_util import log
from mx_util import scored64
from op_util import U

pytestmark = pytest.mark.gpu


def _ml():
    import rank_adapter_gemm_segmented_amd as ml
    return ml


def _check(logits, k, scores, bias, groups, top_groups, renorm, scale):
    got = _ml().route(logits, k, renormalize=renorm, scores=scores, bias=bias, n_groups=groups, top_groups=top_groups, scale=scale)
    torch.cuda.synchronize()
    want = scored64(logits, k, scores, bias, groups, top_groups, renorm, scale)
    for name, g, w in zip(("expert", "weight", "token_index", "seg_start", "position"), got, want):
        if name == "weight":
            # each score rounded once; a sum of k, the division and the factor (k + 2 more, k of them relative to the sum);
            # and below the normal range a step of fp32's smallest
            err = (g.double().cpu() - w).abs()
            assert torch.all(err <= 2 * (k + 4) * U * w + 2.0 ** -126), name
        else:
            assert torch.equal(g.cpu(), w), name


SIZES = [(1, 1, 1, 1, 1), (1, 8, 2, 2, 1), (3, 6, 3, 6, 3), (16, 64, 8, 8, 4), (64, 256, 8, 8, 4), (65, 160, 6, 8, 3), (100, 3, 1, 1, 1),
         (63, 64, 64, 1, 1), (1000, 60, 6, 4, 2), (130, 1024, 32, 64, 20), (129, 1008, 5, 63, 5), (4096, 256, 8, 8, 4), (300, 64, 40, 2, 2),
         (200, 128, 2, 64, 1)]


@pytest.mark.parametrize("T,E,k,groups,top", SIZES)
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sizes(T, E, k, groups, top, scores, dtype):
    log(f"[route scored] T={T} E={E} k={k} groups={groups}/{top} {scores} {dtype}")
    g = torch.Generator().manual_seed(T * 131 + E)
    logits = (2 * torch.randn((T, E), generator=g)).to(dtype).cuda()   # (bf16: many ties)
    bias = 0.1 * torch.randn(E, generator=g).cuda() if (T + E) % 2 else None
    _check(logits, k, scores, bias, groups, top, renorm=(T + k) % 2 == 0, scale=1.0 if T % 3 else 2.5)


@pytest.mark.parametrize("T", [9, 64, 200])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top", [(1, 1), (4, 2), (12, 5), (2, 2)])
def test_masked_tied_and_infinite(T, scores, groups, top):
    log(f"[route scored] special values T={T} {scores} groups={groups}/{top}")
    E, k, inf = 12, 4, float("inf")
    g = torch.Generator().manual_seed(T)
    l = torch.randn((T, E), generator=g)
    l[0] = -inf                                     # a padded token
    l[1] = 0.0                                      # all equal: the first of the first groups
    l[1, 3] = -0.0
    l[2] = float("nan")
    l[2, 7] = 1.0                                   # one logit that counts
    l[3, ::2] = inf
    l[4] = torch.finfo(torch.float32).min           # a mask of the lowest value: still a choice
    l[4, 5] = 0.0
    l[5] = torch.finfo(torch.float32).min           # scores of 0 (sigmoid): chosen, weight 0
    l[6, :11] = -inf                                # one expert left
    l[7] = 40.0 + l[7]                              # scores that round to 1 (sigmoid): ties
    l[8] = -inf
    l[8, 2], l[8, 10] = -3.0, -4.0                  # groups of one expert each
    if T > 64:
        l[T - 70:] = -inf                           # a padded end over several blocks
    k = min(k, top * (E // groups))
    bias = 0.2 * torch.randn(E, generator=g)
    for renorm in (True, False):
        _check(l.cuda(), k, scores, None, groups, top, renorm, 1.5)
        _check(l.cuda(), k, scores, bias.cuda(), groups, top, renorm, 1.0)
        wild = bias.clone()
        wild[1], wild[4], wild[9], wild[11] = inf, -inf, float("nan"), -50.0
        _check(l.cuda(), k, scores, wild.cuda(), groups, top, renorm, 1.0)


def test_near_scores():
    """Neighbouring logits whose scores round to the same fp32 or to neighbours: the order is that of the rounded sums."""
    log("[route scored] near scores")
    g = torch.Generator().manual_seed(1)
    base = torch.randn((256, 1), generator=g)
    l = base + 3e-8 * torch.randint(-9, 10, (256, 96), generator=g)
    for scores in ("softmax", "sigmoid"):
        _check(l.cuda(), 8, scores, None, 1, 1, True, 1.0) if scores == "sigmoid" else _check(l.cuda(), 8, scores, None, 8, 3, True, 1.0)
        _check(l.cuda(), 8, scores, (1e-7 * torch.randn(96, generator=g)).cuda(), 8, 3, False, 1.0)


def test_into_given_outputs_and_refusals():
    log("[route scored] out, refusals")
    ml = _ml()
    l = torch.randn((70, 24), device="cuda")
    want = ml.route(l, 3, scores="sigmoid", n_groups=4, top_groups=2)
    out = tuple(torch.full_like(t, 77) for t in want)
    ml.route(l, 3, scores="sigmoid", n_groups=4, top_groups=2, out=out)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    for bad in (dict(n_groups=5), dict(n_groups=4, top_groups=5), dict(n_groups=4, top_groups=0), dict(n_groups=24, top_groups=2), dict(n_groups=0)):
        with pytest.raises(ml.MloraError) as e:
            ml.route(l, 3, scores="sigmoid", **bad)
        assert e.value.name == "MLORA_ERR_SHAPE"
    for bad in (dict(scores="tanh"), dict(bias=torch.zeros(23, device="cuda")), dict(bias=torch.zeros(24, dtype=torch.bfloat16, device="cuda")),
                dict(top_groups=2), dict(bias=torch.zeros(24))):
        with pytest.raises((TypeError, ValueError)):
            ml.route(l, 3, **bad)
    none = ml.route(torch.empty((0, 24), device="cuda"), 3, scores="sigmoid")
    torch.cuda.synchronize()
    assert none[0].shape == (0, 3) and torch.all(none[3] == 0)
