"""Operands past 2^32 bytes and results past 2^31 elements: epilogue, routing and expert operators, sampled against 64 bits."""
import pytest
import torch

from gpu_util import log
from op_util import U, check, epilogue64, normal, product64

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")
BF16 = dict(dtype=torch.bfloat16, device="cuda")


def _ml():
    import rank_adapter_gemm_segmented_amd as ml
    return ml


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("per_expert,d_out", [(1, 64), (6, 16384), (40, 16384), (200, 16384)])
def test_expert_rows_from_a_long_x(per_expert, d_out):
    """Rows of x and experts' weights behind 4 GB: streamed, and in tiles of 32 to 256 positions."""
    log(f"[far] {per_expert} rows per expert, d_out {d_out}")
    E, d_in, n_rows = 40, 4096, 600_000
    used = (0, E - 2, E - 1)
    W = torch.zeros((E, d_out, d_in), **BF16)
    x = torch.zeros((n_rows, d_in), **BF16)
    rows = torch.tensor([0, 1, 524_287, 524_288, 524_289, n_rows - 1], device="cuda")
    x[rows] = normal((len(rows), d_in), 1)
    for e in used:
        W[e] = normal((64, d_in), 2 + e, 0.05).repeat(d_out // 64, 1)
    counts = torch.zeros(E, dtype=torch.int64)
    counts[list(used)] = per_expert * E // len(used)
    start = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
    idx = rows[torch.arange(int(start[-1]), device="cuda") % len(rows)]
    y = _ml().experts_linear(x, W, start.to(**I32), idx.int())
    torch.cuda.synchronize()
    for e in used:
        a, b = int(start[e]), int(start[e + 1])
        for c in (0, d_out - 64):
            check(y[a:b, c:c + 64], *product64(x[idx[a:b]], W[e, c:c + 64]), f"expert {e}, columns from {c}")


@pytest.mark.parametrize("gated", [True, False])
def test_many_positions(gated):
    """y of 2^33 elements and, on the way back, an fp32 workspace of 34 GB."""
    log(f"[far] 2^20 positions, gated={gated}")
    ml = _ml()
    T, k, E, d_in, d_y = 1 << 19, 2, 4, 16, 8192
    d_out = 2 * d_y if gated else d_y
    x = torch.randn((T, d_in), generator=torch.Generator("cuda").manual_seed(1), device="cuda").bfloat16()
    logits = torch.randn((T, E), generator=torch.Generator("cuda").manual_seed(2), device="cuda")
    W = normal((E, d_out, d_in), 3, 0.2)
    _, weight, index, start, position = ml.route(logits, k)
    y = ml.experts_linear(x, W, start, index, act="silu", gated=gated)
    torch.cuda.synchronize()
    at = start.tolist()
    for e in range(E):
        p = torch.tensor([at[e], (at[e] + at[e + 1]) // 2, at[e + 1] - 1], device="cuda")
        z, dz = product64(x[index[p].long()], W[e])
        check(y[p], *epilogue64(z, dz, "silu", gated, None, None), f"expert {e}")
    del y
    if gated:
        return
    h = torch.randn((T * k, d_in), generator=torch.Generator("cuda").manual_seed(4), device="cuda").bfloat16()
    res = torch.randn((T, d_y), generator=torch.Generator("cuda").manual_seed(5), dtype=torch.bfloat16, device="cuda")
    out = ml.experts_combine(h, W, start, position, weight, residual=res)
    torch.cuda.synchronize()
    for t in (0, T // 2, T - 1):
        ref, bound = res[t].double(), 0.0
        for j in range(k):
            p, w = int(position[t, j]), float(weight[t, j])
            e = max(e for e in range(E) if at[e] <= p)
            z, dz = product64(h[p:p + 1], W[e])
            ref = ref + w * z[0]
            bound = bound + w * dz[0] + (k + 2) * U * (w * z[0].abs() + res[t].double().abs())
        check(out[t], ref, bound, f"token {t}")


@pytest.mark.parametrize("gated", [True, False])
def test_layer_on_a_long_batch(gated):
    """A batch of more than 4 GB, with the epilogue."""
    log(f"[far] 600,000 tokens, gated={gated}")
    ml = _ml()
    T, d_in, d_out = 600_000, 4096, 512
    d_y = d_out // 2 if gated else d_out
    x = torch.zeros((T, d_in), **BF16)
    rows = torch.tensor([0, 1, 524_287, 524_288, T - 1], device="cuda")
    x[rows] = normal((len(rows), d_in), 1)
    W, b = normal((d_out, d_in), 2, 0.05), normal((d_out,), 3)
    res = torch.randn((T, d_y), generator=torch.Generator("cuda").manual_seed(4), dtype=torch.bfloat16, device="cuda")
    pool = ml.Pool(d_in, d_out, torch.bfloat16, 16, 1)
    y = ml.linear_epilogue(x, W, pool, lora_on=0, bias=b, act="silu", gated=gated, residual=res)
    torch.cuda.synchronize()
    z, dz = product64(x[rows], W)
    check(y[rows], *epilogue64(z, dz, "silu", gated, b, res[rows]), "long batch")
