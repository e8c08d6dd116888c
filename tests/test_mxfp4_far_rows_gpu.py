"""Expert products with MXFP4 weights on rows whose bytes lie past 4 GB, in bf16 and in codes, there and back."""
import pytest
import torch

from gpu_util import log
from mx_util import decode, random_mx
from op_util import U, check, product64

pytestmark = pytest.mark.gpu

D_IN, D_OUT, E = 32768, 258, 2


def _ml():
    import rank_adapter_gemm_segmented_amd as ml
    return ml


def _rows(n, x_mx):
    """(operand, keywords, values in 64 bits of chosen rows) of n rows past 4 GB."""
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    if x_mx:
        codes = torch.randint(0, 256, (n, D_IN // 2), generator=g, device="cuda", dtype=torch.uint8)
        assert codes.numel() > 1 << 32
        scale = torch.randint(118, 127, (D_IN // 128, n, 4), generator=g, device="cuda", dtype=torch.uint8)
        return codes, {"x_scale": scale}, lambda r: decode(codes[r], scale[:, r].contiguous(), D_IN)
    x = torch.randn((n, D_IN), generator=g, device="cuda", dtype=torch.bfloat16)
    assert 2 * x.numel() > 1 << 32
    return x, {}, lambda r: x[r].double()


@pytest.mark.parametrize("x_mx", [False, True])
def test_rows_past_4_gb(x_mx):
    log(f"[mxfp4 far rows] x_mx={x_mx}")
    n = 263000 if x_mx else 66000
    x, kw, values = _rows(n, x_mx)
    W, s, W64 = random_mx((E, D_OUT, D_IN), 1)
    for counts in ([1, 3], [15, 20], [70, 40], [300, 257]):   # streamed, and tiles of 32, 64 or 128 and more positions
        total = sum(counts)
        rows = torch.randint(0, n, (total,), generator=torch.Generator().manual_seed(total))
        rows[::2] = n - 1 - rows[::2] % 100                   # (half of them at the far end)
        start = torch.tensor([0, counts[0], total], dtype=torch.int32, device="cuda")
        y = _ml().experts_linear(x, W, start, rows.int().cuda(), w_scale=s, **kw)
        torch.cuda.synchronize()
        for e, (a, b) in enumerate(((0, counts[0]), (counts[0], total))):
            check(y[a:b], *product64(values(rows[a:b].cuda()), W64[e]), f"expert {e} of {counts}")


@pytest.mark.parametrize("x_mx", [False, True])
def test_way_back_past_4_gb(x_mx):
    log(f"[mxfp4 far rows] way back, x_mx={x_mx}")
    n, k = (263000 if x_mx else 66000), 2
    h, kw, values = _rows(n, x_mx)
    T, half = n // k, n // 2
    W, s, W64 = random_mx((E, D_OUT, D_IN), 2)
    g = torch.Generator().manual_seed(3)
    weight = torch.rand((T, k), generator=g)
    # token t has row t of the first expert and row T + t of the second
    position = torch.stack([torch.arange(T), T + torch.arange(T)], 1).int()
    start = torch.tensor([0, half, n], dtype=torch.int32, device="cuda")
    y = _ml().experts_combine(h, W, start, position.cuda(), weight.cuda(), w_scale=s, **kw)
    torch.cuda.synchronize()
    t = torch.cat([torch.arange(20), torch.arange(T // 2, T // 2 + 20), torch.arange(T - 60, T)])
    ref = bound = mass = 0
    for e in range(E):
        z, dz = product64(values((t + e * T).cuda()), W64[e])
        w = weight[t, e].double().cuda()[:, None]
        ref, bound, mass = ref + w * z, bound + w * dz, mass + w * z.abs()
    check(y[t.cuda()], ref, bound + (k + 2) * U * mass, "way back")
