"""Every form of the MXFP4 products by the sizes that choose it, and metadata that lies."""
import pytest
import torch

from gpu_util import log
from mx_util import random_mx
from op_util import check, epilogue64, normal, product64
from test_experts_gpu import _segments
from test_mxfp4_layers_gpu import Layer, _ml, _product, _quantised

pytestmark = pytest.mark.gpu

# rows per expert and widths of each form: 32 rows with two and eight waves, 64 and 128 rows, many positions on few rows,
# tiles of 32, 64 (both heights), 128 positions
EXPERTS = {
    "few items": ([3, 1, 0, 2], 2080, 130),
    "long rows, a few tokens": ([1, 0, 2, 3, 1, 4], 4128, 1026),
    "five per expert": ([5, 4, 6, 0, 9, 3, 4, 5] * 4, 2336, 1540),
    "ten per expert": ([10, 3, 17, 12, 0, 16, 9, 11] * 2, 2336, 2500),
    "many positions, few rows": ([60, 33, 1], 544, 260),
    "sixteen per expert": ([16, 15, 33, 0, 1, 31, 14, 17] * 4, 1056, 1026),
    "forty per expert": ([40, 64, 65, 1, 0, 33, 50, 63] * 2, 672, 2050),
    "forty, many rows": ([40, 64, 65, 1, 0, 33, 50, 63] * 2, 416, 8200),
    "ninety per expert": ([90, 129, 0, 128, 64, 100, 91, 33] * 2, 416, 1030),
}


@pytest.mark.parametrize("x_mx", [False, True])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("counts,d_in,d_out", EXPERTS.values(), ids=EXPERTS.keys())
def test_experts(counts, d_in, d_out, gated, x_mx):
    log(f"[mxfp4 forms] experts {len(counts)} with {sum(counts)} rows, {d_in}->{d_out} gated={gated} x_mx={x_mx}")
    _product(x_mx, counts, d_in, d_out, "silu" if gated else "relu", gated, True, seed=d_in)


@pytest.mark.parametrize("x_mx", [False, True])
@pytest.mark.parametrize("T,d_out", [(100, 3002), (513, 3002), (300, 7000), (513, 9100)])
def test_one_round_of_tiles(x_mx, T, d_out):
    log(f"[mxfp4 forms] T={T} 160->{d_out} x_mx={x_mx}")
    Layer(T, 160, d_out, False, x_mx, seed=T, max_run=30).check("gelu", "plain")
    Layer(T, 160, d_out, True, x_mx, seed=T, max_run=30, residual=False).check("silu", "gated")


@pytest.mark.parametrize("x_mx", [False, True])
def test_largest_tile_without_an_epilogue(x_mx):
    log(f"[mxfp4 forms] 256x256, no epilogue, x_mx={x_mx}")
    Layer(1030, 416, 10006, False, x_mx, seed=1, max_run=70, bias=False, residual=False).check("none", "no epilogue")


@pytest.mark.parametrize("x_mx", [False, True])
@pytest.mark.parametrize("gated", [True, False])
def test_largest_tile_adapters(x_mx, gated):
    """Ranks past a chunk of 64 columns; a segment per token; fused pools; shuffled rows; one segment."""
    log(f"[mxfp4 forms] 256x256 adapters, gated={gated} x_mx={x_mx}")
    Layer(1030, 96, 10006, gated, x_mx, seed=2, ranks=(3, 64, 100, 200), max_run=60, residual=False).check("relu", "high ranks")
    Layer(1030, 96, 10006, gated, x_mx, seed=3, ranks=(16, 5), max_run=1, bias=False, shuffled=True).check("silu", "a segment per token")
    Layer(1030, 96, 10006, gated, x_mx, seed=4, ranks=(16, 40), fused=True, max_run=50).check("gelu_tanh", "fused")
    Layer(1030, 96, 10006, gated, x_mx, seed=5, ranks=(24,), max_run=2000).check("gelu", "long segments")


@pytest.mark.parametrize("x_mx", [False, True])
def test_few_tokens_of_many_adapters(x_mx):
    log(f"[mxfp4 forms] few tokens, x_mx={x_mx}")
    for T in (16, 17, 40, 64):
        Layer(T, 1056, 258, T % 2 == 0, x_mx, seed=T, max_run=2, shuffled=True, ranks=(8, 70, 1)).check("silu", f"T={T}")
        Layer(T, 288, 130, False, x_mx, seed=T, bias=False, residual=False, ranks=(16, 4), fused=True).check("none", f"fused T={T}")


@pytest.mark.parametrize("x_mx", [False, True])
@pytest.mark.parametrize("T,d_out", [(3, 130), (50, 130), (200, 130), (1030, 10006)])
def test_layer_metadata_that_lies(x_mx, T, d_out):
    """Adapters, ranks, bounds and rows out of range are clamped: finite results, and nothing outside y is written."""
    log(f"[mxfp4 forms] lying metadata T={T} ->{d_out} x_mx={x_mx}")
    l = Layer(T, 160, d_out, False, x_mx, seed=6, bias=False, residual=False, ranks=(8, 16))
    guard = torch.full((T * d_out + 4096,), 3.0, dtype=torch.bfloat16, device="cuda")
    y = guard[2048:2048 + T * d_out].view(T, d_out)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    n = T // 2
    start, scale = i32(-7, n, 1 << 29, T + 100), torch.ones(3, device="cuda")
    for ids, ranks in ((i32(1 << 20, -5, 2), i32(4, 4, 4)), (i32(0, 1, 0), i32(1 << 20, 64, -3)), (i32(2, 2, -1), i32(16, 8, 16))):
        guard.fill_(3.0)
        _ml().linear_mxfp4(l.x, l.W, l.w_scale, l.pool, start, ids, ranks, scale, out=y, **l.kw)
        torch.cuda.synchronize()
        assert torch.all(guard[:2048] == 3.0) and torch.all(guard[2048 + T * d_out:] == 3.0)
        assert torch.isfinite(y).all()
    index = torch.full((T,), 1 << 27, dtype=torch.int32, device="cuda")
    guard.fill_(3.0)
    _ml().linear_mxfp4(l.x, l.W, l.w_scale, l.pool, *l.meta, token_index=index, out=y, **l.kw)
    torch.cuda.synchronize()
    assert torch.all(guard[:2048] == 3.0) and torch.all(guard[2048 + T * d_out:] == 3.0)


def test_another_device_or_host_is_refused():
    log("[mxfp4 forms] host tensors")
    ml = _ml()
    l = Layer(4, 64, 32)
    for bad in (dict(W=l.W.cpu()), dict(w_scale=l.w_scale.cpu()), dict(x=l.x.cpu())):
        kw = dict(x=l.x, W=l.W, w_scale=l.w_scale)
        kw.update(bad)
        with pytest.raises(ValueError):
            ml.linear_mxfp4(kw["x"], kw["W"], kw["w_scale"], l.pool, lora_on=0, out=torch.empty((4, 32), dtype=torch.bfloat16, device="cuda"),
                            workspace=l.pool.workspace(4))


def test_same_bits_from_call_to_call():
    """No sum's order goes by timing."""
    log("[mxfp4 forms] same bits")
    for T, d_out in ((5, 16500), (64, 514), (300, 514), (1030, 10006)):
        l = Layer(T, 544, d_out, True, T % 2 == 0, seed=T)
        want = l.run("silu")
        for _ in range(3):
            assert torch.equal(l.run("silu"), want)


def test_two_streams_at_once():
    """Two calls that share no workspace run side by side with the results of one after the other."""
    log("[mxfp4 forms] two streams")
    layers = [Layer(T, 544, 1026, True, x, seed=T) for T, x in ((40, False), (300, True))]
    want = [l.run("silu") for l in layers]
    ws = [l.pool.workspace(l.T) for l in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for l, w, s in zip(layers, ws, streams):
            with torch.cuda.stream(s):
                got.append(_ml().linear_mxfp4(l.x, l.W, l.w_scale, l.pool, *l.meta, bias=l.bias, act="silu", gated=True,
                                              residual=l.residual, workspace=w, **l.kw))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 2])


def test_widest_scales_and_large_values():
    """Scales from 2^-60 to 2^60 in one row: products far apart in size, sums bounded by the largest."""
    log("[mxfp4 forms] wide scales")
    W, s, W64 = random_mx((70, 672), 1, low=67, high=187)
    for T in (3, 40, 200):
        x = normal((T, 672), T)
        pool = _ml().Pool(672, 70, torch.bfloat16, 8, 1)
        for kw, x64 in (({}, x.double()), (None, None)):
            if kw is None:
                c, xs, x64 = _quantised(x)
                kw = dict(x_codes=c, x_scale=xs)
            y = _ml().linear_mxfp4(x, W, s, pool, lora_on=0, **kw)
            torch.cuda.synchronize()
            check(y, *epilogue64(*product64(x64, W64), "none", False, None, None), f"T={T}")


def test_experts_on_a_side_stream_reuse_their_workspace():
    log("[mxfp4 forms] experts, side stream")
    ml = _ml()
    W, s, _ = random_mx((4, 130, 96), 1)
    h = normal((40, 96), 2)
    seg = _segments([10, 10, 10, 10])
    pos, wt = torch.arange(40, dtype=torch.int32, device="cuda").view(20, 2), torch.rand((20, 2), device="cuda")
    ws = ml.experts_workspace(20, 2, 4, 130, torch.bfloat16)
    want = ml.experts_combine(h, W, seg, pos, wt, w_scale=s, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [ml.experts_combine(h, W, seg, pos, wt, w_scale=s, workspace=ws) for _ in range(3)]
    side.synchronize()
    assert all(torch.equal(g, want) for g in got)


@pytest.mark.parametrize("x_mx", [False, True])
def test_x_past_4_gb(x_mx):
    """Rows of x beyond 32-bit offsets: the largest tile's addressing gives way to a smaller tile's."""
    log(f"[mxfp4 forms] x past 4 GB, x_mx={x_mx}")
    ml, T, d_in, d_out = _ml(), 16500, 131072, 770
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn((T, d_in), generator=g, device="cuda", dtype=torch.bfloat16)
    assert x.numel() * 2 > 1 << 32
    W, s, W64 = random_mx((d_out, d_in), 2)
    pool = ml.Pool(d_in, d_out, torch.bfloat16, 8, 1)
    kw = {}
    if x_mx:
        kw["x_codes"], kw["x_scale"] = ml.quantize_mxfp4(x)
    y = ml.linear_mxfp4(x, W, s, pool, lora_on=0, **kw)
    torch.cuda.synchronize()
    for lo in (0, 8200, T - 20):
        rows = x[lo:lo + 20].contiguous()
        x64 = _quantised(rows)[2] if x_mx else rows.double()
        check(y[lo:lo + 20], *product64(x64, W64), f"rows from {lo}")
