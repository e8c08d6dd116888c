"""mlora_experts_linear and mlora_experts_combine against 64-bit products, alone and together with mlora_route."""
import pytest
import torch

from gpu_util import log
from op_util import U, check, e4m3, epilogue64, normal, product64

pytestmark = pytest.mark.gpu


def _ml():
    import rank_adapter_gemm_segmented_amd as ml
    return ml


DT = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8w": torch.bfloat16}


def _weight(E, d_out, d_in, kind, seed):
    """W, its row scales (FP8) and the weight in 64 bits."""
    W = normal((E, d_out, d_in), seed, 0.05, DT[kind])
    if kind != "fp8w":
        return W, None, W.double()
    codes, scale, exact = e4m3(W)
    return codes, scale, exact


def _segments(counts):
    s = torch.zeros(len(counts) + 1, dtype=torch.int32)
    s[1:] = torch.cumsum(torch.tensor(counts), 0)
    return s.cuda()


def _product(kind, counts, d_in, d_out, act, gated, bias, tail=3, n_rows=0, seed=0):
    """One experts_linear call: segments of the given sizes, `tail` unused rows behind them."""
    ml = _ml()
    E, n = len(counts), sum(counts)
    W, scale, W64 = _weight(E, d_out, d_in, kind, seed)
    n_rows = n_rows or max(1, n // 2)
    x = normal((n_rows, d_in), seed + 1, 1.0, DT[kind])
    idx = torch.randint(0, n_rows, (n + tail,), generator=torch.Generator().manual_seed(seed)).int()
    idx[n:] = -1
    b = normal((E, d_out), seed + 2, 0.5, DT[kind]) if bias else None
    y = torch.full((n + tail, d_out // 2 if gated else d_out), 7.0, dtype=DT[kind], device="cuda")
    ml.experts_linear(x, W, _segments(counts), idx.cuda(), bias=b, act=act, gated=gated, w_scale=scale, out=y)
    torch.cuda.synchronize()
    assert torch.all(y[n:] == 7.0), "rows behind the last segment were written"
    at = 0
    for e, c in enumerate(counts):
        if c:
            z, dz = product64(x[idx[at:at + c].long().cuda()], W64[e])
            z, dz = epilogue64(z, dz, act, gated, b[e] if bias else None, None)
            check(y[at:at + c], z, dz, f"{kind} expert {e} ({c} rows) {d_in}->{d_out} {act} gated={gated}")
        at += c


COUNTS = [[1], [0, 1, 0, 2, 0], [5, 0, 17, 1, 33], [16, 16, 16], [64, 65, 0, 1, 130], [300, 3]]


@pytest.mark.parametrize("kind", ["bf16", "fp8w", "f32"])
@pytest.mark.parametrize("i", range(len(COUNTS)))
def test_ragged_counts(kind, i):
    log(f"[experts] {kind} counts {COUNTS[i]}")
    act = ["none", "silu", "relu", "gelu", "gelu_tanh", "silu"][i]
    _product(kind, COUNTS[i], 272, 192, act, gated=False, bias=i % 2 == 0, seed=10 * i)
    _product(kind, COUNTS[i], 272, 192, act, gated=True, bias=i % 2 == 1, seed=10 * i + 5)


# d_in below a unit, not whole units, larger; d_out below a tile, odd, gated halves that are not whole blocks
SHAPES = [(16, 2), (48, 6), (80, 30), (144, 66), (528, 130), (1040, 250), (2064, 34)]


@pytest.mark.parametrize("kind", ["bf16", "fp8w", "f32"])
@pytest.mark.parametrize("d_in,d_out", SHAPES)
def test_odd_shapes(kind, d_in, d_out):
    log(f"[experts] {kind} {d_in}->{d_out}")
    for counts in ([3, 0, 20], [70, 1]):
        _product(kind, counts, d_in, d_out, "silu", gated=True, bias=True, seed=d_in)
        _product(kind, counts, d_in, d_out - 1, "none", gated=False, bias=True, seed=d_in)


@pytest.mark.parametrize("kind,d_in", [("bf16", 8), ("bf16", 24), ("f32", 4), ("f32", 20)])
def test_smallest_rows(kind, d_in):
    log(f"[experts] {kind} d_in={d_in}")
    _product(kind, [2, 1], d_in, 10, "none", gated=False, bias=False)


@pytest.mark.parametrize("counts", [[600, 513], [1024, 0, 700, 256], [2000]])
@pytest.mark.parametrize("gated", [True, False])
def test_long_segments(counts, gated):
    log(f"[experts] bf16 counts {counts} gated={gated}")
    _product("bf16", counts, 520, 1056, "silu" if gated else "none", gated, bias=True, seed=3)
    _product("bf16", counts, 136, 520, "gelu", gated, bias=False, seed=4)


# Sixteen experts on layers wide enough for the tiled forms: means of 5, 30, 100 (tiles of 32, 64, 128 positions) and
# 200 rows (256). The last by how an XCD's tiles fill rounds of 32: 2 over (quarters), 11 over (halves), none, and runs
# of at most 128 positions.
TILED = {
    "mean 5": [5, 1, 0, 9, 12, 3, 4, 8, 2, 5, 7, 6, 0, 33, 1, 4],
    "mean 30": [30, 65, 0, 1, 64, 63, 12, 40, 31, 33, 32, 2, 70, 20, 0, 35],
    "mean 100": [128, 129, 1, 0, 127, 257, 100, 90, 64, 110, 96, 140, 33, 200, 95, 60],
    "200 each": [200] * 16,
    "short runs": [2000, 1100, 90, 10] + [0] * 12,
    "one expert": [0] * 7 + [3301] + [0] * 8,
    "20 runs": [257, 513, 129, 1, 256, 255, 128, 0, 385, 300, 290, 130, 140, 260, 127, 100],
}


@pytest.mark.parametrize("counts", TILED.values(), ids=TILED.keys())
@pytest.mark.parametrize("d_in,d_out", [(72, 2056), (520, 4104), (264, 4344)])
@pytest.mark.parametrize("gated", [True, False])
def test_tiled(counts, d_in, d_out, gated):
    log(f"[experts] tiled, {len(counts)} experts, {sum(counts)} rows, {d_in}->{d_out} gated={gated}")
    _product("bf16", counts, d_in, d_out, "silu" if gated else "gelu_tanh", gated, bias=True, seed=d_in)


@pytest.mark.parametrize("name", ["mean 30", "mean 100", "200 each"])
@pytest.mark.parametrize("gated", [True, False])
def test_tiled_fp8(name, gated):
    log(f"[experts] tiled FP8, {name} gated={gated}")
    _product("fp8w", TILED[name], 272, 2056, "silu", gated, bias=True, seed=8)


def test_many_experts():
    log("[experts] 200 experts, most of them empty")
    counts = [0] * 200
    counts[0], counts[63], counts[64], counts[130], counts[199] = 2, 1, 3, 40, 1
    _product("bf16", counts, 128, 64, "none", False, True)


def test_every_segment_empty():
    log("[experts] no rows at all")
    ml = _ml()
    x, W = normal((4, 64), 1), normal((3, 32, 64), 2)
    y = torch.full((4, 32), 5.0, dtype=torch.bfloat16, device="cuda")
    ml.experts_linear(x, W, _segments([0, 0, 0]), torch.full((4,), -1, dtype=torch.int32, device="cuda"), out=y)
    torch.cuda.synchronize()
    assert torch.all(y == 5.0)


def test_rows_without_an_index():
    log("[experts] position p reads row p")
    ml = _ml()
    x, W = normal((9, 64), 1), normal((2, 40, 64), 2, 0.1)
    y = ml.experts_linear(x, W, _segments([4, 5]))
    torch.cuda.synchronize()
    for e, (a, b) in enumerate(((0, 4), (4, 9))):
        check(y[a:b], *product64(x[a:b], W[e]), "no index")


def test_unused_rows_may_hold_anything():
    log("[experts] NaN and inf in rows that no position reads")
    ml = _ml()
    x, W = normal((20, 64), 1), normal((2, 40, 64), 2, 0.1)
    x[10:] = float("nan")
    W[1, :, :] = float("inf")          # an expert without rows
    idx = torch.arange(10, dtype=torch.int32, device="cuda")
    y = ml.experts_linear(x, W, _segments([10, 0]), idx)
    torch.cuda.synchronize()
    check(y, *product64(x[:10], W[0]), "unused rows")
    z = ml.experts_combine(x, W, _segments([10, 0]), torch.cat([idx, torch.full_like(idx, -1)]).reshape(10, 2),
                           torch.full((10, 2), 0.5, device="cuda"))
    torch.cuda.synchronize()
    assert torch.isfinite(z).all()


def _layer(kind, T, E, k, d, f, bias, pad, seed, act="silu"):
    """route -> experts_linear (gated) -> experts_combine, each step against 64 bits on its own inputs."""
    ml = _ml()
    dt = DT[kind]
    logits = normal((T, E), seed, 1.0, torch.float32)
    if pad:
        logits[T - pad:] = float("-inf")
    x = normal((T, d), seed + 1, 1.0, dt)
    W1, s1, W1_64 = _weight(E, 2 * f, d, kind, seed + 2)
    W2, s2, W2_64 = _weight(E, d, f, kind, seed + 3)
    b1 = normal((E, 2 * f), seed + 4, 0.2, dt) if bias else None
    b2 = normal((E, d), seed + 5, 0.2, dt) if bias else None

    def run(out=None, ws=None):
        r = ml.route(logits, k)
        h = ml.experts_linear(x, W1, r[3], r[2], bias=b1, act=act, gated=True, w_scale=s1)
        return r, h, ml.experts_combine(h, W2, r[3], r[4], r[1], bias=b2, residual=x, w_scale=s2, out=out, workspace=ws)

    (expert, weight, token_index, seg_start, position), h, y = run()
    torch.cuda.synchronize()
    starts = seg_start.tolist()
    z = torch.zeros((T * k, d), dtype=torch.float64, device="cuda")
    dz = torch.zeros_like(z)
    for e in range(E):
        a, b = starts[e], starts[e + 1]
        if a == b:
            continue
        ref, bound = product64(x[token_index[a:b].long()], W1_64[e])
        check(h[a:b], *epilogue64(ref, bound, act, True, b1[e] if bias else None, None), f"{kind} up, expert {e}")
        z[a:b], dz[a:b] = epilogue64(*product64(h[a:b], W2_64[e]), "none", False, b2[e] if bias else None, None)
    p = position.clamp(min=0).long()
    w = torch.where(position >= 0, weight.double(), 0.0)[:, :, None]
    ref = (z[p] * w).sum(1) + x.double()
    bound = ((dz[p] + (k + 2) * U * z[p].abs()) * w).sum(1) + (k + 2) * U * (x.double().abs() + (z[p].abs() * w).sum(1))
    check(y, ref, bound, f"{kind} combine T={T}")
    if pad:
        assert torch.equal(y[T - pad:], x[T - pad:])
    return run, y, x


@pytest.mark.parametrize("kind", ["bf16", "fp8w", "f32"])
@pytest.mark.parametrize("T,E,k,d,f,pad", [(1, 8, 2, 256, 96, 0), (5, 4, 4, 64, 32, 2), (37, 5, 2, 256, 176, 4),
                                           (64, 32, 8, 512, 144, 0), (300, 6, 2, 272, 304, 11)])
def test_layer(kind, T, E, k, d, f, pad):
    log(f"[experts] layer {kind} T={T} E={E} k={k} {d}->{f}")
    _layer(kind, T, E, k, d, f, bias=T % 2 == 1, pad=pad, seed=T)


def test_layer_large():
    log("[experts] layer bf16, 1500 tokens")
    _layer("bf16", 1500, 4, 2, 512, 768, bias=True, pad=100, seed=5)


@pytest.mark.parametrize("kind,T,E,k,d,f,pad", [("bf16", 1600, 16, 2, 4104, 136, 0), ("bf16", 1024, 8, 2, 4104, 520, 9),
                                                ("bf16", 2048, 8, 2, 4096, 264, 0), ("bf16", 350, 16, 4, 2056, 1040, 0),
                                                ("bf16", 40, 16, 2, 2056, 1032, 3), ("fp8w", 400, 16, 2, 2064, 1040, 0)])
def test_layer_tiled(kind, T, E, k, d, f, pad):
    log(f"[experts] layer {kind}, tiled, T={T} E={E} k={k} {d}->{f}")
    _layer(kind, T, E, k, d, f, bias=True, pad=pad, seed=T)


def test_layer_repeats_in_place_and_captured():
    log("[experts] layer: same bits on every run, residual in place, graph replays")
    ml = _ml()
    run, y, x = _layer("bf16", 40, 8, 2, 256, 96, bias=True, pad=0, seed=9)
    assert torch.equal(run()[2], y)
    ws = ml.experts_workspace(40, 2, 8, 256, torch.bfloat16)
    r = ml.route(normal((40, 8), 9, 1.0, torch.float32), 2)
    h, W2 = normal((80, 96), 1), normal((8, 256, 96), 2, 0.1)
    want = ml.experts_combine(h, W2, r[3], r[4], r[1], residual=x)
    inplace = x.clone()
    ml.experts_combine(h, W2, r[3], r[4], r[1], residual=inplace, out=inplace)
    assert torch.equal(inplace, want)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(x)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run(out=out, ws=ws)
    for _ in range(3):
        out.zero_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y)


def test_metadata_that_lies():
    log("[experts] lying segments and indices stay in bounds")
    ml = _ml()
    x, W = normal((6, 64), 1), normal((3, 32, 64), 2, 0.1)
    idx = torch.tensor([0, -5, 99, 3, 1 << 30, -(1 << 30)], dtype=torch.int32, device="cuda")
    for seg in ([0, 100, 200, 300], [-7, 2, 1, 4], [6, 5, 4, 3], [1 << 30, 0, 1 << 30, 6]):
        y = ml.experts_linear(x, W, torch.tensor(seg, dtype=torch.int32, device="cuda"), idx)
        torch.cuda.synchronize()
        assert y.shape == (6, 32)
    pos = torch.tensor([[0, 99], [-5, 1 << 30], [2, 3]], dtype=torch.int32, device="cuda")
    y = ml.experts_combine(x, W, torch.tensor([0, 2, 4, 6], dtype=torch.int32, device="cuda"),
                           pos, torch.ones((3, 2), device="cuda"))
    torch.cuda.synchronize()
    assert torch.isfinite(y).all()


def test_refusals():
    log("[experts] refusals")
    ml = _ml()
    x, W, seg = normal((4, 64), 1), normal((2, 32, 64), 2), _segments([2, 2])
    idx = torch.zeros(4, dtype=torch.int32, device="cuda")
    E = ml.STATUS_CODE
    for bad, code in ((lambda: ml.experts_linear(normal((4, 60), 1), normal((2, 32, 60), 2), seg, idx), "MLORA_ERR_SHAPE"),
                      (lambda: ml.experts_linear(x[:0], W, seg, idx), "MLORA_ERR_SHAPE"),
                      (lambda: ml.experts_combine(x, W, seg, idx.reshape(2, 2), torch.ones((2, 2), device="cuda"),
                                                  workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), "MLORA_ERR_WORKSPACE")):
        with pytest.raises(ml.MloraError) as e:
            bad()
        assert e.value.code == E[code]
    for bad in (lambda: ml.experts_linear(x.float(), W, seg, idx), lambda: ml.experts_linear(x, W.float(), seg, idx),
                lambda: ml.experts_linear(x.half(), W.half(), seg, idx),
                lambda: ml.experts_linear(x, W, seg, idx.long()),
                lambda: ml.experts_linear(x, W.view(torch.uint8)[:, :, :64].contiguous(), seg, idx)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: ml.experts_linear(x, W, seg[:2], idx), lambda: ml.experts_linear(x, W[0], seg, idx),
                lambda: ml.experts_linear(x, W, seg, idx, act="swish"), lambda: ml.experts_linear(x, W, seg, idx, bias=W[0, :, 0]),
                lambda: ml.experts_linear(x, W[:, :31], seg, idx, gated=True),
                lambda: ml.experts_linear(x, W.transpose(1, 2).contiguous().transpose(1, 2), seg, idx),
                lambda: ml.experts_linear(x, W, seg, idx, out=torch.empty((4, 33), dtype=torch.bfloat16, device="cuda")),
                lambda: ml.experts_linear(x.cpu(), W, seg, idx),
                lambda: ml.experts_combine(x[:3], W, seg, idx.reshape(2, 2), torch.ones((2, 2), device="cuda")),
                lambda: ml.experts_combine(x, W, seg, idx, torch.ones(4, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
