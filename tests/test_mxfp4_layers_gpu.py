"""The layer and the expert products with an MXFP4 weight, activations in bf16 and in MXFP4, against 64 bits."""
import pytest
import torch

from gpu_util import log
from mx_util import decode, encode, random_mx, tiled
from op_util import U, check, epilogue64, normal, product64
from test_experts_gpu import COUNTS, TILED, _segments

pytestmark = pytest.mark.gpu


def _ml():
    import rank_adapter_gemm_segmented_amd as ml
    return ml


def _quantised(x):
    """MXFP4 of x by the library: (codes, scale, values in 64 bits)."""
    codes, scale = _ml().quantize_mxfp4(x)
    torch.cuda.synchronize()
    return codes, scale, decode(codes, scale, x.shape[-1])


class Layer:
    """A layer with an MXFP4 weight, adapters of mixed ranks (some tokens without one, an empty segment) and a batch."""

    def __init__(self, T, d_in, d_out, gated=False, x_mx=False, seed=0, ranks=(8, 16, 33, 64), bias=True, residual=True,
                 shuffled=False, max_run=9, fused=False):
        ml = _ml()
        self.T, self.gated = T, gated
        self.W, self.w_scale, W64 = random_mx((d_out, d_in), seed)
        self.x = normal((T, d_in), seed + 1)
        x64 = self.x.double()
        self.kw = {}
        if x_mx:
            self.kw["x_codes"], self.kw["x_scale"], x64 = _quantised(self.x)
        n, total = len(ranks), [2 * r if fused else r for r in ranks]
        self.pool = ml.Pool(d_in, d_out, torch.bfloat16, max(total), n + 1)
        AB = {}
        for a, r in enumerate(ranks):
            if fused:
                half = d_out // 2
                sl = [(normal((r, d_in), seed + 10 * a + m, 0.05), normal((half, r), seed + 10 * a + 5 + m, 0.05)) for m in range(2)]
                self.pool.register_fused(a, sl)
                B = torch.zeros((d_out, 2 * r), dtype=torch.bfloat16, device="cuda")
                B[:half, :r], B[half:, r:] = sl[0][1], sl[1][1]
                AB[a] = torch.cat([s[0] for s in sl]), B
            else:
                AB[a] = normal((r, d_in), seed + 10 * a, 0.05), normal((d_out, r), seed + 10 * a + 5, 0.05)
                self.pool.register(a, *AB[a])
        g = torch.Generator().manual_seed(seed)
        ids, starts, at, a = [], [0], 0, 0
        while at < T:
            run = min(T - at, int(torch.randint(1, max_run + 1, (1,), generator=g)))
            ids.append(a % (n + 1) - 1)
            at, a = at + run, a + 1
            starts.append(at)
            if a == 3:
                ids.append(0)
                starts.append(at)
        scale = [0.0 if i < 0 else 0.5 + i for i in ids]
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        self.meta = (i32(starts), i32(ids), i32([total[i] if i >= 0 else 0 for i in ids]), torch.tensor(scale, device="cuda"))
        self.index = torch.randperm(T, generator=g).int().cuda() if shuffled else None
        self.bias = normal((d_out,), seed + 2, 0.5) if bias else None
        self.residual = normal((T, d_out // 2 if gated else d_out), seed + 3) if residual else None
        self.z, self.dz = product64(x64, W64)
        self.off = self.z.clone(), self.dz.clone()
        for s, i in enumerate(ids):
            if i < 0 or starts[s] == starts[s + 1]:
                continue
            rows = self.index[starts[s]:starts[s + 1]].long() if shuffled else torch.arange(starts[s], starts[s + 1], device="cuda")
            A, B = AB[i]
            v, dv = product64(self.x[rows], A)
            dv = dv + 2.0 ** -16 * v.abs()   # (v as two bf16 parts in the expand)
            b = B.double()
            self.z[rows] += scale[s] * (v @ b.T)
            self.dz[rows] += scale[s] * (dv @ b.abs().T) + 2 * scale[s] * (B.shape[1] + 2) * U * (v.abs() @ b.abs().T) \
                + 2 * U * self.z[rows].abs()

    def run(self, act="none", lora_on=1, **kw):
        kw = {"bias": self.bias, "residual": self.residual, **self.kw, **kw}
        y = _ml().linear_mxfp4(self.x, self.W, self.w_scale, self.pool, *(self.meta if lora_on else ()), lora_on=lora_on,
                               token_index=self.index if lora_on else None, act=act, gated=self.gated, **kw)
        torch.cuda.synchronize()
        return y

    def check(self, act="none", what=""):
        for lora_on in (1, 0):
            z, dz = (self.z, self.dz) if lora_on else self.off
            z, dz = epilogue64(z, dz, act, self.gated, self.bias, self.residual)
            check(self.run(act, lora_on), z, dz, f"{what} lora_on={lora_on}")


# tokens on both sides of the switches between the paths (8, 16, 32, 48, 64, 128) by widths of one block, of odd blocks,
# of part planes and part stages
WIDTHS = [(32, 66), (96, 130), (160, 34), (544, 258), (1056, 98), (2080, 192), (4128, 40)]


@pytest.mark.parametrize("x_mx", [False, True])
@pytest.mark.parametrize("d_in,d_out", WIDTHS)
def test_widths(x_mx, d_in, d_out):
    for i, T in enumerate((1, 7, 16, 31, 64, 65, 130)):
        log(f"[mxfp4 layer] x_mx={x_mx} T={T} {d_in}->{d_out}")
        Layer(T, d_in, d_out, gated=i % 2 == 0, x_mx=x_mx, seed=T, shuffled=i % 3 == 0).check(("silu", "gelu", "none")[i % 3], f"T={T}")


@pytest.mark.parametrize("x_mx", [False, True])
@pytest.mark.parametrize("T", [1, 5, 8, 9, 33, 50])
def test_wide_layers(x_mx, T):
    """From 256 tiles of 64 rows on a few tokens stream the whole of d_in, and 48 tokens go by tiles."""
    log(f"[mxfp4 layer] wide, x_mx={x_mx} T={T}")
    Layer(T, 288, 16500, gated=True, x_mx=x_mx, seed=T).check("silu", "wide gated")
    Layer(T, 672, 16390, x_mx=x_mx, seed=T, residual=False).check("relu", "wide")


@pytest.mark.parametrize("x_mx", [False, True])
@pytest.mark.parametrize("d_in", [224, 288, 800])
@pytest.mark.parametrize("gated", [True, False])
def test_large_tiles(x_mx, d_in, gated):
    log(f"[mxfp4 layer] large tiles, x_mx={x_mx} {d_in} gated={gated}")
    Layer(1030, d_in, 10006, gated, x_mx, seed=d_in, max_run=90, shuffled=gated).check("gelu_tanh", "256x256")
    Layer(513, d_in, 5000, gated, x_mx, seed=d_in, max_run=40).check("silu", "128x128")
    Layer(200, d_in, 1002, gated, x_mx, seed=d_in).check("none", "64x128")


@pytest.mark.parametrize("x_mx", [False, True])
@pytest.mark.parametrize("T", [4, 40, 100, 300])
def test_fused_pools_and_low_ranks(x_mx, T):
    log(f"[mxfp4 layer] fused, x_mx={x_mx} T={T}")
    Layer(T, 192, 256, True, x_mx, seed=T, ranks=(8, 16), fused=True).check("silu", "fused")
    Layer(T, 192, 256, False, x_mx, seed=T, ranks=(4, 1, 16), bias=False, residual=False).check("none", "no epilogue")


def test_no_epilogue_and_in_place_residual():
    log("[mxfp4 layer] residual in place")
    for T in (3, 64, 200):
        l = Layer(T, 160, 96, seed=T)
        want = l.run("silu")
        buf = l.residual.clone()
        assert l.run("silu", residual=buf, out=buf) is buf and torch.equal(buf, want)


def test_zero_tokens():
    l = Layer(2, 64, 32)
    y = _ml().linear_mxfp4(l.x[:0], l.W, l.w_scale, l.pool, lora_on=0)
    assert y.shape == (0, 32)


@pytest.mark.parametrize("T", [4, 64, 300])
def test_nan_scales_stay_in_their_rows(T):
    """A block of scale 255 makes its W row's outputs NaN and no others, in activations its token's."""
    log(f"[mxfp4 layer] NaN scales T={T}")
    W, s, W64 = random_mx((70, 416), 1)
    x = normal((T, 416), 2)
    pool = _ml().Pool(416, 70, torch.bfloat16, 8, 1)
    clean = _ml().linear_mxfp4(x, W, s, pool, lora_on=0)
    s2 = s.clone()
    s2[0, 5, 1] = s2[3, 69, 0] = 255
    y = _ml().linear_mxfp4(x, W, s2, pool, lora_on=0)
    torch.cuda.synchronize()
    rows = torch.tensor([i in (5, 69) for i in range(70)], device="cuda")
    assert torch.isnan(y[:, rows]).all() and torch.equal(y[:, ~rows], clean[:, ~rows])
    xc, xs = _ml().quantize_mxfp4(x)
    clean = _ml().linear_mxfp4(x, W, s, pool, lora_on=0, x_codes=xc, x_scale=xs)
    xs[2, T - 1, 3] = 255
    y = _ml().linear_mxfp4(x, W, s, pool, lora_on=0, x_codes=xc, x_scale=xs)
    torch.cuda.synchronize()
    assert torch.isnan(y[T - 1]).all() and torch.equal(y[:T - 1], clean[:T - 1])


def test_layer_refusals():
    log("[mxfp4 layer] refusals")
    ml = _ml()
    l = Layer(4, 64, 32, x_mx=True)
    f32 = ml.Pool(64, 32, torch.float32, 8, 1)
    xc, xs = l.kw["x_codes"], l.kw["x_scale"]
    for bad in (lambda: ml.linear_mxfp4(l.x, l.W, l.w_scale, f32, lora_on=0), lambda: ml.linear_mxfp4(l.x.float(), l.W, l.w_scale, l.pool, lora_on=0),
                lambda: ml.linear_mxfp4(l.x, l.W[:31], l.w_scale, l.pool, lora_on=0), lambda: ml.linear_mxfp4(l.x, l.W, l.w_scale[:, :31], l.pool, lora_on=0),
                lambda: ml.linear_mxfp4(l.x, l.W, l.w_scale.float(), l.pool, lora_on=0),
                lambda: ml.linear_mxfp4(l.x, l.W, l.w_scale, l.pool, lora_on=0, x_codes=xc),
                lambda: ml.linear_mxfp4(l.x, l.W, l.w_scale, l.pool, lora_on=0, x_codes=xc[:3], x_scale=xs[:, :3]),
                lambda: ml.linear_mxfp4(l.x[:, :32], l.W, l.w_scale, l.pool, lora_on=0),
                lambda: ml.linear_mxfp4(l.x, l.W, l.w_scale, l.pool, *l.meta, bias=normal((31,), 0)),
                lambda: ml.linear_mxfp4(l.x, l.W, l.w_scale, l.pool, l.meta[0][:-1], *l.meta[1:]),
                lambda: ml.linear_mxfp4(l.x, l.W, l.w_scale, l.pool, lora_on=0, act="tanh")):
        with pytest.raises((TypeError, ValueError)):
            bad()
    with pytest.raises(ml.MloraError) as e:
        ml.linear_mxfp4(l.x, l.W, l.w_scale, l.pool, lora_on=0, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.name == "MLORA_ERR_WORKSPACE"


# ---- experts -----------------------------------------------------------------


def _product(x_mx, counts, d_in, d_out, act, gated, bias, tail=3, n_rows=0, seed=0):
    ml = _ml()
    E, n = len(counts), sum(counts)
    W, scale, W64 = random_mx((E, d_out, d_in), seed)
    n_rows = n_rows or max(1, n // 2)
    x = normal((n_rows, d_in), seed + 1)
    x64, kw = x.double(), {}
    if x_mx:
        x, kw["x_scale"], x64 = _quantised(x)
    idx = torch.randint(0, n_rows, (n + tail,), generator=torch.Generator().manual_seed(seed)).int()
    idx[n:] = -1
    b = normal((E, d_out), seed + 2, 0.5) if bias else None
    y = torch.full((n + tail, d_out // 2 if gated else d_out), 7.0, dtype=torch.bfloat16, device="cuda")
    ml.experts_linear(x, W, _segments(counts), idx.cuda(), bias=b, act=act, gated=gated, w_scale=scale, out=y, **kw)
    torch.cuda.synchronize()
    assert torch.all(y[n:] == 7.0), "rows behind the last segment were written"
    at = 0
    for e, c in enumerate(counts):
        if c:
            z, dz = epilogue64(*product64(x64[idx[at:at + c].long().cuda()], W64[e]), act, gated, b[e] if bias else None, None)
            check(y[at:at + c], z, dz, f"expert {e} ({c} rows) {d_in}->{d_out} {act} gated={gated} x_mx={x_mx}")
        at += c


@pytest.mark.parametrize("x_mx", [False, True])
@pytest.mark.parametrize("i", range(len(COUNTS)))
def test_experts_ragged(x_mx, i):
    log(f"[mxfp4 experts] counts {COUNTS[i]} x_mx={x_mx}")
    act = ["none", "silu", "relu", "gelu", "gelu_tanh", "silu"][i]
    _product(x_mx, COUNTS[i], 288, 192, act, False, i % 2 == 0, seed=10 * i)
    _product(x_mx, COUNTS[i], 288, 192, act, True, i % 2 == 1, seed=10 * i + 5)


@pytest.mark.parametrize("x_mx", [False, True])
@pytest.mark.parametrize("d_in,d_out", [(32, 2), (64, 6), (96, 30), (160, 66), (544, 130), (1056, 250), (2080, 34)])
def test_experts_odd_shapes(x_mx, d_in, d_out):
    log(f"[mxfp4 experts] {d_in}->{d_out} x_mx={x_mx}")
    for counts in ([3, 0, 20], [70, 1]):
        _product(x_mx, counts, d_in, d_out, "silu", True, True, seed=d_in)
        _product(x_mx, counts, d_in, d_out - 1, "none", False, True, seed=d_in)


@pytest.mark.parametrize("x_mx", [False, True])
@pytest.mark.parametrize("counts", TILED.values(), ids=TILED.keys())
@pytest.mark.parametrize("d_in,d_out", [(96, 2056), (544, 4104), (288, 4344)])
@pytest.mark.parametrize("gated", [True, False])
def test_experts_tiled(x_mx, counts, d_in, d_out, gated):
    log(f"[mxfp4 experts] tiled, {sum(counts)} rows, {d_in}->{d_out} gated={gated} x_mx={x_mx}")
    _product(x_mx, counts, d_in, d_out, "silu" if gated else "gelu_tanh", gated, True, seed=d_in)


@pytest.mark.parametrize("x_mx", [False, True])
def test_experts_without_an_index(x_mx):
    log(f"[mxfp4 experts] position p reads row p, x_mx={x_mx}")
    x, (W, s, W64) = normal((9, 64), 1), random_mx((2, 40, 64), 2)
    xq, kw, x64 = x, {}, x.double()
    if x_mx:
        xq, kw["x_scale"], x64 = _quantised(x)
    y = _ml().experts_linear(xq, W, _segments([4, 5]), w_scale=s, **kw)
    torch.cuda.synchronize()
    for e, (a, b) in enumerate(((0, 4), (4, 9))):
        check(y[a:b], *product64(x64[a:b], W64[e]), "no index")


def _combine(x_mx, T, k, E, d_in, d_out, bias, residual, pad=0, seed=0):
    ml = _ml()
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn((T, E), generator=g)
    logits[T - pad:] = -float("inf")
    _, weight, _, start, position = ml.route(logits.cuda(), k)
    W, s, W64 = random_mx((E, d_out, d_in), seed)
    h = normal((T * k, d_in), seed + 1)
    hq, kw, h64 = h, {}, h.double()
    if x_mx:
        hq, kw["x_scale"], h64 = _quantised(h)
    b = normal((E, d_out), seed + 2, 0.5) if bias else None
    r = normal((T, d_out), seed + 3) if residual else None
    y = ml.experts_combine(hq, W, start, position, weight, bias=b, residual=r, w_scale=s, **kw)
    torch.cuda.synchronize()
    ref = r.double() if residual else torch.zeros((T, d_out), dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(ref)
    mass = ref.abs()
    start, position, w64 = start.tolist(), position.cpu(), weight.double().cpu()
    for e in range(E):
        rows = [(t, j) for t in range(T) for j in range(k) if start[e] <= int(position[t, j]) < start[e + 1]]
        if not rows:
            continue
        p = torch.tensor([int(position[t, j]) for t, j in rows], device="cuda")
        z, dz = product64(h64[p], W64[e])
        if bias:
            z, dz = z + b[e].double(), dz + U * (z.abs() + b[e].double().abs())
        t = torch.tensor([t for t, _ in rows], device="cuda")
        w = torch.tensor([float(w64[t, j]) for t, j in rows], dtype=torch.float64, device="cuda")[:, None]
        ref.index_add_(0, t, w * z)
        bound.index_add_(0, t, w * dz)
        mass.index_add_(0, t, w * z.abs())
    check(y, ref, bound + (k + 2) * U * mass, f"combine T={T} k={k} E={E} {d_in}->{d_out} x_mx={x_mx}")


@pytest.mark.parametrize("x_mx", [False, True])
@pytest.mark.parametrize("T,k,E,d_in,d_out,pad", [(1, 1, 1, 32, 3, 0), (1, 2, 8, 160, 258, 0), (5, 2, 4, 544, 129, 2), (64, 8, 16, 288, 514, 9),
                                                  (300, 2, 4, 416, 2050, 0), (700, 3, 3, 288, 5000, 11), (2, 2, 3, 1056, 16, 2)])
def test_combine(x_mx, T, k, E, d_in, d_out, pad):
    log(f"[mxfp4 combine] T={T} k={k} E={E} {d_in}->{d_out} x_mx={x_mx}")
    _combine(x_mx, T, k, E, d_in, d_out, T % 2 == 1, T % 3 != 0, pad, seed=T)


@pytest.mark.parametrize("counts", [[1], [40, 3], [300, 200, 700]])
def test_metadata_that_lies(counts):
    """Segments and rows out of range are clamped: finite results, nothing behind the outputs is written."""
    log(f"[mxfp4 experts] lying metadata {counts}")
    ml, E, n = _ml(), len(counts), sum(counts)
    W, s, _ = random_mx((E, 2080, 96), 1)
    x = normal((n, 96), 2)
    xc, xs = ml.quantize_mxfp4(x)
    buf = torch.full((n * 2080 + 4096,), 3.0, dtype=torch.bfloat16, device="cuda")
    start = torch.tensor([-5, 1 << 30] + [n + 9] * (E - 1), dtype=torch.int32, device="cuda")[: E + 1]
    idx = torch.full((n,), 1 << 28, dtype=torch.int32, device="cuda")
    idx[::2] = -7
    for kw in ({"x": x}, {"x": xc, "x_scale": xs}):
        buf.fill_(3.0)
        y = buf[2048:2048 + n * 2080].view(n, 2080)
        ml.experts_linear(kw["x"], W, start, idx, w_scale=s, x_scale=kw.get("x_scale"), out=y)
        torch.cuda.synchronize()
        assert torch.isfinite(y).all() and torch.all(buf[:2048] == 3.0) and torch.all(buf[2048 + n * 2080:] == 3.0)


def test_a_weight_past_4_gb():
    """Offsets of the last of 160 experts pass 32 bits in the codes."""
    log("[mxfp4 experts] codes past 4 GB")
    ml, E, d_out, d_in = _ml(), 160, 14336, 4096
    W = torch.zeros((E, d_out, d_in // 2), dtype=torch.uint8, device="cuda")
    assert W.numel() > 1 << 32
    s = torch.full((E, d_in // 128, d_out, 4), 120, dtype=torch.uint8, device="cuda")
    c, sc, W64 = random_mx((d_out, d_in), 3)
    W[E - 1], s[E - 1] = c, sc
    start = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    for n in (2, 60, 300):
        start[E] = n
        x = normal((n, d_in), n)
        y = ml.experts_linear(x, W, start, w_scale=s)
        xc, xs, x64 = _quantised(x)
        yq = ml.experts_linear(xc, W, start, w_scale=s, x_scale=xs)
        torch.cuda.synchronize()
        check(y, *product64(x, W64), f"{n} rows")
        check(yq, *product64(x64, W64), f"{n} rows of codes")


def test_experts_refusals():
    log("[mxfp4 experts] refusals")
    ml = _ml()
    x, (W, s, _) = normal((9, 64), 1), random_mx((2, 40, 64), 2)
    xc, xs = ml.quantize_mxfp4(x)
    seg = _segments([4, 5])
    pos, wt = torch.zeros((9, 1), dtype=torch.int32, device="cuda"), torch.ones((9, 1), device="cuda")
    for bad in (lambda: ml.experts_linear(x.float(), W, seg, w_scale=s), lambda: ml.experts_linear(x[:, :32], W, seg, w_scale=s),
                lambda: ml.experts_linear(xc, W, seg, w_scale=s), lambda: ml.experts_linear(xc, W, seg, w_scale=s, x_scale=xs[:, :8]),
                lambda: ml.experts_linear(x, W, seg, w_scale=s[:1]), lambda: ml.experts_linear(x, W, seg[:2], w_scale=s),
                lambda: ml.experts_linear(x, normal((2, 40, 64), 3), seg, x_scale=xs),
                lambda: ml.experts_linear(x, W, seg, w_scale=s, bias=normal((2, 39), 1)),
                lambda: ml.experts_combine(xc, W, seg, pos, wt, w_scale=s), lambda: ml.experts_combine(x, W, seg, pos[:8], wt[:8], w_scale=s),
                lambda: ml.experts_linear(x, W[0], seg, w_scale=s)):
        with pytest.raises((TypeError, ValueError)):
            bad()


# ---- together ------------------------------------------------------------------


@pytest.mark.parametrize("x_mx", [False, True])
@pytest.mark.parametrize("T", [1, 20, 333])
def test_a_layer_of_experts(x_mx, T):
    """Routing by scores, the products there and back: each against 64 bits of what it was given, and captured into a
    graph and replayed with the same result."""
    log(f"[mxfp4 chain] T={T} x_mx={x_mx}")
    ml = _ml()
    E, k, d, f = 16, 4, 288, 160
    x, logits = normal((T, d), 1), normal((T, E), 2, dtype=torch.float32)
    rb = normal((E,), 3, 0.1, torch.float32)
    W1, s1, W1v = random_mx((E, 2 * f, d), 4)
    W2, s2, W2v = random_mx((E, d, f), 5)
    rws, ews = ml.route_workspace(T, E, k), ml.experts_workspace(T, k, E, d, torch.bfloat16)

    def run():
        expert, weight, index, start, pos = ml.route(logits, k, workspace=rws, scores="sigmoid", bias=rb, n_groups=4, top_groups=2, scale=2.5)
        xq, xs = ml.quantize_mxfp4(x) if x_mx else (x, None)
        h = ml.experts_linear(xq, W1, start, index, act="silu", gated=True, w_scale=s1, x_scale=xs)
        hq, hs = ml.quantize_mxfp4(h) if x_mx else (h, None)
        y = ml.experts_combine(hq, W2, start, pos, weight, residual=x, w_scale=s2, x_scale=hs, workspace=ews)
        return expert, weight, h, y, pos, hq, hs

    expert, weight, h, y, pos, hq, hs = run()
    torch.cuda.synchronize()
    x64 = _quantised(x)[2] if x_mx else x.double()
    h64 = decode(hq, hs, f) if x_mx else h.double()
    if x_mx:
        v, _ = encode(h)
        assert torch.equal(h64.cpu(), v)
    ref, bound, mass = x.double(), torch.zeros((T, d), dtype=torch.float64, device="cuda"), x.double().abs()
    for e in range(E):
        t, j = torch.nonzero(expert == e, as_tuple=True)
        if t.numel() == 0:
            continue
        p = pos[t, j].long()
        check(h[p], *epilogue64(*product64(x64[t], W1v[e]), "silu", True, None, None), f"expert {e}")
        z, dz = product64(h64[p], W2v[e])
        w = weight[t, j].double()[:, None]
        ref.index_add_(0, t, w * z)
        bound.index_add_(0, t, w * dz)
        mass.index_add_(0, t, w * z.abs())
    check(y, ref, bound + (k + 2) * U * mass, "way back")

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(3):
        x.copy_(normal((T, d), 20 + i))
        logits.copy_(normal((T, E), 30 + i, dtype=torch.float32))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out[:4]]
        for g, w in zip(got, run()[:4]):
            assert torch.equal(g, w), f"replay {i}"


@pytest.mark.parametrize("x_mx", [False, True])
@pytest.mark.parametrize("T", [3, 64, 400])
def test_layer_in_a_graph_and_on_another_stream(x_mx, T):
    log(f"[mxfp4 layer] graph, stream, T={T} x_mx={x_mx}")
    l = Layer(T, 288, 514, True, False, seed=T)
    ws = l.pool.workspace(T)

    def run():
        xc, xs = _ml().quantize_mxfp4(l.x) if x_mx else (None, None)
        return _ml().linear_mxfp4(l.x, l.W, l.w_scale, l.pool, *l.meta, x_codes=xc, x_scale=xs, bias=l.bias, act="silu",
                                  gated=True, residual=l.residual, workspace=ws)

    want = run().clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = run()
    side.synchronize()
    assert torch.equal(there, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(3):
        l.x.copy_(normal(tuple(l.x.shape), 50 + i))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, run()), f"replay {i}"
