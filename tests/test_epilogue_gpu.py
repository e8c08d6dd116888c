"""The layer with bias, activation, gate and residual (mlora_*_epilogue) against 64 bits."""
import pytest
import torch

from gpu_util import log
from op_util import U, check, e4m3, epilogue64, normal, product64

pytestmark = pytest.mark.gpu


def _ml():
    import rank_adapter_gemm_segmented_amd as ml
    return ml


class Layer:
    """A layer, its adapters (mixed ranks, some tokens without one, an empty segment) and its batch."""

    def __init__(self, dtype, T, d_in, d_out, gated, seed=0, ranks=(8, 16, 33, 64), bias=True, residual=True, fused=False,
                 shuffled=False, fp8=False, max_run=9):
        ml = _ml()
        self.T, self.d_in, self.d_out, self.gated, self.dtype = T, d_in, d_out, gated, dtype
        self.W = normal((d_out, d_in), seed, 0.05, dtype)
        self.w_scale, self.W64 = None, self.W.double()
        if fp8:
            self.W, self.w_scale, self.W64 = e4m3(self.W)
        self.x = normal((T, d_in), seed + 1, 1.0, dtype)
        n = len(ranks)
        total = [2 * r if fused else r for r in ranks]
        self.pool = ml.Pool(d_in, d_out, dtype, max(total), n + 1)
        self.AB = {}
        for a, r in enumerate(ranks):
            if fused:
                half = d_out // 2
                sl = [(normal((r, d_in), seed + 10 * a + m, 0.05, dtype), normal((half, r), seed + 10 * a + 5 + m, 0.05, dtype))
                      for m in range(2)]
                self.pool.register_fused(a, sl)
                A = torch.cat([s[0] for s in sl])
                B = torch.zeros((d_out, 2 * r), dtype=dtype, device="cuda")
                B[:half, :r], B[half:, r:] = sl[0][1], sl[1][1]
            else:
                A, B = normal((r, d_in), seed + 10 * a, 0.05, dtype), normal((d_out, r), seed + 10 * a + 5, 0.05, dtype)
                self.pool.register(a, A, B)
            self.AB[a] = (A, B)
        g = torch.Generator().manual_seed(seed)
        ids, starts, at, a = [], [0], 0, 0
        while at < T:
            run = min(T - at, int(torch.randint(1, max_run + 1, (1,), generator=g)))
            ids.append(a % (n + 1) - 1)      # -1, 0, 1, ...
            at, a = at + run, a + 1
            starts.append(at)
            if a == 3:                        # an empty segment
                ids.append(0)
                starts.append(at)
        self.ids, self.starts = ids, starts
        scale = [0.0 if i < 0 else 0.5 + i for i in ids]
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        self.meta = (i32(starts), i32(ids), i32([total[i] if i >= 0 else 0 for i in ids]), torch.tensor(scale, device="cuda"))
        self.index = torch.randperm(T, generator=g).int().cuda() if shuffled else None
        self.bias = normal((d_out,), seed + 2, 0.5, dtype) if bias else None
        d_y = d_out // 2 if gated else d_out
        self.residual = normal((T, d_y), seed + 3, 1.0, dtype) if residual else None
        # z in 64 bits and its bound, in batch order
        self.z, self.dz = product64(self.x, self.W64)
        self.z_off, self.dz_off = self.z.clone(), self.dz.clone()
        for i, s in zip(ids, scale):
            lo, hi = starts.pop(0), starts[0]
            if i < 0 or hi == lo:
                continue
            rows = self.index[lo:hi].long() if shuffled else torch.arange(lo, hi, device="cuda")
            A, B = self.AB[i]
            v, dv = product64(self.x[rows], A)
            # the MFMA expand takes v as two bf16 parts (2^-16 relative); sums over the rank as products
            dv = dv + 2.0 ** -16 * v.abs()
            self.z[rows] += s * (v @ B.double().T)
            self.dz[rows] += s * (dv @ B.double().abs().T) + 2 * s * (B.shape[1] + 2) * U * (v.abs() @ B.double().abs().T) \
                + 2 * U * self.z[rows].abs()

    def run(self, act, lora_on=1, **kw):
        kw = {"bias": self.bias, "residual": self.residual, **kw}
        y = _ml().linear_epilogue(self.x, self.W, self.pool, *self.meta, lora_on=lora_on, token_index=self.index if lora_on else None,
                                  act=act, gated=self.gated, w_scale=self.w_scale, **kw)
        torch.cuda.synchronize()
        return y

    def check(self, act, lora_on=1, what=""):
        z, dz = (self.z, self.dz) if lora_on else (self.z_off, self.dz_off)
        worst = check(self.run(act, lora_on), *epilogue64(z, dz, act, self.gated, self.bias, self.residual),
                      f"{what} T={self.T} {self.d_in}->{self.d_out} {act} gated={self.gated} lora={lora_on}")
        log(f"  error / bound {worst:.3f}")


ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]

# (T, d_in, d_out): decode tiles of 16, 32 and 64 tokens, whole and ragged rows; the tiled paths (64x128, 128x128,
# 64x256, 256x256 tiles); fewer columns than a k step
DECODE = [(1, 264, 192), (1, 4104, 34), (9, 72, 2), (17, 520, 250), (33, 264, 1026), (64, 1048, 1000)]
TILED = [(65, 136, 322), (130, 264, 250), (100, 264, 24640), (300, 72, 12800), (1100, 264, 12290)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("i", range(len(DECODE)))
def test_decode(i, gated):
    T, d_in, d_out = DECODE[i]
    log(f"[epilogue] decode T={T} {d_in}->{d_out} gated={gated}")
    layer = Layer(torch.bfloat16, T, d_in, d_out, gated, seed=i, shuffled=i % 2 == 1)
    layer.check(ACTS[i % 5])
    layer.check(ACTS[(i + 2) % 5], lora_on=0)


# a few tokens on layers of many rows: W streamed over the whole of d_in
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,d_in,d_out,fp8", [(1, 264, 16640, False), (5, 1040, 16390, False), (8, 72, 16400, False),
                                              (8, 528, 17000, True), (3, 16, 16386, True), (9, 272, 16640, True)])
def test_wide_decode(T, d_in, d_out, fp8, gated):
    log(f"[epilogue] wide decode T={T} {d_in}->{d_out} fp8={fp8} gated={gated}")
    layer = Layer(torch.bfloat16, T, d_in, d_out, gated, seed=T, shuffled=T > 3, fp8=fp8, max_run=2)
    layer.check("silu")
    layer.check("gelu", lora_on=0)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("i", range(len(TILED)))
def test_tiled(i, gated):
    T, d_in, d_out = TILED[i]
    log(f"[epilogue] tiled T={T} {d_in}->{d_out} gated={gated}")
    layer = Layer(torch.bfloat16, T, d_in, d_out, gated, seed=i, shuffled=i % 2 == 0, max_run=40)
    layer.check(ACTS[i % 5])
    layer.check(ACTS[(i + 2) % 5], lora_on=0)


# the 64x256 tile, and the largest one over many stages, with many short segments, high ranks and fused pools
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,d_in,d_out,kw", [
    (257, 264, 6402, {}), (769, 1040, 16402, {"max_run": 100}), (2050, 520, 6146, {"max_run": 3}),
    (1100, 264, 12320, {"max_run": 2, "ranks": (64, 16, 33, 128)}), (1030, 136, 12288, {"max_run": 60, "ranks": (200, 8)}),
    (1100, 264, 12320, {"max_run": 30, "ranks": (16, 24), "fused": True})])
def test_tiled_segments(T, d_in, d_out, kw, gated):
    log(f"[epilogue] tiled T={T} {d_in}->{d_out} {kw} gated={gated}")
    layer = Layer(torch.bfloat16, T, d_in, d_out, gated, seed=T, shuffled=True, **kw)
    layer.check("silu")
    layer.check("relu", lora_on=0)


@pytest.mark.parametrize("gated", [False, True])
def test_tiled_mfma_and_dense_expand(gated, monkeypatch):
    log(f"[epilogue] both expand forms gated={gated}")
    layer = Layer(torch.bfloat16, 140, 264, 2048, gated, seed=3)
    for form in ("dense", "mfma"):
        monkeypatch.setenv("MLORA_EXPAND", form)
        layer.check("silu", what=form)


@pytest.mark.parametrize("T", [7, 64, 200])
@pytest.mark.parametrize("gated", [False, True])
def test_low_rank_and_fused_pools(T, gated):
    log(f"[epilogue] low-rank and fused pools T={T} gated={gated}")
    Layer(torch.bfloat16, T, 264, 320, gated, seed=1, ranks=(8, 16), max_run=2).check("silu")
    Layer(torch.bfloat16, T, 264, 320, gated, seed=2, ranks=(16, 16), fused=True).check("silu", what="fused")
    Layer(torch.bfloat16, T, 264, 320, gated, seed=3, ranks=(8, 24), fused=True).check("gelu", what="fused, unequal")


@pytest.mark.parametrize("T,d_in,d_out", [(1, 16, 64), (16, 256, 256), (50, 516, 90), (33, 4, 6)])
@pytest.mark.parametrize("gated", [False, True])
def test_f32(T, d_in, d_out, gated):
    log(f"[epilogue] f32 T={T} {d_in}->{d_out} gated={gated}")
    layer = Layer(torch.float32, T, d_in, d_out, gated, seed=T, ranks=(8, 3), shuffled=T > 20)
    for act in ACTS:
        layer.check(act)
    layer.check("gelu", lora_on=0)


@pytest.mark.parametrize("T,d_in,d_out,kw", [(300, 256, 256, {}), (600, 516, 130, {"ranks": (64, 40, 17), "max_run": 90}),
                                             (3, 1024, 64, {"ranks": (200, 9), "max_run": 1}), (77, 260, 514, {"ranks": (16,), "max_run": 2})])
@pytest.mark.parametrize("gated", [False, True])
def test_f32_by_position(T, d_in, d_out, kw, gated):
    log(f"[epilogue] f32 T={T} {d_in}->{d_out} {kw} gated={gated}")
    layer = Layer(torch.float32, T, d_in, d_out, gated, seed=T, shuffled=T > 20, **kw)
    layer.check("silu")
    layer.check("none", lora_on=0)


@pytest.mark.parametrize("T,d_in,d_out", [(1, 1040, 450), (20, 272, 64), (64, 2064, 520)])
@pytest.mark.parametrize("gated", [False, True])
def test_fp8_weight(T, d_in, d_out, gated):
    log(f"[epilogue] FP8 weight T={T} {d_in}->{d_out} gated={gated}")
    layer = Layer(torch.bfloat16, T, d_in, d_out, gated, seed=T, fp8=True)
    layer.check("silu")
    layer.check("gelu_tanh", lora_on=0)


@pytest.mark.parametrize("T", [5, 64, 150, 300])
@pytest.mark.parametrize("parts", ["bias", "residual", "act", "nothing"])
def test_each_part_alone(T, parts):
    log(f"[epilogue] {parts} alone, T={T}")
    ml = _ml()
    layer = Layer(torch.bfloat16, T, 264, 328, False, seed=4, bias=parts == "bias", residual=parts == "residual")
    layer.check("silu" if parts == "act" else "none")
    if parts == "nothing":
        y = ml.linear(layer.x, layer.W, layer.pool, *layer.meta)
        assert torch.equal(layer.run("none"), y)


@pytest.mark.parametrize("T", [5, 64, 150, 300])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_residual_in_place_and_repeats(T, dtype):
    log(f"[epilogue] residual in place T={T} {dtype}")
    layer = Layer(dtype, T, 264, 328, True, seed=5)
    y = layer.run("silu")
    assert torch.equal(layer.run("silu"), y)
    inplace = layer.residual.clone()
    assert torch.equal(layer.run("silu", residual=inplace, out=inplace), y)


@pytest.mark.parametrize("T", [6, 64, 200])
@pytest.mark.parametrize("gated", [False, True])
def test_unsorted_batch(T, gated):
    log(f"[epilogue] unsorted T={T} gated={gated}")
    ml = _ml()
    layer = Layer(torch.bfloat16, T, 264, 640, gated, seed=6, ranks=(16, 16, 16))
    ids = torch.randint(-1, 3, (T,), generator=torch.Generator().manual_seed(T)).int().cuda()
    scale = torch.tensor([0.5, 1.5, 2.0, 0.0], device="cuda")
    y = ml.linear_tokens_epilogue(layer.x, layer.W, layer.pool, ids, scale, bias=layer.bias, act="silu", gated=gated,
                                  residual=layer.residual)
    z, dz = layer.z_off.clone(), layer.dz_off.clone()
    for a in range(3):
        rows = torch.nonzero(ids == a)[:, 0]
        A, B = layer.AB[a]
        v, dv = product64(layer.x[rows], A)
        dv = dv + 2.0 ** -16 * v.abs()
        s = float(scale[a])
        z[rows] += s * (v @ B.double().T)
        dz[rows] += s * (dv @ B.double().abs().T) + 2 * s * 18 * U * (v.abs() @ B.double().abs().T) + 2 * U * z[rows].abs()
    check(y, *epilogue64(z, dz, "silu", gated, layer.bias, layer.residual), "unsorted")


@pytest.mark.parametrize("T", [30, 200])
def test_captured_and_on_another_stream(T):
    log(f"[epilogue] graph replays T={T}")
    ml = _ml()
    layer = Layer(torch.bfloat16, T, 264, 640, True, seed=7)
    ws = layer.pool.workspace(T)
    out = torch.empty((T, 320), dtype=torch.bfloat16, device="cuda")
    run = lambda y: ml.linear_epilogue(layer.x, layer.W, layer.pool, *layer.meta, bias=layer.bias, act="silu", gated=True,  # noqa: E731
                                       residual=layer.residual, out=y, workspace=ws)
    run(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out)
    for i in range(3):
        layer.x.copy_(normal((T, 264), 100 + i))
        graph.replay()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            y = run(torch.empty_like(out))
        s.synchronize()
        assert torch.equal(out, y)


def test_no_tokens():
    log("[epilogue] no tokens")
    layer = Layer(torch.bfloat16, 4, 64, 32, True)
    y = _ml().linear_epilogue(layer.x[:0], layer.W, layer.pool, lora_on=0, act="silu", gated=True)
    assert y.shape == (0, 16)


def test_extreme_values_pass_through():
    log("[epilogue] saturated activations and NaN")
    ml = _ml()
    pool = ml.Pool(64, 32, torch.bfloat16, 8, 1)
    for T in (2, 70):
        x, W = torch.zeros((T, 64), dtype=torch.bfloat16, device="cuda"), normal((32, 64), 1)
        bias = torch.zeros(32, dtype=torch.bfloat16, device="cuda")
        bias[0], bias[1], bias[2], bias[3] = 1e30, -1e30, float("nan"), float("inf")
        for act in ACTS:
            y = ml.linear_epilogue(x, W, pool, lora_on=0, bias=bias, act=act)
            torch.cuda.synchronize()
            assert torch.all(y[:, 0] == bias[0]) and torch.all(torch.isnan(y[:, 2])) and torch.all(y[:, 3] == float("inf")), act
            assert torch.all(y[:, 1] == (bias[1] if act == "none" else 0)), act


def test_refusals():
    log("[epilogue] refusals")
    ml = _ml()
    layer = Layer(torch.bfloat16, 8, 64, 31, False)
    x, W, pool = layer.x, layer.W, layer.pool
    call = lambda **kw: ml.linear_epilogue(x, W, pool, lora_on=0, **kw)  # noqa: E731
    buf = torch.zeros(8 * 31 + 8, dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: call(act="swish"), lambda: call(gated=True), lambda: call(bias=layer.bias[:30]),
                lambda: call(bias=layer.bias.float()), lambda: call(residual=layer.residual[:, :30]),
                lambda: call(residual=layer.residual.float()), lambda: call(residual=layer.residual.cpu()),
                lambda: call(out=torch.empty((8, 30), dtype=torch.bfloat16, device="cuda")),
                lambda: call(residual=torch.zeros((31, 8), dtype=torch.bfloat16, device="cuda").T)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ml.MloraError) as e:      # not 16-byte aligned
        call(residual=buf[1:1 + 8 * 31].view(8, 31))
    assert e.value.code == ml.STATUS_CODE["MLORA_ERR_INVALID_ARG"]
    fp8 = Layer(torch.bfloat16, 65, 64, 32, False, fp8=True)
    with pytest.raises(ml.MloraError) as e:
        fp8.run("silu")
    assert e.value.code == ml.STATUS_CODE["MLORA_ERR_SHAPE"]
