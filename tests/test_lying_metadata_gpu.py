"""Expert products on segments, indices and positions that lie: nothing outside the call's own arrays is written, whatever
form the batch takes, and an index out of range reads the row that it is clamped to."""
import pytest
import torch

from gpu_util import log
from op_util import check, e4m3, normal, product64

pytestmark = pytest.mark.gpu

GUARD = 8          # rows before and behind y (whole multiples of 16 bytes)
MARK = 7.0

# streamed, then tiles of 32, 64, 128 and 256 positions; FP8 streamed, 64 and 128; fp32
FORMS = {
    "stream": ("bf16", 1, 72, 2056), "32": ("bf16", 5, 72, 2056), "64": ("bf16", 30, 72, 2056), "128": ("bf16", 100, 72, 2056),
    "256": ("bf16", 201, 72, 4104), "FP8 stream": ("fp8w", 8, 80, 2056), "FP8 64": ("fp8w", 30, 80, 2056),
    "FP8 128": ("fp8w", 100, 80, 2056), "f32": ("f32", 20, 72, 264),
}
E = 16


def _ml():
    import rank_adapter_gemm_segmented_amd as ml
    return ml


def _lies(n):
    g = torch.Generator().manual_seed(n)
    yield "far too many", [i * n for i in range(E + 1)]
    yield "descending", [n - i for i in range(E + 1)]
    yield "every other one the whole batch", [0 if i % 2 == 0 else n for i in range(E + 1)]
    yield "far out of range", [-(1 << 30) if i % 2 == 0 else 1 << 30 for i in range(E + 1)]
    yield "anything", torch.randint(-n, 2 * n, (E + 1,), generator=g).tolist()


def _operands(form):
    kind, per, d_in, d_out = FORMS[form]
    n = E * per
    dt = torch.float32 if kind == "f32" else torch.bfloat16
    W, scale = normal((E, d_out, d_in), 1, 0.05, dt), None
    W64 = W.double()
    if kind == "fp8w":
        W, scale, W64 = e4m3(W)
    return n, normal((n, d_in), 2, 1.0, dt), W, scale, W64


def _guarded(rows, cols, dtype):
    """rows x cols in the middle of a buffer of marks, and the buffer."""
    buf = torch.full((GUARD + rows + GUARD, cols), MARK, dtype=dtype, device="cuda")
    return buf[GUARD:GUARD + rows], buf


def _whole(buf, rows):
    assert torch.all(buf[:GUARD] == MARK) and torch.all(buf[GUARD + rows:] == MARK), "written outside"


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("form", FORMS, ids=[f.replace(" ", "_") for f in FORMS])
def test_segments(form, gated):
    n, x, W, scale, _ = _operands(form)
    d_out = W.shape[1]
    index = torch.randint(-5, n + 5, (n,), generator=torch.Generator().manual_seed(1)).int().cuda()
    for what, seg in _lies(n):
        log(f"[lies] experts {form} gated={gated} {what}")
        y, buf = _guarded(n, d_out // 2 if gated else d_out, x.dtype)
        _ml().experts_linear(x, W, _i32(seg), index, act="silu", gated=gated, w_scale=scale, out=y)
        torch.cuda.synchronize()
        _whole(buf, n)


@pytest.mark.parametrize("form", FORMS, ids=[f.replace(" ", "_") for f in FORMS])
def test_way_back(form):
    ml = _ml()
    n, h, W, scale, _ = _operands(form)
    T, d_out = n // 2, W.shape[1]
    need = ml.library().mlora_experts_workspace_bytes(T, 2, E, d_out, 0 if h.dtype == torch.float32 else 1)
    for what, seg in _lies(n):
        log(f"[lies] way back {form} {what}")
        out, buf = _guarded(T, d_out, h.dtype)
        space = torch.full((need + 512,), 165, dtype=torch.uint8, device="cuda")
        position = torch.randint(-n, 2 * n, (T, 2), generator=torch.Generator().manual_seed(2)).int().cuda()
        ml.experts_combine(h, W, _i32(seg), position, torch.rand((T, 2), device="cuda"), w_scale=scale, out=out,
                           workspace=space[256:256 + need])
        torch.cuda.synchronize()
        _whole(buf, T)
        assert torch.all(space[:256] == 165) and torch.all(space[256 + need:] == 165), "written outside the workspace"


@pytest.mark.parametrize("form", FORMS, ids=[f.replace(" ", "_") for f in FORMS])
def test_index_is_clamped(form):
    log(f"[lies] index of {form}")
    n, x, W, scale, W64 = _operands(form)
    index = torch.randint(-n, 2 * n, (n,), generator=torch.Generator().manual_seed(3))
    index[0], index[1] = -(1 << 31), (1 << 31) - 1
    start = [e * (n // E) for e in range(E + 1)]
    y, buf = _guarded(n, W.shape[1], x.dtype)
    _ml().experts_linear(x, W, _i32(start), index.int().cuda(), w_scale=scale, out=y)
    torch.cuda.synchronize()
    _whole(buf, n)
    rows = index.clamp(0, n - 1).cuda()
    for e in range(E):
        p = slice(start[e], start[e + 1])
        check(y[p], *product64(x[rows[p]], W64[e]), f"{form} expert {e}")
