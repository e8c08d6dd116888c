"""Host-side refusals of the epilogue, routing and expert entry points: statuses that return before any HIP call."""
import ctypes

import pytest

FAKE = ctypes.c_void_p(256)        # aligned, never dereferenced
ODD = ctypes.c_void_p(264)


def _lib():
    import rank_adapter_gemm_segmented_amd as ml
    return ml.library(), ml.STATUS_CODE


class Epi(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("act", ctypes.c_int)]


def _route(**kw):
    a = dict(logits=FAKE, dtype=0, T=8, E=16, k=2, renorm=1, expert=FAKE, weight=FAKE, index=FAKE, start=FAKE, pos=FAKE,
             ws=FAKE, bytes=1 << 20)
    a.update(kw)
    return _lib()[0].mlora_route(*a.values(), None)


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), "DTYPE"), (dict(k=0), "SHAPE"), (dict(k=17), "SHAPE"), (dict(E=0), "SHAPE"), (dict(E=1025), "SHAPE"),
    (dict(E=1024, k=65), "SHAPE"), (dict(T=-1), "SHAPE"), (dict(T=(1 << 20) + 1), "SHAPE"), (dict(T=1 << 20, k=16), "SHAPE"),
    (dict(renorm=2), "INVALID_ARG"), (dict(logits=None), "INVALID_ARG"), (dict(logits=ODD), "INVALID_ARG"),
    (dict(expert=None), "INVALID_ARG"), (dict(weight=None), "INVALID_ARG"), (dict(index=None), "INVALID_ARG"),
    (dict(start=None), "INVALID_ARG"), (dict(pos=None), "INVALID_ARG"), (dict(ws=None), "INVALID_ARG"), (dict(bytes=16), "WORKSPACE"),
])
def test_route(bad, status):
    assert _route(**bad) == _lib()[1]["MLORA_ERR_" + status]


def _linear(**kw):
    a = dict(x=FAKE, W=FAKE, w_scale=None, dtype=1, rows=8, E=4, d_in=64, d_out=32, start=FAKE, index=FAKE, n_pos=16, epi=None, y=FAKE)
    a.update(kw)
    return _lib()[0].mlora_experts_linear(*a.values(), None)


def _epi(bias=None, residual=None, act=0):
    return ctypes.cast(ctypes.pointer(Epi(bias, residual, act)), ctypes.c_void_p)


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=5), "DTYPE"), (dict(dtype=0, w_scale=FAKE), "DTYPE"), (dict(E=0), "SHAPE"), (dict(E=1025), "SHAPE"),
    (dict(d_in=0), "SHAPE"), (dict(d_in=60), "SHAPE"), (dict(d_in=72, w_scale=FAKE), "SHAPE"), (dict(dtype=0, d_in=6), "SHAPE"),
    (dict(d_in=(1 << 17) + 8), "SHAPE"), (dict(d_out=0), "SHAPE"), (dict(d_out=(1 << 17) + 1), "SHAPE"), (dict(n_pos=-1), "SHAPE"),
    (dict(n_pos=(1 << 23) + 1), "SHAPE"), (dict(rows=-1), "SHAPE"), (dict(rows=0), "SHAPE"), (dict(index=None), "SHAPE"),
    (dict(x=None), "INVALID_ARG"), (dict(W=None), "INVALID_ARG"), (dict(start=None), "INVALID_ARG"), (dict(y=None), "INVALID_ARG"),
    (dict(x=ODD), "INVALID_ARG"), (dict(W=ODD), "INVALID_ARG"), (dict(y=ODD), "INVALID_ARG"),
])
def test_experts_linear(bad, status):
    assert _linear(**bad) == _lib()[1]["MLORA_ERR_" + status]


def test_experts_linear_epilogue():
    E = _lib()[1]
    assert _linear(epi=_epi(act=5)) == E["MLORA_ERR_INVALID_ARG"]
    assert _linear(epi=_epi(act=-1)) == E["MLORA_ERR_INVALID_ARG"]
    assert _linear(epi=_epi(act=32)) == E["MLORA_ERR_INVALID_ARG"]
    assert _linear(epi=_epi(residual=256)) == E["MLORA_ERR_INVALID_ARG"]
    assert _linear(epi=_epi(bias=264)) == E["MLORA_ERR_INVALID_ARG"]
    assert _linear(epi=_epi(act=16), d_out=31) == E["MLORA_ERR_SHAPE"]
    assert _linear(n_pos=0, x=None, y=None) == 0


def _combine(**kw):
    a = dict(h=FAKE, W=FAKE, w_scale=None, dtype=1, T=8, k=2, E=4, d_in=64, d_out=32, start=FAKE, pos=FAKE, weight=FAKE,
             bias=None, residual=None, out=FAKE, ws=FAKE, bytes=1 << 20)
    a.update(kw)
    return _lib()[0].mlora_experts_combine(*a.values(), None)


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=5), "DTYPE"), (dict(T=-1), "SHAPE"), (dict(k=0), "SHAPE"), (dict(k=5), "SHAPE"), (dict(d_in=60), "SHAPE"),
    (dict(d_out=0), "SHAPE"), (dict(h=None), "INVALID_ARG"), (dict(W=None), "INVALID_ARG"), (dict(start=None), "INVALID_ARG"),
    (dict(pos=None), "INVALID_ARG"), (dict(weight=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"), (dict(ws=None), "INVALID_ARG"),
    (dict(bias=ODD), "INVALID_ARG"), (dict(residual=ODD), "INVALID_ARG"), (dict(bytes=16), "WORKSPACE"),
])
def test_experts_combine(bad, status):
    assert _combine(**bad) == _lib()[1]["MLORA_ERR_" + status]


def test_no_work_and_sizes():
    lib, _ = _lib()
    assert _combine(T=0, h=None, out=None) == 0
    assert lib.mlora_route_workspace_bytes(0, 8, 2) >= 256 and lib.mlora_route_workspace_bytes(1, 8, 9) == 0
    assert lib.mlora_route_workspace_bytes(4096, 64, 8) >= 64 * 4
    assert lib.mlora_experts_workspace_bytes(64, 8, 64, 4096, 1) >= 64 * 8 * 4096 * 4
    assert lib.mlora_experts_workspace_bytes(64, 8, 4, 4096, 1) == 0 and lib.mlora_experts_workspace_bytes(64, 8, 64, 0, 1) == 0


@pytest.mark.parametrize("n_experts", [1, 8, 127, 1024])
def test_a_workspace_for_a_batch_holds_every_smaller_one(n_experts):
    lib, _ = _lib()
    T = sorted({1 << i for i in range(21)} | {(1 << i) + 1 for i in range(20)} | set(range(8000, 8400, 7)) | set(range(127, 131)))
    sizes = [lib.mlora_route_workspace_bytes(t, n_experts, 1) for t in T]
    assert sizes == sorted(sizes)
    sizes = [lib.mlora_experts_workspace_bytes(t, 1, n_experts, 48, 0) for t in T]
    assert sizes == sorted(sizes)


def test_products_past_the_largest_are_refused():
    lib, E = _lib()
    assert lib.mlora_experts_workspace_bytes(1 << 20, 8, 8, 1 << 13, 1) == 1 << 38      # 2^36 elements in fp32
    assert lib.mlora_experts_workspace_bytes(1 << 20, 8, 8, (1 << 13) + 8, 1) == 0
    assert lib.mlora_experts_linear(FAKE, FAKE, None, 1, 1 << 20, 8, 64, (1 << 13) + 8, FAKE, FAKE, 1 << 23, None, FAKE, None) == E["MLORA_ERR_SHAPE"]
    assert _combine(T=1 << 20, k=8, E=8, d_out=(1 << 13) + 8) == E["MLORA_ERR_SHAPE"]


def test_epilogue_of_no_pool():
    lib, E = _lib()
    none = ctypes.c_void_p(None)
    assert lib.mlora_linear_epilogue(FAKE, FAKE, none, None, None, None, None, None, 4, 0, 0, None, FAKE, FAKE, 1 << 20, None) == E["MLORA_ERR_INVALID_ARG"]
    assert lib.mlora_linear_tokens_epilogue(FAKE, FAKE, none, None, None, 4, 0, None, FAKE, FAKE, 1 << 20, None) == E["MLORA_ERR_INVALID_ARG"]
    assert lib.mlora_linear_fp8w_epilogue(FAKE, FAKE, FAKE, none, None, None, None, None, None, 4, 0, 0, None, FAKE, FAKE, 1 << 20, None) == E["MLORA_ERR_INVALID_ARG"]
