"""Host-side refusals of the MXFP4 entry points and of routing by scores: statuses that return before any HIP call."""
import ctypes

import pytest

FAKE = ctypes.c_void_p(256)        # aligned, never dereferenced
ODD = ctypes.c_void_p(264)


def _lib():
    import rank_adapter_gemm_segmented_amd as ml
    return ml.library(), ml.STATUS_CODE


def _quantize(**kw):
    a = dict(x=FAKE, dtype=1, batch=2, rows=8, d=64, codes=FAKE, scale=FAKE)
    a.update(kw)
    lib = _lib()[0]
    x, dtype, batch, rows, d, codes, scale = a.values()
    there = lib.mlora_quantize_mxfp4(x, dtype, batch, rows, d, codes, scale, None)
    assert lib.mlora_dequantize_mxfp4(codes, scale, dtype, batch, rows, d, x, None) == there
    return there


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), "DTYPE"), (dict(batch=-1), "SHAPE"), (dict(batch=1025), "SHAPE"), (dict(rows=-1), "SHAPE"),
    (dict(rows=(1 << 23) + 1), "SHAPE"), (dict(d=0), "SHAPE"), (dict(d=48), "SHAPE"), (dict(d=(1 << 17) + 32), "SHAPE"),
    (dict(x=None), "INVALID_ARG"), (dict(codes=None), "INVALID_ARG"), (dict(scale=None), "INVALID_ARG"),
    (dict(x=ODD), "INVALID_ARG"), (dict(codes=ODD), "INVALID_ARG"), (dict(scale=ODD), "INVALID_ARG"),
])
def test_quantize(bad, status):
    assert _quantize(**bad) == _lib()[1]["MLORA_ERR_" + status]


def test_nothing_to_quantize():
    assert _quantize(rows=0, x=None) == 0 and _quantize(batch=0, codes=None) == 0


def _linear(**kw):
    a = dict(x=FAKE, x_scale=None, W=FAKE, w_scale=FAKE, rows=8, E=4, d_in=64, d_out=32, start=FAKE, index=FAKE, n_pos=16, epi=None, y=FAKE)
    a.update(kw)
    return _lib()[0].mlora_experts_linear_mxfp4(*a.values(), None)


@pytest.mark.parametrize("bad,status", [
    (dict(E=0), "SHAPE"), (dict(E=1025), "SHAPE"), (dict(d_in=0), "SHAPE"), (dict(d_in=48), "SHAPE"), (dict(d_in=(1 << 17) + 32), "SHAPE"),
    (dict(d_out=0), "SHAPE"), (dict(n_pos=-1), "SHAPE"), (dict(n_pos=(1 << 23) + 1), "SHAPE"), (dict(rows=0), "SHAPE"),
    (dict(index=None), "SHAPE"), (dict(x=None), "INVALID_ARG"), (dict(W=None), "INVALID_ARG"), (dict(w_scale=None), "INVALID_ARG"),
    (dict(start=None), "INVALID_ARG"), (dict(y=None), "INVALID_ARG"), (dict(x=ODD), "INVALID_ARG"), (dict(W=ODD), "INVALID_ARG"),
    (dict(w_scale=ODD), "INVALID_ARG"), (dict(x_scale=ODD), "INVALID_ARG"),
])
def test_experts_linear(bad, status):
    assert _linear(**bad) == _lib()[1]["MLORA_ERR_" + status]


def _combine(**kw):
    a = dict(h=FAKE, h_scale=None, W=FAKE, w_scale=FAKE, T=8, k=2, E=4, d_in=64, d_out=32, start=FAKE, pos=FAKE, weight=FAKE,
             bias=None, residual=None, out=FAKE, ws=FAKE, bytes=1 << 20)
    a.update(kw)
    return _lib()[0].mlora_experts_combine_mxfp4(*a.values(), None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), "SHAPE"), (dict(k=5), "SHAPE"), (dict(d_in=48), "SHAPE"), (dict(d_out=0), "SHAPE"), (dict(h=None), "INVALID_ARG"),
    (dict(w_scale=None), "INVALID_ARG"), (dict(pos=None), "INVALID_ARG"), (dict(weight=None), "INVALID_ARG"), (dict(out=None), "INVALID_ARG"),
    (dict(h_scale=ODD), "INVALID_ARG"), (dict(w_scale=ODD), "INVALID_ARG"), (dict(bytes=16), "WORKSPACE"),
])
def test_experts_combine(bad, status):
    assert _combine(**bad) == _lib()[1]["MLORA_ERR_" + status]


def test_layer_of_no_pool():
    lib, E = _lib()
    assert lib.mlora_linear_mxfp4(FAKE, None, None, FAKE, FAKE, None, None, None, None, None, None, 4, 0, 0, None, FAKE, FAKE,
                                  1 << 20, None) == E["MLORA_ERR_INVALID_ARG"]


class Scoring(ctypes.Structure):
    _fields_ = [("scores", ctypes.c_int), ("bias", ctypes.c_void_p), ("n_groups", ctypes.c_int), ("top_groups", ctypes.c_int),
                ("scale", ctypes.c_float)]


def _route(scoring=(1, None, 4, 2, 1.0), **kw):
    a = dict(logits=FAKE, dtype=0, T=8, E=16, k=2, renorm=1, scoring=ctypes.pointer(Scoring(*scoring)) if scoring else None, expert=FAKE,
             weight=FAKE, index=FAKE, start=FAKE, pos=FAKE, ws=FAKE, bytes=1 << 20)
    a.update(kw)
    return _lib()[0].mlora_route_scored(*a.values(), None)


@pytest.mark.parametrize("bad,status", [
    (dict(scoring=None), "INVALID_ARG"), (dict(scoring=(2, None, 4, 2, 1.0)), "INVALID_ARG"), (dict(scoring=(0, 264, 4, 2, 1.0)), "INVALID_ARG"),
    (dict(scoring=(0, None, 0, 1, 1.0)), "SHAPE"), (dict(scoring=(0, None, 3, 1, 1.0)), "SHAPE"), (dict(scoring=(0, None, 4, 0, 1.0)), "SHAPE"),
    (dict(scoring=(0, None, 4, 5, 1.0)), "SHAPE"), (dict(scoring=(0, None, 16, 1, 1.0)), "SHAPE"), (dict(scoring=(0, None, 128, 128, 1.0), E=128), "SHAPE"),
    (dict(dtype=2), "DTYPE"), (dict(k=0), "SHAPE"), (dict(k=17), "SHAPE"), (dict(E=1025), "SHAPE"), (dict(T=-1), "SHAPE"), (dict(renorm=2), "INVALID_ARG"),
    (dict(logits=None), "INVALID_ARG"), (dict(start=None), "INVALID_ARG"), (dict(ws=None), "INVALID_ARG"), (dict(bytes=16), "WORKSPACE"),
])
def test_route_scored(bad, status):
    assert _route(**bad) == _lib()[1]["MLORA_ERR_" + status]
