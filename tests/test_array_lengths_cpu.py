"""Arrays shorter than a call reads are refused before it is made. No device is needed: the pool is none (its handle is
NULL), so a call whose arrays are long enough ends with the library's own MLORA_ERR_INVALID_ARG."""
import pytest
import torch

T, N, D_IN, D_OUT = 6, 3, 64, 32
LENGTHS = {"seg_start": N + 1, "seg_adapter": N, "seg_rank": N, "seg_scale": N, "token_index": T}


def _pool(ml, dtype=torch.bfloat16):
    pool = object.__new__(ml.Pool)
    pool.d_in, pool.d_out, pool.dtype, pool.max_rank, pool.capacity, pool.handle = D_IN, D_OUT, dtype, 8, 4, None
    return pool


def _meta(**short):
    n = {**LENGTHS, **short}
    return {k: torch.zeros(v, dtype=torch.float32 if k == "seg_scale" else torch.int32) for k, v in n.items()}


@pytest.fixture
def ml(monkeypatch):
    import rank_adapter_gemm_segmented_amd as ml
    from rank_adapter_gemm_segmented_amd import binding
    monkeypatch.setattr(binding, "_device", lambda: -1)          # the device of host tensors
    monkeypatch.setattr(binding, "_raw_stream", lambda dev: None)
    return ml


def _epilogue(ml, lora_on=1, fp8=False, **short):
    W = torch.zeros((D_OUT, D_IN), dtype=torch.uint8 if fp8 else torch.bfloat16)
    return ml.linear_epilogue(torch.zeros((T, D_IN), dtype=torch.bfloat16), W, _pool(ml), lora_on=lora_on, act="silu",
                              w_scale=torch.ones(D_OUT) if fp8 else None, workspace=torch.empty(256, dtype=torch.uint8),
                              **_meta(**short))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name,n", [("seg_start", N), ("seg_start", 0), ("seg_rank", N - 1), ("seg_scale", N - 1),
                                    ("seg_scale", 0), ("token_index", T - 1), ("seg_adapter", N + 1)])
def test_epilogue_refuses_short_arrays(ml, name, n, fp8):
    # (a longer seg_adapter makes the others short: it gives the number of segments)
    with pytest.raises(ValueError, match="n_seg" if name != "token_index" else "token_index"):
        _epilogue(ml, fp8=fp8, **{name: n})


@pytest.mark.parametrize("longer", [{}, {"seg_start": N + 5}, {"seg_rank": N + 1, "seg_scale": N + 1}, {"token_index": T + 3},
                                    {"seg_adapter": N - 1}])
def test_epilogue_takes_arrays_that_hold_the_batch(ml, longer):
    with pytest.raises(ml.MloraError) as e:      # (the missing pool)
        _epilogue(ml, **longer)
    assert e.value.code == ml.STATUS_CODE["MLORA_ERR_INVALID_ARG"]


def test_epilogue_does_not_read_them_with_the_adapters_off(ml):
    with pytest.raises(ml.MloraError) as e:
        _epilogue(ml, lora_on=0, seg_start=0, token_index=0)
    assert e.value.code == ml.STATUS_CODE["MLORA_ERR_INVALID_ARG"]


# ---- the plain layer and its helpers: on host tensors an accepted call ends at the check for device tensors

def _plain(ml, name, lora_on=1, out=None, **short):
    m, pool = _meta(**short), _pool(ml)
    x, W = torch.zeros((T, D_IN), dtype=torch.bfloat16), torch.zeros((D_OUT, D_IN), dtype=torch.bfloat16)
    ws = {} if name == "linear_noalloc" else {"workspace": torch.empty(256, dtype=torch.uint8)}
    if name == "linear_fp8w":
        return ml.linear_fp8w(x, W.to(torch.uint8), torch.ones(D_OUT), pool, lora_on=lora_on, out=out, **ws, **m)
    return getattr(ml, name)(x, W, pool, lora_on=lora_on, out=out, **ws, **m)


PLAIN = ["linear", "linear_noalloc", "linear_fp8w"]


@pytest.mark.parametrize("call", PLAIN)
@pytest.mark.parametrize("name,n", [("seg_start", N), ("seg_rank", N - 1), ("seg_scale", N - 1), ("token_index", T - 1),
                                    ("seg_adapter", N + 1)])
def test_layer_refuses_short_arrays(ml, call, name, n):
    with pytest.raises(ValueError, match="n_seg" if name != "token_index" else "token_index"):
        _plain(ml, call, **{name: n})


@pytest.mark.parametrize("call", PLAIN)
@pytest.mark.parametrize("longer", [{}, {"seg_start": N + 5}, {"token_index": T + 3}, {"lora_on": 0, "seg_rank": 0}])
def test_layer_takes_arrays_that_hold_the_batch(ml, call, longer):
    with pytest.raises(TypeError, match="device tensor"):
        _plain(ml, call, **longer)


@pytest.mark.parametrize("n", [T - 1, 0])
def test_unsorted_layer_refuses_short_arrays(ml, n):
    x, W = torch.zeros((T, D_IN), dtype=torch.bfloat16), torch.zeros((D_OUT, D_IN), dtype=torch.bfloat16)
    ids, scale, ws = torch.zeros(T, dtype=torch.int32), torch.ones(4), torch.empty(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="token_adapter"):
        ml.linear_tokens(x, W, _pool(ml), ids[:n], scale, workspace=ws)
    with pytest.raises(TypeError, match="device tensor"):
        ml.linear_tokens(x, W, _pool(ml), ids, scale, workspace=ws)


@pytest.mark.parametrize("n", [0, 4, 6])
def test_route_refuses_another_number_of_outputs(ml, n):
    P, E = T * 2, 8
    out = [torch.zeros(P, dtype=torch.int32), torch.zeros(P), torch.zeros(P, dtype=torch.int32),
           torch.zeros(E + 1, dtype=torch.int32), torch.zeros(P, dtype=torch.int32), torch.zeros(P, dtype=torch.int32)]
    with pytest.raises(ValueError, match="out must be"):
        ml.route(torch.zeros((T, E)), 2, out=tuple(out[:n]), workspace=torch.empty(4096, dtype=torch.uint8))


@pytest.mark.parametrize("call", PLAIN + ["linear_epilogue"])
def test_no_tokens_need_no_arrays(ml, call):
    none = {k: v[:0] for k, v in _meta().items()}
    x, W, ws = torch.zeros((0, D_IN), dtype=torch.bfloat16), torch.zeros((D_OUT, D_IN), dtype=torch.bfloat16), {}
    if call != "linear_noalloc":
        ws = {"workspace": torch.empty(256, dtype=torch.uint8)}
    args = (W.to(torch.uint8), torch.ones(D_OUT)) if call == "linear_fp8w" else (W,)
    with pytest.raises(ml.MloraError if call == "linear_epilogue" else TypeError):   # as with any batch here: no pool, no device
        getattr(ml, call)(x, *args, _pool(ml), **ws, **none)
