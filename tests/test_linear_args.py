"""linear, linear_nvfp4 and what calls them refuse an output or an activation that
does not fit the weight before anything is launched, with and without an epilogue
(CPU: tensors that say they are on a device; a call that is not refused ends
with the library's status for a machine without one)."""
import pytest
import torch

import structured_sparse_quantized_b200 as ss
from test_stream_memory import OnDevice, on_device

BF = torch.bfloat16


def zeros(*shape, dtype=BF):
    return on_device(torch.zeros(*shape, dtype=dtype))


def packed(pattern, q, N, K):
    """A compressed weight's tensors, empty."""
    dense = pattern == "dense"
    if q == "nvfp4":
        _, K_lp = ss.ss_fp4_shape(pattern, K)
        return (zeros(N, K_lp // (2 if dense else 4), dtype=torch.uint8),
                None if dense else zeros(*ss.meta_shape(N, K_lp // 2), dtype=torch.uint8),
                zeros(ss.ss_fp4_scale_bytes(N, K_lp, 16 if dense else 32), dtype=torch.uint8),
                zeros(4, dtype=torch.float32))
    K_lp = ss.ss_slide_shape(pattern, K)[2]
    return (zeros(N, K_lp if dense else K_lp // 2, dtype=BF if q == "bf16" else torch.uint8),
            None if dense else zeros(*ss.meta_shape(N, K_lp), dtype=torch.uint8),
            None if q == "bf16" else zeros(N, dtype=torch.float32))


@pytest.fixture
def device(monkeypatch):
    """The quantisation leaves empty codes; the products are not reached."""
    from structured_sparse_quantized_b200 import _build
    _build.build()
    monkeypatch.setattr(ss, "_stream", lambda s: None)
    monkeypatch.setattr(ss, "_raw_stream", lambda s, d: None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(ss, "_new", lambda like, shape, dtype, stream: zeros(*shape, dtype=dtype))
    for name in ("ss_quant_lift_act", "ss_quant_lift_act_nvfp4", "ss_norm_quant_lift_act"):
        monkeypatch.setattr(ss, name, lambda *a, **k: None)


def call(pattern, q, X, w, **kw):
    if q == "nvfp4":
        return ss.linear_nvfp4(X, w, pattern, **kw)
    return ss.linear(X, w, pattern, q, **kw)


CASES = [(p, q) for q in ("int8", "bf16", "nvfp4") for p in ("6:8", "dense")]


@pytest.mark.parametrize("pattern,q", CASES)
@pytest.mark.parametrize("shape", [(3, 32), (4, 31), (4, 33), (32, 4), (128,), (4, 32, 1), (1, 4, 32)])
def test_output_of_another_shape(device, pattern, q, shape):
    w = packed(pattern, q, 32, 256)
    for e in (None, ss.Epilogue(act="relu")):
        with pytest.raises(ValueError):
            call(pattern, q, zeros(4, 256), w, out=zeros(*shape), epilogue=e)


@pytest.mark.parametrize("pattern,q", CASES)
def test_gated_output_is_half_as_wide(device, pattern, q):
    with pytest.raises(ValueError):
        call(pattern, q, zeros(4, 256), packed(pattern, q, 32, 256), out=zeros(4, 32),
             epilogue=ss.Epilogue(act="silu", gated=True))


@pytest.mark.parametrize("pattern,q", CASES)
@pytest.mark.parametrize("K", [64, 1024])
def test_activation_of_another_length(device, pattern, q, K):
    w = packed(pattern, q, 32, 512)
    norms = [None] if q == "nvfp4" else [None, (zeros(K), 1e-5)]
    for e in (None, ss.Epilogue(act="relu")):
        for norm in norms:
            with pytest.raises(ValueError):
                call(pattern, q, zeros(4, K), w, epilogue=e, **({} if norm is None else {"norm": norm}))
    if q != "nvfp4":
        with pytest.raises(ValueError):
            ss.project_qkv(zeros(4, K), w, pattern, q, 2, 1, None, None)


@pytest.mark.parametrize("pattern,q", CASES)
def test_what_fits_is_not_refused(device, pattern, q):
    """It gets as far as the library, which finds no device here."""
    w = packed(pattern, q, 32, 256)
    if torch.cuda.is_available():
        pytest.skip("CPU tensors must not reach a device")
    for kw in ({}, {"out": zeros(4, 32)}, {"out": zeros(4, 32, dtype=torch.float32)}):
        for e in (None, ss.Epilogue(act="relu")):
            with pytest.raises(ss.SSError):
                call(pattern, q, zeros(4, 256), w, epilogue=e, **kw)
