"""The layer's calls run on the device of their tensors, whatever device is current
(CPU: tensors that say they are on cuda:1, with cuda:0 current; the library's
kernels are replaced by notes of the device that is current at their launch)."""
import contextlib

import pytest
import torch

import structured_sparse_quantized_b200 as ss
from test_stream_memory import HOST

BF = torch.bfloat16


class OnSecond(torch.Tensor):
    is_cuda = True

    def get_device(self):
        return 1


def zeros(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnSecond)


@pytest.fixture
def launches(monkeypatch):
    """The device current at each launch, and the stream's device."""
    from structured_sparse_quantized_b200 import _build
    _build.build()
    real, current, notes = ss.lib(), [0], []

    class Lib:
        def __getattr__(self, name):
            if name in HOST:
                return getattr(real, name)
            return lambda *a: notes.append((name, current[-1], a[-1])) or 0

    @contextlib.contextmanager
    def device(d):
        current.append(1 if isinstance(d, torch.device) else d)
        yield
        current.pop()
    monkeypatch.setattr(ss, "lib", Lib)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[-1], raising=False)
    monkeypatch.setattr(ss, "_stream", lambda s: current[-1])
    monkeypatch.setattr(ss, "_raw_stream", lambda s, d: d)
    monkeypatch.setattr(ss, "_new", lambda like, shape, dtype, stream: zeros(*shape, dtype=dtype))
    return notes


def weight(N, K, pattern="6:8", q="int8"):
    K_lp = ss.ss_slide_shape(pattern, K)[2]
    return (zeros(N, K_lp if pattern == "dense" else K_lp // 2, dtype=BF if q == "bf16" else torch.uint8),
            None if pattern == "dense" else zeros(*ss.meta_shape(N, K_lp), dtype=torch.uint8),
            None if q == "bf16" else zeros(N, dtype=torch.float32))


def weight_fp4(N, K):
    _, K_lp = ss.ss_fp4_shape("2:4", K)
    return (zeros(N, K_lp // 4, dtype=torch.uint8), zeros(*ss.meta_shape(N, K_lp // 2), dtype=torch.uint8),
            zeros(ss.ss_fp4_scale_bytes(N, K_lp, 32), dtype=torch.uint8), zeros(4, dtype=torch.float32))


def qkv(norm=None, bias=None):
    return ss.project_qkv(zeros(4, 64), weight(4 * 16, 64), "6:8", "int8", 2, 1,
                          zeros(4, dtype=torch.int64), zeros(8, dtype=torch.float64), norm=norm, bias=bias)


CALLS = {
    "linear": lambda: ss.linear(zeros(4, 64), weight(32, 64), "6:8", "int8"),
    "linear_dense": lambda: ss.linear(zeros(4, 64), weight(32, 64, "dense", "bf16"), "dense", "bf16"),
    "linear_epilogue": lambda: ss.linear(zeros(4, 64), weight(32, 64), "6:8", "int8",
                                         epilogue=ss.Epilogue(act="silu")),
    "linear_norm": lambda: ss.linear(zeros(4, 64), weight(32, 64), "6:8", "int8", norm=(zeros(64), 1e-5)),
    "linear_nvfp4": lambda: ss.linear_nvfp4(zeros(4, 64), weight_fp4(32, 64), "2:4"),
    "linear_nvfp4_epilogue": lambda: ss.linear_nvfp4(zeros(4, 64), weight_fp4(32, 64), "2:4",
                                                     epilogue=ss.Epilogue(act="silu")),
    "project_qkv": qkv,
    "project_qkv_norm_bias": lambda: qkv((zeros(64), 1e-5), zeros(64)),
    "feed_forward": lambda: ss.feed_forward(zeros(4, 64), weight(2 * 32, 64), weight(64, 32), "6:8", "int8"),
    "norm": lambda: ss.norm_quant_lift_act(zeros(4, 64), zeros(64), 1e-5, "6:8", "int8"),
}


@pytest.mark.parametrize("name", CALLS)
def test_runs_where_its_tensors_are(launches, name):
    CALLS[name]()
    assert launches and all(note[1:] == (1, 1) for note in launches), launches
