"""Memory that a call takes for itself belongs to the stream that it runs on: the
caching allocator gives it out again in that stream's order.  Intermediates taken
on the current stream and used on another would be given to the current stream's
next work while the other one still reads them.  (CPU: the CUDA calls are
replaced, allocations are watched; the last test runs on the device.)"""
import contextlib

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import structured_sparse_quantized_b200 as ss


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is on cuda:0."""
    is_cuda = True

    def get_device(self):
        return 0


def on_device(t):
    return t.as_subclass(OnDevice)


class Watch(TorchDispatchMode):
    """Notes the current stream at every allocation, and puts it on cuda:0."""

    def __init__(self, current):
        super().__init__()
        self.current, self.at = current, []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if "empty" in func.name():
            self.at.append(self.current[-1])
            return out.as_subclass(OnDevice)
        return out


HOST = ("ss_parse_pattern", "ss_slide_shape", "ss_fp4_shape", "ss_fp4_scale_bytes", "ss_act_2to4_shape",
        "ss_meta_bytes")


@pytest.fixture
def watched(monkeypatch):
    """-> (allocations' streams, kernels' streams), with the current stream "current"."""
    from structured_sparse_quantized_b200 import _build
    _build.build()
    real, current, kernels = ss.lib(), ["current"], []

    class Lib:
        def __getattr__(self, name):
            if name in HOST:
                return getattr(real, name)
            return lambda *a: kernels.append(a[-1]) or 0

    @contextlib.contextmanager
    def as_current(stream, like):
        current.append(stream)
        yield
        current.pop()
    monkeypatch.setattr(ss, "lib", Lib)
    monkeypatch.setattr(ss, "_as_current", as_current)
    monkeypatch.setattr(ss, "_stream", lambda s: current[-1] if s is None else s)
    monkeypatch.setattr(ss, "_raw_stream", lambda s, d: current[-1] if s is None else s)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    with Watch(current) as w:
        yield w.at, kernels


def X(M=4, K=64):
    return on_device(torch.ones(M, K, dtype=torch.bfloat16))


def packed(pattern, q, stream):
    return ss.compress_weight(X(32), pattern, q, stream)


CALLS = {
    "compress_weight": lambda s: ss.compress_weight(X(), "6:8", "int8", s),
    "compress_weight_dense": lambda s: ss.compress_weight(X(), "dense", "bf16", s),
    "compress_weight_nvfp4": lambda s: ss.compress_weight_nvfp4(X(), "2:4", s),
    "compress_weight_nvfp4_dense": lambda s: ss.compress_weight_nvfp4(X(), "dense", s),
    "quant_lift_act": lambda s: ss.quant_lift_act(X(), "6:8", "fp8", s),
    "quant_lift_act_nvfp4": lambda s: ss.quant_lift_act_nvfp4(X(), "2:4", 32, s),
    "prune_act_2to4": lambda s: ss.prune_act_2to4(X(), "int8", s),
    "norm": lambda s: ss.norm_quant_lift_act(X(), on_device(torch.ones(64)), 1e-5, "6:8", "int8", s),
}
for _p in ("6:8", "dense"):
    for _q in ("int8", "bf16"):
        CALLS[f"linear_{_p}_{_q}"] = lambda s, p=_p, q=_q: ss.linear(X(), packed(p, q, s), p, q, stream=s)
    CALLS[f"linear_{_p}_norm"] = lambda s, p=_p: ss.linear(
        X(), packed(p, "int8", s), p, "int8", stream=s, norm=(on_device(torch.ones(64)), 1e-5))
    CALLS[f"linear_{_p}_epilogue"] = lambda s, p=_p: ss.linear(
        X(), packed(p, "int8", s), p, "int8", stream=s, epilogue=ss.Epilogue(act="relu"))
    CALLS[f"linear_{_p}_out"] = lambda s, p=_p: ss.linear(
        X(), packed(p, "int8", s), p, "int8", stream=s, out=on_device(torch.zeros(4, 32)))
for _p in ("2:4", "dense"):
    CALLS[f"linear_nvfp4_{_p}"] = lambda s, p=_p: ss.linear_nvfp4(
        X(), ss.compress_weight_nvfp4(X(32), p, s), p, stream=s)
    CALLS[f"linear_nvfp4_{_p}_epilogue"] = lambda s, p=_p: ss.linear_nvfp4(
        X(), ss.compress_weight_nvfp4(X(32), p, s), p, stream=s, epilogue=ss.Epilogue(act="relu"))


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("stream", ["other", None])
def test_memory_is_the_streams(watched, name, stream):
    allocations, kernels = watched
    CALLS[name](stream)
    want = {stream or "current"}
    assert allocations and set(allocations) == want
    assert kernels and set(kernels) == want


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["torch", "handle"])
def test_linear_on_a_stream_beside_work_on_the_current_one(kind):
    """Results on another stream while the current one keeps allocating and
    writing blocks of the sizes that the linear's intermediates have."""
    g = torch.Generator().manual_seed(9)
    x = torch.randn(512, 1024, generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn(768, 1024, generator=g) * 0.05).cuda()
    s = torch.cuda.Stream()
    stream = s if kind == "torch" else s.cuda_stream
    for pattern in ("6:8", "dense"):
        p8, p4 = ss.compress_weight(w, pattern, "int8"), ss.compress_weight_nvfp4(w, "dense")
        want8, want4 = ss.linear(x, p8, pattern, "int8"), ss.linear_nvfp4(x, p4, "dense")
        s.wait_stream(torch.cuda.current_stream())
        got = []
        for _ in range(30):
            got.append((ss.linear(x, p8, pattern, "int8", stream=stream),
                        ss.linear_nvfp4(x, p4, "dense", stream=stream)))
            for n in (512 * 1536, 512 * 1024, 512 * 512, 2048, 16):
                torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        s.synchronize()
        for y8, y4 in got:
            assert torch.equal(y8, want8) and torch.equal(y4, want4)
