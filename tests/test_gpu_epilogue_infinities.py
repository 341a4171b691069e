"""The activations at minus infinity, as the header states them: NaN where the
formula is 0 times infinity (SiLU, tanh GELU), 0 for ReLU and the exact GELU."""
import numpy as np
import pytest
import torch

import structured_sparse_quantized_b200 as ss
import _layer as ref
from _helpers import dev
from test_gpu_epilogue import BF, F32, Product

pytestmark = pytest.mark.gpu


# K split; TMA ways by channels and tokens; straight from registers
@pytest.mark.parametrize("M,N,form", [(3, 512, "w"), (300, 1040, "w"), (300, 1040, "x"), (300, 1040, "dense"),
                                      (300, 1041, "w"), (300, 1041, "x")])
@pytest.mark.parametrize("out", [BF, F32])
def test_minus_infinity(M, N, form, out):
    p = Product(M, N, 256, "int8", form)
    b = torch.linspace(-90, 90, N)
    b[7], b[8] = float("-inf"), -3e38
    keep = [i for i in range(N) if i not in (7, 8)]
    for act in ("relu", "silu", "gelu", "gelu_erf"):
        y = p.run(ss.Epilogue(bias=dev(b), act=act), out)
        assert ss.ss_get_device_status() == ss.SS_OK
        if act in ("silu", "gelu"):
            assert torch.isnan(y[:, 7]).all()
        else:
            assert (y[:, 7] == 0).all()
        assert (y[:, 8] == 0).all()  # the largest negative values are still finite
        want, bound = ref.epilogue(p.d[:, keep], b[keep], act, False, None, out)
        ref.assert_within(y[:, keep], want, bound)


@pytest.mark.parametrize("M", [3, 300])
def test_minus_infinity_gated(M):
    """Only the outputs of that gate; a partner's infinity is the output's."""
    p = Product(M, 512, 256, "int8", "w")
    b = torch.randn(512, generator=torch.Generator().manual_seed(1))
    b[16 * 2 + 3] = float("-inf")   # gate of output 19
    b[16 * 5 + 8 + 1] = float("inf")  # partner of output 41
    y = p.run(ss.Epilogue(bias=dev(b), act="silu", gated=True), BF)
    assert torch.isnan(y[:, 19]).all() and torch.isinf(y[:, 41]).all()
    keep = [i for i in range(256) if i not in (19, 41)]
    with np.errstate(invalid="ignore"):
        want, bound = ref.epilogue(p.d, b, "silu", True, None, BF)
    ref.assert_within(y[:, keep], want[:, keep], bound[:, keep])
