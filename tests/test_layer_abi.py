"""CPU checks of the calls around the products: refusals before any launch,
host-side frequency tables, the weight order of gated products."""
import ctypes
import math

import numpy as np
import pytest
import torch

import structured_sparse_quantized_b200 as ss

vp = ctypes.c_void_p
GOOD, ODD = 0x10000, 0x10008  # never dereferenced: every call below fails first


@pytest.fixture(scope="module")
def L():
    from structured_sparse_quantized_b200 import _build
    _build.build()
    return ss.lib()


def epi(bias=None, residual=None, bt=ss.SS_IN_BF16, rt=ss.SS_IN_BF16, act=0, gated=0):
    return ctypes.byref(ss.ss_epilogue(bias, residual, bt, rt, act, gated))


def every_gemm(L, e, N=64, y=GOOD):
    """The status of the four fused products with epilogue e."""
    return {L.ss_sparse_gemm_fused(0, GOOD, GOOD, GOOD, GOOD, GOOD, 16, N, 128, 0, e, y, 1, None),
            L.ss_dense_gemm_fused(GOOD, GOOD, GOOD, GOOD, 16, N, 128, 0, e, y, 1, None),
            L.ss_sparse_gemm_nvfp4_fused(GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, 16, N, 256, e, y, 1, None),
            L.ss_dense_gemm_nvfp4_fused(GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, 16, N, 256, e, y, 1, None)}


def test_epilogue_refusals(L):
    bad = ss.SS_ERR_INVALID_ARG
    assert every_gemm(L, epi(act=5)) == {bad}
    assert every_gemm(L, epi(act=-1)) == {bad}
    assert every_gemm(L, epi(gated=2)) == {bad}
    assert every_gemm(L, epi(bias=GOOD, bt=2)) == {bad}
    assert every_gemm(L, epi(residual=GOOD, rt=7)) == {bad}
    assert every_gemm(L, epi(gated=1, act=2), N=72) == {bad}
    assert every_gemm(L, epi(gated=1, residual=GOOD)) == {ss.SS_ERR_UNSUPPORTED}
    assert every_gemm(L, epi(bias=ODD)) == {ss.SS_ERR_ALIGNMENT}
    assert every_gemm(L, epi(residual=ODD)) == {ss.SS_ERR_ALIGNMENT}
    # scales are read in vectors by a fused product
    for sa, sb in ((ODD, GOOD), (GOOD, ODD)):
        assert L.ss_sparse_gemm_fused(0, GOOD, GOOD, sa, GOOD, sb, 16, 64, 128, 0, epi(act=1), GOOD, 1,
                                      None) == ss.SS_ERR_ALIGNMENT
        assert L.ss_dense_gemm_fused(GOOD, sa, GOOD, sb, 16, 64, 128, 0, epi(act=1), GOOD, 1,
                                     None) == ss.SS_ERR_ALIGNMENT
    # the plain calls' own checks come first
    assert every_gemm(L, epi(act=1), y=None) == {bad}
    assert every_gemm(L, epi(act=1), y=ODD) == {ss.SS_ERR_ALIGNMENT}


def heads(i=GOOD, o=GOOD, n=4, s=(512, 128, 512, 128)):
    return ctypes.byref(ss.ss_rope_heads(i, o, n, *s))


def test_rope_refusals(L):
    def call(q=None, k=None, dtype=1, pos=GOOD, p64=1, f=GOOD, T=8, D=128, rot=128, layout=0):
        return L.ss_rope(q or heads(), k, dtype, pos, p64, f, 1.0, T, D, rot, layout, None)
    bad = ss.SS_ERR_INVALID_ARG
    assert L.ss_rope(None, None, 1, GOOD, 1, GOOD, 1.0, 8, 128, 128, 0, None) == bad
    for kw in (dict(dtype=2), dict(pos=None), dict(f=None), dict(p64=2), dict(T=0), dict(T=-1),
               dict(T=2 ** 31 - 8), dict(D=1), dict(rot=0), dict(rot=3), dict(rot=130), dict(layout=2),
               dict(q=heads(n=0)), dict(q=heads(n=65537)), dict(q=heads(i=None)), dict(q=heads(o=None)),
               dict(k=heads(n=-1)), dict(k=heads(o=None))):
        assert call(**kw) == bad, kw
    assert call(D=1026) == ss.SS_ERR_UNSUPPORTED
    for kw in (dict(q=heads(i=GOOD + 1)), dict(k=heads(o=GOOD + 1)), dict(pos=GOOD + 4), dict(f=GOOD + 4),
               dict(pos=GOOD + 2, p64=0), dict(dtype=0, q=heads(i=GOOD + 2))):
        assert call(**kw) == ss.SS_ERR_ALIGNMENT, kw


def test_norm_refusals(L):
    pat = ss.ss_pattern(6, 8)

    def call(x=GOOD, xt=1, w=GOOD, wt=1, eps=1e-5, M=4, K=64, p=pat, q=0, xq=GOOD, s=GOOD):
        return L.ss_norm_quant_lift_act(x, xt, w, wt, eps, M, K, p, q, xq, s, None)
    for kw in (dict(x=None), dict(w=None), dict(xq=None), dict(s=None), dict(xt=2), dict(wt=-1),
               dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(M=0), dict(M=2 ** 31),
               dict(K=0), dict(K=2 ** 30 + 1), dict(q=3), dict(p=ss.ss_pattern(3, 4))):
        assert call(**kw) == ss.SS_ERR_INVALID_ARG, kw
    for kw in (dict(x=ODD), dict(w=ODD), dict(xq=ODD), dict(s=ODD)):
        assert call(**kw) == ss.SS_ERR_ALIGNMENT, kw


def test_python_refusals():
    """Shapes, types and devices are checked before the C call."""
    with pytest.raises(ValueError):
        ss.Epilogue(act="tanh")
    cpu = torch.zeros(16, 64)
    with pytest.raises(ValueError):
        ss.dense_gemm(cpu, None, cpu, None, "bf16", epilogue=ss.Epilogue(act="relu"), out=cpu)
    with pytest.raises(ValueError):
        ss.rope(torch.zeros(4, 2, 8), None, torch.arange(4), torch.zeros(4, dtype=torch.float64))
    with pytest.raises(ValueError):
        ss.norm_quant_lift_act(cpu, torch.ones(64), 1e-5, "2:4", "int8")
    with pytest.raises(ValueError):
        ss.rope_frequencies(64, kind="other", device="cpu")
    with pytest.raises(ValueError):
        ss.interleave_gate_up(torch.zeros(12, 4), torch.zeros(12, 4))


def test_interleave_gate_up():
    gate, up = torch.arange(24.0).view(24, 1) + 0.5, torch.arange(24.0).view(24, 1) + 100.5
    both = ss.interleave_gate_up(gate, up)
    assert both.shape == (48, 1)
    for f in range(24):
        row = 16 * (f // 8) + f % 8
        assert both[row] == gate[f] and both[row + 8] == up[f]
    assert torch.equal(ss.interleave_gate_up(gate[:, 0], up[:, 0]), both[:, 0])


def test_frequencies():
    """Against the published formulas, each pair on its own."""
    base, d, factor, orig = 500000.0, 128, 8.0, 8192.0
    inv = [base ** (-2 * i / d) for i in range(d // 2)]
    close = lambda a, b: np.testing.assert_allclose(a, b, rtol=1e-13)
    f, s = ss.rope_frequencies(d, base, device="cpu")
    close(f.numpy(), inv)
    assert s == 1.0 and f.dtype == torch.float64
    close(ss.rope_frequencies(d, base, "linear", factor, device="cpu")[0].numpy(), [v / factor for v in inv])
    close(ss.rope_frequencies(d, base, "ntk", factor, device="cpu")[0].numpy(),
          [(base * factor ** (d / (d - 2))) ** (-2 * i / d) for i in range(d // 2)])
    f, s = ss.rope_frequencies(d, base, "llama3", factor, orig, device="cpu")
    for got, v in zip(f.tolist(), inv):
        wave = 2 * math.pi / v
        if wave < orig / 4:
            want = v
        elif wave > orig / 1:
            want = v / factor
        else:
            m = (orig / wave - 1) / (4 - 1)
            want = (1 - m) * v / factor + m * v
        assert abs(got / want - 1) < 1e-13
    assert s == 1.0
    f, s = ss.rope_frequencies(d, base, "yarn", factor, orig, device="cpu")
    lo = math.floor(d * math.log(orig / (32 * 2 * math.pi)) / (2 * math.log(base)))
    hi = math.ceil(d * math.log(orig / (1 * 2 * math.pi)) / (2 * math.log(base)))
    for i, (got, v) in enumerate(zip(f.tolist(), inv)):
        ramp = min(1, max(0, (i - lo) / (hi - lo)))
        assert abs(got / (v / factor * ramp + v * (1 - ramp)) - 1) < 1e-13
    assert abs(s - (0.1 * math.log(8) + 1)) < 1e-15


@pytest.mark.parametrize("args", [dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=1026), dict(base=1.0),
                                  dict(base=math.nan), dict(kind="linear", factor=0.0),
                                  dict(kind="ntk", factor=math.inf), dict(kind="llama3", factor=8.0),
                                  dict(kind="yarn", factor=8.0, original=100.0, low=2.0, high=2.0)])
def test_frequency_refusals(args):
    with pytest.raises(ss.SSError) as e:
        ss.rope_frequencies(**({"rot_dim": 64, "device": "cpu"} | args))
    assert e.value.status == ss.SS_ERR_INVALID_ARG
