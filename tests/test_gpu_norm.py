"""RMS norm fused into the quantisation and lift, against 64 bits."""
import numpy as np
import pytest
import torch

import oracle
import structured_sparse_quantized_b200 as ss
import _layer as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
TOP = {"int8": 127.0, "fp8": 448.0}


def check(X, w, eps, pattern, tier):
    M, K = X.shape
    Xq, s_x = ss.norm_quant_lift_act(X.cuda(), w.cuda(), eps, pattern, tier)
    assert ss.ss_get_device_status() == ss.SS_OK
    x = X.double().numpy()
    y = x / np.sqrt((x * x).mean(1, keepdims=True) + eps) * w.double().numpy()
    # fp32: the sum of squares, in at most K / 32 + 32 terms in a row, is off by
    # that many half units and its root by half as much, plus root, quotient and
    # two products: `root` bounds y's relative error.  max|y| / Q shares the root.
    root = (K / 32 + 32 + 16) * 2.0 ** -25 + 8 * 2.0 ** -24
    if tier == "bf16":
        assert s_x is None
        want = ref.lift(y, pattern)
        ref.assert_within(Xq, want, np.abs(want) * (root + 2.0 ** -8) * 1.01 + ref.TINY)
        return
    a = np.abs(y).max(1)
    np.testing.assert_allclose(s_x.cpu().double().numpy(), a / TOP[tier], rtol=root + 2.0 ** -23, atol=0)
    scaled = np.where(a[:, None] > 0, y * (TOP[tier] / np.where(a > 0, a, 1.0))[:, None], 0.0)
    v = ref.lift(scaled, pattern)
    # the code is the nearest value to y Q / max|y|, which the root does not
    # change: four roundings on each side of the quotient, 8 * 2^-24 of |v|
    slack = np.abs(v) * 2.0 ** -21
    if tier == "int8":
        got = Xq.cpu().view(torch.int8).double().numpy()
        assert (np.abs(got - v) <= 0.5 + slack).all()
    else:
        got = Xq.cpu().view(torch.float8_e4m3fn).double().numpy()
        # half a step: 2^-4 of the value's power of two, at least half of 2^-9
        step = np.maximum(2.0 ** np.floor(np.log2(np.maximum(np.abs(v), 1e-30))) * 2.0 ** -4, 2.0 ** -10)
        assert (np.abs(got - v) <= step * 1.0001 + slack).all()
    # the padding and the largest element are exact
    _, K_lift, _ = oracle.slide_shape(pattern, K)
    assert (got[:, K_lift:] == 0).all()
    assert (np.abs(got).max(1) == np.where(a > 0, TOP[tier], 0)).all()


def rows(M, K, dtype, seed=0):
    g = torch.Generator().manual_seed(seed + M + K)
    X = torch.randn(M, K, generator=g)
    X[:, torch.randperm(K, generator=g)[:max(1, K // 100)]] *= 20
    return X.to(dtype), (1 + 0.2 * torch.randn(K, generator=g))


@pytest.mark.parametrize("pattern", ["dense", "2:4", "4:6", "6:8", "8:10"])
@pytest.mark.parametrize("tier", ["int8", "fp8", "bf16"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,K", [(1, 4096), (3, 64), (130, 1000), (33, 151), (9, 3584), (2, 1),
                                 (17, 16), (5, 8192), (3, 14336), (4, 5008), (2, 16384), (2, 20000)])
def test_patterns_tiers_sizes(pattern, tier, dtype, M, K):
    X, w = rows(M, K, dtype)
    check(X, w.to(BF if K % 3 else F32), 1e-5, pattern, tier)


@pytest.mark.parametrize("pattern", ["dense", "4:6", "6:8", "8:10"])
@pytest.mark.parametrize("tier", ["int8", "fp8", "bf16"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,K", [(1500, 4096), (2500, 264), (4003, 1000), (1300, 2040), (1200, 5000),
                                 (1184, 8), (1200, 4097)])
def test_many_rows(pattern, tier, dtype, M, K):
    X, w = rows(M, K, dtype)
    check(X, w.to(BF if M % 2 else F32), 1e-5, pattern, tier)


@pytest.mark.parametrize("tier", ["int8", "fp8", "bf16"])
def test_zero_rows_tiny_rows_and_eps(tier):
    X, w = rows(8, 256, F32)
    X[0] = 0
    X[2] *= 1e-12
    X[3] *= 1e12
    check(X, w, 1e-5, "6:8", tier)
    check(X[1:], w, 0.0, "6:8", tier)
    check(X, torch.zeros(256), 1e-5, "2:4", tier)


def test_norm_then_product_equals_the_separate_calls():
    """linear(norm=...) is the fused call, then the product on what it returned."""
    X, w = rows(70, 512, BF)
    W = torch.randn(144, 512, generator=torch.Generator().manual_seed(1)).to(BF) * 0.05
    packed = ss.compress_weight(W.cuda(), "6:8", "int8")
    Xq, s = ss.norm_quant_lift_act(X.cuda(), w.cuda(), 1e-5, "6:8", "int8")
    want = ss.sparse_gemm(0, *packed, Xq, s, 70, 144, "int8")
    got = ss.linear(X.cuda(), packed, "6:8", "int8", norm=(w.cuda(), 1e-5))
    assert torch.equal(got, want)


def test_captured_graph():
    X, w = rows(300, 4096, BF)
    x, w = X.cuda(), w.cuda()
    out = ss.norm_quant_lift_act(x, w, 1e-5, "6:8", "fp8")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ss.norm_quant_lift_act(x, w, 1e-5, "6:8", "fp8", out=out)
    x.mul_(2).add_(0.5)
    want = ss.norm_quant_lift_act(x, w, 1e-5, "6:8", "fp8")
    out[0].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
