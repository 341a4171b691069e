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


MANY = [(p, M, K) for M, K in [(1500, 4096), (2500, 264), (4003, 1000), (1300, 2040), (1184, 8), (1200, 4097)]
        for p in ("dense", "4:6", "6:8", "8:10")]
MANY += [(p, M, K) for M, K in [(1200, 5000), (1190, 6144), (1190, 6136), (1184, 16384), (1190, 8200),
                                (1184, 13313), (1300, 12304)] for p in ("6:8", "8:10")]
MANY += [(p, M, K) for M, K in [(1190, 2560), (1185, 7000), (1190, 8192), (1187, 10240), (1190, 14336)]
         for p in ("dense", "8:10")]


@pytest.mark.parametrize("tier", ["int8", "fp8", "bf16"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pattern,M,K", MANY)
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


def test_nothing_past_the_rows_is_written():
    for M, K, pattern in [(3, 64, "6:8"), (1300, 264, "4:6"), (1300, 4096, "6:8"), (5, 1000, "8:10")]:
        X, w = rows(M, K, BF)
        _, _, K_lp = oracle.slide_shape(pattern, K)
        for tier, dtype in (("int8", torch.uint8), ("bf16", BF)):
            buf = torch.full((M * K_lp + 4096,), 7, dtype=dtype, device="cuda")
            s = torch.full((M + 64,), 7.0, device="cuda")
            out = (buf[:M * K_lp].view(M, K_lp), None if tier == "bf16" else s[:M])
            ss.norm_quant_lift_act(X.cuda(), w.cuda(), 1e-5, pattern, tier, out=out)
            assert (buf[M * K_lp:] == 7).all() and (s[M:] == 7.0).all()


def test_ties_go_to_the_even_code():
    """Q z / max|z| on the border between two codes: the quotient is exact, and
    the even code is taken (max 448, so that a code is z itself)."""
    z = torch.tensor([448.0, 424.0, 440.0, 17.0, 19.0, 2.125, 2.375, 0.0009765625, 0.0029296875])
    X = torch.zeros(4, 64)
    X[:, :9] = z
    Xq, _ = ss.norm_quant_lift_act(X.to(BF).cuda(), torch.ones(64, device="cuda"), 1e-5, "dense", "fp8")
    got = Xq.view(torch.float8_e4m3fn).float().cpu()[:, :9]
    want = torch.tensor([448.0, 416.0, 448.0, 16.0, 20.0, 2.0, 2.5, 0.0, 0.00390625])
    assert torch.equal(got, want.expand(4, 9))
    X = torch.zeros(4, 64)
    X[:, :6] = torch.tensor([254.0, 1.0, 3.0, 5.0, -3.0, 253.0])  # codes z / 2
    Xq, _ = ss.norm_quant_lift_act(X.to(BF).cuda(), torch.ones(64, device="cuda"), 1e-5, "dense", "int8")
    assert torch.equal(Xq.view(torch.int8).cpu()[:, :6],
                       torch.tensor([127, 0, 2, 2, -2, 126], dtype=torch.int8).expand(4, 6))


def test_refusals_on_the_device():
    X, w = rows(4, 64, BF)
    X, w = X.cuda(), w.cuda()
    for bad in (dict(X=X[0]), dict(X=X.half()), dict(X=X.t()), dict(weight=w[:32]), dict(weight=w.cpu()),
                dict(weight=None), dict(weight=w.half()), dict(out=(torch.empty(4, 96, device="cuda"), None))):
        with pytest.raises(ValueError):
            ss.norm_quant_lift_act(**({"X": X, "weight": w, "eps": 1e-5, "pattern": "6:8", "q": "int8"} | bad))
    for bad in (dict(eps=-1.0), dict(pattern="3:4")):
        with pytest.raises(ss.SSError):
            ss.norm_quant_lift_act(**({"X": X, "weight": w, "eps": 1e-5, "pattern": "6:8", "q": "int8"} | bad))


def test_stream_argument():
    X, w = rows(300, 4096, BF)
    s = torch.cuda.Stream()
    x, wc = X.cuda(), w.cuda()
    s.wait_stream(torch.cuda.current_stream())
    got = ss.norm_quant_lift_act(x, wc, 1e-5, "6:8", "int8", stream=s)
    s.synchronize()
    want = ss.norm_quant_lift_act(x, wc, 1e-5, "6:8", "int8")
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
