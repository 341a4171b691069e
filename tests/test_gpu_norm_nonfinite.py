"""The fused norm of rows that have no finite norm: the row's product is NaN, as
the definition's is, in every tier and kernel, and the other rows are untouched."""
import pytest
import torch

import structured_sparse_quantized_b200 as ss

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


# few rows (row kernel: whole and ragged words), many (streaming kernel, with one
# and with several warps a row), rows past the registers of a block
@pytest.mark.parametrize("M,K", [(6, 64), (8, 151), (6, 4096), (9, 5008), (1300, 264), (1200, 4096), (1190, 8200),
                                 (6, 20000)])
@pytest.mark.parametrize("tier", ["int8", "fp8", "bf16"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pattern", ["dense", "6:8", "8:10"])
def test_rows(M, K, tier, dtype, pattern):
    g = torch.Generator().manual_seed(K)
    X, w = torch.randn(M, K, generator=g), 1 + 0.2 * torch.randn(K, generator=g)
    want = ss.norm_quant_lift_act(X.to(dtype).cuda(), w.cuda(), 1e-5, pattern, tier)
    bad = {0: {K // 2: INF}, 1: {K - 1: -INF}, 2: {0: NAN}, 3: {k: NAN for k in range(K)},
           4: {0: NAN} | {k: 0.0 for k in range(1, K)}}
    if dtype == F32:
        bad[5] = {K // 3: 1e30}  # finite, but the sum of squares is not in fp32
    for m, at in bad.items():
        for k, v in at.items():
            X[m, k] = v
    Xq, s = ss.norm_quant_lift_act(X.to(dtype).cuda(), w.cuda(), 1e-5, pattern, tier)
    assert ss.ss_get_device_status() == ss.SS_OK
    rows = torch.ones(M, dtype=torch.bool)
    rows[list(bad)] = False
    if tier == "bf16":
        assert torch.isnan(Xq[~rows.cuda(), :K if pattern == "dense" else 4]).all()
    else:
        assert torch.isnan(s[~rows.cuda()]).all()
        assert torch.equal(s[rows.cuda()], want[1][rows.cuda()])
    assert torch.equal(Xq[rows.cuda()], want[0][rows.cuda()])


@pytest.mark.parametrize("M,K", [(3, 64), (3, 5008), (1300, 264), (1200, 4096), (3, 20000)])
@pytest.mark.parametrize("tier", ["int8", "fp8"])
@pytest.mark.parametrize("value", [INF, NAN])
def test_weights(M, K, tier, value):
    """A weight that is not finite is every row's largest |y|."""
    g = torch.Generator().manual_seed(K)
    w = torch.ones(K)
    w[K // 2] = value
    _, s = ss.norm_quant_lift_act(torch.randn(M, K, generator=g).cuda(), w.cuda(), 1e-5, "6:8", tier)
    assert torch.isnan(s).all()


@pytest.mark.parametrize("tier", ["int8", "fp8", "bf16"])
@pytest.mark.parametrize("value", [INF, -INF, NAN])
def test_through_the_product(tier, value):
    g = torch.Generator().manual_seed(3)
    X, W = torch.randn(40, 512, generator=g).to(BF), torch.randn(144, 512, generator=g) * 0.05
    packed = ss.compress_weight(W.to(BF).cuda(), "6:8", tier)
    norm = (torch.ones(512, device="cuda"), 1e-5)
    want = ss.linear(X.cuda(), packed, "6:8", tier, norm=norm)
    X[7, 100] = value
    y = ss.linear(X.cuda(), packed, "6:8", tier, norm=norm)
    assert torch.isnan(y[7]).all()
    others = [m for m in range(40) if m != 7]
    assert torch.equal(y[others], want[others])
