"""The fused epilogue where a cluster works on several output tiles: its second
accumulator and the barriers' phases, the residual that is loaded for the next
tile during this one's, the tile orders."""
import pytest
import torch

import structured_sparse_quantized_b200 as ss
import _layer as ref
from _helpers import dev
from test_gpu_epilogue import BF, F32, Product, check

pytestmark = pytest.mark.gpu

PLAIN = (BF, "none", False, None, BF)
RESIDUAL = (F32, "gelu", False, BF, BF)
GATED = (None, "silu", True, None, BF)
# straight from registers: fp32 Y, fp32 residual
STRAIGHT = [(BF, "relu", False, F32, BF), (None, "silu", False, BF, F32), (BF, "silu", True, None, F32)]


def tiles_per_cluster(rows_a, rows_b, widest, per_a=256):
    """At least this many: tiles of per_a A rows and at most `widest` B rows."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    clusters = sms // 2 if per_a > 128 else sms
    return -(-rows_a // per_a) * -(-rows_b // widest) / clusters


def run(p, epilogues):
    for e in epilogues:
        check(p, *e)


@pytest.mark.parametrize("tier", ["int8", "fp8", "bf16", "nvfp4"])
@pytest.mark.parametrize("form", ["w", "dense"])
def test_channel_rows(tier, form):
    M, N = 530, 19600
    assert tiles_per_cluster(N, M, 256) > 3
    run(Product(M, N, 256, tier, form), [PLAIN, RESIDUAL, GATED] + STRAIGHT[:1])


@pytest.mark.parametrize("tier", ["int8", "bf16", "nvfp4"])
@pytest.mark.parametrize("form", ["w", "dense"])
def test_channel_rows_straight(tier, form):
    assert tiles_per_cluster(19600, 520, 256) > 3
    run(Product(520, 19600, 128, tier, form), STRAIGHT[1:])
    run(Product(520, 19601, 128, tier, form), [PLAIN, RESIDUAL])  # rows of Y not 16-byte aligned


@pytest.mark.parametrize("tier", ["int8", "fp8", "bf16"])
def test_token_rows(tier):
    M, N = 19601, 464
    assert tiles_per_cluster(M, N, 224) > 3
    run(Product(M, N, 256, tier, "x"), [PLAIN, RESIDUAL, GATED, STRAIGHT[0]])
    run(Product(M, 453, 128, tier, "x"), [RESIDUAL, STRAIGHT[1]])


@pytest.mark.parametrize("tier,form", [("int8", "w"), ("fp8", "w"), ("bf16", "dense"), ("nvfp4", "w")])
@pytest.mark.parametrize("M", [20, 33, 64])
def test_few_tokens(tier, form, M):
    N = 57616
    assert tiles_per_cluster(N, M, 64) > 3
    run(Product(M, N, 384, tier, form), [PLAIN, RESIDUAL, GATED, STRAIGHT[0]])


@pytest.mark.parametrize("tier", ["int8", "bf16"])
@pytest.mark.parametrize("M", [20, 64])
def test_few_channels_of_token_rows(tier, M):
    """A sparse activation's B rows are channels: 64 of them at most."""
    assert tiles_per_cluster(57616, M, 64) > 3
    run(Product(57616, 16 * (M // 16), 256, tier, "x"), [PLAIN, RESIDUAL, GATED])


@pytest.mark.parametrize("tier,form", [("int8", "w"), ("fp8", "dense"), ("bf16", "w"), ("nvfp4", "w"),
                                       ("nvfp4", "dense")])
def test_one_cta(tier, form):
    M, N = 76001, 112  # one A tile of 128 rows: no CTA pairs
    assert tiles_per_cluster(N, M, 256, 128) > 2
    run(Product(M, N, 256, tier, form), [PLAIN, RESIDUAL, GATED, STRAIGHT[0]])


@pytest.mark.parametrize("tier", ["int8", "fp8"])
def test_two_b_tiles(tier, monkeypatch):
    monkeypatch.setenv("SS_SPARSE_KERNEL", "wide")
    M, N = 900, 19600
    assert tiles_per_cluster(N, M, 448) > 3
    run(Product(M, N, 256, tier, "w"), [PLAIN, RESIDUAL, GATED])


@pytest.mark.parametrize("kernel", ["narrow", "wide"])
def test_a_tiles_in_groups(kernel, monkeypatch):
    """50 MB of weight: its tiles are walked in two groups."""
    monkeypatch.setenv("SS_SPARSE_KERNEL", kernel)
    run(Product(900, 19600, 4096, "int8", "w"), [RESIDUAL, GATED])


@pytest.mark.parametrize("tier,form,M,N", [("int8", "w", 530, 19600), ("int8", "x", 19601, 464),
                                           ("nvfp4", "w", 530, 19600), ("fp8", "w", 530, 19601)])
@pytest.mark.parametrize("out", [BF, F32])
def test_residual_updated_in_place(tier, form, M, N, out):
    p = Product(M, N, 256, tier, form)
    y = dev((torch.randn(M, N, generator=torch.Generator().manual_seed(1)) * 2).to(out))
    r = y.cpu().clone()
    for _ in range(2):  # twice: the second call finds what the first left
        p.run(ss.Epilogue(act="relu", residual=y), out, y)
        assert ss.ss_get_device_status() == ss.SS_OK
        want, bound = ref.epilogue(p.d, None, "relu", False, r, out)
        ref.assert_within(y, want, bound)
        r = y.cpu().clone()
