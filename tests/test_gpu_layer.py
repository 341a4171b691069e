"""The operators of a layer's linear path together, as they would be used."""
import numpy as np
import pytest
import torch

import structured_sparse_quantized_b200 as ss

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def dense_of(packed, pattern, K, tier="int8"):
    """The compressed weight's values: the product with the identity's rows."""
    eye = torch.eye(K, device="cuda", dtype=BF)
    return ss.linear(eye, packed, pattern, tier, torch.float32).t().double()


def rel(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("pattern", ["6:8", "dense"])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_layer_path(M, pattern):
    """norm -> q/k/v with bias -> rotary -> (attention left out: the values of
    the query heads go on) -> output product + residual -> feed-forward, against
    64 bits on the weights as quantised.  INT8 rounding of the activations
    (half of 1/127 of the row's largest element, about 4 deviations: 0.9% of a
    value of one deviation, in quadrature over independent elements) enters four
    times; 3% covers the chain."""
    K, H, Hk, D, F = 512, 8, 2, 64, 704
    g = torch.Generator().manual_seed(M)
    rand = lambda *s: torch.randn(*s, generator=g)
    X = rand(M, K).to(BF).cuda()
    w1, w2 = (1 + 0.1 * rand(K)).cuda(), (1 + 0.1 * rand(K)).cuda()
    bias = rand((H + 2 * Hk) * D).cuda()
    Wqkv, Wo = rand((H + 2 * Hk) * D, K) * K ** -0.5, rand(K, H * D) * (H * D) ** -0.5
    Wg, Wu, Wd = rand(F, K) * K ** -0.5, rand(F, K) * K ** -0.5, rand(K, F) * F ** -0.5
    pack = lambda W: ss.compress_weight(W.to(BF).cuda(), pattern, "int8")
    pq, po, pg, pd = pack(Wqkv), pack(Wo), pack(ss.interleave_gate_up(Wg, Wu)), pack(Wd)
    pos = torch.arange(M, device="cuda") + 1000
    f, s = ss.rope_frequencies(D, 500000.0, "llama3", 8.0, 8192)
    q, k, v = ss.project_qkv(X, pq, pattern, "int8", H, Hk, pos, f, scale=s, norm=(w1, 1e-5), bias=bias)
    mid = ss.linear(q.reshape(M, H * D).contiguous(), po, pattern, "int8", epilogue=ss.Epilogue(residual=X))
    out = ss.feed_forward(mid, pg, pd, pattern, "int8", norm=(w2, 1e-5))
    assert ss.ss_get_device_status() == ss.SS_OK

    def norm64(x, w):
        return x / (x.square().mean(1, keepdim=True) + 1e-5).sqrt() * w.double()

    def turn(x):
        a = (pos.double()[:, None] * f)[:, None]
        p, r = x[..., :D // 2], x[..., D // 2:]
        return torch.cat((p * a.cos() - r * a.sin(), r * a.cos() + p * a.sin()), -1)

    y = norm64(X.double(), w1) @ dense_of(pq, pattern, K).t() + bias.double()
    y = y.view(M, H + 2 * Hk, D)
    rq, rk, rv = turn(y[:, :H]), turn(y[:, H:H + Hk]), y[:, H + Hk:]
    assert rel(q, rq) < 0.02 and rel(k, rk) < 0.02 and rel(v, rv) < 0.02
    rmid = X.double() + rq.reshape(M, -1) @ dense_of(po, pattern, H * D).t()
    assert rel(mid, rmid) < 0.02
    gu = (norm64(rmid, w2) @ dense_of(pg, pattern, K).t()).view(M, F // 8, 2, 8)
    h = (torch.nn.functional.silu(gu[:, :, 0]) * gu[:, :, 1]).reshape(M, F)
    want = rmid + h @ dense_of(pd, pattern, F).t()
    assert rel(out, want) < 0.03


@pytest.mark.parametrize("M", [1, 200])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_feed_forward_on_a_stream_repeats(M, dtype):
    """The same call on the current stream and, repeatedly, on another one (its
    intermediates are reused there while calls are in flight); fp32 stream too."""
    g = torch.Generator().manual_seed(M)
    K, F = 256, 352
    X = torch.randn(M, K, generator=g).to(dtype).cuda()
    w = torch.ones(K, device="cuda")
    pg = ss.compress_weight(ss.interleave_gate_up(torch.randn(F, K, generator=g) * 0.06,
                                                  torch.randn(F, K, generator=g) * 0.06).cuda(), "6:8", "int8")
    pd = ss.compress_weight((torch.randn(K, F, generator=g) * 0.05).cuda(), "6:8", "int8")
    want = ss.feed_forward(X, pg, pd, "6:8", "int8", norm=(w, 1e-5))
    assert want.dtype == dtype
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [ss.feed_forward(X, pg, pd, "6:8", "int8", norm=(w, 1e-5), stream=s) for _ in range(10)]
    s.synchronize()
    for y in got:
        assert torch.equal(y, want)


def test_nvfp4_linear_with_epilogue():
    """linear_nvfp4's epilogue against the plain call's fp32 output."""
    g = torch.Generator().manual_seed(3)
    X, W = torch.randn(70, 512, generator=g).to(BF).cuda(), (torch.randn(272, 512, generator=g) * 0.05).to(BF).cuda()
    b, r = torch.randn(272, generator=g).cuda(), torch.randn(70, 272, generator=g).to(BF).cuda()
    for pattern in ("2:4", "dense"):
        packed = ss.compress_weight_nvfp4(W, pattern)
        plain = ss.linear_nvfp4(X, packed, pattern, torch.float32).double()
        v = plain + b.double()
        want = v * torch.sigmoid(v) + r.double()
        got = ss.linear_nvfp4(X, packed, pattern, BF, epilogue=ss.Epilogue(bias=b, act="silu", residual=r))
        # half a step of bf16, and fp32 arithmetic on values of order one
        assert ((got.double() - want).abs() <= want.abs() * 2.0 ** -8 + 1e-5).all()
