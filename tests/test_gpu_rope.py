"""Rotary positions against 64 bits: layouts, partial heads, far positions,
scaled frequencies, strided views, in place."""
import numpy as np
import pytest
import torch

import structured_sparse_quantized_b200 as ss
import _layer as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def make(T, Hq, Hk, D, dtype, far=131072, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed + T + D)
    qkv = torch.randn(T, (Hq + 2 * Hk) * D + pad, generator=g).to(dtype).cuda()
    q = qkv[:, pad:pad + Hq * D].unflatten(1, (Hq, D))
    k = qkv[:, pad + Hq * D:pad + (Hq + Hk) * D].unflatten(1, (Hk, D))
    pos = torch.randint(0, far, (T,), generator=g)
    return qkv, q, k, pos


def check(q, k, pos, freqs, scale, layout, out=None):
    want = [ref.rope(t.clone(), pos, freqs.cpu().numpy(), layout, scale) for t in (q, k)]
    got = ss.rope(q, k, pos.cuda(), freqs, layout, scale, out=out)
    assert ss.ss_get_device_status() == ss.SS_OK
    for y, w in zip(got, want):
        ref.assert_within(y, *w)
    return got


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,Hq,Hk,D,rot", [
    (1, 32, 8, 128, 128), (64, 28, 4, 128, 128), (257, 5, 5, 64, 64), (33, 16, 2, 80, 32),
    (19, 7, 1, 96, 96), (130, 3, 3, 256, 64), (7, 1, 1, 2, 2), (40, 9, 3, 66, 42),
    (3, 2, 1, 1024, 1022), (5, 64, 64, 72, 72), (70, 3, 1, 104, 72), (31, 2, 2, 64, 24),
    (40, 4, 2, 96, 40), (33, 5, 1, 128, 90), (50, 2, 2, 68, 36),
])
def test_layouts_and_sizes(layout, dtype, T, Hq, Hk, D, rot):
    _, q, k, pos = make(T, Hq, Hk, D, dtype)
    f, s = ss.rope_frequencies(rot, 500000.0)
    check(q, k, pos, f, s, layout)


@pytest.mark.parametrize("kind", ["none", "linear", "ntk", "llama3", "yarn"])
@pytest.mark.parametrize("far", [1, 8192, 1 << 20, 1 << 31])
def test_scaled_and_far_positions(kind, far):
    _, q, k, pos = make(50, 4, 2, 128, F32, far=far)
    f, s = ss.rope_frequencies(128, 500000.0, kind, 8.0, 8192)
    check(q, k, pos, f, s, "half")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot,pad", [(128, 128, 0), (128, 64, 8), (80, 32, 3), (64, 64, 1)])
def test_in_place_leaves_the_rest(layout, D, rot, pad):
    """In place inside a projection's output: values, padding and the elements
    past rot keep their bits.  pad = 1, 3: rows that are not 16-byte aligned."""
    qkv, q, k, pos = make(21, 6, 2, D, BF, pad=pad)
    before = qkv.clone()
    f, s = ss.rope_frequencies(rot, 10000.0)
    check(q, k, pos, f, s, layout, out=(q, k))
    assert torch.equal(qkv[:, :pad], before[:, :pad])
    assert torch.equal(qkv[:, pad + 8 * D:], before[:, pad + 8 * D:])
    if rot < D:
        assert torch.equal(q[..., rot:], before[:, pad:pad + 6 * D].unflatten(1, (6, D))[..., rot:])


def test_positions_int32_and_negative():
    """Negated positions turn back what positions turned (the gradient's map)."""
    _, q, k, pos = make(40, 4, 2, 64, F32, far=1000)
    f, s = ss.rope_frequencies(64, 10000.0)
    q1, k1 = ss.rope(q, k, pos.int().cuda(), f)
    q2, k2 = ss.rope(q1, k1, (-pos).cuda(), f)
    q64, _ = ss.rope(q, None, pos.cuda(), f)
    assert torch.equal(q1, q64)
    for a, b in ((q, q2), (k, k2)):
        # two turns, each off by 3 * 2^-23 of |a| + |b| and a rounding
        assert ((a - b).abs() <= 2.0 ** -19 * a.abs().amax()).all()


def test_gradient_is_the_negated_call():
    """d/dx of sum(g * rope(x)) is rope(g) at negated positions, against
    central differences of the 64-bit reference."""
    T, H, D = 3, 2, 16
    g = torch.Generator().manual_seed(3)
    x, up = torch.randn(T, H, D, generator=g), torch.randn(T, H, D, generator=g)
    pos = torch.tensor([0, 5, 77])
    f, s = ss.rope_frequencies(12, 10000.0, "yarn", 4.0, 32)
    for layout in ("half", "interleaved"):
        got = ss.rope(up.cuda(), None, (-pos).cuda(), f, layout, s)[0].cpu().double().numpy()
        for t, h, d in [(0, 0, 0), (1, 1, 5), (2, 0, 7), (2, 1, 11), (1, 0, 15)]:
            hi, lo = x.double().clone(), x.double().clone()
            hi[t, h, d] += 1e-3
            lo[t, h, d] -= 1e-3
            fn = lambda v: (ref.rope(v, pos, f.cpu().numpy(), layout, s)[0] * up.double().numpy()).sum()
            # the map is linear, so the difference quotient is exact to 64-bit rounding
            assert abs((fn(hi) - fn(lo)) / 2e-3 - got[t, h, d]) < 1e-5


def test_strided_heads_and_outputs():
    """Heads before tokens, outputs of other strides, one tensor in place."""
    g = torch.Generator().manual_seed(0)
    q = torch.randn(4, 50, 64, generator=g).to(BF).cuda().transpose(0, 1)
    k = torch.randn(50, 2, 128, generator=g).to(BF).cuda()[..., 64:]
    pos = torch.arange(50)
    f, s = ss.rope_frequencies(48, 10000.0)
    out = torch.full((50, 9, 64), 5.0, dtype=BF, device="cuda")
    check(q, k, pos, f, s, "half", out=(out[:, 2:6], k))
    assert (out[:, :2] == 5).all() and (out[:, 6:] == 5).all()


def test_long_tensor_offsets():
    """Offsets past 2^31 elements: a token stride of 2^22 over 600 tokens."""
    T, stride = 600, 1 << 22
    buf = torch.empty(T * stride, dtype=BF, device="cuda")
    q = buf.as_strided((T, 2, 64), (stride, 64, 1))
    q.copy_(torch.randn(T, 2, 64, generator=torch.Generator().manual_seed(0)))
    pos = torch.arange(T)
    f, s = ss.rope_frequencies(64, 10000.0)
    want = ref.rope(q.clone(), pos, f.cpu().numpy(), "half", s)
    got, _ = ss.rope(q, None, pos.cuda(), f)
    ref.assert_within(got, *want)
    ss.rope(q, None, pos.cuda(), f, out=(q, None))
    assert torch.equal(q, got)


def test_captured_graph():
    _, q, k, pos = make(64, 32, 8, 128, BF)
    f, s = ss.rope_frequencies(128, 500000.0)
    p = pos.cuda()
    out = (torch.empty(64, 32, 128, dtype=BF, device="cuda"), torch.empty(64, 8, 128, dtype=BF, device="cuda"))
    ss.rope(q, k, p, f, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ss.rope(q, k, p, f, out=out)
    new = pos + 17
    p.copy_(new)
    graph.replay()
    torch.cuda.synchronize()
    for y, x in zip(out, (q, k)):
        ref.assert_within(y, *ref.rope(x, new, f.cpu().numpy(), "half", s))


def test_refusals_on_the_device():
    _, q, k, pos = make(8, 4, 2, 64, BF)
    f, s = ss.rope_frequencies(64)
    p = pos.cuda()
    for bad in (dict(q=q[:4]), dict(k=k.float()), dict(k=k[:, :, :32]), dict(positions=p[:4]),
                dict(positions=p.float()), dict(positions=pos), dict(freqs=f.float()), dict(freqs=f.cpu()),
                dict(q=q.half()), dict(q=q.transpose(1, 2)), dict(q=q[0]),
                dict(out=(torch.empty(8, 4, 64, device="cuda", dtype=BF), None)),
                dict(out=(torch.empty(1, 1, 64, device="cuda", dtype=BF).expand(8, 4, 64), k))):
        with pytest.raises(ValueError):
            ss.rope(**({"q": q, "k": k, "positions": p, "freqs": f} | bad))
    with pytest.raises(ss.SSError):  # more frequencies than pairs
        ss.rope(q, k, p, torch.ones(33, dtype=torch.float64, device="cuda"))
    with pytest.raises(ss.SSError):
        ss.rope(q[:0], None, p[:0], f)


def test_one_token_any_strides():
    """With one token its stride means nothing, whatever it says."""
    x = torch.randn(2, 64, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    q = x.as_strided((1, 2, 64), (7, 64, 1))
    f, s = ss.rope_frequencies(64)
    pos = torch.tensor([5])
    got, _ = ss.rope(q, None, pos.cuda(), f)
    ref.assert_within(got, *ref.rope(q, pos, f.cpu().numpy(), "half", s))


def test_stream_argument():
    _, q, k, pos = make(64, 8, 2, 128, BF)
    f, sc = ss.rope_frequencies(128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p = pos.cuda()
    s.wait_stream(torch.cuda.current_stream())
    got = ss.rope(q, k, p, f, stream=s)
    s.synchronize()
    for y, x in zip(got, (q, k)):
        ref.assert_within(y, *ref.rope(x, pos, f.cpu().numpy(), "half", sc))
