"""The GEMMs' fused epilogue (bias, activation plain and gated, residual)
against 64 bits, in every kernel shape, tier and operand form."""
import numpy as np
import pytest
import torch

import structured_sparse_quantized_b200 as ss
import _layer as ref
from _helpers import dev

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
# bias, act, gated, residual, out
EPILOGUES = [
    (BF, "none", False, None, BF),
    (None, "none", False, BF, BF),
    (F32, "relu", False, F32, F32),
    (None, "silu", True, None, BF),
    (BF, "gelu", True, None, F32),
    (F32, "gelu_erf", False, BF, BF),
    (BF, "silu", False, F32, BF),
    (F32, "none", True, None, BF),
    (None, "gelu", False, BF, F32),
    (F32, "gelu_erf", True, None, BF),
]
# M, N, L: single rows, ragged tiles, every kernel shape's edges
SHAPES = [
    (1, 16, 128),       # one tile, one token
    (5, 48, 384),       # K split over a cluster, ragged rows
    (64, 1008, 640),    # K split, the most tokens
    (33, 4096, 512),    # K split
    (65, 144, 128),     # CTA pair, second CTA almost empty
    (300, 272, 1152),   # several token tiles
    (129, 131, 256),    # rows of Y not 16-byte aligned
    (700, 520, 256),    # 520 = 4 * 128 + 8
]
FORMS = [(t, f) for t in ("int8", "fp8", "bf16") for f in ("w", "x", "dense")] + \
        [("nvfp4", "w"), ("nvfp4", "dense")]


class Product:
    """Random operands of one product on the device and its exact fp32 value."""

    def __init__(self, M, N, L, tier, form, seed=0):
        rng = np.random.default_rng(seed + M * 7 + N * 3 + L)
        self.M, self.N, self.tier, self.form = M, N, tier, form
        if tier == "nvfp4":
            L = -(-L // 256) * 256
            block = 32 if form == "w" else 16
            wv, wm, ws, w = ref.operand_fp4(rng, N, L, form == "w", block)
            xv, _, xs, x = ref.operand_fp4(rng, M, L, False, block)
            gx, gw = np.float32(0.37), np.float32(0.03)
            self.d = ref.dequantised(x, w, [gx], gw)
            g = lambda v: dev(np.full(4, v, np.float32))
            self.w = (dev(wv), None if wm is None else dev(wm), dev(ws), g(gw))
            self.x = (dev(xv), dev(xs), g(gx))
            return
        wv, wm, w = ref.operand(rng, N, L, tier, form == "w")
        xv, xm, x = ref.operand(rng, M, L, tier, form == "x")
        s_x = s_w = None
        if tier != "bf16":
            s_x = rng.uniform(0.02, 0.06, M).astype(np.float32)
            s_w = rng.uniform(0.1, 0.5, N).astype(np.float32)
        self.d = ref.dequantised(x, w, s_x, s_w)
        put = lambda t: None if t is None else dev(t)
        self.w, self.x = [put(t) for t in (wv, wm, s_w)], [put(t) for t in (xv, xm, s_x)]

    def run(self, e, out, y=None):
        M, N = self.M, self.N
        if self.tier == "nvfp4":
            if self.form == "w":
                return ss.sparse_gemm_nvfp4(self.w, self.x, M, N, out, out=y, epilogue=e)
            return ss.dense_gemm_nvfp4(self.x, self.w, M, N, out, out=y, epilogue=e)
        (wv, wm, sw), (xv, xm, sx) = self.w, self.x
        if self.form == "w":
            return ss.sparse_gemm(0, wv, wm, sw, xv, sx, M, N, self.tier, out, out=y, epilogue=e)
        if self.form == "x":
            return ss.sparse_gemm(1, xv, xm, sx, wv, sw, M, N, self.tier, out, out=y, epilogue=e)
        return ss.dense_gemm(xv, sx, wv, sw, self.tier, out, out=y, epilogue=e)


def check(p: Product, bias, act, gated, residual, out, seed=5):
    g = torch.Generator().manual_seed(seed)
    b = None if bias is None else torch.randn(p.N, generator=g).to(bias)
    r = None if residual is None else (torch.randn(p.M, p.N, generator=g) * 3).to(residual)
    e = ss.Epilogue(bias=None if b is None else dev(b), act=act, gated=gated,
                    residual=None if r is None else dev(r))
    y = p.run(e, out)
    assert y.dtype == out
    assert ss.ss_get_device_status() == ss.SS_OK
    ref.assert_within(y, *ref.epilogue(p.d, b, act, gated, r, out))
    return y


@pytest.mark.parametrize("tier,form", FORMS)
@pytest.mark.parametrize("M,N,L", SHAPES)
def test_epilogues(tier, form, M, N, L):
    p = Product(M, N, L, tier, form)
    for e in EPILOGUES:
        if e[2] and N % 16:
            continue
        check(p, *e)


@pytest.mark.parametrize("tier,form", [("int8", "w"), ("fp8", "x"), ("int8", "x"), ("fp8", "w")])
@pytest.mark.parametrize("kernel", ["wide", "narrow", "splitk"])
@pytest.mark.parametrize("M,N,L", [(50, 1024, 1024), (1000, 656, 512), (460, 2064, 256)])
def test_pinned_kernel_shapes(tier, form, kernel, M, N, L, monkeypatch):
    monkeypatch.setenv("SS_SPARSE_KERNEL", kernel)
    p = Product(M, N, L, tier, form)
    for e in EPILOGUES:
        check(p, *e)


@pytest.mark.parametrize("M,N,L", [(1, 512, 512), (300, 1040, 256)])
def test_wide_values_and_extremes(M, N, L):
    """Pre-activations over the activations' whole range: large magnitudes of
    both signs, where exponentials overflow, and a bias of infinities and NaN."""
    p = Product(M, N, L, "int8", "w")
    for act in ("relu", "silu", "gelu", "gelu_erf"):
        b = torch.linspace(-120, 120, N)
        y = p.run(ss.Epilogue(bias=dev(b), act=act), F32)
        ref.assert_within(y, *ref.epilogue(p.d, b, act, False, None, F32))
        b[3], b[5], b[9] = float("inf"), float("nan"), 3e38
        y = p.run(ss.Epilogue(bias=dev(b), act=act), F32)
        assert torch.isposinf(y[:, 3]).all() and torch.isnan(y[:, 5]).all()
        assert (y[:, 9] > 1e38).all()
        keep = [i for i in range(N) if i not in (3, 5, 9)]
        want, bound = ref.epilogue(p.d[:, keep], b[keep], act, False, None, F32)
        ref.assert_within(y[:, keep], want, bound)


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,N,L", [(3, 256, 512), (300, 1032, 256), (70, 131, 128)])
def test_residual_updated_in_place(out, M, N, L):
    p = Product(M, N, L, "int8", "w")
    y = dev((torch.randn(M, N, generator=torch.Generator().manual_seed(1)) * 2).to(out))
    r = y.cpu().clone()
    got = p.run(ss.Epilogue(residual=y), out, y)
    assert got.data_ptr() == y.data_ptr()
    ref.assert_within(y, *ref.epilogue(p.d, None, "none", False, r, out))


def test_rows_and_columns_past_the_output_stay():
    """Nothing is written past the M x N output, whatever the tile."""
    for M, N, L, gated in [(1, 16, 128, False), (70, 144, 128, True), (129, 131, 128, False),
                           (300, 272, 256, False), (300, 272, 256, True)]:
        for out in (BF, F32):
            p = Product(M, N, L, "int8", "w")
            n = M * (N // 2 if gated else N)
            buf = torch.full((n + 4096,), 7.0, dtype=out, device="cuda")
            y = buf[:n].view(M, -1)
            p.run(ss.Epilogue(act="silu", gated=gated), out, y)
            assert (buf[n:] == 7.0).all()


def test_empty_epilogue_equals_plain_call():
    for tier, form in FORMS:
        p = Product(130, 144, 256, tier, form)
        y = p.run(ss.Epilogue(), BF)
        want = torch.from_numpy(p.d).float().to(BF)  # the fp32 value, then bf16
        assert torch.equal(y.cpu(), want)


def test_captured_graph_replays_on_new_inputs():
    p = Product(300, 272, 512, "int8", "w")
    r = torch.zeros(300, 272, dtype=BF, device="cuda")
    y = torch.empty_like(r)
    e = ss.Epilogue(act="silu", residual=r)
    p.run(e, BF, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run(e, BF, y)
    for seed in range(3):
        new = torch.randn(300, 272, generator=torch.Generator().manual_seed(seed)).to(BF)
        r.copy_(new)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        ref.assert_within(y, *ref.epilogue(p.d, None, "silu", False, new, BF))


def test_another_stream():
    p = Product(300, 272, 512, "fp8", "w")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = dev(torch.randn(272))
    with torch.cuda.stream(s):
        ys = [p.run(ss.Epilogue(bias=b, act="gelu"), BF) for _ in range(4)]
    s.synchronize()
    want = ref.epilogue(p.d, b.cpu(), "gelu", False, None, BF)
    for y in ys:
        ref.assert_within(y, *want)


@pytest.mark.parametrize("kind", ["torch", "handle"])
def test_stream_argument(kind):
    """Results and their memory belong to the stream that is passed."""
    p = Product(300, 272, 512, "int8", "w")
    b = dev(torch.randn(272))
    want = ref.epilogue(p.d, b.cpu(), "silu", False, None, BF)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    (wv, wm, sw), (xv, _, sx) = p.w, p.x
    ys = [ss.sparse_gemm(0, wv, wm, sw, xv, sx, 300, 272, "int8", BF,
                         stream=s if kind == "torch" else s.cuda_stream,
                         epilogue=ss.Epilogue(bias=b, act="silu")) for _ in range(8)]
    s.synchronize()
    for y in ys:
        ref.assert_within(y, *want)


def test_two_streams_and_two_graphs_at_once():
    """Calls in flight on two streams, then two captured graphs that share
    their inputs, replayed together: nothing is shared but what is read."""
    p = Product(700, 528, 512, "fp8", "w")
    r = dev((torch.randn(700, 528, generator=torch.Generator().manual_seed(2))).to(BF))
    cases = [ss.Epilogue(act="gelu", residual=r), ss.Epilogue(act="silu", gated=True)]
    wants = [ref.epilogue(p.d, None, "gelu", False, r.cpu(), BF),
             ref.epilogue(p.d, None, "silu", True, None, BF)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.empty(700, 528, dtype=BF, device="cuda"), torch.empty(700, 264, dtype=BF, device="cuda")]
    torch.cuda.synchronize()
    for _ in range(6):
        for s, e, y in zip(streams, cases, outs):
            with torch.cuda.stream(s):
                p.run(e, BF, y)
    torch.cuda.synchronize()
    for y, want in zip(outs, wants):
        ref.assert_within(y, *want)
    graphs = []
    for s, e, y in zip(streams, cases, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            p.run(e, BF, y)
        graphs.append(g)
        y.zero_()
    torch.cuda.synchronize()
    for _ in range(4):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for y, want in zip(outs, wants):
        ref.assert_within(y, *want)


@pytest.mark.parametrize("kernel", ["narrow", "wide"])
@pytest.mark.parametrize("form", ["w", "x", "dense"])
def test_wait_runs_out_then_next_call_is_clean(kernel, form, monkeypatch):
    """A K stage that is never loaded (a wait that nothing satisfies, limited to
    20 ms): the call records the timeout, residual loads in flight land, and the
    next call is right."""
    if form != "w" and kernel == "wide":
        pytest.skip("channel rows of a sparse weight only")
    monkeypatch.setenv("SS_SPARSE_KERNEL", kernel)
    p = Product(500, 1024, 2048, "int8", form)
    assert ss.ss_get_device_status() == ss.SS_OK
    r = dev(torch.randn(500, 1024, generator=torch.Generator().manual_seed(4)).to(BF))
    e = ss.Epilogue(act="silu", residual=r)
    try:
        ss.ss_debug_set_wait_limit(20_000_000)
        ss.ss_debug_skip_stage(1)
        p.run(e, BF)
        assert ss.ss_get_device_status() == ss.SS_ERR_TIMEOUT
        assert ss.ss_get_device_status() == ss.SS_OK
    finally:
        ss.ss_debug_skip_stage(-1)
        ss.ss_debug_set_wait_limit(4_000_000_000)
    y = p.run(e, BF)
    assert ss.ss_get_device_status() == ss.SS_OK
    ref.assert_within(y, *ref.epilogue(p.d, None, "silu", False, r.cpu(), BF))


def test_refusals_on_the_device():
    p = Product(32, 48, 256, "int8", "w")
    (wv, wm, sw), (xv, _, sx) = p.w, p.x

    def run(e=ss.Epilogue(act="relu"), M=32, N=48, y=None, w=wv, m=wm, s=sw, x=xv):
        return ss.sparse_gemm(0, w, m, s, x, sx, M, N, "int8", out=y, epilogue=e)
    run()
    bad = [dict(e=ss.Epilogue(bias=torch.zeros(47, device="cuda"))),
           dict(e=ss.Epilogue(bias=torch.zeros(48, device="cuda", dtype=torch.float16))),
           dict(e=ss.Epilogue(bias=torch.zeros(48))),
           dict(e=ss.Epilogue(bias=torch.zeros(96, device="cuda")[::2])),
           dict(e=ss.Epilogue(residual=torch.zeros(32, 24, device="cuda"))),
           dict(M=31), dict(N=47), dict(y=torch.empty(32, 24, device="cuda", dtype=BF)),
           dict(y=torch.empty(32, 48, device="cuda", dtype=torch.float16)), dict(m=wm.flatten()[1:]),
           dict(w=wv.float()), dict(s=None), dict(s=sw[:-1]), dict(x=xv[:-1])]
    for kw in bad:
        with pytest.raises(ValueError):
            run(**kw)
    for e, status in ((ss.Epilogue(act="silu", gated=True, residual=torch.zeros(32, 48, device="cuda")),
                       ss.SS_ERR_UNSUPPORTED),
                      (ss.Epilogue(bias=torch.zeros(52, device="cuda")[1:49]), ss.SS_ERR_ALIGNMENT)):
        with pytest.raises(ss.SSError) as err:
            run(e)
        assert err.value.status == status
    q = Product(32, 40, 256, "int8", "w")
    with pytest.raises(ss.SSError) as err:
        q.run(ss.Epilogue(act="silu", gated=True), BF)
    assert err.value.status == ss.SS_ERR_INVALID_ARG
