"""The operators that a transformer layer's linear path needs around the quantised matmul, as cases:

  gemm   sparse or dense matrix product with bias, activation (plain or gated) and residual in its epilogue
  rope   rotary positions of the query and key heads
  norm   RMS norm fused into the per-token quantisation and lift of the next product's input

`run` computes them from elementary torch operations, or, where `own` is true, by the package's own calls on the same
inputs.  Operands are drawn directly in their stored form (quantised codes, 2:4 selectors, scales)."""
import math

import torch

own = False

DEV = "cuda"
OUT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"2:4": 2, "4:6": 3, "6:8": 4, "8:10": 5, "dense": 0}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def up(x, m):
    return (x + m - 1) // m * m


def lifted(K, pattern, tier):
    """Padded length of the lifted reduction axis that the product runs over."""
    if tier == "nvfp4":
        return up(K, 256) if pattern == "dense" else 2 * lifted((K + 1) // 2, pattern, "int8")
    h = HALF[pattern]
    return up(K, 128) if h == 0 else up(-(-K // (2 * h)) * (h - 1) * 4, 128)


# ---------------------------------------------------------------------------------------------- cases
def gemm(name, M, N, K, pattern, tier, sparse="w", bias="none", act="none", gated=False, residual="none", out="bf16"):
    c = dict(op="gemm", M=M, N=N, K=K, pattern=pattern, tier=tier, sparse=sparse, bias=bias, act=act, gated=gated,
             residual=residual, out=out)
    return dict(c, name=name) if name else c


def rope(name, T, Hq, Hk, D, rot, layout, scaling, dtype="bf16", far=131072):
    c = dict(op="rope", T=T, Hq=Hq, Hk=Hk, D=D, rot=rot, layout=layout, scaling=scaling, dtype=dtype, far=far)
    return dict(c, name=name) if name else c


def norm(name, M, K, pattern, tier, dtype="bf16", weight="bf16"):
    c = dict(op="norm", M=M, K=K, pattern=pattern, tier=tier, dtype=dtype, weight=weight)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of a Llama-3.1-8B query projection with a bias: the smallest call, latency
        gemm("decode_q_bias", 1, 4096, 4096, "2:4", "int8", bias="bf16"),
        # a decode batch through the gate and up projections, SwiGLU in the epilogue: reads the weight once
        gemm("decode_gate_up", 16, 28672, 4096, "6:8", "fp8", act="silu", gated=True),
        # prefill of the output projection, added to the residual stream
        gemm("prefill_o_residual", 8192, 4096, 4096, "2:4", "int8", residual="bf16"),
        # prefill of the Qwen2.5-7B gate and up projections with SwiGLU
        gemm("prefill_gate_up", 8192, 37888, 3584, "6:8", "fp8", act="silu", gated=True),
        # prefill of the down projection into the residual stream: the longest reduction
        gemm("prefill_down_residual", 16384, 4096, 14336, "6:8", "int8", residual="bf16"),
        # the 16-bit tier without sparsity: a feed-forward with bias and GELU
        gemm("bf16_dense_gelu", 2048, 14336, 4096, "dense", "bf16", bias="f32", act="gelu"),
        # odd sizes, every operand of the epilogue, fp32 residual stream
        gemm("ragged_f32_stream", 1000, 1001, 650, "4:6", "int8", bias="f32", act="relu", residual="f32", out="f32"),
        # block-scaled FP4 with pairwise sparsity
        gemm("nvfp4_bias_gelu", 8192, 14336, 4096, "2:4", "nvfp4", bias="bf16", act="gelu"),
        # a decode batch's query and key heads, at far positions
        rope("rope_decode", 64, 32, 8, 128, 128, "half", "llama3"),
        # a prompt's heads, YaRN-scaled
        rope("rope_prefill", 16384, 28, 4, 128, 128, "half", "yarn"),
        # one token's input of a projection
        norm("norm_decode", 1, 4096, "6:8", "int8"),
        # a prompt's inputs
        norm("norm_prefill", 16384, 4096, "6:8", "fp8"),
    ]


def log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "gemm", "rope", "norm"])
    if op == "rope":
        D = rng.choice([64, 80, 96, 128, 256])
        rot = D if rng.random() < 0.6 else up(rng.randrange(2, D + 1), 2)
        Hq = rng.randrange(1, 65)
        Hk = rng.choice([h for h in range(1, Hq + 1) if Hq % h == 0])
        T = min(log_int(rng, 1, 16384), 16384 * 32 * 128 // ((Hq + Hk) * D))
        return rope(None, T, Hq, Hk, D, rot, rng.choice(["half", "interleaved"]), rng.choice(["none", "linear", "ntk", "llama3", "yarn"]),
                    rng.choice(["bf16", "bf16", "f32"]), rng.choice([4096, 131072, 1048576]))
    if op == "norm":
        K = log_int(rng, 64, 16384)
        K = K if rng.random() < 0.4 else up(K, 64)
        M = min(log_int(rng, 1, 16384), 16384 * 4096 // K)
        return norm(None, M, K, rng.choice(list(HALF)), rng.choice(["int8", "fp8", "bf16"]), rng.choice(["bf16", "bf16", "f32"]),
                    rng.choice(["bf16", "f32"]))
    while True:
        tier = rng.choice(["int8", "fp8", "bf16", "nvfp4"])
        sparse = rng.choice(["w", "w", "x", "no"]) if tier != "nvfp4" else rng.choice(["w", "w", "no"])
        pattern = "dense" if sparse == "no" else "2:4" if sparse == "x" else rng.choice(["2:4", "4:6", "6:8", "8:10"])
        gated = rng.random() < 0.3
        M, N, K = log_int(rng, 1, 16384), log_int(rng, 16, 28672), log_int(rng, 64, 14336)
        if rng.random() < 0.7:
            N, K = up(N, 16), up(K, 16)
        if gated:
            N = up(N, 16)
        # fp32 results of the 16-bit tier are for short reductions: the tensor core's own fp32 sum is off by about 1e-9 a step
        out = rng.choice(["bf16", "bf16", "f32"]) if tier != "bf16" or K <= 4096 else "bf16"
        if M * N * lifted(K, pattern, tier) <= 8192 * 37888 * 5376:
            return gemm(None, M, N, K, pattern, tier, sparse, rng.choice(["none", "bf16", "f32"]),
                        rng.choice(["silu", "gelu", "relu", "gelu_erf"] + ([] if gated else ["none", "none"])), gated,
                        "none" if gated else rng.choice(["none", "bf16", "f32"]), out)


# ---------------------------------------------------------------------------------------------- inputs
def codes(g, rows, cols, tier):
    """Stored values of standard deviation about 32 (int8), 64 (fp8), 1 (bf16); random E2M1 pairs for nvfp4."""
    if tier == "nvfp4":
        return torch.randint(0, 256, (rows, cols), generator=g, device=DEV, dtype=torch.uint8)
    out = torch.empty((rows, cols), dtype=torch.bfloat16 if tier == "bf16" else torch.uint8, device=DEV)
    for a in range(0, rows, 4096):
        x = torch.randn((min(4096, rows - a), cols), generator=g, device=DEV)
        if tier == "int8":
            out[a:a + 4096] = (x * 32).round_().clamp_(-127, 127).to(torch.int8).view(torch.uint8)
        elif tier == "fp8":
            out[a:a + 4096] = (x * 64).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            out[a:a + 4096] = x.to(torch.bfloat16)
    return out


def selectors(g, rows, windows, tier):
    """Two kept positions in each window of four, as the tile-major metadata of 128 rows x 16 bytes."""
    pair = torch.tensor([4, 8, 12, 9, 13, 14], dtype=torch.uint8, device=DEV)
    nib = pair[torch.randint(0, 6, (rows, windows), generator=g, device=DEV, dtype=torch.uint8).int()]
    b = torch.zeros((up(rows, 128), windows // 2), dtype=torch.uint8, device=DEV)
    b[:rows] = nib[:, 0::2] | (nib[:, 1::2] << 4)
    b = b.view(b.shape[0] // 128, 128, -1, 16).permute(0, 2, 1, 3).contiguous()
    return swap_halves(b) if tier == "bf16" else b


def swap_halves(tiles):
    """The 16-bit tier exchanges row bit 3 and byte bit 1 inside each tile."""
    t = tiles.view(-1, 8, 2, 8, 4, 2, 2)
    return t.permute(0, 1, 5, 3, 4, 2, 6).contiguous().view(tiles.shape)


def scale_tiles(s):
    """[rows, blocks] scales as 512-byte blocks: rows 32-strided, four blocks of K together."""
    rows, n = s.shape
    p = torch.zeros((up(rows, 128), n), dtype=torch.uint8, device=DEV)
    p[:rows] = s
    return p.view(-1, 4, 32, n // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def lift_index(K, pattern, L):
    """Source of each lifted element, and where there is one."""
    h = HALF[pattern]
    k = torch.arange(L, device=DEV)
    if h <= 2:
        return k.clamp(max=K - 1), k < K
    win, t = k // 4, k % 4
    at = 2 * h * (win // (h - 1)) + 2 * (win % (h - 1)) + t
    ok = (at < K) & (k < -(-K // (2 * h)) * (h - 1) * 4)
    return at.clamp(max=K - 1), ok


def frequencies(rot, scaling, base=500000.0, factor=8.0, first=8192.0):
    """Radians per position of each rotated pair, in 64 bits, and the factor on cos and sin."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    f = base ** (-2 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "ntk":
        return (base * factor ** (rot / max(1, rot - 2))) ** (-2 * i / rot), 1.0
    if scaling == "llama3":
        turns = first * f / (2 * math.pi)
        mix = ((turns - 1.0) / 3.0).clamp(0, 1)
        return f * (mix + (1 - mix) / factor), 1.0
    if scaling == "yarn":
        edge = [rot * math.log(first / (b * 2 * math.pi)) / (2 * math.log(base)) for b in (32.0, 1.0)]
        lo, hi = max(0, math.floor(edge[0])), min(rot - 1, math.ceil(edge[1]))
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    rand = lambda *s: torch.rand(s, generator=g, device=DEV)  # noqa: E731
    if case["op"] == "rope":
        T, Hq, Hk, D = case["T"], case["Hq"], case["Hk"], case["D"]
        # query, key and value heads as one projection leaves them
        qkv = randn(T, (Hq + 2 * Hk) * D).to(OUT[case["dtype"]])
        # packed sequences: positions start anew, the last ones reach far
        pos = (torch.arange(T, device=DEV) % max(1, T // 3 + 1) + torch.randint(0, max(1, case["far"] - T), (1,), generator=g, device=DEV))
        f, scale = frequencies(case["rot"], case["scaling"])
        return dict(case=case, q=qkv[:, :Hq * D].view(T, Hq, D), k=qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D), pos=pos, freqs=f,
                    scale=scale)
    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        X = randn(M, K)
        X[:, torch.randperm(K, generator=g, device=DEV)[:max(1, K // 100)]] *= 20  # outlier channels
        return dict(case=case, X=X.to(OUT[case["dtype"]]), w=(1 + 0.1 * randn(K)).to(OUT[case["weight"]]), eps=1e-5)
    M, N, K, tier, sparse = case["M"], case["N"], case["K"], case["tier"], case["sparse"]
    L = lifted(K, case["pattern"], tier)
    s = dict(case=case, L=L, bias=None, residual=None)
    W, X = {}, {}
    if tier == "nvfp4":
        W["v"] = codes(g, N, L // 4 if sparse == "w" else L // 2, tier)
        W["m"] = selectors(g, N, L // 8, tier) if sparse == "w" else None
        block = 32 if sparse == "w" else 16
        for t, rows in ((W, N), (X, M)):
            t["s"] = scale_tiles((rand(rows, L // block) * 4 + 0.5).to(torch.float8_e4m3fn).view(torch.uint8))
        at, ok = lift_index((K + 1) // 2, case["pattern"], L // 2)
        X["v"] = codes(g, M, (K + 1) // 2, tier)[:, at] * ok.to(torch.uint8)
        n = K / 2 if sparse == "w" else K
        X["g"] = torch.full((4,), 1 / 7.6, device=DEV)
        W["g"] = torch.full((4,), 1 / (7.6 * math.sqrt(n)), device=DEV)
    else:
        std = {"int8": 32.0, "fp8": 64.0, "bf16": 1.0}[tier]
        n = K if sparse == "no" else L / 2
        at, ok = lift_index(K, case["pattern"], L)
        for t, rows, other in ((W, N, "x"), (X, M, "w")):
            if sparse != "no" and sparse != other:  # the sparse operand
                t["v"], t["m"] = codes(g, rows, L // 2, tier), selectors(g, rows, L // 4, tier)
            else:
                v = codes(g, rows, K, tier)
                t["v"], t["m"] = torch.where(ok, v[:, at], torch.zeros((), dtype=v.dtype, device=DEV)), None
        X["s"] = (0.5 + rand(M)) / std if tier != "bf16" else None
        W["s"] = (0.5 + rand(N)) / (std * math.sqrt(n)) if tier != "bf16" else None
        if tier == "bf16":
            W["v"] = W["v"] / math.sqrt(n)
    if case["bias"] != "none":
        s["bias"] = (0.5 * randn(N)).to(OUT[case["bias"]])
    if case["residual"] != "none":
        s["residual"] = randn(M, N).to(OUT[case["residual"]])
    return dict(s, W=W, X=X)


# ---------------------------------------------------------------------------------------------- plain forms
def values(v, tier):
    if tier == "int8":
        return v.view(torch.int8).float()
    if tier == "fp8":
        return v.view(torch.float8_e4m3fn).float()
    if tier == "bf16":
        return v.float()
    table = torch.tensor(E2M1 + [-x for x in E2M1], device=DEV)
    return torch.stack((table[(v & 15).int()], table[(v >> 4).int()]), -1).flatten(1)


def unpack(t, rows, L, tier):
    """The operand as a matrix of 32-bit values, [rows, L] (without its per-row scale)."""
    v = t["v"]
    if t["m"] is not None:
        tiles = swap_halves(t["m"]) if tier == "bf16" else t["m"]
        b = tiles.permute(0, 2, 1, 3).reshape(tiles.shape[0] * 128, -1)[:rows]
        nib = torch.stack((b & 15, b >> 4), -1).flatten(1)  # one per window
        at = torch.stack((nib & 3, nib >> 2), -1).long()
        n = nib.shape[1]
        wide = torch.zeros((rows, n, 4), dtype=v.dtype, device=DEV)
        v = wide.scatter_(2, at, v.view(rows, n, 2)).view(rows, 4 * n)
    x = values(v, tier)
    if tier == "nvfp4":
        n = t["s"].numel() // up(rows, 128)
        e = t["s"].view(-1, n // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, n)[:rows]
        x = (x.view(rows, n, L // n) * e.view(torch.float8_e4m3fn).float()[:, :, None]).view(rows, L)
    return x


def activate(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "gelu_erf":
        return 0.5 * v * torch.erfc(v * -math.sqrt(0.5))
    return v


def plain_gemm(s):
    c, L = s["case"], s["L"]
    tier, W, X = c["tier"], s["W"], s["X"]
    x = unpack(dict(m=None) | X, c["M"], L, tier)
    v = x @ unpack(W, c["N"], L, tier).t()
    if tier == "nvfp4":
        v = v * X["g"][0] * W["g"][0]
    elif tier != "bf16":
        v = v * X["s"][:, None] * W["s"]
    if s["bias"] is not None:
        v = v + s["bias"].float()
    if c["gated"]:  # rows of the weight: eight gates, then their eight partners
        v = v.view(c["M"], -1, 2, 8)
        v = (activate(v[:, :, 0], c["act"]) * v[:, :, 1]).reshape(c["M"], -1)
    else:
        v = activate(v, c["act"])
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return v.to(OUT[c["out"]])


def plain_rope(x, s):
    c = s["case"]
    r = c["rot"]
    a = s["pos"].double()[:, None] * s["freqs"]
    cos, sin = ((f(a) * s["scale"]).float()[:, None] for f in (torch.cos, torch.sin))
    y = x.float()
    u = y[..., :r]
    p, q = (u[..., :r // 2], u[..., r // 2:]) if c["layout"] == "half" else (u[..., 0::2], u[..., 1::2])
    t = torch.stack((p * cos - q * sin, q * cos + p * sin), -2 if c["layout"] == "half" else -1)
    return torch.cat((t.flatten(-2), y[..., r:]), -1).to(x.dtype)


def quantised(y, tier):
    """Codes and scale of each row: the largest magnitude becomes the largest code."""
    a = y.abs().amax(1, keepdim=True)
    top = 127.0 if tier == "int8" else 448.0
    inv = torch.where(a > 0, top / a, torch.zeros_like(a))
    v = y * inv
    return (v.round().clamp(-127, 127) if tier == "int8" else v.clamp(-448, 448)), (a / top)[:, 0]


def plain_norm(s):
    c = s["case"]
    x = s["X"].float()
    y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + s["eps"]) * s["w"].float()
    at, ok = lift_index(c["K"], c["pattern"], lifted(c["K"], c["pattern"], c["tier"]))
    if c["tier"] == "bf16":
        return dict(x=y.to(torch.bfloat16)[:, at] * ok.to(torch.bfloat16))
    v, scale = quantised(y, c["tier"])
    v = torch.where(ok, v[:, at], torch.zeros((), device=DEV))
    return dict(x=v.to(torch.bfloat16 if c["tier"] == "int8" else torch.float8_e4m3fn), scale=scale)


def run(s):
    c = s["case"]
    if not own:
        if c["op"] == "gemm":
            return plain_gemm(s)
        return dict(q=plain_rope(s["q"], s), k=plain_rope(s["k"], s)) if c["op"] == "rope" else plain_norm(s)
    import structured_sparse_quantized_b200 as ss
    if c["op"] == "rope":
        q, k = ss.rope(s["q"], s["k"], s["pos"], s["freqs"], layout=c["layout"], scale=s["scale"])
        return dict(q=q, k=k)
    if c["op"] == "norm":
        x, scale = ss.norm_quant_lift_act(s["X"], s["w"], s["eps"], c["pattern"], c["tier"])
        if c["tier"] == "bf16":
            return dict(x=x)
        return dict(x=x.view(torch.int8).to(torch.bfloat16) if c["tier"] == "int8" else x.view(torch.float8_e4m3fn), scale=scale)
    W, X, M, N, out = s["W"], s["X"], c["M"], c["N"], OUT[c["out"]]
    e = ss.Epilogue(bias=s["bias"], act=c["act"], gated=c["gated"], residual=s["residual"])
    if c["tier"] == "nvfp4":
        packed, act = (W["v"], W["m"], W["s"], W["g"]), (X["v"], X["s"], X["g"])
        if c["sparse"] == "w":
            return ss.sparse_gemm_nvfp4(packed, act, M, N, out_dtype=out, epilogue=e)
        return ss.dense_gemm_nvfp4(act, packed, M, N, out_dtype=out, epilogue=e)
    if c["sparse"] == "w":
        return ss.sparse_gemm(0, W["v"], W["m"], W["s"], X["v"], X["s"], M, N, c["tier"], out_dtype=out, epilogue=e)
    if c["sparse"] == "x":
        return ss.sparse_gemm(1, X["v"], X["m"], X["s"], W["v"], W["s"], M, N, c["tier"], out_dtype=out, epilogue=e)
    return ss.dense_gemm(X["v"], X["s"], W["v"], W["s"], c["tier"], out_dtype=out, epilogue=e)


# ---------------------------------------------------------------------------------------------- the definition in 64 bits
def exact_operand(t, rows, L, tier, i16):
    """Element (r, k) by the storage formulas: byte offsets of selectors and scales, window arithmetic."""
    pairs = 2 if tier == "nvfp4" else 1  # stored units per window element
    v = t["v"]
    r = torch.arange(rows, device=DEV)[:, None]
    if t.get("m") is not None:
        n = L // (4 * pairs)
        b = torch.arange(n // 2, device=DEV)[None]
        rr, bb = ((r & ~8) | ((b & 2) << 2), (b & ~2) | ((r & 8) >> 2)) if i16 else (r, b)
        byte = t["m"].reshape(-1)[((rr // 128) * (n // 32) + bb // 16) * 2048 + (rr % 128) * 16 + bb % 16]
        dense = torch.zeros(rows * 4 * n, dtype=v.dtype, device=DEV)
        for half in range(2):
            nib = (byte >> (4 * half)) & 15
            win = (2 * b + half).expand(rows, -1)
            for j in range(2):
                at = r * 4 * n + 4 * win + ((nib >> (2 * j)) & 3).long()
                dense[at.reshape(-1)] = torch.gather(v, 1, 2 * win + j).reshape(-1)
        v = dense.view(rows, 4 * n)
    if tier == "int8":
        return v.view(torch.int8).double()
    if tier == "fp8":
        return v.view(torch.float8_e4m3fn).double()
    if tier == "bf16":
        return v.double()
    x = torch.empty((rows, L), dtype=torch.float64, device=DEV)
    for j in range(2):
        u = (v >> (4 * j)) & 15
        mag = torch.tensor(E2M1, dtype=torch.float64, device=DEV)[(u & 7).long()]
        x[:, j::2] = torch.where(u > 7, -mag, mag)
    n = t["s"].numel() // up(rows, 128)
    j = torch.arange(n, device=DEV)[None]
    e = t["s"][((r // 128) * (n // 4) + j // 4) * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4 + j % 4]
    return x * e.view(torch.float8_e4m3fn).double().repeat_interleave(L // n, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        out = {}
        for n in ("q", "k"):
            x, r = s[n].double(), case["rot"]
            i = torch.arange(r // 2, device=DEV)
            a, b = (i, i + r // 2) if case["layout"] == "half" else (2 * i, 2 * i + 1)
            z = torch.complex(x[..., a], x[..., b])
            angle = s["pos"].double()[:, None] * s["freqs"]
            z = z * torch.polar(torch.full_like(angle, s["scale"]), angle)[:, None]
            y = x.clone()
            y[..., a], y[..., b] = z.real, z.imag
            out[n] = y
        return out
    if case["op"] == "norm":
        x = s["X"].double()
        y = x / torch.sqrt((x * x).sum(1, keepdim=True) / case["K"] + s["eps"]) * s["w"].double()
        L, h = lifted(case["K"], case["pattern"], case["tier"]), HALF[case["pattern"]]
        scale = None
        if case["tier"] != "bf16":
            top = {"int8": 127.0, "fp8": 448.0}[case["tier"]]
            a = y.abs().max(1, keepdim=True).values
            scale = (a / top)[:, 0]
            y = torch.where(a > 0, y * (top / a), torch.zeros_like(y))
            y = torch.round(y) if case["tier"] == "int8" else y.clamp(-448, 448).to(torch.float8_e4m3fn).double()
        if h > 2:  # overlapping windows of four, two apart, in each group
            G = -(-case["K"] // (2 * h))
            y = torch.nn.functional.pad(y, (0, G * 2 * h - case["K"])).view(case["M"], G, 2 * h)
            y = torch.cat([y[:, :, 2 * j:2 * j + 4] for j in range(h - 1)], 2).flatten(1)
        y = torch.nn.functional.pad(y, (0, L - y.shape[1]))
        return dict(x=y) if scale is None else dict(x=y, scale=scale)
    c, L, tier = case, s["L"], case["tier"]
    W = exact_operand(s["W"], c["N"], L, tier, tier == "bf16").t()
    M, per = c["M"], max(1, (1 << 30) // max(L, 2 * c["N"]))
    parts = []
    X = exact_operand(s["X"], M, L, tier, tier == "bf16")
    for a in range(0, M, per):
        v = X[a:a + per] @ W
        if tier == "nvfp4":
            v *= s["X"]["g"][0].double() * s["W"]["g"][0].double()
        elif tier != "bf16":
            v *= s["X"]["s"][a:a + per, None].double()
            v *= s["W"]["s"].double()
        if s["bias"] is not None:
            v += s["bias"].double()
        col = torch.arange(c["N"], device=DEV)
        gate = v[:, (col % 16) < 8] if c["gated"] else v
        if c["act"] == "relu":
            y = torch.maximum(gate, torch.zeros_like(gate))
        elif c["act"] == "silu":
            y = gate * torch.sigmoid(gate)
        elif c["act"] == "gelu":
            y = gate * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (gate + 0.044715 * gate ** 3))
        elif c["act"] == "gelu_erf":
            y = gate * torch.special.ndtr(gate)
        else:
            y = gate
        if c["gated"]:
            y = y * v[:, (col % 16) >= 8]
        if s["residual"] is not None:
            y = y + s["residual"][a:a + per].double()
        parts.append(y.float() if c["out"] == "bf16" else y)
    return torch.cat(parts)


# ---------------------------------------------------------------------------------------------- work
def work(case):
    size = {"bf16": 2, "f32": 4, "none": 0}
    if case["op"] == "rope":
        n = case["T"] * (case["Hq"] + case["Hk"]) * case["D"]
        return {"bytes": 2 * n * size[case["dtype"]] + 8 * case["T"] + 4 * case["rot"],
                "flops": 3 * case["T"] * (case["Hq"] + case["Hk"]) * case["rot"]}
    L = lifted(case["K"], case["pattern"], case["tier"])
    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        return {"bytes": M * (K * size[case["dtype"]] + L * (2 if case["tier"] == "bf16" else 1) + 4) + K * size[case["weight"]],
                "flops": 6 * M * K}
    M, N, sparse = case["M"], case["N"], case["sparse"]
    unit = {"int8": 1, "fp8": 1, "bf16": 2, "nvfp4": 0.5}[case["tier"]]
    half = lambda yes: L * unit / 2 + L / (16 if case["tier"] == "nvfp4" else 8) if yes else L * unit  # noqa: E731
    n = M * (N // 2 if case["gated"] else N)
    b = N * half(sparse == "w") + M * half(sparse == "x") + N * size[case["bias"]] + M * N * size[case["residual"]] + n * size[case["out"]]
    b += (M + N) * (L / (32 if sparse == "w" else 16) if case["tier"] == "nvfp4" else 0 if case["tier"] == "bf16" else 4)
    return {"bytes": b, "flops": M * N * L * (2 if sparse == "no" else 1)}
