"""Operands and 64-bit references for the tests of the fused epilogue, the
rotary positions and the fused norm.

Operands of the products are small integers (or E2M1 values with power-of-two
block scales), so every partial sum of a product is an fp32 value and the
accumulator is the same in any order: the dequantised fp32 value that enters
the epilogue is then known exactly, and the tolerances below are those of the
epilogue's own arithmetic."""
import numpy as np
import torch

import oracle

ULP = 2.0 ** -23   # spacing of fp32 just above 1; a rounding is off by half of it
# Activations this small may come out as 0: __fdividef returns 0 for
# denominators from 2^126 on, i.e. for 1 + e^t with t >= 126 ln 2 = 87.33; there
# |v| / (1 + e^t) <= |v| 2^-126, which is largest at silu's t = -v = 87.34:
# 87.34 * 2^-126 = 1.03e-36 (it falls with |v| from there on; gelu's |v| at t =
# 87.33 is below 11).  A gated output is that times the partner.
TINY = 88 * 2.0 ** -126


def _codes(x: np.ndarray, tier: str) -> torch.Tensor:
    t = torch.from_numpy(x.astype(np.float32))
    if tier == "int8":
        return t.to(torch.int8).view(torch.uint8)
    if tier == "fp8":
        return t.to(torch.float8_e4m3fn).view(torch.uint8)
    return t.to(torch.bfloat16)


def _nibbles(rng, rows, windows):
    pairs = np.array([4, 8, 12, 9, 13, 14], dtype=np.uint8)
    nib = pairs[rng.integers(0, 6, (rows, windows))]
    return nib, (nib[:, 0::2] | (nib[:, 1::2] << 4)).astype(np.uint8)


def operand(rng, rows, L, tier, sparse):
    """-> (stored values, metadata tiles or None, the matrix [rows, L] in 64 bits)."""
    if not sparse:
        x = rng.integers(-4, 5, (rows, L)).astype(np.float64)
        return _codes(x, tier), None, x
    v = rng.integers(-4, 5, (rows, L // 2)).astype(np.float64)
    nib, b = _nibbles(rng, rows, L // 4)
    x = np.zeros((rows, L // 4, 4))
    np.put_along_axis(x, np.stack((nib & 3, nib >> 2), -1).astype(np.int64),
                      v.reshape(rows, -1, 2), 2)
    meta = torch.from_numpy(oracle.meta_to_tiles(b, L, i16=tier == "bf16"))
    return _codes(v, tier), meta, x.reshape(rows, L)


def operand_fp4(rng, rows, L, sparse, block):
    """-> (stored codes, metadata tiles or None, scale tiles, matrix [rows, L])."""
    scale = np.array([0x30, 0x38, 0x40], dtype=np.uint8)  # UE4M3 0.5, 1, 2
    S = scale[rng.integers(0, 3, (rows, L // block))]
    tiles = torch.from_numpy(oracle.scales_to_tiles(S, L, block))
    if not sparse:
        v = rng.integers(0, 256, (rows, L // 2), dtype=np.uint8)
        return torch.from_numpy(v), None, tiles, oracle.decode_dense_nvfp4(v, S, L, block).astype(np.float64)
    v = rng.integers(0, 256, (rows, L // 4), dtype=np.uint8)
    _, b = _nibbles(rng, rows, L // 8)
    meta = torch.from_numpy(oracle.meta_to_tiles(b, L // 2))
    return torch.from_numpy(v), meta, tiles, oracle.decode_sparse_nvfp4(v, b, S, L).astype(np.float64)


def dequantised(x, w, s_x, s_w):
    """(float)acc * s_x in fp32 (the accumulator is exact), times s_w in 64 bits:
    v of the epilogue before the bias and the one rounding of their sum."""
    acc = (x @ w.T).astype(np.float32)
    if s_x is None:
        return acc.astype(np.float64)
    d = acc * np.asarray(s_x, np.float32).reshape(-1, 1)
    return d.astype(np.float64) * np.asarray(s_w, np.float32).astype(np.float64)


def activate(v, act):
    """act(v) in 64 bits, and a bound on the kernel's relative error against it
    for an fp32 v that is off by half a unit in the last place (units of 2^-23).

    2^x and 1/x are off by at most 2 units and 1 unit (their documented bounds),
    every product or sum by half.  silu: the exponent -v log2 e carries 1 unit
    of itself (its constant's rounding and the product's), i.e. |v| units in
    e^-v, and v's own half unit |v| / 2 more: 2 + 1.5 |v|, then 1/2 + 1 + 1/2:
    below 7 + 2 |v|.  gelu: the exponent u2 = 2 sqrt(2/pi) (v + 0.044715 v^3)
    carries 2.5 units (two constants, three operations), and v's half unit
    changes it by at most 3 |u2| / 2 units: below 8 + 5 |u2|.  gelu_erf: with
    u = |v|, Phi(-u) = e^(-u^2 / 2) t Q(t): 2.7 units for the polynomial in fp32,
    1 for the reciprocal t (the product t Q changes less than t does), 2 and
    1.5 u^2 / 2 for the power, 1.5 for the products, u^2 / 2 for v's half unit
    (and 1/2 in the factor v): 7.7 + 1.25 u^2, rounded up to 9 + 2 v^2; for v > 0
    it enters with a factor below 1."""
    if act == "relu":
        return np.where(v < 0, 0.0, v), np.full_like(v, ULP)
    if act == "silu":
        e = np.exp(np.minimum(-v, 700.0))
        return v / (1 + e), (7 + 2 * np.abs(v)) * ULP
    if act == "gelu":
        u2 = 2 * np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)
        return v / (1 + np.exp(np.minimum(-u2, 700.0))), (8 + 5 * np.abs(u2)) * ULP
    if act == "gelu_erf":
        phi = 0.5 * torch.special.erfc(torch.from_numpy(-v / np.sqrt(2.0))).numpy()
        return v * phi, (9 + 2 * v * v) * ULP
    return v, np.full_like(v, ULP / 2)


def half_step(out):
    return 2.0 ** -8 if out == torch.bfloat16 else 2.0 ** -24


def epilogue(d, bias, act, gated, residual, out):
    """(the epilogue of dequantised()'s d in 64 bits, bound on |Y - that|)."""
    v = d
    if bias is not None:
        v = v + bias.double().numpy()
    if gated:
        g = v.reshape(v.shape[0], -1, 2, 8)
        y, rel = activate(g[:, :, 0], act)
        y = (y * g[:, :, 1]).reshape(v.shape[0], -1)
        tiny = TINY * (1 + np.abs(g[:, :, 1]).reshape(y.shape))
        rel = rel.reshape(y.shape) + 1.5 * ULP  # the partner's rounding and the product's
    else:
        y, rel = activate(v, act)
        tiny = TINY
    off = np.abs(y) * rel
    if residual is not None:
        y = y + residual.double().numpy()
        off = off + np.abs(y) * ULP
    return y, off * 1.01 + np.abs(y) * half_step(out) * 1.01 + tiny


def assert_within(got: torch.Tensor, want: np.ndarray, bound: np.ndarray):
    g = got.detach().cpu().double().numpy()
    assert g.shape == want.shape
    bad = ~(np.abs(g - want) <= bound)
    if bad.any():
        at = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{bad.sum()} of {bad.size} off; first at {at}: {g[at]} against "
                             f"{want[at]}, allowed {bound[at]}")


def rope(x, pos, freqs, layout, scale):
    """(rotated x in 64 bits, bound for an fp32 computation rounded to x's type).

    cos and sin: the angle in turns is off by 2^-26 (its fraction rounded to
    fp32) plus |turns| 2^-52 (products in 64 bits), sincospif by 1 unit, the
    scale's product by half: at most 2^-22 + 2 pi |turns| 2^-51.  Two products and a
    sum add 3 half units of |a| + |b|."""
    x64, r = x.double().cpu().numpy(), 2 * len(freqs)
    ang = pos.double().cpu().numpy()[:, None] * freqs[None]
    c, s = scale * np.cos(ang)[:, None], scale * np.sin(ang)[:, None]
    a, b = (x64[..., :r // 2], x64[..., r // 2:r]) if layout == "half" else \
        (x64[..., 0:r:2], x64[..., 1:r:2])
    y, off = x64.copy(), np.zeros_like(x64)
    one = (np.abs(a) + np.abs(b)) * abs(scale) * \
        (3 * 2.0 ** -23 + np.abs(ang)[:, None] * 2.0 ** -51)
    at = (slice(0, r // 2), slice(r // 2, r)) if layout == "half" else \
        (slice(0, r, 2), slice(1, r, 2))
    for where, v in zip(at, (a * c - b * s, b * c + a * s)):
        y[..., where] = v
        off[..., where] = one + np.abs(v) * half_step(x.dtype) * 1.01 + TINY
    return y, off


def lift(v, pattern):
    """[M, K] in the lifted order, zero padded to K_lp."""
    M, K = v.shape
    _, _, K_lp = oracle.slide_shape(pattern, K)
    out = np.zeros((M, K_lp))
    if pattern in ("dense", "2:4"):
        out[:, :K] = v
        return out
    nh = int(pattern.split(":")[1]) // 2
    G = -(-K // (2 * nh))
    g = np.pad(v, ((0, 0), (0, G * 2 * nh - K))).reshape(M, G, 2 * nh)
    w = np.concatenate([g[:, :, 2 * j:2 * j + 4] for j in range(nh - 1)], 2).reshape(M, -1)
    out[:, :w.shape[1]] = w
    return out
