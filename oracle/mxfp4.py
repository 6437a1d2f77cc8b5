"""MXFP4: E2M1 elements with one power-of-two (UE8M0) scale per 32 elements,
and the gated feed-forward block on such operands.

Test infrastructure: see the package header in ``oracle/__init__.py``.

Per block of 32 consecutive elements along K (the OCP microscaling definition,
with the conversion saturating like the other formats here):

    E      = floor(log2(amax_b)) - 2            (2 = exponent of E2M1's 6),
             clamped to [-127, 127]; E = -127 for an all-zero block
    scale  = UE8M0 code E + 127; 255 (NaN) for a block with an infinity or a
             NaN, whose codes are 0
    code   = E2M1 of x / 2^E, nearest, ties to the even code, saturating at 6
    DQ     = E2M1dec(code) * 2^E                (exact)

Products are fp64 sums of the exact block values.  The gated projection is
H = act(X Wg^T) * (X Wu^T) with act(g) = g s(g) (silu) or
g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2 (gelu_tanh); its gradients for
an upstream dH are dG = dH U act'(G), dU = dH act(G), dX = dG Wg + dU Wu,
dWg = dG^T X, dWu = dU^T X.
"""
from __future__ import annotations

import numpy as np

from .formats import e2m1_decode, e2m1_encode

MX_BLOCK = 32
E2M1_EMAX = 2            # 6 = 1.5 * 2^2
UE8M0_BIAS = 127
UE8M0_NAN = 255


def quantize(x):
    """MXFP4 of fp32 x [R, C]: (codes uint8 [R, C], one per element; scales
    uint8 [R, C/32])."""
    x = np.asarray(x, np.float32)
    R, C = x.shape
    if C % MX_BLOCK:
        raise ValueError("row length must be a multiple of 32")
    b = x.reshape(R, C // MX_BLOCK, MX_BLOCK)
    bad = ~np.isfinite(b).all(axis=2)
    b64 = np.where(bad[:, :, None], 0.0, b).astype(np.float64)
    amax = np.abs(b64).max(axis=2)
    e = np.full(amax.shape, -UE8M0_BIAS, np.int64)
    nz = amax > 0
    e[nz] = np.frexp(amax[nz])[1] - 1 - E2M1_EMAX
    e = np.clip(e, -UE8M0_BIAS, UE8M0_BIAS)
    q = np.ldexp(b64, -e[:, :, None])                      # exact
    codes = np.where(bad[:, :, None], np.uint8(0), e2m1_encode(q)).astype(np.uint8)
    return codes.reshape(R, C), np.where(bad, UE8M0_NAN, e + UE8M0_BIAS).astype(np.uint8)


def dequantize(codes, scales):
    """E2M1dec(code) * 2^(scale - 127) per element, float64 (exact); NaN for scale 255."""
    codes, scales = np.asarray(codes, np.uint8), np.asarray(scales, np.uint8)
    s = np.where(scales == UE8M0_NAN, np.nan, np.ldexp(1.0, scales.astype(np.int64) - UE8M0_BIAS))
    return e2m1_decode(codes) * np.repeat(s, MX_BLOCK, axis=1)


def qdq(x):
    return dequantize(*quantize(x))


def tiled_index(rows, cols):
    """Byte offset of every (row, block) scale in the MMA-tiled layout."""
    r = np.arange(rows, dtype=np.int64)[:, None]
    c = np.arange(cols // MX_BLOCK, dtype=np.int64)[None, :]
    return ((r >> 7) * -(-cols // 128) + (c >> 2)) * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4 + (c & 3)


def logistic(w):
    """1 / (1 + e^-w) in fp64, to a few units of the last place on both sides."""
    e = np.exp(-np.abs(w))
    return np.where(w >= 0, 1 / (1 + e), e / (1 + e))


def act(g, kind):
    """(act(g), act'(g)) in fp64.  (1 + tanh z) / 2 is the logistic function of
    2 z, which does not cancel at negative z."""
    g = np.asarray(g, np.float64)
    if kind == "silu":
        s = logistic(g)
        return g * s, s + g * s * (1 - s)
    c = 2 * np.sqrt(2 / np.pi)
    s = logistic(c * (g + 0.044715 * g ** 3))
    return g * s, s + g * s * (1 - s) * c * (1 + 3 * 0.044715 * g * g)


def gated(x, wg, wu, kind, dh=None):
    """H, and with dh the gradients (dx, dwg, dwu), of fp64 operands."""
    g, u = x @ wg.T, x @ wu.T
    a, da = act(g, kind)
    if dh is None:
        return a * u
    dg, du = dh * u * da, dh * a
    return a * u, (dg @ wg + du @ wu, dg.T @ x, du.T @ x)
