"""Edges of the MXFP4 and gated calls: infinities, NaN and overflow through every
kernel, outputs inside wider buffers, decode batches, results that repeat.

Tolerances of the decode batches as in the oracle tests of these calls (derived
there), with the 64-bit products formed on the GPU."""
import math

import numpy as np
import pytest
import torch

from oracle import mxfp4 as mx
from tests.gpu_common import need_gpu
from tests.layout import unpack_codes

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -23
NAN, INF = float("nan"), float("inf")


def bf16(M, K, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(M, K, generator=g)).to(torch.bfloat16)


def ok(b):
    torch.cuda.synchronize()
    assert b.stream_status() == 0


def lines(M, N, rows=(), cols=()):
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[list(rows)] = True
    bad[:, list(cols)] = True
    return bad


# ---- infinities and NaN ----------------------------------------------------------
@pytest.mark.parametrize("M", [2, 4, 8, 9, 16, 40, 600])
def test_nonfinite_through_the_linear(M):
    """Tokens quantized in the product, few-token tiles, CTA pairs."""
    b = need_gpu()
    x, w = bf16(M, 2048, M), bf16(300, 2048, 1)
    x[1, 2047], w[299, 0] = -INF, NAN
    qw = b.mxfp4_quantize(w.cuda())
    for dt in (torch.float32, torch.bfloat16):
        y = b.mxfp4_linear(x.cuda(), qw, dt)
        ok(b)
        assert torch.equal(torch.isnan(y.cpu()), lines(M, 300, [1], [299]))


@pytest.mark.parametrize("M,K,F", [(3, 256, 160), (20, 2048, 1024), (50, 256, 160), (300, 256, 160), (700, 320, 2080)])
@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_nonfinite_through_the_gated_product(M, K, F, kind):
    b = need_gpu()
    x, wg, wu = bf16(M, K, M), bf16(F, K, 1, 0.05), bf16(F, K, 2)
    x[1, 200], x[M - 1, 0], wg[5, 7], wu[70, 3] = INF, NAN, -INF, NAN
    qx, qg, qu = (b.mxfp4_quantize(t.cuda()) for t in (x, wg, wu))
    y = b.mxfp4_gated_gemm(qx, qg, qu, act=kind, out_dtype=torch.float32)
    y16 = b.mxfp4_gated_gemm(qx, qg, qu, act=kind)
    q = b.mxfp4_gated_gemm(qx, qg, qu, act=kind, out_dtype="mxfp4")
    ok(b)
    bad = lines(M, F, [1, M - 1], [5, 70])
    assert torch.equal(torch.isnan(y.cpu()), bad) and torch.equal(torch.isnan(y16.cpu()), bad)
    assert torch.isfinite(y.cpu()[~bad]).all()
    # a block with a NaN: scale 255, codes 0; the others as ever
    codes, scales = mx.quantize(y.cpu().numpy())
    got = q.scales.cpu().numpy()[mx.tiled_index(M, F)]
    assert np.array_equal(got, scales) and np.array_equal(unpack_codes(q.codes.cpu().numpy()), codes)
    assert (got == 255).any() and (got != 255).any()


@pytest.mark.parametrize("M", [1, 3, 20, 50, 300])
def test_overflow_in_the_gated_product(M):
    """Projections beyond fp32 make infinite values, and those a NaN block of the
    quantized form; the other rows stay finite."""
    b = need_gpu()
    K, F = 256, 96
    x, wg, wu = bf16(M, K, M), bf16(F, K, 1).abs() + 1, bf16(F, K, 2).abs() + 1
    x[0] = 3e38
    qx, qg, qu = (b.mxfp4_quantize(t.cuda()) for t in (x, wg, wu))
    y = b.mxfp4_gated_gemm(qx, qg, qu, out_dtype=torch.float32)
    q = b.mxfp4_gated_gemm(qx, qg, qu, out_dtype="mxfp4")
    ok(b)
    assert torch.equal(torch.isfinite(y.cpu()), ~lines(M, F, [0]))
    codes, scales = mx.quantize(y.cpu().numpy())
    got = q.scales.cpu().numpy()[mx.tiled_index(M, F)]
    assert (got[0] == 255).all() and np.array_equal(got, scales)
    assert np.array_equal(unpack_codes(q.codes.cpu().numpy()), codes)


@pytest.mark.parametrize("M", [1, 20, 50, 300])
def test_nonfinite_through_the_block(M):
    b = need_gpu()
    K, F, N = 256, 320, 130
    x, wg, wu, wd = bf16(M, K, M), bf16(F, K, 1, 0.05), bf16(F, K, 2), bf16(N, F, 3)
    x[M - 1, 31], wd[129, 319] = NAN, INF
    y = b.mxfp4_gated_mlp(x.cuda(), *(b.mxfp4_quantize(w.cuda()) for w in (wg, wu, wd)))
    ok(b)
    assert torch.equal(torch.isnan(y.cpu()), lines(M, N, [M - 1], [129]))


@pytest.mark.parametrize("M,K,F", [(40, 64, 72), (300, 136, 264)])
@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_nonfinite_through_the_bf16_gated_projection(M, K, F, kind):
    """A bad token makes its rows of H and dX NaN or infinite, and (as every
    weight meets it) all of dW; a bad gradient its token's dX and its row of dW."""
    b = need_gpu()
    x, wg, wu, dh = (t.cuda() for t in (bf16(M, K, M), bf16(F, K, 1, 0.2), bf16(F, K, 2, 0.2), bf16(M, F, 3)))
    h0, saved0 = b.gated_linear_forward(x, wg, wu, kind, save=True)
    g0 = b.gated_linear_backward(x, wg, wu, dh, kind, saved0)
    for v in (NAN, INF, -INF):
        xb = x.clone()
        xb[7, 3] = v
        h, saved = b.gated_linear_forward(xb, wg, wu, kind, save=True)
        dx, dwg, dwu = b.gated_linear_backward(xb, wg, wu, dh, kind, saved)
        ok(b)
        keep = torch.arange(M, device="cuda") != 7
        assert not torch.isfinite(h[7]).any() and torch.equal(h[keep], h0[keep])
        assert not torch.isfinite(dx[7]).any() and torch.equal(dx[keep], g0[0][keep])
        assert not torch.isfinite(dwu[:, 3]).any() and not torch.isfinite(dwg[:, 3]).any()
    db = dh.clone()
    db[9, 5] = NAN
    dx, dwg, dwu = b.gated_linear_backward(x, wg, wu, db, kind, saved0)
    ok(b)
    assert torch.isnan(dx[9]).all() and torch.equal(torch.isnan(dx).any(1), torch.arange(M, device="cuda") == 9)
    for d, ref in ((dwg, g0[1]), (dwu, g0[2])):
        keep = torch.arange(F, device="cuda") != 5
        assert torch.isnan(d[5]).all() and torch.equal(d[keep], ref[keep])


# ---- outputs inside wider buffers ---------------------------------------------------
@pytest.mark.parametrize("M,K,F", [(3, 96, 130), (20, 64, 33), (50, 64, 34), (300, 64, 1030), (700, 96, 2001)])
@pytest.mark.parametrize("left", [2, 3, 8])
def test_gated_output_inside_a_wider_buffer(M, K, F, left):
    b = need_gpu()
    qx, qg, qu = (b.mxfp4_quantize(t.cuda()) for t in (bf16(M, K, 1), bf16(F, K, 2, 0.05), bf16(F, K, 3)))
    for dt in (torch.bfloat16, torch.float32):
        ref = b.mxfp4_gated_gemm(qx, qg, qu, out_dtype=dt)
        for pad in (7, 8):
            wide = torch.full((M + 4, left + F + pad), 5.0, dtype=dt, device="cuda")
            b.mxfp4_gated_gemm(qx, qg, qu, out_dtype=dt, out=wide[:M, left:left + F])
            ok(b)
            assert torch.equal(wide[:M, left:left + F], ref)
            assert (wide[M:] == 5).all() and (wide[:, :left] == 5).all() and (wide[:, left + F:] == 5).all()


@pytest.mark.parametrize("M", [1, 40, 300])
def test_block_and_codes_inside_larger_buffers(M):
    """The block's output in a wider buffer; quantized outputs in buffers of more
    rows: what lies behind stays."""
    b = need_gpu()
    K, F, N = 128, 160, 96
    x = bf16(M, K, M).cuda()
    qg, qu, qd = (b.mxfp4_quantize(t.cuda()) for t in (bf16(F, K, 1, 0.05), bf16(F, K, 2), bf16(N, F, 3)))
    ref = b.mxfp4_gated_mlp(x, qg, qu, qd)
    wide = torch.full((M + 2, N + 9), 5.0, dtype=torch.bfloat16, device="cuda")
    b.mxfp4_gated_mlp(x, qg, qu, qd, out=wide[:M, 3:3 + N])
    ok(b)
    assert torch.equal(wide[:M, 3:3 + N], ref) and (wide[M:] == 5).all()
    assert (wide[:, :3] == 5).all() and (wide[:, 3 + N:] == 5).all()
    qx = b.mxfp4_quantize(x)
    h = b.mxfp4_gated_gemm(qx, qg, qu, out_dtype="mxfp4")
    big = b.MxFP4Tensor(torch.full((M + 4, F // 2), 77, dtype=torch.uint8, device="cuda"),
                        torch.full((h.scales.numel() + 512,), 77, dtype=torch.uint8, device="cuda"), M, F, 1)
    b.mxfp4_gated_gemm(qx, qg, qu, out_dtype="mxfp4", out=big)
    ok(b)
    assert torch.equal(big.codes[:M], h.codes) and (big.codes[M:] == 77).all()
    assert torch.equal(big.scales[:h.scales.numel()], h.scales) and (big.scales[h.scales.numel():] == 77).all()


# ---- decode batches -------------------------------------------------------------------
def act64(g, kind):
    if kind == "silu":
        return g * torch.sigmoid(g), g
    w = 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    return g * torch.sigmoid(w), w


@pytest.mark.parametrize("M", [16, 64, 100, 128, 200, 256])
@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_decode_batch_through_the_block(M, kind):
    b = need_gpu()
    K, F = 4096, 11008
    x = bf16(M, K, M).cuda()
    qg, qu, qd = (b.mxfp4_quantize(t.cuda()) for t in (bf16(F, K, 1, 0.02), bf16(F, K, 2, 0.02), bf16(K, F, 3, 0.02)))
    qx = b.mxfp4_quantize(x)
    xv, gv, uv = (b.mxfp4_dequantize(q, torch.float32).double() for q in (qx, qg, qu))

    def product(a, w):
        return a @ w.t(), (2 * (a.shape[1] // 64) + 17) * F32 * (a.abs() @ w.abs().t())

    (g, tg), (u, tu) = product(xv, gv), product(xv, uv)
    a, w = act64(g, kind)
    ta = 1.2 * tg + (8 + 6 * w.abs().clamp(max=90)) * F32 * a.abs() + 1e-35
    h, tol = a * u, ta * u.abs() + a.abs() * tu + ta * tu
    y = b.mxfp4_gated_gemm(qx, qg, qu, act=kind, out_dtype=torch.float32)
    assert ((y.double() - h).abs() <= tol + 3 * F32 * h.abs()).all()
    q = b.mxfp4_gated_gemm(qx, qg, qu, act=kind, out_dtype="mxfp4")
    # the quantized form is that of the same fp32 values
    codes, scales = mx.quantize(y.cpu().numpy())
    assert np.array_equal(q.scales.cpu().numpy()[mx.tiled_index(M, F)], scales)
    assert np.array_equal(unpack_codes(q.codes.cpu().numpy()), codes)
    # the down projection reduces over 11008
    d, td = product(b.mxfp4_dequantize(q, torch.float32).double(), b.mxfp4_dequantize(qd, torch.float32).double())
    z = b.mxfp4_gated_mlp(x, qg, qu, qd, act=kind, out_dtype=torch.float32)
    ok(b)
    assert ((z.double() - d).abs() <= td + F32 * d.abs()).all()
    assert torch.equal(b.mxfp4_gated_mlp(x, qg, qu, qd, act=kind), z.to(torch.bfloat16))


# ---- results that repeat ----------------------------------------------------------------
@pytest.mark.parametrize("M", [1, 7, 64, 300, 777])
def test_results_repeat_bit_for_bit(M):
    """Sums split over CTAs are added in a fixed order; nothing is accumulated by
    atomics, forward or backward."""
    b = need_gpu()
    K, F = 2048, 1024
    x, wg, wu, dh = bf16(M, K, 1), bf16(F, K, 2, 0.02), bf16(F, K, 3, 0.02), bf16(M, F, 4)
    wd = bf16(K, F, 5, 0.02)
    leaves = [t.cuda().requires_grad_(True) for t in (x, wg, wu)]
    q = [b.mxfp4_quantize(t.cuda()) for t in (wg, wu, wd)]

    def once():
        h = b.qat_gated_linear(*leaves, fmt="mxfp4")
        y = b.mxfp4_gated_mlp(leaves[0].detach(), *q)
        return (h.detach(), *torch.autograd.grad(h, leaves, dh.cuda()), y, b.mxfp4_linear(y, q[0], torch.float32))

    first = once()
    for _ in range(10):
        junk = torch.full((1 << 22,), NAN, device="cuda")           # (what freed buffers are handed on with)
        del junk
        assert all(torch.equal(p, r) for p, r in zip(once(), first))
    ok(b)


# ---- outputs over the inputs, and far offsets -----------------------------------------------
@pytest.mark.parametrize("M", [1, 2, 4, 5, 8, 9, 40, 300])
def test_output_over_the_input(M):
    """The linear and the block read all of x before they write y."""
    b = need_gpu()
    K, F = 2048, 512
    x = bf16(M, K, M).cuda()
    qw = b.mxfp4_quantize(bf16(K, K, 1, 0.02).cuda())
    block = [b.mxfp4_quantize(t.cuda()) for t in (bf16(F, K, 2, 0.02), bf16(F, K, 3, 0.02), bf16(K, F, 4, 0.02))]
    ref, ref_block = b.mxfp4_linear(x, qw), b.mxfp4_gated_mlp(x, *block)
    for _ in range(20):
        for f, want in ((lambda t: b.mxfp4_linear(t, qw, out=t), ref),
                        (lambda t: b.mxfp4_gated_mlp(t, *block, out=t), ref_block)):
            y = x.clone()
            f(y)
            assert torch.equal(y, want)
    # y starts inside x's rows
    buf = torch.zeros(M, K + 64, dtype=torch.bfloat16, device="cuda")
    buf[:, :K] = x
    b.mxfp4_linear(buf[:, :K], qw, out=buf[:, 64:])
    ok(b)
    assert torch.equal(buf[:, 64:], ref)


def test_gated_projection_beyond_32_bit_offsets():
    """More than 2^31 outputs: the last tokens' results are those of a call of
    their own; the tokens before them are zero and add nothing to dW."""
    b = need_gpu()
    K, F, n = 16, 8192, 300
    M = 64 * 4219 + n                              # (the last tokens start on a step of the reduction)
    x, wg, wu, dh = (t.cuda() for t in (bf16(n, K, 1), bf16(F, K, 2), bf16(F, K, 3), bf16(n, F, 4)))
    xs, ds = (torch.zeros(M, c, dtype=torch.bfloat16, device="cuda") for c in (K, F))
    xs[-n:], ds[-n:] = x, dh
    h, saved = b.gated_linear_forward(xs, wg, wu, save=True)
    few, few_saved = b.gated_linear_forward(x, wg, wu, save=True)
    assert M * F > 1 << 31 and torch.equal(h[-n:], few) and not h[:-n].any()
    del h
    got = b.gated_linear_backward(xs, wg, wu, ds, saved=saved)
    want = b.gated_linear_backward(x, wg, wu, dh, saved=few_saved)
    ok(b)
    assert torch.equal(got[0][-n:], want[0]) and not got[0][:-n].any()
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])


@pytest.mark.parametrize("M", range(1, 18))
@pytest.mark.parametrize("K,N", [(32, 40), (288, 130), (2080, 300), (8224, 260)])
def test_few_tokens_quantized_in_the_product_or_before_it(M, K, N):
    """The linear is its parts bit for bit on both sides of the rule, from rows of
    a wider buffer too."""
    b = need_gpu()
    wide = bf16(M, K + 24, M).cuda()
    qw = b.mxfp4_quantize(bf16(N, K, 1, 0.05).cuda())
    for x in (wide[:, :K].contiguous(), wide[:, 8:8 + K]):
        for dt in (torch.float32, torch.bfloat16):
            assert torch.equal(b.mxfp4_linear(x, qw, dt), b.mxfp4_gemm(b.mxfp4_quantize(x), qw, dt))
    ok(b)
