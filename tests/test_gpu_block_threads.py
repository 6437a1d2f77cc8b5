"""Host threads that share a stream, or run side by side on their own: the MXFP4
and gated calls see each buffer as stream order has it, whole."""
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

from tests.gpu_common import need_gpu

pytestmark = pytest.mark.gpu


def weight(N, K, seed, scale=0.05):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(N, K, generator=g)).to(torch.bfloat16).cuda()


def rows(M, K, seed):
    return weight(M, K, seed, 1.0)


def together(*work):
    """Runs the functions in one thread each; an exception in any is raised here."""
    with ThreadPoolExecutor(len(work)) as pool:
        for f in [pool.submit(w) for w in work]:
            f.result()


def ok(b):
    torch.cuda.synchronize()
    assert b.stream_status() == 0


def match(got, refs):
    return [i for i, r in enumerate(refs) if torch.equal(got, r)]


@pytest.mark.parametrize("M", [3, 40, 300])
def test_weight_requantized_by_another_thread_on_the_same_stream(M):
    """Every product reads one quantization of the weight or the other, never a
    mixture: the two are queued on one stream, in whatever order."""
    b = need_gpu()
    K, N = 2048, 4096
    x, ws = rows(M, K, M), [weight(N, K, 1), weight(N, K, 2)]
    refs = [b.mxfp4_linear(x, b.mxfp4_quantize(w)) for w in ws]
    qw = b.mxfp4_quantize(ws[0])
    torch.cuda.synchronize()
    got, n = [], 300

    def multiply():
        got.extend(b.mxfp4_linear(x, qw) for _ in range(n))

    def refresh():
        for i in range(n):
            b.mxfp4_quantize(ws[(i + 1) % 2], out=qw)

    together(multiply, refresh)
    ok(b)
    assert len(got) == n and all(match(y, refs) for y in got)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_block_beside_a_thread_that_refreshes_its_weights(M):
    b = need_gpu()
    K, F = 512, 2048
    x = rows(M, K, M)
    sets = [[weight(F, K, s), weight(F, K, s + 1), weight(K, F, s + 2)] for s in (1, 11)]
    qs = [[b.mxfp4_quantize(w) for w in s] for s in sets]
    # each weight is refreshed by a call of its own: any of the eight combinations
    refs = [b.mxfp4_gated_mlp(x, qs[i][0], qs[j][1], qs[k][2]) for i in (0, 1) for j in (0, 1) for k in (0, 1)]
    kept = [b.mxfp4_quantize(w) for w in sets[0]]
    torch.cuda.synchronize()
    got, n = [], 200

    def block():
        got.extend(b.mxfp4_gated_mlp(x, *kept) for _ in range(n))

    def refresh():
        for i in range(n):
            for w, q in zip(sets[(i + 1) % 2], kept):
                b.mxfp4_quantize(w, out=q)

    together(block, refresh)
    ok(b)
    assert len(got) == n and all(match(y, refs) for y in got)


def test_weight_gradients_beside_a_thread_that_refills_the_activations():
    """dW reads X where its launch stands in the stream: all old or all new."""
    b = need_gpu()
    M, K, F = 600, 512, 1024
    qx = [b.mxfp4_quantize(rows(M, K, s)) for s in (1, 2)]
    xs = [b.mxfp4_dequantize(q) for q in qx]
    wg, wu, dh = weight(F, K, 3), weight(F, K, 4), rows(M, F, 5)
    x = xs[0].clone()
    _, saved = b.gated_linear_forward(x, wg, wu, save=True)
    # (with the projections given, X enters the weights' gradients alone)
    refs = [b.gated_linear_backward(v, wg, wu, dh, saved=saved) for v in xs]
    torch.cuda.synchronize()
    got, n = [], 100

    def backward():
        got.extend(b.gated_linear_backward(x, wg, wu, dh, saved=saved) for _ in range(n))

    def refill():
        for i in range(2 * n):
            b.mxfp4_dequantize(qx[(i + 1) % 2], out=x)

    together(backward, refill)
    ok(b)
    assert len(got) == n and torch.equal(refs[0][0], refs[1][0])
    for dx, dg, du in got:
        assert torch.equal(dx, refs[0][0])
        assert set(match(dg, [r[1] for r in refs])) & set(match(du, [r[2] for r in refs]))


def test_threads_on_streams_of_their_own():
    """Calls and backward passes from several threads at once, each on its own
    stream; every pass of every thread is counted."""
    b = need_gpu()
    n, work = 20, []
    for M in (40, 300, 1):
        x, wg, wu, dh = rows(M, 96, M), weight(96, 96, 1, 0.3), weight(96, 96, 2, 0.3), rows(M, 96, M + 1)
        leaves = [t.requires_grad_(True) for t in (x, wg, wu)]
        want = torch.autograd.grad(b.gated_linear(*leaves), leaves, dh)
        qs = [b.mxfp4_quantize(t.detach()) for t in (wg, wu, wg)]
        work.append(([x, wg, wu, dh], want, qs, b.mxfp4_gated_mlp(x.detach(), *qs)))
    torch.cuda.synchronize()
    done = [0] * len(work)

    def run(i):
        (*ops, dh), want, qs, y = work[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(n):
                leaves = [t.detach().clone().requires_grad_(True) for t in ops]
                got = torch.autograd.grad(b.gated_linear(*leaves), leaves, dh)
                z = b.mxfp4_gated_mlp(leaves[0].detach(), *qs)
                torch.cuda.current_stream().synchronize()
                assert all(torch.equal(p, q) for p, q in zip(got, want)) and torch.equal(z, y)
                done[i] += 1

    together(*[lambda i=i: run(i) for i in range(len(work))])
    ok(b)
    assert done == [n] * len(work)
