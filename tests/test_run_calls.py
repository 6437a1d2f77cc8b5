"""run_calls makes the inputs of the MXFP4 and gated calls only where one of
them is asked for, and of those only what the asked ones take (no GPU needed:
the library's calls are recorded, not made)."""
from types import SimpleNamespace

import torch

from precision_rl_rollout_nvfp4_b200 import run_calls as R
from precision_rl_rollout_nvfp4_b200 import synthetic as S


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def f(*args, **kw):
            self.calls.append((name, [tuple(t.shape) for t in args if isinstance(t, torch.Tensor)]))
            return name, name
        return f


def ask(names, M=8, K=64, N=96):
    b = Recorder()
    a = SimpleNamespace(M=M, K=K, N=N, y_dtype="fp32")
    return b, R.block_calls(b, S, a, torch.device("cpu"), names)


def test_steps_of_the_plan_make_nothing():
    b, block = ask(["prepare_weight", "quantize", "gemm"], N=1001)
    assert block == {} and b.calls == []


def test_each_call_makes_only_its_operands():
    # N = 1001 cannot be a reduction of an MXFP4 product: only the block's down projection has it as one
    for name in R.BLOCK_CALLS:
        b, block = ask([name, "gemm"], N=1001)
        assert list(block) == [name]
        quantized = [shape for n, (shape, *_) in b.calls if n == "mxfp4_quantize"]
        assert ((64, 1001) in quantized) == (name == "mxfp4_gated_mlp")
        assert ((8, 64) in quantized) == (name in ("mxfp4_dequantize", "mxfp4_gemm", "mxfp4_gated_gemm"))
        b.calls.clear()
        block[name]()
        assert len(b.calls) == 1


def test_backward_takes_what_the_forward_call_kept():
    b, block = ask(["gated_forward", "gated_backward"])
    b.calls.clear()
    block["gated_forward"]()
    block["gated_backward"]()
    assert [n for n, _ in b.calls] == ["gated_linear_forward", "gated_linear_backward"]
