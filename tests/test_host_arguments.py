"""The native host module converts its integer and truth arguments before
anything else, under the interpreter's lock, and passes on what the conversion
raises.  (No GPU: the tensors are refused right after.)"""
import pytest
import torch

from precision_rl_rollout_nvfp4_b200 import binding as B

X = torch.zeros(4, 64, dtype=torch.bfloat16)
Q = B.MxFP4Tensor(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 4, 64, 1)
# calls with one integer argument left open
INTS = {
    "quantize": lambda v: B._host.quantize(X, v, None, False),
    "dequantize": lambda v: B._host.dequantize(Q, v, None),
    "gemm": lambda v: B._host.gemm(Q, Q, v, None),
    "gated_gemm act": lambda v: B._host.gated_gemm(Q, Q, Q, v, 1, None),
    "gated_gemm dtype": lambda v: B._host.gated_gemm(Q, Q, Q, 0, v, None),
    "linear": lambda v: B._host.linear(X, Q, v, None),
    "mlp act": lambda v: B._host.mlp(X, Q, Q, Q, v, 1, None),
    "mlp dtype": lambda v: B._host.mlp(X, Q, Q, Q, 0, v, None),
    "gated_forward": lambda v: B._host.gated_forward(X, X, X, v, False),
    "gated_backward": lambda v: B._host.gated_backward(X, X, X, X, v, None, (True, True, True)),
    "gated_linear act": lambda v: B._host.gated_linear(X, X, X, v, False, 0, False, True),
    "gated_linear fmt": lambda v: B._host.gated_linear(X, X, X, 0, False, v, False, True),
}
TRUTHS = {
    "quantize": lambda v: B._host.quantize(X, 1, None, v),
    "gated_forward": lambda v: B._host.gated_forward(X, X, X, 0, v),
    "gated_backward": lambda v: B._host.gated_backward(X, X, X, X, 0, None, (True, v, True)),
    "gated_linear recompute": lambda v: B._host.gated_linear(X, X, X, 0, v, 0, False, True),
    "gated_linear act_quant": lambda v: B._host.gated_linear(X, X, X, 0, False, 0, v, True),
    "gated_linear grad": lambda v: B._host.gated_linear(X, X, X, 0, False, 0, False, v),
}


class Raises:
    def __index__(self):
        raise KeyError("index")

    def __bool__(self):
        raise KeyError("bool")


@pytest.mark.parametrize("call", INTS)
def test_integer_arguments(call):
    f = INTS[call]
    with pytest.raises(TypeError, match="integer"):
        f("silu")
    with pytest.raises(KeyError):
        f(Raises())
    for v in (1 << 40, -1 << 33, 1 << 80):
        with pytest.raises(OverflowError):
            f(v)
    with pytest.raises(ValueError, match="CUDA"):
        f(0)


@pytest.mark.parametrize("call", TRUTHS)
def test_truth_arguments(call):
    f = TRUTHS[call]
    with pytest.raises(KeyError):
        f(Raises())
    for v in (0, 1, True):
        with pytest.raises(ValueError, match="CUDA"):
            f(v)


def test_public_calls():
    with pytest.raises(TypeError):
        B.mxfp4_quantize(X, layout="1")
    with pytest.raises(ValueError, match="CUDA"):
        B.gated_linear_backward(X, X, X, X, need=[1, 0, True])
