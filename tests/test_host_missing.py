"""Without the native host module the ctypes calls import and run; each call
that needs it raises an ImportError that says what to build."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import sys
sys.modules["precision_rl_rollout_nvfp4_b200._host"] = None        # its import raises
import torch
from precision_rl_rollout_nvfp4_b200 import binding as B
assert B.workspace_size(B.OP_QUANTIZE, 64, 0, 64) > 0 and B.rac_nsel(50.0, 64) == 32
assert B.mxfp4_scale_bytes(64, 512, 0) == 1024
assert B.MxFP4Tensor.empty(4, 64, device="cpu").codes.shape == (4, 32)
x = torch.zeros(4, 64, dtype=torch.bfloat16)
q = B.MxFP4Tensor.empty(4, 64, device="cpu")
calls = [lambda: B.mxfp4_quantize(x), lambda: B.mxfp4_qdq(x), lambda: B.mxfp4_dequantize(q), lambda: B.mxfp4_gemm(q, q),
         lambda: B.mxfp4_gated_gemm(q, q, q), lambda: B.mxfp4_linear(x, q), lambda: B.mxfp4_gated_mlp(x, q, q, q),
         lambda: B.gated_linear_forward(x, x, x), lambda: B.gated_linear_backward(x, x, x, x),
         lambda: B.gated_linear(x, x, x), lambda: B.qat_gated_linear(x, x, x), lambda: B.fake_quant(x, "mxfp4")]
for f in calls:
    try:
        f()
    except ImportError as e:
        assert "build_lib" in str(e) and e.__cause__ is not None
    else:
        raise AssertionError("no error")
print("done")
'''


def test_binding_without_the_host_module():
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=dict(os.environ, PYTHONPATH=ROOT),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, r.stderr[-3000:]
