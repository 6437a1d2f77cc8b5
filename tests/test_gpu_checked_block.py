"""The MXFP4 and gated calls in the index-checked build (compiled with
NVFP4_CHECKS): every store and gathered load compares its offset with its
buffer's end, and a failure makes the stream's status an error.  The checks
against the oracle run on small and ragged shapes of every kernel variant, in a
child process (one library per process); each ends by asking for the status."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import torch
from precision_rl_rollout_nvfp4_b200 import binding as b
from tests import test_gpu_gated as G, test_gpu_mx4 as T
assert b._lib.nvfp4_build_flags() & 1, "not the checked build"
for layout in (0, 1):
    for M, K in [(1, 32), (2, 160), (129, 2080), (257, 1056)]:
        T.test_quantize_matches_oracle(M, K, layout)
for cut in ("wide", "offset", "transposed", "expanded", "3d"):
    T.test_quantize_strides(cut)
# few tokens (quantized in the product up to 8), 16, 32 and 64 token tiles, split over K, CTA pairs
for dt in (torch.float32, torch.bfloat16):
    for M, K, N in [(1, 32, 1), (3, 96, 7), (4, 2080, 130), (16, 288, 128), (17, 256, 33), (33, 160, 64), (100, 544, 1001),
                    (300, 1504, 1001), (2600, 352, 2600)]:
        T.test_gemm_matches_oracle(M, K, N, dt)
T.test_gemm_split_over_k(13, 8992, 5300)
T.test_gemm_split_over_k(64, 2048, 600)
for left in (2, 3, 8):
    for M, K, N in [(20, 64, 33), (50, 64, 34), (300, 64, 1030)]:
        T.test_out_keeps_what_lies_between_and_behind_its_rows(M, K, N, left)
for kind in ("silu", "gelu_tanh"):
    # F % 32 == 0 also with an MXFP4 output
    for M, K, F in [(1, 32, 32), (3, 96, 8), (17, 256, 160), (33, 160, 64), (65, 96, 128), (130, 544, 1001), (300, 1504, 992),
                    (32, 2304, 1024), (2100, 320, 1312)]:
        T.test_gated_matches_oracle(M, K, F, kind)
    T.test_mlp_is_its_parts(150, 320, 256, 320, kind)
    for M, K, F in [(1, 8, 8), (7, 72, 40), (65, 520, 136), (300, 1032, 520), (1300, 1400, 2600)]:
        G.test_forward_and_backward_match_oracle(M, K, F, kind)
for need in [(True, False, False), (False, True, False), (False, False, True), (False, True, True)]:
    G.test_only_the_gradients_asked_for(need)
G.test_strides_and_no_tokens()
torch.cuda.synchronize()
assert b.stream_status() == 0
print("checked build ok")
'''


def test_block_in_checked_build():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lib = os.path.join(ROOT, "precision_rl_rollout_nvfp4_b200", "libnvfp4rac_checked.so")
    assert os.path.exists(lib), "build the checked library (build_lib.build(checked=True))"
    env = dict(os.environ, NVFP4_LIB="checked", PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, capture_output=True, text=True,
                       timeout=900)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "checked build ok" in r.stdout
