"""The gated bf16 calls refuse reductions that one bounded wait cannot cover,
before any CUDA work (no GPU needed)."""
import ctypes

from precision_rl_rollout_nvfp4_b200 import binding as B

SHAPE = 3
MOST = 1 << 26                      # terms of a reduction: 2^20 steps of 64
lib = B.library_handle()
P = ctypes.c_void_p
X, G, U, H, D, WS = (P(0x1000 * i) for i in range(1, 7))    # aligned; nothing is read
HUGE = (1 << 62)                    # workspace bytes: never the reason


def forward(M=4, K=64, F=48):
    return lib.gated_linear_forward(X, M, K, K, G, U, F, K, 0, H, F, None, None)


def backward(M=4, K=64, F=48, dx=H, dg=G, du=U):
    return lib.gated_linear_backward(X, M, K, K, G, U, F, K, 0, D, F, P(0x9000), dx, K, dg, du, WS, HUGE, None)


def test_reductions_beyond_the_limit_are_refused():
    assert forward(K=MOST + 8) == SHAPE                                  # H: over K
    assert backward(K=MOST + 8) == SHAPE                                 # and computed again
    assert backward(F=MOST // 2 + 8, dg=None, du=None) == SHAPE          # dX: over F twice
    assert backward(M=MOST + 1, dx=None) == SHAPE                        # dW: over the tokens
    assert backward(M=MOST + 1, dx=None, du=None) == backward(M=MOST + 1, dx=None, dg=None) == SHAPE


def test_what_does_not_reduce_is_not_limited():
    """Past the shape checks: without tokens, or nothing asked for, the calls
    end there with nothing to do."""
    assert forward(M=0, K=MOST, F=MOST) == 0
    assert backward(M=MOST + 1, F=MOST // 2 + 8, dx=None, dg=None, du=None) == 0
    # refused for the missing output or workspace, not for the shape
    assert lib.gated_linear_forward(X, MOST + 1, 64, 64, G, U, 48, 64, 0, None, 48, None, None) == 1
    for dx, dg, M, F in ((H, None, MOST + 1, 48), (None, G, 4, MOST // 2 + 8), (H, G, MOST, MOST // 2)):
        assert lib.gated_linear_backward(X, M, 64, 64, G, U, F, 64, 0, D, F, P(0x9000), dx, 64, dg, None, None, 0,
                                         None) == 4
