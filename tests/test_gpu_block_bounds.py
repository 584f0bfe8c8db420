"""The operators around the convolution on the index-checked build
(libhyena_nd_bounds.so): every kernel access to a caller buffer that is not a
TMA copy, and every plain access to the ahead-copied slots in shared memory, is
checked against the call's buffers; a stray one is redirected, so that it shows
as a wrong result here (and in the feed-forward block's status word).  One
case per kernel runs in a child process (the binding loads one library per
process), against the float64 oracle within the parity tolerances."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BOUNDS_LIB = os.path.join(ROOT, "dimensional_long_convolution_b200", "libhyena_nd_bounds.so")

JOIN = [((1,), 5, 96, "bf16", "layer", "rms", 0.3), ((1,), 3, 101, "f32", "rms", "layer", 0.3),
        ((8, 8), 2, 40, "f32", "layer", "layer", 0.3), ((64,), 2, 130, "bf16", "rms", "layer", 0.3),
        ((13,), 3, 70, "bf16", "layer", "rms", 0.3), ((7,), 2, 30, "f32", "rms", "rms", 0.3),
        ((12,), 2, 700, "bf16", "layer", "layer", 0.3), ((5,), 1, 5000, "f32", "rms", "layer", 0.3)]
FFN = [((1,), 3, 64, 72, "bf16", "silu"), ((5,), 2, 64, 72, "f32", "gelu"), ((8, 8), 2, 64, 136, "bf16", "gelu"),
       ((37,), 3, 40, 72, "bf16", "silu"), ((40,), 2, 72, 136, "f32", "silu"), ((1,), 40, 64, 72, "f32", "silu"),
       ((1,), 50, 64, 72, "bf16", "gelu")]


def _child() -> None:
    sys.path.insert(0, ROOT)
    sys.path.insert(0, os.path.join(ROOT, "tests"))
    from dimensional_long_convolution_b200 import hyena_nd as H
    H.load(BOUNDS_LIB)
    import numpy as np
    import test_gpu_block as T
    from dimensional_long_convolution_b200 import hyena_nd_block as K
    from oracle import block_oracle as O
    for dims, B, C, dt, post, pre, p in JOIN:
        c = T.JoinCase(dims, B, C, dt, post, pre, "wbgs", p)
        c.check_forward()
        c.check_backward()
    for dims, B, C, F, dt, act in FFN:
        T.FfnCase(dims, B, C, F, dt, act).check()
    for dt in ("f32", "bf16"):
        x = T.dev(np.random.default_rng(1).standard_normal((2, 3, 37)), dt)
        want = O.dropout(T.host(x), O.drop_factors(T.SEED, T.OFFSET, 0.4, tuple(x.shape)))
        T.close(T.host(K.GridDropout((37,), 2, 3, io_dtype=dt, p=0.4)(x, T.rng_state())), want, abs(want), dt, 0, "y")
    print("checked %d" % (len(JOIN) + len(FFN) + 2))


@pytest.mark.gpu
def test_block_operators_on_the_checked_build():
    if not os.path.exists(BOUNDS_LIB):
        pytest.fail("libhyena_nd_bounds.so not built")
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "checked %d" % (len(JOIN) + len(FFN) + 2) in r.stdout


if __name__ == "__main__":
    _child()
