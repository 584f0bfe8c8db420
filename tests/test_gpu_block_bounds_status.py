"""The index-checked build (libhyena_nd_bounds.so) reports for the operators
that have no status word of their own: the join, the norm and dropout record a
stray access in the library's word, which is read for a null workspace.  A
probe that exists in that build alone reads a byte of a torch tensor inside
and outside the part it registers (both the tensor's own memory); then one
case per kernel runs and has to leave the word clean.  In a child process, as
the binding loads one library per process."""
import ctypes
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _child() -> None:
    sys.path.insert(0, ROOT)
    sys.path.insert(0, os.path.join(ROOT, "tests"))
    import test_gpu_block_bounds as cases
    from dimensional_long_convolution_b200 import hyena_nd as H
    H.load(cases.BOUNDS_LIB)
    import numpy as np
    import test_gpu_block as T
    from dimensional_long_convolution_b200 import hyena_nd_block as K

    t = T.torch()

    def status():
        return H.device_status(0, t.cuda.current_stream().cuda_stream)

    buf, out = t.arange(64, dtype=t.uint8, device="cuda"), t.zeros(1, dtype=t.uint8, device="cuda")
    probe = K.load().hyena_nd_debug_bounds_probe
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    probe.restype, probe.argtypes = ctypes.c_int, [vp, sz, sz, vp, vp]

    def read(registered, at):
        assert probe(buf.data_ptr(), registered, at, out.data_ptr(), t.cuda.current_stream().cuda_stream) == H.OK
        return status()

    assert read(32, 31) == H.OK and int(out) == 31
    assert read(32, 32) == H.ERR_DEVICE_BOUNDS
    assert read(64, 63) == H.OK and int(out) == 63          # read and cleared
    ran = 0
    for dims, B, C, dt, post, pre, p in cases.JOIN + [((40,), 2, 2500, "f32", "rms", "layer", 0.1),
                                                      ((1,), 400, 96, "bf16", "layer", "rms", 0.3)]:
        c = T.JoinCase(dims, B, C, dt, post, pre, "wbgs", p)
        c.check_forward()
        assert status() == H.OK, (dims, B, C, "forward")
        c.check_backward()
        assert status() == H.OK, (dims, B, C, "backward")
        c.op.norm(c.t["x"])
        assert status() == H.OK, (dims, B, C, "norm")
        c.op.norm_backward(c.t["x"], c.t["dn"])
        assert status() == H.OK, (dims, B, C, "norm, backward")
        ran += 1
    for dt in ("f32", "bf16"):
        for n in (1, 7, 37, 64):
            x = T.dev(np.random.default_rng(1).standard_normal((2, 3, n)), dt)
            K.GridDropout((n,), 2, 3, io_dtype=dt, p=0.4)(x, T.rng_state())
            assert status() == H.OK, (dt, n)
            ran += 1
    print("clean: %d" % ran)


@pytest.mark.gpu
def test_checked_build_reports_for_join_norm_and_dropout():
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "clean: 18" in r.stdout


if __name__ == "__main__":
    _child()
