"""What lies beside the buffers of the operators around the convolution.

Every buffer of a C call (inputs, parameters, outputs, the workspace at its
exact size) lies in the middle of a larger one whose margins are all ones,
which reads as NaN in every type.  The results have to be those of torch's own
buffers, so nothing read from a margin counts, and the margins have to stay as
they were.  TMA copies, which no index check covers, have only the extents in
their descriptors to hold them back; these are the sizes that fill no tile."""
import ctypes

import numpy as np
import pytest

import test_gpu_block as T
from dimensional_long_convolution_b200 import hyena_nd as H
from dimensional_long_convolution_b200 import hyena_nd_block as K

pytestmark = pytest.mark.gpu
MARGIN = 1 << 16


class Buffers:
    def __init__(self):
        self.t, self.held = T.torch(), []

    def room(self, nbytes, align=16):
        """The address of nbytes bytes at `align` modulo 2 `align`."""
        t = self.t
        buf = t.full((nbytes + 2 * MARGIN + 2 * align,), 255, dtype=t.uint8, device="cuda")
        at = MARGIN + (align - buf.data_ptr()) % (2 * align)
        self.held.append((buf, at, nbytes))
        return buf[at:at + nbytes]

    def put(self, v, align=16):
        if v is None:
            return None
        r = self.room(v.numel() * v.element_size(), align)
        r.copy_(v.contiguous().reshape(-1).view(self.t.uint8))
        return r.data_ptr()

    def out(self, want, align=16):
        """Room for a result like `want`, and its address."""
        r = self.room(want.numel() * want.element_size(), align)
        return r, r.data_ptr()

    def same(self, rooms, wants):
        for k in wants:
            assert self.t.equal(rooms[k], wants[k].contiguous().reshape(-1).view(self.t.uint8)), k

    def margins_hold(self):
        for buf, at, n in self.held:
            assert (buf[:at] == 255).all() and (buf[at + n:] == 255).all(), (n, at)

    @property
    def stream(self):
        return self.t.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("dims,B,C,F,dt", [
    ((1,), 1, 8, 8, "bf16"), ((5,), 3, 136, 72, "f32"),                      # a few positions
    ((1,), 200, 72, 200, "bf16"), ((1,), 130, 64, 264, "f32"),               # token-major
    ((1,), 40, 72, 2088, "bf16"), ((1,), 40, 24, 2088, "f32"),               # sums split
    ((7,), 30, 64, 96, "bf16"), ((37, 41), 2, 24, 40, "bf16"),               # positions gathered
    ((130,), 2, 200, 264, "f32"), ((37, 41), 1, 24, 40, "f32"),
    ((40,), 1, 72, 136, "bf16"), ((16, 24), 2, 136, 344, "bf16"),            # as they lie
    ((2056,), 1, 8, 1032, "bf16"), ((256,), 2, 40, 2560, "bf16"), ((72,), 2, 1032, 8, "bf16"),
    ((1000,), 1, 264, 1032, "bf16")])
def test_ffn_margins(dims, B, C, F, dt):
    c, m = T.FfnCase(dims, B, C, F, dt, "silu"), Buffers()
    y, g = c.run()
    wants = dict(zip(("y", "dx", "dwg", "dwu", "dwd"), (y, *g)))
    ins = [m.put(c.t[k]) for k in ("x", "wg", "wu", "wd")]
    dy, control = m.put(c.t["dy"]), m.put(m.t.zeros(256, dtype=m.t.uint8, device="cuda"))
    rooms, ptr = {}, {}
    for k, v in wants.items():
        rooms[k], ptr[k] = m.out(v)
    f, need = ctypes.byref(c.op.f), c.op.ws_bytes
    ws = [m.room(n).data_ptr() for n in need]
    lib = K.load()
    assert lib.hyena_nd_ffn_forward(f, *ins, ptr["y"], control, ws[0], need[0], m.stream) == H.OK
    assert lib.hyena_nd_ffn_backward(f, *ins, dy, ptr["dx"], ptr["dwg"], ptr["dwu"], ptr["dwd"], control, ws[1],
                                     need[1], m.stream) == H.OK
    assert H.device_status(control, m.stream) == H.OK
    m.same(rooms, wants)
    m.margins_hold()


@pytest.mark.parametrize("dims,B,C,dt", [
    ((1,), 1, 1, "f32"), ((1,), 5, 96, "bf16"), ((1,), 3, 101, "bf16"), ((1,), 700, 40, "f32"), ((1,), 2, 9000, "bf16"),
    ((8, 8), 2, 64, "bf16"), ((64,), 2, 40, "f32"), ((12,), 3, 40, "f32"),
    ((13,), 3, 70, "bf16"), ((7,), 2, 30, "f32"), ((777,), 2, 9, "bf16"), ((2,), 9, 30, "bf16"),
    ((24,), 2, 1000, "bf16"), ((24,), 2, 3000, "bf16"), ((9,), 2, 1100, "f32"), ((33,), 1, 2500, "bf16"),
    ((8,), 1, 9000, "bf16")])
def test_join_and_norm_margins(dims, B, C, dt):
    c, m = T.JoinCase(dims, B, C, dt, "layer", "rms", "wbgs", 0.3), Buffers()
    t, op = c.t, c.op
    h, n = op(t["x"], t["y"], rng=c.rng)
    grads = op.backward(t["x"], t["y"], t["dh"], t["dn"], rng=c.rng)
    alone = op.norm_backward(t["x"], t["dn"])
    wants = {"h": h, "n": n, "norm": op.norm(t["x"]), **grads, **{"norm_" + k: v for k, v in alone.items()}}
    rooms, ptr = {}, {}
    for k, v in wants.items():
        rooms[k], ptr[k] = m.out(v, 16 if v.shape == t["x"].shape else 4)
    x, y, dh, dn = (m.put(t[k]) for k in ("x", "y", "dh", "dn"))
    par = {k: m.put(v, 4) for k, v in c.pt.items()}
    j = K.Join.from_buffer_copy(op.j)
    j.post.w, j.post.b, j.pre.w, j.pre.b = par["post_w"], par["post_b"], par["pre_w"], par["pre_b"]
    j.gate, j.scale, j.rng = par["gate"], par["scale"], m.put(c.rng, 8)
    lib, s, need = K.load(), ctypes.byref(op.s), op.ws_bytes
    ws = [m.room(need).data_ptr() for _ in range(2)]
    gs = K.JoinGrads(**{k: ptr["d" + k] for k in op.PARAMS})
    assert lib.hyena_nd_join_forward(s, ctypes.byref(j), x, y, ptr["h"], ptr["n"], m.stream) == H.OK
    assert lib.hyena_nd_join_backward(s, ctypes.byref(j), x, y, dh, dn, ptr["dx"], ptr["dy"], ctypes.byref(gs), ws[0],
                                      need, m.stream) == H.OK
    assert lib.hyena_nd_norm_forward(s, ctypes.byref(j.pre), x, ptr["norm"], m.stream) == H.OK
    assert lib.hyena_nd_norm_backward(s, ctypes.byref(j.pre), x, dn, ptr["norm_dx"], ptr["norm_dpre_w"],
                                      ptr["norm_dpre_b"], ws[1], need, m.stream) == H.OK
    m.same(rooms, wants)
    m.margins_hold()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 7, 8, 37, 4096, 8197])
def test_dropout_margins(n, dt):
    m = Buffers()
    x = T.dev(np.random.default_rng(3).standard_normal((1, 3, n)), dt)
    op = K.GridDropout((n,), 1, 3, io_dtype=dt, p=0.3)
    want = {"y": op(x, T.rng_state())}
    room, ptr = m.out(want["y"])
    code = K.load().hyena_nd_dropout(ctypes.byref(op.s), 0.3, m.put(T.rng_state(), 8), m.put(x), ptr, m.stream)
    assert code == H.OK
    m.same({"y": room}, want)
    m.margins_hold()
