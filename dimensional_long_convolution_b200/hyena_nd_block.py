"""Binding of the block operators of libhyena_nd.so (include/hyena_nd_block.h)
and their torch wrappers: ``BlockJoin`` (residual join with the norms on both
sides of it, the block's gate, the residual scale and dropout),
``GridDropout`` and ``GatedFFN``.

They work on the [B, C, *dims] activations of the convolution
(``hyena_nd.HyenaND``) and follow its manner: an object is bound to one
problem shape and device, ``__call__`` is the forward pass, ``backward`` takes
the gradients explicitly, and everything runs in the CUDA kernels of the
library on the current stream of the object's device.  dims may have any
extents here (single tokens, odd lengths).  Scratch memory is taken per call
from torch's allocator, so that one object may serve several streams and
captured graphs.  Tensors are read and written only by the call that takes
them; a tensor made on another stream is ordered by the caller, as for any
torch operation.
"""
from __future__ import annotations

import ctypes
import math
import threading
from typing import Optional, Sequence

from . import hyena_nd as H

NORM_KINDS = {"none": 0, "rms": 1, "layer": 2}
ACTS = {"silu": 0, "gelu": 1}

EXPORTED = (
    "hyena_nd_norm_forward",
    "hyena_nd_norm_backward",
    "hyena_nd_join_forward",
    "hyena_nd_join_backward",
    "hyena_nd_join_workspace_bytes",
    "hyena_nd_dropout",
    "hyena_nd_ffn_workspace_bytes",
    "hyena_nd_ffn_forward",
    "hyena_nd_ffn_backward",
)


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("C", ctypes.c_int64), ("L", ctypes.c_int64), ("io_dtype", ctypes.c_int)]


class Norm(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("eps", ctypes.c_float), ("w", ctypes.c_void_p), ("b", ctypes.c_void_p)]


class Join(ctypes.Structure):
    _fields_ = [
        ("post", Norm),
        ("pre", Norm),
        ("gate", ctypes.c_void_p),
        ("scale", ctypes.c_void_p),
        ("p", ctypes.c_double),
        ("rng", ctypes.c_void_p),
    ]


class JoinGrads(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("post_w", "post_b", "gate", "scale", "pre_w", "pre_b")]


class FFN(ctypes.Structure):
    _fields_ = [("s", Shape), ("F", ctypes.c_int64), ("act", ctypes.c_int)]


_lib: Optional[ctypes.CDLL] = None


def load() -> ctypes.CDLL:
    """The library that ``hyena_nd.load()`` loads, with this header's calls declared."""
    global _lib
    lib = H.load()
    if _lib is lib:
        return lib
    vp, sz, c_int = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    S, N, J, G, FP = (ctypes.POINTER(t) for t in (Shape, Norm, Join, JoinGrads, FFN))
    sigs = {
        "hyena_nd_norm_forward": (c_int, [S, N, vp, vp, vp]),
        "hyena_nd_norm_backward": (c_int, [S, N, vp, vp, vp, vp, vp, vp, sz, vp]),
        "hyena_nd_join_forward": (c_int, [S, J, vp, vp, vp, vp, vp]),
        "hyena_nd_join_backward": (c_int, [S, J, vp, vp, vp, vp, vp, vp, G, vp, sz, vp]),
        "hyena_nd_join_workspace_bytes": (sz, [S]),
        "hyena_nd_dropout": (c_int, [S, ctypes.c_double, vp, vp, vp, vp]),
        "hyena_nd_ffn_workspace_bytes": (sz, [FP, c_int]),
        "hyena_nd_ffn_forward": (c_int, [FP, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "hyena_nd_ffn_backward": (c_int, [FP] + [vp] * 11 + [sz, vp]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


_CONTROL_BYTES = 256
_controls: dict = {}        # of each device, cleared control words for new objects
_control_lock = threading.Lock()


# ------------------------------------------------------------ torch wrappers
class _GridOp:
    """What the operators share: shape, device, argument checks, stream."""

    def __init__(self, dims: Sequence[int], B: int, C: int, io_dtype: str, device):
        import torch

        self.torch = torch
        self.dims = tuple(int(d) for d in dims)
        if not 1 <= len(self.dims) <= 3 or min(self.dims) < 1:
            raise ValueError("dims must be one to three extents of at least 1")
        if io_dtype not in ("f32", "bf16"):
            raise ValueError("io_dtype must be 'f32' or 'bf16'")
        self.B, self.C = int(B), int(C)
        self.io_dtype = io_dtype
        self.tdtype = torch.bfloat16 if io_dtype == "bf16" else torch.float32
        dev = torch.device(device if device is not None else "cuda")
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        self.shape = torch.Size((self.B, self.C) + self.dims)
        self.s = Shape(self.B, self.C, math.prod(self.dims), H.BF16 if io_dtype == "bf16" else H.F32)
        self.lib = load()
        self.ref = ctypes.byref(self.s)
        # the current stream's handle without a Stream object around it (4 us a call less), where torch has that
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)

    def _stream(self) -> int:
        if self.device.type != "cuda":
            raise ValueError("the operators run on CUDA devices, not on %s" % self.device)
        if self.raw_stream is not None:
            return self.raw_stream(self.device.index)
        return self.torch.cuda.current_stream(self.device).cuda_stream

    def _run(self, call, what: str, *args) -> None:
        """A library call on the current stream of the object's device, which
        launches need as the current one."""
        cuda, stream = self.torch.cuda, self._stream()
        if cuda.current_device() == self.device.index:
            code = call(*args, stream)
        else:
            with cuda.device(self.device):
                code = call(*args, stream)
        if code != H.OK:
            raise H.HyenaNDError(code, what)

    def _check(self, name: str, t) -> int:
        """An activation (contiguous, of the problem's shape, dtype and device); its address."""
        if t.shape != self.shape or t.dtype != self.tdtype or t.device != self.device or not t.is_contiguous():
            raise ValueError("%s must be a contiguous %s tensor of shape %s on %s"
                             % (name, self.tdtype, tuple(self.shape), self.device))
        return t.data_ptr()

    def _check_param(self, name: str, t, shape, dtype) -> int:
        if t.shape != shape or t.dtype != dtype or t.device != self.device or not t.is_contiguous():
            raise ValueError("%s must be a contiguous %s tensor of shape %s on %s"
                             % (name, dtype, tuple(shape), self.device))
        return t.data_ptr()

    def _check_rng(self, rng) -> int:
        if rng is None:
            raise ValueError("dropout needs rng, an int64 tensor (seed, offset)")
        return self._check_param("rng", rng, (2,), self.torch.int64)

    def _control_word(self):
        """256 zero bytes that calls on any stream may use at once: no caller could order another stream behind
        their clearing.  They come from a block that was cleared, and waited for, for many objects; where a capture
        needs a new one, the bytes are the graph's own and are cleared by each replay."""
        torch = self.torch

        def zeros(n):
            return torch.zeros(n * _CONTROL_BYTES, dtype=torch.uint8, device=self.device)

        if self.device.type != "cuda":
            return zeros(1)
        with _control_lock:
            left = _controls.setdefault(self.device.index, [])
            if not left:
                with torch.cuda.device(self.device):
                    if torch.cuda.is_current_stream_capturing():
                        return zeros(1)
                    left.extend(zeros(64).split(_CONTROL_BYTES))
                    torch.cuda.current_stream().synchronize()
            return left.pop()

    def _scratch(self, nbytes: int):
        return self.torch.empty(max(nbytes, 16), dtype=self.torch.uint8, device=self.device)


class BlockJoin(_GridOp):
    """h = x + scale_c gate_bc drop(norm_post(y)),  n = norm_pre(h): the join
    of a block's output y to the residual stream x with the norms around it.

    post, pre: "rms", "layer" or "none"; p: dropout probability.  Parameters
    (all optional, fp32) are set by set_params; the object keeps the tensors
    themselves, so values written into them later are seen.  Calls with p > 0
    take ``rng``, an int64 tensor (seed, offset) on the device; the backward
    call must be given the values of its forward call."""

    PARAMS = ("post_w", "post_b", "gate", "scale", "pre_w", "pre_b")

    def __init__(self, dims: Sequence[int], B: int, C: int, io_dtype: str = "f32", post: str = "rms",
                 pre: str = "rms", eps: float = 1e-6, p: float = 0.0, device=None):
        super().__init__(dims, B, C, io_dtype, device)
        if post not in NORM_KINDS or pre not in NORM_KINDS:
            raise ValueError("post and pre must be 'rms', 'layer' or 'none'")
        if not 0.0 <= p <= 1.0:
            raise ValueError("p must be in [0, 1]")
        if not (eps > 0.0 and math.isfinite(eps)):
            raise ValueError("eps must be finite and positive")
        self.p = float(p)
        self.drops = math.floor(self.p * 65536 + 0.5) > 0
        self.post, self.pre = post, pre
        self.params = dict.fromkeys(self.PARAMS)
        self.j = Join()
        self.j.post.kind, self.j.pre.kind = NORM_KINDS[post], NORM_KINDS[pre]
        self.j.post.eps = self.j.pre.eps = float(eps)
        self.j.p = self.p
        self.jref = ctypes.byref(self.j)
        self.ws_bytes = int(self.lib.hyena_nd_join_workspace_bytes(ctypes.byref(self.s)))
        if self.ws_bytes == 0:
            raise H.HyenaNDError(H.ERR_UNSUPPORTED, "join_workspace_bytes")

    def set_params(self, post_w=None, post_b=None, gate=None, scale=None, pre_w=None, pre_b=None) -> None:
        given = dict(zip(self.PARAMS, (post_w, post_b, gate, scale, pre_w, pre_b)))
        for name, t in given.items():
            if t is None:
                continue
            if getattr(self, name.split("_")[0], "") == "none":
                raise ValueError("%s given, but there is no such norm" % name)
            self._check_param(name, t, (self.B, self.C) if name == "gate" else (self.C,), self.torch.float32)
        self.params = given
        ptr = {k: None if t is None else t.data_ptr() for k, t in given.items()}
        self.j.post.w, self.j.post.b = ptr["post_w"], ptr["post_b"]
        self.j.pre.w, self.j.pre.b = ptr["pre_w"], ptr["pre_b"]
        self.j.gate, self.j.scale = ptr["gate"], ptr["scale"]

    def _with_rng(self, rng):
        if not self.drops:
            return self.jref
        j = Join.from_buffer_copy(self.j)       # one object may be called from several threads
        j.rng = self._check_rng(rng)
        return ctypes.byref(j)

    def __call__(self, x, y, rng=None, h=None, n=None):
        """(h, n); n is None without a pre norm."""
        xp, yp = self._check("x", x), self._check("y", y)
        j = self._with_rng(rng)
        if n is not None and self.pre == "none":
            raise ValueError("n given, but there is no pre norm")
        h = self.torch.empty_like(x) if h is None else h
        if n is None and self.pre != "none":
            n = self.torch.empty_like(x)
        self._run(self.lib.hyena_nd_join_forward, "join_forward", self.ref, j, xp, yp, self._check("h", h),
                  None if n is None else self._check("n", n))
        return h, n

    def backward(self, x, y, dh, dn=None, rng=None) -> dict:
        """Gradients "dx", "dy" and "d" + name for each parameter that is set.
        dh: gradient that reaches h past the pre norm (None: zero); dn: that
        of n (exactly where there is a pre norm)."""
        xp, yp = self._check("x", x), self._check("y", y)
        if (dn is None) != (self.pre == "none"):
            raise ValueError("dn goes with the pre norm")
        dhp = None if dh is None else self._check("dh", dh)
        dnp = None if dn is None else self._check("dn", dn)
        j = self._with_rng(rng)
        torch = self.torch
        out = {"dx": torch.empty_like(x), "dy": torch.empty_like(x)}
        grads = JoinGrads()
        for name, t in self.params.items():
            if t is not None:
                out["d" + name] = g = torch.empty_like(t)
                setattr(grads, name, g.data_ptr())
        ws = self._scratch(self.ws_bytes)
        self._run(self.lib.hyena_nd_join_backward, "join_backward", self.ref, j, xp, yp, dhp, dnp,
                  out["dx"].data_ptr(), out["dy"].data_ptr(), ctypes.byref(grads), ws.data_ptr(), self.ws_bytes)
        return out

    def norm(self, x, n=None):
        """norm_pre(x) alone: the head of a stack."""
        if self.pre == "none":
            raise ValueError("there is no pre norm")
        xp = self._check("x", x)
        n = self.torch.empty_like(x) if n is None else n
        self._run(self.lib.hyena_nd_norm_forward, "norm_forward", self.ref, ctypes.byref(self.j.pre), xp,
                  self._check("n", n))
        return n

    def norm_backward(self, x, dn) -> dict:
        """Gradients "dx" and "dpre_w", "dpre_b" where set, of norm(x) for dn."""
        if self.pre == "none":
            raise ValueError("there is no pre norm")
        xp, dnp = self._check("x", x), self._check("dn", dn)
        out = {"dx": self.torch.empty_like(x)}
        for name in ("pre_w", "pre_b"):
            if self.params[name] is not None:
                out["d" + name] = self.torch.empty_like(self.params[name])
        dw, db = (out[k].data_ptr() if k in out else None for k in ("dpre_w", "dpre_b"))
        ws = self._scratch(self.ws_bytes)
        self._run(self.lib.hyena_nd_norm_backward, "norm_backward", self.ref, ctypes.byref(self.j.pre), xp, dnp,
                  out["dx"].data_ptr(), dw, db, ws.data_ptr(), self.ws_bytes)
        return out


class GridDropout(_GridOp):
    """Inverted dropout of a [B, C, *dims] tensor from a counter-based
    generator: kept where a 16-bit lot of Philox4x32-10 at (seed, offset,
    element) reaches round(65536 p), and then multiplied by the reciprocal of
    the kept share.  The mask is never stored: backward recomputes it from the
    same rng, an int64 tensor (seed, offset) on the device."""

    def __init__(self, dims: Sequence[int], B: int, C: int, io_dtype: str = "f32", p: float = 0.1, device=None):
        super().__init__(dims, B, C, io_dtype, device)
        if not 0.0 <= p <= 1.0:
            raise ValueError("p must be in [0, 1]")
        self.p = float(p)
        self.drops = math.floor(self.p * 65536 + 0.5) > 0

    def __call__(self, x, rng=None, y=None):
        xp = self._check("x", x)
        ptr = self._check_rng(rng) if self.drops else None
        y = self.torch.empty_like(x) if y is None else y
        self._run(self.lib.hyena_nd_dropout, "dropout", self.ref, self.p, ptr, xp, self._check("y", y))
        return y

    def backward(self, dy, rng=None, dx=None):
        """dx for dy, with the rng values of the forward call: the same map."""
        return self(dy, rng, dx)


class GatedFFN(_GridOp):
    """y = Wd (act(Wg x) * (Wu x)) over the channels of every position.
    act: "silu" or "gelu".  Weights in the activations' dtype: Wg, Wu [F, C],
    Wd [C, F]; C and F multiples of 8."""

    def __init__(self, dims: Sequence[int], B: int, C: int, F: int, io_dtype: str = "bf16", act: str = "silu",
                 device=None):
        super().__init__(dims, B, C, io_dtype, device)
        if act not in ACTS:
            raise ValueError("act must be 'silu' or 'gelu'")
        self.F, self.act = int(F), act
        self.f = FFN(self.s, self.F, ACTS[act])
        self.ws_bytes = [int(self.lib.hyena_nd_ffn_workspace_bytes(ctypes.byref(self.f), k)) for k in (0, 1)]
        if 0 in self.ws_bytes:
            raise H.HyenaNDError(H.ERR_UNSUPPORTED, "ffn_workspace_bytes")
        self.control = self._control_word()
        self.fref = ctypes.byref(self.f)
        self.up, self.down = self.torch.Size((self.F, self.C)), self.torch.Size((self.C, self.F))

    def _check_weights(self, wg, wu, wd):
        return (self._check_param("wg", wg, self.up, self.tdtype), self._check_param("wu", wu, self.up, self.tdtype),
                self._check_param("wd", wd, self.down, self.tdtype))

    def __call__(self, x, wg, wu, wd, y=None):
        xp, w = self._check("x", x), self._check_weights(wg, wu, wd)
        y = self.torch.empty_like(x) if y is None else y
        ws = self._scratch(self.ws_bytes[0])
        self._run(self.lib.hyena_nd_ffn_forward, "ffn_forward", self.fref, xp, *w, self._check("y", y),
                  self.control.data_ptr(), ws.data_ptr(), self.ws_bytes[0])
        return y

    def backward(self, x, wg, wu, wd, dy):
        """(dx, dwg, dwu, dwd) for dy; the hidden activations are recomputed."""
        xp, dyp, w = self._check("x", x), self._check("dy", dy), self._check_weights(wg, wu, wd)
        out = tuple(self.torch.empty_like(t) for t in (x, wg, wu, wd))
        ws = self._scratch(self.ws_bytes[1])
        self._run(self.lib.hyena_nd_ffn_backward, "ffn_backward", self.fref, xp, *w, dyp,
                  *(t.data_ptr() for t in out), self.control.data_ptr(), ws.data_ptr(), self.ws_bytes[1])
        return out

    def status(self) -> int:
        """Waits for the current stream, then reads and clears the device-side
        status: that of the calls which the current stream comes after.  A call
        still running on another stream may record one later."""
        stream = self._stream()
        with self.torch.cuda.device(self.device):
            return H.device_status(self.control.data_ptr(), stream)
