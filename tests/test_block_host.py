"""Host-only checks of the operators around the convolution: the oracle
against closed forms and differences, the exported symbols, sizes, and the
refusals of the C ABI (no call here reaches a kernel launch)."""
import ctypes
import os
import re

import numpy as np
import pytest

from dimensional_long_convolution_b200 import hyena_nd as H
from dimensional_long_convolution_b200 import hyena_nd_block as K
from oracle import block_oracle as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x7F0000000000          # fake device addresses, far apart
STEP = 1 << 33


def test_library_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "hyena_nd_block.h")).read()
    names = set(re.findall(r"HYENA_ND_API\s+[\w\s\*]+?\b(hyena_nd_\w+)\s*\(", text))
    assert names == set(K.EXPORTED)
    lib = K.load()
    for n in names:
        assert getattr(lib, n) is not None


# ------------------------------------------------------------------ oracle
@pytest.mark.parametrize("ctr,key,want", [
    # the published known answers of Philox4x32-10
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_oracle_philox_known_answers(ctr, key, want):
    got = O.philox([np.array([c], dtype=np.uint64) for c in ctr], key)
    assert tuple(int(g[0]) for g in got) == want


def test_oracle_lots_are_uniform_and_addressed_by_element():
    v = O.lots(1234, 5, 0, 1 << 16)
    assert abs(v.mean() / 65535 - 0.5) < 5 * 0.2887 / 256
    np.testing.assert_array_equal(v[1003:1100], O.lots(1234, 5, 1003, 97))
    assert (O.lots(1234, 6, 0, 64) != v[:64]).any() and (O.lots(1235, 5, 0, 64) != v[:64]).any()


@pytest.mark.parametrize("post,pre", [("rms", "layer"), ("layer", "rms"), ("none", "layer"), ("layer", "none")])
def test_oracle_join_gradients_against_differences(post, pre):
    rng = np.random.default_rng(7)
    B, C, L, eps = 2, 5, 3, 1e-3
    x, y, dh, dn = (rng.standard_normal((B, C, L)) for _ in range(4))
    P = {"post_w": rng.standard_normal(C), "post_b": rng.standard_normal(C), "gate": rng.standard_normal((B, C)),
         "scale": rng.standard_normal(C), "pre_w": rng.standard_normal(C), "pre_b": rng.standard_normal(C)}
    for s in ("post", "pre"):
        if (post if s == "post" else pre) == "none":
            P[s + "_w"] = P[s + "_b"] = None
    m = O.drop_factors(3, 4, 0.3, x.shape)
    assert 0 < (m == 0).sum() < m.size

    def loss():
        h, n = O.join(x, y, m, P, post, pre, eps)
        return (h * dh).sum() + (0.0 if n is None else (n * dn).sum())

    g = O.join_backward(x, y, m, P, post, pre, eps, dh, dn)
    for name, t in [("dx", x), ("dy", y)] + [("d" + k, v) for k, v in P.items() if v is not None]:
        flat, got = t.reshape(-1), np.asarray(g[name]).reshape(-1)
        for i in range(flat.size):
            keep, step = flat[i], 1e-5
            flat[i] = keep + step
            up = loss()
            flat[i] = keep - step
            down = loss()
            flat[i] = keep
            # central difference: error of order step^2 times the third derivative, plus rounding / step
            assert abs((up - down) / (2 * step) - got[i]) < 1e-5 * max(1.0, np.abs(got).max()), (name, i)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_oracle_ffn_gradients_against_differences(kind):
    rng = np.random.default_rng(8)
    x, dy = rng.standard_normal((2, 4, 3)), rng.standard_normal((2, 4, 3))
    wg, wu, wd = rng.standard_normal((6, 4)), rng.standard_normal((6, 4)), rng.standard_normal((4, 6))
    grads = O.ffn_backward(x, wg, wu, wd, dy, kind)
    for t, g in zip((x, wg, wu, wd), grads):
        flat, got = t.reshape(-1), g.reshape(-1)
        for i in range(flat.size):
            keep, step = flat[i], 1e-5
            flat[i] = keep + step
            up = (O.ffn(x, wg, wu, wd, kind) * dy).sum()
            flat[i] = keep - step
            down = (O.ffn(x, wg, wu, wd, kind) * dy).sum()
            flat[i] = keep
            assert abs((up - down) / (2 * step) - got[i]) < 1e-5 * max(1.0, np.abs(got).max())


# ---------------------------------------------------------------- refusals
def _ptr(i):
    return A + i * STEP


def _shape(B=2, C=8, L=16, dt=0):
    return K.Shape(B, C, L, dt)


def _join(post=1, pre=1, eps=1e-6, p=0.0, **kw):
    j = K.Join()
    j.post.kind, j.pre.kind = post, pre
    j.post.eps = j.pre.eps = eps
    j.p = p
    for k, v in kw.items():
        if "_" in k:
            s, f = k.split("_")
            setattr(getattr(j, s), f, v)
        else:
            setattr(j, k, v)
    return j


def _fwd(s, j, x=_ptr(0), y=_ptr(1), h=_ptr(2), n=_ptr(3)):
    return K.load().hyena_nd_join_forward(ctypes.byref(s), ctypes.byref(j), x, y, h, n, None)


def test_join_forward_refusals():
    inv, uns, mis = H.ERR_INVALID_ARG, H.ERR_UNSUPPORTED, H.ERR_MISALIGNED
    for bad in (_shape(B=0), _shape(C=0), _shape(L=0), _shape(B=-1), _shape(dt=2)):
        assert _fwd(bad, _join()) == inv
    for big in (_shape(C=65537), _shape(B=1 << 31), _shape(L=1 << 31), _shape(B=1 << 20, L=1 << 20),
                _shape(B=1 << 15, C=1 << 16, L=1), _shape(B=4, C=1 << 16, L=1 << 28)):
        assert _fwd(big, _join()) == uns
        assert K.load().hyena_nd_join_workspace_bytes(ctypes.byref(big)) == 0
    s = _shape()
    for j in (_join(post=3), _join(pre=-1), _join(eps=0.0), _join(eps=-1.0), _join(eps=float("nan")),
              _join(eps=float("inf")), _join(p=-0.1), _join(p=1.1), _join(p=float("nan")), _join(p=0.5),
              _join(post=0, post_w=_ptr(9))):
        assert _fwd(s, j) == inv
    assert _fwd(s, _join(post=0, pre=0, eps=0.0, pre_b=_ptr(9)), n=None) == inv
    for k in ("x", "y", "h", "n"):
        assert _fwd(s, _join(), **{k: None}) == inv
        assert _fwd(s, _join(), **{k: _ptr(7) + 8}) == mis
    assert _fwd(s, _join(pre=0)) == inv                     # n without a pre norm
    for kw in (dict(post_w=_ptr(9) + 2), dict(pre_b=_ptr(9) + 1), dict(gate=_ptr(9) + 2), dict(scale=_ptr(9) + 3),
               dict(rng=_ptr(9) + 4, p=0.5)):
        assert _fwd(s, _join(**kw)) == mis
    n = 2 * 8 * 16 * 4
    assert _fwd(s, _join(), h=_ptr(0)) == inv               # in place
    assert _fwd(s, _join(), h=_ptr(1) + n - 16) == inv      # the last bytes of y
    assert _fwd(s, _join(), n=_ptr(2) + 16) == inv          # outputs over each other
    assert _fwd(s, _join(scale=_ptr(2) + 4)) == inv         # a parameter inside an output


def test_join_backward_refusals():
    lib, s, j = K.load(), _shape(), _join()
    need = lib.hyena_nd_join_workspace_bytes(ctypes.byref(s))
    assert need > 0

    def call(j=j, ws=_ptr(8), ws_bytes=need, grads=None, **kw):
        a = dict(x=_ptr(0), y=_ptr(1), dh=_ptr(2), dn=_ptr(3), dx=_ptr(4), dy=_ptr(5))
        a.update(kw)
        g = K.JoinGrads(**(grads or {}))
        return lib.hyena_nd_join_backward(ctypes.byref(s), ctypes.byref(j), *a.values(), ctypes.byref(g), ws,
                                          ws_bytes, None)

    for k in ("x", "y", "dn", "dx", "dy"):
        assert call(**{k: None}) == H.ERR_INVALID_ARG
    assert call(ws=None) == H.ERR_INVALID_ARG
    assert call(ws_bytes=need - 1) == H.ERR_WORKSPACE_TOO_SMALL
    assert call(ws=_ptr(8) + 4) == H.ERR_MISALIGNED
    assert call(dx=_ptr(2)) == H.ERR_INVALID_ARG
    assert call(dy=_ptr(4)) == H.ERR_INVALID_ARG
    assert call(ws=_ptr(3)) == H.ERR_INVALID_ARG
    assert call(grads=dict(gate=_ptr(9) + 2)) == H.ERR_MISALIGNED
    assert call(grads=dict(gate=_ptr(5))) == H.ERR_INVALID_ARG
    assert call(j=_join(pre=0)) == H.ERR_INVALID_ARG                                     # dn without a pre norm
    assert call(j=_join(pre=0), dn=None, grads=dict(pre_w=_ptr(9))) == H.ERR_INVALID_ARG
    assert call(j=_join(post=0), grads=dict(post_b=_ptr(9))) == H.ERR_INVALID_ARG


def test_norm_refusals():
    lib, s = K.load(), _shape()
    n, none = K.Norm(1, 1e-6, None, None), K.Norm(0, 1e-6, None, None)
    f = lambda n, x=_ptr(0), o=_ptr(1): lib.hyena_nd_norm_forward(ctypes.byref(s), ctypes.byref(n), x, o, None)  # noqa: E731
    assert f(none) == H.ERR_INVALID_ARG and f(n, x=None) == H.ERR_INVALID_ARG and f(n, o=None) == H.ERR_INVALID_ARG
    assert f(n, o=_ptr(0)) == H.ERR_INVALID_ARG and f(n, x=_ptr(0) + 2) == H.ERR_MISALIGNED
    assert lib.hyena_nd_norm_forward(None, ctypes.byref(n), _ptr(0), _ptr(1), None) == H.ERR_INVALID_ARG
    assert lib.hyena_nd_norm_forward(ctypes.byref(s), None, _ptr(0), _ptr(1), None) == H.ERR_INVALID_ARG
    need = lib.hyena_nd_join_workspace_bytes(ctypes.byref(s))
    b = lambda n, dn=_ptr(1), dx=_ptr(2), ws=_ptr(3), nb=need: lib.hyena_nd_norm_backward(  # noqa: E731
        ctypes.byref(s), ctypes.byref(n), _ptr(0), dn, dx, None, None, ws, nb, None)
    assert b(none) == H.ERR_INVALID_ARG and b(n, dn=None) == H.ERR_INVALID_ARG and b(n, ws=None) == H.ERR_INVALID_ARG
    assert b(n, dx=_ptr(1)) == H.ERR_INVALID_ARG and b(n, nb=need - 1) == H.ERR_WORKSPACE_TOO_SMALL


def test_dropout_refusals():
    lib = K.load()

    def call(s=_shape(), p=0.5, rng=_ptr(5), x=_ptr(0), y=_ptr(1)):
        return lib.hyena_nd_dropout(ctypes.byref(s), p, rng, x, y, None)

    assert call(s=_shape(L=0)) == H.ERR_INVALID_ARG
    for p in (-1e-9, 1.0 + 1e-9, float("nan"), float("inf")):
        assert call(p=p) == H.ERR_INVALID_ARG
    assert call(rng=None) == H.ERR_INVALID_ARG and call(x=None) == H.ERR_INVALID_ARG and call(y=None) == H.ERR_INVALID_ARG
    assert call(rng=_ptr(5) + 4) == H.ERR_MISALIGNED and call(x=_ptr(0) + 4) == H.ERR_MISALIGNED
    assert call(y=_ptr(0)) == H.ERR_INVALID_ARG and call(y=_ptr(5) - 16) == H.ERR_INVALID_ARG


def _ffn(B=2, C=8, L=16, F=16, dt=1, act=0):
    return K.FFN(K.Shape(B, C, L, dt), F, act)


def test_ffn_refusals():
    lib = K.load()
    size = lambda f, b=0: lib.hyena_nd_ffn_workspace_bytes(ctypes.byref(f), b)  # noqa: E731
    for f in (_ffn(C=12), _ffn(F=20), _ffn(C=65544), _ffn(F=65544), _ffn(F=0), _ffn(act=2), _ffn(dt=3), _ffn(L=0),
              _ffn(B=1 << 16, L=1 << 14, F=1 << 16)):
        assert size(f) == 0 and size(f, 1) == 0
    f = _ffn()
    need = size(f), size(f, 1)
    assert 0 < need[0] <= need[1]

    def fwd(f=f, nb=need[0], **kw):
        a = dict(x=_ptr(0), wg=_ptr(1), wu=_ptr(2), wd=_ptr(3), y=_ptr(4), control=_ptr(5), ws=_ptr(6))
        a.update(kw)
        return lib.hyena_nd_ffn_forward(ctypes.byref(f), *a.values(), nb, None)

    def bwd(f=f, nb=need[1], **kw):
        names = ("x", "wg", "wu", "wd", "dy", "dx", "dwg", "dwu", "dwd", "control", "ws")
        a = {k: _ptr(i) for i, k in enumerate(names)}
        a.update(kw)
        return lib.hyena_nd_ffn_backward(ctypes.byref(f), *a.values(), nb, None)

    for call, names in ((fwd, ("x", "wg", "wu", "wd", "y", "control", "ws")),
                        (bwd, ("x", "wg", "wu", "wd", "dy", "dx", "dwg", "dwu", "dwd", "control", "ws"))):
        for k in names:
            assert call(**{k: None}) == H.ERR_INVALID_ARG
            assert call(**{k: _ptr(30) + 2}) == H.ERR_MISALIGNED
        assert call(f=_ffn(C=12)) == H.ERR_UNSUPPORTED
        assert call(nb=0) == H.ERR_WORKSPACE_TOO_SMALL
    assert fwd(y=_ptr(0)) == H.ERR_INVALID_ARG and fwd(ws=_ptr(3)) == H.ERR_INVALID_ARG
    assert bwd(dwg=_ptr(1)) == H.ERR_INVALID_ARG and bwd(dwu=_ptr(6)) == H.ERR_INVALID_ARG


@pytest.mark.parametrize("B,C,L,F", [(40, 24, 1, 2088), (2, 64, 1024, 136), (5, 72, 37, 40), (1, 8, 1, 8)])
def test_ffn_workspace_has_room_for_32_byte_stores(B, C, L, F):
    """A workspace starts on 16 bytes; the fp32 hidden planes, which leave in stores of 32, start on the next 32
    from there.  All parts are multiples of 256 bytes, so what is above a multiple is the room for that: 16 bytes or
    more in each fp32 call that has such planes (up to 32 positions forward: none)."""
    lib, f = K.load(), _ffn(B, C, L, F, dt=0)
    for backward in (0, 1):
        if backward or B * L > 32:
            assert lib.hyena_nd_ffn_workspace_bytes(ctypes.byref(f), backward) % 256 >= 16


def test_wrapper_refusals():
    import torch

    cpu = torch.device("cpu")
    with pytest.raises(ValueError):
        K.BlockJoin((8, 0), 1, 4, device=cpu)
    with pytest.raises(ValueError):
        K.BlockJoin((8,), 1, 4, io_dtype="f16", device=cpu)
    with pytest.raises(ValueError):
        K.BlockJoin((8,), 1, 4, post="batch", device=cpu)
    with pytest.raises(ValueError):
        K.BlockJoin((8,), 1, 4, p=1.5, device=cpu)
    with pytest.raises(ValueError):
        K.BlockJoin((8,), 1, 4, eps=0.0, device=cpu)
    with pytest.raises(H.HyenaNDError):
        K.BlockJoin((8,), 1, 1 << 17, device=cpu)
    with pytest.raises(ValueError):
        K.GridDropout((8,), 1, 4, p=-0.5, device=cpu)
    with pytest.raises(ValueError):
        K.GatedFFN((8,), 1, 8, 8, act="relu", device=cpu)
    with pytest.raises(H.HyenaNDError):
        K.GatedFFN((8,), 1, 4, 8, device=cpu)
    op = K.BlockJoin((4, 4), 2, 3, post="rms", pre="none", p=0.5, device=cpu)
    x = torch.zeros(2, 3, 4, 4)
    rng = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        op(x, torch.zeros(2, 3, 16), rng)                   # shape
    with pytest.raises(ValueError):
        op(x, x.to(torch.bfloat16), rng)                    # dtype
    with pytest.raises(ValueError):
        op(x, torch.zeros(2, 4, 4, 3).movedim(3, 1), rng)   # strides
    with pytest.raises(ValueError):
        op(x, x.clone())                                    # no rng
    with pytest.raises(ValueError):
        op(x, x.clone(), rng.to(torch.int32))
    with pytest.raises(ValueError):
        op(x, x.clone(), rng, n=x.clone())                  # no pre norm
    with pytest.raises(ValueError):
        op.backward(x, x.clone(), x.clone(), x.clone(), rng)
    with pytest.raises(ValueError):
        op.norm(x)
    with pytest.raises(ValueError):
        op.set_params(pre_w=torch.ones(3))
    with pytest.raises(ValueError):
        op.set_params(gate=torch.ones(3))
    with pytest.raises(ValueError):
        op.set_params(scale=torch.ones(3, dtype=torch.float64))
    with pytest.raises(ValueError):
        op(x, x.clone(), rng)                               # host tensors: nothing is launched
    ffn = K.GatedFFN((4,), 2, 8, 16, io_dtype="f32", device=cpu)
    with pytest.raises(ValueError):
        ffn(torch.zeros(2, 8, 4), torch.zeros(16, 8), torch.zeros(8, 16), torch.zeros(8, 16))
