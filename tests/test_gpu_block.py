"""Parity of the operators around the convolution (residual join with its
norms, counter-based dropout, gated feed-forward block) with the float64
oracle, over the shapes, types and values where they can go wrong.

Tolerances are elementwise and derived.  A stored value is rounded once: half
a step, 2^-8 (bf16) or 2^-24 (fp32) of it.  fp32 arithmetic adds at most
(k + length of the longest serial sum) 2^-24 of the magnitudes of the terms
that are added up (the oracle's "mag" arrays): k = 64 covers the operations
before and after the sums, and a sum of n terms that is split over at least 8
lanes has at most n / 8 + 16 additions in a row."""
import numpy as np
import pytest

from dimensional_long_convolution_b200 import hyena_nd as H
from dimensional_long_convolution_b200 import hyena_nd_block as K
from oracle import block_oracle as O

pytestmark = pytest.mark.gpu

HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def torch():
    import torch as _t
    return _t


def dev(a, dt="f32"):
    t = torch()
    v = t.from_numpy(np.ascontiguousarray(a)).to(t.float32)
    return (v.to(t.bfloat16) if dt == "bf16" else v).cuda()


def host(t, B=None, C=None):
    v = t.detach().double().cpu().numpy()
    return v if B is None else v.reshape(B, C, -1)


def close(got, want, mag, dt, n, what):
    """Elementwise: half a step of the value plus fp32 error of its terms (sums of n)."""
    tol = HALF_STEP[dt] * np.abs(want) * 1.001 + (80 + n / 8) * 2.0 ** -24 * mag + 1e-37
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of the tolerance" % (
        what, bad.sum(), bad.size, np.nanmax(np.abs(got - want) / tol))


SEED, OFFSET = 0x1234567890ABCDEF, (7 << 32) + 3


def rng_state(seed=SEED, offset=OFFSET):
    t = torch()
    return t.tensor([seed, offset], dtype=t.int64, device="cuda")


class JoinCase:
    def __init__(self, dims, B, C, dt, post, pre, params="wbgs", p=0.0, seed=0, values=None, eps=1e-6):
        r = np.random.default_rng(seed + 31)
        self.dims, self.B, self.C, self.dt, self.post, self.pre, self.p, self.eps = dims, B, C, dt, post, pre, p, eps
        L = int(np.prod(dims))
        shape = (B, C, L)
        raw = {k: r.standard_normal(shape) for k in ("x", "y", "dh", "dn")}
        raw["y"] *= 0.4
        if values:
            values(raw)
        self.t = {k: dev(v.reshape((B, C) + tuple(dims)), dt) for k, v in raw.items()}
        self.v = {k: host(t, B, C) for k, t in self.t.items()}      # the stored values
        par = {}
        for s in ("post", "pre"):
            on = (post if s == "post" else pre) != "none"
            par[s + "_w"] = 1 + 0.3 * r.standard_normal(C) if on and "w" in params else None
            par[s + "_b"] = 0.3 * r.standard_normal(C) if on and "b" in params else None
        par["gate"] = 1 + 0.5 * r.standard_normal((B, C)) if "g" in params else None
        par["scale"] = 0.5 + 0.2 * r.standard_normal(C) if "s" in params else None
        self.pt = {k: None if a is None else dev(a) for k, a in par.items()}
        self.P = {k: None if a is None else host(a) for k, a in self.pt.items()}
        self.op = K.BlockJoin(dims, B, C, io_dtype=dt, post=post, pre=pre, eps=eps, p=p)
        self.op.set_params(**self.pt)
        self.rng = rng_state() if self.op.drops else None
        self.m = O.drop_factors(SEED, OFFSET, p, shape)
        if pre == "none":
            self.t["dn"] = self.v["dn"] = None

    def mags(self):
        """Magnitudes of the terms of h and n."""
        P, v = self.P, self.v
        one = lambda a: 1.0 if a is None else np.abs(a)[None, :, None]  # noqa: E731
        g = 1.0 if P["gate"] is None else np.abs(P["gate"])[:, :, None]
        y = np.abs(v["y"])
        if self.post != "none":
            _, rho = O.stats(v["y"], self.post, self.eps)
            y = rho * (y + y.mean(1, keepdims=True))
            y = y * one(P["post_w"]) + (0.0 if P["post_b"] is None else np.abs(P["post_b"])[None, :, None])
        h = np.abs(v["x"]) + g * one(P["scale"]) * self.m * y
        if self.pre == "none":
            return h, None
        hv = O.join(v["x"], v["y"], self.m, P, self.post, "none", self.eps)[0]
        _, rho = O.stats(hv, self.pre, self.eps)
        n = rho * (h + h.mean(1, keepdims=True)) * one(P["pre_w"])
        return h, n + (0.0 if P["pre_b"] is None else np.abs(P["pre_b"])[None, :, None])

    def check_forward(self):
        h, n = self.op(self.t["x"], self.t["y"], rng=self.rng)
        wh, wn = O.join(self.v["x"], self.v["y"], self.m, self.P, self.post, self.pre, self.eps)
        mh, mn = self.mags()
        close(host(h, self.B, self.C), wh, mh, self.dt, self.C, "h")
        if self.pre == "none":
            assert n is None
        else:
            # the error of the statistics of h reaches every channel: twice the magnitudes
            close(host(n, self.B, self.C), wn, 2 * mn, self.dt, self.C, "n")
        return h, n

    def check_backward(self, dh=True):
        t, v = self.t, self.v
        got = self.op.backward(t["x"], t["y"], t["dh"] if dh else None, t["dn"], rng=self.rng)
        want = O.join_backward(v["x"], v["y"], self.m, self.P, self.post, self.pre, self.eps, v["dh"] if dh else None,
                               v["dn"])
        assert set(got) == {"dx", "dy"} | {"d" + k for k, a in self.P.items() if a is not None}
        T = self.B * v["x"].shape[2]
        for k, g in got.items():
            act = k in ("dx", "dy")
            close(host(g, self.B, self.C) if act else host(g), want[k], 2 * want["mag_" + k],
                  self.dt if act else "f32", self.C + (0 if act else T), k)
        return got


JOIN = [
    # dims, B, C, dtype, post, pre, parameters, p
    ((1,), 1, 1, "f32", "rms", "layer", "wbgs", 0.0),            # one value
    ((1,), 5, 8, "bf16", "layer", "rms", "wbgs", 0.5),           # tokens: channels lie together
    ((1,), 37, 96, "f32", "layer", "layer", "wbgs", 0.25),
    ((1,), 3, 101, "bf16", "rms", "rms", "wg", 0.3),             # odd channel count, tokens
    ((1,), 16, 1024, "bf16", "rms", "rms", "wgs", 0.0),
    ((1,), 4, 7777, "f32", "layer", "layer", "wb", 0.1),
    ((1,), 2, 40000, "bf16", "rms", "layer", "wbgs", 0.1),       # wide tokens
    ((2,), 3, 5, "f32", "rms", "rms", "", 0.0),
    ((7,), 3, 5, "f32", "none", "layer", "wbs", 0.9),
    ((8, 8), 2, 64, "bf16", "rms", "none", "wgs", 0.0),
    ((8, 8), 2, 64, "f32", "none", "none", "", 0.4),
    ((37, 41), 2, 5, "bf16", "layer", "rms", "wbgs", 0.1),       # odd rows
    ((64, 64), 2, 96, "f32", "layer", "layer", "wbgs", 0.1),
    ((24,), 2, 1000, "bf16", "rms", "layer", "wbgs", 0.2),
    ((777,), 2, 204, "bf16", "rms", "layer", "wbg", 0.25),
    ((777,), 2, 204, "f32", "layer", "rms", "wbs", 0.25),
    ((16, 8, 8), 1, 1, "f32", "rms", "rms", "wbgs", 0.0),        # one channel
    ((16, 8, 8), 3, 33, "bf16", "layer", "layer", "", 0.5),
    ((40,), 2, 2500, "f32", "rms", "layer", "wbgs", 0.1),        # many channels
    ((33,), 1, 2500, "bf16", "layer", "rms", "wbgs", 0.1),
    ((8,), 1, 9000, "bf16", "layer", "layer", "wbgs", 0.1),      # more channels than a block holds
    ((3,), 1, 9000, "f32", "rms", "rms", "wbgs", 0.1),
    ((8,), 1, 65536, "bf16", "rms", "layer", "wgs", 0.0),        # the most channels
    ((8,), 1200, 16, "f32", "layer", "rms", "wbgs", 0.1),        # many short samples
    # rows of 16 bytes: one to many lanes of positions, channels that fill a block or not
    ((24,), 2, 300, "bf16", "layer", "rms", "wbgs", 0.1),
    ((40,), 2, 700, "f32", "rms", "layer", "wbgs", 0.1),
    ((12,), 3, 40, "f32", "layer", "layer", "wbgs", 0.3),        # rows of half a counter group
    ((16, 128), 3, 9, "bf16", "rms", "layer", "wbgs", 0.3),
    ((1024,), 1, 256, "f32", "layer", "rms", "wbgs", 0.3),
    ((512,), 5, 512, "bf16", "rms", "rms", "wgs", 0.1),
    # rows that start anywhere: every shift, short and long, a last vector of each length
    ((2,), 9, 30, "bf16", "layer", "rms", "wbgs", 0.4),
    ((3,), 5, 700, "f32", "rms", "layer", "wbgs", 0.4),
    ((5,), 4, 1000, "f32", "layer", "rms", "wbgs", 0.2),
    ((7,), 40, 70, "bf16", "rms", "layer", "wbgs", 0.2),
    ((9,), 2, 500, "bf16", "layer", "layer", "wbgs", 0.2),
    ((11,), 3, 129, "f32", "layer", "layer", "wbgs", 0.2),
    ((255,), 1, 129, "f32", "rms", "rms", "wbgs", 0.2),
    ((257,), 2, 40, "bf16", "layer", "rms", "wbgs", 0.2),
    ((1003,), 2, 7, "bf16", "rms", "layer", "wbgs", 0.5),
    ((4097,), 1, 33, "f32", "layer", "rms", "wbgs", 0.5),
    ((31, 33), 2, 512, "bf16", "rms", "layer", "gs", 0.1),
    ((6,), 3, 2000, "f32", "rms", "rms", "wbgs", 0.1),
    ((4,), 3, 900, "bf16", "layer", "layer", "wbgs", 0.1),
]


@pytest.mark.parametrize("dims,B,C,dt,post,pre,params,p", JOIN)
def test_join_parity(dims, B, C, dt, post, pre, params, p):
    c = JoinCase(dims, B, C, dt, post, pre, params, p)
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("dims,C,dt", [
    # the most channels of each kind of block, and one more: persistent, registers, any number
    ((24,), 512, "bf16"), ((24,), 513, "bf16"), ((24,), 1024, "f32"), ((24,), 1025, "f32"), ((25,), 513, "f32"),
    ((24,), 2048, "bf16"), ((24,), 2049, "bf16"), ((24,), 3000, "bf16"), ((24,), 4096, "f32"), ((24,), 4097, "f32"),
    ((25,), 4096, "bf16"), ((25,), 4097, "f32"), ((25,), 16384, "bf16"), ((25,), 16385, "f32"),
    ((1,), 4095, "bf16"), ((1,), 4097, "f32"), ((1,), 8192, "bf16"), ((1,), 8193, "f32"), ((1,), 8200, "bf16"),
    ((1,), 16384, "f32"), ((1,), 16392, "bf16"), ((4,), 1024, "bf16"), ((3,), 2048, "f32"), ((3,), 2049, "f32")])
def test_join_parity_at_the_limits_of_its_kernels(dims, C, dt):
    c = JoinCase(dims, 2, C, dt, "layer", "rms", "wbgs", 0.1)
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("dims,C", [((13,), 24), ((8, 8), 64), ((777,), 9)])
def test_join_writes_its_outputs_only(dims, C, dt):
    """Outputs in the middle of larger buffers: what lies before and behind stays as it was."""
    t = torch()
    c = JoinCase(dims, 2, C, dt, "rms", "layer", "wbgs", 0.2)
    want_h, want_n = c.op(c.t["x"], c.t["y"], rng=c.rng)
    size, pad = want_h.numel(), 64
    h, n = (t.full((size + 2 * pad,), 7.0, dtype=want_h.dtype, device="cuda") for _ in range(2))
    c.op(c.t["x"], c.t["y"], rng=c.rng, h=h[pad:pad + size].view(want_h.shape), n=n[pad:pad + size].view(want_h.shape))
    for buf, want in ((h, want_h), (n, want_n)):
        assert t.equal(buf[pad:pad + size].view(want.shape), want)
        assert (buf[:pad] == 7).all() and (buf[pad + size:] == 7).all()


@pytest.mark.parametrize("dims,C", [((1,), 64), ((8, 8), 64), ((13,), 30)])
def test_join_without_the_gradient_past_the_norm(dims, C):
    JoinCase(dims, 3, C, "f32", "rms", "layer", "wbgs", 0.1).check_backward(dh=False)


def _zero_rows(raw):
    raw["x"][:, :, 0] = 0
    raw["y"][:, :, 0] = 0
    raw["y"][:, :, -1] = 0.5          # a constant row: no variance


def _far_mean(raw):
    raw["x"] += 300
    raw["y"] += 40


def _tiny(raw):
    for k in ("x", "y"):
        raw[k] *= 1e-12               # squares far below eps


@pytest.mark.parametrize("dims", [(1,), (24,), (11,)])
@pytest.mark.parametrize("values", [_zero_rows, _far_mean, _tiny])
def test_join_values(dims, values):
    for post, pre in (("rms", "layer"), ("layer", "rms")):
        c = JoinCase(dims, 3, 48, "f32", post, pre, "wbgs", 0.0, values=values)
        c.check_forward()
        c.check_backward()


@pytest.mark.parametrize("dims", [(1,), (16,), (7,)])
def test_join_drops_infinities_and_nan(dims):
    """A dropped value is gone even where it is NaN (no post norm); a kept one shows."""
    c = JoinCase(dims, 4, 40, "f32", "none", "none", "gs", 0.5)
    y = c.t["y"].clone()
    flat = y.view(c.B, c.C, -1)
    gone = torch().from_numpy(c.m == 0).cuda()
    flat[gone] = float("nan")
    flat[0, 0, 0] = float("inf")
    h, _ = c.op(c.t["x"], y, rng=c.rng)
    got = host(h, c.B, c.C)
    want, _ = O.join(c.v["x"], c.v["y"], c.m, c.P, "none", "none", c.eps)
    keep = np.ones(want.shape, dtype=bool)
    keep[0, 0, 0] = False
    close(got[keep], want[keep], np.abs(c.v["x"] + 0 * want)[keep] + np.abs(want)[keep], "f32", 1, "h")
    assert np.isinf(got[0, 0, 0]) == (c.m[0, 0, 0] > 0)


@pytest.mark.parametrize("pre", ["none", "layer"])
@pytest.mark.parametrize("dims,B,C,dt", [((1,), 4, 40, "f32"), ((1,), 400, 96, "bf16"), ((1,), 3, 33, "f32"),
                                         ((16,), 4, 40, "f32"), ((64,), 2, 70, "bf16"), ((7,), 4, 40, "bf16"),
                                         ((13,), 2, 40, "f32"), ((24,), 2, 700, "bf16"), ((9,), 2, 1100, "f32"),
                                         ((8,), 1, 9000, "f32")])
def test_join_gradients_drop_infinities_and_nan(dims, B, C, dt, pre):
    """A dropped value of y reaches nothing, so the gradients (those of gate and scale sum over products with y) are
    the ones of any finite value in its place."""
    c = JoinCase(dims, B, C, dt, "none", pre, "wbgs", 0.5)
    gone = np.argwhere(c.m == 0)
    flat = c.t["y"].view(c.B, c.C, -1)
    for k, value in enumerate((float("nan"), float("inf"), -float("inf"))):
        i = torch().from_numpy(np.ascontiguousarray(gone[k::3].T)).cuda()
        flat[i[0], i[1], i[2]] = value
    c.v["y"][c.m == 0] = 0
    c.check_forward()
    got = c.check_backward()
    assert (host(got["dy"], B, C)[c.m == 0] == 0).all()


def test_join_nan_stays_in_its_position():
    for dims in ((16,), (7,), (1,)):
        c = JoinCase(dims, 3, 40, "f32", "layer", "rms", "wb", 0.0)
        c.t["y"].view(3, 40, -1)[1, 5, 0] = float("nan")
        h, n = c.op(c.t["x"], c.t["y"])
        for t in (h, n):
            bad = np.isnan(host(t, 3, 40))
            assert bad[1, :, 0].all()
            bad[1, :, 0] = False
            assert not bad.any()


@pytest.mark.parametrize("dims,B,C,dt", [((1,), 9, 96, "bf16"), ((64,), 2, 40, "f32"), ((13,), 2, 40, "bf16"),
                                         ((1,), 2, 33, "f32")])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_alone(dims, B, C, dt, kind):
    c = JoinCase(dims, B, C, dt, "none", kind, "wb", 0.0)
    x, dn, P = c.v["x"], c.v["dn"], c.P
    n = c.op.norm(c.t["x"])
    _, rho = O.stats(x, kind, c.eps)
    mag = rho * (np.abs(x) + np.abs(x).mean(1, keepdims=True)) * np.abs(P["pre_w"])[None, :, None] \
        + np.abs(P["pre_b"])[None, :, None]
    close(host(n, B, C), O.norm(x, kind, P["pre_w"], P["pre_b"], c.eps), 2 * mag, dt, C, "n")
    got = c.op.norm_backward(c.t["x"], c.t["dn"])
    dx, dw, db, mdx, mdw, mdb = O.norm_backward(x, kind, P["pre_w"], dn, c.eps)
    close(host(got["dx"], B, C), dx, 2 * mdx, dt, C, "dx")
    close(host(got["dpre_w"]), dw, 2 * mdw, "f32", C + n.numel() // C, "dw")
    close(host(got["dpre_b"]), db, mdb, "f32", n.numel() // C, "db")


def test_results_repeat_bit_for_bit():
    t = torch()
    for dims, C in (((1,), 96), ((64, 64), 40), ((777,), 20)):
        c = JoinCase(dims, 4, C, "f32", "layer", "layer", "wbgs", 0.1)
        first = c.op.backward(c.t["x"], c.t["y"], c.t["dh"], c.t["dn"], rng=c.rng)
        again = c.op.backward(c.t["x"], c.t["y"], c.t["dh"], c.t["dn"], rng=c.rng)
        for k in first:
            assert t.equal(first[k], again[k])


# ----------------------------------------------------------------- dropout
@pytest.mark.parametrize("dims,B,C,dt", [((1,), 1, 1, "f32"), ((1,), 1, 7, "bf16"), ((1,), 3, 3, "f32"),
                                         ((37, 41), 3, 5, "f32"), ((37, 41), 3, 5, "bf16"),
                                         ((64, 64), 2, 16, "bf16"), ((32, 16, 8), 2, 9, "f32")])
@pytest.mark.parametrize("p", [0.0, 2.0 ** -18, 0.1, 0.5, 0.999, 1.0])
def test_dropout_parity(dims, B, C, dt, p):
    r = np.random.default_rng(5)
    x = dev(r.standard_normal((B, C) + dims), dt)
    op = K.GridDropout(dims, B, C, io_dtype=dt, p=p)
    rng = rng_state() if op.drops else None
    m = O.drop_factors(SEED, OFFSET, p, tuple(x.shape))
    want = O.dropout(host(x), m)
    got = host(op(x, rng))
    close(got, want, np.abs(want), dt, 0, "y")
    np.testing.assert_array_equal(got == 0, (m == 0) | (host(x) == 0))
    close(host(op.backward(x, rng)), want, np.abs(want), dt, 0, "dx")


def test_dropout_of_infinities_and_nan():
    t = torch()
    x = t.full((1, 4, 33), float("nan"), device="cuda")
    x[:, 2:] = float("inf")
    m = O.drop_factors(SEED, OFFSET, 0.5, tuple(x.shape))
    got = host(K.GridDropout((33,), 1, 4, p=0.5)(x, rng_state()))
    assert (got[m == 0] == 0).all() and not np.isfinite(got[m > 0]).any()


def test_dropout_negative_state_words():
    """The state's 64 bits count as they stand, the sign bit too."""
    r = np.random.default_rng(6)
    x = dev(r.standard_normal((2, 3, 50)))
    got = host(K.GridDropout((50,), 2, 3, p=0.3)(x, rng_state(-5, -(1 << 63))))
    m = O.drop_factors(-5, -(1 << 63), 0.3, tuple(x.shape))
    np.testing.assert_array_equal(got == 0, m == 0)


def test_beyond_32_bits():
    """Elements past 2^32 bytes and past 2^31 indices: the tail of a large
    tensor, through dropout and the join (which share the index)."""
    t = torch()
    B, C, L = 1, 64, (1 << 25) + 72
    free, _ = t.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    x = t.empty(B, C, L, dtype=t.bfloat16, device="cuda").normal_()
    y = K.GridDropout((L,), B, C, io_dtype="bf16", p=0.3)(x, rng_state())
    first = (C - 1) * L + L - 1000
    m = O.drop_factors(SEED, OFFSET, 0.3, (1000,), first=first)
    tail = host(x[0, -1, -1000:])
    close(host(y[0, -1, -1000:]), tail * m, np.abs(tail * m), "bf16", 0, "tail")
    op = K.BlockJoin((L,), B, C, io_dtype="bf16", post="rms", pre="layer", p=0.3)
    h, n = op(x, y, rng=rng_state())
    cols = slice(L - 40, L)
    mm = np.stack([O.drop_factors(SEED, OFFSET, 0.3, (40,), first=c * L + L - 40) for c in range(C)])[None]
    none = dict.fromkeys(op.PARAMS)
    xv, yv = host(x[:, :, cols]), host(y[:, :, cols])
    wh, wn = O.join(xv, yv, mm, none, "rms", "layer", 1e-6)
    close(host(h[:, :, cols]), wh, np.abs(xv) + 4 * np.abs(wh - xv), "bf16", C, "h")
    close(host(n[:, :, cols]), wn, 8 + np.abs(wn), "bf16", C, "n")


# --------------------------------------------------------------------- ffn
class FfnCase:
    def __init__(self, dims, B, C, F, dt, act, seed=0):
        r = np.random.default_rng(seed + 77)
        self.B, self.C, self.F, self.dt, self.act = B, C, F, dt, act
        shape = (B, C) + tuple(dims)
        self.t = {"x": dev(r.standard_normal(shape), dt), "wg": dev(r.standard_normal((F, C)) / np.sqrt(C), dt),
                  "wu": dev(r.standard_normal((F, C)) / np.sqrt(C), dt),
                  "wd": dev(r.standard_normal((C, F)) / np.sqrt(F), dt), "dy": dev(r.standard_normal(shape), dt)}
        self.v = {k: host(t, B, C) if k in ("x", "dy") else host(t) for k, t in self.t.items()}
        self.op = K.GatedFFN(dims, B, C, F, io_dtype=dt, act=act)

    def run(self):
        w = [self.t[k] for k in ("wg", "wu", "wd")]
        return self.op(self.t["x"], *w), self.op.backward(self.t["x"], *w, self.t["dy"])

    def check(self, outs=None):
        y, (dx, dwg, dwu, dwd) = outs or self.run()
        assert self.op.status() == H.OK
        v, B, C, F = self.v, self.B, self.C, self.F
        q = O.ffn_terms(v["x"], v["wg"], v["wu"], v["wd"], v["dy"], self.act)
        a = {k: np.abs(t) for k, t in q.items()}
        W = {k: np.abs(v[k]) for k in ("wg", "wu", "wd")}
        T = q["X"].shape[1]
        # one rounding of each hidden value to the activations' type (bf16), fp32 sums of C terms before it
        half, acc = HALF_STEP[self.dt], lambda n: (80 + n / 8) * 2.0 ** -24  # noqa: E731
        eG, eU, eD = acc(C) * (W["wg"] @ a["X"]), acc(C) * (W["wu"] @ a["X"]), acc(C) * (W["wd"].T @ a["DY"])
        # |act'| <= 1.13, |act''| <= 1: what an error of G does to act and act'
        eH = half * a["H"] + eG * 1.13 * a["U"] + eU * a["a"] + 2.0 ** -20 * a["H"]
        eDG = half * a["DG"] + eD * a["U"] * np.abs(q["da"]) + eU * a["DH"] * np.abs(q["da"]) + eG * a["DH"] * a["U"] \
            + 2.0 ** -20 * a["DH"] * a["U"]
        eDU = half * a["DU"] + eD * a["a"] + eG * 1.13 * a["DH"] + 2.0 ** -20 * a["DU"]
        wy, (wdx, wdg, wdu, wdd) = (O.ffn(v["x"], v["wg"], v["wu"], v["wd"], self.act),
                                    O.ffn_backward(v["x"], v["wg"], v["wu"], v["wd"], v["dy"], self.act))
        wt, gt, ut = W["wd"], W["wg"].T, W["wu"].T
        err = {
            "y": O.uncols(wt @ eH + acc(F) * (wt @ a["H"]), B),
            "dx": O.uncols(gt @ eDG + ut @ eDU + acc(2 * F) * (gt @ a["DG"] + ut @ a["DU"]), B),
            "dwg": eDG @ a["X"].T + acc(T) * (a["DG"] @ a["X"].T),
            "dwu": eDU @ a["X"].T + acc(T) * (a["DU"] @ a["X"].T),
            "dwd": a["DY"] @ eH.T + acc(T) * (a["DY"] @ a["H"].T),
        }
        for k, got, want in (("y", y, wy), ("dx", dx, wdx), ("dwg", dwg, wdg), ("dwu", dwu, wdu), ("dwd", dwd, wdd)):
            g = host(got, B, C) if k in ("y", "dx") else host(got)
            tol = err[k] + half * 1.001 * (np.abs(want) + err[k]) + 1e-37
            bad = ~(np.abs(g - want) <= tol)
            assert not bad.any(), "%s: %d of %d off, worst %.3g of the tolerance" % (
                k, bad.sum(), bad.size, np.nanmax(np.abs(g - want) / tol))
            # the errors of independent roundings add up in squares: the norm is far below the bound
            rel = np.linalg.norm(g - want) / max(np.linalg.norm(want), 1e-300)
            assert rel <= {"bf16": 2.0 ** -8, "f32": 2.0 ** -20}[self.dt], (k, rel)


FFN = [
    # dims, B, C, F, dtype, act
    ((1,), 1, 8, 8, "bf16", "silu"),
    ((1,), 1, 8, 8, "f32", "gelu"),
    ((1,), 4, 256, 520, "bf16", "silu"),          # single tokens
    ((1,), 7, 264, 136, "f32", "silu"),
    ((1,), 16, 128, 512, "bf16", "gelu"),
    ((1,), 8, 2048, 40, "bf16", "silu"),
    ((1,), 9, 40, 2048, "f32", "gelu"),
    ((1,), 32, 264, 328, "bf16", "silu"),
    ((1,), 33, 264, 328, "bf16", "silu"),
    ((1,), 25, 72, 136, "f32", "silu"),
    ((2, 3), 4, 72, 104, "bf16", "gelu"),         # a few positions of short samples
    ((5,), 3, 136, 72, "f32", "silu"),
    ((32,), 1, 64, 96, "bf16", "silu"),
    ((1,), 17, 128, 512, "bf16", "gelu"),
    ((1,), 200, 72, 200, "bf16", "silu"),         # token-major
    ((1,), 130, 64, 264, "f32", "gelu"),
    ((3,), 5, 64, 96, "bf16", "silu"),            # short odd samples
    ((7,), 30, 64, 96, "bf16", "gelu"),
    ((8,), 20, 40, 72, "bf16", "silu"),
    ((8, 8), 2, 64, 128, "bf16", "silu"),
    ((8, 8), 2, 64, 128, "f32", "silu"),
    ((16, 24), 2, 136, 344, "bf16", "gelu"),
    ((37, 41), 2, 24, 40, "bf16", "silu"),        # odd rows
    ((37, 41), 1, 24, 40, "f32", "gelu"),
    ((777,), 3, 200, 536, "bf16", "gelu"),
    ((130,), 2, 200, 264, "f32", "silu"),
    ((1000,), 1, 256, 1024, "bf16", "silu"),
    ((16, 16, 16), 1, 64, 256, "f32", "gelu"),
    ((64, 32), 2, 512, 640, "bf16", "silu"),
    ((2056,), 1, 8, 1032, "bf16", "silu"),        # few channels, many hidden
    ((1,), 40, 24, 2088, "f32", "silu"),          # few tiles, long sums: their depth is split
    ((1,), 40, 72, 2088, "bf16", "gelu"),
    ((50,), 2, 64, 2056, "bf16", "silu"),
    ((256,), 2, 40, 2560, "bf16", "silu"),
    ((30,), 3, 40, 1112, "f32", "gelu"),
    ((72,), 2, 1032, 8, "bf16", "gelu"),
]


@pytest.mark.parametrize("dims,B,C,F,dt,act", FFN)
def test_ffn_parity(dims, B, C, F, dt, act):
    FfnCase(dims, B, C, F, dt, act).check()


def test_ffn_repeats_bit_for_bit():
    t = torch()
    for dims, B, dt in (((64, 64), 1, "bf16"), ((1,), 3, "bf16"), ((777,), 1, "bf16"), ((64,), 2, "f32")):
        c = FfnCase(dims, B, 128, 256, dt, "silu")
        (y1, g1), (y2, g2) = c.run(), c.run()
        assert t.equal(y1, y2) and all(t.equal(a, b) for a, b in zip(g1, g2))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_ffn_extreme_gates(dt):
    """Gates far outside the range of exp: act is 0 or the gate itself, its slope 0 or 1."""
    for act in ("silu", "gelu"):
        c = FfnCase((24,), 2, 16, 32, dt, act)
        c.t["wg"].mul_(2000)
        c.v["wg"] = host(c.t["wg"])
        c.check()


@pytest.mark.parametrize("gate", [1e3, 1e15, 1e20, 1e30, 3e38])
@pytest.mark.parametrize("dims,dt", [((1,), "bf16"), ((40,), "bf16"), ((1,), "f32"), ((40,), "f32")])
def test_ffn_gates_of_any_size(dims, dt, gate):
    """silu(g) and its slope are 0 at g = -gate (below 1e-400), however large the gate: the sigmoid has to be 0
    there, not small, since g multiplies it.  Every other hidden channel has g = 0, act 0 and slope 1/2, so that
    only dwg has values: its odd rows, (sum of wd) / 2 at each position.  All of them are exact in bf16; fp32's
    reciprocal is off by 2^-22 at most."""
    C = F = 8
    L = int(np.prod(dims))
    x = np.zeros((1, C) + dims)
    x[:, 0] = 1
    wg, wu, wd = np.zeros((F, C)), np.zeros((F, C)), np.ones((C, F))
    wg[::2, 0] = -gate
    wu[:, 0] = 1
    x, wg, wu, wd, dy = (dev(v, dt) for v in (x, wg, wu, wd, np.ones((1, C) + dims)))
    op = K.GatedFFN(dims, 1, C, F, io_dtype=dt, act="silu")
    y = op(x, wg, wu, wd)
    dx, dwg, dwu, dwd = (host(v) for v in op.backward(x, wg, wu, wd, dy))
    assert op.status() == H.OK
    want = np.zeros((F, C))
    want[1::2, 0] = C / 2 * L
    for name, got in (("y", host(y)), ("dx", dx), ("dwu", dwu), ("dwd", dwd)):
        assert (got == 0).all(), (name, np.abs(got).max())
    assert (np.abs(dwg - want) <= 2.0 ** -22 * want).all()


def _single_gates(dims, dt, kind, gates, act, slope, slopes, tol):
    """One gate a hidden channel, u = 2^13, Wd the unit matrix: every result but dx is a single term of the formula at
    each position.  act and its slope at the gates, magnitudes of the slope's terms, tol relative to the terms."""
    C = F = gates.size
    L, u = int(np.prod(dims)), 2.0 ** 13
    x = np.zeros((1, C) + dims)
    x[:, 0] = 1
    wg, wu = np.zeros((F, C)), np.zeros((F, C))
    wg[:, 0], wu[:, 0] = gates, u
    x, wg, wu, wd, dy = (dev(v, dt) for v in (x, wg, wu, np.eye(C), np.ones((1, C) + dims)))
    op = K.GatedFFN(dims, 1, C, F, io_dtype=dt, act=kind)
    y = host(op(x, wg, wu, wd), 1, C)
    dx, dwg, dwu, dwd = (host(v) for v in op.backward(x, wg, wu, wd, dy))
    assert op.status() == H.OK
    for name, got, want, mag in (("y", y[0].T, act * u, act * u), ("dwg", dwg[:, 0], slope * u * L, slopes * u * L),
                                 ("dwu", dwu[:, 0], act * L, act * L), ("dwd", np.diag(dwd), act * u * L, act * u * L)):
        off = np.abs(got - want) / np.abs(mag)
        assert (off <= tol * 1.001).all(), (name, off / tol)
    # the first channel's dx sums over the hidden channels
    want, mag = gates * slope * u + u * act, np.abs(gates) * slopes * u + np.abs(u * act)
    assert (np.abs(dx[0, 0] - want.sum()) <= (tol * mag).sum() + HALF_STEP[dt] * 1.001 * abs(want.sum())).all()


SINGLE = [((1,), "bf16"), ((40,), "bf16"), ((1,), "f32"), ((40,), "f32")]


@pytest.mark.parametrize("dims,dt", SINGLE)
def test_ffn_gelu_far_below_zero(dims, dt):
    """gelu(g) = g Phi(g) keeps its relative accuracy where Phi(g) is small, as g u may be large.  With bf16 the
    hidden value and the stored result are rounded, half a step each, and Phi is good to 2^-13; fp32 functions are off
    by a few steps, an argument by 2^-23, which moves exp(-g^2/2) by g^2 2^-23 of itself; 40 more steps of 2^-24 for
    the sums of planes and of the positions.  The slope is a difference above -0.75: its tolerance is relative to both
    terms."""
    import math

    gates = host(dev(np.linspace(-12.5, 12.5, 64), "bf16"))
    phi = np.array([0.5 * math.erfc(-g / math.sqrt(2)) for g in gates])
    bell = gates * np.exp(-0.5 * gates ** 2) / math.sqrt(2 * math.pi)
    tol = (2 * HALF_STEP["bf16"] + 2.0 ** -13 if dt == "bf16" else 0) + (gates ** 2 + 40) * 2.0 ** -23
    _single_gates(dims, dt, "gelu", gates, gates * phi, phi + bell, phi + np.abs(bell), tol)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("dims", [(1,), (33,)])
def test_ffn_gelu_where_its_slope_is_zero(dims, dt):
    """gelu's slope crosses zero near -0.7518: what its error is there, is to the terms of Phi + g phi no more than
    elsewhere.  One gate a hidden channel around the crossing, one for all positions."""
    import math

    gates = host(dev(np.linspace(-0.8, -0.7, 64), dt))
    phi = np.array([0.5 * math.erfc(-g / math.sqrt(2)) for g in gates])
    bell = gates * np.exp(-0.5 * gates ** 2) / math.sqrt(2 * math.pi)
    C = F = gates.size
    x = np.zeros((1, C) + dims)
    x[:, 0] = 1
    wg, wu = np.zeros((F, C)), np.zeros((F, C))
    wg[:, 0], wu[:, 0] = gates, 1
    x, wg, wu, wd, dy = (dev(v, dt) for v in (x, wg, wu, np.eye(C), np.ones((1, C) + dims)))
    got = host(K.GatedFFN(dims, 1, C, F, io_dtype=dt, act="gelu").backward(x, wg, wu, wd, dy)[1])[:, 0]
    L, want = int(np.prod(dims)), phi + bell
    # the slope and its sum over L equal terms are rounded, each half a step of itself (bf16); 16 steps of 2^-24 of the
    # slope's terms and L / 8 + 16 of the sum's for the arithmetic
    tol = (2 * HALF_STEP[dt] * 1.01 + (L / 8 + 16) * 2.0 ** -24) * np.abs(want) + 16 * 2.0 ** -24 * (phi - bell)
    assert (np.abs(got / L - want) <= tol).all(), np.abs(got / L - want) / tol


@pytest.mark.parametrize("dims,dt", SINGLE)
def test_ffn_silu_far_below_zero(dims, dt):
    """silu(g) = g s, s = 1 / (1 + exp(-g)), keeps its relative accuracy where s is small.  Roundings as above; the
    exponential's argument is off by 2^-23 of itself."""
    gates = host(dev(np.linspace(-60.0, 60.0, 64), "bf16"))
    s = 1.0 / (1.0 + np.exp(-gates))
    bend = gates * s * (1.0 / (1.0 + np.exp(gates)))
    tol = (2 * HALF_STEP["bf16"] if dt == "bf16" else 0) + (np.abs(gates) + 40) * 2.0 ** -23
    _single_gates(dims, dt, "silu", gates, gates * s, s + bend, s + np.abs(bend), tol)


def test_ffn_weight_gradients_over_a_million_positions():
    """The tensor cores cut what they add to an accumulator, which is off by as much as 2^-23 of the sum an addition
    and always the same way; no loop may be so deep that this shows next to bf16's 2^-8.  Gates of 64, where silu is
    the gate itself and its slope 1, one channel of x that is 1 and one row of Wd: the gradients are 2^20 equal terms,
    known exactly.  A sum that grows evenly loses half of 2^-23 an addition: 2^-12 in 4096, the most of a loop, and
    2^-11 on average is allowed for a product of 16 that is added in two steps."""
    t = torch()
    C, F, L = 1024, 1536, 1 << 20
    if t.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB of device memory")
    r = np.random.default_rng(4)
    u, d = (host(dev(1 + r.random(n), "bf16")) for n in (F, C))
    wg, wu, wd = np.zeros((F, C)), np.zeros((F, C)), np.zeros((C, F))
    wg[:, 0], wu[:, 0], wd[0] = 64, u, 1
    x = t.zeros(1, C, L, dtype=t.bfloat16, device="cuda")
    x[:, 0] = 1
    dy = dev(d, "bf16").view(1, C, 1).expand(1, C, L).contiguous()
    op = K.GatedFFN((L,), 1, C, F, io_dtype="bf16", act="silu")
    _, dwg, dwu, dwd = op.backward(x, *(dev(v, "bf16") for v in (wg, wu, wd)), dy)
    assert op.status() == H.OK
    stored = lambda v: host(dev(v, "bf16"))  # noqa: E731  (one rounding of exact products of 16 bits)
    for name, got, want in (("dwg", dwg[:, 0], stored(d[0] * u) * L), ("dwu", dwu[:, 0], stored(np.full(F, 64 * d[0])) * L),
                            ("dwd", dwd, 64.0 * L * d[:, None] * u[None, :])):
        off = host(got) / want - 1
        assert np.abs(off).max() <= HALF_STEP["bf16"] * 1.01 + 2.0 ** -12, (name, off.min(), off.max())
        if name == "dwd":
            assert abs(off.mean()) <= 2.0 ** -11, off.mean()


@pytest.mark.parametrize("dims,B,C,F,dt", [(((1 << 28) + 8,), 1, 8, 16, "bf16"), (((1 << 27) + 5,), 2, 8, 16, "bf16"),
                                           ((1,), (1 << 28) - 5, 8, 16, "bf16"), (((1 << 26) + 7,), 1, 8, 40, "f32")])
def test_ffn_beyond_32_bits(dims, B, C, F, dt):
    """Activations and hidden values past 2^31 elements: the last positions, against the oracle on them alone."""
    t = torch()
    t.cuda.empty_cache()
    if t.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("needs 120 GB of device memory")
    c = FfnCase((40,), 1, C, F, dt, "silu")
    w = [c.t[k] for k in ("wg", "wu", "wd")]
    x, dy = (t.empty((B, C) + dims, dtype=c.t["x"].dtype, device="cuda").normal_() for _ in range(2))
    op = K.GatedFFN(dims, B, C, F, io_dtype=dt)
    y = op(x, *w)
    n = 40 if dims != (1,) else 1

    def tail(v):
        return host(v[-1:, :, -n:] if n > 1 else v[-40:], 1 if n > 1 else 40, C)

    V = c.v
    q = O.ffn_terms(tail(x), V["wg"], V["wu"], V["wd"], tail(dy), "silu")
    want = O.ffn(tail(x), V["wg"], V["wu"], V["wd"], "silu")
    mag = O.uncols(np.abs(V["wd"]) @ np.abs(q["H"]), want.shape[0])
    step = 3 * HALF_STEP[dt] + 2.0 ** -18          # hidden value, result; fp32 arithmetic of the planes
    assert (np.abs(tail(y) - want) <= step * mag + 1e-37).all()
    del y
    dx = op.backward(x, *w, dy)[0]
    assert op.status() == H.OK
    want = O.ffn_backward(tail(x), V["wg"], V["wu"], V["wd"], tail(dy), "silu")[0]
    mag = np.abs(V["wg"]).T @ (np.abs(q["DH"] * q["U"]) * 1.2) + np.abs(V["wu"]).T @ np.abs(q["DU"])
    assert (np.abs(tail(dx) - want) <= step * O.uncols(mag, want.shape[0]) + 1e-37).all()


@pytest.mark.parametrize("dims", [(1,), (40,), (7,)])
def test_ffn_nan_stays_in_its_position(dims):
    c = FfnCase(dims, 3, 64, 96, "bf16", "silu")
    c.t["x"].view(3, 64, -1)[1, 5, 0] = float("nan")
    y = host(c.op(c.t["x"], c.t["wg"], c.t["wu"], c.t["wd"]), 3, 64)
    bad = np.isnan(y)
    assert bad[1, :, 0].all()
    bad[1, :, 0] = False
    assert not bad.any()


@pytest.mark.parametrize("dims,B,C,F,dt", [((1,), 40, 24, 2088, "f32"), ((1,), 3, 24, 40, "f32"),
                                           ((8, 8), 2, 64, 136, "f32"), ((37,), 3, 40, 72, "f32"),
                                           ((37,), 3, 40, 72, "bf16"), ((8, 8), 2, 64, 136, "bf16"),
                                           ((1,), 3, 24, 40, "bf16"), ((1,), 40, 24, 2088, "bf16")])
def test_ffn_pointers_on_16_bytes(dims, B, C, F, dt):
    """Every buffer of the C calls at 16 modulo 32, the least they ask for: the results are those of torch's own
    buffers, and nothing beside a buffer changes, the workspace's exact size included."""
    import ctypes

    t = torch()
    c = FfnCase(dims, B, C, F, dt, "gelu")
    want_y, want_g = c.run()
    held = []

    def room(nbytes):
        """nbytes at 16 modulo 32, in the middle of a buffer of sevens."""
        buf = t.full((nbytes + 512,), 7, dtype=t.uint8, device="cuda")
        at = 128 + (16 - buf.data_ptr()) % 32
        assert (buf.data_ptr() + at) % 32 == 16
        held.append((buf, at, nbytes))
        return buf[at:at + nbytes]

    def placed(v):
        r = room(v.numel() * v.element_size())
        r.copy_(v.reshape(-1).view(t.uint8))
        return r

    ins = [placed(c.t[k]) for k in ("x", "wg", "wu", "wd")]
    dy, control = placed(c.t["dy"]), placed(t.zeros(256, dtype=t.uint8, device="cuda"))
    y, *g = (room(v.numel() * v.element_size()) for v in (want_y, *want_g))
    stream, f = t.cuda.current_stream().cuda_stream, ctypes.byref(c.op.f)
    need = c.op.ws_bytes
    ptr = lambda *v: [b.data_ptr() for b in v]  # noqa: E731
    assert K.load().hyena_nd_ffn_forward(f, *ptr(*ins, y, control, room(need[0])), need[0], stream) == H.OK
    assert K.load().hyena_nd_ffn_backward(f, *ptr(*ins, dy, *g, control, room(need[1])), need[1], stream) == H.OK
    assert H.device_status(control.data_ptr(), stream) == H.OK
    for got, want in zip((y, *g), (want_y, *want_g)):
        assert t.equal(got.view(want.dtype), want.reshape(-1))
    for buf, at, n in held:
        assert (buf[:at] == 7).all() and (buf[at + n:] == 7).all()


# ------------------------------------------------------- streams and graphs
def test_ffn_control_is_set_up_before_the_object_is_used():
    """The status word is cleared by the time the constructor returns: a code that a call on another stream records
    stays, however late the constructing stream gets to its work."""
    t = torch()
    late, other = t.cuda.Stream(), t.cuda.Stream()
    with t.cuda.stream(late):      # memory and kernels are there: nothing below waits for either
        t.zeros(256, dtype=t.uint8, device="cuda")
        t.zeros(64, dtype=t.int32, device="cuda")[0].fill_(H.ERR_DEVICE_TIMEOUT)
        t.cuda._sleep(1)
    t.cuda.synchronize()
    with t.cuda.stream(late):
        t.cuda._sleep(100_000_000)          # some 50 ms
        op = K.GatedFFN((8,), 1, 8, 8)
    with t.cuda.stream(other):
        op.control.view(t.int32)[0].fill_(H.ERR_DEVICE_TIMEOUT)      # as a kernel would
    t.cuda.synchronize()
    assert op.status() == H.ERR_DEVICE_TIMEOUT
    assert op.status() == H.OK               # read and cleared


def test_two_streams_share_an_object():
    t = torch()
    c = FfnCase((32, 32), 2, 64, 256, "bf16", "silu")
    x2 = c.t["x"].flip(0).contiguous()
    w = [c.t[k] for k in ("wg", "wu", "wd")]
    want1, want2 = c.op(c.t["x"], *w), c.op(x2, *w)
    s1, s2 = t.cuda.Stream(), t.cuda.Stream()
    t.cuda.synchronize()
    got = []
    for _ in range(10):
        with t.cuda.stream(s1):
            a = c.op(c.t["x"], *w)
        with t.cuda.stream(s2):
            b = c.op(x2, *w)
        got.append((a, b))
    t.cuda.synchronize()
    assert all(t.equal(a, want1) and t.equal(b, want2) for a, b in got)


def test_host_threads_share_objects():
    """Two threads, each on a stream of its own and with a generator state of its own, call the same objects; another
    object is made meanwhile in each."""
    import threading

    t = torch()
    c = JoinCase((64,), 3, 72, "bf16", "rms", "layer", "wbgs", 0.3)
    f = FfnCase((64,), 3, 72, 136, "f32", "gelu")
    drop = K.GridDropout((64,), 3, 72, io_dtype="bf16", p=0.4)
    w = [f.t[k] for k in ("wg", "wu", "wd")]
    states = [rng_state(5, 6), rng_state(7, 8)]

    def step(rng):
        h, n = c.op(c.t["x"], c.t["y"], rng=rng)
        g = c.op.backward(c.t["x"], c.t["y"], c.t["dh"], c.t["dn"], rng=rng)
        own = K.GatedFFN((64,), 3, 72, 136, io_dtype="f32", act="gelu")
        return [h, n, drop(n, rng)] + [g[k] for k in sorted(g)] + [f.op(f.t["x"], *w), own(f.t["x"], *w)] \
            + list(f.op.backward(f.t["x"], *w, f.t["dy"]))

    want = [step(s) for s in states]
    t.cuda.synchronize()
    wrong, done = [], []

    def work(i):
        with t.cuda.stream(t.cuda.Stream()):
            for _ in range(20):
                got = step(states[i])
                t.cuda.current_stream().synchronize()
                if not all(t.equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append(i)
        done.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert sorted(done) == [0, 1] and not wrong and not t.equal(want[0][0], want[1][0]) and f.op.status() == H.OK


def test_graphs_follow_the_generator_state():
    """A captured forward and backward replays with the state's new values;
    two graphs of one object do not share scratch."""
    t = torch()
    c = JoinCase((64,), 2, 40, "f32", "layer", "rms", "wbgs", 0.3)
    f = FfnCase((64,), 2, 40, 64, "bf16", "silu")
    w = [f.t[k] for k in ("wg", "wu", "wd")]

    def step():
        h, n = c.op(c.t["x"], c.t["y"], rng=c.rng)
        g = c.op.backward(c.t["x"], c.t["y"], c.t["dh"], c.t["dn"], rng=c.rng)
        return [h, n] + [g[k] for k in sorted(g)] + [f.op(f.t["x"], *w)] + list(f.op.backward(f.t["x"], *w, f.t["dy"]))

    step()
    t.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    for k in range(3):
        c.rng.add_(k)
        want = [v.clone() for v in step()]
        t.cuda.synchronize()
        s1, s2 = t.cuda.Stream(), t.cuda.Stream()
        with t.cuda.stream(s1):
            graphs[0][0].replay()
        with t.cuda.stream(s2):
            graphs[1][0].replay()
        t.cuda.synchronize()
        for _, out in graphs:
            assert all(t.equal(a, b) for a, b in zip(out, want))
    assert f.op.status() == H.OK


# ------------------------------------------------------------ a whole block
@pytest.mark.parametrize("dims", [(16, 16), (64,)])
def test_a_block_runs_forward_and_backward(dims):
    """norm -> convolution -> join -> feed-forward -> join -> dropout, and all
    the way back, against the oracle.  fp32: each stage is within 1e-5 of the
    oracle in norm (the convolution's own parity), five stages in a row."""
    from oracle import hyena_nd_oracle as HO
    from dimensional_long_convolution_b200 import workloads as W

    t = torch()
    B, C, F = 2, 16, 32
    wl = W.custom(dims, B, C, io_dtype="f32", seed=11)
    inp = W.make_inputs(wl)
    conv = H.HyenaND(dims, B, C, "f32")
    f = inp.filt
    conv.set_filter(*(t.from_numpy(a) for a in (f.W1, f.b1, f.W2, f.b2, f.alpha)), f.decay_scale, f.num_freqs)
    j1 = JoinCase(dims, B, C, "f32", "rms", "layer", "wbgs", 0.2, seed=1)
    j2 = JoinCase(dims, B, C, "f32", "none", "rms", "ws", 0.0, seed=2)
    ff = FfnCase(dims, B, C, F, "f32", "silu")
    drop = K.GridDropout(dims, B, C, p=0.25)
    w = [ff.t[k] for k in ("wg", "wu", "wd")]
    x, dy = j1.t["x"], j1.t["dh"]
    rng2 = rng_state(99, 1)

    n0 = j1.op.norm(x)
    mix = conv(n0, n0, n0)
    h1, n1 = j1.op(x, mix, rng=j1.rng)
    y2 = ff.op(n1, *w)
    h2, n2 = j2.op(h1, y2)
    out = drop(n2, rng2)
    dn2 = drop.backward(dy, rng2)
    g2 = j2.op.backward(h1, y2, None, dn2)
    dn1, dwg, dwu, dwd = ff.op.backward(n1, *w, g2["dy"])
    g1 = j1.op.backward(x, mix, g2["dx"], dn1, rng=j1.rng)
    dq, dk, dv = conv.backward(n0, n0, n0, g1["dy"])
    g0 = j1.op.norm_backward(x, dq + dk + dv)
    dx = g0["dx"] + g1["dx"]
    assert conv.status() == H.OK and ff.op.status() == H.OK

    # the same in 64 bits
    xv, dyv, P1, P2 = host(x, B, C), host(dy, B, C), j1.P, j2.P
    V = ff.v
    on0 = O.norm(xv, "layer", P1["pre_w"], P1["pre_b"], 1e-6)

    S = HO.spectrum_full(HO.implicit_kernel(f, dims), dims)

    def grid(v):
        return v.reshape((B, C) + dims)

    omix = HO.conv_dft(grid(on0), grid(on0), grid(on0), S, dims).reshape(B, C, -1)
    oh1, on1 = O.join(xv, omix, j1.m, P1, "rms", "layer", 1e-6)
    oy2 = O.ffn(on1, V["wg"], V["wu"], V["wd"], "silu")
    one = np.ones(xv.shape)
    oh2, on2 = O.join(oh1, oy2, one, P2, "none", "rms", 1e-6)
    m2 = O.drop_factors(99, 1, 0.25, xv.shape)
    odn2 = dyv * m2
    og2 = O.join_backward(oh1, oy2, one, P2, "none", "rms", 1e-6, None, odn2)
    odn1, odwg, odwu, odwd = O.ffn_backward(on1, V["wg"], V["wu"], V["wd"], og2["dy"], "silu")
    og1 = O.join_backward(xv, omix, j1.m, P1, "rms", "layer", 1e-6, og2["dx"], odn1)
    odn0 = sum(HO.backward_dft(*[grid(on0)] * 3, grid(og1["dy"]), S, dims)).reshape(B, C, -1)
    odx, odw0 = O.norm_backward(xv, "layer", P1["pre_w"], odn0, 1e-6)[:2]
    odx = odx + og1["dx"]
    for name, got, want in (("out", host(out, B, C), on2 * m2), ("dx", host(dx, B, C), odx),
                            ("dwg", host(dwg), odwg), ("dwu", host(dwu), odwu), ("dwd", host(dwd), odwd),
                            ("dgate", host(g1["dgate"]), og1["dgate"]), ("dscale", host(g2["dscale"]), og2["dscale"]),
                            ("dpost_w", host(g1["dpost_w"]), og1["dpost_w"]),
                            ("dpre_w", host(g0["dpre_w"]), odw0)):
        rel = np.linalg.norm(got - want) / np.linalg.norm(want)
        assert rel < 5e-5, (name, rel)
