"""float64 CPU oracle of the operators around the convolution: the residual
join with its norms, counter-based dropout and the gated feed-forward block,
with their gradients.  Written from the formulas; shares no code with the GPU
path.  Activations are numpy arrays [B, C, L]."""
from __future__ import annotations

import math

import numpy as np

U64 = np.uint64
LOW = U64(0xFFFFFFFF)


def philox(counter, key):
    """Philox4x32-10 (Salmon et al. 2011): four uint64 arrays holding 32-bit
    counter words, two key words -> four arrays of 32-bit words."""
    c = [np.asarray(v, dtype=U64) for v in counter]
    k = [int(v) for v in key]
    for _ in range(10):
        a, b = U64(0xD2511F53) * c[0], U64(0xCD9E8D57) * c[2]
        c = [(b >> U64(32)) ^ c[1] ^ U64(k[0]), b & LOW, (a >> U64(32)) ^ c[3] ^ U64(k[1]), a & LOW]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def lots(seed: int, offset: int, first: int, count: int):
    """16-bit lots of elements first .. first + count - 1."""
    i = np.arange(first, first + count, dtype=U64)
    g = i >> U64(3)
    seed, offset = seed % (1 << 64), offset % (1 << 64)
    o = np.full_like(g, offset & 0xFFFFFFFF), np.full_like(g, offset >> 32)
    w = philox([g & LOW, g >> U64(32), o[0], o[1]], [seed & 0xFFFFFFFF, seed >> 32])
    j = (i & U64(7)).astype(np.int64)
    word = np.choose(j // 2, w)
    return np.where(j % 2 == 1, word >> U64(16), word & U64(0xFFFF)).astype(np.int64)


def border(p: float) -> int:
    return math.floor(p * 65536 + 0.5)


def drop_factors(seed, offset, p, shape, first=0):
    """The factor of each element: 0 or 65536 / (65536 - border)."""
    t = border(p)
    n = int(np.prod(shape))
    if t == 0:
        return np.ones(shape)
    if t == 65536:
        return np.zeros(shape)
    return np.where(lots(seed, offset, first, n) >= t, 65536.0 / (65536 - t), 0.0).reshape(shape)


def dropout(x, m):
    return np.where(m > 0, x, 0.0) * m


def stats(v, kind, eps):
    """(vhat, rho) over axis 1."""
    mu = v.mean(1, keepdims=True) if kind == "layer" else 0.0
    d = v - mu
    rho = 1.0 / np.sqrt((d * d).mean(1, keepdims=True) + eps)
    return d * rho, rho


def _col(v):
    return v[None, :, None]


def norm(v, kind, w, b, eps):
    if kind == "none":
        return v
    vhat, _ = stats(v, kind, eps)
    return vhat * (1.0 if w is None else _col(w)) + (0.0 if b is None else _col(b))


def hat_magnitude(vhat, rho, mv):
    """Magnitudes of vhat's terms where v's terms have magnitudes mv: vhat =
    (v - mean) rho carries an error e mv of v as e rho (mv + mean mv), and one
    of rho, whose relative size is the mean of |vhat| times the former."""
    hm = rho * (mv + mv.mean(1, keepdims=True))
    return hm + np.abs(vhat) * (np.abs(vhat) * hm).mean(1, keepdims=True)


def norm_backward(v, kind, w, dn, eps, mv=None, mdn=None):
    """dv, dw, db, and the magnitudes of their terms where v and dn are sums
    of terms of magnitudes mv and mdn."""
    mv, mdn = np.abs(v) if mv is None else mv, np.abs(dn) if mdn is None else mdn
    if kind == "none":
        return dn, None, None, mdn, None, None
    vhat, rho = stats(v, kind, eps)
    hm = hat_magnitude(vhat, rho, mv)
    a, ma = (t * (1.0 if w is None else np.abs(_col(w)) if t is mdn else _col(w)) for t in (dn, mdn))
    m1 = a.mean(1, keepdims=True) if kind == "layer" else 0.0
    m2 = (a * vhat).mean(1, keepdims=True)
    off = 1.0 + (np.abs(vhat) * hm).mean(1, keepdims=True)          # of rho
    mag = rho * off * (ma + ma.mean(1, keepdims=True) + hm * (ma * hm).mean(1, keepdims=True))
    return (rho * (a - m1 - vhat * m2), (dn * vhat).sum((0, 2)), dn.sum((0, 2)), mag, (mdn * hm).sum((0, 2)),
            mdn.sum((0, 2)))


def join(x, y, m, P, post, pre, eps):
    """h, n; P: dict of post_w, post_b, gate, scale, pre_w, pre_b (None: absent)."""
    z = norm(np.where(m > 0, y, np.where(np.isfinite(y), y, 0.0)), post, P["post_w"], P["post_b"], eps)
    s = 1.0
    if P["gate"] is not None:
        s = s * P["gate"][:, :, None]
    if P["scale"] is not None:
        s = s * _col(P["scale"])
    h = x + s * m * z
    return h, (None if pre == "none" else norm(h, pre, P["pre_w"], P["pre_b"], eps))


def join_backward(x, y, m, P, post, pre, eps, dh, dn):
    """Gradients by name, and under "mag_" + name the magnitudes of the terms summed in them."""
    one = np.ones(x.shape)
    g = one * (1.0 if P["gate"] is None else P["gate"][:, :, None])
    sc = one * (1.0 if P["scale"] is None else _col(P["scale"]))
    w1 = 1.0 if P["post_w"] is None else _col(P["post_w"])
    b1 = 0.0 if P["post_b"] is None else _col(P["post_b"])
    yhat, ym = y, np.abs(y)
    if post != "none":
        yhat, rho = stats(y, post, eps)
        ym = hat_magnitude(yhat, rho, ym)
    z = w1 * yhat + b1
    # z is itself a sum: an error e of yhat moves it by e |w1| however small z is
    zm = np.abs(w1) * ym + np.abs(b1)
    h = x + g * sc * m * z
    hm = np.abs(x) + np.abs(g * sc) * m * zm
    d = np.zeros(x.shape) if dh is None else dh
    mag = np.abs(d)
    out = {}
    if pre != "none":
        dv, dw, db, vm, mw, mb = norm_backward(h, pre, P["pre_w"], dn, eps, hm)
        d, mag = d + dv, mag + vm
        out["dpre_w"], out["dpre_b"], out["mag_dpre_w"], out["mag_dpre_b"] = dw, db, mw, mb
    out["dx"], out["mag_dx"] = d, mag
    dz, mz = d * g * sc * m, mag * np.abs(g * sc * m)
    dy, dw, db, my, mw, mb = norm_backward(y, post, P["post_w"], dz, eps, None, mz)
    out["dy"], out["mag_dy"] = dy, my
    if post != "none":
        out["dpost_w"], out["dpost_b"], out["mag_dpost_w"], out["mag_dpost_b"] = dw, db, mw, mb
    each, meach = (d * m * z).sum(2), (mag * m * zm).sum(2)
    out["dgate"], out["mag_dgate"] = each * sc[:, :, 0], meach * np.abs(sc[:, :, 0])
    out["dscale"], out["mag_dscale"] = (each * g[:, :, 0]).sum(0), (meach * np.abs(g[:, :, 0])).sum(0)
    return out


_erf = np.vectorize(math.erf, otypes=[float])


def act(g, kind):
    """The activation and its derivative."""
    if kind == "silu":
        s = np.where(g >= 0, 1.0 / (1.0 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1.0 + np.exp(-np.abs(g))))
        return g * s, s * (1.0 + g * (1.0 - s))
    cdf = 0.5 * (1.0 + _erf(g / math.sqrt(2.0)))
    return g * cdf, cdf + g * np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)


def cols(v):
    """[B, C, L] -> [C, B L]."""
    return v.transpose(1, 0, 2).reshape(v.shape[1], -1)


def uncols(v, B):
    return v.reshape(v.shape[0], B, -1).transpose(1, 0, 2)


def ffn(x, wg, wu, wd, kind):
    X = cols(x)
    H = act(wg @ X, kind)[0] * (wu @ X)
    return uncols(wd @ H, x.shape[0])


def ffn_terms(x, wg, wu, wd, dy, kind):
    """Everything of the two passes, as [channels, positions] matrices."""
    X, DY = cols(x), cols(dy)
    G, U = wg @ X, wu @ X
    a, da = act(G, kind)
    DH = wd.T @ DY
    DG, DU = DH * U * da, DH * a
    return {"X": X, "DY": DY, "G": G, "U": U, "H": a * U, "DH": DH, "DG": DG, "DU": DU, "a": a, "da": da}


def ffn_backward(x, wg, wu, wd, dy, kind):
    t = ffn_terms(x, wg, wu, wd, dy, kind)
    return (uncols(wg.T @ t["DG"] + wu.T @ t["DU"], x.shape[0]), t["DG"] @ t["X"].T, t["DU"] @ t["X"].T,
            t["DY"] @ t["H"].T)
