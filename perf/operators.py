"""What is timed of the operators around the long convolution of a block.

A block of this framework mixes a [B, C, *grid] activation with the gated long
convolution.  The operators here are the rest of such a block on the same
layout:

* join     the residual join after a mixer with the norms on both sides of it:
           h = x + scale_c gate_bc drop(norm_post(y)),  n = norm_pre(h)
* dropout  inverted dropout whose mask comes from a counter (Philox4x32-10)
           and is recomputed wherever it is needed
* ffn      the gated feed-forward block  Wd (act(Wg x) * (Wu x))  over channels

Each runs forward, and forward with its backward pass ("train").  ``own``
chooses between the plain form and the framework's kernels.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # the join of a 2D vision token grid in training: layer norms, adaptive gate, layer scale, dropout
        dict(name="join 64x64 f32 train", op="join", grid="64x64", B=8, C=256, dtype="f32", train=True,
             post="layer", pre="layer", affine=True, gate=True, scale=True, p=0.1),
        # high-resolution images being served: RMS norms, layer scale, no dropout
        dict(name="join 256x256 bf16", op="join", grid="256x256", B=2, C=128, dtype="bf16", train=False,
             post="rms", pre="rms", affine=True, gate=False, scale=True, p=0.0),
        # ragged 1D sequences in training: no axis is a multiple of anything
        dict(name="join 777 bf16 train", op="join", grid="777", B=13, C=204, dtype="bf16", train=True,
             post="rms", pre="layer", affine=True, gate=True, scale=False, p=0.25),
        # one token of each of 16 sequences, as when a model is stepped: latency counts
        dict(name="join 1 token bf16", op="join", grid="1", B=16, C=1024, dtype="bf16", train=False,
             post="rms", pre="rms", affine=True, gate=True, scale=True, p=0.0),
        # a large volume's activations: the streaming rate
        dict(name="dropout 128x128x128 bf16", op="dropout", grid="128x128x128", B=1, C=32, dtype="bf16",
             train=False, p=0.1),
        # a small odd image, forward and backward
        dict(name="dropout 37x41 f32 train", op="dropout", grid="37x41", B=3, C=5, dtype="f32", train=True, p=0.5),
        # the channel mixer of the 2D vision grid being served
        dict(name="ffn 64x64 bf16", op="ffn", grid="64x64", B=8, C=256, F=1024, dtype="bf16", train=False, act="silu"),
        # the same in training
        dict(name="ffn 64x64 bf16 train", op="ffn", grid="64x64", B=8, C=256, F=1024, dtype="bf16", train=True,
             act="silu"),
        # a wide model on long sequences in training: the matrix products decide
        dict(name="ffn 4096 wide bf16 train", op="ffn", grid="4096", B=2, C=2048, F=5632, dtype="bf16", train=True,
             act="silu"),
        # one token of each of 4 sequences through the wide model: the weights are read once
        dict(name="ffn 1 token bf16", op="ffn", grid="1", B=4, C=2048, F=5632, dtype="bf16", train=False, act="silu"),
        # a small 3D volume in full precision, in training
        dict(name="ffn 16x16x16 f32 train", op="ffn", grid="16x16x16", B=2, C=64, F=256, dtype="f32", train=True,
             act="gelu"),
        # ragged sequences, sizes that fill no tile
        dict(name="ffn 777 bf16", op="ffn", grid="777", B=3, C=200, F=536, dtype="bf16", train=False, act="gelu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _grid(rng, positions):
    """A grid of one to three axes with about `positions` points, odd extents among them."""
    d = rng.choice((1, 1, 2, 3))
    n = max(1, int(round(positions ** (1.0 / d))))
    axes = [max(1, n + rng.randint(-(n // 4), n // 4)) for _ in range(d)]
    if rng.random() < 0.4:      # the powers of two that the convolution takes
        axes = [1 << max(0, int(round(math.log2(a)))) for a in axes]
    return axes


def draw(rng):
    op = rng.choice(("join", "join", "dropout", "ffn", "ffn"))
    dtype = rng.choice(("f32", "bf16", "bf16"))
    train = rng.random() < 0.5
    while True:
        B = _log(rng, 1, 64)
        axes = [1] if rng.random() < 0.2 else _grid(rng, _log(rng, 2, 300000))
        L = math.prod(axes)
        case = dict(op=op, grid="x".join(map(str, axes)), B=B, dtype=dtype, train=train)
        if op == "ffn":
            C, F = 8 * _log(rng, 1, 256), 8 * _log(rng, 2, 704)
            if B * L * C * F * (6 if dtype == "f32" else 1) > 2 * 4096 * 2048 * 5632 or B * L * max(C, F) > 1 << 26:
                continue
            return dict(case, C=C, F=F, act=rng.choice(("silu", "gelu")))
        C = _log(rng, 4, 2048)
        if op == "dropout":
            if B * C * L > 1 << 26:
                continue
            return dict(case, C=C, p=rng.choice((0.1, 0.5, round(rng.uniform(0.0, 0.9), 3))))
        if B * C * L > 1 << 25:
            continue
        return dict(case, C=C, post=rng.choice(("rms", "layer", "none")), pre=rng.choice(("rms", "layer", "none")),
                    affine=rng.random() < 0.8, gate=rng.random() < 0.5, scale=rng.random() < 0.5,
                    p=rng.choice((0.0, 0.1, 0.3)))


def _axes(case):
    return [int(n) for n in case["grid"].split("x")]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    axes, B, C, dt = _axes(case), case["B"], case["C"], DTYPES[case["dtype"]]
    shape = [B, C] + axes

    def normal(*s):
        return torch.randn(*s, generator=g, device="cuda", dtype=torch.float32)

    s = {"case": case}
    s["rng"] = torch.tensor([0x9E3779B9 * (seed + 1) % (1 << 62), 1000 + seed], dtype=torch.int64, device="cuda")
    if case["op"] == "dropout":
        s["x"] = normal(*shape).to(dt)
        s["dy"] = normal(*shape).to(dt) if case["train"] else None
    elif case["op"] == "join":
        per = (1, C) + (1,) * len(axes)
        # a residual stream whose channels have their own means and scales, a mixer's output that is smaller
        s["x"] = (normal(*shape) * (0.5 + normal(*per).abs()) + 0.5 * normal(*per)).to(dt)
        s["y"] = (normal(*shape) * 0.3 + 0.1 * normal(*per)).to(dt)
        for stage in ("post", "pre"):
            norm = case[stage] != "none" and case["affine"]
            s[stage + "_w"] = 1 + 0.2 * normal(C) if norm else None
            s[stage + "_b"] = 0.1 * normal(C) if norm and case[stage] == "layer" else None
        s["gate"] = 1 + 0.5 * normal(B, C) if case["gate"] else None
        s["scale"] = 0.3 + 0.1 * normal(C) if case["scale"] else None
        if case["train"]:
            s["dh"] = normal(*shape).to(dt)
            s["dn"] = normal(*shape).to(dt) if case["pre"] != "none" else None
    else:
        F = case["F"]
        s["x"] = normal(*shape).to(dt)
        s["wg"] = (normal(F, C) / math.sqrt(C)).to(dt)
        s["wu"] = (normal(F, C) / math.sqrt(C)).to(dt)
        s["wd"] = (normal(C, F) / math.sqrt(F)).to(dt)
        s["dy"] = normal(*shape).to(dt) if case["train"] else None
    if own:
        from dimensional_long_convolution_b200 import hyena_nd_block as K

        io = case["dtype"]
        if case["op"] == "dropout":
            s["layer"] = K.GridDropout(axes, B, C, io_dtype=io, p=case["p"])
        elif case["op"] == "join":
            s["layer"] = K.BlockJoin(axes, B, C, io_dtype=io, post=case["post"], pre=case["pre"], p=case["p"])
            s["layer"].set_params(post_w=s["post_w"], post_b=s["post_b"], gate=s["gate"], scale=s["scale"],
                                  pre_w=s["pre_w"], pre_b=s["pre_b"])
        else:
            s["layer"] = K.GatedFFN(axes, B, C, case["F"], io_dtype=io, act=case["act"])
    return s


def run(s):
    if own:
        return _own(s)
    return {"dropout": _dropout, "join": _join, "ffn": _ffn}[s["case"]["op"]](s)


def _own(s):
    case, layer = s["case"], s["layer"]
    if case["op"] == "dropout":
        out = {"y": layer(s["x"], s["rng"])}
        if case["train"]:
            out["dx"] = layer.backward(s["dy"], s["rng"])
        return out
    if case["op"] == "join":
        h, n = layer(s["x"], s["y"], rng=s["rng"] if case["p"] > 0 else None)
        out = {"h": h, "n": n}
        if case["train"]:
            out.update(layer.backward(s["x"], s["y"], s["dh"], s["dn"], rng=s["rng"] if case["p"] > 0 else None))
        return out
    out = {"y": layer(s["x"], s["wg"], s["wu"], s["wd"])}
    if case["train"]:
        out["dx"], out["dwg"], out["dwu"], out["dwd"] = layer.backward(s["x"], s["wg"], s["wu"], s["wd"], s["dy"])
    return out


# ------------------------------------------------------------- plain forms
def _philox_words(rng, groups):
    """The four 32-bit words of Philox4x32-10 (Salmon et al. 2011) for each counter (group, offset), as int64."""
    low = 0xFFFFFFFF

    def product(a, b):          # high and low word of a 32 x 32 bit product
        return (a * (b >> 16) + ((a * (b & 0xFFFF)) >> 16)) >> 16, (a * b) & low

    i = torch.arange(groups, device=rng.device, dtype=torch.int64)
    k0, k1 = rng[0] & low, (rng[0] >> 32) & low
    c0, c1 = i & low, i >> 32
    c2, c3 = (rng[1] & low).expand(groups), ((rng[1] >> 32) & low).expand(groups)
    for _ in range(10):
        h0, l0 = product(0xD2511F53, c0)
        h1, l1 = product(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack((c0, c1, c2, c3), dim=1)


def _mask(case, rng, shape):
    """Which elements stay, and what they are multiplied by: eight 16-bit lots a counter, compared with p."""
    count = math.prod(shape)
    words = _philox_words(rng, (count + 7) // 8)
    lots = torch.stack((words & 0xFFFF, words >> 16), dim=2).reshape(-1)[:count]
    border = math.floor(case["p"] * 65536 + 0.5)
    return (lots >= border).reshape(shape), 65536 / (65536 - border)


def _drop(keep, factor, v):
    return torch.where(keep, v * factor, 0.0)


def _dropout(s):
    case, x = s["case"], s["x"]
    keep, factor = _mask(case, s["rng"], x.shape)
    out = {"y": _drop(keep, factor, x.float()).to(x.dtype)}
    if case["train"]:
        out["dx"] = _drop(keep, factor, s["dy"].float()).to(x.dtype)
    return out


def _hat(v, kind, eps=1e-6):
    """The normalised value and the factor it was normalised with, over axis 1."""
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    rho = torch.rsqrt((v * v).mean(1, keepdim=True) + eps)
    return v * rho, rho


def _affine(v, w, b):
    v = v if w is None else v * w[:, None]
    return v if b is None else v + b[:, None]


def _hat_backward(e, hat, rho, kind):
    d = e - hat * (e * hat).mean(1, keepdim=True)
    if kind == "layer":
        d = d - e.mean(1, keepdim=True)
    return d * rho


def _join(s):
    case, dt, shape = s["case"], s["x"].dtype, s["x"].shape
    B, C = shape[:2]
    x, y = (s[k].float().reshape(B, C, -1) for k in ("x", "y"))
    post, pre = case["post"], case["pre"]
    yhat, rho1 = _hat(y, post) if post != "none" else (y, None)
    z = _affine(yhat, s["post_w"], s["post_b"])
    if case["p"] > 0:
        keep, factor = _mask(case, s["rng"], x.shape)
        z = _drop(keep, factor, z)
    mult = torch.ones(B, C, device=x.device)
    mult = mult if s["gate"] is None else mult * s["gate"]
    mult = mult if s["scale"] is None else mult * s["scale"]
    h = x + mult[:, :, None] * z
    out = {"h": h.to(dt).reshape(shape), "n": None}
    if pre != "none":
        hhat, rho2 = _hat(h, pre)
        out["n"] = _affine(hhat, s["pre_w"], s["pre_b"]).to(dt).reshape(shape)
    if not case["train"]:
        return out
    dht = s["dh"].float().reshape(B, C, -1)
    if pre != "none":
        dn = s["dn"].float().reshape(B, C, -1)
        a = dn if s["pre_w"] is None else dn * s["pre_w"][:, None]
        dht = dht + _hat_backward(a, hhat, rho2, pre)
        if s["pre_w"] is not None:
            out["dpre_w"] = (dn * hhat).sum((0, 2))
        if s["pre_b"] is not None:
            out["dpre_b"] = dn.sum((0, 2))
    out["dx"] = dht.to(dt).reshape(shape)
    each = (dht * z).sum(2)
    if s["gate"] is not None:
        out["dgate"] = each if s["scale"] is None else each * s["scale"]
    if s["scale"] is not None:
        out["dscale"] = (each if s["gate"] is None else each * s["gate"]).sum(0)
    dz = dht * mult[:, :, None]
    if case["p"] > 0:
        dz = _drop(keep, factor, dz)
    if s["post_w"] is not None:
        out["dpost_w"] = (dz * yhat).sum((0, 2))
    if s["post_b"] is not None:
        out["dpost_b"] = dz.sum((0, 2))
    e = dz if s["post_w"] is None else dz * s["post_w"][:, None]
    dy = e if post == "none" else _hat_backward(e, yhat, rho1, post)
    out["dy"] = dy.to(dt).reshape(shape)
    return out


def _act(g, kind):
    """The activation and its derivative."""
    if kind == "silu":
        sig = 1 / (1 + torch.exp(-g))
        return g * sig, sig * (1 + g * (1 - sig))
    cdf = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
    return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))


def _ffn(s):
    case, dt, shape = s["case"], s["x"].dtype, s["x"].shape
    B, C = shape[:2]
    wg, wu, wd = (s[k].float() for k in ("wg", "wu", "wd"))
    # one column a position: [C, B L]
    x = s["x"].float().reshape(B, C, -1).transpose(0, 1).reshape(C, -1)

    def back(v):
        return v.reshape(C, B, -1).transpose(0, 1).reshape(shape).to(dt)

    g, u = wg @ x, wu @ x
    a, da = _act(g, case["act"])
    out = {"y": back(wd @ (a * u))}
    if case["train"]:
        dy = s["dy"].float().reshape(B, C, -1).transpose(0, 1).reshape(C, -1)
        dh = wd.t() @ dy
        dg, du = dh * u * da, dh * a
        out["dx"] = back(wg.t() @ dg + wu.t() @ du)
        out["dwg"], out["dwu"] = (dg @ x.t()).to(dt), (du @ x.t()).to(dt)
        out["dwd"] = (dy @ (a * u).t()).to(dt)
    return out


# ------------------------------------------------------------------- work
def work(case):
    E, es = case["B"] * case["C"] * math.prod(_axes(case)), SIZE[case["dtype"]]
    if case["op"] == "dropout":
        return {"bytes": (4 if case["train"] else 2) * E * es, "flops": 0}
    if case["op"] == "join":
        n = 1 if case["pre"] != "none" else 0
        tensors = 3 + n + ((3 + n) if case["train"] else 0)
        params = 4 * case["C"] * (4 + case["B"]) * (2 if case["train"] else 1)
        return {"bytes": tensors * E * es + params, "flops": (40 if case["train"] else 12) * E}
    weights = 3 * case["C"] * case["F"]
    T = E // case["C"]
    return {"bytes": ((4 if case["train"] else 2) * E + (2 if case["train"] else 1) * weights) * es,
            "flops": (18 if case["train"] else 6) * T * case["C"] * case["F"]}


# ------------------------------------------------------- the definition, in 64 bits
def _lots64(rng, count):
    """The 16-bit lots of elements 0 .. count - 1, on the host."""
    seed, offset = (int(v) for v in rng.tolist())
    u, mask = np.uint64, np.uint64(0xFFFFFFFF)
    groups = np.arange(-(-count // 8), dtype=np.uint64)
    ctr = [groups & mask, groups >> u(32), np.full_like(groups, offset & 0xFFFFFFFF), np.full_like(groups, offset >> 32)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = ctr[0] * u(0xD2511F53), ctr[2] * u(0xCD9E8D57)
        ctr = [(b >> u(32)) ^ ctr[1] ^ u(key[0]), b & mask, (a >> u(32)) ^ ctr[3] ^ u(key[1]), a & mask]
        key = [(key[0] + 0x9E3779B9) % (1 << 32), (key[1] + 0xBB67AE85) % (1 << 32)]
    lots = np.empty((groups.size, 8), dtype=np.uint16)
    for w in range(4):
        lots[:, 2 * w], lots[:, 2 * w + 1] = ctr[w] & u(0xFFFF), ctr[w] >> u(16)
    return lots.reshape(-1)[:count]


def _factors64(case, s):
    """What dropout multiplies each element by."""
    t = int(math.floor(case["p"] * 65536 + 0.5))
    stay = torch.from_numpy(_lots64(s["rng"], s["x"].numel()) >= t).to(s["x"].device)
    return stay.double().mul_(65536.0 / (65536 - t)).reshape(s["x"].shape)


def _norm64(v, kind, w, b):
    v = v.movedim(1, -1)
    if kind == "layer":
        v = torch.nn.functional.layer_norm(v, v.shape[-1:], w, b, 1e-6)
    else:
        v = v / torch.sqrt(v.square().mean(-1, keepdim=True) + 1e-6)
        v = v if w is None else v * w
    return v.movedim(-1, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "dropout":
        m = _factors64(case, s)
        out = {"y": s["x"].double() * m}
        if case["train"]:
            out["dx"] = s["dy"].double() * m
        return out
    train = case["train"]
    if case["op"] == "join":
        names = ["x", "y"] + [k for k in ("post_w", "post_b", "gate", "scale", "pre_w", "pre_b") if s[k] is not None]
        v = {k: s[k].double().requires_grad_(train) for k in names}
        z = v["y"] if case["post"] == "none" else _norm64(v["y"], case["post"], v.get("post_w"), v.get("post_b"))
        if case["p"] > 0:
            z = z * _factors64(case, s)
        tail = (1,) * (s["x"].ndim - 2)
        if "gate" in v:
            z = z * v["gate"].reshape(v["gate"].shape + tail)
        if "scale" in v:
            z = z * v["scale"].reshape((-1,) + tail)
        h = v["x"] + z
        n = None if case["pre"] == "none" else _norm64(h, case["pre"], v.get("pre_w"), v.get("pre_b"))
        out = {"h": h.detach(), "n": None if n is None else n.detach()}
        if train:
            heads, seeds = ([h], [s["dh"].double()]) if n is None else ([h, n], [s["dh"].double(), s["dn"].double()])
            grads = torch.autograd.grad(heads, list(v.values()), seeds)
            out.update({"d" + k: g for k, g in zip(names, grads)})
        return out
    v = {k: s[k].double().requires_grad_(train) for k in ("x", "wg", "wu", "wd")}
    tokens = v["x"].movedim(1, -1)
    act = torch.nn.functional.silu if case["act"] == "silu" else torch.nn.functional.gelu
    y = (act(tokens @ v["wg"].t()) * (tokens @ v["wu"].t()) @ v["wd"].t()).movedim(-1, 1)
    out = {"y": y.detach()}
    if train:
        grads = torch.autograd.grad(y, list(v.values()), s["dy"].double())
        out.update({"d" + k: g for k, g in zip(v, grads)})
    return out
