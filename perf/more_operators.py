"""What the row operators of a training step beside the norms are measured on:
group norm with an activation (channels last), rows kept in 8 bits for the
backward pass, and embedding rows with their gradient.

`listed()` names the cases, `draw(rng)` gives more of the same ranges,
`prepare` makes what a caller has in hand, `run` makes one pass: with `own`
false in elementary torch operations, with `own` true through this package.
`exact` restates the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
GN_EPS, RMS_EPS = 1e-5, 1e-6
BLOCK = 32  # values that share a scale in an 8-bit row


def _gn(name, op, b, s, c, g, act, dt, w32):
    return {"name": name, "op": op, "b": b, "s": s, "c": c, "g": g, "act": act, "dt": dt, "w32": w32}


def _rows(name, op, m, n, fused, dt, w32):
    return {"name": name, "op": op, "m": m, "n": n, "fused": fused, "dt": dt, "w32": w32}


def _embed(name, op, t, v, n, norm, pad, dt):
    return {"name": name, "op": op, "t": t, "v": v, "n": n, "norm": norm, "pad": pad, "dt": dt}


def listed():
    return [
        # the innermost, 8 x 8 stage of an image model, one image: the call's latency
        _gn("groupnorm 8x8 c1280", "gn_fwd", 1, 64, 1280, 32, "silu", "bf16", False),
        # its outer stage, a batch of latents: groups of 10 channels, no 16-byte chunk of their own
        _gn("groupnorm 64x64 c320", "gn_fwd", 8, 4096, 320, 32, "silu", "bf16", True),
        # a decoder's pixels: one sample is larger than what the SMs hold
        _gn("groupnorm 256x256 c256", "gn_fwd", 8, 65536, 256, 32, "silu", "bf16", False),
        # the outer stage's gradient in a training step
        _gn("groupnorm grad 64x64 c320", "gn_bwd", 8, 4096, 320, 32, "silu", "bf16", True),
        # odd channels, sizes and activation in fp32
        _gn("groupnorm grad odd f32", "gn_bwd", 3, 1001, 90, 9, "gelu", "f32", False),
        # a training step whose saved rows are held in 8 bits
        _gn("groupnorm kept in 8 bits", "gn_kept", 4, 4096, 512, 32, "silu", "f16", True),
        # the headline workload's rows, kept in 8 bits between the norm and its gradient
        _rows("norm kept 16384x8192", "norm_kept", 16384, 8192, False, "bf16", False),
        # the fused residual add of a small batch
        _rows("add norm kept 256x4096", "norm_kept", 256, 4096, True, "f16", True),
        # rows kept and restored by themselves, no whole chunks
        _rows("kept and restored odd", "kept", 2049, 5003, False, "bf16", False),
        # a batch's embedding rows, scaled, and the first norm
        _embed("embed norm 16384x4096", "embed", 16384, 32768, 4096, True, False, "bf16"),
        # the table's gradient for a padded batch of that size
        _embed("embed grad 16384x4096", "embed_grad", 16384, 32768, 4096, False, True, "bf16"),
        # the rows of eight sequences that are being decoded
        _embed("embed 8 tokens", "embed", 8, 32768, 8192, False, False, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gn_fwd", "gn_fwd", "gn_bwd", "gn_bwd", "gn_kept", "norm_kept", "norm_kept", "kept", "embed", "embed_grad"])
    dt = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op.startswith("gn"):
        b, g = _log(rng, 1, 16), rng.choice([1, 4, 8, 16, 32, 32, rng.randint(2, 40)])
        c = g * rng.choice([4, 8, 10, 16, 20, 30, 40, rng.randint(1, 48)])
        s = min(_log(rng, 16, 65536), max(1, 60_000_000 // (b * c * BYTES[dt] // 2)))
        return _gn("", op, b, s, c, g, rng.choice(["silu", "silu", "gelu", "none"]), dt, rng.random() < 0.5)
    if op in ("norm_kept", "kept"):
        n = rng.choice([64 * _log(rng, 1, 256), _log(rng, 16, 16384)])
        m = min(_log(rng, 1, 32768), max(1, 60_000_000 // (n * BYTES[dt] // 2)))
        return _rows("", op, m, n, op == "norm_kept" and rng.random() < 0.5, dt, rng.random() < 0.5)
    n = rng.choice([64 * _log(rng, 2, 128), _log(rng, 32, 8192)])
    t = min(_log(rng, 1, 32768), 60_000_000 // n)
    v = min(_log(rng, 100, 150_000), 120_000_000 // n)
    return _embed("", op, t, v, n, op == "embed" and rng.random() < 0.6, rng.random() < 0.5, dt)


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def prepare(case, seed):
    c, gen = case, torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt, s = DTYPES[c["dt"]], {"case": c}
    wt = torch.float32 if c.get("w32") else dt
    if c["op"].startswith("gn"):
        # channels of unlike means and widths, as a convolution leaves them
        mean, width = _normal(gen, c["c"]), _normal(gen, c["c"]).mul_(0.3).exp_()
        s["x"] = _normal(gen, c["b"], c["s"], c["c"]).mul_(width).add_(mean).to(dt)
        s["gamma"], s["beta"] = (1 + 0.1 * _normal(gen, c["c"])).to(wt), (0.1 * _normal(gen, c["c"])).to(wt)
        if c["op"] != "gn_fwd":
            s["dy"] = _normal(gen, c["b"], c["s"], c["c"]).to(dt)
        if c["op"] == "gn_bwd":  # what the forward pass saved
            x = s["x"].view(c["b"], c["s"], c["g"], -1)
            s["mean"] = x.mean((1, 3), dtype=torch.float64).float()
            s["rstd"] = ((x.double() - s["mean"][:, None, :, None]).square().mean((1, 3)) + GN_EPS).rsqrt().float()
    elif c["op"] in ("norm_kept", "kept"):
        s["x"] = _normal(gen, c["m"], c["n"])
        s["x"][:, torch.randperm(c["n"], generator=gen, device="cuda")[:-(-c["n"] // 100)]] *= 20  # outlier channels
        s["x"] = s["x"].to(dt)
        if c["op"] == "norm_kept":
            s["w"], s["dy"] = (1 + 0.1 * _normal(gen, c["n"])).to(wt), _normal(gen, c["m"], c["n"]).to(dt)
            if c["fused"]:
                s["residual"], s["dres"] = _normal(gen, c["m"], c["n"]).to(dt), _normal(gen, c["m"], c["n"]).to(dt)
    else:
        # a vocabulary's tokens, the k-th as often as 1 / k, in no order; some places are padding
        rank = torch.rand(c["t"], generator=gen, device="cuda", dtype=torch.float64).mul_(math.log(c["v"] + 1)).exp_().long() - 1
        ids = torch.randperm(c["v"], generator=gen, device="cuda")[rank.clamp_(0, c["v"] - 1)]
        if c["pad"]:
            ids = torch.where(torch.rand(c["t"], generator=gen, device="cuda") < 0.1, -1, ids)
        s["ids"], s["scale"] = ids, math.sqrt(c["n"])
        if c["op"] == "embed":
            s["table"] = _normal(gen, c["v"], c["n"]).mul_(0.02).to(dt)
            s["w"] = (1 + 0.1 * _normal(gen, c["n"])).to(dt)
        else:
            s["dh"] = _normal(gen, c["t"], c["n"]).mul_(0.02).to(dt)
    return s


# ------------------------------------------------------------- plain forms --

def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_slope(z, act):
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    return torch.ones_like(z)


def _gn_forward(s, c):
    x = s["x"].float().view(c["b"], c["s"], c["g"], -1)
    mean = x.mean((1, 3))
    d = x - mean[:, None, :, None]
    rstd = 1 / torch.sqrt(d.square().mean((1, 3)) + GN_EPS)
    z = (d * rstd[:, None, :, None]).view(c["b"], c["s"], c["c"]) * s["gamma"].float() + s["beta"].float()
    return {"y": _act(z, c["act"]).to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _gn_backward(s, c, x, mean, rstd):
    x = x.float().view(c["b"], c["s"], c["g"], -1)
    xhat = ((x - mean[:, None, :, None]) * rstd[:, None, :, None]).view(c["b"], c["s"], c["c"])
    gamma = s["gamma"].float()
    u = s["dy"].float() * _act_slope(xhat * gamma + s["beta"].float(), c["act"])
    dgamma, dbeta = (u * xhat).sum((0, 1)), u.sum((0, 1))
    g, xhat = (u * gamma).view(x.shape), xhat.view(x.shape)
    dx = rstd[:, None, :, None] * (g - g.mean((1, 3), keepdim=True) - xhat * (g * xhat).mean((1, 3), keepdim=True))
    return {"dx": dx.view(c["b"], c["s"], c["c"]).to(s["dy"].dtype), "dgamma": dgamma.to(s["gamma"].dtype),
            "dbeta": dbeta.to(s["beta"].dtype)}


def _kept(x):
    """The fp32 values that x's rows are kept as: in each block of 32 along the
    last dimension whole multiples, -127 to 127, of the smallest power of two
    that can hold them."""
    n = x.shape[-1]
    v = torch.nn.functional.pad(x.float(), (0, -n % BLOCK)).unflatten(-1, (-1, BLOCK))
    top = v.abs().amax(-1, keepdim=True)
    frac, exp = torch.frexp(top)
    step = exp - 7 + (frac >= 255 / 256).int()  # 127.5 steps would round to 128
    most = 9 if x.dtype == torch.float16 else 121  # 64 steps of more are no finite value of the type
    step = torch.where(top > 0, step, -127).clamp(-127, most)
    scale = torch.exp2(step.double()).float()
    return (torch.round(v / scale).clamp(-127, 127) * scale).flatten(-2)[..., :n]


def _norm_forward(h, w, offset=0.0):
    v = h.float()
    rstd = 1 / torch.sqrt(v.square().mean(-1) + RMS_EPS)
    return (v * rstd[..., None] * (offset + w.float())).to(h.dtype), rstd


def _plain(s, c):
    if c["op"] == "gn_fwd":
        return _gn_forward(s, c)
    if c["op"] == "gn_bwd":
        return _gn_backward(s, c, s["x"], s["mean"], s["rstd"])
    if c["op"] == "gn_kept":
        out = _gn_forward(s, c)
        return {**out, **_gn_backward(s, c, _kept(s["x"]), out["mean"], out["rstd"])}
    if c["op"] == "kept":
        return {"x": _kept(s["x"]).to(s["x"].dtype)}
    if c["op"] == "norm_kept":
        h = (s["x"].float() + s["residual"].float()).to(s["x"].dtype) if c["fused"] else s["x"]
        y, rstd = _norm_forward(h, s["w"])
        xhat = _kept(h) * rstd[:, None]
        dy = s["dy"].float()
        g = dy * s["w"].float()
        dx = rstd[:, None] * (g - xhat * (g * xhat).mean(-1, keepdim=True))
        dx = dx + s["dres"].float() if c["fused"] else dx
        out = {"y": y, "rstd": rstd, "dx": dx.to(h.dtype), "dw": (dy * xhat).sum(0).to(s["w"].dtype)}
        return {**out, "h": h} if c["fused"] else out
    there = s["ids"] >= 0
    if c["op"] == "embed":
        h = (s["table"][s["ids"].clamp(min=0)].float() * s["scale"] * there[:, None]).to(s["table"].dtype)
        if not c["norm"]:
            return {"h": h}
        y, rstd = _norm_forward(h, s["w"])
        return {"y": y, "h": h, "rstd": rstd}
    grad = torch.zeros(c["v"], c["n"], device="cuda")
    grad.index_add_(0, s["ids"].clamp(min=0), s["dh"].float() * there[:, None])
    return {"dtable": (grad * s["scale"]).to(s["dh"].dtype)}


# ------------------------------------------------------ the package's calls --

def _package(s, c):
    import row_wise_normalization_rmsnorm_gb300 as rn

    act = None if c.get("act") == "none" else c.get("act")
    if c["op"] == "gn_fwd":
        return rn.groupnorm_fwd(s["x"], s["gamma"], s["beta"], c["g"], act=act, eps=GN_EPS)
    if c["op"] == "gn_bwd":
        return rn.groupnorm_bwd(s["dy"], s["x"], s["gamma"], s["beta"], s["mean"], s["rstd"], c["g"], act=act)
    if c["op"] == "gn_kept":
        f = rn.groupnorm_fwd_ckpt8(s["x"], s["gamma"], s["beta"], c["g"], act=act, eps=GN_EPS)
        b = rn.groupnorm_bwd_ckpt8(s["dy"], f["codes"], f["scales"], s["gamma"], s["beta"], f["mean"], f["rstd"], c["g"], act=act)
        return {"y": f["y"], "mean": f["mean"], "rstd": f["rstd"], **b}
    if c["op"] == "kept":
        return {"x": rn.ckpt8_unpack(*rn.ckpt8_pack(s["x"]), s["x"].dtype)}
    if c["op"] == "norm_kept":
        f = rn.rmsnorm_fwd_ckpt8(s["x"], s["w"], residual=s.get("residual"), eps=RMS_EPS)
        dx, dw = rn.rmsnorm_bwd_ckpt8(s["dy"], f["codes"], f["scales"], s["w"], f["rstd"], dresidual_out=s.get("dres"))
        out = {"y": f["y"], "rstd": f["rstd"], "dx": dx, "dw": dw}
        return {**out, "h": f["residual_out"]} if c["fused"] else out
    if c["op"] == "embed":
        if not c["norm"]:
            return {"h": rn.embed_fwd(s["ids"], s["table"], scale=s["scale"])}
        y, h, rstd = rn.rmsnorm_embed_fwd(s["ids"], s["table"], s["w"], scale=s["scale"], eps=RMS_EPS)
        return {"y": y, "h": h, "rstd": rstd}
    return {"dtable": rn.embed_bwd(s["dh"], s["ids"], c["v"], scale=s["scale"])}


def run(state):
    if own:
        return _package(state, state["case"])
    return _plain(state, state["case"])


def work(case):
    c, e = case, BYTES[case["dt"]]
    kept = 1 + 1 / BLOCK  # bytes a value is kept in
    if c["op"].startswith("gn"):
        n = c["b"] * c["s"] * c["c"]
        each = {"gn_fwd": 2 * e, "gn_bwd": 3 * e, "gn_kept": 4 * e + 2 * kept}[c["op"]]
        return {"bytes": n * each, "flops": n * {"gn_fwd": 10, "gn_bwd": 25, "gn_kept": 40}[c["op"]]}
    if c["op"] in ("norm_kept", "kept"):
        n = c["m"] * c["n"]
        each = 2 * e + 2 * kept if c["op"] == "kept" else 4 * e + 2 * kept + (3 * e if c["fused"] else 0)
        return {"bytes": n * each, "flops": n * (6 if c["op"] == "kept" else 20)}
    if c["op"] == "embed":
        k = np.arange(c["v"])
        p = np.log((k + 2) / (k + 1)) / math.log(c["v"] + 1)
        rows = float((1 - (1 - p) ** (c["t"] * (0.9 if c["pad"] else 1))).sum())  # of the table that are read
        return {"bytes": c["n"] * e * (rows + c["t"] * (2 if c["norm"] else 1)) + 8 * c["t"],
                "flops": c["t"] * c["n"] * (5 if c["norm"] else 1)}
    return {"bytes": c["n"] * e * (c["t"] * (0.9 if c["pad"] else 1) + c["v"]) + 8 * c["t"], "flops": c["t"] * c["n"]}


# ------------------------------------------------------ the definition in 64 --

def _held(x):
    """What an 8-bit row of x stands for, from its definition."""
    v = x.double()
    n = v.shape[-1]
    out = torch.empty_like(v)
    lead = v.shape[:-1]
    whole = n // BLOCK * BLOCK
    for lo, hi in ((0, whole), (whole, n)):
        if hi == lo:
            continue
        part = v[..., lo:hi].reshape(*lead, -1, min(BLOCK, hi - lo))
        top = part.abs().amax(-1, keepdim=True)
        # the largest value lies in [64, 127.5) steps of 2^k
        k = torch.floor(torch.log2(top.clamp(min=2.0 ** -200))) - 6
        k = torch.where(top / torch.exp2(k) >= 128, k + 1, k)  # a logarithm that came out one low or high
        k = torch.where(top / torch.exp2(k) < 64, k - 1, k)
        k = torch.where(top / torch.exp2(k) >= 127.5, k + 1, k)
        k = k.clamp(-127, 9 if x.dtype == torch.float16 else 121)
        out[..., lo:hi] = ((part / torch.exp2(k)).round().clamp(-127, 127) * torch.exp2(k)).reshape(*lead, hi - lo)
    return out


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"].startswith("gn"):
        shape = (c["b"], c["s"], c["g"], c["c"] // c["g"])
        gamma, beta = s["gamma"].double().view(shape[2:]), s["beta"].double().view(shape[2:])
        x = s["x"].double().view(shape)
        out = {}
        if c["op"] == "gn_bwd":
            mean, rstd = s["mean"].double()[:, None, :, None], s["rstd"].double()[:, None, :, None]
        else:
            var, mean = torch.var_mean(x, (1, 3), correction=0, keepdim=True)
            rstd = (var + GN_EPS) ** -0.5
            z = (x - mean) * rstd * gamma + beta
            y = z * torch.sigmoid(z) if c["act"] == "silu" else z * torch.special.ndtr(z) if c["act"] == "gelu" else z
            out = {"y": y.view(c["b"], c["s"], c["c"]), "mean": mean[:, 0, :, 0], "rstd": rstd[:, 0, :, 0]}
            del z, y
        if c["op"] == "gn_fwd":
            return out
        if c["op"] == "gn_kept":
            x = _held(s["x"]).view(shape)
        x = (x - mean) * rstd
        z = x * gamma + beta
        if c["act"] == "silu":
            p = torch.sigmoid(z)
            z = p + z * p * (1 - p)
        elif c["act"] == "gelu":
            z = torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        else:
            z = torch.ones_like(z)
        u = z * s["dy"].double().view(shape)
        dgamma, dbeta = (u * x).sum((0, 1)).view(-1), u.sum((0, 1)).view(-1)
        u = u * gamma
        n = c["s"] * shape[3]
        dx = (u - u.sum((1, 3), keepdim=True) / n - x * ((u * x).sum((1, 3), keepdim=True) / n)) * rstd
        return {**out, "dx": dx.view(c["b"], c["s"], c["c"]), "dgamma": dgamma, "dbeta": dbeta}
    if c["op"] == "kept":
        return {"x": _held(s["x"])}
    if c["op"] == "norm_kept":
        h = s["x"]
        if c["fused"]:
            h = (h.double() + s["residual"].double()).to(h.dtype)  # stored, and normalised as stored
        v, w, dy = h.double(), s["w"].double(), s["dy"].double()
        rstd = (v.square().sum(-1, keepdim=True) / c["n"] + RMS_EPS) ** -0.5
        out = {"y": v * rstd * w, "rstd": rstd[:, 0]}
        if c["fused"]:
            out["h"] = h.double()
        v = _held(h) * rstd
        g = dy * w
        dx = (g - v * ((g * v).sum(-1, keepdim=True) / c["n"])) * rstd
        out["dx"], out["dw"] = dx + s["dres"].double() if c["fused"] else dx, (dy * v).sum(0)
        return out
    scale = float(np.float32(s["scale"]))
    if c["op"] == "embed_grad":
        grad = torch.zeros(c["v"] + 1, c["n"], dtype=torch.float64, device="cuda")
        grad.index_add_(0, torch.where(s["ids"] < 0, c["v"], s["ids"]), s["dh"].double())
        return {"dtable": grad[:-1] * scale}
    h = torch.cat([s["table"], torch.zeros_like(s["table"][:1])])[s["ids"]].double() * scale
    if not c["norm"]:
        return {"h": h}
    h = h.to(s["table"].dtype)  # stored, and normalised as stored
    v = h.double()
    rstd = (v.square().sum(-1, keepdim=True) / c["n"] + RMS_EPS) ** -0.5
    return {"y": v * rstd * s["w"].double(), "h": v, "rstd": rstd[:, 0]}
