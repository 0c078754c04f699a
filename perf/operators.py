"""What the serving operators on head rows are measured on: multi-axis rotary
positions (forward and gradient), appending keys and values to a paged cache,
and attention of new tokens over that cache.

`listed()` names the cases, `draw(rng)` gives more of the same ranges,
`prepare` makes what a caller has in hand, `run` makes one pass: with `own`
false in elementary torch operations, with `own` true through this package.
`exact` restates the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


def _rope(name, grad, t, hq, hk, d, r, sections, mixed, pairing, dt):
    return {"name": name, "op": "rope", "grad": grad, "t": t, "hq": hq, "hk": hk, "d": d, "r": r,
            "sections": sections, "mixed": mixed, "pairing": pairing, "dt": dt}


def _append(name, t, hq, hk, d, r, sections, pairing, norm, page, pad, dt):
    return {"name": name, "op": "append", "t": t, "hq": hq, "hk": hk, "d": d, "r": r, "sections": sections,
            "mixed": False, "pairing": pairing, "norm": norm, "page": page, "pad": pad, "dt": dt}


def _attend(name, b, q, kv, ragged, hq, hk, d, page, dt):
    return {"name": name, "op": "attend", "b": b, "q": q, "kv": kv, "ragged": ragged, "hq": hq, "hk": hk, "d": d,
            "page": page, "dt": dt}


def listed():
    return [
        # the q and k heads of a few tokens being generated: the call's latency
        _rope("rope 8 tokens", False, 8, 32, 8, 128, 128, "64", False, "half", "bf16"),
        # a video batch (time, height, width) in 16384 rows of 32 heads, the per-head norm's shape
        _rope("rope video 16384", False, 16384, 32, 8, 128, 128, "16,24,24", False, "half", "bf16"),
        # the same rotation's gradient in a training step, axes dealt in turn
        _rope("rope video grad 4096", True, 4096, 32, 8, 128, 128, "24,20,20", True, "half", "f16"),
        # odd heads, part of the head rotated, adjacent pairs, two axes (an image), fp32
        _rope("rope image odd f32", True, 1001, 12, 3, 80, 64, "16,16", False, "adjacent", "f32"),
        # one decoding step of 32 sequences: normalise and rotate q and k, append k and v
        _append("append 32 tokens", 32, 32, 8, 128, 128, "64", "half", True, 16, False, "bf16"),
        # a prefill chunk's tokens appended
        _append("append chunk 8192", 8192, 32, 8, 128, 128, "64", "half", True, 64, False, "bf16"),
        # a padded batch: some tokens have no slot; odd heads and pages
        _append("append padded odd", 777, 10, 5, 96, 64, "12,10,10", "half", False, 24, True, "f16"),
        # a single sequence being decoded over a long context
        _attend("attend 1 token 4095", 1, 1, 4095, False, 32, 8, 128, 16, "bf16"),
        # a decoding batch of unequal contexts
        _attend("attend 64 tokens 8192", 64, 1, 8192, True, 32, 8, 128, 16, "bf16"),
        # chunks of prompts over the context that precedes them
        _attend("attend chunk 512 over 8192", 4, 512, 8192, True, 32, 8, 128, 64, "bf16"),
        # whole prompts
        _attend("attend prompt 8192", 2, 8192, 8192, False, 32, 8, 128, 64, "bf16"),
        # a ragged batch of odd lengths, seven heads a group, small heads, pages of 24
        _attend("attend ragged odd", 7, 301, 2047, True, 14, 2, 64, 24, "f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _split(rng, n, half):
    """`half` frequencies over n axes, none empty."""
    cuts = sorted(rng.sample(range(1, half), n - 1)) if n > 1 else []
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [half]))


def draw(rng):
    op = rng.choice(["rope", "rope", "append", "attend", "attend", "attend"])
    hk = rng.randint(1, 8)
    if op == "attend":
        group, d, page = rng.randint(1, 8), 8 * rng.randint(8, 16), 8 * rng.randint(1, 16)
        dt = rng.choice(["bf16", "bf16", "f16"])
        kind = rng.choice(["one", "few", "chunk", "prompt"])
        if kind == "one":
            b, q, kv = _log(rng, 1, 64), 1, _log(rng, 64, 16384)
        elif kind == "few":
            b, q, kv = _log(rng, 1, 16), rng.randint(2, 16), _log(rng, 64, 16384)
        elif kind == "chunk":
            b, q, kv = _log(rng, 1, 4), _log(rng, 32, 1024), _log(rng, 1024, 8192)
        else:
            b, q = _log(rng, 1, 4), _log(rng, 128, 4000)
            kv = q
        c = _attend("", b, q, max(q, kv), rng.random() < 0.6, hk * group, hk, d, page, dt)
    else:
        d = 8 * rng.randint(8, 16)
        r = rng.choice([d, d, 2 * rng.randint(16, d // 2)])
        sections = _split(rng, rng.randint(1, 3), r // 2)
        pairing = rng.choice(["half", "half", "adjacent"])
        dt = rng.choice(["bf16", "bf16", "f16", "f32"])
        hq, t = hk * rng.randint(1, 8), _log(rng, 1, 8192)
        if op == "rope":
            c = _rope("", rng.random() < 0.5, t, hq, hk, d, r, sections, rng.random() < 0.5, pairing, dt)
        else:
            c = _append("", t, hq, hk, d, r, sections, pairing, rng.random() < 0.5, 8 * rng.randint(1, 16),
                        rng.random() < 0.5, dt)
    del c["name"]
    return c


# ------------------------------------------------------------ what a case is --

def _axes(c):
    """The axis of each frequency, one byte each: blocks of the given sizes,
    or dealt in turn among the axes that have frequencies left."""
    left = [int(s) for s in c["sections"].split(",")]
    if not c["mixed"]:
        return bytes(a for a, n in enumerate(left) for _ in range(n))
    out = []
    while any(left):
        for a, n in enumerate(left):
            if n:
                out.append(a)
                left[a] -= 1
    return bytes(out)


def _lens(c):
    """(new tokens, length after them) of each sequence."""
    n = c["b"]
    if not c["ragged"]:
        return [c["q"]] * n, [c["kv"]] * n
    q = [max(1, c["q"] - (c["q"] * ((5 * i) % 8)) // 11) for i in range(n)]
    kv = [max(q[i], c["kv"] - (c["kv"] * ((3 * i) % 16)) // 17) for i in range(n)]
    return q, kv


def _pages(c):
    return [-(-n // c["page"]) for n in _lens(c)[1]]


def work(c):
    size = 4 if c["dt"] == "f32" else 2
    if c["op"] == "attend":
        q, kv = _lens(c)
        pairs = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(q, kv))
        nbytes = 2 * size * c["d"] * (sum(q) * c["hq"] + sum(kv) * c["hk"]) + 4 * sum(_pages(c)) + 4 * sum(q) * c["hq"]
        return {"bytes": nbytes, "flops": 4 * c["d"] * pairs * c["hq"]}
    naxes = c["sections"].count(",") + 1
    heads = c["hq"] + (2 if c["op"] == "append" else 1) * c["hk"]
    rot = (c["hq"] + c["hk"]) * c["r"]
    return {"bytes": c["t"] * (2 * size * heads * c["d"] + 4 * naxes + (8 if c["op"] == "append" else 0)),
            "flops": c["t"] * (3 * rot + (4 * (c["hq"] + c["hk"]) * c["d"] if c.get("norm") else 0))}


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[c["dt"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    s = {"case": c}
    if c["op"] == "attend":
        q, kv = _lens(c)
        pages = _pages(c)
        total = sum(pages) + 3  # a cache has pages that no sequence holds
        order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros(c["b"], max(pages), dtype=torch.int32, device="cuda")
        at = 0
        for i, n in enumerate(pages):
            table[i, :n] = order[at:at + n]
            at += n
        s["q"] = normal(sum(q), c["hq"], c["d"])
        s["k_cache"] = normal(total, c["page"], c["hk"], c["d"])
        s["v_cache"] = normal(total, c["page"], c["hk"], c["d"])
        s["table"] = table
        s["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
        s["cu_q"] = torch.tensor([sum(q[:i]) for i in range(c["b"] + 1)], dtype=torch.int32, device="cuda")
        s["max_q"], s["max_kv"] = max(q), max(kv)
        return s
    naxes = c["sections"].count(",") + 1
    half = c["r"] // 2
    s["inv_freq"] = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).to(torch.float32).cuda()
    s["axes"] = _axes(c)
    first = torch.randint(0, 100000, (), generator=g, device="cuda", dtype=torch.int32)
    if naxes == 1:
        s["positions"] = (first + torch.arange(c["t"], device="cuda", dtype=torch.int32)).view(1, -1)
    else:  # a grid of frames of 24 x 32 patches
        i = torch.arange(c["t"], device="cuda", dtype=torch.int32)
        s["positions"] = (first + torch.stack([i // 768, i // 32 % 24, i % 32][-naxes:])).contiguous()
    # q, k and v are the parts of one projection's output
    heads = c["hq"] + 2 * c["hk"]
    qkv = normal(c["t"], heads, c["d"])
    s["q"], s["k"], s["v"] = qkv.split([c["hq"], c["hk"], c["hk"]], dim=1)
    if c["op"] == "append":
        total = -(-c["t"] // c["page"]) + 3
        slots = torch.randperm(total * c["page"], generator=g, device="cuda")[:c["t"]]
        if c["pad"]:
            slots[::5] = -1
        s["slots"] = slots
        s["k_cache"] = normal(total, c["page"], c["hk"], c["d"])
        s["v_cache"] = normal(total, c["page"], c["hk"], c["d"])
        s["wq"] = s["wk"] = None
        if c["norm"]:
            s["wq"] = 1 + 0.1 * normal(c["d"])
            s["wk"] = 1 + 0.1 * normal(c["d"])
    return s


# -------------------------------------------------------------- plain forms --

def _cos_sin(s, sign):
    """cos and sin of every token's angles, [t, 1, r / 2]: the products in 64
    bits, because a far position's angle has lost its fraction in 32."""
    axis = torch.tensor(list(s["axes"]), device="cuda")
    angle = s["positions"].double()[axis].t() * s["inv_freq"].double()
    return angle.cos().float()[:, None], (sign * angle.sin()).float()[:, None]


def _rotate(x, cos, sin, c):
    """Rotates the first r values of each head of x (32 bits)."""
    r = c["r"]
    rot, rest = x[..., :r], x[..., r:]
    if c["pairing"] == "half":
        a, b = rot[..., :r // 2], rot[..., r // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], dim=-1)
    a, b = rot[..., 0::2], rot[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2), rest], dim=-1)


def _norm(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _plain_rope(s):
    c, dt = s["case"], s["q"].dtype
    cos, sin = _cos_sin(s, -1.0 if c["grad"] else 1.0)
    return _rotate(s["q"].float(), cos, sin, c).to(dt), _rotate(s["k"].float(), cos, sin, c).to(dt)


def _plain_append(s):
    c, dt = s["case"], s["q"].dtype
    cos, sin = _cos_sin(s, 1.0)
    q, k = s["q"].float(), s["k"].float()
    if c["norm"]:
        q, k = _norm(q, s["wq"]), _norm(k, s["wk"])
    q, k = _rotate(q, cos, sin, c).to(dt), _rotate(k, cos, sin, c).to(dt)
    kept = s["slots"] >= 0
    at = s["slots"][kept]
    s["k_cache"].view(-1, c["hk"], c["d"])[at] = k[kept]
    s["v_cache"].view(-1, c["hk"], c["d"])[at] = s["v"][kept]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attend(s):
    c = s["case"]
    b, mq, mk, hq, hk, d = c["b"], s["max_q"], s["max_kv"], c["hq"], c["hk"], c["d"]
    group = hq // hk
    cu, kv = s["cu_q"].long(), s["kv_lens"].long()
    nq = cu[1:] - cu[:-1]
    i = torch.arange(mq, device="cuda")
    j = torch.arange(mk, device="cuda")
    token = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)                       # [b, mq]
    page = torch.gather(s["table"].long(), 1, (j // c["page"]).expand(b, mk))       # [b, mk]
    slot = page * c["page"] + j % c["page"]
    q = s["q"][token].float().view(b, mq, hk, group, d).permute(0, 2, 3, 1, 4).reshape(b, hk, group * mq, d)
    k = s["k_cache"].view(-1, hk, d)[slot].float().permute(0, 2, 3, 1)               # [b, hk, d, mk]
    v = s["v_cache"].view(-1, hk, d)[slot].float().permute(0, 2, 1, 3)               # [b, hk, mk, d]
    seen = (j <= (kv - nq)[:, None, None] + i[:, None]) & (j < kv[:, None, None])    # [b, mq, mk]
    x = torch.matmul(q, k).view(b, hk, group, mq, mk).mul_(1.0 / math.sqrt(d))
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(b, hk, group * mq, mk), v).view(b, hk, group, mq, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (total.log() + top).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(b * mq, hq, d)
    lse = lse.permute(0, 3, 1, 2).reshape(b * mq, hq)
    # back to the ragged rows: sequence and place of each token
    row = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    at = seq * mq + row - cu[seq]
    return {"out": o[at].to(s["q"].dtype), "lse": lse[at]}


# ---------------------------------------------------------- the package's --

def _own(s):
    import row_wise_normalization_rmsnorm_gb300 as rn
    c = s["case"]
    if c["op"] == "rope":
        call = rn.rope_bwd if c["grad"] else rn.rope_fwd
        return call(s["q"], s["k"], s["positions"], s["inv_freq"], axes=s["axes"], pairing=c["pairing"])
    if c["op"] == "append":
        q = rn.paged_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], s["positions"], s["inv_freq"],
                               axes=s["axes"], pairing=c["pairing"], q=s["q"], wq=s["wq"], wk=s["wk"], eps=EPS)
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    out, lse = rn.paged_attn_fwd(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], s["cu_q"],
                                 max_q=s["max_q"], max_kv=s["max_kv"], lse=True)
    return {"out": out, "lse": lse}


def run(s):
    if own:
        return _own(s)
    return {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend}[s["case"]["op"]](s)


# ------------------------------------------------------------------- 64 bits --

def _turned(x, s, c, sign):
    """Each head's pairs as complex numbers, times exp(i angle)."""
    r, half = c["r"], c["r"] // 2
    first = torch.arange(half, device="cuda") * (1 if c["pairing"] == "half" else 2)
    second = first + (half if c["pairing"] == "half" else 1)
    pos = torch.stack([s["positions"][a] for a in s["axes"]], dim=1).double()
    turn = torch.polar(torch.ones_like(pos), sign * pos * s["inv_freq"].double())
    z = torch.complex(x[..., first], x[..., second]) * turn[:, None, :]
    y = x.clone()
    y[..., first] = z.real
    y[..., second] = z.imag
    assert r == 2 * half
    return y


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope":
        sign = -1.0 if c["grad"] else 1.0
        return _turned(s["q"].double(), s, c, sign), _turned(s["k"].double(), s, c, sign)
    if c["op"] == "append":
        q, k = s["q"].double(), s["k"].double()
        if c["norm"]:
            q = q / (q.square().sum(-1, keepdim=True) / c["d"] + EPS).sqrt() * s["wq"].double()
            k = k / (k.square().sum(-1, keepdim=True) / c["d"] + EPS).sqrt() * s["wk"].double()
        q, k = _turned(q, s, c, 1.0), _turned(k, s, c, 1.0)
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        for t, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                kc[slot // c["page"], slot % c["page"]] = k[t]
                vc[slot // c["page"], slot % c["page"]] = s["v"][t].double()
        return {"q": q, "k_cache": kc, "v_cache": vc}
    group = c["hq"] // c["hk"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    at = 0
    for b, (nq, nk) in enumerate(zip(*_lens(c))):
        held = s["table"][b, :-(-nk // c["page"])].long()
        hidden = torch.ones(nq, nk, dtype=torch.bool, device="cuda").triu(nk - nq + 1)
        for h in range(c["hk"]):
            k = s["k_cache"][held, :, h].reshape(-1, c["d"])[:nk].double()
            v = s["v_cache"][held, :, h].reshape(-1, c["d"])[:nk].double()
            for m in range(h * group, (h + 1) * group):
                x = s["q"][at:at + nq, m].double() @ k.t() / math.sqrt(c["d"])
                x[hidden] = -math.inf
                lse[at:at + nq, m] = torch.logsumexp(x, -1)
                out[at:at + nq, m] = torch.softmax(x, -1) @ v
        at += nq
    return {"out": out, "lse": lse}
