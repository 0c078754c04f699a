"""Rotary positions, paged append and paged attention on a GPU, against their
definitions in 64 bits.

Tolerances, derived from the arithmetic (u = 2^-24, half an fp32 step at 1):
  rotation   The angle is a fraction of a turn in fp32, in [-1/2, 1/2): at
             most 2^-26 (u / 4) from its rounding and 2^-32 from the integer
             product, i.e. 2 pi u / 4 < 2 u in the angle; sincospi 2 u each
             for the two, the two products and their sum 3 u more: below
             16 u (|x1| + |x2|) with room, plus the output's rounding.
  norm       rstd: the sum of squares adds at most 10 terms in sequence and 5
             in a tree (15 u), the mean and eps 2 u, rsqrt 4 u of its own,
             halved by the root: below 13 u; two products more 2 u. With the
             rotation: below 32 u (|z1| + |z2|).
  attention  With the weights w_j = exp(x_j - lse): a score's error dx is at
             most 2^-20 scale sum_d |q_d k_jd| (128 products summed in fp32 by
             the tensor cores, u each, at worst truncated) plus 2^-22 |x_j|
             (the fp32 exponent's argument); it moves lse by max dx and w_j
             by twice that. exp2 2 u, the sum of w 16 u. Rounding w to the
             type: half a step of it, h = eps / 2, in fp16 at least 2^-25 of
             the largest weight. So o is off by at most
             sum_j w_j |v_j| (h + 2 max dx + 2^-19) + 2^-25 sum |v_j| (fp16)
             + h |o| (its own rounding), lse by max dx + 2^-20 (1 + |lse|).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def half_step(dt):
    return torch.finfo(dt).eps / 2


@pytest.fixture(scope="module")
def rn():
    from row_wise_normalization_rmsnorm_gb300 import build
    build.build()
    import row_wise_normalization_rmsnorm_gb300 as pkg
    yield pkg
    assert pkg.lib().rmsnorm_device_status(0) == 0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dt=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dt)


def offset_view(x, k):
    """The same values, `k` elements past a 16-byte boundary."""
    buf = torch.empty(x.numel() + k + 16, dtype=x.dtype, device=x.device)
    v = buf[k:k + x.numel()].view(x.shape)
    v.copy_(x)
    return v


# ------------------------------------------------------------------ rotary --

def rotated(x, pos, f, axes, pairing, sign=1.0):
    """(R x in 64 bits, |x1| + |x2| of each value's pair). pos [n, T], axes a list."""
    r = 2 * f.numel()
    first = torch.arange(r // 2, device=x.device) * (1 if pairing == "half" else 2)
    second = first + (r // 2 if pairing == "half" else 1)
    ang = sign * pos[torch.tensor(axes, device=x.device)].double().t() * f.double()
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    x = x.double()
    y, mag = x.clone(), torch.zeros_like(x)
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    mag[..., first] = mag[..., second] = a.abs() + b.abs()
    return y, mag


def near(got, ref, bound):
    assert got.shape == ref.shape
    if got.numel() == 0:
        return
    err = (got.double() - ref).abs()
    worst = (err / (bound + 1e-300)).max().item()
    assert bool((err <= bound).all()), f"worst error {worst:.3g} of its bound"


def freqs(n, base=10000.0):
    return (base ** (-torch.arange(n, dtype=torch.float64) / n)).float().cuda()


def positions(g, n, t, dt, high=100000):
    return torch.randint(0, high, (n, t), generator=g, device="cuda", dtype=dt)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pairing", ["half", "adjacent"])
@pytest.mark.parametrize("T,hq,hk,D,R,sections,mixed", [
    (1, 1, 1, 128, 128, (64,), False), (5, 32, 8, 128, 128, (16, 24, 24), False), (33, 3, 1, 64, 64, (20, 12), True),
    (257, 7, 7, 80, 80, (10, 10, 10, 10), True), (64, 2, 3, 96, 32, (16,), False), (19, 5, 2, 256, 256, (64, 64), False),
    (11, 3, 2, 72, 46, (23,), False), (7, 9, 4, 2, 2, (1,), False), (6, 4, 2, 33, 10, (3, 2), False),
    (1000, 12, 3, 112, 64, (8, 0, 24), False),
])
def test_rope_both_ways(rn, dt, pairing, T, hq, hk, D, R, sections, mixed):
    g, t = gen(T * D + R), TYPES[dt]
    qkv = normal(g, T, hq + 2 * hk, D, dt=t)
    q, k, _ = qkv.split([hq, hk, hk], dim=1)
    f = freqs(R // 2)
    pos = positions(g, len(sections), T, torch.int32)
    axes = rn.rope_axes(sections, mixed)
    for fn, sign in ((rn.rope_fwd, 1.0), (rn.rope_bwd, -1.0)):
        got = fn(q, k, pos, f, axes=axes, pairing=pairing)
        for x, y in zip((q, k), got):
            assert y.dtype == t and y.is_contiguous()
            ref, mag = rotated(x, pos, f, list(axes), pairing, sign)
            near(y, ref, half_step(t) * ref.abs() + 16 * U * mag)
            assert torch.equal(y[..., R:], x[..., R:])


@pytest.mark.parametrize("dt,ptype", [("bf16", torch.int64), ("f32", torch.int32)])
def test_rope_far_and_negative_positions(rn, dt, ptype):
    t = TYPES[dt]
    g = gen(3)
    p = torch.tensor([0, 1, -1, 4095, 4096, -4096, 2 ** 24 + 1, 2 ** 30 + 12345, 2 ** 31 - 1, -2 ** 31 + 1], dtype=ptype,
                     device="cuda")
    x = normal(g, p.numel(), 4, 128, dt=t)
    f = freqs(64)
    y, none = rn.rope_fwd(x, None, p, f)
    assert none is None
    ref, mag = rotated(x, p[None], f, [0] * 64, "half")
    near(y, ref, half_step(t) * ref.abs() + 16 * U * mag)


@pytest.mark.parametrize("pairing", ["half", "adjacent"])
def test_rope_angles_keep_the_bits_that_fp32_holds(rn, pairing):
    """Pairs (1, 0) come back as (cos, sin). In units of u, for values up to 1:
    sincospi 1 (an ulp below 1), the sum with the angle's lower bits 1/2, the
    integer product's 2^-32 of a turn below 0.03. An angle held in one fp32
    fraction of a turn adds up to pi / 2."""
    g = gen(29)
    T, H, D = 8192, 1, 256
    pos = torch.randint(-2 ** 24, 2 ** 24, (T,), generator=g, device="cuda", dtype=torch.int64)
    f = freqs(128)
    x = torch.zeros(T, H, D, device="cuda")
    first = torch.arange(128, device="cuda") * (1 if pairing == "half" else 2)
    second = first + (128 if pairing == "half" else 1)
    x[..., first] = 1.0
    y = rn.rope_fwd(x, None, pos, f, pairing=pairing)[0].double()
    ang = pos.double()[:, None, None] * f.double()  # exact: 25 and 24 bits
    near(y[..., first], ang.cos(), torch.full_like(ang, 1.6 * U))
    near(y[..., second], ang.sin(), torch.full_like(ang, 1.6 * U))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rope_layouts_give_the_same_bits(rn, dt):
    """In place, strided, off a 16-byte boundary and transposed layouts, int64
    positions: the vectorised and the element-wise kernel agree bit for bit."""
    t = TYPES[dt]
    g = gen(4)
    T, H, D = 37, 6, 96
    x = normal(g, T, H, D, dt=t)
    pos, f = positions(g, 1, T, torch.int32), freqs(32)
    y = rn.rope_fwd(x, None, pos, f)[0]
    assert torch.equal(rn.rope_fwd(offset_view(x, 1), None, pos[0].long(), f)[0], y)
    z = x.clone()
    assert rn.rope_fwd(z, None, pos, f, q_out=z)[0] is z and torch.equal(z, y)
    heads_first = x.transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.empty(T, H, 2 * D, dtype=t, device="cuda")[..., :D]
    assert torch.equal(rn.rope_fwd(heads_first, None, pos, f, q_out=out)[0], y)
    odd = torch.zeros(T, H, D + 1, dtype=t, device="cuda")[..., :D]
    odd.copy_(x)
    assert torch.equal(rn.rope_fwd(odd, None, pos, f)[0], y)
    assert torch.equal(rn.rope_fwd(x, None, pos, offset_view(f, 1))[0], y)
    assert torch.equal(rn.rope_fwd(x[:0], None, pos[:, :0], f)[0], y[:0])


def test_rope_gradient_against_differences(rn):
    """<dy, (R(x + h e) - R(x - h e)) / 2h> = <bwd(dy), e> for random e (the
    map is linear; in fp32 the difference carries 2^-24 |R x| / h a value)."""
    g = gen(5)
    T, H, D = 9, 3, 64
    x, e, dy = (normal(g, T, H, D) for _ in range(3))
    pos, f = positions(g, 2, T, torch.int32), freqs(24)
    kw = dict(axes=rn.rope_axes((10, 14)), pairing="adjacent")
    h = 0.5
    up, down = (rn.rope_fwd(x + s * h * e, None, pos, f, **kw)[0].double() for s in (1, -1))
    left = (dy.double() * (up - down) / (2 * h)).sum()
    dx = rn.rope_bwd(dy, None, pos, f, **kw)[0].double()
    right = (dx * e.double()).sum()
    scale = (dy.abs().double() * (x.abs() + e.abs()).double().amax()).sum().item()
    assert abs((left - right).item()) <= 64 * U * scale


@pytest.mark.parametrize("dt", ["bf16"])
def test_rope_refusals(rn, dt):
    t = TYPES[dt]
    x = torch.zeros(4, 2, 64, dtype=t, device="cuda")
    p, f = torch.zeros(4, dtype=torch.int32, device="cuda"), freqs(32)
    bad = [
        lambda: rn.rope_fwd(x[0], None, p, f), lambda: rn.rope_fwd(x, x[:3], p, f), lambda: rn.rope_fwd(x, x.float(), p, f),
        lambda: rn.rope_fwd(x, None, p[:3], f), lambda: rn.rope_fwd(x, None, p.float(), f),
        lambda: rn.rope_fwd(x, None, p, f.double()), lambda: rn.rope_fwd(x, None, p, freqs(33)),
        lambda: rn.rope_fwd(x, None, p.expand(2, 4), f), lambda: rn.rope_fwd(x, None, p, f, axes=bytes(31)),
        lambda: rn.rope_fwd(x, None, p, f, axes=bytes([1] * 32)), lambda: rn.rope_fwd(x, None, p, f, pairing="x"),
        lambda: rn.rope_fwd(x, None, p, f, q_out=x[:2]), lambda: rn.rope_fwd(x.transpose(1, 2), None, p, freqs(1)),
        lambda: rn.rope_fwd(x, None, p, f, k_out=x), lambda: rn.rope_fwd(x, None, p.cpu(), f),
        lambda: rn.rope_fwd(x, None, p[::2], f),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(rn.RMSNormError):
        rn.rope_fwd(torch.zeros(4, 2, 258, dtype=t, device="cuda"), None, p, f)


# ------------------------------------------------------------------ append --

@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,hq,hk,D,R,page,norm,wtype", [
    (1, 4, 1, 128, 128, 16, True, "same"), (77, 8, 2, 64, 64, 1, True, "f32"), (130, 6, 6, 80, 32, 24, False, "same"),
    (33, 0, 3, 96, 96, 5, True, "same"), (19, 5, 5, 50, 20, 3, True, "f32"), (300, 32, 8, 128, 128, 64, True, "same"),
    (12, 3, 1, 256, 0, 16, False, "same"), (9, 2, 2, 7, 6, 2, True, "same"),
])
def test_append(rn, dt, T, hq, hk, D, R, page, norm, wtype):
    g, t = gen(T + D), TYPES[dt]
    pages = -(-T // page) + 2
    q = normal(g, T, hq, D, dt=t) if hq else None
    k, v = normal(g, T, hk, D, dt=t), normal(g, T, hk, D, dt=t)
    kc, vc = normal(g, pages, page, hk, D, dt=t), normal(g, pages, page, hk, D, dt=t)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T]
    slots[::4] = -1
    slots[1::7] = pages * page + 3     # behind the cache: left out as well
    kept = (slots >= 0) & (slots < pages * page)
    wdt = torch.float32 if wtype == "f32" else t
    wq = (1 + 0.1 * normal(g, D)).to(wdt) if norm and hq else None
    wk = (1 + 0.1 * normal(g, D)).to(wdt) if norm else None
    pos, f = positions(g, 1, T, torch.int32), freqs(max(R // 2, 1))
    eps, offset = 1e-5, 0.25
    before = kc.clone(), vc.clone()
    rope = dict(positions=pos, inv_freq=f, pairing="half") if R else {}
    qo = rn.paged_kv_append(k, v, kc, vc, slots, q=q, wq=wq, wk=wk, eps=eps, offset=offset, **rope)

    def ref(x, w):
        z = x.double()
        if w is not None:
            z = z / (z.square().mean(-1, keepdim=True) + eps).sqrt() * (offset + w.double())
        y, mag = rotated(z, pos, f, [0] * f.numel(), "half") if R else (z, torch.zeros_like(z))
        exact = 0.0 if w is None else 32 * U
        return y, half_step(t) * y.abs() + (32 * U * mag if w is not None or R else 0) + exact * z.abs()

    if hq:
        near(qo, *ref(q, wq))
    else:
        assert qo is None
    y, bound = ref(k, wk)
    at = slots[kept]
    near(kc.view(-1, hk, D)[at], y[kept], bound[kept])
    assert torch.equal(vc.view(-1, hk, D)[at], v[kept])
    # nothing else has changed
    others = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    others[at] = False
    for c, b in zip((kc, vc), before):
        assert torch.equal(c.view(-1, hk, D)[others], b.view(-1, hk, D)[others])


def test_append_into_one_tensor_of_keys_and_values(rn):
    """A cache [pages, 2, heads, page_size, D], its k and v views with the
    heads before the places; inputs off a 16-byte boundary give the same bits."""
    g = gen(8)
    T, H, D, page = 21, 3, 64, 8
    both = torch.zeros(5, 2, H, page, D, dtype=torch.bfloat16, device="cuda")
    kc, vc = (both[:, i].transpose(1, 2) for i in (0, 1))
    k, v = normal(g, T, H, D, dt=torch.bfloat16), normal(g, T, H, D, dt=torch.bfloat16)
    slots = torch.randperm(40, generator=g, device="cuda")[:T]
    pos, f, w = positions(g, 1, T, torch.int32), freqs(32), normal(g, D)
    rn.paged_kv_append(k, v, kc, vc, slots, pos, f, wk=w)
    plain = [torch.zeros(5, page, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    rn.paged_kv_append(k, v, *plain, slots, pos, f, wk=w)
    assert torch.equal(kc, plain[0]) and torch.equal(vc, plain[1])
    odd = [torch.zeros(5, page, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    rn.paged_kv_append(k, offset_view(v, 3), *odd, slots, pos, f)
    rn.paged_kv_append(k, v, *plain, slots, pos, f)
    assert torch.equal(odd[0], plain[0]) and torch.equal(odd[1], plain[1])


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("off,D,R", [(0, 64, 32), (1, 64, 32), (0, 50, 22), (0, 33, 10), (1, 33, 0)])
def test_what_passes_unturned_keeps_its_bits(rn, dt, off, D, R):
    """v, and q and k values that are neither normalised nor turned, are every
    bit pattern of their type, NaN payloads and signs among them, in the
    vectorised and the element-wise kernel."""
    t = TYPES[dt]
    word = torch.int32 if dt == "f32" else torch.int16
    g = gen(28)
    T, H, page = 65, 3, 8
    pages = -(-T // page) + 1

    def bits(*shape):
        info = torch.iinfo(word)
        x = torch.randint(info.min, info.max + 1, shape, generator=g, device="cuda", dtype=torch.int64).to(word)
        return offset_view(x, off).view(t)

    q, k, v = bits(T, H, D), bits(T, H, D), bits(T, H, D)
    assert bool(torch.isnan(v).any())
    kc, vc = (torch.zeros(pages, page, H, D, dtype=t, device="cuda") for _ in range(2))
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T]
    pos, f = positions(g, 1, T, torch.int32), freqs(max(R // 2, 1))
    rope = dict(positions=pos, inv_freq=f) if R else {}
    got = rn.paged_kv_append(k, v, kc, vc, slots, q=q, **rope)

    def same(a, b):
        return torch.equal(a.contiguous().view(word), b.contiguous().view(word))

    assert same(vc.view(-1, H, D)[slots], v)
    assert same(kc.view(-1, H, D)[slots][..., R:], k[..., R:]) and same(got[..., R:], q[..., R:])
    if R:
        for fn in (rn.rope_fwd, rn.rope_bwd):
            for x, y in zip((q, k), fn(q, k, pos, f)):
                assert same(y[..., R:], x[..., R:])


def test_append_far_into_a_large_cache(rn):
    """Offsets past 2^32 bytes and 2^31 elements."""
    T, H, D, page = 3, 8, 128, 64
    pages = 2 ** 31 // (page * H * D) + 40
    kc, vc = (torch.empty(pages, page, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = gen(9)
    k, v = normal(g, T, H, D, dt=torch.bfloat16), normal(g, T, H, D, dt=torch.bfloat16)
    slots = torch.tensor([pages * page - 1, 2 ** 31 // (H * D) + 5, 7], device="cuda")
    rn.paged_kv_append(k, v, kc, vc, slots)
    assert torch.equal(kc.view(-1, H, D)[slots], k) and torch.equal(vc.view(-1, H, D)[slots], v)


def test_append_refusals(rn):
    g = gen(10)
    k = normal(g, 4, 2, 64, dt=torch.bfloat16)
    c = torch.zeros(3, 8, 2, 64, dtype=torch.bfloat16, device="cuda")
    s = torch.arange(4, device="cuda")
    p, f = torch.zeros(4, dtype=torch.int32, device="cuda"), freqs(32)
    w = torch.ones(64, device="cuda")
    bad = [
        lambda: rn.paged_kv_append(k, k[:3], c, c, s), lambda: rn.paged_kv_append(k, k, c, c[:2], s),
        lambda: rn.paged_kv_append(k, k, c[:, :, :1], c[:, :, :1], s), lambda: rn.paged_kv_append(k, k, c.half(), c.half(), s),
        lambda: rn.paged_kv_append(k, k, c, c, s.int()), lambda: rn.paged_kv_append(k, k, c, c, s[:3]),
        lambda: rn.paged_kv_append(k, k, c, c, s, inv_freq=f), lambda: rn.paged_kv_append(k, k, c, c, s, wq=w),
        lambda: rn.paged_kv_append(k, k, c, c, s, q=k[:2]), lambda: rn.paged_kv_append(k, k, c, c, s, wk=w[:32]),
        lambda: rn.paged_kv_append(k, k, c, c, s, wk=w.half()), lambda: rn.paged_kv_append(k, k, c, c, s[::2]),
        lambda: rn.paged_kv_append(k, k, c, c, s, q=k, wq=w, wk=w.bfloat16()),
        lambda: rn.paged_kv_append(k, k, c, c, s, p[:3], f),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(rn.RMSNormError):
        rn.paged_kv_append(k, k, c, c, s, eps=-1.0)


# --------------------------------------------------------------- attention --

def paged(g, lens, page, hk, D, dt, spare=3, fill=None):
    """Caches, table and lens for sequences of these lengths; what no sequence
    holds (spare pages, the places behind its end) is `fill`."""
    n = [-(-x // page) for x in lens]
    total = sum(n) + spare
    order = torch.randperm(total, generator=g, device="cuda").int()
    table = torch.full((len(lens), max(n + [1])), -7, dtype=torch.int32, device="cuda")
    kc, vc = normal(g, total, page, hk, D, dt=dt), normal(g, total, page, hk, D, dt=dt)
    held = torch.zeros(total, page, dtype=torch.bool, device="cuda")
    at = 0
    for b, m in enumerate(n):
        table[b, :m] = order[at:at + m]
        at += m
        slot = torch.arange(lens[b], device="cuda")
        held[table[b].long()[slot // page], slot % page] = True
    if fill is not None:
        kc[~held] = fill
        vc[~held] = fill
    return kc, vc, table, torch.tensor(lens, dtype=torch.int32, device="cuda")


def starts(nq):
    return torch.tensor([sum(nq[:i]) for i in range(len(nq) + 1)], dtype=torch.int32, device="cuda")


def attended(q, kc, vc, table, lens, nq, causal, scale):
    """(o, lse, bound of o, bound of lse) in 64 bits."""
    T, hq, D = q.shape
    page, hk = kc.shape[1], kc.shape[2]
    h = half_step(q.dtype)
    o = torch.zeros(T, hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device="cuda")
    bo, bl = torch.zeros_like(o), torch.zeros_like(lse)
    at = 0
    for b, (n, m) in enumerate(zip(nq, lens)):
        j = torch.arange(m, device="cuda")
        pg = table[b].long()[j // page] if m else j
        k, v = kc[pg, j % page].double(), vc[pg, j % page].double()     # [m, hk, D]
        i = torch.arange(n, device="cuda")
        seen = (j <= m - n + i[:, None]) if causal else torch.ones(n, m, dtype=torch.bool, device="cuda")
        for head in range(hq):
            kk, vv = k[:, head * hk // hq], v[:, head * hk // hq]
            qq = q[at:at + n, head].double()
            x = (scale * qq @ kk.t()).masked_fill(~seen, -math.inf)
            some = seen.any(-1)
            ls = torch.logsumexp(x, -1)
            w = torch.exp(x - torch.where(some, ls, 0.0)[:, None])
            dx = 2.0 ** -20 * scale * (qq.abs() @ kk.abs().t()) + 2.0 ** -22 * x.abs()
            dx = dx.masked_fill(~seen, 0.0).amax(-1) if m else torch.zeros(n, dtype=torch.float64, device="cuda")
            o[at:at + n, head] = w @ vv
            lse[at:at + n, head] = ls
            bo[at:at + n, head] = (w @ vv.abs()) * (h + 2 * dx + 2.0 ** -19)[:, None] + h * (w @ vv).abs()
            if q.dtype == torch.float16:
                bo[at:at + n, head] += 2.0 ** -25 * (seen.double() @ vv.abs()) * w.amax(-1, keepdim=True) if m else 0
            bl[at:at + n, head] = dx + 2.0 ** -20 * (1 + torch.where(some, ls, 0.0).abs())
        at += n
    return o, lse, bo, bl


def check_attention(rn, q, kc, vc, table, lens, nq, causal=True, scale=None, **kw):
    lens_l = lens.tolist()
    s = 1 / math.sqrt(q.shape[2]) if scale is None else scale
    out, lse = rn.paged_attn_fwd(q, kc, vc, table, lens, starts(nq), max_q=max(nq), max_kv=max(lens_l), causal=causal,
                                 scale=scale, lse=True, **kw)
    o, l, bo, bl = attended(q[:sum(nq)], kc, vc, table, lens_l, nq, causal, s)
    n = sum(nq)
    near(out[:n], o, bo)
    some = torch.isfinite(l)
    assert torch.equal(torch.isfinite(lse[:n]), some) and bool((lse[:n][~some] == -math.inf).all())
    near(lse[:n][some], l[some], bl[some])
    return out, lse


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("nq,lens,hq,hk,D,page", [
    ([1], [1], 1, 1, 64, 8),                        # one token, one key
    ([1], [129], 8, 1, 128, 16),                    # a tile and one key
    ([1, 1, 1], [5, 0, 700], 4, 2, 128, 16),        # a sequence without keys
    ([1] * 9, [64, 1, 2, 127, 128, 129, 255, 256, 1000], 16, 2, 80, 24),
    ([1, 1], [2048, 3000], 32, 8, 128, 128),        # split over the keys
    ([3, 7, 1, 5], [3, 300, 1, 640], 12, 4, 96, 40),
    ([16], [16], 4, 4, 32, 8),
    ([64], [64], 1, 1, 128, 64),                    # 64 rows: the small geometry's most
    ([65], [65], 1, 1, 128, 64),                    # 65: the large one's least
    ([128, 129], [128, 400], 2, 1, 64, 64),
    ([300, 1, 77], [300, 513, 1000], 6, 2, 128, 256),
    ([40, 3], [90, 333], 7, 1, 112, 56),            # seven heads a group
    ([9], [500], 16, 1, 72, 8),
    ([2, 5], [260, 77], 128, 1, 128, 16),           # 128 heads a group
    ([257], [1100], 3, 3, 8, 16),                   # the smallest head
    ([20, 30], [10, 40], 4, 2, 64, 16),             # more new tokens than keys: empty rows
])
@pytest.mark.parametrize("causal", [True, False])
def test_attention(rn, dt, nq, lens, hq, hk, D, page, causal):
    g, t = gen(sum(lens) + D), TYPES[dt]
    kc, vc, table, ln = paged(g, lens, page, hk, D, t)
    q = normal(g, sum(nq), hq, D, dt=t)
    check_attention(rn, q, kc, vc, table, ln, nq, causal)


@pytest.mark.parametrize("nq,lens,hq,hk,D,page", [
    ([1], [20011], 4, 1, 128, 16),                               # more splits than a cluster has: joined by a kernel
    ([2, 1], [9000, 16500], 2, 1, 64, 32),
    ([1] * 40, [5000 - 97 * i for i in range(40)], 16, 8, 64, 16),   # several items a CTA, 40 sequences
    ([1, 3, 0, 2] * 5, [4200, 17, 900, 5001] * 5, 32, 16, 64, 8),    # in the order of their lengths, one without tokens
    ([300, 0, 70, 129, 1], [2100, 40, 3333, 1000, 1], 8, 4, 128, 8),  # the same with row tiles, small pages
    ([1500, 700], [1500, 700], 32, 16, 64, 24),                  # several row tiles a CTA, pages that end inside a tile
    ([700], [900], 10, 10, 96, 16),
    ([33, 5], [4000, 2500], 5, 5, 128, 64),                      # row tiles whose keys are split
])
def test_attention_many_items(rn, nq, lens, hq, hk, D, page):
    """Every way of cutting the work: clusters, splits joined by a kernel, items
    handed from CTA to CTA, row tiles that one split holds beside ones that are
    split."""
    g = gen(sum(nq) + D)
    kc, vc, table, ln = paged(g, lens, page, hk, D, torch.bfloat16, fill=float("nan"))
    q = normal(g, sum(nq), hq, D, dt=torch.bfloat16)
    a, _ = check_attention(rn, q, kc, vc, table, ln, nq)
    b = rn.paged_attn_fwd(q, kc, vc, table, ln, starts(nq), max_q=max(nq), max_kv=max(lens))[0]
    assert torch.equal(a, b)


@pytest.mark.parametrize("nq,lens,hq,hk,max_kv", [
    ([1] * 40, [5000 - 97 * i for i in range(40)], 16, 8, 2 ** 20),     # more than one CTA a place, lengths far below
    ([1] * 24, [4200, 17, 900, 5001] * 6, 16, 8, 2 ** 18),              # the same in the order of their lengths
    ([2] * 70, [1, 2100, 350, 0, 4097] * 14, 16, 16, 2 ** 22),
    ([1], [4095], 8, 2, 2 ** 21), ([90, 200], [500, 3000], 4, 2, 2 ** 21),
])
def test_attention_with_a_bound_far_above_the_lengths(rn, nq, lens, hq, hk, max_kv):
    """max_kv is the largest length of all replays of a captured call: results
    and the memory taken do not go by it."""
    g = gen(27)
    D, page = 64, 16
    kc, vc, table, ln = paged(g, lens, page, hk, D, torch.bfloat16, fill=float("nan"))
    wide = torch.full((len(lens), max_kv // page), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    q = normal(g, sum(nq), hq, D, dt=torch.bfloat16)
    out, lse = rn.paged_attn_fwd(q, kc, vc, wide, ln, starts(nq), max_q=max(nq), max_kv=max_kv, lse=True)
    o, l, bo, bl = attended(q, kc, vc, table, lens, nq, True, 1 / math.sqrt(D))
    near(out, o, bo)
    some = torch.isfinite(l)
    assert bool((lse[~some] == -math.inf).all())
    near(lse[some], l[some], bl[some])


@pytest.mark.parametrize("batch,hk", [(1, 13), (7, 2), (15, 1), (4, 4), (19, 1), (1, 23), (5, 6), (6, 8)])
@pytest.mark.parametrize("kv", [2100, 9000])
def test_attention_as_many_clusters_as_the_device_holds(rn, batch, hk, kv):
    """Numbers of clusters around those that run at once."""
    g = gen(batch * hk + kv)
    lens = [kv - 97 * i for i in range(batch)]
    kc, vc, table, ln = paged(g, lens, 16, hk, 128, torch.bfloat16, fill=float("nan"))
    q = normal(g, batch, 2 * hk, 128, dt=torch.bfloat16)
    check_attention(rn, q, kc, vc, table, ln, [1] * batch)


def test_attention_workspace_is_bounded_in_max_kv(rn):
    """Partial results of at most 32 items for each CTA that the device holds
    (two of 64 rows an SM), whatever the bound on the lengths."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    D = 128
    most = 32 * (2 * sms) * 64 * (D + 1) * 4 + 512
    for batch, hq, hk, max_q in ((128, 64, 8, 1), (128, 64, 8, 4), (40, 16, 8, 8), (24, 32, 8, 1), (1, 8, 1, 8), (7, 8, 8, 64)):
        for max_kv in (4096, 8192, 2 ** 15, 2 ** 20, 2 ** 30):
            assert rn.paged_attn_workspace_bytes(batch * max_q, batch, hq, hk, D, max_q, max_kv) <= most


@pytest.mark.parametrize("fill", [None, float("nan")])
@pytest.mark.parametrize("hq,hk,D,page", [(128, 8, 112, 256), (24, 8, 128, 256), (16, 8, 64, 128), (32, 8, 128, 16)])
def test_attention_last_piece_of_one_or_four_tiles(rn, fill, hq, hk, D, page):
    """Keys cut over a cluster, the last piece one tile (or four) whose values
    end inside a page: the rows' statistics take shared memory that the tile's
    values are still read from until its last product is done."""
    lens = [729, 636, 974, 667, 518, 965, 706, 297, 0, 1133, 839, 20, 996, 93, 1085, 0, 295]
    nq = [1, 1, 1, 1, 1, 0] + [1] * 11
    for seed in range(4):
        g = gen(seed + D)
        kc, vc, table, ln = paged(g, lens, page, hk, D, torch.float16, fill=fill)
        q = normal(g, sum(nq), hq, D, dt=torch.float16)
        check_attention(rn, q, kc, vc, table, ln, nq, causal=False)


@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 56), (24, 8)])
def test_attention_short_items_that_end_inside_a_page(rn, off, D, page):
    """Four items a CTA and one key tile each: the copies run two items ahead of
    the products, and so does the mending of the values past the end."""
    lens = [1 + (37 * i) % 127 for i in range(80)]
    nq = [128] * 80
    g = gen(D + off)
    kc, vc, table, ln = paged(g, lens, page, 8, D, torch.bfloat16, fill=float("nan"))
    q = offset_view(normal(g, sum(nq), 16, D, dt=torch.bfloat16), off)
    check_attention(rn, q, kc, vc, table, ln, nq, causal=False)


@pytest.mark.parametrize("hk,group,D", [(3, 128, 104), (3, 16, 16), (6, 5, 128)])
def test_attention_items_with_an_empty_row_tile_and_unaligned_q(rn, hk, group, D):
    """Several items a CTA, the second row tile of most empty, q by plain loads:
    a tile without rows does not get ahead of the other's q."""
    per = 2 * (128 // group)
    nq = [(1, per // 2, per + 1, 0, per)[i % 5] for i in range(120)]
    lens = [16 * (1 + (7 * i) % 40) for i in range(120)]
    g = gen(D)
    kc, vc, table, ln = paged(g, lens, 16, hk, D, torch.bfloat16)
    q = offset_view(normal(g, sum(nq), hk * group, D, dt=torch.bfloat16), 1)
    check_attention(rn, q, kc, vc, table, ln, nq, causal=False)


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("nq,lens,page", [([1, 1], [77, 1030], 16), ([1], [3], 256), ([200, 9], [205, 130], 48),
                                          ([1], [0], 8)])
def test_attention_never_sees_what_lies_behind_a_sequence(rn, fill, nq, lens, page):
    g = gen(11)
    kc, vc, table, ln = paged(g, lens, page, 2, 128, torch.bfloat16, fill=fill)
    q = normal(g, sum(nq), 8, 128, dt=torch.bfloat16)
    check_attention(rn, q, kc, vc, table, ln, nq)


def test_attention_key_of_nan_stays_with_the_rows_that_see_it(rn):
    """A masked key's score may be anything: only its value has to be finite."""
    g = gen(12)
    nq, lens = [40], [200]
    kc, vc, table, ln = paged(g, lens, 16, 1, 64, torch.bfloat16)
    q = normal(g, 40, 2, 64, dt=torch.bfloat16)
    cu = starts(nq)
    a = rn.paged_attn_fwd(q, kc, vc, table, ln, cu, max_q=40, max_kv=200)[0]
    last = table[0, 199 // 16].item(), 199 % 16
    kc[last] = float("nan")
    b = rn.paged_attn_fwd(q, kc, vc, table, ln, cu, max_q=40, max_kv=200)[0]
    assert torch.equal(a[:39], b[:39]) and bool(torch.isnan(b[39]).all())


@pytest.mark.parametrize("nq", [[1, 1], [150, 60]])
def test_attention_rows_of_growing_scores(rn, nq):
    """Scores that grow (and fall) by far more than the rescaling threshold
    from tile to tile, and a few hundred times larger than usual."""
    g = gen(13)
    lens = [900, 1500]
    kc, vc, table, ln = paged(g, lens, 16, 1, 128, torch.bfloat16)
    q = normal(g, sum(nq), 2, 128, dt=torch.bfloat16)
    for b, m in enumerate(lens):
        j = torch.arange(m, device="cuda")
        pg = table[b].long()[j // 16]
        ramp = (j // 128).float() if b == 0 else (m // 128 - j // 128).float()
        kc[pg, j % 16] = (kc[pg, j % 16].float() * (0.2 + ramp)[:, None, None]).bfloat16()
    check_attention(rn, q, kc, vc, table, ln, nq, scale=0.5)


def test_attention_layouts(rn):
    """Strided q and out, off a 16-byte boundary, a cache with the heads before
    the places, a table wider than needed: the same bits."""
    g = gen(14)
    nq, lens, hq, hk, D, page = [5, 70], [200, 333], 6, 2, 96, 16
    t = torch.bfloat16
    kc, vc, table, ln = paged(g, lens, page, hk, D, t)
    q = normal(g, sum(nq), hq, D, dt=t)
    a, lse = check_attention(rn, q, kc, vc, table, ln, nq)
    kw = dict(max_q=70, max_kv=333)
    cu = starts(nq)
    wide = torch.full((2, 64), 2 ** 30, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    assert torch.equal(rn.paged_attn_fwd(q, kc, vc, wide, ln, cu, **kw)[0], a)
    assert torch.equal(rn.paged_attn_fwd(offset_view(q, 1), kc, vc, table, ln, cu, **kw)[0], a)
    big = torch.zeros(sum(nq), hq + 3, D + 8, dtype=t, device="cuda")
    big[:, 1:hq + 1, :D] = q
    assert torch.equal(rn.paged_attn_fwd(big[:, 1:hq + 1, :D], kc, vc, table, ln, cu, **kw)[0], a)
    out = torch.zeros(sum(nq), hq, D + 1, dtype=t, device="cuda")[..., :D]
    assert rn.paged_attn_fwd(q, kc, vc, table, ln, cu, out=out, **kw)[0] is out and torch.equal(out, a)
    both = torch.empty(kc.shape[0], 2, hk, page, D, dtype=t, device="cuda")
    both[:, 0], both[:, 1] = kc.transpose(1, 2), vc.transpose(1, 2)
    got = rn.paged_attn_fwd(q, both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2), table, ln, cu, **kw)
    assert torch.equal(got[0], a) and got[1] is None
    given = torch.zeros_like(lse)
    assert rn.paged_attn_fwd(q, kc, vc, table, ln, cu, lse=given, **kw)[1] is given and torch.equal(given, lse)


@pytest.mark.parametrize("nq,lens", [([1, 2], [900, 40]), ([90, 3], [900, 40])])
def test_attention_leaves_rows_behind_the_last_sequence(rn, nq, lens):
    g = gen(15)
    kc, vc, table, ln = paged(g, lens, 16, 2, 64, torch.bfloat16)
    q = normal(g, sum(nq) + 70, 4, 64, dt=torch.bfloat16)
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    rn.paged_attn_fwd(q, kc, vc, table, ln, starts(nq), max_q=max(nq), max_kv=900, out=out, lse=lse)
    assert bool((out[sum(nq):] == 7.0).all()) and bool((lse[sum(nq):] == 7.0).all())
    assert not bool((out[:sum(nq)] == 7.0).all(-1).any())


def test_attention_lengths_are_held_to_the_call(rn):
    """Lengths beyond max_kv or the table, rows beyond max_q or T, negative
    lengths, table entries that are no page: in bounds, and the rest right."""
    g = gen(16)
    kc, vc, table, ln = paged(g, [100, 60], 16, 2, 64, torch.float16)
    q = normal(g, 4, 4, 64, dt=torch.float16)
    cu = starts([2, 2])
    a = rn.paged_attn_fwd(q, kc, vc, table, ln, cu, max_q=2, max_kv=100)[0]
    lens = torch.tensor([100, 10 ** 9], dtype=torch.int32, device="cuda")
    b = rn.paged_attn_fwd(q, kc, vc, table, lens, cu, max_q=2, max_kv=100)[0]
    assert torch.equal(a[:2], b[:2]) and bool(torch.isfinite(b).all())
    lens = torch.tensor([-5, 60], dtype=torch.int32, device="cuda")
    b = rn.paged_attn_fwd(q, kc, vc, table, lens, cu, max_q=2, max_kv=100)[0]
    assert torch.equal(a[2:], b[2:]) and bool((b[:2] == 0).all())
    out = torch.full_like(q, 7.0)
    far = torch.tensor([0, 2, 10 ** 6], dtype=torch.int32, device="cuda")
    rn.paged_attn_fwd(q, kc, vc, table, ln, far, max_q=1, max_kv=100, out=out)
    assert bool((out[[1, 3]] == 7.0).all())
    bad = table.clone()
    bad[1] = torch.tensor([2 ** 31 - 1, -1, 10 ** 6, 3] + [0] * (table.shape[1] - 4), dtype=torch.int32)[:table.shape[1]]
    b = rn.paged_attn_fwd(q, kc, vc, bad, ln, cu, max_q=2, max_kv=100)[0]
    assert torch.equal(a[:2], b[:2]) and bool(torch.isfinite(b).all())


def test_attention_of_an_empty_cache(rn):
    q = torch.ones(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    c = torch.zeros(0, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(1, 0, dtype=torch.int32, device="cuda")
    ln = torch.tensor([9], dtype=torch.int32, device="cuda")
    out, lse = rn.paged_attn_fwd(q, c, c, table, ln, starts([3]), max_q=3, max_kv=9, lse=True)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    none = rn.paged_attn_fwd(q[:0], c, c, table, ln, starts([0]), max_q=0, max_kv=0)[0]
    assert none.shape == (0, 4, 64)


def test_attention_far_in_a_large_cache(rn):
    """Pages whose offsets pass 2^32 bytes and 2^31 elements."""
    g = gen(17)
    H, D, page = 8, 128, 64
    pages = 2 ** 31 // (page * H * D) + 40
    kc, vc = (torch.empty(pages, page, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.tensor([[pages - 1, 3, pages - 17]], dtype=torch.int32, device="cuda")
    for i in table[0].tolist():
        kc[i], vc[i] = normal(g, page, H, D, dt=torch.bfloat16), normal(g, page, H, D, dt=torch.bfloat16)
    q = normal(g, 2, 16, D, dt=torch.bfloat16)
    check_attention(rn, q, kc, vc, table, torch.tensor([150], dtype=torch.int32, device="cuda"), [2])


@pytest.mark.parametrize("nq,lens", [([1, 1], [1000, 4000]), ([100, 30], [100, 700])])
def test_attention_same_bits_stream_workspace_and_graph(rn, nq, lens):
    """The same call twice, on another stream (its memory stream-ordered), with
    a workspace given (its contents do not matter), and captured into a graph
    that is replayed on other lengths, tables and queries."""
    g = gen(18)
    hq, hk, D, page = 8, 2, 128, 16
    kc, vc, table, ln = paged(g, lens, page, hk, D, torch.bfloat16)
    q = normal(g, sum(nq), hq, D, dt=torch.bfloat16)
    cu = starts(nq)
    kw = dict(max_q=max(nq), max_kv=max(lens))
    a, la = rn.paged_attn_fwd(q, kc, vc, table, ln, cu, lse=True, **kw)
    again = rn.paged_attn_fwd(q, kc, vc, table, ln, cu, lse=True, **kw)
    assert torch.equal(a, again[0]) and torch.equal(la, again[1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = torch.empty_like(q)
    rn.paged_attn_fwd(q, kc, vc, table, ln, cu, out=out, stream=side, **kw)
    side.synchronize()
    assert torch.equal(a, out)
    need = rn.paged_attn_workspace_bytes(sum(nq), len(nq), hq, hk, D, max(nq), max(lens))
    if need:
        ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
        assert torch.equal(rn.paged_attn_fwd(q, kc, vc, table, ln, cu, workspace=ws, **kw)[0], a)
        with pytest.raises(rn.RMSNormError, match="WORKSPACE"):
            rn.paged_attn_fwd(q, kc, vc, table, ln, cu, workspace=ws[:need - 256], **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = rn.paged_attn_fwd(q, kc, vc, table, ln, cu, **kw)[0]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(captured, a)
    q.copy_(normal(g, *q.shape, dt=torch.bfloat16))
    ln.copy_(torch.tensor([lens[0] - 99, lens[1] // 2], dtype=torch.int32))
    table.copy_(table.roll(1, 0).clamp(min=0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(captured, rn.paged_attn_fwd(q, kc, vc, table, ln, cu, **kw)[0])


@pytest.mark.parametrize("nq,lens", [([1, 2], [3000, 77]), ([150, 64], [900, 64]), ([60], [3000])])
def test_attention_in_place(rn, nq, lens):
    """out may be q."""
    g = gen(21)
    kc, vc, table, ln = paged(g, lens, 16, 2, 128, torch.bfloat16)
    q = normal(g, sum(nq), 8, 128, dt=torch.bfloat16)
    kw = dict(max_q=max(nq), max_kv=max(lens))
    a = rn.paged_attn_fwd(q, kc, vc, table, ln, starts(nq), **kw)[0]
    rn.paged_attn_fwd(q, kc, vc, table, ln, starts(nq), out=q, **kw)
    assert torch.equal(q, a)


def test_calls_on_two_streams_at_once(rn):
    """Attention with a join's workspace and appends on two streams, many times
    over, each with its own results."""
    g = gen(22)
    sides = []
    for i in range(2):
        lens = [20011 + 999 * i]
        kc, vc, table, ln = paged(g, lens, 16, 1, 64, torch.bfloat16)
        q = normal(g, 1, 4, 64, dt=torch.bfloat16)
        sides.append((torch.cuda.Stream(), q, kc, vc, table, ln, max(lens), []))
    want = [rn.paged_attn_fwd(q, kc, vc, t, ln, starts([1]), max_q=1, max_kv=m)[0]
            for _, q, kc, vc, t, ln, m, _ in sides]
    cu = starts([1])
    torch.cuda.synchronize()
    for _ in range(20):
        for s, q, kc, vc, t, ln, m, got in sides:
            with torch.cuda.stream(s):
                got.append(rn.paged_attn_fwd(q, kc, vc, t, ln, cu, max_q=1, max_kv=m)[0])
    torch.cuda.synchronize()
    for w, side in zip(want, sides):
        assert all(torch.equal(w, x) for x in side[-1])


def test_appends_and_rotations_on_two_streams_at_once(rn):
    """Each stream appends to its own cache and rotates in place, many times
    over, beside the other."""
    g = gen(31)
    T, H, D, page, pages = 4096, 8, 128, 16, 300
    pos, f, w = torch.arange(T, device="cuda"), freqs(64), normal(g, D)
    sides = []
    for _ in range(2):
        q, k, v = (normal(g, T, H, D, dt=torch.bfloat16) for _ in range(3))
        slots = torch.randperm(pages * page, generator=g, device="cuda")[:T]
        caches = [torch.zeros(pages, page, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        sides.append((torch.cuda.Stream(), q, k, v, slots, caches, q.clone()))

    def step(q, k, v, slots, caches, x):
        a = rn.paged_kv_append(k, v, *caches, slots, pos, f, q=q, wq=w, wk=w)
        rn.rope_fwd(x, None, pos, f, q_out=x)
        rn.rope_bwd(x, None, pos, f, dq_out=x)
        return a, x.clone()

    want = []
    for _, q, k, v, slots, caches, x in sides:
        first = step(q, k, v, slots, caches, x.clone())
        want.append([*first, *(c.clone() for c in caches)])
        for c in caches:
            c.zero_()
    torch.cuda.synchronize()
    got = [None, None]
    for i in range(20):
        for n, (s, q, k, v, slots, caches, x) in enumerate(sides):
            with torch.cuda.stream(s):
                got[n] = step(q, k, v, slots, caches, x) if i == 0 else (step(q, k, v, slots, caches, x)[0], got[n][1])
    torch.cuda.synchronize()
    for side, w4, g2 in zip(sides, want, got):
        assert all(torch.equal(a, b) for a, b in zip(w4, [*g2, *side[5]]))


def test_results_made_for_a_named_stream(rn):
    """With stream= and no result given, the call makes them and their memory
    is not handed out again while that stream still writes it."""
    g = gen(24)
    T, H, D = 4000, 8, 128
    q = normal(g, T, H, D, dt=torch.bfloat16)
    pos, f = torch.arange(T, device="cuda"), freqs(64)
    want = rn.rope_fwd(q, q, pos, f)
    kc, vc, table, ln = paged(g, [300], 16, 8, D, torch.bfloat16)
    kw = dict(max_q=200, max_kv=300, lse=True)
    o, l = rn.paged_attn_fwd(q[:200], kc, vc, table, ln, starts([200]), **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        a = rn.rope_fwd(q, q, pos, f, stream=handle)
        b = rn.paged_attn_fwd(q[:200], kc, vc, table, ln, starts([200]), stream=handle, **kw)
        rn.rope_fwd(q, q, pos, f, stream=handle)          # dropped at once
        other = torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(a[0], want[0]) and torch.equal(a[1], want[1])
        assert torch.equal(b[0], o) and torch.equal(b[1], l) and not bool(other.any())


@pytest.mark.parametrize("op", ["rope", "append", "attn", "lse"])
def test_results_for_a_named_stream_are_not_memory_in_use_on_the_current_one(rn, op):
    """The current stream still has a late read and a late write of a block
    queued that has been dropped. What a call on another stream makes, which
    waits for none of that, must lie elsewhere."""
    g = gen(25)
    T, H, D = 2048, 8, 128
    q, k = (normal(g, T, H, D, dt=torch.bfloat16) for _ in range(2))
    pos, f = torch.arange(T, device="cuda"), freqs(64)
    kc, vc, table, ln = paged(g, [T], 16, H, D, torch.bfloat16)
    cu, slots = starts([T]), torch.arange(T, device="cuda")
    lse = torch.empty(T, H, device="cuda")
    out = torch.empty_like(q)

    def call(**kw):
        if op == "rope":
            return rn.rope_fwd(q, None, pos, f, **kw)[0]
        if op == "append":
            return rn.paged_kv_append(k, k, kc, vc, slots, pos, f, q=q, **kw)
        if op == "attn":
            return rn.paged_attn_fwd(q, kc, vc, table, ln, cu, max_q=T, max_kv=T, lse=lse, **kw)[0]
        return rn.paged_attn_fwd(q, kc, vc, table, ln, cu, max_q=T, max_kv=T, lse=True, out=out, **kw)[1]

    want = call()
    kept = torch.empty_like(want)
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        block = torch.full_like(want, 3.0)  # of the result's size: the next one of this pool
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)
        kept.copy_(block)
        block.fill_(5.0)
        del block
        got = call(stream=handle)
        torch.cuda.synchronize()
        assert bool((kept == 3.0).all()) and torch.equal(got, want)
        del got


@pytest.mark.parametrize("handle", [0, 1, 2])
def test_results_on_the_default_streams_by_handle(rn, handle):
    """CUDA's handles of the legacy default stream (0 and 1) and of the
    thread's own default one (2)."""
    g = gen(26)
    q, pos, f = normal(g, 9, 4, 64), torch.arange(9, device="cuda"), freqs(32)
    want = rn.rope_fwd(q, None, pos, f)[0]
    torch.cuda.synchronize()
    got = rn.rope_fwd(q, None, pos, f, stream=handle)[0]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    del got
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def test_append_and_rope_in_a_graph(rn):
    g = gen(23)
    T, H, D = 33, 4, 64
    q, k, v = (normal(g, T, H, D, dt=torch.float16) for _ in range(3))
    kc, vc = (torch.zeros(8, 8, H, D, dtype=torch.float16, device="cuda") for _ in range(2))
    slots, pos, f = torch.arange(T, device="cuda"), torch.arange(T, device="cuda").int(), freqs(32)

    def run():
        r, _ = rn.rope_fwd(q, None, pos, f)
        b, _ = rn.rope_bwd(r, None, pos, f)
        a = rn.paged_kv_append(k, v, kc, vc, slots, pos, f, q=q)
        return r, b, a

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, b, a = run()
    q.copy_(normal(g, T, H, D, dt=torch.float16))
    k.copy_(normal(g, T, H, D, dt=torch.float16))
    pos.add_(1000)
    slots.copy_(torch.arange(T, device="cuda").flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(r, a)
    want = [x.clone() for x in (r, kc, vc)]
    run()
    torch.cuda.synchronize()
    assert torch.equal(rn.rope_fwd(q, None, pos, f)[0], want[0])
    assert torch.equal(kc, want[1]) and torch.equal(vc, want[2])
    near(b, q.double(), 8 * half_step(torch.float16) * (q.double().abs() + q.double().abs().roll(D // 2, -1)))


def test_results_that_overlap_themselves_are_refused(rn):
    """An expanded tensor as a result or a cache; as an input it is fine, and
    so is a stride of 0 over a single entry."""
    g = gen(30)
    t = torch.bfloat16
    kc, vc, table, ln = paged(g, [20], 16, 2, 64, t)
    q, k = normal(g, 4, 4, 64, dt=t), normal(g, 4, 2, 64, dt=t)
    p, f, s = torch.arange(4, device="cuda"), freqs(32), torch.arange(4, device="cuda")
    cu, kw = starts([4]), dict(max_q=4, max_kv=20)
    for out in (q[:1].expand(4, 4, 64), q[:, :1].expand(4, 4, 64)):
        for call in (lambda: rn.rope_fwd(q, None, p, f, q_out=out), lambda: rn.rope_bwd(q, None, p, f, dq_out=out),
                     lambda: rn.paged_kv_append(k, k, kc, vc, s, q=q, q_out=out),
                     lambda: rn.paged_attn_fwd(q, kc, vc, table, ln, cu, out=out, **kw)):
            with pytest.raises(rn.RMSNormError, match="INVALID"):
                call()
    for c in (kc[:1].expand_as(kc), kc[:, :1].expand_as(kc), kc[:, :, :1].expand_as(kc)):
        for pair in ((c, vc), (kc, c)):
            with pytest.raises(rn.RMSNormError, match="INVALID"):
                rn.paged_kv_append(k, k, *pair, s)
    assert torch.equal(rn.rope_fwd(q[:1].expand(4, 4, 64), None, p, f)[0], rn.rope_fwd(q[[0] * 4], None, p, f)[0])
    one = torch.empty(1, 1, 64, dtype=t, device="cuda").as_strided((1, 1, 64), (0, 0, 1))
    assert torch.equal(rn.rope_fwd(q[:1, :1], None, p[:1], f, q_out=one)[0], rn.rope_fwd(q[:1, :1], None, p[:1], f)[0])


def test_attention_refusals(rn):
    g = gen(19)
    kc, vc, table, ln = paged(g, [20], 16, 2, 64, torch.bfloat16)
    q = normal(g, 1, 4, 64, dt=torch.bfloat16)
    cu = starts([1])
    kw = dict(max_q=1, max_kv=20)
    bad = [
        lambda: rn.paged_attn_fwd(q[0], kc, vc, table, ln, cu, **kw), lambda: rn.paged_attn_fwd(q, kc[0], vc[0], table, ln, cu, **kw),
        lambda: rn.paged_attn_fwd(q, kc, vc[:-1], table, ln, cu, **kw), lambda: rn.paged_attn_fwd(q.half(), kc, vc, table, ln, cu, **kw),
        lambda: rn.paged_attn_fwd(q, kc, vc, table.long(), ln, cu, **kw), lambda: rn.paged_attn_fwd(q, kc, vc, table[0], ln, cu, **kw),
        lambda: rn.paged_attn_fwd(q, kc, vc, table, ln.long(), cu, **kw), lambda: rn.paged_attn_fwd(q, kc, vc, table, ln, cu[:1], **kw),
        lambda: rn.paged_attn_fwd(q, kc, vc, table, ln, cu, max_q=-1, max_kv=20),
        lambda: rn.paged_attn_fwd(q, kc, vc, table, ln, cu, max_q=1, max_kv=2 ** 40),
        lambda: rn.paged_attn_fwd(q, kc, vc, table, ln, cu, out=q[:, :2], **kw),
        lambda: rn.paged_attn_fwd(q, kc, vc, table, ln, cu, lse=torch.zeros(3, device="cuda"), **kw),
        lambda: rn.paged_attn_fwd(q, kc, vc, table.cpu(), ln, cu, **kw),
        lambda: rn.paged_attn_fwd(q, kc, vc, table, ln, cu, workspace=torch.zeros(4), **kw),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("accepted", i)
    for call in (lambda: rn.paged_attn_fwd(q, kc, vc, table, ln, cu, scale=0.0, **kw),
                 lambda: rn.paged_attn_fwd(q.float(), kc.float(), vc.float(), table, ln, cu, **kw),
                 lambda: rn.paged_attn_fwd(q[..., :60], kc[..., :60], vc[..., :60], table, ln, cu, **kw),
                 lambda: rn.paged_attn_fwd(q, kc[:, :12], vc[:, :12], table, ln, cu, **kw),
                 lambda: rn.paged_attn_fwd(q[:, :3], kc, vc, table, ln, cu, **kw)):
        with pytest.raises(rn.RMSNormError):
            call()
    with pytest.raises(TypeError):
        rn.paged_attn_fwd(q, kc, vc, table, ln, cu, max_q="1", max_kv=20)


# --------------------------------------------------------- a run of them --

@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_prompt_then_tokens(rn, dt):
    """Per-head norm, rotation, append and attention as a model runs them: a
    prompt in two chunks, then single tokens, for two sequences. The fused
    append agrees with rmsnorm_fwd and rope_fwd one after the other within
    the rounding between them, and every step's attention with the definition
    on the cache as it then stands."""
    g, t = gen(20), TYPES[dt]
    hq, hk, D, page = 8, 2, 128, 16
    lens, width = [0, 0], 12
    kc, vc = (torch.full((40, page, hk, D), float("nan"), dtype=t, device="cuda") for _ in range(2))
    table = torch.randperm(40, generator=g, device="cuda").int()[:2 * width].view(2, width)
    wq, wk = (1 + 0.1 * normal(g, D)).to(t), (1 + 0.1 * normal(g, D)).to(t)
    f, axes = freqs(64), rn.rope_axes((32, 32))
    for new in ([70, 33], [50, 1], [1, 1], [1, 1], [1, 1]):
        T = sum(new)
        qkv = normal(g, T, hq + 2 * hk, D, dt=t)
        q, k, v = qkv.split([hq, hk, hk], dim=1)
        where = torch.cat([torch.arange(n, n + m) for n, m in zip(lens, new)]).cuda()
        seq = torch.cat([torch.full((m,), b) for b, m in enumerate(new)]).cuda()
        slots = table[seq, where // page].long() * page + where % page
        pos = torch.stack([where, where // 3]).int()
        lens = [n + m for n, m in zip(lens, new)]
        qr = rn.paged_kv_append(k, v, kc, vc, slots, pos, f, axes=axes, q=q, wq=wq, wk=wk)
        qn = rn.rmsnorm_fwd(q.contiguous(), wq)[0]
        kn = rn.rmsnorm_fwd(k.contiguous(), wk)[0]
        q2, k2 = rn.rope_fwd(qn, kn, pos, f, axes=axes)
        # the unfused path rounds the normalised values once more
        slack = 4 * half_step(t)
        for a, b in ((qr, q2), (kc.view(-1, hk, D)[slots], k2)):
            pair = b.double().abs() + b.double().abs().roll(D // 2, -1)
            near(a, b.double(), slack * pair)
        check_attention(rn, qr, kc, vc, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), new)
