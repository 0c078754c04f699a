"""Rows of a training step on a GPU (8-bit checkpoints, group norm, embedding
rows) against their definitions in 64 bits.

Tolerances, derived from the arithmetic (u = 2^-24, half an fp32 step at 1;
h half a step of the output's type):
  codes      none: scales are powers of two, so a code's only rounding is its
             own, of an exact quotient, and the definition gives the same one.
  norms      rstd: N / 256 terms in sequence at most, a tree and the root: below
             (N / 256 + 40) u. Three products more for y.
  group norm A sum of n terms in sequence is off by n u times the sum of their
             magnitudes. L = rows of a lane + lanes + chunks + 100 bounds the terms
             in sequence. Deviations are taken from a value of the group, at most
             D = max |x - mean| away: the mean is off by L u (mean |x - mean| + D)
             + 4 u |mean|, the variance by 2 L u (var + D^2). z carries both and 4 u
             of its own terms; activations have slopes below 1.2 and an error of
             their own of (10 + 3 |z|) u (the fast exponential's 2 + 1.2 |z| ulp and
             a division; erf's 2 ulp), and the slopes' slopes are below 1.2 too.
  gradients  the errors of u = dy act'(z) summed as magnitudes, and L u times the
             sum of the magnitudes of what is added.
  embedding  32 terms in sequence in a piece, then its row's pieces: 8 lanes of
             them, in order.
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


def near(got, ref, bound, what=""):
    assert got.shape == ref.shape, what
    if got.numel() == 0:
        return
    err = (got.double() - ref).abs()
    worst = (err / (bound + 1e-300)).max().item()
    assert bool((err <= bound).all()), f"{what}: worst error {worst:.3g} of its bound"


def bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


# -------------------------------------------------------------------- 8 bits --

def kept(x):
    """codes, scales and values of x's rows by the definition, in 64 bits."""
    n = x.shape[-1]
    v = torch.nn.functional.pad(x.double(), (0, -n % 32)).unflatten(-1, (-1, 32))
    top = v.abs().amax(-1, keepdim=True)
    fine = torch.isfinite(top)
    frac, exp = torch.frexp(torch.where(fine, top, 1.0))
    k = exp - 7 + (frac >= 255 / 256).int()
    k = torch.where(top > 0, k, -127).clamp(-127, 9 if x.dtype == torch.float16 else 121)
    step = torch.exp2(k.double())  # (torch.ldexp multiplies by a power in fp32, which need not be exact)
    codes = (torch.where(fine, v, 0.0) / step).round().clamp(-127, 127)
    values = torch.where(fine, codes * step, math.nan)
    scales = torch.where(fine, k + 127, 255)[..., 0]
    return codes.flatten(-2)[..., :n], scales, values.flatten(-2)[..., :n]


def check_kept(x, codes, scales, values=None):
    c, s, v = kept(x)
    assert codes.dtype == torch.int8 and scales.dtype == torch.uint8
    assert torch.equal(scales.long(), s.long())
    fine = torch.isfinite(v)
    assert torch.equal(codes.double()[fine], c[fine])
    if values is not None:
        assert torch.equal(torch.isnan(values), ~fine)
        want = v.to(values.dtype)  # a code has 7 bits
        assert torch.equal(values[fine], want[fine])


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N", [(1, 1), (3, 31), (5, 32), (2, 33), (7, 64), (64, 1000), (1, 4096), (129, 257), (1000, 96)])
def test_pack_and_unpack(rn, dt, M, N):
    g, t = gen(M * N), TYPES[dt]
    x = (normal(g, M, N) * torch.exp2(torch.randint(-12, 12, (M, N), generator=g, device="cuda").float())).to(t)
    for k in (0, 1):
        xx = offset_view(x, k) if k else x
        codes, scales = rn.ckpt8_pack(xx)
        y = rn.ckpt8_unpack(codes, scales, t)
        check_kept(x, codes, scales, y)
        _, _, v = kept(x)
        top = torch.nn.functional.pad(x.double().abs(), (0, -N % 32)).unflatten(-1, (-1, 32)).amax(-1, keepdim=True)
        far = (torch.nn.functional.pad(y.double() - x.double(), (0, -N % 32)).unflatten(-1, (-1, 32))).abs()
        assert bool((far <= top / 127.5 + torch.finfo(t).smallest_normal * torch.finfo(t).eps).all())


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N", [256, 250])
def test_pack_at_the_types_borders(rn, dt, N):
    """Largest and smallest values, blocks of zeros, ties, the value that would round to 128 steps."""
    t = TYPES[dt]
    f = torch.finfo(t)
    x = torch.zeros(12, N, dtype=t, device="cuda")
    x[0, ::7] = f.max
    x[1, 3] = -f.max
    x[2, ::5] = f.smallest_normal
    x[3, 40] = f.smallest_normal * f.eps  # the smallest subnormal
    x[4] = torch.arange(N, device="cuda").to(t) * 0.5 - 60  # ties
    x[5, 10], x[5, 11] = 255 / 128, 1.0
    x[6, 10], x[6, 11] = 254 / 128, 1 / 128
    x[7, 100] = math.inf
    x[8, 33] = -math.inf
    x[9, 70] = math.nan
    x[10, 0], x[10, 1] = f.max, f.smallest_normal
    codes, scales = rn.ckpt8_pack(x)
    y = rn.ckpt8_unpack(codes, scales, t)
    check_kept(x, codes, scales, y)
    assert bool(torch.isfinite(y[:7]).all())


def norm_reference(h, w, offset, eps=1e-6):
    v = h.double()
    rstd = 1 / (v.square().mean(-1) + eps).sqrt()
    f = 1.0 if w is None else offset + w.double()
    return v * rstd[..., None] * f, rstd


def check_norm(y, rstd, h, w, offset):
    n = h.shape[-1]
    ref, r = norm_reference(h, w, offset)
    near(rstd, r, (n / 256 + 40) * U * r, "rstd")
    near(y, ref, (half_step(y.dtype) + (n / 256 + 48) * U) * ref.abs() + 2.0 ** -25 * (y.dtype == torch.float16), "y")


NORM_SHAPES = [(1, 1), (3, 8), (70, 64), (33, 96), (5, 250), (9, 256), (17, 1000), (4, 1024), (130, 2048), (6, 5120), (3, 8192),
               (2, 16384), (2, 20000), (3, 65536), (5, 4097)]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("M,N", NORM_SHAPES)
def test_norm_forward_keeps_its_rows(rn, dt, fused, M, N):
    g, t = gen(M + N), TYPES[dt]
    x, res = normal(g, M, N, dt=t), normal(g, M, N, dt=t) if fused else None
    wt = torch.float32 if N % 3 == 0 else t
    w = None if M == 9 else (1 + 0.1 * normal(g, N)).to(wt)
    out = rn.rmsnorm_fwd_ckpt8(x, w, residual=res, offset=0.5)
    h = x
    if fused:
        h = (x.double() + res.double()).to(t)
        assert torch.equal(out["residual_out"], h)
    else:
        assert out["residual_out"] is None
    check_norm(out["y"], out["rstd"], h, w, 0.5)
    check_kept(h, out["codes"], out["scales"])


def bwd_reference(dy, v, w, rstd, offset, dres):
    """dx, dw and the magnitudes their errors go by."""
    n = dy.shape[-1]
    f = torch.ones(n, dtype=torch.float64, device="cuda") if w is None else offset + w.double()
    xhat, r, dy = v * rstd.double()[:, None], rstd.double()[:, None], dy.double()
    g = dy * f
    c = (g * xhat).mean(-1, keepdim=True)
    dx = r * (g - xhat * c)
    err = r * U * (8 * (g.abs() + (xhat * c).abs()) + (n / 256 + 48) * xhat.abs() * (g * xhat).abs().mean(-1, keepdim=True))
    if dres is not None:
        dx, err = dx + dres.double(), err + 2 * U * dres.double().abs()
    return dx, err, (dy * xhat).sum(0), (dy * xhat).abs().sum(0)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("M,N", NORM_SHAPES + [(3000, 64), (1000, 512), (700, 1000), (2000, 33), (1, 4096)])
def test_norm_gradient_from_kept_rows(rn, dt, fused, M, N):
    g, t = gen(M * 3 + N), TYPES[dt]
    x, dy = normal(g, M, N, dt=t), normal(g, M, N, dt=t)
    dres = normal(g, M, N, dt=t) if fused else None
    wt = torch.float32 if N % 3 == 0 else t
    w = None if M == 9 else (1 + 0.1 * normal(g, N)).to(wt)
    codes, scales = rn.ckpt8_pack(x)
    _, rstd = rn.rmsnorm_fwd(x, w, offset=0.5)
    dx, dw = rn.rmsnorm_bwd_ckpt8(dy, codes, scales, w, rstd, dresidual_out=dres, offset=0.5)
    ref, err, rw, mag = bwd_reference(dy, kept(x)[2], w, rstd, 0.5, dres)
    small = 2.0 ** -25 * (t == torch.float16)
    near(dx, ref, half_step(t) * ref.abs() + err + small, "dx")
    if w is None:
        assert dw is None
    else:
        assert dw.dtype == wt
        near(dw, rw, half_step(wt) * rw.abs() + (M + 600) * U * mag + small, "dw")
    again = rn.rmsnorm_bwd_ckpt8(dy, codes, scales, w, rstd, dresidual_out=dres, offset=0.5)
    assert torch.equal(bits(again[0]), bits(dx)) and (w is None or torch.equal(bits(again[1]), bits(dw)))


@pytest.mark.parametrize("dt,N", [("bf16", 512), ("f32", 512), ("f16", 500)])
def test_norm_gradient_in_place_and_at_offsets(rn, dt, N):
    g, t, M = gen(7), TYPES[dt], 37
    x, dy, dres, w = normal(g, M, N, dt=t), normal(g, M, N, dt=t), normal(g, M, N, dt=t), normal(g, N, dt=t)
    codes, scales = rn.ckpt8_pack(x)
    _, rstd = rn.rmsnorm_fwd(x, w)
    want, wdw = rn.rmsnorm_bwd_ckpt8(dy, codes, scales, w, rstd, dresidual_out=dres)
    for name in ("dy", "dres"):
        a, b = dy.clone(), dres.clone()
        dx, dw = rn.rmsnorm_bwd_ckpt8(a, codes, scales, w, rstd, dresidual_out=b, dx=a if name == "dy" else b)
        assert torch.equal(dx, want) and torch.equal(dw, wdw)
    ref, err, rw, mag = bwd_reference(dy, kept(x)[2], w, rstd, 0.0, dres)
    small = 2.0 ** -25 * (t == torch.float16)
    # codes, scales and rstd anywhere; dy off its boundary takes the other kernels
    for k in (8, 1, 3):
        for ky in (0, 1):
            dx, dw = rn.rmsnorm_bwd_ckpt8(offset_view(dy, ky), offset_view(codes, k), offset_view(scales, k), w,
                                          offset_view(rstd, k), dresidual_out=offset_view(dres, ky))
            near(dx, ref, half_step(t) * ref.abs() + err + small, "dx")
            near(dw, rw, half_step(t) * rw.abs() + (M + 600) * U * mag + small, "dw")


def test_norm_gradient_leaves_its_surroundings(rn):
    """Codes of a view with poison behind it; results between guards."""
    M, N = 50, 200
    g = gen(3)
    x, dy, w = normal(g, M, N, dt=torch.bfloat16), normal(g, M, N, dt=torch.bfloat16), normal(g, N, dt=torch.bfloat16)
    _, rstd = rn.rmsnorm_fwd(x, w)
    codes, scales = rn.ckpt8_pack(x)
    want = rn.rmsnorm_bwd_ckpt8(dy, codes, scales, w, rstd)
    cb = torch.full((M * N + 64,), 77, dtype=torch.int8, device="cuda")
    sb = torch.full((scales.numel() + 64,), 255, dtype=torch.uint8, device="cuda")
    db = torch.full((M * N + 128,), 9.0, dtype=torch.bfloat16, device="cuda")
    cb[32:32 + M * N] = codes.flatten()
    sb[32:32 + scales.numel()] = scales.flatten()
    dx = db[64:64 + M * N].view(M, N)
    got = rn.rmsnorm_bwd_ckpt8(dy, cb[32:32 + M * N].view(M, N), sb[32:32 + scales.numel()].view(scales.shape), w, rstd, dx=dx)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((db[:64] == 9).all()) and bool((db[64 + M * N:] == 9).all())


def test_a_block_that_is_not_finite_makes_its_row_nan_and_no_other(rn):
    g = gen(5)
    x, dy, w = normal(g, 40, 256, dt=torch.bfloat16), normal(g, 40, 256, dt=torch.bfloat16), normal(g, 256, dt=torch.bfloat16)
    _, rstd = rn.rmsnorm_fwd(x, w)
    clean, _ = rn.rmsnorm_bwd_ckpt8(dy, *rn.ckpt8_pack(x), w, rstd)
    x[7, 40] = math.inf
    dx, dw = rn.rmsnorm_bwd_ckpt8(dy, *rn.ckpt8_pack(x), w, rstd)
    assert bool(torch.isnan(dx[7]).all()) and bool(torch.isnan(dw[32:64]).all())
    assert bool(torch.isfinite(dw[:32]).all()) and bool(torch.isfinite(dw[64:]).all())
    rest = torch.arange(40, device="cuda") != 7
    assert torch.equal(dx[rest], clean[rest])


# ---------------------------------------------------------------- group norm --

def act64(z, act):
    """act(z), act'(z)."""
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    if act == "gelu":
        c = torch.special.ndtr(z)
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return z, torch.ones_like(z)


def terms(B, S, C):
    """A bound of the terms in sequence in any sum over a group or over the batch."""
    return 128 + 600 + B + 100


def gn_stats(x, G, eps):
    B, C = x.shape[0], x.shape[-1]
    v = x.double().reshape(B, -1, G, C // G)
    mean = v.mean((1, 3))
    d = v - mean[:, None, :, None]
    var = d.square().mean((1, 3))
    D = d.abs().amax((1, 3))
    L = terms(B, v.shape[1], C)
    em = L * U * (d.abs().mean((1, 3)) + D) + 4 * U * mean.abs()
    rstd = 1 / (var + eps).sqrt()
    er = rstd * (L * U * (var + D.square()) / (var + eps) + 4 * U) + rstd ** 3 * em.square()
    return v, mean, rstd, em, er


def gn_forward(x, gamma, beta, G, act, eps):
    B, C = x.shape[0], x.shape[-1]
    v, mean, rstd, em, er = gn_stats(x, G, eps)
    ga = torch.ones(C, device="cuda").double() if gamma is None else gamma.double()
    be = torch.zeros(C, device="cuda").double() if beta is None else beta.double()
    ga, be = ga.view(G, C // G), be.view(G, C // G)

    def wide(t):
        return t[:, None, :, None]

    xhat = (v - wide(mean)) * wide(rstd)
    z = xhat * ga + be
    y, _ = act64(z, act)
    ez = ga.abs() * (wide(rstd) * wide(em) + (v - wide(mean)).abs() * wide(er) + 4 * U * xhat.abs()) + 4 * U * (z.abs() + be.abs())
    ey = 1.2 * ez + (10 + 3 * z.abs()) * U * (z.abs() + y.abs())
    return y.view(x.shape), ey.view(x.shape), mean, em, rstd, er


GN_SHAPES = [  # B, places, C, G
    (1, (64,), 1280, 32), (2, (8, 8), 320, 32), (3, (1001,), 90, 9), (2, (17, 3), 64, 64), (1, (1,), 64, 4), (1, (1,), 8, 8),
    (5, (7,), 33, 11), (2, (300,), 128, 1), (1, (4096,), 32, 32), (2, (50,), 5000, 5), (1, (9,), 5120, 1280), (1, (40,), 1025, 1),
    (2, (2000,), 960, 32), (300, (5,), 16, 4), (1, (20000,), 40, 2), (2, (3,), 8000, 10), (1, (70,), 8192, 1), (3, (30000,), 12, 4),
    (2, (9001,), 321, 3),
]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("act", [None, "silu", "gelu"])
@pytest.mark.parametrize("B,places,C,G", GN_SHAPES)
def test_groupnorm_forward(rn, dt, act, B, places, C, G):
    g, t = gen(B * C + G), TYPES[dt]
    x = (normal(g, B, *places, C) * torch.exp(0.3 * normal(g, C)) + 2 * normal(g, C)).to(t)
    wt = torch.float32 if C % 3 else t
    gamma, beta = ((1 + 0.2 * normal(g, C)).to(wt), (0.3 * normal(g, C)).to(wt)) if B != 5 else (None, None)
    y, ey, mean, em, rstd, er = gn_forward(x, gamma, beta, G, act, 1e-5)
    small = 2.0 ** -25 * (t == torch.float16)
    kept_out = rn.groupnorm_fwd_ckpt8(x, gamma, beta, G, act=act)
    check_kept(x, kept_out["codes"], kept_out["scales"])
    for out in (rn.groupnorm_fwd(x, gamma, beta, G, act=act), kept_out):
        near(out["mean"], mean, em, "mean")
        near(out["rstd"], rstd, er, "rstd")
        near(out["y"], y, half_step(t) * y.abs() + ey + small, "y")


@pytest.mark.parametrize("dt,C,G", [("f32", 64, 4), ("bf16", 320, 32), ("f32", 30, 3)])
def test_groupnorm_of_a_mean_far_from_zero(rn, dt, C, G):
    """Means 1000 widths away: the variance loses no digits but those that x's type has lost."""
    g, t = gen(11), TYPES[dt]
    x = (normal(g, 2, 3000, C) + 1000).to(t)
    x[:, 0] += 50  # the first value a thread sees is far from the others
    out = rn.groupnorm_fwd(x, None, None, G)
    y, ey, mean, em, rstd, er = gn_forward(x, None, None, G, None, 1e-5)
    near(out["mean"], mean, em, "mean")
    near(out["rstd"], rstd, er, "rstd")
    near(out["y"], y, half_step(t) * y.abs() + ey, "y")


def gn_backward(dy, x, gamma, beta, mean, rstd, G, act):
    B, C = dy.shape[0], dy.shape[-1]
    shape = (B, dy.numel() // (B * C), G, C // G)
    ga = torch.ones(C, device="cuda").double() if gamma is None else gamma.double()
    be = torch.zeros(C, device="cuda").double() if beta is None else beta.double()
    ga, be = ga.view(shape[2:]), be.view(shape[2:])
    m, r = mean.double()[:, None, :, None], rstd.double()[:, None, :, None]
    v, d = x.double().reshape(shape), dy.double().reshape(shape)
    xhat = (v - m) * r
    z = xhat * ga + be
    _, slope = act64(z, act)
    u = d * slope
    ez = 5 * U * ((xhat * ga).abs() + be.abs())
    eu = d.abs() * (1.2 * ez + (10 + 3 * z.abs()) * (1 + z.abs()) * U) + 2 * U * u.abs()
    L = terms(B, shape[1], C)
    dgamma, dbeta = (u * xhat).sum((0, 1)), u.sum((0, 1))
    eg = (eu * xhat.abs() + 4 * U * (u * xhat).abs()).sum((0, 1)) + L * U * (u * xhat).abs().sum((0, 1))
    eb = eu.sum((0, 1)) + L * U * u.abs().sum((0, 1))
    w, ew = u * ga, eu * ga.abs()
    m1, m2 = w.mean((1, 3), keepdim=True), (w * xhat).mean((1, 3), keepdim=True)
    e1 = ew.mean((1, 3), keepdim=True) + L * U * w.abs().mean((1, 3), keepdim=True)
    e2 = (ew * xhat.abs()).mean((1, 3), keepdim=True) + (L + 4) * U * (w * xhat).abs().mean((1, 3), keepdim=True)
    dx = r * (w - m1 - xhat * m2)
    ex = r * (ew + e1 + xhat.abs() * e2 + 8 * U * (w.abs() + m1.abs() + (xhat * m2).abs()))
    return dx.view(dy.shape), ex.view(dy.shape), dgamma.view(-1), eg.view(-1), dbeta.view(-1), eb.view(-1)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("act", [None, "silu", "gelu"])
@pytest.mark.parametrize("B,places,C,G", GN_SHAPES)
def test_groupnorm_gradient(rn, dt, act, B, places, C, G):
    g, t = gen(B * C + 2 * G), TYPES[dt]
    x = (normal(g, B, *places, C) * torch.exp(0.3 * normal(g, C)) + 2 * normal(g, C)).to(t)
    dy = normal(g, B, *places, C, dt=t)
    wt = torch.float32 if C % 3 else t
    gamma, beta = ((1 + 0.2 * normal(g, C)).to(wt), (0.3 * normal(g, C)).to(wt)) if B != 5 else (None, None)
    f = rn.groupnorm_fwd_ckpt8(x, gamma, beta, G, act=act)
    small = 2.0 ** -25 * (t == torch.float16)
    for from_kept in (False, True):
        if from_kept:
            out = rn.groupnorm_bwd_ckpt8(dy, f["codes"], f["scales"], gamma, beta, f["mean"], f["rstd"], G, act=act)
        else:
            out = rn.groupnorm_bwd(dy, x, gamma, beta, f["mean"], f["rstd"], G, act=act)
        v = kept(x)[2] if from_kept else x
        dx, ex, dg, eg, db, eb = gn_backward(dy, v, gamma, beta, f["mean"], f["rstd"], G, act)
        near(out["dx"], dx, half_step(t) * dx.abs() + ex + small, "dx")
        pt = wt if gamma is not None else t
        near(out["dbeta"], db, half_step(pt) * db.abs() + eb + 2.0 ** -25 * (pt == torch.float16), "dbeta")
        if gamma is None:
            assert out["dgamma"] is None
        else:
            near(out["dgamma"], dg, half_step(pt) * dg.abs() + eg + 2.0 ** -25 * (pt == torch.float16), "dgamma")


def test_groupnorm_gradient_is_that_of_differences(rn):
    """Central differences of sum(y w) along random directions, in fp64 arithmetic of the definition, against the
    kernel's gradients in fp32: off by the step's square and the kernel's rounding."""
    g, B, S, C, G = gen(21), 2, 40, 24, 4
    x, gamma, beta, w = normal(g, B, S, C), 1 + 0.2 * normal(g, C), 0.3 * normal(g, C), normal(g, B, S, C)

    def loss(xx, gg, bb, act):
        v = xx.view(B, S, G, -1)
        m = v.mean((1, 3), keepdim=True)
        r = 1 / ((v - m).square().mean((1, 3), keepdim=True) + 1e-5).sqrt()
        z = ((v - m) * r).view(B, S, C) * gg + bb
        return (act64(z, act)[0] * w.double()).sum().item()

    for act in (None, "silu", "gelu"):
        f = rn.groupnorm_fwd(x, gamma, beta, G, act=act)
        out = rn.groupnorm_bwd(w, x, gamma, beta, f["mean"], f["rstd"], G, act=act)
        for name, at in (("dx", 0), ("dgamma", 1), ("dbeta", 2)):
            args = [x.double(), gamma.double(), beta.double()]
            d = normal(g, *args[at].shape).double()
            step = 1e-4
            lo, hi = list(args), list(args)
            lo[at], hi[at] = args[at] - step * d, args[at] + step * d
            slope = (loss(*hi, act) - loss(*lo, act)) / (2 * step)
            got = (out[name].double() * d).sum().item()
            scale = (out[name].double() * d).abs().sum().item()
            assert abs(got - slope) <= 1e-5 * scale + 1e-5, (act, name)


def test_groupnorm_in_place_and_at_offsets(rn):
    g = gen(2)
    for dt, C, G in ((torch.bfloat16, 64, 8), (torch.float32, 64, 8), (torch.float16, 30, 3)):
        x, dy = normal(g, 3, 50, C, dt=dt), normal(g, 3, 50, C, dt=dt)
        gamma, beta = normal(g, C, dt=dt), normal(g, C, dt=dt)
        want = rn.groupnorm_fwd(x, gamma, beta, G, act="silu")
        back = rn.groupnorm_bwd(dy, x, gamma, beta, want["mean"], want["rstd"], G, act="silu")
        y = x.clone()
        assert rn.groupnorm_fwd(y, gamma, beta, G, act="silu", y=y)["y"] is y and torch.equal(y, want["y"])
        y = x.clone()
        got = rn.groupnorm_fwd_ckpt8(y, gamma, beta, G, act="silu", y=y)
        assert torch.equal(y, rn.groupnorm_fwd_ckpt8(x, gamma, beta, G, act="silu")["y"])
        check_kept(x, got["codes"], got["scales"])
        for into in ("dy", "x"):
            a, b = dy.clone(), x.clone()
            r = rn.groupnorm_bwd(a, b, gamma, beta, want["mean"], want["rstd"], G, act="silu", dx=a if into == "dy" else b)
            assert torch.equal(r["dx"], back["dx"]) and torch.equal(r["dgamma"], back["dgamma"])
        ref, ey, *_ = gn_forward(x, gamma, beta, G, "silu", 1e-5)
        off = rn.groupnorm_fwd(offset_view(x, 1), offset_view(gamma, 1), offset_view(beta, 1), G, act="silu")
        near(off["y"], ref, half_step(dt) * ref.abs() + ey + 2.0 ** -25 * (dt == torch.float16), "y")
        dx, ex, *_ = gn_backward(dy, x, gamma, beta, want["mean"], want["rstd"], G, "silu")
        off = rn.groupnorm_bwd(offset_view(dy, 1), offset_view(x, 1), gamma, beta, want["mean"], want["rstd"], G, act="silu")
        near(off["dx"], dx, half_step(dt) * dx.abs() + ex + 2.0 ** -25 * (dt == torch.float16), "dx")


def test_groupnorm_of_a_constant_group_and_of_nothing(rn):
    x = torch.full((2, 30, 16), 7.0, device="cuda")
    f = rn.groupnorm_fwd(x, None, None, 4)
    assert torch.equal(f["y"], torch.zeros_like(x)) and torch.equal(f["mean"], torch.full((2, 4), 7.0, device="cuda"))
    for shape in ((0, 5, 16), (3, 0, 16)):
        e = torch.empty(shape, device="cuda")
        w = torch.ones(16, device="cuda")
        f = rn.groupnorm_fwd_ckpt8(e, w, w, 4)
        assert f["y"].shape == shape and not f["mean"].any()
        b = rn.groupnorm_bwd(e, e, w, w, f["mean"], f["rstd"], 4)
        assert not b["dgamma"].any() and not b["dbeta"].any()


def test_groupnorm_nan_stays_in_its_group(rn):
    x = normal(gen(4), 2, 100, 64)
    want = rn.groupnorm_fwd(x, None, None, 8)["y"]
    x[1, 50, 20] = math.nan
    y = rn.groupnorm_fwd(x, None, None, 8)["y"]
    assert bool(torch.isnan(y[1, :, 16:24]).all())
    y[1, :, 16:24] = want[1, :, 16:24]
    assert torch.equal(y, want)


@pytest.mark.parametrize("S,C,G", [(100, 64, 8), (40000, 32, 4), (30, 33, 3)])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_groupnorm_of_what_is_not_finite(rn, S, C, G, bad):
    """One value that is no number leaves no number in its group (the mean is not finite, the variance none), and
    every other group its bits."""
    g = gen(6)
    x, dy = normal(g, 2, S, C), normal(g, 2, S, C)
    clean = rn.groupnorm_fwd(x, None, None, G, act="silu")
    at = (1, S // 2, C // 2)
    x[at] = bad
    f = rn.groupnorm_fwd(x, None, None, G, act="silu")
    lo = (C // 2) // (C // G) * (C // G)
    hit = slice(lo, lo + C // G)
    assert bool(torch.isnan(f["rstd"][1, lo // (C // G)])) and bool(torch.isnan(f["y"][1, :, hit]).all())
    b = rn.groupnorm_bwd(dy, x, None, None, f["mean"], f["rstd"], G, act="silu", want_dbeta=False)
    assert bool(torch.isnan(b["dx"][1, :, hit]).all())
    f["y"][1, :, hit] = clean["y"][1, :, hit]
    assert torch.equal(f["y"], clean["y"])
    b["dx"][1, :, hit] = 0
    assert bool(torch.isfinite(b["dx"]).all())


# ----------------------------------------------------------------- embedding --

EMBED_SHAPES = [(1, 10, 64), (8, 1000, 8192), (33, 50, 100), (1000, 300, 33), (257, 7, 4096), (5000, 2, 24), (300, 100000, 128),
                (3, 5, 1), (40, 17, 20000)]


def some_ids(g, T, V, dt=torch.int64, pad=True):
    ids = (torch.rand(T, generator=g, device="cuda").square() * V).to(dt).clamp_(max=V - 1)
    if pad and T > 4:
        ids[1], ids[T // 2], ids[T - 1] = -1, V, -2 ** 31
    return ids


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,V,N", EMBED_SHAPES)
def test_embedding_rows(rn, dt, T, V, N):
    g, t = gen(T + V), TYPES[dt]
    table = normal(g, V, N, dt=t)
    ids = some_ids(g, T, V, torch.int32 if T % 2 else torch.int64)
    there = (ids >= 0) & (ids < V)
    scale = 1.7
    ref = table[ids.clamp(0, V - 1).long()].double() * float(torch.tensor(scale)) * there[:, None]
    h = rn.embed_fwd(ids, table, scale=scale)
    small = 2.0 ** -25 * (t == torch.float16)
    near(h, ref, (half_step(t) + U) * ref.abs() + small, "h")
    assert not h[~there].any()
    assert torch.equal(rn.embed_fwd(ids, table)[there], table[ids[there].long()])
    wt = torch.float32 if N % 3 else t
    w = (1 + 0.1 * normal(g, N)).to(wt)
    y, h2, rstd = rn.rmsnorm_embed_fwd(ids, table, w, scale=scale, offset=0.25)
    assert torch.equal(bits(h2), bits(h))
    check_norm(y, rstd, h, w, 0.25)
    y, h2, rstd = rn.rmsnorm_embed_fwd(ids, table, None, scale=scale)
    check_norm(y, rstd, h, None, 0.0)


GRAD_SHAPES = EMBED_SHAPES + [(1, 1, 8), (2048, 3, 512), (9000, 40000, 64), (20000, 1, 16), (70000, 300, 8), (70000, 300000, 16),
                              (140000, 5, 32), (65536, 600, 24), (65537, 70000, 9), (32, 33, 264), (64, 1, 2056), (8193, 1 << 20, 8)]


@pytest.mark.parametrize("dt,out", [("bf16", None), ("bf16", "f32"), ("f16", None), ("f32", None)])
@pytest.mark.parametrize("T,V,N", GRAD_SHAPES)
def test_embedding_gradient(rn, dt, out, T, V, N):
    g, t = gen(T + V + N), TYPES[dt]
    ot = TYPES[out] if out else t
    dh = normal(g, T, N, dt=t)
    ids = some_ids(g, T, V, torch.int32 if T % 2 else torch.int64)
    scale = 1.3
    keep = (ids >= 0) & (ids < V)
    to = ids[keep].long()
    ref = torch.zeros(V, N, dtype=torch.float64, device="cuda").index_add_(0, to, dh[keep].double()) * float(torch.tensor(scale))
    mag = torch.zeros(V, N, dtype=torch.float64, device="cuda").index_add_(0, to, dh[keep].double().abs()) * scale
    most = int(torch.bincount(to, minlength=1).max()) if to.numel() else 0
    L = 32 + most / 32 / 8 + 20
    small = 2.0 ** -25 * (ot == torch.float16)
    got = rn.embed_bwd(dh, ids, V, scale=scale, dtype=None if out is None else ot)
    assert got.dtype == ot and got.shape == (V, N)
    near(got, ref, half_step(ot) * ref.abs() + L * U * mag + small, "dtable")
    touched = torch.zeros(V, dtype=torch.bool, device="cuda")
    touched[to] = True
    assert not got[~touched].any()
    assert torch.equal(bits(rn.embed_bwd(dh, ids, V, scale=scale, dtype=None if out is None else ot)), bits(got))
    # added to what is there; rows without a token keep their bits
    base = normal(g, V, N, dt=ot)
    acc = base.clone()
    assert rn.embed_bwd(dh, ids, V, scale=scale, dtable=acc, accumulate=True) is acc
    ref = ref + base.double()
    near(acc, ref, half_step(ot) * ref.abs() + L * U * (mag + base.double().abs()) + small, "accumulated")
    assert torch.equal(acc[~touched], base[~touched])


def test_embedding_gradient_of_nothing(rn):
    dh, ids = torch.empty(0, 16, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    assert not rn.embed_bwd(dh, ids, 5).any()
    table = torch.ones(5, 16, device="cuda")
    assert rn.embed_fwd(ids, table).shape == (0, 16)
    acc = table.clone()
    rn.embed_bwd(dh, ids, 5, dtable=acc, accumulate=True)
    assert torch.equal(acc, table)
    none = torch.full((7,), -1, device="cuda")
    assert not rn.embed_bwd(torch.ones(7, 16, device="cuda"), none, 5).any()


# ------------------------------------------------------------ the step's run --

def test_a_training_step_of_rows(rn):
    """Embedding rows into a norm, a second norm after a residual add whose rows are kept in 8 bits, and the way
    back to the table, each call fed by the one before. Against the same step in 64 bits from the same kept rows."""
    T, V, N, scale = 300, 97, 512, 22.5
    g = gen(31)
    ids = some_ids(g, T, V)
    table = (0.05 * normal(g, V, N)).float()
    w1, w2, mix, dy = 1 + 0.1 * normal(g, N), 1 + 0.1 * normal(g, N), normal(g, N), normal(g, T, N)
    y1, h1, r1 = rn.rmsnorm_embed_fwd(ids, table, w1, scale=scale)
    branch = y1 * mix
    f = rn.rmsnorm_fwd_ckpt8(branch, w2, residual=h1)
    dh2, dw2 = rn.rmsnorm_bwd_ckpt8(dy, f["codes"], f["scales"], w2, f["rstd"])
    dh1, dw1 = rn.rmsnorm_add_bwd(dh2 * mix, dh2, h1, w1, r1)
    dtable = rn.embed_bwd(dh1, ids, V, scale=scale)
    # the same in 64 bits
    tab = table.double().requires_grad_()
    v1, v2 = w1.double().requires_grad_(), w2.double().requires_grad_()
    there = ((ids >= 0) & (ids < V)).double()[:, None]
    e1 = tab[ids.clamp(0, V - 1)] * scale * there
    n1 = e1 / (e1.square().mean(-1, keepdim=True) + 1e-6).sqrt() * v1
    e2 = n1 * mix.double() + e1
    rs = 1 / (e2.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    held = kept(f["residual_out"])[2]
    xhat = held * rs.detach()
    gy = dy.double() * w2.double()
    d2 = rs.detach() * (gy - xhat * (gy * xhat).mean(-1, keepdim=True))
    e2.backward(d2)
    near(f["y"], (e2 * rs * v2).detach(), 1e-5 * (e2 * rs * v2).detach().abs() + 1e-6, "y")
    for got, want in ((dtable, tab.grad), (dw1, v1.grad), (dw2, (dy.double() * xhat).sum(0))):
        assert (got.double() - want).norm() <= 1e-5 * want.norm()


def test_an_image_step_with_kept_rows(rn):
    """Two group norms in a row, the second's rows kept in 8 bits, and back."""
    B, S, C, G = 2, 16 * 16, 64, 8
    g = gen(41)
    x, dy = normal(g, B, 16, 16, C), normal(g, B, 16, 16, C)
    ga, be = 1 + 0.1 * normal(g, C), 0.1 * normal(g, C)
    f1 = rn.groupnorm_fwd(x, ga, be, G, act="silu")
    f2 = rn.groupnorm_fwd_ckpt8(f1["y"], ga, be, G, act="gelu")
    b2 = rn.groupnorm_bwd_ckpt8(dy, f2["codes"], f2["scales"], ga, be, f2["mean"], f2["rstd"], G, act="gelu")
    b1 = rn.groupnorm_bwd(b2["dx"], x, ga, be, f1["mean"], f1["rstd"], G, act="silu")
    d2, _, dg2, _, db2, _ = gn_backward(dy, kept(f1["y"])[2], ga, be, f2["mean"], f2["rstd"], G, "gelu")
    d1, _, dg1, _, db1, _ = gn_backward(d2, x, ga, be, f1["mean"], f1["rstd"], G, "silu")
    for got, want in ((b2["dx"], d2), (b2["dgamma"], dg2), (b2["dbeta"], db2), (b1["dx"], d1), (b1["dgamma"], dg1), (b1["dbeta"], db1)):
        assert (got.double() - want).norm() <= 1e-5 * want.norm()


# ------------------------------------------------- streams, graphs, devices --

def all_calls(rn):
    """name -> a call without arguments that makes its results anew."""
    g, bf = gen(51), torch.bfloat16
    x, dy, w = normal(g, 96, 256, dt=bf), normal(g, 96, 256, dt=bf), normal(g, 256, dt=bf)
    codes, scales = rn.ckpt8_pack(x)
    _, rstd = rn.rmsnorm_fwd(x, w)
    img, dimg = x.view(2, 48, 256), dy.view(2, 48, 256)
    f = rn.groupnorm_fwd(img, w, w, 16, act="silu")
    ids = some_ids(g, 96, 40)
    return {
        "pack": lambda **k: rn.ckpt8_pack(x, **k),
        "unpack": lambda **k: (rn.ckpt8_unpack(codes, scales, bf, **k),),
        "norm_fwd": lambda **k: tuple(v for v in rn.rmsnorm_fwd_ckpt8(x, w, residual=dy, **k).values()),
        "norm_bwd": lambda **k: rn.rmsnorm_bwd_ckpt8(dy, codes, scales, w, rstd, **k),
        "gn_fwd": lambda **k: tuple(rn.groupnorm_fwd_ckpt8(img, w, w, 16, act="silu", **k).values()),
        "gn_bwd": lambda **k: tuple(rn.groupnorm_bwd(dimg, img, w, w, f["mean"], f["rstd"], 16, act="silu", **k).values()),
        "embed": lambda **k: (rn.embed_fwd(ids, x, **k),),
        "embed_norm": lambda **k: rn.rmsnorm_embed_fwd(ids, x, w, **k),
        "embed_bwd": lambda **k: (rn.embed_bwd(dy, ids, 40, **k),),
    }


CALLS = ["pack", "unpack", "norm_fwd", "norm_bwd", "gn_fwd", "gn_bwd", "embed", "embed_norm", "embed_bwd"]


@pytest.mark.parametrize("op", CALLS)
def test_named_streams_graphs_and_two_at_once(rn, op):
    call = all_calls(rn)[op]
    want = [t.clone() for t in call()]

    def same(got):
        return all(torch.equal(bits(a), bits(b)) for a, b in zip(got, want))

    torch.cuda.synchronize()
    for stream in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream, 0):
        got = call(stream=stream)
        torch.cuda.synchronize()
        assert same(got)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    results = []
    for _ in range(20):
        for s in (a, b):
            with torch.cuda.stream(s):
                results.append(call())
    torch.cuda.synchronize()
    assert all(same(r) for r in results)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got)


def test_given_results_and_workspaces(rn):
    g = gen(61)
    x, dy, w = normal(g, 64, 128), normal(g, 64, 128), normal(g, 128)
    f = rn.rmsnorm_fwd_ckpt8(x, w)
    mine = {k: torch.empty_like(v) for k, v in f.items() if v is not None}
    again = rn.rmsnorm_fwd_ckpt8(x, w, **mine)
    assert all(again[k] is mine[k] and torch.equal(mine[k], f[k]) for k in mine)
    want = rn.rmsnorm_bwd_ckpt8(dy, f["codes"], f["scales"], w, f["rstd"])
    ws = torch.full((rn.rmsnorm_bwd_ckpt8_workspace_bytes(64, 128, torch.float32),), 255, dtype=torch.uint8, device="cuda")
    got = rn.rmsnorm_bwd_ckpt8(dy, f["codes"], f["scales"], w, f["rstd"], workspace=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(rn.RMSNormError):
        rn.rmsnorm_bwd_ckpt8(dy, f["codes"], f["scales"], w, f["rstd"], workspace=ws[:256])
    img = x.view(2, 32, 128)
    fw = rn.groupnorm_fwd(img, w, w, 8)
    bw = rn.groupnorm_bwd(img, img, w, w, fw["mean"], fw["rstd"], 8)
    for back in (False, True):
        ws = torch.full((rn.groupnorm_workspace_bytes(2, 32, 128, 8, torch.float32, backward=back),), 255, dtype=torch.uint8, device="cuda")
        if back:
            r = rn.groupnorm_bwd(img, img, w, w, fw["mean"], fw["rstd"], 8, workspace=ws)
            assert all(torch.equal(r[k], bw[k]) for k in bw)
        else:
            r = rn.groupnorm_fwd(img, w, w, 8, workspace=ws)
            assert all(torch.equal(r[k], fw[k]) for k in fw)
    ids = some_ids(g, 64, 30)
    want = rn.embed_bwd(dy, ids, 30)
    ws = torch.full((rn.embed_bwd_workspace_bytes(64, 128, 30),), 255, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        assert torch.equal(rn.embed_bwd(dy, ids, 30, workspace=ws), want)
