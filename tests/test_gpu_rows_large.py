"""Training rows whose offsets pass 32 bits, compared at the places where an
index would come round: the first rows, those about element 2^31 and 2^32, and
the last ones. Definitions and tolerances are those of test_gpu_rows."""
import pytest
import torch

from test_gpu_rows import U, bits, bwd_reference, check_kept, check_norm, gen, half_step, kept, near, normal, rn  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.slow]

BF = torch.bfloat16


def rows_to_look_at(M, N):
    """A few rows at each border."""
    at = {0, 1, M - 2, M - 1}
    for k in (31, 32):
        r = (1 << k) // N
        at |= {r - 1, r, r + 1}
    return torch.tensor(sorted(r for r in at if 0 <= r < M), device="cuda")


def big(M, N, seed):
    """Rows that all differ, made a block at a time."""
    g, x = gen(seed), torch.empty(M, N, dtype=BF, device="cuda")
    for r in range(0, M, 16384):
        x[r:r + 16384] = normal(g, min(16384, M - r), N)
    return x


@pytest.mark.parametrize("M,N", [(140000, 32768), (70000, 65535)])
def test_rows_kept_and_restored(rn, M, N):
    x = big(M, N, 1)
    codes, scales = rn.ckpt8_pack(x)
    y = rn.ckpt8_unpack(codes, scales, BF)
    at = rows_to_look_at(M, N)
    check_kept(x[at], codes[at], scales[at], y[at])


@pytest.mark.parametrize("M,N", [(300000, 8192), (300000, 7999)])
@pytest.mark.parametrize("fused", [False, True])
def test_norms_keeping_their_rows(rn, M, N, fused):
    x, res = big(M, N, 2), big(M, N, 3) if fused else None
    w = (1 + 0.1 * normal(gen(4), N)).to(BF)
    f = rn.rmsnorm_fwd_ckpt8(x, w, residual=res)
    at = rows_to_look_at(M, N)
    h = (x[at].double() + res[at].double()).to(BF) if fused else x[at]
    if fused:
        assert torch.equal(f["residual_out"][at], h)
    check_norm(f["y"][at], f["rstd"][at], h, w, 0.0)
    check_kept(h, f["codes"][at], f["scales"][at])
    dy, dres = f["y"], res
    dx, dw = rn.rmsnorm_bwd_ckpt8(dy, f["codes"], f["scales"], w, f["rstd"], dresidual_out=dres)
    ref, err, _, _ = bwd_reference(dy[at], kept(h)[2], w, f["rstd"][at], 0.0, dres[at] if fused else None)
    near(dx[at], ref, half_step(BF) * ref.abs() + err, "dx")
    # every row counts in dw
    total = torch.zeros(N, dtype=torch.float64, device="cuda")
    mag = total.clone()
    for r in range(0, M, 8192):
        s = slice(r, r + 8192)
        values = rn.ckpt8_unpack(f["codes"][s], f["scales"][s], torch.float32).double()
        p = dy[s].double() * values * f["rstd"][s].double()[:, None]
        total += p.sum(0)
        mag += p.abs().sum(0)
    near(dw, total, half_step(BF) * total.abs() + (M / 32 + 600) * U * mag, "dw")  # (rows of a CTA or of a slice in sequence)


@pytest.mark.parametrize("B,S,C,G", [(1, 2200000, 1024, 32), (2, 1100001, 1021, 1021), (290000, 1, 8192, 64), (70000, 33, 960, 30)])
def test_group_norms(rn, B, S, C, G):
    """Statistics and rows of the first, the middle and the last samples (or of the one), and the gradient's sums."""
    x = big(B * S, C, 5).view(B, S, C)
    gamma, beta = (1 + 0.1 * normal(gen(6), C)).to(BF), (0.1 * normal(gen(7), C)).to(BF)
    f = rn.groupnorm_fwd_ckpt8(x, gamma, beta, G)
    samples = sorted({0, B // 2, ((1 << 31) // (S * C)) % B, B - 1})
    n = S * C // G
    for b in samples:
        s1, s2 = (torch.zeros(G, dtype=torch.float64, device="cuda") for _ in range(2))
        for r in range(0, S, 65536):
            v = x[b, r:r + 65536].double().view(-1, G, C // G)
            s1 += v.sum((0, 2))
            s2 += v.square().sum((0, 2))
        mean = s1 / n
        var = s2 / n - mean.square()
        # (values about 0 and of width 1: deviations below 8 of a chain of at most 12000 terms)
        near(f["mean"][b].double(), mean, torch.full_like(mean, 12000 * U * 9), "mean")
        near(f["rstd"][b].double(), (var + 1e-5).rsqrt(), 12000 * U * 10 * (var + 1e-5).rsqrt(), "rstd")
    at = rows_to_look_at(B * S, C)
    rows = x.view(-1, C)[at]
    m, r = (f[k][at // S].double()[:, :, None] for k in ("mean", "rstd"))

    def xhat(v):
        return ((v.double().view(len(at), G, -1) - m) * r).view(len(at), C)

    z = xhat(rows) * gamma.double() + beta.double()
    near(f["y"].view(-1, C)[at], z, half_step(BF) * z.abs() + 8 * U * (1 + z.abs()), "y")
    check_kept(rows, f["codes"].view(-1, C)[at], f["scales"].view(len(x.view(-1, C)), -1)[at])
    dy = f["y"]
    for held in (False, True):
        if held:
            o = rn.groupnorm_bwd_ckpt8(dy, f["codes"], f["scales"], gamma, beta, f["mean"], f["rstd"], G)
        else:
            o = rn.groupnorm_bwd(dy, x, gamma, beta, f["mean"], f["rstd"], G)
        db, dg, ab, ag = (torch.zeros(C, dtype=torch.float64, device="cuda") for _ in range(4))
        m1, m2 = (torch.zeros(B, G, dtype=torch.float64, device="cuda") for _ in range(2))
        step = max(1, 60000 // S)  # samples, or rows of one
        for b in range(0, B, step):
            for q in range(0, S, 65536):
                d = dy[b:b + step, q:q + 65536].double()
                v = x[b:b + step, q:q + 65536]
                if held:
                    c = f["codes"][b:b + step, q:q + 65536].contiguous()
                    v = rn.ckpt8_unpack(c, f["scales"][b:b + step, q:q + 65536].contiguous(), torch.float32)
                h = ((v.double().view(*v.shape[:2], G, -1) - f["mean"][b:b + step].double()[:, None, :, None])
                     * f["rstd"][b:b + step].double()[:, None, :, None]).view(v.shape)
                db += d.sum((0, 1))
                ab += d.abs().sum((0, 1))
                dg += (d * h).sum((0, 1))
                ag += (d * h).abs().sum((0, 1))
                u = (d * gamma.double()).view(*v.shape[:2], G, -1)
                m1[b:b + step] += u.sum((1, 3)) / n
                m2[b:b + step] += (u * h.view(u.shape)).sum((1, 3)) / n
        L = B / 32 + 12000  # (the finalizer takes a 32nd of the samples' rows in sequence)
        near(o["dbeta"], db, half_step(BF) * db.abs() + L * U * ab, "dbeta")
        near(o["dgamma"], dg, half_step(BF) * dg.abs() + L * U * ag, "dgamma")
        v = rows
        if held:
            v = rn.ckpt8_unpack(f["codes"].view(-1, C)[at], f["scales"].view(B * S, -1)[at], torch.float32)
        h, u = xhat(v).view(len(at), G, -1), (dy.view(-1, C)[at].double() * gamma.double()).view(len(at), G, -1)
        a, b = m1[at // S][:, :, None], m2[at // S][:, :, None]
        dx = (r * (u - a - h * b)).view(len(at), C)
        e = (r * U * (8 * (u.abs() + a.abs() + (h * b).abs()) + 12000 * (1.5 + 3 * h.abs()))).view(len(at), C)
        near(o["dx"].view(-1, C)[at], dx, half_step(BF) * dx.abs() + e, "dx")


@pytest.mark.parametrize("T,V,N", [(300000, 290000, 8192), (290000, 300000, 7999)])
def test_embedding_rows(rn, T, V, N):
    g = gen(8)
    table, w = big(V, N, 9), (1 + 0.1 * normal(gen(10), N)).to(BF)
    ids = torch.randint(-1, V, (T,), generator=g, device="cuda")
    at = rows_to_look_at(T, N)
    ids[at] = V - 1 - torch.arange(len(at), device="cuda")  # the table's last rows
    y, h, rstd = rn.rmsnorm_embed_fwd(ids, table, w, scale=2.0)
    assert torch.equal(h[at], (table[ids[at]].float() * 2).to(BF))
    check_norm(y[at], rstd[at], h[at], w, 0.0)
    alone = rn.embed_fwd(ids, table, scale=2.0)
    assert torch.equal(bits(alone[at]), bits(h[at]))
    del y, alone, table
    got = rn.embed_bwd(h, ids, V, scale=0.5)
    look = torch.unique(torch.cat([rows_to_look_at(V, N), ids[at].clamp(min=0)]))
    for v in look.tolist():
        of = (ids == v).nonzero()[:, 0]
        ref, mag = h[of].double().sum(0) * 0.5, h[of].double().abs().sum(0) * 0.5
        near(got[v].double(), ref, half_step(BF) * ref.abs() + (len(of) + 8) * U * mag, f"row {v}")
