"""Group norms of samples that no cluster holds (pieces by ticket), against the
definitions and tolerances of test_gpu_rows: their workspaces, streams, graphs,
in-place results and rings of stages."""
import ctypes

import pytest
import torch

from test_gpu_rows import TYPES, bits, check_kept, gen, gn_backward, gn_forward, half_step, near, normal, offset_view, rn  # noqa: F401
from test_rows_plan_cpu import Plan

pytestmark = pytest.mark.gpu


def sample(seed, B, S, C, t):
    g = gen(seed)
    x = (normal(g, B, S, C) * torch.exp(0.3 * normal(g, C)) + 2 * normal(g, C)).to(t)
    return x, (1 + 0.2 * normal(g, C)).to(t), (0.3 * normal(g, C)).to(t)


def check_forward(out, x, gamma, beta, G, act):
    t = x.dtype
    y, ey, mean, em, rstd, er = gn_forward(x, gamma, beta, G, act, 1e-5)
    near(out["mean"], mean, em, "mean")
    near(out["rstd"], rstd, er, "rstd")
    near(out["y"], y, half_step(t) * y.abs() + ey + 2.0 ** -25 * (t == torch.float16), "y")


def check_backward(out, dy, x, gamma, beta, f, G, act):
    t = dy.dtype
    dx, ex, dg, eg, db, eb = gn_backward(dy, x, gamma, beta, f["mean"], f["rstd"], G, act)
    small = 2.0 ** -25 * (t == torch.float16)
    near(out["dx"], dx, half_step(t) * dx.abs() + ex + small, "dx")
    near(out["dgamma"], dg, half_step(gamma.dtype) * dg.abs() + eg + small, "dgamma")
    near(out["dbeta"], db, half_step(beta.dtype) * db.abs() + eb + small, "dbeta")


def cut(rn, B, S, C, G, t, backward=False, kept=False, row=16, code=16):
    p, dt = Plan(), {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}[t]
    assert rn.lib().groupnorm_plan_query(B, S, C, G, dt, backward, kept, row, code, 0, ctypes.byref(p)) == 0
    return p


def full_workspace(rn, shape, G, t, backward=False):
    B, S, C = shape
    n = rn.groupnorm_workspace_bytes(B, S, C, G, t, backward=backward)
    return torch.full((n,), 255, dtype=torch.uint8, device="cuda")


# A cluster holds the groups of the plain call (spans of 40 or 80 channels), none those of the call that keeps x
# (spans are whole blocks of 32), which goes by pieces.
@pytest.mark.parametrize("dt,B,S,C,G", [("bf16", 1, 16384, 320, 32), ("bf16", 4, 9216, 320, 32), ("f16", 8, 5184, 320, 32),
                                        ("bf16", 1, 9216, 640, 32), ("f32", 4, 4096, 320, 32), ("bf16", 1, 1024, 736, 32),
                                        ("bf16", 16, 9216, 192, 32)])
def test_the_keeping_forward_has_the_workspace_that_it_takes(rn, dt, B, S, C, G):
    t = TYPES[dt]
    x, gamma, beta = sample(S + C, B, S, C, t)
    out = rn.groupnorm_fwd_ckpt8(x, gamma, beta, G, act="silu")
    check_kept(x, out["codes"], out["scales"])
    check_forward(out, x, gamma, beta, G, "silu")
    ws = full_workspace(rn, (B, S, C), G, t)
    assert ws.numel() > 0
    again = rn.groupnorm_fwd_ckpt8(x, gamma, beta, G, act="silu", workspace=ws)
    assert all(torch.equal(bits(again[k]), bits(out[k])) for k in out)
    with pytest.raises(rn.RMSNormError):
        rn.groupnorm_fwd_ckpt8(x, gamma, beta, G, act="silu", workspace=ws[:256])


# ------------------------------------------------------ a wait that gives up --

@pytest.mark.parametrize("dt,B,S,C,G,stages", [("bf16", 2, 140000, 128, 8, 2), ("f32", 3, 3000, 1030, 10, 1), ("f16", 2, 5001, 321, 3, 1)])
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("lost", [0, 1])
def test_a_launch_whose_wait_gives_up_ends_and_says_so(rn, dt, B, S, C, G, stages, backward, lost):
    """One sample is never joined and the wait for it is a short one: the launch ends, the status word is set, no row
    is written that was not normalised, and the next call is as ever."""
    t, status = TYPES[dt], rn.lib().rmsnorm_device_status
    x, dy = sample(1, B, S, C, t)[0], normal(gen(2), B, S, C, dt=t)
    p = cut(rn, B, S, C, G, t, backward)
    assert p.cluster == 0 and p.stages >= 2 and (stages == 1 or p.rows * C * x.element_size() > 2 * 28 * 1024)
    f = rn.groupnorm_fwd(x, None, None, G)
    want = rn.groupnorm_bwd(dy, x, None, None, f["mean"], f["rstd"], G, want_dbeta=False)["dx"] if backward else f["y"]
    assert status(0) == 0
    out, mean, rstd = torch.full_like(x, 7.0), f["mean"].clone(), f["rstd"].clone()
    code = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}[t]
    got = rn.lib().groupnorm_give_up_check(dy.data_ptr() if backward else None, x.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                                           out.data_ptr(), B, S, C, G, code, lost, 2000, torch.cuda.current_stream().cuda_stream)
    assert got == 0
    torch.cuda.synchronize()
    assert status(1) == 1 and status(0) == 0
    assert bool((out[lost] == 7).all())
    untouched = (out == 7).all(-1)
    assert torch.equal(out[~untouched], want[~untouched])
    again = rn.groupnorm_fwd(x, None, None, G)
    assert torch.equal(bits(again["y"]), bits(f["y"])) and status(0) == 0


# -------------------------------------------------------------- rings of stages --

@pytest.mark.parametrize("act", [None, "silu"])
def test_a_gradient_whose_ring_has_one_stage(rn, act):
    """8192 fp32 channels in 4096 groups at an odd address: copies and sums take turns."""
    t, (B, S, C, G) = torch.float32, (2, 300, 8192, 4096)
    x, gamma, beta = sample(3, B, S, C, t)
    x, dy = offset_view(x, 1), offset_view(normal(gen(4), B, S, C), 1)
    assert cut(rn, B, S, C, G, t, backward=True, row=4).stages == 1
    f = rn.groupnorm_fwd(x, gamma, beta, G, act=act)
    check_forward(f, x, gamma, beta, G, act)
    check_backward(rn.groupnorm_bwd(dy, x, gamma, beta, f["mean"], f["rstd"], G, act=act), dy, x, gamma, beta, f, G, act)
