"""Group norms of samples that no cluster holds (pieces by ticket), against the
definitions and tolerances of test_gpu_rows: their workspaces, streams, graphs,
in-place results and rings of stages."""
import pytest
import torch

from test_gpu_rows import TYPES, bits, check_kept, gen, gn_backward, gn_forward, half_step, kept, near, normal, offset_view, rn  # noqa: F401

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
