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
    assert rn.lib().groupnorm_plan_query(B, S, C, G, dt, backward, kept, row, code, 0, 0, ctypes.byref(p)) == 0
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


# ------------------------------------- workspaces, streams, graphs, in place --

FLOWS = [("bf16", 2, 40000, 32, 4), ("f32", 2, 40000, 33, 3), ("f16", 1, 20001, 90, 9)]


def flow_calls(rn, dt, B, S, C, G):
    """name -> (whether backward, a call that makes its results anew or into what it is given)."""
    t = TYPES[dt]
    x, gamma, beta = sample(5, B, S, C, t)
    dy = normal(gen(6), B, S, C, dt=t)
    f = rn.groupnorm_fwd_ckpt8(x, gamma, beta, G, act="silu")
    for backward, held in ((False, False), (False, True), (True, False), (True, True)):
        assert cut(rn, B, S, C, G, t, backward, held).cluster == 0
    a = (gamma, beta, G)
    m = (f["mean"], f["rstd"])
    return {
        "forward": (False, lambda **k: rn.groupnorm_fwd(x, *a, act="silu", **k)),
        "keeping": (False, lambda **k: rn.groupnorm_fwd_ckpt8(x, *a, act="silu", **k)),
        "gradient": (True, lambda **k: rn.groupnorm_bwd(dy, x, gamma, beta, *m, G, act="silu", **k)),
        "gradient from kept": (True, lambda **k: rn.groupnorm_bwd_ckpt8(dy, f["codes"], f["scales"], gamma, beta, *m, G, act="silu", **k)),
    }


def same(got, want):
    return got.keys() == want.keys() and all(torch.equal(bits(got[k]), bits(want[k])) for k in want)


@pytest.mark.parametrize("op", ["forward", "keeping", "gradient", "gradient from kept"])
@pytest.mark.parametrize("dt,B,S,C,G", FLOWS)
def test_flows_on_streams_in_graphs_and_in_given_workspaces(rn, dt, B, S, C, G, op):
    backward, call = flow_calls(rn, dt, B, S, C, G)[op]
    want = {k: v.clone() for k, v in call().items()}
    # the workspace that the query names, whatever is in it; none that is smaller than the cut's
    ws = full_workspace(rn, (B, S, C), G, TYPES[dt], backward)
    need = cut(rn, B, S, C, G, TYPES[dt], backward, "kept" in op or op == "keeping").workspace_bytes
    assert ws.numel() >= need > 256
    for _ in range(2):
        assert same(call(workspace=ws), want)
    assert same(call(workspace=ws[:need]), want)
    with pytest.raises(rn.RMSNormError):
        call(workspace=ws[:need - 16])
    torch.cuda.synchronize()
    for stream in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream, 0):
        got = call(stream=stream)
        torch.cuda.synchronize()
        assert same(got, want)
    # two streams at once, each call in a workspace of its own
    streams, results = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                results.append(call())
    torch.cuda.synchronize()
    assert all(same(r, want) for r in results)
    # captured and replayed: the tickets begin anew
    for given in (None, ws):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = call(workspace=given)
        for _ in range(3):
            for t in got.values():
                t.zero_()
            if given is not None:
                given.fill_(255)
            graph.replay()
            torch.cuda.synchronize()
            assert same(got, want)


@pytest.mark.parametrize("dt,B,S,C,G", FLOWS)
def test_two_graphs_share_a_workspace_of_a_flow(rn, dt, B, S, C, G):
    """One after the other on one stream, in either order, forward and gradient in the same memory."""
    calls = flow_calls(rn, dt, B, S, C, G)
    want = {op: {k: v.clone() for k, v in calls[op][1]().items()} for op in ("keeping", "gradient")}
    ws = torch.full((max(rn.groupnorm_workspace_bytes(B, S, C, G, TYPES[dt], backward=b) for b in (False, True)),), 255, dtype=torch.uint8,
                    device="cuda")
    graphs = {}
    for op in want:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = calls[op][1](workspace=ws)
        graphs[op] = (g, got)
    for op in ("keeping", "gradient", "gradient", "keeping", "keeping", "gradient"):
        for t in graphs[op][1].values():
            t.zero_()
        graphs[op][0].replay()
        torch.cuda.synchronize()
        assert same(graphs[op][1], want[op])


@pytest.mark.parametrize("dt,B,S,C,G", FLOWS)
def test_flows_in_place(rn, dt, B, S, C, G):
    t = TYPES[dt]
    x, gamma, beta = sample(7, B, S, C, t)
    dy = normal(gen(8), B, S, C, dt=t)
    want = rn.groupnorm_fwd(x, gamma, beta, G, act="gelu")
    check_forward(want, x, gamma, beta, G, "gelu")
    y = x.clone()
    assert rn.groupnorm_fwd(y, gamma, beta, G, act="gelu", y=y)["y"] is y and torch.equal(bits(y), bits(want["y"]))
    keeping = rn.groupnorm_fwd_ckpt8(x, gamma, beta, G, act="gelu")
    y = x.clone()
    got = rn.groupnorm_fwd_ckpt8(y, gamma, beta, G, act="gelu", y=y)
    assert same(got, keeping)
    check_kept(x, got["codes"], got["scales"])
    back = rn.groupnorm_bwd(dy, x, gamma, beta, want["mean"], want["rstd"], G, act="gelu")
    check_backward(back, dy, x, gamma, beta, want, G, "gelu")
    for into in ("dy", "x"):
        a, b = dy.clone(), x.clone()
        assert same(rn.groupnorm_bwd(a, b, gamma, beta, want["mean"], want["rstd"], G, act="gelu", dx=a if into == "dy" else b), back)
    a = dy.clone()
    kept_back = rn.groupnorm_bwd_ckpt8(dy, keeping["codes"], keeping["scales"], gamma, beta, want["mean"], want["rstd"], G, act="gelu")
    assert same(rn.groupnorm_bwd_ckpt8(a, keeping["codes"], keeping["scales"], gamma, beta, want["mean"], want["rstd"], G, act="gelu", dx=a), kept_back)


def test_the_device_is_asked_for_the_clusters_that_it_holds(rn):
    """The cut on this device is that for the largest cluster that it says it holds; clusters of 8 are every device's."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for size in ((3, 2000, 90, 9), (8, 4096, 320, 32), (2, 16384, 64, 8)):
        for backward in (False, True):
            here = cut(rn, *size, torch.float32, backward)
            for_most = {}
            for most in (8, 16):
                for_most[most] = Plan()
                assert rn.lib().groupnorm_plan_query(*size, 0, backward, 0, 16, 16, sms, most, ctypes.byref(for_most[most])) == 0
            assert bytes(here) in (bytes(for_most[8]), bytes(for_most[16]))
