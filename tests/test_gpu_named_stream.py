"""Results that the norms' calls make for a named stream (``stream=``)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

M, N = 2048, 4096


@pytest.fixture(scope="module")
def rn():
    from row_wise_normalization_rmsnorm_gb300 import build
    build.build()
    import row_wise_normalization_rmsnorm_gb300 as pkg
    return pkg


def inputs():
    g = torch.Generator(device="cuda")
    g.manual_seed(5)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    return normal(M, N), normal(M, N), normal(N)


def calls(rn, x, dy, w):
    """Each call with its one large result that is made here."""
    rows = [torch.empty(M, device="cuda") for _ in range(2)]
    y, rstd = rn.rmsnorm_fwd(x, w)
    ln = rn.layernorm_fwd(x, w, w)
    dw = torch.empty_like(w)
    return {
        "fwd": lambda **kw: rn.rmsnorm_fwd(x, w, rstd=rows[0], **kw)[0],
        "fwd_by_name": lambda **kw: rn.rmsnorm_fwd(w=w, x=x, rstd=rows[0], **kw)[0],
        "fwd_ex": lambda **kw: rn.rmsnorm_fwd_ex(x, w, rstd=rows[0], **kw)[0],
        "add_fwd": lambda **kw: rn.rmsnorm_add_fwd(x, dy, w, rstd=rows[0], residual_out=y, **kw)[0],
        "bwd": lambda **kw: rn.rmsnorm_bwd(dy, x, w, rstd, dw=dw, **kw)[0],
        "bwd_ex": lambda **kw: rn.rmsnorm_bwd_ex(dy, x, w, rstd, dw=dw, **kw)[0],
        "add_bwd": lambda **kw: rn.rmsnorm_add_bwd(dy, dy, x, w, rstd, dw=dw, **kw)[0],
        "ln_fwd": lambda **kw: rn.layernorm_fwd(x, w, w, mean=rows[0], rstd=rows[1], **kw)["y"],
        "ln_bwd": lambda **kw: rn.layernorm_bwd(dy, x, w, ln["mean"], ln["rstd"], dgamma=dw, want_dbeta=False, **kw)["dx"],
        "fp8": lambda **kw: rn.rmsnorm_fwd_fp8(x, w, rstd=rows[0], scale_inv=rows[1], **kw)["y"],
    }


@pytest.mark.parametrize("op", ["fwd", "fwd_by_name", "fwd_ex", "add_fwd", "bwd", "bwd_ex", "add_bwd", "ln_fwd", "ln_bwd", "fp8"])
def test_results_for_a_named_stream_are_not_memory_in_use_on_the_current_one(rn, op):
    """The current stream still has a late read and a late write of a block
    queued that has been dropped. What a call on another stream makes, which
    waits for none of that, must lie elsewhere."""
    call = calls(rn, *inputs())[op]
    want = call()
    kept = torch.empty_like(want)
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        block = torch.full_like(want, 3)  # of the result's size: the next one of this pool
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)
        kept.copy_(block)
        block.fill_(5)
        del block
        got = call(stream=handle)
        torch.cuda.synchronize()
        assert bool((kept == 3).all()) and torch.equal(got, want)
        del got


@pytest.mark.parametrize("handle", [0, 1, 2])
def test_default_streams_by_handle(rn, handle):
    x, _, w = inputs()
    want, rstd = rn.rmsnorm_fwd(x, w)
    torch.cuda.synchronize()
    y = torch.empty_like(x)
    got = rn.rmsnorm_fwd(x, w, y=y, stream=handle)
    torch.cuda.synchronize()
    assert got[0] is y and torch.equal(y, want) and torch.equal(got[1], rstd)
