"""The order in which the gradient of embedding rows is summed, and what it may cost.

A row of m tokens is summed in pieces of P (8 where T N <= 2^23 values, else 32) of the sorted tokens, in sequence; its
at most m / P + 2 parts by four lanes, each a quarter of them in sequence; the lanes in sequence; then one product (and,
accumulating, one sum, fused). So a sum has at most L = P + (m / P + 2) / 4 + 1 + 3 + 1 roundings in a chain, each off by
half a step of a value no larger than the sum of the magnitudes: |error| <= L 2^-24 scale sum |dh|, and the result's own
rounding."""
import pytest
import torch

from test_gpu_rows import TYPES, U, bits, gen, half_step, near, normal, offset_view, rn  # noqa: F401

pytestmark = pytest.mark.gpu


def chain(T, N, most):
    P = 8 if T * N <= 1 << 23 else 32
    return P + (most / P + 2) / 4 + 5


def power_law(g, T, V):
    return (torch.rand(T, generator=g, device="cuda").pow(6) * V).long().clamp_(max=V - 1)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,V,N", [(20000, 1, 16), (5000, 2, 24), (140000, 5, 32), (70000, 1, 264), (3000, 50, 4096), (33, 1, 8), (9, 2, 5)])
def test_long_runs_within_their_chain(rn, dt, T, V, N):
    """Values of one sign, so that a sum is as large as the sum of its magnitudes."""
    g, t = gen(T + N), TYPES[dt]
    ids = power_law(g, T, V)
    dh = (normal(g, T, N).abs() * 0.01).to(t)
    got = rn.embed_bwd(dh, ids, V, scale=1.5, dtype=torch.float32)
    ref = torch.zeros(V, N, dtype=torch.float64, device="cuda").index_add_(0, ids, dh.double()) * 1.5
    L = chain(T, N, int(torch.bincount(ids).max()))
    near(got, ref, (U + L * U) * ref, "dtable")
    base = normal(g, V, N).abs()
    acc = rn.embed_bwd(dh, ids, V, scale=1.5, dtable=base.clone(), accumulate=True)
    near(acc, ref + base.double(), (U + L * U) * (ref + base.double()), "accumulated")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,N", [(5000, 200, 24), (70000, 300, 32), (70000, 30, 264)])
def test_the_order_is_that_of_the_ids(rn, dt, T, V, N):
    """The same ids, number and row length: the same bits wherever the arrays lie, whatever the ids' type, and however
    many rows the table has beside those that have tokens."""
    g, t = gen(T + V), TYPES[dt]
    ids, dh = power_law(g, T, V), normal(g, T, N, dt=t)
    want = rn.embed_bwd(dh, ids, V)
    assert torch.equal(bits(rn.embed_bwd(offset_view(dh, 1), ids, V)), bits(want))
    assert torch.equal(bits(rn.embed_bwd(dh, ids.int(), V)), bits(want))
    more = rn.embed_bwd(dh, ids, V + 100000)
    assert torch.equal(bits(more[:V]), bits(want)) and not more[V:].any()
    assert torch.equal(rn.embed_bwd(dh, ids, V, dtype=torch.float32).to(t), want)
