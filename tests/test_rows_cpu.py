"""Host-side tests of the entry points on training rows (8-bit checkpoints,
group norm, embedding rows) that need no GPU: refusals as status codes before
any CUDA call, and the Python binding's checks."""
import math

import pytest
import torch

from row_wise_normalization_rmsnorm_gb300 import build as rn_build

OK, INVALID, UNSUPPORTED = 0, 1, 2
A = 4096  # a pointer that no refused call follows
F32, BF16, F16, W32 = 0, 1, 2, 0x100


@pytest.fixture(scope="module")
def rn():
    rn_build.build()
    import row_wise_normalization_rmsnorm_gb300 as pkg
    return pkg


def call(rn, name, defaults, bad):
    args = dict(defaults)
    assert set(bad) <= set(args)
    args.update(bad)
    return getattr(rn.lib(), name)(*args.values())


PACK = {"x": A, "codes": A, "scales": A, "M": 4, "N": 64, "dt": BF16, "stream": None}
UNPACK = {"codes": A, "scales": A, "x": A, "M": 4, "N": 64, "dt": BF16, "stream": None}


@pytest.mark.parametrize("bad", [{"x": None}, {"codes": None}, {"scales": None}, {"x": A + 1}, {"M": -1}, {"N": 0}, {"N": 65537},
                                 {"dt": 3}, {"dt": BF16 | W32}, {"M": 2 ** 62}])
def test_pack_and_unpack_refuse(rn, bad):
    assert call(rn, "ckpt8_pack", PACK, bad) == INVALID
    assert call(rn, "ckpt8_unpack", UNPACK, bad) == INVALID


FWD = {"x": A, "residual": A, "w": A, "y": A, "h": A, "rstd": A, "codes": A, "scales": A, "M": 4, "N": 64, "dt": BF16, "eps": 1e-6,
       "offset": 0.0, "stream": None}


@pytest.mark.parametrize("bad", [{"x": None}, {"y": None}, {"rstd": None}, {"codes": None}, {"scales": None}, {"residual": None},
                                 {"h": None}, {"x": A + 1}, {"w": A + 1}, {"rstd": A + 2}, {"M": -1}, {"M": 2 ** 31}, {"N": 0},
                                 {"N": 65537}, {"dt": 3}, {"dt": 0x201}, {"eps": -1.0}, {"eps": math.nan}, {"offset": math.inf},
                                 {"dt": BF16 | W32, "w": A + 2}])
def test_norm_forward_refuses(rn, bad):
    assert call(rn, "rmsnorm_fwd_ckpt8", FWD, bad) == INVALID


BWD = {"dy": A, "dres": A, "codes": A, "scales": A, "w": A, "rstd": A, "dx": A, "dw": A, "ws": None, "ws_bytes": 0, "M": 4, "N": 64,
       "dt": BF16, "offset": 0.0, "stream": None}


@pytest.mark.parametrize("bad", [{"dy": None}, {"codes": None}, {"scales": None}, {"rstd": None}, {"dx": None}, {"w": None},
                                 {"dw": None}, {"dy": A + 1}, {"dres": A + 1}, {"dx": A + 1}, {"dw": A + 1}, {"rstd": A + 1},
                                 {"M": -1}, {"N": 0}, {"N": 65537}, {"dt": 5}, {"offset": math.nan}])
def test_norm_backward_refuses(rn, bad):
    assert call(rn, "rmsnorm_bwd_ckpt8", BWD, bad) == INVALID


GN = {"x": A, "gamma": A, "beta": A, "y": A, "mean": A, "rstd": A, "codes": A, "scales": A, "ws": None, "ws_bytes": 0, "B": 2, "S": 9,
      "C": 64, "G": 8, "act": 1, "dt": BF16, "eps": 1e-5, "stream": None}


@pytest.mark.parametrize("bad", [{"x": None}, {"y": None}, {"mean": None}, {"rstd": None}, {"codes": None}, {"scales": None},
                                 {"x": A + 1}, {"y": A + 1}, {"gamma": A + 1}, {"beta": A + 1}, {"mean": A + 2}, {"B": -1}, {"S": -1},
                                 {"C": 0}, {"C": 8200, "G": 8}, {"G": 0}, {"G": 7}, {"G": 65}, {"act": 3}, {"act": -1}, {"dt": 3},
                                 {"eps": -1.0}, {"eps": math.inf}, {"B": 2 ** 31}, {"B": 2 ** 30, "S": 2 ** 30, "C": 8192}])
def test_groupnorm_forward_refuses(rn, bad):
    assert call(rn, "groupnorm_fwd", GN, bad) == INVALID


def test_groupnorm_refuses_too_many_groups(rn):
    assert call(rn, "groupnorm_fwd", GN, {"C": 8192, "G": 8192}) == UNSUPPORTED
    assert call(rn, "groupnorm_bwd", GNB, {"C": 8192, "G": 8192}) == UNSUPPORTED
    assert call(rn, "groupnorm_fwd", GN, {"B": 0}) == OK


GNB = {"dy": A, "x": A, "codes": None, "scales": None, "gamma": A, "beta": A, "mean": A, "rstd": A, "dx": A, "dgamma": A, "dbeta": A,
       "ws": None, "ws_bytes": 0, "B": 2, "S": 9, "C": 64, "G": 8, "act": 1, "dt": BF16, "stream": None}


@pytest.mark.parametrize("bad", [{"dy": None}, {"x": None}, {"codes": A}, {"codes": A, "scales": A}, {"x": None, "codes": A},
                                 {"gamma": None}, {"mean": None}, {"rstd": None}, {"dx": None}, {"dgamma": A + 1}, {"dbeta": A + 1},
                                 {"dy": A + 1}, {"G": 7}, {"act": 3}, {"dt": 9}, {"rstd": A + 1}])
def test_groupnorm_backward_refuses(rn, bad):
    assert call(rn, "groupnorm_bwd", GNB, bad) == INVALID


EMBED = {"ids": A, "table": A, "h": A, "T": 4, "N": 64, "rows": 10, "id_bytes": 8, "dt": BF16, "scale": 1.0, "stream": None}
EMBED_NORM = {"ids": A, "table": A, "w": A, "y": A, "h": A, "rstd": A, "T": 4, "N": 64, "rows": 10, "id_bytes": 8, "dt": BF16,
              "scale": 1.0, "eps": 1e-6, "offset": 0.0, "stream": None}
EMBED_BWD = {"dh": A, "ids": A, "dtable": A, "ws": None, "ws_bytes": 0, "T": 4, "N": 64, "rows": 10, "id_bytes": 8, "dt": BF16,
             "scale": 1.0, "accumulate": 0, "stream": None}


@pytest.mark.parametrize("bad", [{"ids": None}, {"ids": A + 4}, {"T": -1}, {"N": 0}, {"N": 65537}, {"rows": -1}, {"id_bytes": 2},
                                 {"dt": 3}, {"scale": math.nan}])
def test_embedding_refuses(rn, bad):
    assert call(rn, "embed_fwd", EMBED, bad) == INVALID
    assert call(rn, "rmsnorm_embed_fwd", EMBED_NORM, bad) == INVALID
    assert call(rn, "embed_bwd", EMBED_BWD, bad) == INVALID


@pytest.mark.parametrize("name,defaults,bad", [
    ("embed_fwd", EMBED, {"table": None}), ("embed_fwd", EMBED, {"h": None}), ("embed_fwd", EMBED, {"dt": BF16 | W32}),
    ("embed_fwd", EMBED, {"h": A + 1}), ("rmsnorm_embed_fwd", EMBED_NORM, {"y": None}), ("rmsnorm_embed_fwd", EMBED_NORM, {"rstd": None}),
    ("rmsnorm_embed_fwd", EMBED_NORM, {"eps": -1.0}), ("rmsnorm_embed_fwd", EMBED_NORM, {"w": A + 1}),
    ("embed_bwd", EMBED_BWD, {"dh": None}), ("embed_bwd", EMBED_BWD, {"dtable": None}), ("embed_bwd", EMBED_BWD, {"rows": 2 ** 31 - 1}),
    ("embed_bwd", EMBED_BWD, {"dtable": A + 1}), ("embed_bwd", EMBED_BWD, {"dt": F16 | W32, "dtable": A + 2}),
])
def test_embedding_refuses_its_own(rn, name, defaults, bad):
    assert call(rn, name, defaults, bad) == INVALID


def test_calls_of_nothing_succeed(rn):
    assert call(rn, "ckpt8_pack", PACK, {"M": 0, "x": None, "codes": None, "scales": None}) == OK
    assert call(rn, "rmsnorm_fwd_ckpt8", FWD, {"M": 0}) == OK
    assert call(rn, "embed_fwd", EMBED, {"T": 0}) == OK
    assert call(rn, "embed_bwd", EMBED_BWD, {"T": 0, "accumulate": 1}) == OK
    assert call(rn, "embed_bwd", EMBED_BWD, {"rows": 0}) == OK


def test_embedding_workspace(rn):
    need = rn.embed_bwd_workspace_bytes
    assert need(0, 64, 10) == 0 and need(64, 0, 10) == 0 and need(64, 64, 0) == 0
    # keys and tokens, a bit a row, the pieces' two partial rows
    assert need(64, 64, 100) >= 64 * 8 + 16 + 2 * 2 * 64 * 4
    assert need(70000, 8, 100) > need(65536, 8, 100)


def test_python_refuses(rn):
    x = torch.zeros(4, 8)
    w = torch.zeros(8)
    i8, u8 = torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4, 1, dtype=torch.uint8)
    ids = torch.zeros(4, dtype=torch.int64)
    for f in (lambda: rn.ckpt8_pack(x), lambda: rn.ckpt8_unpack(i8, u8, torch.bfloat16), lambda: rn.rmsnorm_fwd_ckpt8(x, w),
              lambda: rn.rmsnorm_bwd_ckpt8(x, i8, u8, w, x[:, 0]), lambda: rn.groupnorm_fwd(x, w, w, 2),
              lambda: rn.groupnorm_bwd(x, x, w, w, w, w, 2), lambda: rn.embed_fwd(ids, x), lambda: rn.embed_bwd(x, ids, 5)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            f()
    for f in (lambda: rn.ckpt8_pack(3), lambda: rn.groupnorm_fwd(None, w, w, 2), lambda: rn.embed_fwd(ids, None)):
        with pytest.raises(TypeError, match="torch.Tensor"):
            f()
    with pytest.raises(TypeError):
        rn.groupnorm_fwd(x, w, w)
