"""Host-side tests of the entry points on head rows (rotary positions, the
paged cache, its attention) that need no GPU: refusals as status codes before
any CUDA call, the Python binding's checks, and the axes' map."""
import ctypes

import pytest
import torch

from row_wise_normalization_rmsnorm_gb300 import build as rn_build

_p, _q, _i, _f = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


class Rows(ctypes.Structure):
    _fields_ = [("in_", _p), ("out", _p), ("in_token", _q), ("in_head", _q), ("out_token", _q), ("out_head", _q)]


class Angles(ctypes.Structure):
    _fields_ = [("positions", _p), ("inv_freq", _p), ("axis_stride", _q), ("position_bytes", _i), ("n_axes", _i),
                ("rotary_dim", _i), ("pairing", _i)]


class RopeCall(ctypes.Structure):
    _fields_ = [("q", Rows), ("k", Rows), ("angles", Angles), ("tokens", _q), ("q_heads", _i), ("k_heads", _i),
                ("head_dim", _i), ("dtype", _i)]


class Cache(ctypes.Structure):
    _fields_ = [("k", _p), ("v", _p), ("pages", _q), ("k_page", _q), ("k_slot", _q), ("k_head", _q), ("v_page", _q),
                ("v_slot", _q), ("v_head", _q), ("page_size", _i), ("heads", _i)]


class AppendCall(ctypes.Structure):
    _fields_ = [("q", Rows), ("k", Rows), ("v", Rows), ("angles", Angles), ("cache", Cache), ("slots", _p), ("wq", _p),
                ("wk", _p), ("tokens", _q), ("eps", _f), ("offset", _f), ("q_heads", _i), ("head_dim", _i),
                ("dtype", _i), ("reserved", _i)]


class AttnCall(ctypes.Structure):
    _fields_ = [("q", _p), ("out", _p), ("lse", _p), ("q_token", _q), ("q_head", _q), ("out_token", _q),
                ("out_head", _q), ("cache", Cache), ("block_table", _p), ("kv_lens", _p), ("cu_q", _p),
                ("table_stride", _q), ("tokens", _q), ("workspace", _p), ("workspace_bytes", ctypes.c_size_t),
                ("scale", _f), ("batch", _i), ("table_width", _i), ("q_heads", _i), ("head_dim", _i), ("max_q", _i),
                ("max_kv", _i), ("causal", _i), ("dtype", _i)]


@pytest.fixture(scope="module")
def rn():
    rn_build.build()
    import row_wise_normalization_rmsnorm_gb300 as pkg
    return pkg


A = 4096  # a pointer that no refused call follows


def rope_call(**kw):
    c = RopeCall()
    c.q = Rows(A, A, 512, 64, 512, 64)
    c.k = Rows(A, A, 128, 64, 128, 64)
    c.angles = Angles(A, A, 0, 4, 1, 64, 0)
    c.tokens, c.q_heads, c.k_heads, c.head_dim, c.dtype = 4, 8, 2, 64, 1
    for name, v in kw.items():
        at = c
        *path, last = name.split("__")
        for part in path:
            at = getattr(at, part)
        setattr(at, last, v)
    return c


@pytest.mark.parametrize("bad", [
    {"dtype": 3}, {"dtype": 0x101}, {"head_dim": 0}, {"head_dim": 257}, {"tokens": -1}, {"q_heads": 0}, {"k_heads": -1},
    {"q__in_": None}, {"q__out": None}, {"k__in_": None}, {"q__in_": A + 1}, {"k__out": A + 1},
    {"angles__positions": None}, {"angles__positions": A + 2}, {"angles__inv_freq": None}, {"angles__inv_freq": A + 2},
    {"angles__position_bytes": 2}, {"angles__n_axes": 0}, {"angles__n_axes": 5}, {"angles__rotary_dim": 0},
    {"angles__rotary_dim": 63}, {"angles__rotary_dim": 66}, {"angles__pairing": 2},
])
def test_rope_refuses(rn, bad):
    for fn in (rn.lib().rope_fwd, rn.lib().rope_bwd):
        assert fn(ctypes.byref(rope_call(**bad)), None, None) == INVALID


def test_rope_refuses_an_axis_it_has_not(rn):
    c = rope_call()
    assert rn.lib().rope_fwd(ctypes.byref(c), bytes([0] * 31 + [1]), None) == INVALID
    assert rn.lib().rope_fwd(None, None, None) == INVALID


def test_rope_of_no_tokens_is_done(rn):
    c = rope_call(tokens=0, q__in_=None, q__out=None)
    assert rn.lib().rope_fwd(ctypes.byref(c), None, None) == 0


def append_call(**kw):
    c = AppendCall()
    c.q = Rows(A, A, 512, 64, 512, 64)
    c.k = Rows(A, None, 128, 64, 0, 0)
    c.v = Rows(A, None, 128, 64, 0, 0)
    c.angles = Angles(A, A, 0, 4, 1, 64, 0)
    c.cache = Cache(A, A, 10, 2048, 128, 64, 2048, 128, 64, 16, 2)
    c.slots = A
    c.tokens, c.eps, c.q_heads, c.head_dim, c.dtype = 4, 1e-6, 8, 64, 1
    for name, v in kw.items():
        at = c
        *path, last = name.split("__")
        for part in path:
            at = getattr(at, part)
        setattr(at, last, v)
    return c


@pytest.mark.parametrize("bad", [
    {"dtype": 3}, {"head_dim": 0}, {"head_dim": 257}, {"tokens": -1}, {"q_heads": -1}, {"cache__heads": 0},
    {"cache__page_size": 0}, {"cache__pages": -1}, {"cache__k": None}, {"cache__v": None}, {"cache__k": A + 1},
    {"k__in_": None}, {"v__in_": None}, {"v__in_": A + 1}, {"q__out": None}, {"slots": None}, {"slots": A + 4},
    {"wq": A + 1}, {"wk": A + 1}, {"dtype": 0x101, "wk": A + 2}, {"eps": -1.0}, {"eps": float("nan")},
    {"offset": float("inf")}, {"angles__inv_freq": None}, {"angles__rotary_dim": 66},
])
def test_append_refuses(rn, bad):
    assert rn.lib().paged_kv_append(ctypes.byref(append_call(**bad)), None, None) == INVALID


@pytest.mark.parametrize("bad", [{"q__out_token": 0}, {"q__out_head": 0}, {"k__out_token": 0}, {"k__out_head": 0}])
def test_rope_refuses_rows_that_overwrite_one_another(rn, bad):
    assert rn.lib().rope_fwd(ctypes.byref(rope_call(**bad)), None, None) == INVALID
    assert rn.lib().rope_bwd(ctypes.byref(rope_call(**bad)), None, None) == INVALID


@pytest.mark.parametrize("bad", [
    {"q__out_token": 0}, {"q__out_head": 0}, {"cache__k_page": 0}, {"cache__k_slot": 0}, {"cache__k_head": 0},
    {"cache__v_page": 0}, {"cache__v_slot": 0}, {"cache__v_head": 0},
    {"cache__pages": 2 ** 40, "cache__page_size": 2 ** 30},   # places that 64 bits do not count
])
def test_append_refuses_places_that_overwrite_one_another(rn, bad):
    assert rn.lib().paged_kv_append(ctypes.byref(append_call(**bad)), None, None) == INVALID


@pytest.mark.parametrize("bad", [{"out_token": 0}, {"out_head": 0}])
def test_attention_refuses_rows_that_overwrite_one_another(rn, bad):
    assert rn.lib().paged_attn_fwd(ctypes.byref(attn_call(**bad)), None) == INVALID


def test_append_of_no_tokens_is_done(rn):
    assert rn.lib().paged_kv_append(ctypes.byref(append_call(tokens=0, slots=None)), None, None) == 0
    assert rn.lib().paged_kv_append(None, None, None) == INVALID


def attn_call(**kw):
    c = AttnCall()
    c.q, c.out, c.lse = A, A, A
    c.q_token, c.q_head, c.out_token, c.out_head = 512, 64, 512, 64
    c.cache = Cache(A, A, 10, 2048, 128, 64, 2048, 128, 64, 16, 2)
    c.block_table, c.kv_lens, c.cu_q, c.table_stride, c.tokens = A, A, A, 4, 4
    c.scale, c.batch, c.table_width, c.q_heads, c.head_dim, c.max_q, c.max_kv = 0.125, 4, 4, 8, 64, 1, 64
    c.causal, c.dtype = 1, 1
    for name, v in kw.items():
        at = c
        *path, last = name.split("__")
        for part in path:
            at = getattr(at, part)
        setattr(at, last, v)
    return c


@pytest.mark.parametrize("bad,status", [
    ({"dtype": 0}, UNSUPPORTED), ({"dtype": 7}, INVALID), ({"dtype": 0x101}, INVALID), ({"head_dim": 0}, INVALID),
    ({"head_dim": 68}, UNSUPPORTED), ({"head_dim": 136}, UNSUPPORTED), ({"q_heads": 9}, INVALID),
    ({"q_heads": 0}, INVALID), ({"q_heads": 258}, UNSUPPORTED), ({"cache__heads": 0}, INVALID), ({"batch": -1}, INVALID),
    ({"tokens": -1}, INVALID), ({"max_q": -1}, INVALID), ({"max_kv": -1}, INVALID), ({"table_width": -1}, INVALID),
    ({"scale": 0.0}, INVALID), ({"scale": -1.0}, INVALID), ({"scale": float("nan")}, INVALID),
    ({"scale": float("inf")}, INVALID), ({"scale": 3e38}, INVALID), ({"max_kv": 2 ** 31 - 1}, UNSUPPORTED), ({"cache__page_size": 0}, INVALID), ({"cache__page_size": 12}, UNSUPPORTED),
    ({"cache__pages": -1}, INVALID), ({"q": None}, INVALID), ({"out": None}, INVALID), ({"q": A + 1}, INVALID),
    ({"lse": A + 2}, INVALID), ({"kv_lens": None}, INVALID), ({"cu_q": None}, INVALID), ({"block_table": None}, INVALID),
    ({"kv_lens": A + 2}, INVALID), ({"cache__k": None}, INVALID), ({"cache__k": A + 2}, UNSUPPORTED),
    ({"cache__v_slot": 68}, UNSUPPORTED), ({"cache__k_page": 2052}, UNSUPPORTED), ({"cache__k_head": 0}, UNSUPPORTED),
    ({"workspace": A + 8, "workspace_bytes": 1 << 20}, WORKSPACE),
])
def test_attention_refuses(rn, bad, status):
    assert rn.lib().paged_attn_fwd(ctypes.byref(attn_call(**bad)), None) == status


def test_attention_of_nothing_is_done(rn):
    for kw in ({"tokens": 0, "q": None, "out": None}, {"batch": 0}, {"max_q": 0}):
        assert rn.lib().paged_attn_fwd(ctypes.byref(attn_call(**kw)), None) == 0
    assert rn.lib().paged_attn_fwd(None, None) == INVALID
    assert rn.lib().paged_attn_workspace_bytes(None) == 0
    assert rn.lib().paged_attn_workspace_bytes(ctypes.byref(attn_call(head_dim=68))) == 0


class AttnPlan(ctypes.Structure):
    _fields_ = [("row_tiles", _i), ("tile_tokens", _i), ("q_tiles", _i), ("splits", _i), ("chunk", _i),
                ("clustered", _i), ("workspace_bytes", _q)]


# clusters of 0 .. 16 CTAs that a device holds at once: as a GB300 of 152 SMs
# answers, a device without room for any, and one of whole parts
GB300 = [0, 304, 152, 97, 74, 58, 46, 38, 36, 30, 28, 23, 23, 19, 14, 14, 14]
NONE = [0] * 17
WHOLE = [0, 304] + [8 * (38 // s) for s in range(2, 17)]


def attn_plan(rn, clusters, batch, heads, kv_heads, max_q, max_kv, sms=152):
    p = AttnPlan()
    c = attn_call(tokens=batch * max_q, batch=batch, q_heads=heads, cache__heads=kv_heads, max_q=max_q, max_kv=max_kv)
    held = (_i * 17)(*clusters)
    assert rn.lib().paged_attn_plan_query(ctypes.byref(c), sms, held, ctypes.byref(p)) == 0
    return p


@pytest.mark.parametrize("held", [GB300, NONE, WHOLE])
@pytest.mark.parametrize("batch,kv_heads", [(1, 1), (1, 8), (2, 8), (15, 1), (16, 1), (5, 3), (3, 16), (6, 8), (7, 8), (19, 8)])
def test_attention_clusters_are_as_many_as_the_device_holds(rn, held, batch, kv_heads):
    """A row's keys are cut over a cluster only where all of the call's
    clusters run at once; else a second kernel joins the pieces."""
    for max_kv in (500, 4095, 8192, 20000, 32768, 65536, 2 ** 20):
        p = attn_plan(rn, held, batch, 4 * kv_heads, kv_heads, 1, max_kv)
        assert p.row_tiles == 1 and (p.splits - 1) * p.chunk < max_kv
        assert p.splits == 1 or p.splits * p.chunk >= max_kv
        if p.clustered:
            assert 2 <= p.splits <= 16 and held[p.splits] >= batch * kv_heads and p.workspace_bytes == 0
        else:
            assert (p.workspace_bytes > 0) == (p.splits > 1)
    if held == GB300 and batch * kv_heads == 16:
        # 14 clusters of 16 are held, and of 13 enough
        assert attn_plan(rn, held, batch, 4 * kv_heads, kv_heads, 1, 128 * 128).splits <= 13


def test_attention_items_are_bounded_in_max_kv(rn):
    for batch, heads, kv_heads, max_q in ((128, 64, 8, 1), (128, 64, 8, 4), (40, 16, 8, 8), (64, 32, 8, 1), (90, 7, 7, 9)):
        for max_kv in (4096, 8192, 2 ** 15, 2 ** 20, 2 ** 30):
            p = attn_plan(rn, GB300, batch, heads, kv_heads, max_q, max_kv)
            assert p.splits == 1 or p.splits * batch * kv_heads * p.q_tiles <= 32 * 304


def test_attention_plan_refuses(rn):
    p, held = AttnPlan(), (_i * 17)(*GB300)
    ask = rn.lib().paged_attn_plan_query
    assert ask(None, 152, held, ctypes.byref(p)) == INVALID
    assert ask(ctypes.byref(attn_call()), 152, held, None) == INVALID
    assert ask(ctypes.byref(attn_call()), 152, None, ctypes.byref(p)) == INVALID
    assert ask(ctypes.byref(attn_call(head_dim=68)), 152, held, ctypes.byref(p)) == UNSUPPORTED
    for kw in ({"tokens": 0}, {"batch": 0}, {"max_q": 0}):
        assert ask(ctypes.byref(attn_call(**kw)), 152, held, ctypes.byref(p)) == INVALID


def test_library_exports_the_head_row_calls(rn):
    from row_wise_normalization_rmsnorm_gb300._binding import SIGNATURES
    for name in ("rope_fwd", "rope_bwd", "paged_kv_append", "paged_attn_fwd", "paged_attn_workspace_bytes"):
        assert name in SIGNATURES and hasattr(rn.lib(), name)


def test_axes_in_blocks_and_dealt(rn):
    assert rn.rope_axes((2, 1, 3)) == bytes([0, 0, 1, 2, 2, 2])
    assert rn.rope_axes((2, 1, 3), interleaved=True) == bytes([0, 1, 2, 0, 2, 2])
    assert rn.rope_axes([4]) == bytes(4)
    for bad in ((), (1, 2, 3, 4, 5), (2, -1)):
        with pytest.raises(ValueError):
            rn.rope_axes(bad)


def test_python_calls_refuse_what_is_not_on_a_gpu(rn):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    f = torch.ones(32)
    with pytest.raises(ValueError, match="CUDA"):
        rn.rope_fwd(x, None, torch.zeros(4, dtype=torch.int32), f)
    with pytest.raises(TypeError, match="torch.Tensor"):
        rn.rope_bwd([1.0], None, torch.zeros(4, dtype=torch.int32), f)
    with pytest.raises(TypeError, match="dtype"):
        rn.rope_fwd(x.double(), None, torch.zeros(4, dtype=torch.int32), f)
    c = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        rn.paged_kv_append(x, x, c, c, torch.zeros(4, dtype=torch.int64))
    t = torch.zeros(1, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        rn.paged_attn_fwd(x, c, c, t, t[0, :1], t[0, :2], max_q=4, max_kv=8)
