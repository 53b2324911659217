"""Host-side checks of the paged-pool entry points: refusals, sizes, the rotary
layout.  No call here launches a kernel."""
import ctypes as C
import math

import pytest


@pytest.fixture(scope="module")
def kvq():
    from quantized_kv_cache_kv8_gb300 import kvq as K
    K.lib()
    return K


D = C.c_void_p(1 << 20)          # dummy device addresses, never dereferenced
E = C.c_void_p(1 << 21)
ODD = C.c_void_p((1 << 20) + 2)
BIG = 1 << 30


def reserve(L, n_seq=2, page=64, lens=D, new=E, table=D, stride=4, free=D, n_free=D, n_pages=8, out=D, cu=D, slots=D,
            pos=None, max_new=4, ws=D, size=BIG):
    return L.kv_pages_reserve(n_seq, page, lens, new, table, stride, free, n_free, n_pages, out, cu, slots, pos, max_new,
                              ws, size, None)


@pytest.mark.parametrize("bad,status", [
    (dict(n_seq=-1), 1), (dict(page=0), 1), (dict(stride=-1), 1), (dict(n_pages=-1), 1), (dict(max_new=-1), 1),
    (dict(page=48), 5), (dict(page=1 << 17), 5), (dict(n_seq=65536), 5), (dict(n_pages=1 << 26), 5),
    (dict(max_new=1 << 31), 5), (dict(lens=None), 1), (dict(new=None), 1), (dict(table=None), 1), (dict(free=None), 1),
    (dict(n_free=None), 1), (dict(out=None), 1), (dict(cu=None), 1), (dict(slots=None), 1), (dict(out=E), 1),
    (dict(lens=C.c_void_p((1 << 20) + 4)), 1), (dict(table=ODD), 1), (dict(pos=ODD), 1), (dict(ws=None), 3),
    (dict(size=128), 3),
])
def test_reserve_refuses(kvq, bad, status):
    assert reserve(kvq.lib(), **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(n_seq=-1), 1), (dict(page=3), 5), (dict(lens=None), 1), (dict(keep=None), 1), (dict(keep=D), 1),
    (dict(n_free=None), 1), (dict(ws=None), 3), (dict(size=0), 3), (dict(free=ODD), 1),
])
def test_trim_refuses(kvq, bad, status):
    a = dict(n_seq=2, page=64, lens=D, keep=E, table=D, stride=4, free=D, n_free=D, n_pages=8, ws=D, size=BIG)
    a.update(bad)
    assert kvq.lib().kv_pages_trim(a["n_seq"], a["page"], a["lens"], a["keep"], a["table"], a["stride"], a["free"],
                                   a["n_free"], a["n_pages"], a["ws"], a["size"], None) == status


def rope_call(kvq, **kw):
    a = dict(fmt=1, layout=kvq.mla_layout(), rope=kvq.rope_layout([1.0] * 32), x=D, xd=1, xs=576, n=4, pos=D, ps=4,
             slots=D, qi=D, qd=1, qit=64 * 8, qih=64, qo=E, qot=576 * 8, qoh=576, heads=8, codes=D, scales=D, rows=8,
             err=None)
    a.update(kw)
    rope = a["rope"]
    return kvq.lib().kv_rope_append(a["fmt"], C.byref(a["layout"]), None if rope is None else C.byref(rope), a["x"],
                                    a["xd"], a["xs"], a["n"], a["pos"], a["ps"], a["slots"], a["qi"], a["qd"], a["qit"],
                                    a["qih"], a["qo"], a["qot"], a["qoh"], a["heads"], a["codes"], a["scales"],
                                    a["rows"], a["err"], None)


def test_rope_append_refuses(kvq):
    lay = kvq.mla_layout
    two = kvq.rope_layout([1.0] * 32, [0] * 16 + [1] * 16)
    wrong_axis = kvq.rope_layout([1.0] * 32)
    wrong_axis.axis[3] = 1
    odd = kvq.rope_layout([1.0] * 32)
    odd.dim = 63
    wide = kvq.rope_layout([1.0] * 64)
    wide.dim = 130
    nan = kvq.rope_layout([1.0] * 31 + [math.inf])
    for kw, status in [
        (dict(fmt=3), 1), (dict(fmt=14), 5), (dict(fmt=2, layout=lay((500, 76))), 2), (dict(rope=None), 1),
        (dict(rope=wrong_axis), 1), (dict(rope=odd), 1), (dict(rope=wide), 5), (dict(rope=nan), 1),
        (dict(layout=lay((1024, 64)), xs=1088), 5), (dict(layout=lay((32,), v_dim=32)), 1), (dict(xd=7), 1),
        (dict(qd=7), 1), (dict(n=-1), 1), (dict(heads=-1), 1), (dict(heads=70000), 5), (dict(pos=None), 1),
        (dict(rope=two, ps=3), 1), (dict(slots=None), 1), (dict(xs=575), 1), (dict(codes=None), 1),
        (dict(scales=None), 1), (dict(qi=None), 1), (dict(qo=None), 1), (dict(qo=D), 1),
        (dict(x=C.c_void_p((1 << 20) + 1)), 1), (dict(pos=C.c_void_p((1 << 20) + 4)), 1), (dict(rows=-1), 1),
    ]:
        assert rope_call(kvq, **kw) == status, kw
    assert rope_call(kvq, n=0, x=None, pos=None) == 0
    with pytest.raises(ValueError):
        kvq.rope_layout([])
    with pytest.raises(ValueError):
        kvq.rope_layout([1.0] * 65)
    with pytest.raises(ValueError):
        kvq.rope_layout([1.0, 2.0], [0])


def attn_call(kvq, **kw):
    a = dict(fmt=1, layout=kvq.mla_layout(), q=D, dt=1, n=4, heads=16, n_seq=2, cu=D, codes=D, scales=D, table=D, stride=4,
             lens=D, page=64, n_pages=8, sm=0.1, out=E, ws=D, size=BIG, path=0)
    a.update(kw)
    return kvq.lib().kv_attn_paged(a["fmt"], C.byref(a["layout"]), a["q"], a["dt"], a["n"], a["heads"], a["n_seq"],
                                   a["cu"], a["codes"], a["scales"], a["table"], a["stride"], a["lens"], a["page"],
                                   a["n_pages"], a["sm"], a["out"], a["ws"], a["size"], a["path"], None)


def test_attn_paged_refuses(kvq):
    lay = kvq.mla_layout
    for kw, status in [
        (dict(fmt=14), 5), (dict(fmt=9), 1), (dict(layout=lay((256, 64), v_dim=256)), 5), (dict(fmt=2, layout=lay((576,))), 2),
        (dict(path=3), 1), (dict(dt=4), 1), (dict(dt=0, path=2), 5), (dict(page=8), 5), (dict(page=100), 5),
        (dict(n_pages=1 << 26), 5), (dict(n_seq=-1), 1), (dict(n_seq=70000), 5), (dict(heads=-1), 1), (dict(n=-1), 1),
        (dict(sm=math.nan), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(cu=None), 1), (dict(lens=None), 1),
        (dict(codes=None), 1), (dict(scales=None), 1), (dict(table=None), 1), (dict(codes=C.c_void_p((1 << 20) + 16)), 1),
        (dict(q=C.c_void_p((1 << 20) + 8)), 1), (dict(out=C.c_void_p((1 << 20) + 8)), 1),
        (dict(lens=C.c_void_p((1 << 20) + 4)), 1), (dict(table=ODD), 1), (dict(ws=None), 3), (dict(size=1000), 3),
    ]:
        assert attn_call(kvq, **kw) == status, kw
    for kw in (dict(n=0), dict(heads=0), dict(n_seq=0)):
        assert attn_call(kvq, q=None, out=None, cu=None, ws=None, **kw) == 0


def test_attn_paged_workspace_is_independent_of_lengths(kvq):
    size = kvq.kv_attn_paged_workspace_size
    a = size(1, 1, 16, 1)
    assert a == size(1, 1000, 128, 100000) == size(2, 8, 128, 8) > 2 * 152 * 64 * 512 * 4
    assert size(1, 1, 16, 1, bf16=False) < a
    assert size(14, 1, 16, 1) == 0
    assert size(1, 1, 16, 1, bf16=False, path=kvq.PATH_TENSOR) == 0
    assert kvq.kv_pages_workspace_size() >= 8


def test_rope_append_refuses_outputs_that_overlap(kvq):
    assert rope_call(kvq, qoh=0) == 1 and rope_call(kvq, qot=0) == 1


def test_paged_calls_check_their_tensors(kvq):
    """The extension's own refusals that need no GPU."""
    import torch
    host = kvq._paged()
    t = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        host.trim(t, t, t, t, t, 16, t, 0, 0)          # not on a GPU
    with pytest.raises(TypeError):
        host.trim(1, t, t, t, t, 16, t, 0, 0)          # not a tensor
    with pytest.raises(TypeError):
        host.trim(t, t)
    with pytest.raises(TypeError):
        host.reserve(t, t, t, t, t, 16, t, t, t, t, t, "0", 0)
    with pytest.raises(ValueError):                    # a rotary layout where the row layout belongs
        host.rope_append(1, kvq.rope_layout([1.0]), None, t, t, None, t, t, t, kvq.rope_layout([1.0]), None, 0, 0)
