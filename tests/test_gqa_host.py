"""Host checks of the grouped-query and beam-search calls: what they refuse before any launch."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def kvq():
    from quantized_kv_cache_kv8_gb300 import kvq as K
    K.lib()
    return K


D = C.c_void_p(4096)      # aligned for every operand, never dereferenced
ODD = C.c_void_p(4096 + 8)


def attn(kvq, heads=8, kv=2, dim=128, n=4, seqs=2, stride=4, page=16, pages=8, sm=0.1, dt=1, q=D, k=D, table=D, out=D, ws=D,
         ws_bytes=None):
    if ws_bytes is None:
        ws_bytes = kvq.kv_gqa_attn_paged_workspace_size(2, 8, 2, 256, 4)
    return kvq.lib().kv_gqa_attn_paged(q, dt, n, heads, kv, dim, seqs, D, k, D, D, table, stride, D, page, pages, sm, 1, out, ws,
                                       ws_bytes, None)


def test_attention_refusals(kvq):
    assert attn(kvq, heads=7) == 1 and attn(kvq, kv=0) == 1 and attn(kvq, heads=-2) == 1
    assert attn(kvq, dim=96) == 5 and attn(kvq, dim=0) == 5
    assert attn(kvq, page=8) == 5 and attn(kvq, page=24) == 5 and attn(kvq, page=0) == 1
    assert attn(kvq, n=-1) == 1 and attn(kvq, seqs=-1) == 1 and attn(kvq, dt=2) == 1
    assert attn(kvq, sm=float("nan")) == 1 and attn(kvq, q=None) == 1 and attn(kvq, k=None) == 1
    assert attn(kvq, q=ODD) == 1 and attn(kvq, out=ODD) == 1 and attn(kvq, k=ODD) == 1
    assert attn(kvq, ws=None) == 3 and attn(kvq, ws_bytes=1000) == 3
    assert attn(kvq, pages=1 << 30, page=16) == 5 and attn(kvq, n=1 << 30) == 5
    assert attn(kvq, n=0) == 0 and attn(kvq, seqs=0) == 0 and attn(kvq, heads=0) == 0
    assert kvq.kv_gqa_attn_paged_workspace_size(1, 7, 2, 128, 1) == 0
    assert kvq.kv_gqa_attn_paged_workspace_size(1, 8, 2, 100, 1) == 0


def append(kvq, rope=None, dt=1, n=4, heads=8, kv=2, dim=128, k=D, v=D, pos=D, pos_stride=4, slots=D, q=D, qo=D, qos=(1024, 128),
           codes=D, page=16, pages=8):
    return kvq.lib().kv_gqa_append(C.byref(rope) if rope else None, dt, n, heads, kv, dim, k, 256, 128, v, 256, 128, pos,
                                   pos_stride, slots, q, 1024, 128, qo, qos[0], qos[1], codes, codes, codes, page, pages, None,
                                   None)


def test_append_refusals(kvq):
    rope = kvq.rope_layout([1.0] * 64)
    wide, axes, bad = kvq.rope_layout([1.0] * 64), kvq.rope_layout([1.0], [1]), kvq.rope_layout([float("inf")])
    assert append(kvq, wide, dim=64) == 1            # more rotary dims than the head has
    assert append(kvq, axes, pos_stride=3) == 1 and append(kvq, bad) == 1
    assert append(kvq, rope, pos=None) == 1 and append(kvq, slots=None) == 1
    assert append(kvq, k=None) == 1 and append(kvq, v=None) == 1 and append(kvq, q=None) == 1
    assert append(kvq, heads=9) == 1 and append(kvq, dim=80) == 5 and append(kvq, page=8) == 5 and append(kvq, dt=3) == 1
    assert append(kvq, codes=ODD) == 1 and append(kvq, codes=None) == 1
    assert append(kvq, qo=D, qos=(1024, 64)) == 1    # in place at other strides
    assert append(kvq, qo=C.c_void_p(8192), qos=(0, 128)) == 1
    assert append(kvq, n=0) == 0 and append(kvq, n=-1) == 1


def test_beam_refusals(kvq):
    def select(n=2, beams=4, vocab=100, keep=8, dt=1, stride=100, x=D, ws=D, ws_bytes=1 << 20):
        return kvq.lib().kv_beam_select(x, dt, stride, n, beams, vocab, D, keep, D, D, D, ws, ws_bytes, None)
    assert select(beams=0) == 1 and select(beams=33) == 5 and select(keep=0) == 1 and select(keep=65) == 5
    assert select(vocab=0) == 1 and select(stride=99) == 1 and select(dt=2) == 1 and select(x=None) == 1
    assert select(x=C.c_void_p(4097)) == 1 and select(ws=None) == 3 and select(ws_bytes=100) == 3 and select(n=0) == 0
    assert kvq.kv_beam_workspace_size(2, 40, 100, 8) == 0 and select(n=65536) == 5
    for v in (100, 30000, 200000):   # fewer requests have more slices each, and no larger a workspace
        for b in (1, 4, 32):
            sizes = [kvq.kv_beam_workspace_size(n, b, v, 8) for n in range(1, 600)]
            assert sizes == sorted(sizes)


def test_fork_and_copy_refusals(kvq):
    def forked(n=2, page=16, stride=4, pages=8, parents=D, copies=D, ws=D, ws_bytes=1 << 20):
        return kvq.lib().kv_pages_fork(n, page, parents, D, D, stride, D, D, pages, copies, ws, ws_bytes, None)
    assert forked(n=4097) == 5 and forked(n=-1) == 1 and forked(page=3) == 5 and forked(n=4096, stride=1 << 20) == 5
    assert forked(parents=None) == 1 and forked(copies=None) == 1 and forked(ws=None) == 3 and forked(ws_bytes=256) == 3
    assert forked(n=0) == 0
    assert kvq.kv_pages_fork_workspace_size(4097, 1, 1) == 0

    class PoolEntry(C.Structure):
        _fields_ = [("data", C.c_void_p), ("page_bytes", C.c_int64)]
    pool = (PoolEntry * 1)(PoolEntry(None, 64))
    copy = kvq.lib().kv_pages_copy
    assert copy(1, D, 4, 1, C.byref(pool), None, None) == 1
    pool[0] = PoolEntry(4096, -1)
    assert copy(1, D, 4, 1, C.byref(pool), None, None) == 1
    assert copy(-1, D, 4, 1, C.byref(pool), None, None) == 1 and copy(1, None, 4, 1, C.byref(pool), None, None) == 1
    assert copy(0, D, 4, 1, C.byref(pool), None, None) == 0


def test_wide_heads_turn_128_dims_at_most(kvq):
    rope = kvq.rope_layout([1.0] * 64)
    assert append(kvq, rope, dim=256, n=0) == 0
    rope.dim = 130
    assert append(kvq, rope, dim=256, n=0) == 5
    with pytest.raises(ValueError):
        kvq.rope_layout([1.0] * 65)
