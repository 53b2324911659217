"""The chained launches of the paged calls behind something that is no kernel, behind several streams, and across the
contiguous calls: eager and captured."""
import math

import numpy as np
import pytest
import torch

from gpu_common import to_dev
from quantized_kv_cache_kv8_gb300 import synth
from test_gpu_paged import SM, Paged, freqs, kvq, query  # noqa: F401

pytestmark = pytest.mark.gpu


class Step:
    """A step's rotary append and attention over a pool, its inputs refilled before every run by copies."""

    def __init__(self, kvq, oracle, fmt, past, new, H=16, page=16, seed=6):
        self.kvq, self.fmt = kvq, fmt
        self.p = Paged(kvq, oracle, fmt, past, new, page, seed)
        n = sum(new)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.rope = kvq.rope_layout(freqs(64))
        self.src = torch.randn(n, H, 576, generator=g, device="cuda").bfloat16()
        self.x = torch.randn(n, 576, generator=g, device="cuda").bfloat16()
        self.pos = torch.arange(n, device="cuda") * 7
        slots = []
        for s, (a, m) in enumerate(zip(past, new)):
            slots += [int(self.p.table[s, t // page]) * page + t % page for t in range(a, a + m)]
        self.slots = torch.tensor(slots, device="cuda")
        self.q, self.out = torch.zeros_like(self.src), torch.zeros(n, H, 512, dtype=torch.bfloat16, device="cuda")
        self.cu, self.table, self.lens = to_dev(self.p.cu), to_dev(self.p.table), to_dev(self.p.lens)
        self.page = page
        self.ws = torch.zeros(kvq.kv_attn_paged_workspace_size(fmt, len(new), H, n, self.p.layout), dtype=torch.uint8,
                              device="cuda")

    def append(self):
        self.kvq.kv_rope_append(self.fmt, self.rope, self.x, self.pos, self.slots, self.q[..., 512:], self.q[..., 512:],
                                self.p.codes, self.p.scales, self.p.layout)

    def attend(self):
        self.kvq.kv_attn_paged(self.fmt, self.q, self.cu, self.p.codes, self.p.scales, self.table, self.lens, self.page,
                               self.out, self.ws, SM, self.p.layout)

    def waited(self):
        torch.cuda.synchronize()
        self.q.copy_(self.src)
        torch.cuda.synchronize()
        self.append()
        torch.cuda.synchronize()
        self.attend()
        torch.cuda.synchronize()
        return self.out.clone()


def after_copy(s, side):
    s.out.zero_()               # a memset and a copy of bytes, no kernels
    s.q.copy_(s.src)
    s.append()
    s.out.zero_()
    s.attend()


def after_two_streams(s, side):
    main = torch.cuda.current_stream()
    side.wait_stream(main)
    with torch.cuda.stream(side):
        s.q.copy_(s.src)
    s.out.zero_()
    main.wait_stream(side)
    s.append()
    side.wait_stream(main)
    main.wait_stream(side)
    s.attend()


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("run", [after_copy, after_two_streams])
def test_paged_calls_behind_other_work(kvq, oracle, fmt, run):  # noqa: F811
    s = Step(kvq, oracle, fmt, [40, 0, 300], [1, 5, 2])
    want = s.waited()
    side = torch.cuda.Stream()
    for _ in range(3):
        s.out.fill_(7.0)
        run(s, side)
        torch.cuda.synchronize()
        assert torch.equal(s.out, want)
    graph = torch.cuda.CUDAGraph()
    main = torch.cuda.Stream()
    main.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=main):
        run(s, side)
    for _ in range(3):
        s.out.fill_(7.0)
        s.q.fill_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(s.out, want)
    assert kvq.read_device_error(s.ws) == 0


@pytest.mark.parametrize("fmt", [1, 2])
def test_paged_calls_between_contiguous_ones(kvq, oracle, fmt):  # noqa: F811
    """The contiguous decode's merge and the paged kernels are both launched early: each sees what was before it."""
    s = Step(kvq, oracle, fmt, [40, 0, 300], [1, 5, 2])
    want = s.waited()
    T, H = 5000, 128
    x = to_dev(synth.mla_rows(3, T))
    codes = torch.zeros(T, kvq.row_bytes(fmt, s.p.layout), dtype=torch.uint8, device="cuda")
    scales = torch.zeros(T, 2, device="cuda")
    (kvq.kv8_encode if fmt == 1 else kvq.tq4_encode)(x, codes, scales, s.p.layout)
    q = query(1, H, 3, True)
    cu = to_dev(np.array([0, T]))
    ws = torch.zeros(kvq.kv_attn_workspace_size(fmt, 1, H, T, s.p.layout), dtype=torch.uint8, device="cuda")
    ref, out = torch.zeros(1, H, 512, device="cuda"), torch.zeros(1, H, 512, device="cuda")

    def decode(o):
        kvq.kv_attn_decode(fmt, q, codes, scales, cu, o, ws, T, 1 / math.sqrt(192.0), s.p.layout)

    decode(ref)
    torch.cuda.synchronize()
    for _ in range(5):
        s.out.fill_(7.0)
        out.fill_(7.0)
        s.q.copy_(s.src)
        decode(out)
        s.append()
        decode(out)
        s.attend()
        decode(out)
        torch.cuda.synchronize()
        assert torch.equal(s.out, want) and torch.equal(out, ref)
