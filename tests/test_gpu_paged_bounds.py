"""Paged attention where its rounding could show: 2e-3 of exact attention before the
rounding to bf16, whatever the rows and scores."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

from gpu_common import SIMT_TOL, TENSOR_TOL, to_dev
from quantized_kv_cache_kv8_gb300 import synth
from test_gpu_paged import BF16_STEP, SM, Paged, kvq, query  # noqa: F401

pytestmark = pytest.mark.gpu


def copies(kvq, oracle, fmt, x, seed, order, page=64):
    """A pool whose rows are copies of the rows x: row t is x[order[t]].  Returns (layout, codes, scales, block table,
    reconstructed rows)."""
    layout = kvq.mla_layout(seed=seed)
    codes = torch.empty(len(x), kvq.row_bytes(fmt, layout), dtype=torch.uint8, device="cuda")
    scales = torch.empty(len(x), 2, device="cuda")
    (kvq.kv8_encode if fmt == 1 else kvq.tq4_encode)(to_dev(x), codes, scales, layout)
    xh = np.asarray(oracle.reconstruct(fmt, codes.cpu().numpy(), scales.cpu().numpy(), seed=seed), np.float64)
    pages = -(-len(order) // page)
    rows = torch.zeros(pages * page, dtype=torch.int64, device="cuda")
    rows[:len(order)] = to_dev(np.asarray(order, np.int64))
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None].contiguous()
    return layout, codes[rows].contiguous(), scales[rows].contiguous(), table, xh


def attend(kvq, fmt, q, layout, codes, scales, table, n_rows, page=64):
    n, H = q.shape[:2]
    out = torch.full((n, H, 512), float("nan"), dtype=q.dtype, device="cuda")
    size = kvq.kv_attn_paged_workspace_size(fmt, 1, H, n, layout, bf16=q.dtype == torch.bfloat16)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    kvq.kv_attn_paged(fmt, q, to_dev(np.array([0, n])), codes, scales, table, to_dev(np.array([n_rows])), page, out, ws, SM,
                      layout)
    assert kvq.read_device_error(ws) == 0
    return out.double().cpu().numpy()


def row_weights(out, xh):
    """The weight of row 0 in outputs that mix two rows, by projection, over the exact weight's output."""
    d = xh[0, :512] - xh[1, :512]
    return (out - xh[1, :512]) @ d / (d @ d), d


@pytest.mark.parametrize("fmt", [1, 2])
def test_query_keeps_its_bits(kvq, oracle, fmt):  # noqa: F811
    """Queries for which two rows score alike: the weight of row 0 is near 1/2 and moves by a quarter of what a score is
    off.  Outputs within 2e-3 of the largest put the projected weight off by at most 2e-3 max|out| |d|_1 / |d|_2^2; their
    rounding to bf16, 512 independent errors, each uniform up to 2^-8 of the value, adds 8 sigma (once in 10^15)."""
    H, T, seed = 256, 256, 12
    x = synth.mla_rows(seed, 2)
    layout, codes, scales, table, xh = copies(kvq, oracle, fmt, x, seed, np.arange(T) % 2)
    full = xh[0] - xh[1]
    q = torch.randn(H, 576, generator=torch.Generator().manual_seed(seed)).double().numpy() * 6.0
    q -= np.outer(q @ full, full) / (full @ full)
    q = torch.from_numpy(q).bfloat16()
    out = attend(kvq, fmt, q[None].cuda(), layout, codes, scales, table, T)[0]
    got, d = row_weights(out, xh)
    z = q.double().numpy() @ xh.T * SM
    want = 1.0 / (1.0 + np.exp(z[:, 1] - z[:, 0]))
    ref = want[:, None] * xh[0, :512] + (1.0 - want)[:, None] * xh[1, :512]
    allowed = TENSOR_TOL * np.abs(ref).max(1) * np.abs(d).sum() / (d @ d)
    allowed += 8 * BF16_STEP / math.sqrt(3.0) * np.sqrt(((ref * d) ** 2).sum(1)) / (d @ d)
    ratio = np.abs(got - want) / allowed
    assert ratio.max() <= 1.0, (int(ratio.argmax()), float(ratio.max()))


ORDERS = {"falling": lambda order, rng: order, "rising": lambda order, rng: order[::-1], "mixed": lambda order, rng: rng.permutation(order)}


def kinds_of(kvq, oracle, fmt, binades, counts, order, H, seed):  # noqa: F811
    """Rows of a few kinds, each with dims of its own, so that an output shows what the kind weighs, and queries for which
    their scores lie `binades` apart, times 0.9 to 1.1."""
    rng = np.random.default_rng(seed)
    kinds = len(binades)
    x = 0.3 * rng.standard_normal((kinds, 576)).astype(np.float32)
    for k in range(kinds):
        x[k, 64 * (k + 1):64 * (k + 2)] += 2.0
    kind = ORDERS[order](np.repeat(np.arange(kinds), counts), rng)
    layout, codes, scales, table, xh = copies(kvq, oracle, fmt, x, seed, kind)
    q = rng.standard_normal((H, 576))
    goal = np.outer(np.linspace(0.9, 1.1, H), np.array(binades) * math.log(2.0) / SM)
    steps = xh[1:] - xh[0]
    q += np.linalg.solve(steps @ steps.T, (goal[:, 1:] - goal[:, :1] - q @ steps.T).T).T @ steps
    return layout, codes, scales, table, xh, kind, q


def check_kinds(kvq, oracle, fmt, binades, counts, order):  # noqa: F811
    """80 tiles of 128 heads: a walker has nearly all rows of a tile.  Outputs within 2e-3 of the largest, their rounding to
    bf16 (2^-8 of the value) aside."""
    H, n, seed = 128, 80, 3
    kinds = len(binades)
    layout, codes, scales, table, xh, kind, q = kinds_of(kvq, oracle, fmt, binades, counts, order, H, seed)
    T = len(kind)
    q = torch.from_numpy(q).bfloat16()
    out = attend(kvq, fmt, q.expand(n, H, 576).contiguous().cuda(), layout, codes, scales, table, T)
    z = q.double().numpy() @ xh.T * SM
    w = np.exp(z - z.max(1, keepdims=True))
    worst = 0.0
    seen = np.stack([np.cumsum(kind == k) for k in range(kinds)])       # of each kind up to row t
    for i in range(n):
        m = w * seen[:, T - n + i]
        ref = (m / m.sum(1, keepdims=True)) @ xh[:, :512]
        top = TENSOR_TOL * np.abs(ref).max(1, keepdims=True)
        worst = max(worst, float((np.abs(out[i] - ref) / (top + BF16_STEP * (np.abs(ref) + top))).max()))
    assert worst <= 1.0, worst


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("binades,counts,order", [
    ([0, -20.5], [1, 131071], "falling"), ([0, -9, -18], [1, 700, 130000], "falling"), ([0, 0], [1 << 16, 1 << 16], "mixed"),
    ([0, -17], [33, 131039], "mixed"), ([0, 0], [5, (1 << 20) - 5], "mixed"),
])
def test_exact_path_keeps_its_bound(kvq, oracle, fmt, binades, counts, order):  # noqa: F811
    """The same on the exact path with f32 queries: 1e-5 of the largest output, with rows whose roundings all point one
    way."""
    H, n, seed = 32, 6, 3
    layout, codes, scales, table, xh, kind, q = kinds_of(kvq, oracle, fmt, binades, counts, order, H, seed)
    T = len(kind)
    q = torch.from_numpy(q).float()
    out = attend(kvq, fmt, q.expand(n, H, 576).contiguous().cuda(), layout, codes, scales, table, T)
    z = q.double().numpy() @ xh.T * SM
    w = np.exp(z - z.max(1, keepdims=True))
    for i in range(n):
        m = w * np.bincount(kind[:T - n + i + 1], minlength=len(binades))
        ref = (m / m.sum(1, keepdims=True)) @ xh[:, :512]
        e = np.abs(out[i] - ref).max(1) / np.abs(ref).max(1)
        assert e.max() <= SIMT_TOL, (i, int(e.argmax()), float(e.max()))


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("counts", [[1 << 19, 1 << 19], [5, (1 << 20) - 5]])
def test_long_sums(kvq, oracle, fmt, counts):  # noqa: F811
    """A million rows by one walker: what 65,536 products add to one accumulator."""
    check_kinds(kvq, oracle, fmt, [0, 0], counts, "mixed")


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("binades,counts,order", [
    ([0, -20.5], [1, 131071], "falling"), ([0, -20.5], [1, 131071], "mixed"), ([0, -17], [33, 131039], "mixed"),
    ([0, -9, -18], [1, 700, 130000], "falling"), ([0, -9, -18], [1, 700, 130000], "rising"),
    ([0, -9, -18], [1, 700, 130000], "mixed"), ([0, -14, -28], [1, 3, 90000], "falling"), ([0, -60], [1, 70000], "falling"),
])
def test_many_small_weights_add_up(kvq, oracle, fmt, binades, counts, order):  # noqa: F811
    """One kind outweighs another by many binades, but for the number of its rows."""
    check_kinds(kvq, oracle, fmt, binades, counts, order)


@pytest.mark.parametrize("fmt", [1, 2])
def test_long_walks_over_different_rows(kvq, oracle, fmt):  # noqa: F811
    """70,000 rows and 80 tiles, so that walkers fold their sums twice and their references move in between; some of the
    vectors against f64."""
    T, n, H = 70000, 80, 128
    p = Paged(kvq, oracle, fmt, [T - n], [n], 64, seed=9)
    q = query(n, H, 9, True)
    out = p.run(q, 0)
    assert p.err == 0
    rows = torch.from_numpy(p.xh[0]).cuda()
    rng = np.random.default_rng(1)
    for i in np.concatenate([[0, n - 1], rng.integers(0, n, 30)]):
        heads = torch.from_numpy(rng.integers(0, H, 16)).cuda()
        K = rows[:T - n + int(i) + 1]
        ref = torch.softmax(q[int(i), heads].double() @ K.T * SM, -1) @ K[:, :512]
        top = TENSOR_TOL * ref.abs().amax(1, keepdim=True)
        ratio = (out[int(i), heads].double() - ref).abs() / (top + BF16_STEP * (ref.abs() + top))
        assert float(ratio.max()) <= 1.0, (int(i), float(ratio.max()))


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("path,bf16", [(1, False), (1, True), (2, True)])
def test_tables_without_entries(kvq, fmt, path, bf16):  # noqa: F811
    """A pool that no table can list anything of, its addresses null: nothing is read, every token yields zeros."""
    layout, H, n = kvq.mla_layout(), 4, 3
    dtype = torch.bfloat16 if bf16 else torch.float32
    q, out = torch.ones(n, H, 576, dtype=dtype, device="cuda"), torch.full((n, H, 512), 7.0, dtype=dtype, device="cuda")
    cu, lens = to_dev(np.array([0, 1, 3])), torch.zeros(2, dtype=torch.int64, device="cuda")
    size = kvq.kv_attn_paged_workspace_size(fmt, 2, H, n, layout, bf16, path)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    status = kvq.lib().kv_attn_paged(fmt, C.byref(layout), q.data_ptr(), int(bf16), n, H, 2, cu.data_ptr(), None, None, None, 0,
                                     lens.data_ptr(), 16, 5, SM, out.data_ptr(), ws.data_ptr(), size, path, None)
    torch.cuda.synchronize()
    assert status == 0 and kvq.read_device_error(ws) == 0 and bool((out == 0).all())
