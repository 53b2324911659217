"""Grouped-query attention over value rows of zeros and of extreme sizes, rows that are no numbers,
and weights that a later row dwarfs."""
import math

import pytest
import torch

from gpu_common import kvq_module
from gqa_common import Pool, attention, close
from test_gpu_gqa import attend, check, queries

pytestmark = pytest.mark.gpu

DT = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def kvq():
    return kvq_module()


def place(pool, b, t):
    """(pages, places) of rows t of sequence b."""
    t = torch.as_tensor(t, device="cuda")
    return pool.table[b].long()[t // pool.page], t % pool.page


def blank(pool, b, t, heads=slice(None)):
    """Rows t of sequence b as kv_gqa_append stores values of zero."""
    pg, at = place(pool, b, t)
    v, s = pool.v[pg, :, at], pool.scales[pg, :, at]   # [rows][heads][..]
    v[:, heads] = 0
    s[:, heads, 1] = 0.0
    pool.v[pg, :, at], pool.scales[pg, :, at] = v, s


# So many sequences over the same pages that a CTA takes several steps of each.
MANY = 300


def shared(pool):
    """The table and lengths of MANY sequences with the pages of sequence 0."""
    pool.table = pool.table[:1].expand(MANY, pool.width).contiguous()
    return [int(pool.lens[0])] * MANY


def check_shared(out, q, pool, new, sm, causal, what=""):
    """As check, for sequences that share their rows: token i of all of them at once."""
    n, ref = int(pool.lens[0]), {}
    wide = q.dtype == torch.bfloat16 and new * (q.shape[1] // pool.heads) > 24
    for absolute in (False, True)[:1 + wide]:
        r = ref[absolute] = torch.empty(q.shape, dtype=torch.float64, device="cuda")
        for i in range(new):
            rows = n - new + 1 + i if causal else n
            r[i::new] = attention(q[i::new], pool, [rows], [len(q) // new], sm, False, absolute)
    close(out, ref[False], what, ref.get(True))


# a sequence's new tokens, and the vectors of a tile: 8, 16, 128
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim,heads,kv", [(64, 8, 2), (128, 8, 2), (256, 4, 1)])
@pytest.mark.parametrize("new", [1, 4, 20])
def test_zero_values_in_front(kvq, dtype, causal, dim, heads, kv, new):
    for front in (15, 16, 64, 200):
        pool = Pool(kv, dim, 16, [330], seed=front)
        blank(pool, 0, range(front))
        lens, news = shared(pool), [new] * MANY
        q = queries(new * MANY, heads, dim, dtype)
        out, ws = attend(kvq, pool, q, lens, news, causal)
        check_shared(out, q, pool, new, 1 / math.sqrt(dim), causal, f"{front} rows")
        assert kvq.read_device_error(ws) == 0


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("run", [16, 64, 256])
def test_zero_values_where_a_share_of_the_rows_begins(kvq, dtype, odd, run):
    """Long sequences are cut among the CTAs at multiples of 64 rows: every other run is zero."""
    lens = [30000, 9001]
    for dim in (64, 128, 256):
        pool = Pool(2, dim, 64, lens, seed=run)
        for b, n in enumerate(lens):
            t = torch.arange(n)
            blank(pool, b, t[t // run % 2 == odd], heads=slice(0, 1))
        for causal, new in ((True, [1, 1]), (True, [3, 4]), (False, [2, 1])):
            q = queries(sum(new), 8, dim, dtype)
            out, _ = attend(kvq, pool, q, lens, new, causal)
            check(out, q, pool, lens, new, 1 / math.sqrt(dim), causal, f"dim {dim} {new}")


def test_appended_zero_values(kvq):
    """As an encoder's padding gets there: rows of zero values through the append, then decode steps and cross attention."""
    n, kv, dim = 200, 2, 128
    for front in (16, 64):
        pool = Pool(kv, dim, 16, [n], seed=3)
        pool.k.zero_(), pool.v.zero_(), pool.scales.zero_()
        k, v = queries(n, kv, dim, torch.bfloat16, seed=4), queries(n, kv, dim, torch.bfloat16, seed=5)
        v[:front] = 0
        pg, at = place(pool, 0, range(n))
        kvq.kv_gqa_append(None, k, v, None, pg * pool.page + at, None, None, pool.k, pool.v, pool.scales)
        assert bool((pool.scales[pg[:front], :, at[:front], 1] == 0).all())
        lens, q = shared(pool), queries(2 * MANY, 8, dim, torch.bfloat16)
        for causal in (True, False):
            out, _ = attend(kvq, pool, q, lens, [2] * MANY, causal)
            check_shared(out, q, pool, 2, 1 / math.sqrt(dim), causal, f"{front} causal={causal}")


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("gain", [1e-25, 1e-10, 1e10, 1e25])
def test_sizes_of_values(kvq, dtype, gain):
    for new in ([1, 2], [70, 30]):
        lens = [500, 333]
        pool = Pool(2, 128, 32, lens, seed=7)
        pool.scales[..., 1] *= gain
        q = queries(sum(new), 8, 128, dtype)
        out, _ = attend(kvq, pool, q, lens, new)
        check(out, q, pool, lens, new, 1 / math.sqrt(128), True, f"{new}")


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("new", [1, 3, 20])
@pytest.mark.parametrize("small", [0.0, 1e-25])
def test_large_values_of_no_weight_behind_small_ones(kvq, dtype, new, small):
    """The last rows' values are 1e13, at scores so low that their weights vanish from f32."""
    n, dim = 640, 128
    pool = Pool(1, dim, 64, [n], seed=11)
    q = torch.ones(new, 4, dim, device="cuda").to(dtype)
    pool.k[:] = 0x38   # 1.0
    pool.scales[..., 0] = 1e-3
    pg, at = place(pool, 0, range(512, 640))
    pool.scales[pg, :, at, 0] = -4.0   # scores of -512
    pool.scales[pg, :, at, 1] = 1e13 / 448
    pg, at = place(pool, 0, range(64 if small == 0.0 else 512))
    pool.scales[pg, :, at, 1] *= small
    lens, news = shared(pool), [new] * MANY
    q = q.repeat(MANY, 1, 1)
    out, _ = attend(kvq, pool, q, lens, news, causal=False, sm=1.0)
    check_shared(out, q, pool, new, 1.0, False)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [6, 70])
def test_every_dim_of_a_token_that_sees_no_number(kvq, dtype, causal, dim, new):
    """A key's NaN code or either scale that is no finite number makes every dim NaN, whatever the sign of the product;
    a value's NaN code its own dim; tokens that don't see the row are as without it."""
    lens, news, sm = [330 + new, 150], [new, 20 if new > 6 else 2], 0.1
    row = 330 + new // 2
    for bad in ("k", "v", "sk", "sv"):
        for x in (math.nan, math.inf, -math.inf) if bad in ("sk", "sv") else (None,):
            pool, clean = Pool(2, dim, 16, lens, seed=9), Pool(2, dim, 16, lens, seed=9)
            q = queries(sum(news), 8, dim, dtype)
            pg, at = place(pool, 0, [row])
            pg1 = int(pool.table[1, 150 // 16])   # behind sequence 1's end
            for p_, a in ((int(pg), slice(int(at), int(at) + 1)), (pg1, slice(150 % 16, 16))):
                if x is None:
                    (pool.k if bad == "k" else pool.v)[p_, :, a, 5] = 0x7f
                else:
                    pool.scales[p_, :, a, 0 if bad == "sk" else 1] = x
            out, ws = attend(kvq, pool, q, lens, news, causal, sm=sm)
            sees = [i for i in range(new) if not causal or 330 + i >= row]
            rest = [i for i in range(len(q)) if i not in sees]
            hit = torch.isnan(out[sees])
            assert bool(hit[..., 5].all() if bad == "v" else hit.all()), (bad, x)
            ref = attention(q, clean, lens, news, sm, causal)
            wide = dtype == torch.bfloat16 and new > 6
            mass = attention(q, clean, lens, news, sm, causal, absolute=True)[rest] if wide else None
            close(out[rest], ref[rest], f"{bad} {x}", mass)
            assert kvq.read_device_error(ws) == 0


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("ahead", [20.0, 24.5, 25.5, 30.0])
def test_weights_of_a_step_whose_last_row_dwarfs_them(kvq, dtype, dim, ahead):
    """Rows 128 .. 223 score some binades above the first 128, the next row `ahead` binades: 448 as the values' second
    dim of the 96 makes their share of the output visible."""
    one, most = 0x38, 0x7e   # 1.0, 448
    pool = Pool(1, dim, 64, [256])
    pool.k[:], pool.v[:] = 0, 0
    pool.k[..., 0] = one
    pool.v[..., 0] = one
    pool.scales[..., 0], pool.scales[..., 1] = 0.0, 1.0
    pg, at = place(pool, 0, range(128, 224))
    pool.scales[pg, :, at, 0] = 2.5 if dtype == torch.bfloat16 else 3.5
    v = pool.v[pg, :, at]
    v[..., 1] = most
    pool.v[pg, :, at] = v
    pg, at = place(pool, 0, [224])
    pool.scales[pg, :, at, 0] = ahead
    q = torch.zeros(2, 64, dim, device="cuda", dtype=dtype)
    q[..., 0] = 1.0
    sm = float(torch.tensor(math.log(2.0)))   # scores are binades
    out, _ = attend(kvq, pool, q, [256], [2], causal=False, sm=sm)
    check(out, q, pool, [256], [2], sm, False)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("gain", [1e10, 1e18, 1e25])
def test_large_values_behind_zero_ones(kvq, dtype, dim, gain):
    """The rows of zero values count in the softmax's sum, whatever the size of the values behind them."""
    for new, n in ((1, 330), (20, 330), (20, 2600)):
        for front in (16, 32, 128, n - 70):
            pool = Pool(1, dim, 64, [n], seed=front)
            pool.scales[..., 1] *= gain
            blank(pool, 0, range(front))
            lens, news = shared(pool), [new] * MANY
            q = queries(new * MANY, 4, dim, dtype)
            out, _ = attend(kvq, pool, q, lens, news, causal=False)
            check_shared(out, q, pool, new, 1 / math.sqrt(dim), False, f"{front} of {n} rows, {new} tokens")


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 40])
def test_queries_that_are_no_numbers(kvq, dtype, dim, new):
    """Every dim of their outputs is NaN, on one row too, whose score may be -inf; zeros where no row is seen."""
    lens, news = [1, 3, 0, 200], [new] * 4
    pool = Pool(2, dim, 16, lens, seed=1)
    q = queries(4 * new, 8, dim, dtype)
    ref = attention(q, pool, lens, news, 0.1, False)
    mass = attention(q, pool, lens, news, 0.1, False, absolute=True) if new * 4 > 24 and dtype == torch.bfloat16 else None
    q[:, 1, 5], q[:, 2, 5], q[:, 6, 40] = math.inf, -math.inf, math.nan
    out, _ = attend(kvq, pool, q, lens, news, False, sm=0.1)
    rest = [0, 3, 4, 5, 7]
    some = torch.tensor([n > 0 for n in lens for _ in range(new)], device="cuda")
    assert bool(torch.isnan(out[some][:, [1, 2, 6]]).all()) and bool((out[~some] == 0).all())
    close(out[:, rest], ref[:, rest], "the other heads", None if mass is None else mass[:, rest])
