"""Grouped-query attention over value rows of extreme sizes."""
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


# So many sequences over the same pages that a CTA takes several steps of each.
MANY = 300


def shared(pool):
    """The table and lengths of MANY sequences with the pages of sequence 0."""
    pool.table = pool.table[:1].expand(MANY, pool.width).contiguous()
    return [int(pool.lens[0])] * MANY


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
@pytest.mark.parametrize("small", [1e-25])
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
    check(out, q, pool, lens, news, 1.0, False)
