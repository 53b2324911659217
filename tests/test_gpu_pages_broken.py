"""A block table with an entry that is no page: a trim that would give it back is refused."""
import numpy as np
import pytest
import torch

from gpu_common import to_dev
from test_gpu_paged import Pages, kvq  # noqa: F401

pytestmark = pytest.mark.gpu


def trim(p, keep):
    p.kvq.kv_pages_trim(p.d_lens, to_dev(np.array(keep, np.int64)), p.d_table, p.d_free, p.d_n, p.page, p.ws)


@pytest.mark.parametrize("n_seq", [2, 300, 1500, 9000])       # one CTA and several
@pytest.mark.parametrize("bad", [-1, "n_pages", 2 ** 31 - 1])
def test_trim_refuses_a_page_that_is_none(kvq, n_seq, bad):  # noqa: F811
    rng = np.random.default_rng(n_seq)
    lens = rng.integers(1, 70, n_seq).tolist()
    p = Pages(kvq, lens, 16, 8, sum(-(-n // 16) for n in lens) + 3 * n_seq)
    broken = n_seq // 2
    kept = int(p.d_table[broken, 0].item())
    p.d_table[broken, 0] = p.n_pages if bad == "n_pages" else bad
    trim(p, [0] * n_seq)
    assert kvq.read_device_error(p.ws) == 1
    p.d_table[broken, 0] = kept
    p.check()                                                 # nothing has moved
    p.d_table[broken, 0] = p.n_pages if bad == "n_pages" else bad
    keep = [0] * n_seq                                        # the others can go without it
    keep[broken] = -1
    trim(p, keep)
    p.model_trim(keep)
    assert kvq.read_device_error(p.ws) == 0
    p.d_table[broken, 0] = kept
    p.check()
    add = [40] * n_seq                                        # every page handed out is one
    add[broken] = 0
    _, _, slots, _ = p.reserve(add)
    assert slots.tolist() == p.model_reserve(add)[0]
    assert kvq.read_device_error(p.ws) == 0
    p.check()


def test_trim_keeps_a_broken_entry_that_stays(kvq):  # noqa: F811
    p = Pages(kvq, [100, 40], 16, 8, 20)
    p.d_table[0, 1] = -5                                      # row 16 .. 31: kept
    trim(p, [40, 0])
    p.model_trim([40, 0])
    assert kvq.read_device_error(p.ws) == 0 and p.d_lens.tolist() == [40, 0]
    n = int(p.d_n.item())
    assert n == len(p.stack) and p.d_free.cpu().numpy()[:n].tolist() == p.stack
    assert torch.equal(p.ws[4:8], torch.zeros_like(p.ws[4:8]))
