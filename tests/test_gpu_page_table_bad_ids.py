"""Block tables with ids that are not pages of the pool: what a step and the attention do with them."""
import numpy as np
import pytest
import torch

import attention_tensor_cores_gb300 as F
from paged_util import check_attention
from test_gpu_page_table import Step
from test_gpu_paged import Problem

pytestmark = pytest.mark.gpu


def test_bad_ids_of_a_finished_request_go_on_the_stack_and_are_reported():
    """As the steps say: pushed with the others, handed on, and a token on such a page has no slot."""
    table = np.array([[5, 99, -4], [0, 0, 0], [0, 0, 0]], np.int32)
    s = Step([40, 0, 0], [-1, 0, 0], table, np.array([1, 2, 3, 0, 0, 0, 0, 0]), 3, 0)
    s.call(16)
    assert F.fmha_check_status() == F.FMHA_ERR_PAGES
    assert s.free.tolist()[:6] == [1, 2, 3, 5, 99, -4] and int(s.n_out) == 6 and s.seqlens.tolist() == [0, 0, 0]
    t = Step([0, 0, 0], [0, 20, 17], s.table.cpu().numpy(), s.free.cpu().numpy(), 6, 40)
    t.call(16)
    assert F.fmha_check_status() == F.FMHA_ERR_PAGES
    assert t.table.tolist()[1][:2] == [-4, 99] and t.table.tolist()[2][:2] == [5, 3] and int(t.n_out) == 2
    assert t.slots.tolist() == [-1] * 20 + list(range(80, 96)) + [48] + [-1] * 3
    assert t.positions.tolist() == list(range(20)) + list(range(17)) + [0] * 3
    assert F.fmha_check_status() == 0


@pytest.mark.parametrize("layout", ["hnd", "nhd", "kv"])
@pytest.mark.parametrize("D, P", [(64, 16), (128, 16), (128, 64), (128, 24)])
@pytest.mark.parametrize("Hq, Hkv", [(4, 2), (16, 1)])
def test_attention_over_bad_pages(layout, D, P, Hq, Hkv):
    """Pages out of the pool read as zero rows, just behind it and far away."""
    for bad in (None, -1, -(1 << 31), (1 << 31) - 1):
        p = Problem([4 * P, 3 * P + 1, 200], Hq, Hkv, 1, D, P, layout, seed=D + P, extra=0)
        pages = p.pools[0].shape[0]
        for b, i in ((0, 1), (1, 0), (1, 3)):
            p.table[b, i] = pages if bad is None else bad
            p.k[b, :, i * P:(i + 1) * P] = p.v[b, :, i * P:(i + 1) * P] = 0
        ref = p.ref()
        for split in (True, False):
            out, lse = p.run(split=split)
            assert F.fmha_check_status() == F.FMHA_ERR_PAGES
            check_attention(out, lse, ref)


@pytest.mark.parametrize("layout", ["hnd", "nhd", "kv"])
@pytest.mark.parametrize("D", [64, 128])
def test_a_pool_of_one_page(layout, D):
    p = Problem([30], 4, 2, 1, D, 32, layout, seed=1, spare=0)
    assert p.pools[0].shape[0] == 1
    out, lse = p.run()
    assert F.fmha_check_status() == 0
    check_attention(out, lse, p.ref())
    p.table[0, 0] = 1
    p.k[:], p.v[:] = 0, 0
    out, lse = p.run()
    assert F.fmha_check_status() == F.FMHA_ERR_PAGES
    check_attention(out, lse, p.ref())
