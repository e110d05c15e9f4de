"""Of several causes in the status word the one that says most about the results is reported: a paged-cache call
whose data was out of bounds has defined results, one that timed out has none."""
import pytest
import torch

import attention_tensor_cores_gb300 as F
from test_gpu_page_table import Step
from test_gpu_paged import Problem

pytestmark = pytest.mark.gpu


def late(call):
    """The call with a wait limit of one cycle."""
    F.fmha_set_wait_limit(1)
    try:
        call()
    finally:
        F.fmha_set_wait_limit(0)


def short_of_pages():
    """A page table step that finds no free page."""
    s = Step([16], [1], [[0, -1]], [1, 2, 3], 0, 1)
    s.call(16)


@pytest.mark.parametrize("split", [True, False])
def test_timeout_outlasts_a_bad_length_of_the_same_call(split):
    p = Problem([900, 64, 333], 8, 8, 1, 64, 16, seed=8)
    p.seqlens[1] = 1 << 20
    assert F.fmha_check_status() == 0
    late(lambda: p.run(split=split))
    assert F.fmha_check_status() == F.FMHA_ERR_TIMEOUT
    assert F.fmha_check_status() == 0
    p.run(split=split)
    assert F.fmha_check_status() == F.FMHA_ERR_PAGES


def test_timeout_outlasts_a_step_without_pages():
    p = Problem([900, 64, 333], 8, 8, 1, 64, 16, seed=8)
    late(p.run)
    short_of_pages()
    assert F.fmha_check_status() == F.FMHA_ERR_TIMEOUT
    short_of_pages()
    late(p.run)
    assert F.fmha_check_status() == F.FMHA_ERR_TIMEOUT
    short_of_pages()
    p.run()
    assert F.fmha_check_status() == F.FMHA_ERR_PAGES
    assert F.fmha_check_status() == 0
