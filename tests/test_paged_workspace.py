"""CPU check of the paged attention's workspace: the work split has its place in it wherever a kernel is to read it."""
import pytest

import attention_tensor_cores_gb300 as F
from attention_tensor_cores_gb300 import build as B
from test_paged_refusals import A, cache, opts

# requests whose split the kernel finds itself, and SMs whose partials of one unit it merges itself
INLINE_REQUESTS, MERGE_SMS = 512, 160


@pytest.fixture(scope="module")
def lib():
    B.build()
    return F.load()


@pytest.mark.parametrize("batch", [1, 7, 512, 513, 3000])
@pytest.mark.parametrize("given_scale", [False, True])
def test_the_split_has_a_place_where_it_is_read(lib, batch, given_scale):
    """The combine kernel, which runs for a given NVFP4 scale and on more SMs than the attention merges for, takes
    the split from the workspace, and so does the attention of very large batches."""
    c, Hq, D = cache(D=64), 4, 64
    sms = lib.fmha_num_sms() or 256       # without a device sized for the most SMs there might be
    up = lambda n: -(-n // 256) * 256   # noqa: E731
    units = batch * c.Hkv
    partials = units + sms
    split = batch > INLINE_REQUESTS or given_scale or sms > MERGE_SMS
    want = (up((batch + 2) * 4) if split else 0) + up(units * 8) + up(partials * 16 * 4) + up(partials * 16 * D * 4)
    o = opts(out_kind=F.FMHA_OUT_NVFP4, nvfp4_scale_in=A) if given_scale else opts()
    assert lib.fmha_paged_workspace_size(batch, Hq, 1, c, o) == want
