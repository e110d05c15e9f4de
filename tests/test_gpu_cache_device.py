"""The device of a cache's pools goes along with its descriptor: calls with tensors of another device are refused."""
import pytest
import torch

import attention_tensor_cores_gb300 as F
from test_gpu_paged import Problem

pytestmark = pytest.mark.gpu


def calls(p):
    out = torch.empty_like(p.qd)
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(2, device="cuda")
    return (lambda: F.fmha_fwd_paged(p.qd, p.cache, p.table, p.seqlens, out, None, 0.1),
            lambda: F.fmha_rope_append(x, x, x, None, None, 0.0, None, None, slots, torch.empty_like(x), p.cache))


def test_pools_of_another_device_are_refused():
    p = Problem([20], 4, 2, 1, 64, 16)
    assert p.cache.device == torch.cuda.current_device()
    for other in (p.cache.device + 1, -1, "cuda"):
        p.cache.device = other
        for call in calls(p):
            with pytest.raises(F.FmhaError, match="device") as e:
                call()
            assert e.value.code == F.FMHA_ERR_INVALID
    p.cache.device = torch.cuda.current_device()
    for call in calls(p):
        call()
    assert F.fmha_check_status() == 0


def test_a_descriptor_filled_by_hand():
    p = Problem([20], 4, 2, 1, 64, 16)
    c = F.fmha_kv_cache()
    for name, _ in c._fields_:
        setattr(c, name, getattr(p.cache, name))
    assert c.device is None
    p.cache, keep = c, p.cache
    for call in calls(p):
        call()
    assert F.fmha_check_status() == 0 and keep.pools
