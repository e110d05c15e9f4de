"""fmha_rope_append where a token or a head lies 2^31 elements behind the first (outputs of 4.3 GB)."""
import pytest
import torch

import attention_tensor_cores_gb300 as F
from paged_util import make_pools

pytestmark = pytest.mark.gpu

D, FAR = 128, (1 << 31) // 128


def test_many_tokens_of_one_sequence():
    """q_out [1, 1, Sq, D]: tokens on either side of element 2^31, all others padding."""
    T = FAR + 72
    x = torch.randn(1, 1, D, device="cuda").to(torch.bfloat16)
    rows = x.expand(T, 1, D)                       # every token the same row: a token stride of 0
    real = [0, 5, FAR - 1, FAR, FAR + 1, T - 1]
    slots = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    slots[real] = torch.arange(len(real), device="cuda")
    kp, vp = make_pools(1, 1, 16, D, "hnd", fill=-3.0)
    out = torch.full((1, 1, T, D), -3.0, dtype=torch.bfloat16, device="cuda")
    F.fmha_rope_append(rows, rows, rows, None, None, 0.0, None, None, slots, out, F.make_kv_cache(kp, vp))
    assert F.fmha_check_status() == 0
    written = (out[0, 0, :, 0] != -3).nonzero()[:, 0].tolist()
    assert written == real
    assert (out[0, 0, real] == x[0]).all()
    for pool in (kp, vp):
        assert (pool[0, 0, :len(real)] == x[0]).all() and (pool[0, 0, len(real):] == -3).all()


def test_many_heads_of_one_token():
    """q [1, Hq, D]: heads on either side of element 2^31."""
    Hq = FAR + 6
    q = torch.empty(1, Hq, D, dtype=torch.bfloat16, device="cuda").normal_()
    k = torch.randn(1, 1, D, device="cuda").to(torch.bfloat16)
    kp, vp = make_pools(1, 1, 16, D, "hnd", fill=-3.0)
    out = torch.full((1, Hq, D), -3.0, dtype=torch.bfloat16, device="cuda")
    F.fmha_rope_append(q, k, k, None, None, 0.0, None, None, torch.zeros(1, dtype=torch.int64, device="cuda"), out,
                       F.make_kv_cache(kp, vp))
    assert F.fmha_check_status() == 0
    assert torch.equal(out, q)
