"""fmha_rope_append on more heads than fill the GPU, where a group of threads takes up to four heads of a token."""
import pytest
import torch

import attention_tensor_cores_gb300 as F
from paged_util import make_pools, up
from test_gpu_rope_append import EPS, case, near, ref_heads, table_of

pytestmark = pytest.mark.gpu


def tokens(Hq, Hkv, D, Sq=1):
    """The fewest tokens, a multiple of Sq, whose heads of one group each would be more than 2048 threads per SM; a few on top."""
    T = up(2048 * F.fmha_num_sms() // ((Hq + 2 * Hkv) * (D // 16)) + 5, Sq) * Sq
    assert T * (Hq + 2 * Hkv) * (D // 16) > 2048 * F.fmha_num_sms()
    return T


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("Hq, Hkv, P, layout, Sq, split, norm, R", [
    (7, 1, 16, "hnd", 1, False, True, 64),       # three heads in the last query set, one key head
    (10, 5, 24, "nhd", 3, True, True, 48),       # sets of four, four and two, and of four and one
    (32, 8, 64, "kv", 4, False, False, 32),
    (5, 5, 5, "hnd", 2, True, True, 16),
    (1, 1, 1, "nhd", 1, False, True, 0)])
def test_up_to_four_heads_a_group(D, pairs, Hq, Hkv, P, layout, Sq, split, norm, R):
    T = tokens(Hq, Hkv, D, Sq)
    pad = [0, 1, T // 3, T // 2, T - 1] if Sq == 1 else [Sq, T // 2]
    case(T, Hq, Hkv, D, R * D // 64, pairs, norm, norm, P, layout, Sq, pad=pad, seed=T, split=split)


@pytest.mark.parametrize("D, pairs", [(64, True), (128, False)])
def test_out_of_bounds_tokens_are_left_out(D, pairs):
    Hq, Hkv, P = 7, 1, 16
    T = tokens(Hq, Hkv, D)
    pages = up(T, P) + 1
    g = torch.Generator().manual_seed(D)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(torch.bfloat16)
    d = qkv.cuda()
    slots, pos = torch.randperm(pages * P, generator=g)[:T], torch.randint(0, 500, (T,), generator=g).int()
    out_of = {0: (pages * P, 0), 77: (1 << 40, 0), T // 2: (None, 500), T - 2: (None, -1), T - 1: (-1, 9)}
    for t, (slot, p) in out_of.items():
        slots[t], pos[t] = slots[t] if slot is None else slot, p
    left_out = torch.zeros(T, dtype=torch.bool)
    left_out[list(out_of)] = True
    kp, vp = make_pools(pages, Hkv, P, D, "nhd", fill=-3.0)
    out = torch.full((T, Hq, D), -3.0, dtype=torch.bfloat16, device="cuda")
    table = table_of(500, D)
    F.fmha_rope_append(d[:, :Hq], d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:], None, None, EPS, table.cuda(), pos.cuda(), slots.cuda(), out,
                       F.make_kv_cache(kp, vp), interleaved=pairs)
    assert F.fmha_check_status() == F.FMHA_ERR_PAGES
    assert (out[left_out.cuda()] == -3).all()
    real, st = ~left_out, slots[~left_out].cuda()
    yq, size = ref_heads(qkv[real, :Hq], None, table, pos[real], pairs)
    near(out[real.cuda()], yq, size, "q")
    yk, size = ref_heads(qkv[real, Hq:Hq + Hkv], None, table, pos[real], pairs)
    near(kp[st // P, :, st % P], yk, size, "k")
    assert torch.equal(vp[st // P, :, st % P].cpu(), qkv[real, Hq + Hkv:])
    rest = torch.ones(pages * P, dtype=torch.bool)
    rest[slots[real]] = False
    u = rest.nonzero()[:, 0].cuda()
    assert (kp[u // P, :, u % P] == -3).all() and (vp[u // P, :, u % P] == -3).all()
