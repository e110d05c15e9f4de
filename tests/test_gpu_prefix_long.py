"""Long sums over common keys (fmha_fwd_prefix): a piece of more key tiles than one accumulator takes.

The tensor core cuts off what has no bits in its sum: with C products added up, each less than a step of 2^-23 of what is there, C 2^-23
of sum p |v| in all.  An accumulator takes 64 tiles of 16 products, 2^-13, the bound that check_attention has for sums over keys; what
is merged adds a few 2^-23 a time.
"""
import pytest
import torch

import attention_tensor_cores_gb300 as F
from paged_util import check_attention
from test_gpu_prefix import call
from test_gpu_prefix_common import many

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq, members", [(16, 9), (16, 8), (1, 9)])     # two row tiles; one, on both sides
@pytest.mark.parametrize("tiles", [1024, 2500])
def test_constant_values(tiles, members, Hq, D):
    """Values of 1 add up to 1, whatever their weights.  More groups than SMs, in the same pages, so that a piece is as long as a prefix."""
    groups, P = 320, 128
    B, keys = groups * members, tiles * 128
    k = torch.empty(tiles + 1, 1, P, D, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(tiles))
    gr = type("Case", (), dict(k=k, v=torch.ones_like(k)))
    gr.table = torch.arange(tiles + 1, device="cuda").int().repeat(B, 1)     # all requests' last keys, too
    gr.table[torch.arange(B, device="cuda") % members > 0, :tiles] = -1
    gr.seqlens = torch.full((B,), keys + 7, dtype=torch.int32, device="cuda")
    gr.cu = torch.arange(0, B + 1, members, device="cuda").int()
    gr.prefix_lens = torch.full((groups,), keys, dtype=torch.int32, device="cuda")
    q = torch.empty(B, Hq, 1, D, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    out, lse = call(q, gr, kind=F.FMHA_OUT_F32)
    assert F.fmha_check_status() == F.FMHA_OK
    # the accumulator's 2^-13, two BF16 for a weight 2^-16, and 2^-24 for each of an accumulator's 64 tiles' weights, of the 32 sums
    # in a tile, and four times for each of up to 40 parts: together below 2^-16
    off = float((out - 1).abs().max())
    assert off <= 2.0 ** -13 + 2.0 ** -16 + 2.0 ** -16, off
    b = B // 2
    x = torch.einsum("hd,nd->hn", q[b, :, 0].double(), k[:, 0].reshape(-1, D)[:keys + 7].double()) * D ** -0.5
    assert (torch.logsumexp(x, -1) - lse[b, :, 0]).abs().max() <= 2.0 ** -12 + 2.0 ** -20 * float(lse[b].abs().max())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tiles, groups, Hq, members", [
    (65, 320, 16, 9),      # two row tiles: a tile more than an accumulator takes
    (64, 320, 16, 9),
    (129, 200, 16, 8),     # one row tile: a part with an odd number of key tiles
    (257, 200, 1, 9),
    (200, 170, 16, 9),     # four parts
    (400, 170, 2, 9)])
def test_parts(tiles, groups, Hq, members, D):
    """Parts of a piece are merged; requests that end in an earlier part, and empty slots, keep what they have."""
    gr, q, ref = many([members] * groups, [tiles] * groups, D, Hq, 1, seed=tiles, P=128, short=groups * members // 5)
    out, lse = call(q, gr, kind=F.FMHA_OUT_F32)
    assert F.fmha_check_status() == F.FMHA_OK
    check_attention(out, lse, ref, bf16=False)
    again, lse2 = call(q, gr, kind=F.FMHA_OUT_F32)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("D", [64, 128])
def test_causal_parts(D):
    """Proposed tokens, some of which end in an earlier part, against one token at a time."""
    Sq, members, groups, tiles, P = 4, 9, 170, 140, 128
    gr, q, ref = many([members] * groups, [tiles] * groups, D, 4, 1, seed=3, P=P, short=300)
    gr.table = gr.full     # shorter requests share a tile less
    # token i of request b alone is a request of lens[b] - Sq + 1 + i keys
    qs = torch.empty(q.shape[0], 4, Sq, D, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(5))
    qs[:, :, -1:] = q
    out, lse = call(qs, gr, kind=F.FMHA_OUT_F32, causal=True)
    assert F.fmha_check_status() == F.FMHA_OK
    check_attention(out[:, :, -1:], lse[:, :, -1:], ref, bf16=False)
    keep = gr.seqlens.clone()
    for i in range(Sq - 1):
        gr.seqlens = (keep - Sq + 1 + i).clamp(min=0)
        one, one_lse = call(qs[:, :, i:i + 1].contiguous(), gr, kind=F.FMHA_OUT_F32)
        assert F.fmha_check_status() == F.FMHA_OK
        none = one_lse == -torch.inf
        assert torch.equal(none, lse[:, :, i:i + 1] == -torch.inf)
        # both within check_attention's bound of the same number; sum p |v| <= max |v|
        bound = 2 * float(gr.v.abs().max()) * (2.0 ** -12 + 2.0 ** -13 + 2.0 ** -16)
        assert (out[:, :, i:i + 1] - one).abs().max() <= bound
        assert (lse[:, :, i:i + 1] - one_lse)[~none].abs().max() <= 2 * (2.0 ** -12 + 2.0 ** -20 * 64)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("where", [3, 100, 199])     # tiles in the first, second and last part
def test_nan_in_a_part(where, D):
    """A NaN key makes the rows that see it NaN in whatever part it is; requests that end before it are as they were."""
    gr, q, ref = many([9] * 170, [200] * 170, D, 16, 1, seed=where, P=128, short=300)
    first = next(b for b in gr.cu.tolist()[5:] if gr.seqlens[b] > 0)
    gr.k[int(gr.table[first, where]), :, 5] = float("nan")
    out, lse = call(q, gr, kind=F.FMHA_OUT_F32)
    assert F.fmha_check_status() == F.FMHA_OK
    bad = torch.zeros(q.shape[:3], dtype=torch.bool)
    bad[first:first + 9] = (gr.seqlens[first:first + 9].cpu() > where * 128 + 5)[:, None, None]
    assert bad.any() and torch.equal(lse.isnan().cpu(), bad) and torch.equal(out.isnan().all(-1).cpu(), bad)
    fine = ~bad[:, 0, 0]
    check_attention(out.cpu()[fine], lse.cpu()[fine], tuple(x[fine] for x in ref), bf16=False)


@pytest.mark.parametrize("D", [64, 128])
def test_forced_timeout_in_parts(D):
    """With a wait limit of one cycle the kernel drains and reports, whatever part it is in; the next call is right."""
    gr, q, ref = many([9] * 170, [200] * 170, D, 16, 1, seed=11, P=128, short=300)
    assert F.fmha_check_status() == F.FMHA_OK
    F.fmha_set_wait_limit(1)
    try:
        call(q, gr)
        rc = F.fmha_check_status()
    finally:
        F.fmha_set_wait_limit(0)
    assert rc == F.FMHA_ERR_TIMEOUT
    out, lse = call(q, gr)
    assert F.fmha_check_status() == F.FMHA_OK
    check_attention(out, lse, ref)
