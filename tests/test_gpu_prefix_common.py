"""Common keys of many shapes really read once (fmha_fwd_prefix): what the other rows of a group have in place of them are ids
outside the pool, so a call that reads through those rows is wrong and reports it.

Tolerances are check_attention's (test_gpu_prefix.py says why they hold for this operator).
"""
import math

import pytest
import torch

import attention_tensor_cores_gb300 as F
from paged_util import attention_ref, check_attention
from shared_util import Groups
from test_gpu_prefix import call

pytestmark = pytest.mark.gpu


def reach(gr, g):
    """Keys of group g's whole tiles that its first request reaches."""
    first = sum(gr.members[:g])
    return min(gr.prefix[g], gr.lens[first]) // 128 * 128 if gr.members[g] else 0


def blind(gr):
    """Ids outside the pool in the rows behind each group's first one, where its tiles are read for all."""
    at = 0
    for g, m in enumerate(gr.members):
        gr.table[at + 1:at + m, :reach(gr, g) // gr.P] = -1
        at += m


def queries(gr, Hq, Sq, D, seed=5):
    return torch.randn(len(gr.lens), Hq, Sq, D, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def run(lens, prefix, P=16, Hq=8, Hkv=2, Sq=1, D=64, layout="hnd", causal=False, seed=1):
    gr = Groups(lens, prefix, P, Hkv, D, layout, seed)
    blind(gr)
    q = queries(gr, Hq, Sq, D)
    out, lse = call(q.cuda(), gr, causal=causal)
    assert F.fmha_check_status() == F.FMHA_OK
    check_attention(out, lse, attention_ref(q, *gr.dense, gr.lens, D ** -0.5, causal), what=f"{lens} {prefix}")


# ------------------------------------------------------------------------------------------------
# more groups than threads
# ------------------------------------------------------------------------------------------------
def device_ref(q, k, v, table, lens, P, scale):
    """attention_ref on the GPU for one token a request, a run of requests at a time."""
    outs, run = [], max(1, (1 << 19) // max(lens))
    for b0 in range(0, len(lens), run):
        n = lens[b0:b0 + run]
        at = torch.arange(max(max(n), 1), device="cuda")
        page = table[b0:b0 + run, at // P].long().clamp(min=0)
        see = at < torch.tensor(n, device="cuda")[:, None]
        kk, vv = (torch.where(see[:, :, None, None], pool[page, :, at % P], 0.0).double() for pool in (k, v))       # [b][key][Hkv][D]
        b, Hq, _, D = q[b0:b0 + run].shape
        x = torch.einsum("bhgd,bnhd->bhgn", q[b0:b0 + run].double().reshape(b, kk.shape[2], -1, D), kk) * scale
        x = torch.where(see[:, None, None], x, -math.inf)
        l = torch.logsumexp(x, -1, keepdim=True)
        p = torch.where(see[:, None, None], torch.exp(x - torch.where(l == -math.inf, 0.0, l)), 0.0)
        o, a = (torch.einsum("bhgn,bnhd->bhgd", p, y) for y in (vv, vv.abs()))
        outs.append([y.reshape(b, Hq, 1, -1).cpu() for y in (o, l, a)])
    o, l, a = (torch.cat(x) for x in zip(*outs))
    return o, l.squeeze(-1), a


def many(members, tiles, D, Hq, Hkv, seed, P=16, short=0):
    """Requests of len(members) groups behind tiles[g] tiles each, one in fifty an empty slot and `short` of them ended inside: tables and
    pools on the device, the queries, and the reference."""
    rng = torch.Generator().manual_seed(seed)
    N, B = len(members), sum(members)
    of = torch.arange(N).repeat_interleave(torch.tensor(members))
    t = torch.tensor(tiles)
    common = t * (128 // P)                                                    # pages
    lens = t[of] * 128 + torch.randint(1, 30, (B,), generator=rng)
    lens[torch.randint(0, B, (B // 50,), generator=rng)] = 0                   # empty slots, first ones of groups among them
    cu = torch.tensor([0] + members).cumsum(0)
    head = cu[:-1][of]                                                         # each request's group's first one
    for b in torch.randint(0, B, (short,), generator=rng).tolist():
        if b != head[b]:
            lens[b] = int(torch.randint(0, int(t[of[b]]) * 128, (), generator=rng))
    first = torch.cumsum(common, 0) - common
    total = int(common.sum()) + 2 * B
    ids = torch.randperm(total, generator=rng)
    width = max(int(common.max()) + 3, -(-((6000 // (B * Hkv) + 1) * 128) // P))
    col = torch.arange(width)[None]
    mine = int(common.sum()) + 2 * torch.arange(B)[:, None] + col - common[of][:, None]
    place = torch.where(col < common[of][:, None], first[of][:, None] + col, mine)
    held = col < (lens[:, None] + P - 1) // P
    table = torch.where(held, ids[place.clamp(0, total - 1)], -1).int().cuda()
    dev = torch.Generator("cuda").manual_seed(seed)
    k, v = (torch.empty(total, Hkv, P, D, dtype=torch.bfloat16, device="cuda").normal_(generator=dev) for _ in range(2))
    q = torch.empty(B, Hq, 1, D, dtype=torch.bfloat16, device="cuda").normal_(generator=dev)
    ref = device_ref(q, k, v, table, lens.tolist(), P, D ** -0.5)
    apart = (torch.arange(B) != head) & (lens[head] > 0)                       # read through another row
    full = table.clone()
    table[(apart[:, None] & (col < common[of][:, None])).cuda()] = -1
    gr = type("Case", (), dict(k=k, v=v, table=table, full=full, seqlens=lens.int().cuda(), cu=cu.int().cuda(), prefix_lens=(t * 128).int().cuda()))
    return gr, q, ref


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N, members, tiles", [
    (385, (8,), (5,)),                      # one more than threads
    (400, (8, 9), (16,)),                   # 16 rows a request: a row tile, and two
    (1000, (8, 0, 20, 1, 9), (5, 7, 6)),    # groups without requests, and of one
    (8192, (2,), (10,))])                   # as many as there may be
def test_more_groups_than_threads(N, members, tiles, D):
    if N == 8192 and D == 128:
        tiles = (11,)
    Hq, Hkv = (1, 1) if N == 8192 else (16, 1) if members == (8, 9) else (2, 1)
    gr, q, ref = many([members[g % len(members)] for g in range(N)], [tiles[g % len(tiles)] for g in range(N)], D, Hq, Hkv, seed=N)
    if 1 in members:     # a request alone reads its own keys, which nobody else has
        assert (gr.cu[1:] - gr.cu[:-1] == 1).any()
    out, lse = call(q, gr)
    assert F.fmha_check_status() == F.FMHA_OK
    check_attention(out, lse, ref)
    again, lse2 = call(q, gr)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


# ------------------------------------------------------------------------------------------------
# rows and lengths
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens, prefix", [
    ([[700, 2000, 1900, 1999, 650, 1700, 1800, 1601, 1600]], [1600]),         # the first request ends inside the prefix
    ([[641, 641, 640, 639, 2000, 2000, 1, 0, 129]], [1600]),                  # others too
    ([[1280, 1279, 1281, 1300, 1, 127, 128, 0, 1290]], [1280]),               # the first one at its end
    ([[128 * 9 + 127] * 9], [128 * 10]),                                      # all in the prefix's last tile
    ([[2000] * 20, [], [1500] * 9, [3], [1900, 1000] * 6], [1920, 640, 1280, 0, 1600])])
def test_requests_that_end_inside(lens, prefix, D):
    run(lens, prefix, D=D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq, Hkv, Sq", [(4, 2, 16), (2, 1, 32), (4, 1, 16), (1, 1, 64), (8, 2, 5)])
def test_causal_rows_that_end_inside(Hq, Hkv, Sq, D):
    p = 2560 if D == 64 else 1920
    run([[p, p + 1, p + 3, p + 60, 3, Sq, 0, p - 1, p - 128, p + Sq - 1, p - Sq, p // 2, p + 130]], [p], Hq=Hq, Hkv=Hkv, Sq=Sq, D=D, causal=True)


@pytest.mark.parametrize("P, layout", [(8, "nhd"), (24, "kv"), (64, "kv"), (128, "nhd"), (1000, "hnd")])
@pytest.mark.parametrize("D", [64, 128])
def test_pages(P, layout, D):
    p = 2000 // P * P
    run([[p + 37, p + 1, p + 300, p, p + 9, p + 5, p + 4, p + 3, p + 2]], [p], P=P, layout=layout, D=D)


@pytest.mark.parametrize("D", [64, 128])
def test_far_pages(D):
    """Pages past 2^31 elements of the pool."""
    gr = Groups([[1300 + i for i in range(12)], [40]], [1280, 0], 16, 1, D)
    pages, big = gr.k.shape[0], torch.zeros((1 << 32) + (1 << 20), dtype=torch.bfloat16, device="cuda")
    step = (1 << 32) // pages // (8 * D) * (8 * D)
    k, v = (big.as_strided(gr.k.shape, (step, 16 * D, D, 1), o) for o in (0, 16 * D))
    k.copy_(gr.k)
    v.copy_(gr.v)
    gr.k, gr.v = k, v
    assert int(gr.table[0, :80].max()) * step > 1 << 31
    blind(gr)
    q = queries(gr, 4, 1, D)
    out, lse = call(q.cuda(), gr)
    assert F.fmha_check_status() == 0
    check_attention(out, lse, attention_ref(q, *gr.dense, gr.lens, D ** -0.5, False))


# ------------------------------------------------------------------------------------------------
# what is wrong with the data
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("members", [9, 40])
def test_common_pages_outside_the_pool(members, D):
    """They read as zero keys and values, for all requests, and are reported."""
    gr = Groups([[1300 + i for i in range(members)], [50]], [1280, 0], 16, 2, D)
    blind(gr)
    for j, page in ((0, -1), (13, 1 << 30), (79, gr.k.shape[0])):
        gr.table[0, j] = page
        for dense in gr.dense:
            dense[:members, :, j * 16:j * 16 + 16] = 0
    q = queries(gr, 8, 1, D)
    ref = attention_ref(q, *gr.dense, gr.lens, D ** -0.5, False)
    out, lse = call(q.cuda(), gr)
    assert F.fmha_check_status() == F.FMHA_ERR_PAGES
    check_attention(out, lse, ref)
    assert F.fmha_check_status() == F.FMHA_OK


def test_lists_that_are_none_and_lengths_out_of_bounds():
    gr = Groups([[1300 + i for i in range(9)], [700, 60]], [1280, 48], 16, 2, 64)
    q = queries(gr, 8, 1, 64)
    ref = attention_ref(q, *gr.dense, gr.lens, 0.125, False)
    good, table = gr.cu.clone(), gr.table.clone()
    for cu in ([1, 9, 11], [0, 12, 11], [0, 9, 10], [0, -1, 11], [0, 9, 12], [0, 1 << 30, 11]):     # nothing is shared
        gr.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        out, lse = call(q.cuda(), gr)
        assert F.fmha_check_status() == F.FMHA_ERR_PAGES
        check_attention(out, lse, ref, what=str(cu))
    gr.cu = good
    blind(gr)
    # a prefix that passes the first request's tokens reaches as far as its whole tiles do: 1280 keys here
    gr.prefix_lens = torch.tensor([1 << 30, -5], dtype=torch.int32, device="cuda")
    out, lse = call(q.cuda(), gr)
    assert F.fmha_check_status() == F.FMHA_OK
    check_attention(out, lse, ref)
    # a negative length is 0: of another request; of the first one, which leaves nothing to be shared
    for b in (4, 0):
        gr.table = table.clone()
        if b:
            blind(gr)
        keep = gr.seqlens.clone()
        gr.seqlens[b] = -7
        out, lse = call(q.cuda(), gr)
        assert F.fmha_check_status() == F.FMHA_ERR_PAGES
        assert (out[b] == 0).all() and (lse[b] == -math.inf).all()
        pick = torch.tensor([i for i in range(11) if i != b])
        check_attention(out.cpu()[pick], lse.cpu()[pick], tuple(x[pick] for x in ref))
        gr.seqlens = keep


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("key", [0, 200, 1279, 1285])     # in the first and in other common tiles, and behind them
@pytest.mark.parametrize("members", [9, 40])              # one row tile and two
def test_infinite_scores(members, key, D):
    """A score of +infinity makes its row and LSE NaN, one of -infinity weighs nothing; the other rows are as they were."""
    gr = Groups([[1300 + i for i in range(members)], [300]], [1280, 0], 16, 2, D)
    blind(gr)
    q = queries(gr, 8, 1, D)
    q[..., 0] = 0
    gr.k[..., 0] = 0     # the one key alone has a first feature
    gr.dense[0][..., 0] = 0
    up, down = (1, 2), (members - 1, 5)
    big = torch.finfo(torch.bfloat16).max
    q[up][0, 0], q[down][0, 0] = big, -big
    rows = range(members) if key < 1280 else [up[0], down[0]]
    for b in rows:
        page = int(gr.table[0 if key < 1280 else b, key // 16])
        gr.k[page, :, key % 16, 0] = big
        gr.dense[0][b, :, key, 0] = big
    ref = [x.clone() for x in attention_ref(q, *gr.dense, gr.lens, D ** -0.5, False)]
    # of the row of -infinity: the attention without that key
    b, h = down
    keep = torch.tensor([j for j in range(gr.lens[b]) if j != key])
    one = attention_ref(q[b:b + 1, h:h + 1], *(x[b:b + 1, h // 4:h // 4 + 1][:, :, keep] for x in gr.dense), [len(keep)], D ** -0.5, False)
    for x, y in zip(ref, one):
        x[b, h] = y[0, 0]
    out, lse = call(q.cuda(), gr)
    assert F.fmha_check_status() == F.FMHA_OK
    bad = torch.zeros(len(gr.lens), 8, 1, dtype=torch.bool)
    bad[up] = True
    assert torch.equal(out.isnan().all(-1).cpu(), bad) and torch.equal(lse.isnan().cpu(), bad)
    fine = ~bad[..., 0]
    check_attention(out.cpu()[fine], lse.cpu()[fine], tuple(x[fine] for x in ref))


# ------------------------------------------------------------------------------------------------
# the call
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("D", [64, 128])
def test_other_stream_and_no_lse(D):
    gr = Groups([[1300 + i for i in range(9)], [50]], [1280, 0], 16, 2, D)
    blind(gr)
    q = queries(gr, 8, 1, D)
    ref = attention_ref(q, *gr.dense, gr.lens, D ** -0.5, False)
    q = q.cuda()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    out, lse = call(q, gr, stream=stream)
    stream.synchronize()
    assert F.fmha_check_status(stream) == F.FMHA_OK
    check_attention(out, lse, ref)
    cache = F.make_kv_cache(gr.k, gr.v)
    ws = torch.full((F.fmha_prefix_workspace_size(*q.shape[:3], cache, F.make_opts()),), 0xff, dtype=torch.uint8, device="cuda")
    # without an LSE, into an output that is only 16-byte aligned
    wide = torch.zeros(out.numel() + 4, device="cuda")[4:].view(out.shape)
    F.fmha_fwd_prefix(q, cache, gr.table, gr.seqlens, gr.cu, gr.prefix_lens, wide, None, D ** -0.5, F.make_opts(out_kind=F.FMHA_OUT_F32, workspace=ws))
    assert F.fmha_check_status() == F.FMHA_OK
    check_attention(wide, None, ref, bf16=False)


@pytest.mark.parametrize("groups, members", [(300, 9), (40, 100), (1, 8192)])
def test_large_batches(groups, members):
    gr, q, ref = many([members] * groups, [8] * groups, 64, 2, 1, seed=groups)
    out, lse = call(q, gr, kind=F.FMHA_OUT_F32)
    assert F.fmha_check_status() == F.FMHA_OK
    check_attention(out, lse, ref, bf16=False)
