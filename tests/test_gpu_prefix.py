"""Attention of groups of requests that share their first pages (fmha_fwd_prefix) against the 64-bit statement.

Tolerances are check_attention's: the kernel rounds each weight to two BF16 (2^-17) and the output once, and sums in FP32
over tiles of 128 keys, as the paged attention does; merging partials adds a few 2^-23 of them.
"""
import math

import pytest
import torch

import attention_tensor_cores_gb300 as F
from paged_util import attention_ref, check_attention
from shared_util import Groups

pytestmark = pytest.mark.gpu


def call(q, gr, cache=None, causal=False, scale=None, kind=F.FMHA_OUT_BF16, fill=None, **kw):
    B, Hq, Sq, D = q.shape
    cache = cache or F.make_kv_cache(gr.k, gr.v)
    need = F.fmha_prefix_workspace_size(B, Hq, Sq, cache, F.make_opts(out_kind=kind, causal=causal))
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")       # NaN wherever a partial is not written
    out = torch.full(q.shape, float("nan"), dtype=torch.float32 if kind == F.FMHA_OUT_F32 else torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    F.fmha_fwd_prefix(q, cache, gr.table, gr.seqlens, gr.cu, gr.prefix_lens, out, lse, scale or D ** -0.5,
                      F.make_opts(out_kind=kind, workspace=ws, causal=causal), **kw)
    return out, lse


def run(lens, prefix, P=16, Hq=8, Hkv=2, Sq=1, D=64, layout="hnd", causal=False, kind=F.FMHA_OUT_BF16, seed=1, scale=1.0, wide=True):
    gr = Groups(lens, prefix, P, Hkv, D, layout, seed, scale, wide=wide)
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn(len(gr.lens), Hq, Sq, D, generator=g).to(torch.bfloat16)
    out, lse = call(q.cuda(), gr, causal=causal, kind=kind)
    assert F.fmha_check_status() == F.FMHA_OK
    ref = attention_ref(q, *gr.dense, gr.lens, D ** -0.5, causal)
    check_attention(out, lse, ref, bf16=kind == F.FMHA_OUT_BF16, what=f"{lens} {prefix}")
    return gr, q, out, lse


@pytest.mark.parametrize("wide", [True, False])
def test_one_group(wide):
    before = F.fmha_launch_count()
    run([[600, 590]], [512], D=128, wide=wide)
    assert F.fmha_launch_count() - before == (2 if wide else 1)    # few tiles: the paged attention


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens, prefix", [
    ([[1]], [0]), ([[128]], [0]), ([[129]], [128]), ([[500]], [0]),                      # a request alone
    ([[513, 700, 900, 514]], [512]), ([[512, 512]], [512]), ([[640, 641]], [528]),       # all, none or a part of a tile behind the prefix
    ([[2000, 0, 300, 100]], [1600]), ([[0, 2000, 1900]], [1600]), ([[90, 2000, 1900]], [1600]),   # empty slots, requests that end inside
    ([[0, 0, 0]], [0]), ([[0], [0, 0], [5]], [0, 0, 0]),
    ([[1300] * 3, [], [700, 701], [40], [2100] * 5], [1024, 0, 688, 0, 2096])])
def test_lengths(lens, prefix, D):
    run(lens, prefix, D=D)


@pytest.mark.parametrize("Hq, Hkv, Sq", [(1, 1, 1), (2, 2, 1), (8, 1, 1), (16, 1, 1), (7, 1, 1), (6, 2, 2), (14, 2, 3), (4, 1, 4), (8, 8, 4),
                                         (32, 1, 2), (64, 1, 1), (16, 1, 4), (33, 1, 2), (65, 1, 1), (128, 1, 1), (40, 1, 4), (64, 1, 5)])
@pytest.mark.parametrize("causal", [False, True])
def test_heads_and_rows(Hq, Hkv, Sq, causal):
    run([[1300, 1200, 1157, 1280, 1153], [400, 390]], [1152, 384], Hq=Hq, Hkv=Hkv, Sq=Sq, causal=causal, D=64 if Hq % 2 else 128)


@pytest.mark.parametrize("Sq", [2, 4, 16])
def test_causal_rows_that_end_inside_the_prefix(Sq):
    # the first request reaches to the prefix's end, so its earlier queries do not see all of it; a request shorter than Sq
    # has queries that see nothing
    run([[640, 641, 643, 700, 3, Sq, 0, 512, 513]], [640], Hq=4, Hkv=2, Sq=Sq, causal=True, D=64)


@pytest.mark.parametrize("P", [8, 24, 40, 48, 64, 128, 256, 1000])
@pytest.mark.parametrize("layout", ["hnd", "nhd", "kv"])
def test_pages(P, layout):
    p = 1000 // P * P
    run([[p + 37, p + 1, p + 500], [p + 2, p]], [p, p], P=P, layout=layout, D=128 if P in (24, 64, 1000) else 64)


@pytest.mark.parametrize("members", [2, 31, 32, 33, 64, 100])
def test_many_requests(members):
    run([[700 + 3 * i for i in range(members)]], [640], Hq=8, Hkv=2)


@pytest.mark.parametrize("B", [383, 384, 385, 1000])
def test_many_groups(B):
    # more entries than threads: runs of them per thread
    groups = [[140 + i % 7, 150, 141][:1 + i % 3] for i in range(B // 2)]
    run(groups, [128] * len(groups), Hq=2, Hkv=1)
    run([[n] for n in range(B)], [0] * B, Hq=2, Hkv=1)


def test_long_prefix_over_every_sm():
    run([[20000 + i for i in range(8)]], [19968], Hq=4, Hkv=1, D=128)


@pytest.mark.parametrize("scale", [0.1, 8.0])
def test_reference_moves(scale):
    # large scores: the running maximum moves, and partials of very different weights meet
    run([[1500, 1400, 1300]], [1280], scale=scale)


@pytest.mark.parametrize("kind", [F.FMHA_OUT_F32])
def test_fp32_output(kind):
    run([[700, 800, 650], [50], [0]], [640, 0, 0], kind=kind, D=128)


def test_same_as_paged_attention():
    gr, q, out, lse = run([[3000 + 11 * i for i in range(16)], [77], [400, 500]], [2992, 0, 400], Hq=32, Hkv=8, D=128)
    cache = F.make_kv_cache(gr.k, gr.v)
    ws = torch.empty(F.fmha_paged_workspace_size(len(gr.lens), 32, 1, cache, F.make_opts()), dtype=torch.uint8, device="cuda")
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    F.fmha_fwd_paged(q.cuda(), cache, gr.table, gr.seqlens, o2, l2, 128 ** -0.5, F.make_opts(workspace=ws))
    # each within FP32 roundings of the same number: a step of BF16 apart at most (2^-7 of the value) where they round apart
    assert ((out.float() - o2.float()).abs() <= 2.0 ** -7 * o2.float().abs() + 2.0 ** -12).all()
    assert (lse - l2).abs().max() <= 2.0 ** -12


@pytest.mark.parametrize("single", [False, True])
def test_nvfp4(single):
    import oracle
    import numpy as np
    gr = Groups([[700, 800, 650], [50], [0]], [640, 0, 0], 16, 2, 128)
    q = torch.randn(5, 8, 1, 128, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    cache = F.make_kv_cache(gr.k, gr.v)
    n = q.numel()
    codes, scales = torch.zeros(n // 2, dtype=torch.uint8, device="cuda"), torch.zeros(n // 16, dtype=torch.uint8, device="cuda")
    ts, amax, o32 = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda"), torch.zeros(n, device="cuda")
    given = torch.tensor([2.5e-4], device="cuda") if single else None
    lse = torch.zeros(5, 8, 1, device="cuda")

    def opts(**kw):
        return F.make_opts(F.FMHA_OUT_NVFP4, out_scales=scales, out_tensor_scale=ts, nvfp4_scale_in=given, out_amax=amax, **kw)
    for stage in (o32, None):
        need = F.fmha_prefix_workspace_size(5, 8, 1, cache, opts(out_f32=stage))
        ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
        F.fmha_fwd_prefix(q.cuda(), cache, gr.table, gr.seqlens, gr.cu, gr.prefix_lens, codes, lse, 128 ** -0.5, opts(out_f32=stage, workspace=ws))
        assert F.fmha_check_status() == F.FMHA_OK
        ref = attention_ref(q, *gr.dense, gr.lens, 128 ** -0.5, False)
        check_attention(o32.view(q.shape), lse, ref, bf16=False)
        o = o32.cpu().numpy()
        if single:
            c, s = oracle.nvfp4_quantize_scaled(o, float(given))[:2]
        else:
            c, s, _ = oracle.nvfp4_quantize(o)
        assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s[:n // 16])
        assert float(amax) == np.abs(o).max()


def test_bad_lists_lengths_and_pages():
    lens, prefix = [[700, 800, 650], [50, 60]], [640, 48]
    gr = Groups(lens, prefix, 16, 2, 64)
    q = torch.randn(5, 8, 1, 64, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    ref = attention_ref(q, *gr.dense, gr.lens, 0.125, False)
    good = gr.cu.clone()
    # no list of groups: everything is computed without sharing, and reported
    for cu in ([1, 3, 5], [0, 6, 5], [0, 3, 4], [0, -1, 5], [0, 3, 6], [0, 1 << 30, 5]):
        gr.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        out, lse = call(q.cuda(), gr)
        assert F.fmha_check_status() == F.FMHA_ERR_PAGES
        check_attention(out, lse, ref, what=str(cu))
    gr.cu = good
    # a prefix below 0 is none; one behind the first request's tokens reaches as far as they do
    gr.prefix_lens = torch.tensor([-5, 1 << 30], dtype=torch.int32, device="cuda")
    gr2 = Groups([[700, 800, 650], [48, 48]], [640, 48], 16, 2, 64)
    gr2.prefix_lens = gr.prefix_lens
    out, lse = call(q.cuda(), gr2)
    assert F.fmha_check_status() == F.FMHA_OK
    check_attention(out, lse, attention_ref(q, *gr2.dense, gr2.lens, 0.125, False))
    # lengths out of bounds are clamped
    gr.prefix_lens = torch.tensor(prefix, dtype=torch.int32, device="cuda")
    keep = gr.seqlens.clone()
    gr.seqlens[3] = -7
    out, lse = call(q.cuda(), gr)
    assert F.fmha_check_status() == F.FMHA_ERR_PAGES
    assert (out[3] == 0).all() and (lse[3] == -math.inf).all()
    pick = torch.tensor([0, 1, 2, 4])
    check_attention(out.cpu()[pick], lse.cpu()[pick], tuple(x[pick] for x in ref))
    gr.seqlens = keep
    # a page out of the pool reads as zero keys and values
    gr.table[1, 45] = 1 << 20
    gr.dense[0][1, :, 720:736] = 0
    gr.dense[1][1, :, 720:736] = 0
    out, lse = call(q.cuda(), gr)
    assert F.fmha_check_status() == F.FMHA_ERR_PAGES
    check_attention(out, lse, attention_ref(q, *gr.dense, gr.lens, 0.125, False))
    assert F.fmha_check_status() == F.FMHA_OK


def test_nan_and_infinite_scores():
    gr = Groups([[1500, 1400, 1300], [1300]], [1280, 0], 16, 2, 64)
    q = torch.randn(4, 4, 1, 64, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    q[1, 2] = float("nan")
    q[3, 0] = float("nan")
    out, lse = call(q.cuda(), gr)
    assert F.fmha_check_status() == F.FMHA_OK
    bad = torch.zeros(4, 4, 1, dtype=torch.bool)
    bad[1, 2] = bad[3, 0] = True
    assert torch.equal(out.isnan().all(-1).cpu(), bad) and torch.equal(lse.isnan().cpu(), bad)


@pytest.mark.parametrize("D", [64, 128])
def test_forced_timeout_is_reported(D):
    """With a wait limit of one cycle the kernel drains and reports; the next call is right."""
    gr = Groups([[1500, 1400, 1300], [1300]], [1280, 0], 16, 2, D)
    q = torch.randn(4, 8, 1, D, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    assert F.fmha_check_status() == 0
    F.fmha_set_wait_limit(1)
    try:
        call(q.cuda(), gr)
        rc = F.fmha_check_status()
    finally:
        F.fmha_set_wait_limit(0)
    assert rc == F.FMHA_ERR_TIMEOUT
    out, lse = call(q.cuda(), gr)
    assert F.fmha_check_status() == 0
    check_attention(out, lse, attention_ref(q, *gr.dense, gr.lens, D ** -0.5, False))


def test_other_stream_and_no_lse():
    gr = Groups([[700, 800, 650], [50]], [640, 0], 16, 2, 64)
    q = torch.randn(4, 8, 1, 64, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    out, lse = call(q, gr, stream=stream)
    stream.synchronize()
    ref = attention_ref(q.cpu(), *gr.dense, gr.lens, 0.125, False)
    assert F.fmha_check_status(stream) == 0
    check_attention(out, lse, ref)
    cache = F.make_kv_cache(gr.k, gr.v)
    ws = torch.empty(F.fmha_prefix_workspace_size(4, 8, 1, cache, F.make_opts()), dtype=torch.uint8, device="cuda")
    F.fmha_fwd_prefix(q, cache, gr.table, gr.seqlens, gr.cu, gr.prefix_lens, out.zero_(), None, 0.125, F.make_opts(workspace=ws))
    check_attention(out, None, ref)
    # an output that is only 16-byte aligned
    wide = torch.zeros(out.numel() + 4, device="cuda")[4:].view(out.shape)
    F.fmha_fwd_prefix(q, cache, gr.table, gr.seqlens, gr.cu, gr.prefix_lens, wide, lse, 0.125, F.make_opts(out_kind=F.FMHA_OUT_F32, workspace=ws))
    assert F.fmha_check_status() == 0
    check_attention(wide, lse, ref, bf16=False)


def test_nothing_to_do():
    gr = Groups([[700, 800]], [640], 16, 2, 64)
    cache = F.make_kv_cache(gr.k, gr.v)
    empty = torch.empty(0, 8, 1, 64, dtype=torch.bfloat16, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    F.fmha_fwd_prefix(empty, cache, gr.table[:0], none, torch.zeros(1, dtype=torch.int32, device="cuda"), none, empty, None, 1.0, F.make_opts())
    q = torch.empty(2, 8, 0, 64, dtype=torch.bfloat16, device="cuda")
    F.fmha_fwd_prefix(q, cache, gr.table, gr.seqlens, gr.cu, gr.prefix_lens, q, None, 1.0, F.make_opts())
    with pytest.raises(F.FmhaError) as e:      # no workspace
        F.fmha_fwd_prefix(torch.zeros(2, 8, 1, 64, dtype=torch.bfloat16, device="cuda"), cache, gr.table, gr.seqlens, gr.cu, gr.prefix_lens,
                          torch.zeros(2, 8, 1, 64, dtype=torch.bfloat16, device="cuda"), None, 1.0, F.make_opts())
    assert e.value.code == F.FMHA_ERR_WORKSPACE


def test_far_pages():
    """Pages past 2^31 elements of the pool."""
    gr = Groups([[300, 290, 280, 270, 260], [40]], [256, 0], 16, 1, 64)
    pages, big = gr.k.shape[0], torch.zeros((1 << 32) // 1 + (1 << 20), dtype=torch.bfloat16, device="cuda")
    step = (1 << 32) // pages // 64 * 64
    k, v = (big.as_strided(gr.k.shape, (step, 1024, 64, 1), o) for o in (0, 1024))
    k.copy_(gr.k)
    v.copy_(gr.v)
    gr.k, gr.v = k, v
    q = torch.randn(6, 4, 1, 64, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    out, lse = call(q.cuda(), gr)
    assert F.fmha_check_status() == 0
    check_attention(out, lse, attention_ref(q, *gr.dense, gr.lens, 0.125, False))


@pytest.mark.parametrize("groups, members", [(8192, 1), (3000, 2), (1, 8192), (40, 100)])
def test_large_batches(groups, members):
    """Against the paged attention (the 64-bit statement would take minutes)."""
    rng = torch.Generator().manual_seed(groups)
    B, P, D = groups * members, 16, 64
    m = 20 if members > 1 else 0                     # common pages of each group
    rest = torch.randint(1, 30, (B,), generator=rng)
    lens = (m * P + rest).int()
    table = torch.full((B, m + 3), -1, dtype=torch.int32)
    table[:, :m] = torch.arange(groups * m).view(groups, m).repeat_interleave(members, 0) if m else 0
    table[:, m:m + 2] = groups * m + torch.arange(2 * B).view(B, 2)
    pages = groups * m + 2 * B
    k, v = (torch.randn(pages, 1, P, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    cache = F.make_kv_cache(k, v)
    q = torch.randn(B, 2, 1, D, device="cuda").to(torch.bfloat16)
    table, lens = table.cuda(), lens.cuda()
    cu, prefix = torch.arange(0, B + 1, members).int().cuda(), torch.full((groups,), m * P, dtype=torch.int32, device="cuda")
    outs = []
    for name in ("fmha_prefix_workspace_size", "fmha_paged_workspace_size"):
        ws = torch.full((getattr(F, name)(B, 2, 1, cache, F.make_opts()),), 0xff, dtype=torch.uint8, device="cuda")
        out, lse = torch.zeros(q.shape, device="cuda"), torch.zeros(B, 2, 1, device="cuda")
        opts = F.make_opts(out_kind=F.FMHA_OUT_F32, workspace=ws)
        if "prefix" in name:
            F.fmha_fwd_prefix(q, cache, table, lens, cu, prefix, out, lse, 0.125, opts)
        else:
            F.fmha_fwd_paged(q, cache, table, lens, out, lse, 0.125, opts)
        assert F.fmha_check_status() == 0
        outs.append((out, lse))
    # each is within check_attention's bound of the exact result, (2^-12 + 2^-13 + 2^-16) sum p |v| <= .. max |v|; |lse| stays below 64
    assert (outs[0][0] - outs[1][0]).abs().max() <= 2 * float(v.abs().max()) * (2.0 ** -12 + 2.0 ** -13 + 2.0 ** -16)
    assert float(outs[0][1].abs().max()) < 64
    assert (outs[0][1] - outs[1][1]).abs().max() <= 2 * (2.0 ** -12 + 2.0 ** -14)


@pytest.mark.parametrize("seed", range(40))
def test_sweep(seed):
    r = torch.Generator().manual_seed(1000 + seed)

    def pick(*xs):
        return xs[int(torch.randint(0, len(xs), (1,), generator=r))]

    def upto(n):
        return int(torch.randint(0, n + 1, (1,), generator=r))
    P, Hkv, Sq = pick(8, 16, 24, 64, 128), pick(1, 2, 3, 5), pick(1, 1, 2, 3, 4)
    G = pick(1, 2, 3, 4, 5, 8, 16, 21)
    lens, prefix = [], []
    for _ in range(1 + upto(4)):
        p = upto(1500) // P * P
        kind = upto(5)
        lens.append([0 if kind == 0 and upto(3) == 0 else max(0, p + upto(300) - (upto(200) if kind == 1 else 0)) for _ in range(upto(12))])
        prefix.append(p)
    if not any(lens):
        lens, prefix = [[5]], [0]
    run(lens, prefix, P=P, Hq=G * Hkv, Hkv=Hkv, Sq=Sq, D=pick(64, 128), layout=pick("hnd", "nhd", "kv"), causal=Sq > 1 and upto(2) > 0,
        kind=pick(F.FMHA_OUT_BF16, F.FMHA_OUT_BF16, F.FMHA_OUT_F32), seed=seed, scale=pick(1.0, 1.0, 3.0))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq, Hkv, Sq, members", [(1, 1, 1, 140), (2, 2, 1, 70), (3, 1, 1, 50), (5, 1, 1, 30), (14, 2, 1, 20), (8, 1, 1, 17), (16, 1, 1, 16),
                                                  (17, 1, 1, 9), (4, 1, 4, 9), (21, 1, 1, 7), (32, 1, 1, 9), (31, 1, 1, 5), (11, 1, 3, 9), (43, 1, 1, 6),
                                                  (48, 1, 1, 9), (63, 1, 1, 5), (16, 1, 4, 12), (64, 1, 1, 12)])
def test_common_keys_are_read_through_the_first_row(Hq, Hkv, Sq, members, D):
    """With the common entries of the other rows outside the pool: only a call that does share them is right and reports nothing."""
    prefix = 4096
    gr = Groups([[prefix + 5 * i + Sq - 1 for i in range(members)], [300, 200]], [prefix, 0], 16, Hkv, D)
    gr.table[1:members, :prefix // 16] = -1
    q = torch.randn(members + 2, Hq, Sq, D, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    out, lse = call(q.cuda(), gr, causal=Sq > 1)
    assert F.fmha_check_status() == F.FMHA_OK
    check_attention(out, lse, attention_ref(q, *gr.dense, gr.lens, D ** -0.5, Sq > 1))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("prefixes, members", [([1280] * 6, 9), ([1280, 2560, 640, 3200], 9), ([1280] * 40, 9), ([640, 2560] * 12, 40), ([1280], 64)])
def test_equal_and_other_groups(prefixes, members, D):
    """Units of one length, cut into as many pieces each, and of several."""
    lens = [[p + 3 * i + g % 5 for i in range(members)] for g, p in enumerate(prefixes)]
    gr = Groups(lens, prefixes, 16, 2, D)
    for g, p in enumerate(prefixes):
        gr.table[g * members + 1:(g + 1) * members, :p // 16] = -1
    q = torch.randn(len(gr.lens), 8, 1, D, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    out, lse = call(q.cuda(), gr)
    assert F.fmha_check_status() == F.FMHA_OK
    check_attention(out, lse, attention_ref(q, *gr.dense, gr.lens, D ** -0.5, False))


@pytest.mark.parametrize("D", [64, 128])
def test_two_graphs_share_a_workspace(D):
    """Two captured calls of one workspace, replayed in turn on one stream."""
    grs = [Groups([[2000 + i for i in range(n)], [77]], [1920, 0], 16, 2, D, seed=n) for n in (20, 9)]
    qs = [torch.randn(len(g.lens), 8, 1, D, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16) for g in grs]
    caches = [F.make_kv_cache(g.k, g.v) for g in grs]
    need = max(F.fmha_prefix_workspace_size(*q.shape[:3], c, F.make_opts()) for q, c in zip(qs, caches))
    opts = F.make_opts(workspace=torch.full((need,), 0xff, dtype=torch.uint8, device="cuda"))
    dev = [q.cuda() for q in qs]
    outs = [(torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda")) for q in dev]
    graphs = []
    for q, c, g, (out, lse) in zip(dev, caches, grs, outs):
        F.fmha_fwd_prefix(q, c, g.table, g.seqlens, g.cu, g.prefix_lens, out, lse, D ** -0.5, opts)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            F.fmha_fwd_prefix(q, c, g.table, g.seqlens, g.cu, g.prefix_lens, out, lse, D ** -0.5, opts)
    for _ in range(5):
        for out, lse in outs:
            out.zero_(), lse.zero_()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert F.fmha_check_status() == F.FMHA_OK
        for q, g, (out, lse) in zip(qs, grs, outs):
            check_attention(out, lse, attention_ref(q, *g.dense, g.lens, D ** -0.5, False))


@pytest.mark.parametrize("D", [64, 128])
def test_tables_of_many_tiles(D):
    """Room for more than 2^23 key tiles: the work is cut by tiles, not by what they cost."""
    gr = Groups([[2000 + 9 * i for i in range(9)], [1300 + i for i in range(5)], [77, 0]], [1920, 1280, 0], 16, 2, D)
    gr.table = torch.nn.functional.pad(gr.table, (0, (1 << 23) // 32 * 8 + 8), value=-1)     # 16 requests, 2 heads, 8 entries a tile
    for first, last, p in ((0, 9, 1920), (9, 14, 1280)):
        gr.table[first + 1:last, :p // 16] = -1
    q = torch.randn(16, 8, 1, D, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    out, lse = call(q.cuda(), gr)
    assert F.fmha_check_status() == F.FMHA_OK
    check_attention(out, lse, attention_ref(q, *gr.dense, gr.lens, D ** -0.5, False))
