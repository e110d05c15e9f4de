"""fmha_fwd_paged on the GPU against attention over the gathered keys in 64 bits."""
import numpy as np
import pytest
import torch

import attention_tensor_cores_gb300 as F
import oracle
from paged_util import attention_ref, check_attention, fill_tables, make_pools, scatter, up

pytestmark = pytest.mark.gpu


class Problem:
    """q, a paged cache with NaN wherever no request has a token, its block table and the gathered K and V."""

    def __init__(self, lens, Hq, Hkv, Sq, D, P, layout="hnd", seed=0, spare=3, extra=2, junk=1 << 30):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.P, self.B = list(lens), P, len(lens)
        S = max(max(lens), 1)
        rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)   # noqa: E731
        self.q, self.k, self.v = rnd(self.B, Hq, Sq, D), rnd(self.B, Hkv, S, D), rnd(self.B, Hkv, S, D)
        self.scale = D ** -0.5
        pages = sum(up(n, P) for n in lens) + spare
        table, _ = fill_tables(lens, P, pages, max(1, up(S, P)) + extra, np.random.default_rng(seed), junk)
        self.pools = make_pools(pages, Hkv, P, D, layout)
        for pool, x in zip(self.pools, (self.k, self.v)):
            scatter(pool, table, lens, P, x)
        self.cache = F.make_kv_cache(*self.pools)
        self.table = torch.tensor(table, device="cuda")
        self.seqlens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.qd = self.q.cuda()

    def ref(self, causal=False):
        return attention_ref(self.q, self.k, self.v, self.lens, self.scale, causal)

    def workspace(self, **kw):
        B, Hq, Sq, _ = self.q.shape
        n = F.fmha_paged_workspace_size(B, Hq, Sq, self.cache, F.make_opts(**kw))
        return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN partials if read unwritten

    def run(self, causal=False, split=True, kind=F.FMHA_OUT_BF16, stream=None):
        dt = torch.float32 if kind == F.FMHA_OUT_F32 else torch.bfloat16
        out = torch.full(self.q.shape, float("nan"), dtype=dt, device="cuda")
        lse = torch.full(self.q.shape[:3], float("nan"), device="cuda")
        opts = F.make_opts(kind, causal=causal)
        ws = None
        if split:
            ws = self.workspace(out_kind=kind, causal=causal)
            opts = F.make_opts(kind, workspace=ws, causal=causal)
        F.fmha_fwd_paged(self.qd, self.cache, self.table, self.seqlens, out, lse, self.scale, opts, stream)
        return out, lse


def check(p, causal=False, kinds=(F.FMHA_OUT_BF16, F.FMHA_OUT_F32), splits=(True, False)):
    ref = p.ref(causal)
    for kind in kinds:
        for split in splits:
            out, lse = p.run(causal, split, kind)
            assert F.fmha_check_status() == 0
            check_attention(out, lse, ref, kind == F.FMHA_OUT_BF16, f"kind {kind} split {split}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [8, 16, 24, 48, 64, 128, 256, 384])
def test_page_sizes(D, P):
    check(Problem([0, 1, P - 1, P, P + 1, 127, 128, 129, 700, 385], 8, 2, 1, D, P, seed=P), kinds=(F.FMHA_OUT_BF16,))


@pytest.mark.parametrize("layout", ["hnd", "nhd", "kv"])
@pytest.mark.parametrize("Hq, Hkv, Sq", [(1, 1, 1), (4, 4, 1), (5, 5, 1), (32, 8, 1), (16, 1, 1), (14, 2, 2), (8, 2, 4), (3, 1, 5), (6, 3, 8)])
def test_head_groups(layout, Hq, Hkv, Sq):
    for D in (64, 128):
        check(Problem([333, 5, 0, 129], Hq, Hkv, Sq, D, 16, layout, seed=Hq + Sq), kinds=(F.FMHA_OUT_BF16,))


@pytest.mark.parametrize("Hq, Hkv, Sq, causal", [(17, 1, 1, False), (32, 1, 1, False), (64, 2, 1, False), (8, 1, 4, True), (8, 2, 9, True),
                                                 (33, 1, 1, False), (5, 1, 13, True), (24, 1, 3, True)])
def test_more_than_sixteen_rows(Hq, Hkv, Sq, causal):
    for D in (64, 128):
        check(Problem([300, 2, 0, 1025], Hq, Hkv, Sq, D, 32, seed=Hq), causal)


@pytest.mark.parametrize("Hq, Hkv, Sq", [(4, 4, 2), (2, 2, 16), (8, 2, 4), (16, 8, 3)])
def test_causal_rows_that_see_no_key(Hq, Hkv, Sq):
    check(Problem([0, 1, 2, 3, Sq - 1, Sq, Sq + 1, 128, 130, 515], Hq, Hkv, Sq, 64, 16, seed=Sq), True)


@pytest.mark.parametrize("lens", [[1], [0], [0, 0, 0], [5001], [1, 1, 1, 1, 4097], [4097, 1, 1, 1, 1], [0] * 40 + [3000] + [0] * 40])
@pytest.mark.parametrize("Hq, Hkv, D", [(8, 2, 128), (3, 3, 64)])
def test_uneven_batches(lens, Hq, Hkv, D):
    check(Problem(lens, Hq, Hkv, 1, D, 16, seed=len(lens)))


def test_many_requests():
    rng = np.random.default_rng(3)
    p = Problem(rng.integers(0, 40, 2100).tolist(), 2, 1, 1, 64, 8, seed=9)
    check(p, kinds=(F.FMHA_OUT_BF16,))


def test_one_long_request():
    p = Problem([40001], 8, 2, 1, 128, 16, seed=1)
    check(p, kinds=(F.FMHA_OUT_F32,), splits=(True,))


def test_infinite_and_nan_keys_behind_the_length():
    """Stale rows of a request's last page, of any value, change nothing."""
    ref = None
    for fill in (float("nan"), float("inf"), -float("inf"), 3e38):
        p = Problem([77, 130, 9], 4, 1, 1, 64, 32, seed=2)
        for pool in p.pools:
            pool[torch.isnan(pool)] = fill
        out, lse = p.run()
        assert F.fmha_check_status() == 0
        if ref is None:
            ref = out, lse
            check_attention(out, lse, p.ref())
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


def test_equal_scores_far_apart():
    """Scores of one large value and of equal ones: the softmax's reference moves, and does not."""
    p = Problem([1000], 4, 1, 1, 64, 16, seed=4)
    for value, at in ((30.0, 999), (30.0, 0), (-30.0, 500)):
        q = p.q.clone()
        q[...] = 1.0
        k = torch.zeros_like(p.k)
        k[0, 0, at] = value / 8
        p.q, p.k, p.qd = q, k, q.cuda()
        table = p.table.cpu().numpy()
        scatter(p.pools[0], table, p.lens, p.P, k)
        check(p)


def test_bad_pages_and_lengths_are_reported():
    """Pages out of the pool read as zero rows, lengths out of bounds are clamped; both are reported."""
    p = Problem([64, 64, 64], 4, 2, 1, 64, 16, seed=6, extra=0)
    p.table[0, 1], p.table[1, 0] = -3, 1 << 20
    p.k[0, :, 16:32] = p.v[0, :, 16:32] = p.k[1, :, :16] = p.v[1, :, :16] = 0
    ref = p.ref()
    for split in (True, False):
        out, lse = p.run(split=split)
        assert F.fmha_check_status() == F.FMHA_ERR_PAGES
        check_attention(out, lse, ref)
    p = Problem([64, 64, 0], 4, 2, 1, 64, 16, seed=6, extra=0)
    p.seqlens = torch.tensor([64, 100000, -4], dtype=torch.int32, device="cuda")
    for split in (True, False):
        out, lse = p.run(split=split)
        assert F.fmha_check_status() == F.FMHA_ERR_PAGES
        check_attention(out, lse, p.ref())
    assert F.fmha_check_status() == 0


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("lens, Hq, Hkv, Sq, D", [([300, 0, 17], 8, 2, 1, 128), ([2000], 4, 4, 1, 64), ([130, 40], 32, 1, 2, 64)])
def test_nvfp4_output(given, lens, Hq, Hkv, Sq, D):
    """The codes and scales are the quantiser's of the FP32 output (bit-exact), whose tolerance holds."""
    p = Problem(lens, Hq, Hkv, Sq, D, 16, seed=D)
    n = p.q.numel()
    codes = torch.zeros(n // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(n // 16, dtype=torch.uint8, device="cuda")
    ts, amax = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    f32 = torch.full((n,), float("nan"), device="cuda")
    lse = torch.full(p.q.shape[:3], float("nan"), device="cuda")
    sg = torch.tensor([0.001], device="cuda") if given else None
    kw = dict(out_scales=scales, out_tensor_scale=ts, out_f32=f32, nvfp4_scale_in=sg, out_amax=amax)
    for split in (0, 1):
        n_ws = F.fmha_paged_workspace_size(p.B, Hq, Sq, p.cache, F.make_opts(F.FMHA_OUT_NVFP4, None, split, **kw))
        ws = torch.empty(max(n_ws, 256), dtype=torch.uint8, device="cuda")
        F.fmha_fwd_paged(p.qd, p.cache, p.table, p.seqlens, codes, lse, p.scale, F.make_opts(F.FMHA_OUT_NVFP4, None, split, ws, **kw))
        assert F.fmha_check_status() == 0
        check_attention(f32, lse, p.ref(), False)
        o = f32.cpu().numpy()
        assert float(amax) == np.abs(o).max()
        c, s, t = oracle.nvfp4_quantize_scaled(o, 0.001) + (np.float32(0.001),) if given else oracle.nvfp4_quantize(o)
        assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s[:n // 16])


def test_dense_tensor_as_a_cache():
    """A [B, Hkv, Skv, D] tensor is a cache of B pages: the attention of fmha_fwd_ex, whose weights are rounded once
    to BF16 (2^-8 of sum_j p_j |v_j|) where the paged kernel's are not; both outputs are rounded to BF16."""
    g = torch.Generator("cuda").manual_seed(0)
    B, Hq, Hkv, S, D = 3, 8, 2, 640, 128
    q, k, v = (torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16) for s in ((B, Hq, 1, D), (B, Hkv, S, D), (B, Hkv, S, D)))
    lens = torch.tensor([640, 77, 300], dtype=torch.int32, device="cuda")
    a, b = torch.empty_like(q), torch.empty_like(q)
    F.fmha_fwd_ex(q, k, v, a, None, 0.1, F.make_opts(seqlens_k=lens, num_splits=1))
    F.fmha_fwd_paged(q, F.make_kv_cache(k, v), torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous(), lens, b, None, 0.1)
    assert F.fmha_check_status() == 0
    o, l, size = attention_ref(q.cpu(), k.cpu(), v.cpu(), lens.tolist(), 0.1, False)
    check_attention(b, None, (o, l, size))
    assert ((a.double() - b.double()).abs().cpu() <= 2.0 ** -8 * size * (1 + 3 / 32) + 2.0 ** -7 * o.abs()).all()


def test_cache_beyond_32_bit_offsets():
    """Pages whose elements lie past 2^32 from the pool's start (two pools of 8.6 GB)."""
    Hkv, P, D = 8, 16, 128
    pages = (1 << 32) // (Hkv * P * D) + 64
    pools = [torch.empty(pages, Hkv, P, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    g = torch.Generator().manual_seed(1)
    lens = [100, 50]
    k, v = (torch.randn(2, Hkv, 100, D, generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(2, 32, 1, D, generator=g).to(torch.bfloat16)
    table = np.array([[pages - 1 - 5 * i for i in range(7)], [pages - 3, 2, pages // 2, pages - 2, -1, -1, -1]], np.int32)
    for pool, x in zip(pools, (k, v)):
        scatter(pool, table, lens, P, x)
    cache = F.make_kv_cache(*pools)
    ws = torch.empty(F.fmha_paged_workspace_size(2, 32, 1, cache, F.make_opts()), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty(2, 32, 1, D, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 32, 1, device="cuda")
    F.fmha_fwd_paged(q.cuda(), cache, torch.tensor(table, device="cuda"), torch.tensor(lens, dtype=torch.int32, device="cuda"), out, lse,
                     D ** -0.5, F.make_opts(workspace=ws))
    assert F.fmha_check_status() == 0
    check_attention(out, lse, attention_ref(q, k, v, lens, D ** -0.5, False))
    # the writer reaches the same places
    slots = torch.tensor([(pages - 1) * P + 15, (pages - 40) * P + 3], device="cuda")
    x = torch.randn(2, 8, D, device="cuda").to(torch.bfloat16)
    F.fmha_rope_append(x, x, x, None, None, 0.0, None, None, slots, torch.empty_like(x), cache)
    assert F.fmha_check_status() == 0
    for pool in pools:
        assert torch.equal(pool[pages - 1, :, 15], x[0]) and torch.equal(pool[pages - 40, :, 3], x[1])


def test_two_graphs_of_one_workspace():
    """Two captured calls that share a workspace, replayed in turns, with eager calls between them."""
    a, b = Problem([900, 0, 31], 8, 2, 1, 128, 16, seed=1), Problem([40, 2000], 8, 2, 1, 64, 48, seed=2)
    ws = torch.full((max(a.workspace().numel(), b.workspace().numel()),), 0xFF, dtype=torch.uint8, device="cuda")
    opts = F.make_opts(workspace=ws)
    calls = []
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        for p in (a, b):
            out, lse = torch.empty_like(p.qd), torch.empty(p.q.shape[:3], device="cuda")

            def call(p=p, out=out, lse=lse):
                F.fmha_fwd_paged(p.qd, p.cache, p.table, p.seqlens, out, lse, p.scale, opts)
            call()
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                call()
            calls.append((p, out, lse, g, call))
    for turn in range(6):
        for p, out, lse, g, call in calls:
            out.fill_(float("nan"))
            torch.cuda.synchronize()
            if turn == 3:
                call()
            else:
                g.replay()
            torch.cuda.synchronize()
            check_attention(out, lse, p.ref(), what=f"turn {turn}")
    assert F.fmha_check_status() == 0


def test_streams_with_workspaces_of_their_own():
    ps = [Problem([700, 3, 1500], 8, 2, 1, 128, 16, seed=s) for s in range(3)]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    got = []
    for p, s in zip(ps, streams):
        with torch.cuda.stream(s):
            got.append([p.run() for _ in range(5)])
    torch.cuda.synchronize()
    assert F.fmha_check_status() == 0
    for p, outs in zip(ps, got):
        ref = p.ref()
        for out, lse in outs:
            check_attention(out, lse, ref)
            assert torch.equal(out, outs[0][0])     # the merge's order does not change a result


def test_empty_batches():
    p = Problem([20], 4, 2, 1, 64, 16)
    for shape in ((0, 4, 1, 64), (1, 4, 0, 64)):
        q = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        B = shape[0]
        F.fmha_fwd_paged(q, p.cache, p.table[:B], p.seqlens[:B], q.clone(), torch.empty(shape[:3], device="cuda"), 0.1)
    assert F.fmha_check_status() == 0


def test_refuses_wrong_shapes():
    p = Problem([20], 4, 2, 1, 64, 16)
    out, lse = torch.empty_like(p.qd), torch.empty(1, 4, 1, device="cuda")
    args = lambda **kw: {**dict(q=p.qd, cache=p.cache, block_table=p.table, seqlens=p.seqlens, out=out, lse=lse, scale=0.1), **kw}   # noqa: E731
    F.fmha_fwd_paged(**args())
    for bad in (dict(q=p.qd.float()), dict(q=p.qd[:, :3].contiguous()), dict(out=out.float()), dict(out=out[:, :2].contiguous()),
                dict(lse=lse[:, :2].contiguous()), dict(lse=lse.double()), dict(block_table=p.table.long()), dict(block_table=p.table[0]),
                dict(seqlens=p.seqlens.long()), dict(q=p.q), dict(scale=-1.0), dict(q=torch.zeros(1, 4, 1, 128, dtype=torch.bfloat16, device="cuda")),
                dict(seqlens=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(F.FmhaError):
            F.fmha_fwd_paged(**args(**bad))
    with pytest.raises(F.FmhaError):
        F.fmha_fwd_paged(**args(opts=F.make_opts(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))))


@pytest.mark.parametrize("seed", range(60))
def test_random_shapes(seed):
    rng = np.random.default_rng(1000 + seed)
    pick = lambda *a: a[int(rng.integers(len(a)))]   # noqa: E731
    Sq, group, Hkv, D = pick(1, 1, 2, 3, 4, 7), pick(1, 2, 3, 4, 5, 8, 16), pick(1, 2, 3), pick(64, 128)
    B = pick(1, 2, 5, 17, 60)
    most = int(np.exp(rng.uniform(0, np.log(6000 // B + 2))))
    lens = rng.integers(0, most + 1, B)
    lens[rng.integers(B)] = most
    p = Problem(lens.tolist(), Hkv * group, Hkv, Sq, D, pick(8, 16, 32, 40, 64, 128, 160), pick("hnd", "nhd", "kv"), seed)
    check(p, bool(rng.integers(2)), kinds=(pick(F.FMHA_OUT_BF16, F.FMHA_OUT_F32),))


@pytest.mark.parametrize("Hq, Hkv, D", [(4, 4, 128), (16, 2, 64)])
def test_forced_timeout_is_reported(Hq, Hkv, D):
    """With a wait limit of one cycle the kernel drains and reports; the next call is right."""
    p = Problem([900, 0, 333], Hq, Hkv, 1, D, 16, seed=8)
    assert F.fmha_check_status() == 0
    F.fmha_set_wait_limit(1)
    try:
        p.run()
        rc = F.fmha_check_status()
    finally:
        F.fmha_set_wait_limit(0)
    assert rc == F.FMHA_ERR_TIMEOUT
    check(p)
