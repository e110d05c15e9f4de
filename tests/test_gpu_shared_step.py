"""Beams as a serving loop runs them: a prompt's pages forked, partly filled pages copied in every layer, pages and slots for the new
tokens, norm, rotation and store, attention over the common pages; eagerly, as captured graphs, and from two threads."""
import threading

import pytest
import torch

import attention_tensor_cores_gb300 as F
from paged_util import attention_ref, check_attention, make_pools, up
from test_gpu_rope_append import EPS, table_of

pytestmark = pytest.mark.gpu


class Beams:
    """`prompts` requests of W beams each over L layers, with the host's own copy of every beam's keys and values."""

    def __init__(self, prompts, W, Hq, Hkv, D, P, L=2, layout="hnd", seed=0, pages=None):
        self.prompts, self.W, self.B, self.L, self.P = prompts, W, len(prompts) * W, L, P
        self.Hq, self.Hkv, self.D = Hq, Hkv, D
        self.gen = torch.Generator().manual_seed(seed)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.pages = pages or sum(up(n, P) for n in prompts) + 8 * self.B
        width = up((6000 // (self.B * Hkv) + 1) * 128, P)     # a table of so many key tiles: common keys are read once
        self.free, self.n = torch.randperm(self.pages, generator=self.gen).int().cuda(), torch.tensor([self.pages], **i32)
        self.tables, self.lens = [torch.full((self.B, width), -1, **i32) for _ in range(2)], [torch.zeros(self.B, **i32) for _ in range(2)]
        self.parents, self.new = torch.zeros(self.B, **i32), torch.ones(self.B, **i32)
        self.src, self.dst, self.tok = (torch.zeros(self.B, **i32) for _ in range(3))
        self.cu = torch.zeros(self.B + 1, **i32)
        self.groups = torch.arange(0, self.B + 1, W).int().cuda()
        self.prefix = torch.tensor([n // P * P for n in prompts], **i32)
        self.pools = [make_pools(self.pages, Hkv, P, D, layout) for _ in range(L)]
        self.caches = [F.make_kv_cache(*p) for p in self.pools]
        self.one = torch.ones(D, dtype=torch.bfloat16, device="cuda")
        self.cos_sin = table_of(max(prompts) + 64, D).cuda()
        self.q = [torch.zeros(self.B, Hq, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(L)]
        self.out, self.lse = [torch.zeros_like(self.q[0]) for _ in range(L)], [torch.zeros(self.B, Hq, 1, device="cuda") for _ in range(L)]
        need = F.fmha_prefix_workspace_size(self.B, Hq, 1, self.caches[0], F.make_opts())
        self.opts = F.make_opts(workspace=torch.full((need,), 0xff, dtype=torch.uint8, device="cuda"))
        self.qkv = [torch.zeros(self.B, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(L)]
        self.pos, self.slots = torch.zeros(self.B, **i32), torch.zeros(self.B, dtype=torch.int64, device="cuda")
        self.now = 0
        self.fill()

    def rows(self, slots):
        """Keys and values in these slots, [L][2][tokens, Hkv, D] on the host."""
        s = slots.long()
        return [[p[s // self.P, :, s % self.P].cpu() for p in kv] for kv in self.pools]

    def fill(self):
        """The prompts, one row each, forked into W beams."""
        N, dev = len(self.prompts), dict(dtype=torch.int32, device="cuda")
        T = sum(self.prompts)
        table, lens, cu = self.tables[0][:N].clone(), torch.zeros(N, **dev), torch.zeros(N + 1, **dev)
        pos, slots = torch.zeros(T, **dev), torch.zeros(T, dtype=torch.int64, device="cuda")
        F.fmha_page_table(lens, torch.tensor(self.prompts, **dev), self.P, self.free, self.n, table, lens, cu, pos, slots, self.n)
        a, b = self.Hq, self.Hq + self.Hkv
        for kv in self.caches:
            x = torch.randn(T, b + self.Hkv, self.D, generator=self.gen).to(torch.bfloat16).cuda()
            F.fmha_rope_append(x[:, :a], x[:, a:b], x[:, b:], self.one, self.one, EPS, self.cos_sin, pos, slots,
                               torch.empty(T, a, self.D, dtype=torch.bfloat16, device="cuda"), kv)
        start = [0, *torch.tensor(self.prompts).cumsum(0).tolist()]
        stored = [self.rows(slots[start[i]:start[i + 1]]) for i in range(N)]
        parents = torch.arange(N).repeat_interleave(self.W).int().cuda()
        F.fmha_page_fork(parents, lens, self.P, table, self.free, self.n, self.tables[0], self.lens[0], self.src, self.dst, self.tok, self.n)
        F.fmha_page_copy(self.caches, self.src, self.dst, self.tok)
        self.host = [stored[i // self.W] for i in range(self.B)]
        assert F.fmha_check_status() == 0

    def tokens(self, parents):
        self.parents.copy_(torch.tensor(parents, dtype=torch.int32))
        for x in self.qkv:
            x.copy_(torch.randn(x.shape, generator=self.gen))

    def launch(self, now):
        """What a step launches, from buffers `now` to the others."""
        a, b, nxt = self.Hq, self.Hq + self.Hkv, 1 - now
        table, lens = self.tables[nxt], self.lens[nxt]
        F.fmha_page_fork(self.parents, self.lens[now], self.P, self.tables[now], self.free, self.n, table, lens, self.src, self.dst, self.tok,
                         self.n)
        F.fmha_page_copy(self.caches, self.src, self.dst, self.tok)
        F.fmha_page_table(lens, self.new, self.P, self.free, self.n, table, lens, self.cu, self.pos, self.slots, self.n)
        for i, kv in enumerate(self.caches):
            x = self.qkv[i]
            F.fmha_rope_append(x[:, :a], x[:, a:b], x[:, b:], self.one, self.one, EPS, self.cos_sin, self.pos, self.slots, self.q[i], kv)
            F.fmha_fwd_prefix(self.q[i], kv, table, lens, self.groups, self.prefix, self.out[i], self.lse[i], self.D ** -0.5, self.opts)

    def check(self, parents):
        assert F.fmha_check_status() == 0
        new = self.rows(self.slots)
        self.host = [[[torch.cat([old, x[b:b + 1]]) for old, x in zip(layer, fresh)] for layer, fresh in zip(self.host[p], new)]
                     for b, p in enumerate(parents)]
        lens = [h[0][0].shape[0] for h in self.host]
        assert self.lens[1 - self.now].tolist() == lens
        most = max(lens)
        for i in range(self.L):
            k, v = (torch.zeros(self.B, self.Hkv, most, self.D, dtype=torch.bfloat16) for _ in range(2))
            for b, n in enumerate(lens):
                k[b, :, :n], v[b, :, :n] = (x.transpose(0, 1) for x in self.host[b][i])
            check_attention(self.out[i], self.lse[i], attention_ref(self.q[i].cpu(), k, v, lens, self.D ** -0.5, False), what=f"layer {i}")
        # pages are free or held, and a partly filled one has one holder
        table = self.tables[1 - self.now].cpu()
        held = [set(table[b, :up(n, self.P)].tolist()) for b, n in enumerate(lens)]
        stack = self.free[:int(self.n)].tolist()
        assert len(set(stack)) == len(stack) and not set(stack) & set().union(*held)
        assert len(stack) + len(set().union(*held)) == self.pages
        self.now = 1 - self.now

    def choose(self):
        return [g * self.W + int(torch.randint(0, self.W, (1,), generator=self.gen)) for g in range(len(self.prompts)) for _ in range(self.W)]


@pytest.mark.parametrize("layout, D, P", [("hnd", 128, 16), ("nhd", 64, 8)])
def test_beams(layout, D, P):
    s = Beams([300, 517, 40], 4, 8, 2, D, P, layout=layout, seed=D)
    for _ in range(20):
        parents = s.choose()
        s.tokens(parents)
        s.launch(s.now)
        s.check(parents)
    # every request ends: all pages come back
    s.parents.fill_(-1)
    F.fmha_page_fork(s.parents, s.lens[s.now], P, s.tables[s.now], s.free, s.n, s.tables[1 - s.now], s.lens[1 - s.now], s.src, s.dst, s.tok, s.n)
    assert F.fmha_check_status() == 0
    assert int(s.n) == s.pages and sorted(s.free.tolist()) == list(range(s.pages)) and not s.lens[1 - s.now].any()


def test_captured_steps():
    """A graph for either direction between the two tables, replayed over many steps with other parents."""
    s = Beams([260, 131], 3, 8, 2, 128, 16, seed=5)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        for now in (0, 1):     # once eagerly
            parents = s.choose()
            s.tokens(parents)
            s.launch(now)
            s.check(parents)
        graphs = []
        for now in (0, 1):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=stream):
                s.launch(now)
        for _ in range(16):
            parents = s.choose()
            s.tokens(parents)
            graphs[s.now].replay()
            torch.cuda.synchronize()
            s.check(parents)


def test_two_threads():
    """Two host threads, a stream, caches and a workspace each."""
    servers = [Beams([400, 150], 4, 8, 2, D, 16, seed=D) for D in (64, 128)]
    failures = []

    def work(s):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(6):
                    parents = s.choose()
                    s.tokens(parents)
                    s.launch(s.now)
                    torch.cuda.current_stream().synchronize()
                    s.check(parents)
        except BaseException as e:   # noqa: BLE001
            failures.append(e)

    threads = [threading.Thread(target=work, args=(s,)) for s in servers]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures


def test_compaction_between_steps():
    s = Beams([200, 90], 2, 4, 2, 64, 16, seed=7, pages=300)
    for _ in range(3):
        parents = s.choose()
        s.tokens(parents)
        s.launch(s.now)
        s.check(parents)
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, stack = torch.zeros(300, **i32), s.free.clone()
    src, dst, moves = torch.zeros(150, **i32), torch.zeros(150, **i32), torch.zeros(1, **i32)
    table = s.tables[1 - s.now]
    F.fmha_page_compact(s.lens[s.now], 16, s.tables[s.now], s.free, s.n, ids, table, src, dst, moves, stack)
    F.fmha_page_copy(s.caches, src, dst, None, moves)
    used = 300 - int(s.n)
    assert F.fmha_check_status() == 0 and int(moves) > 0
    assert max(int(table[b, :up(n, 16)].max()) for b, n in enumerate(s.lens[s.now].tolist())) < used
    s.tables[s.now].copy_(table)
    s.free.copy_(stack)
    for _ in range(3):
        parents = s.choose()
        s.tokens(parents)
        s.launch(s.now)
        s.check(parents)
