"""The paged cache's operators together, as a serving loop uses them: pages and slots for the new tokens, norm,
rotation and store, attention over the pages; eagerly and as one captured graph that advances its own state."""
import threading

import numpy as np
import pytest
import torch

import attention_tensor_cores_gb300 as F
from paged_util import attention_ref, check_attention, make_pools, page_table_ref, up
from test_gpu_rope_append import EPS, near, ref_heads, table_of

pytestmark = pytest.mark.gpu


class Server:
    """A batch of B requests over a pool of pages, with the host's own account of pages and lengths."""

    def __init__(self, B, Hq, Hkv, D, P, pages, width, layout="hnd", Sq=1, seed=0):
        self.B, self.Hq, self.Hkv, self.D, self.P, self.Sq = B, Hq, Hkv, D, P, Sq
        self.gen = torch.Generator().manual_seed(seed)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.lens, self.new = torch.zeros(B, **i32), torch.full((B,), Sq, **i32)
        self.free, self.n = torch.randperm(pages, generator=self.gen).int().cuda(), torch.tensor([pages], **i32)
        self.table = torch.full((B, width), -1, **i32)
        self.cu, self.kp_vp = torch.zeros(B + 1, **i32), make_pools(pages, Hkv, P, D, layout)
        self.cache = F.make_kv_cache(*self.kp_vp)
        self.w = [(1 + 0.2 * torch.randn(D, generator=self.gen)).to(torch.bfloat16) for _ in range(2)]
        self.wd = [w.cuda() for w in self.w]
        self.cos_sin = table_of(width * P, D)
        self.cos_sin_d = self.cos_sin.cuda()
        ws = F.fmha_paged_workspace_size(B, Hq, Sq, self.cache, F.make_opts(causal=True))
        self.opts = F.make_opts(workspace=torch.empty(ws, dtype=torch.uint8, device="cuda"), causal=True)
        self.host = dict(lens=[0] * B, free=self.free.cpu().numpy(), n=pages, table=self.table.cpu().numpy())

    def buffers(self, T):
        self.T = T
        self.qkv = torch.zeros(T, self.Hq + 2 * self.Hkv, self.D, dtype=torch.bfloat16, device="cuda")
        self.positions = torch.zeros(T, dtype=torch.int32, device="cuda")
        self.slots = torch.zeros(T, dtype=torch.int64, device="cuda")
        self.q = torch.zeros(T // self.Sq, self.Hq, self.Sq, self.D, dtype=torch.bfloat16, device="cuda")
        self.out = torch.zeros(self.B, self.Hq, self.Sq, self.D, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.zeros(self.B, self.Hq, self.Sq, device="cuda")

    def tokens(self):
        x = torch.randn(self.T, self.Hq + 2 * self.Hkv, self.D, generator=self.gen).to(torch.bfloat16)
        self.qkv.copy_(x)
        return x

    def step(self, attend=True):
        a, b = self.Hq, self.Hq + self.Hkv
        F.fmha_page_table(self.lens, self.new, self.P, self.free, self.n, self.table, self.lens, self.cu, self.positions, self.slots, self.n)
        F.fmha_rope_append(self.qkv[:, :a], self.qkv[:, a:b], self.qkv[:, b:], *self.wd, EPS, self.cos_sin_d, self.positions, self.slots,
                           self.q, self.cache)
        if attend:
            F.fmha_fwd_paged(self.q[:self.B], self.cache, self.table, self.lens, self.out, self.lse, self.D ** -0.5, self.opts)

    def check(self, x, new, attend=True):
        """The step that has just run, x being its projections, against the definitions."""
        h, P = self.host, self.P
        ref = page_table_ref(h["lens"], new, P, h["free"], h["n"], h["table"], self.T)
        self.host = dict(lens=ref["seqlens"].tolist(), free=ref["free"], n=ref["n"], table=ref["table"])
        assert int(self.n) == ref["n"]
        for name, got in (("table", self.table), ("free", self.free), ("seqlens", self.lens), ("cu", self.cu), ("slots", self.slots),
                          ("positions", self.positions)):
            assert np.array_equal(got.cpu().numpy(), ref[name]), name
        real = torch.tensor(ref["slots"] >= 0)
        pos, slots = torch.tensor(ref["positions"])[real], torch.tensor(ref["slots"])[real]
        a, b = self.Hq, self.Hq + self.Hkv
        kp, vp = (p.cpu() for p in self.kp_vp)
        yk, size = ref_heads(x[real, a:b], self.w[1], self.cos_sin, pos, False)
        near(kp[slots // P, :, slots % P], yk, size, "k")
        assert torch.equal(vp[slots // P, :, slots % P], x[real, b:])
        yq, size = ref_heads(x[real, :a], self.w[0], self.cos_sin, pos, False)
        near(self.q.cpu().transpose(1, 2).reshape(self.T, self.Hq, self.D)[real], yq, size, "q")
        if attend:
            lens, most = self.host["lens"], max(1, *self.host["lens"])
            k, v = (torch.zeros(self.B, self.Hkv, most, self.D, dtype=torch.bfloat16) for _ in range(2))
            for i, n in enumerate(lens):
                at = torch.arange(n)
                page = torch.tensor(self.host["table"][i])[at // P].long()
                k[i, :, :n], v[i, :, :n] = kp[page, :, at % P].transpose(0, 1), vp[page, :, at % P].transpose(0, 1)
            check_attention(self.out, self.lse, attention_ref(self.q[:self.B].cpu(), k, v, lens, self.D ** -0.5, True))
        assert F.fmha_check_status() == 0


@pytest.mark.parametrize("layout, D, Sq", [("hnd", 128, 1), ("nhd", 64, 2)])
def test_serving_loop(layout, D, Sq):
    """Prompts of many lengths, decoding steps, requests that end and others that take their place."""
    B, P = 5, 16
    s = Server(B, 8, 2, D, P, 100, 20, layout, Sq, seed=D)

    def go(new, attend):
        s.new.copy_(torch.tensor(new, dtype=torch.int32))
        T = sum(max(n, 0) for n in new)
        s.buffers(up(T + 3, Sq) * Sq if not attend else B * Sq)
        x = s.tokens()
        s.step(attend)
        s.check(x, new, attend)

    go([37, 16 * Sq, 0, 130, 1], False)
    for _ in range(3):
        go([Sq] * B, True)
    go([-1, 0, -1, 0, 0], False)
    go([200, 0, 15, 0, 0], False)
    for _ in range(2):
        go([Sq] * B, True)
    go([-1] * B, False)
    assert int(s.n) == 100 and sorted(s.free.tolist()) == list(range(100))


def test_captured_step_advances_itself():
    """One graph of the three calls, lengths and stack updated in place, replayed over many steps."""
    s = Server(6, 8, 2, 128, 8, 120, 12, seed=3)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        s.buffers(6)
        new = [1, 1, 1, 1, 1, 1]
        x = s.tokens()
        s.step()
        s.check(x, new)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            s.step()
        for i in range(40):
            if i == 20:
                s.new.copy_(torch.tensor([1, -1, 1, 1, -1, 1], dtype=torch.int32))
                new = [1, -1, 1, 1, -1, 1]
            if i == 21:
                s.new.fill_(1)
                new = [1] * 6
            x = s.tokens()
            graph.replay()
            torch.cuda.synchronize()
            s.check(x, new)


def test_two_threads():
    """Two host threads, a stream, a cache and a workspace each."""
    servers = [Server(4, 8, 2, 64, 16, 60, 12, seed=s) for s in (1, 2)]
    failures = []

    def work(s):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for n in (50, 1, 1, 1, 1):
                    s.new.fill_(n)
                    s.buffers(4 * n)
                    x = s.tokens()
                    s.step(n == 1)
                    torch.cuda.current_stream().synchronize()
                    s.check(x, [n] * 4, n == 1)
        except BaseException as e:   # noqa: BLE001
            failures.append(e)

    threads = [threading.Thread(target=work, args=(s,)) for s in servers]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures
