"""Steps of a serving loop whose attention really reads its common keys once: eagerly, as captured graphs whose lengths and parents
change from replay to replay, from two threads, and around a compaction."""
import threading

import pytest
import torch

import attention_tensor_cores_gb300 as F
from test_gpu_rope_append import EPS
from test_gpu_shared_step import Beams

pytestmark = pytest.mark.gpu


class BlindBeams(Beams):
    """Beams whose attention gets a table with ids outside the pool in place of the common tiles of every row but its group's first
    one: what is read through another row is wrong and reported."""

    def __init__(self, prompts, W, Hq, Hkv, D, P, **kw):
        super().__init__(prompts, W, Hq, Hkv, D, P, **kw)
        tiles = torch.tensor([n // P * P // 128 * 128 // P for n in prompts], device="cuda").repeat_interleave(W)     # pages of whole tiles
        assert int(tiles.min()) > 0
        row, col = torch.arange(self.B, device="cuda")[:, None], torch.arange(self.tables[0].shape[1], device="cuda")[None]
        self.hidden = (row % W > 0) & (col < tiles[:, None])
        self.view = torch.zeros_like(self.tables[0])

    def launch(self, now):
        a, b, nxt = self.Hq, self.Hq + self.Hkv, 1 - now
        table, lens = self.tables[nxt], self.lens[nxt]
        F.fmha_page_fork(self.parents, self.lens[now], self.P, self.tables[now], self.free, self.n, table, lens, self.src, self.dst, self.tok,
                         self.n)
        F.fmha_page_copy(self.caches, self.src, self.dst, self.tok)
        F.fmha_page_table(lens, self.new, self.P, self.free, self.n, table, lens, self.cu, self.pos, self.slots, self.n)
        self.view.copy_(table)
        self.view.masked_fill_(self.hidden, -1)
        for i, kv in enumerate(self.caches):
            x = self.qkv[i]
            F.fmha_rope_append(x[:, :a], x[:, a:b], x[:, b:], self.one, self.one, EPS, self.cos_sin, self.pos, self.slots, self.q[i], kv)
            F.fmha_fwd_prefix(self.q[i], kv, self.view, lens, self.groups, self.prefix, self.out[i], self.lse[i], self.D ** -0.5, self.opts)

    def step(self):
        parents = self.choose()
        self.tokens(parents)
        self.launch(self.now)
        torch.cuda.current_stream().synchronize()
        self.check(parents)


@pytest.mark.parametrize("layout, D, P", [("hnd", 128, 16), ("nhd", 64, 8)])
def test_beams(layout, D, P):
    s = BlindBeams([1300, 770], 5, 8, 2, D, P, layout=layout, seed=D)
    for _ in range(12):
        s.step()


@pytest.mark.parametrize("D, W", [(128, 5), (64, 5), (128, 34)])     # 34 beams of 4 rows: two row tiles
def test_captured_steps(D, W):
    """A graph for either direction between the two tables, replayed over many steps with other parents and lengths."""
    s = BlindBeams([1290, 1021], W, 8, 2, D, 16, seed=W, L=1)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(2):     # once eagerly
            s.step()
        graphs = []
        for now in (0, 1):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=stream):
                s.launch(now)
        for i in range(10 if W < 10 else 4):
            if i % 3 == 2:     # the prefix that is shared changes too: less of it, then all again
                s.prefix -= 256
            parents = s.choose()
            s.tokens(parents)
            graphs[s.now].replay()
            torch.cuda.synchronize()
            if i % 3 == 2:
                assert F.fmha_check_status() == F.FMHA_ERR_PAGES     # keys that only the first row has
                s.prefix += 256
                table, lens = s.tables[1 - s.now], s.lens[1 - s.now]
                for k, kv in enumerate(s.caches):
                    F.fmha_fwd_prefix(s.q[k], kv, table, lens, s.groups, s.prefix, s.out[k], s.lse[k], D ** -0.5, s.opts)
            s.check(parents)


def test_two_threads():
    """Two host threads, a stream, caches and a workspace each."""
    servers = [BlindBeams([1300, 900], 5, 8, 2, D, 16, seed=D) for D in (64, 128)]
    failures = []

    def work(s):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(6):
                    s.step()
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
    s = BlindBeams([1200, 910], 5, 8, 2, 64, 16, seed=7, pages=600)
    for _ in range(3):
        s.step()
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, stack = torch.zeros(600, **i32), s.free.clone()
    src, dst, moves = torch.zeros(300, **i32), torch.zeros(300, **i32), torch.zeros(1, **i32)
    table = s.tables[1 - s.now]
    F.fmha_page_compact(s.lens[s.now], 16, s.tables[s.now], s.free, s.n, ids, table, src, dst, moves, stack)
    F.fmha_page_copy(s.caches, src, dst, None, moves)
    assert F.fmha_check_status() == 0 and int(moves) > 0
    s.tables[s.now].copy_(table)
    s.free.copy_(stack)
    for _ in range(3):
        s.step()
