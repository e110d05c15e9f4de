"""fmha_page_table on the GPU against the same steps taken one request after another."""
import numpy as np
import pytest
import torch

import attention_tensor_cores_gb300 as F
from paged_util import fill_tables, page_table_ref, up

pytestmark = pytest.mark.gpu


def setup(ctx, new, P, spare, pad, seed, width=None):
    rng = np.random.default_rng(seed)
    need = sum(up(c + a, P) - up(c, P) for c, a in zip(ctx, new) if a >= 0)
    pages = max(1, sum(up(c, P) for c in ctx) + need + spare)
    width = width or max([1] + [up(c + max(a, 0), P) for c, a in zip(ctx, new)])
    table, left = fill_tables(ctx, P, pages, width, rng)
    free = np.full(pages, -7, np.int32)
    free[:len(left)] = left
    return table, free, len(left), sum(max(a, 0) for a in new) + pad


class Step:
    """Device arrays of one call."""

    def __init__(self, ctx, new, table, free, n, T):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.ctx, self.new = torch.tensor(ctx, **i32), torch.tensor(new, **i32)
        self.table, self.free = torch.tensor(table, **i32), torch.tensor(free, **i32)
        self.n, self.n_out = torch.tensor([n], **i32), torch.full((1,), -9, **i32)
        self.seqlens, self.cu = torch.full((len(ctx),), -9, **i32), torch.full((len(ctx) + 1,), -9, **i32)
        self.positions = torch.full((T,), -9, **i32)
        self.slots = torch.full((T,), -9, dtype=torch.int64, device="cuda")

    def call(self, P, stream=None):
        F.fmha_page_table(self.ctx, self.new, P, self.free, self.n, self.table, self.seqlens, self.cu, self.positions, self.slots,
                          self.n_out, stream)

    def same(self, ref):
        assert int(self.n_out) == ref["n"]
        for name in ("table", "free", "cu", "seqlens", "positions", "slots"):
            got = getattr(self, name).cpu().numpy()
            assert np.array_equal(got, ref[name]), name


def run(ctx, new, P, spare=3, pad=0, seed=0):
    table, free, n, T = setup(ctx, new, P, spare, pad, seed)
    s = Step(ctx, new, table, free, n, T)
    s.call(P)
    assert F.fmha_check_status() == 0
    s.same(page_table_ref(ctx, new, P, free, n, table, T))


@pytest.mark.parametrize("P", [1, 8, 16, 48, 64])
@pytest.mark.parametrize("ctx, new", [
    ([0], [1]), ([0], [0]), ([5], [-1]), ([16], [1]), ([15], [1]), ([15, 16, 17], [1, 1, 1]), ([0, 0, 0], [0, 7, 0]),
    ([100, 0, 33, 64, 1], [-1, 65, 1, 0, -1]), ([64, 64, 64], [-1, -1, -1]), ([1, 2, 3], [200, 300, 1000])])
def test_small_steps(ctx, new, P):
    for pad in (0, 5):
        run(ctx, new, P, pad=pad)
    run(ctx, new, P, spare=0)


@pytest.mark.parametrize("B, most, add, P, done", [
    (1, 40000, 1, 16, 0), (33, 500, 1, 16, 9), (257, 900, 1, 8, 100), (1024, 300, 3, 16, 300), (1025, 64, 2, 32, 1), (8192, 30, 1, 16, 4000),
    (5, 1000, 30000, 64, 1), (32, 2000, 4000, 16, 8), (3, 10, 100001, 8, 0)])
def test_batches(B, most, add, P, done):
    rng = np.random.default_rng(B + most)
    ctx = rng.integers(0, most + 1, B).tolist()
    new = rng.integers(0, add + 1, B)
    new[rng.choice(B, done, replace=False)] = -1
    run(ctx, new.tolist(), P, spare=int(rng.integers(0, 50)), pad=int(rng.integers(0, 700)), seed=B)


@pytest.mark.parametrize("B, add", [(9, 700), (3000, 1)])
def test_in_place_with_many_tokens_or_requests(B, add):
    """More than 2048 of either: the lengths and the height are updated by a second launch."""
    rng = np.random.default_rng(B)
    ctx, new = rng.integers(0, 200, B).tolist(), rng.integers(add, add + 2, B)
    new[::4] = -1
    table, free, n, T = setup(ctx, new.tolist(), 16, 3, 11, B)
    s = Step(ctx, new.tolist(), table, free, n, T)
    s.seqlens, s.n_out = s.ctx, s.n
    s.call(16)
    assert F.fmha_check_status() == 0
    s.same(page_table_ref(ctx, new, 16, free, n, table, T))


def test_no_requests_and_no_tokens():
    s = Step([], [], np.zeros((0, 4), np.int32), np.arange(6), 6, 3)
    s.call(16)
    torch.cuda.synchronize()
    assert s.cu.tolist() == [0] and s.slots.tolist() == [-1] * 3 and s.positions.tolist() == [0] * 3 and int(s.n_out) == 6
    s = Step([3], [0], np.array([[2]], np.int32), np.arange(6), 6, 0)
    s.call(16)
    torch.cuda.synchronize()
    assert s.cu.tolist() == [0, 0] and s.seqlens.tolist() == [3] and F.fmha_check_status() == 0


@pytest.mark.parametrize("what", ["pages", "row", "tokens", "negative", "height", "pushed"])
def test_all_or_nothing(what):
    """A step that cannot be taken leaves the table and the stack, gives no slot and is reported."""
    ctx, new, P = [20, 31, 40], [1, 5, -1], 16
    table, free, n, T = setup(ctx, new, P, 3, 2, 1)
    if what == "pages":
        new, n = [1, 5, 0], 0
    elif what == "row":
        new = [1, 200, -1]
        T = 300
    elif what == "tokens":
        T = 5
    elif what == "negative":
        ctx = [20, -1, 40]
    elif what == "height":
        n = -1
    else:
        n = len(free) - 1      # three pages come back: more than the pool has
    s = Step(ctx, new, table, free, n, T)
    s.call(P)
    assert F.fmha_check_status() == F.FMHA_ERR_PAGES
    assert F.fmha_check_status() == 0
    s.same({"n": n, "table": table, "free": free, "cu": np.zeros(4, np.int32), "seqlens": np.array(ctx, np.int32),
            "positions": np.zeros(T, np.int32), "slots": np.full(T, -1)})


def test_pages_outside_the_pool_give_no_slot():
    table = np.array([[3, 99], [-5, 0]], np.int32)
    s = Step([17, 4], [1, 2], table, np.arange(8), 2, 3)
    s.call(16)
    assert F.fmha_check_status() == F.FMHA_ERR_PAGES
    assert s.slots.tolist() == [-1, -1, -1] and s.seqlens.tolist() == [18, 6] and s.positions.tolist() == [17, 4, 5]


def test_in_place_steps_in_a_graph():
    """Lengths and stack height updated in place: a captured step replayed is the step taken again."""
    P, B = 8, 6
    rng = np.random.default_rng(5)
    ctx = [0, 7, 8, 30, 1, 16]
    table, left = fill_tables(ctx, P, 200, 40, rng)
    free = np.full(200, -1, np.int32)
    free[:len(left)] = left
    s = Step(ctx, [1, 2, 1, 3, 0, 1], table, free, len(left), 10)
    s.seqlens, s.n_out = s.ctx, s.n
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        s.call(P)                       # eager once
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            s.call(P)
    n, lens = len(left), list(ctx)
    for step in range(30):
        if step:
            g.replay()
            torch.cuda.synchronize()
        new = [1, 2, 1, 3, 0, 1]
        ref = page_table_ref(lens, new, P, free, n, table, 10)
        table, free, n, lens = ref["table"], ref["free"], ref["n"], ref["seqlens"].tolist()
        s.same(ref)
    s.new.copy_(torch.tensor([-1, -1, 1, -1, 0, -1], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    s.same(page_table_ref(lens, [-1, -1, 1, -1, 0, -1], P, free, n, table, 10))
    assert F.fmha_check_status() == 0
