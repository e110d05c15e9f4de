"""fmha_page_compact against its plain statement, and with fmha_page_copy: the data follows."""
import numpy as np
import pytest
import torch

import attention_tensor_cores_gb300 as F
from paged_util import up
from shared_util import compact_ref

pytestmark = pytest.mark.gpu


def call(lens, P, table, stack, pages, height=None, spare=0):
    dev = dict(dtype=torch.int32, device="cuda")
    free = np.full(pages, -5, np.int32)
    free[:len(stack)] = stack
    n = len(stack) if height is None else height
    copies = pages // 2 + spare
    start = {"new_ids": np.full(pages, -77, np.int32), "new_table": np.full(table.shape, -9, np.int32), "src": np.full(copies, -77, np.int32),
             "dst": np.full(copies, -77, np.int32), "moves": np.full(1, -77, np.int32), "free_out": np.full(pages, -6, np.int32)}
    t = {k: torch.tensor(v, **dev) for k, v in start.items()}
    F.fmha_page_compact(torch.tensor(lens, **dev), P, torch.tensor(table, **dev), torch.tensor(free, **dev), torch.tensor([n], **dev),
                        t["new_ids"], t["new_table"], t["src"], t["dst"], t["moves"], t["free_out"])
    return {k: v.cpu().numpy() for k, v in t.items()}, free, n, start, copies


def check(lens, P, table, stack, pages, **kw):
    got, free, n, start, copies = call(lens, P, table, stack, pages, **kw)
    assert F.fmha_check_status() == F.FMHA_OK
    want = compact_ref(lens, P, table, free, n, start["new_table"], start["free_out"], copies)
    for k, v in want.items():
        assert np.array_equal(got[k], v if k != "moves" else [v]), k
    return got


def scene(pages, B, used, P, rng, elsewhere=0):
    ids = rng.permutation(pages).astype(np.int32)
    held = [used // B + (1 if b < used % B else 0) for b in range(B)]
    table = np.full((B, max(held) + 2), -9, np.int32)
    at = 0
    for b, k in enumerate(held):
        table[b, :k] = ids[at:at + k]
        at += k
    lens = [k * P - int(rng.integers(0, P)) if k else 0 for k in held]
    return lens, table, ids[at + elsewhere:]


@pytest.mark.parametrize("pages", [1, 2, 31, 32, 33, 255, 256, 257, 1000, 8191, 100_000])
@pytest.mark.parametrize("share", [0.0, 0.1, 0.5, 0.95, 1.0])
def test_pools(pages, share):
    rng = np.random.default_rng(pages)
    check(*_scene(scene(pages, 3, int(share * pages), 16, rng)), pages)


def _scene(s):
    return s[0], 16, s[1], s[2]


def test_limit_of_pages():
    rng = np.random.default_rng(4)
    check(*_scene(scene(1 << 20, 64, 700_000, 16, rng)), 1 << 20)


def test_pages_that_no_request_names_and_a_longer_list():
    rng = np.random.default_rng(6)
    check(*_scene(scene(777, 5, 200, 16, rng, elsewhere=150)), 777, spare=100)


def test_shared_pages():
    table = np.array([[9, 7, 3, -1], [9, 7, 5, 8]], np.int32)
    got = check([40, 64], 16, table, [0, 1, 2, 4, 6], 10)
    assert got["moves"] == 4 and got["new_table"][0, 0] == got["new_table"][1, 0]     # pages 5, 7, 8 and 9


@pytest.mark.parametrize("B", [0, 1, 2000])
def test_batches(B):
    rng = np.random.default_rng(B)
    pages = 5000
    ids = rng.permutation(pages).astype(np.int32)
    lens = [int(x) for x in rng.integers(0, 33, B)]
    table = np.full((B, 2), -9, np.int32)
    at = 0
    for b, c in enumerate(lens):
        k = up(c, 16)
        table[b, :k] = ids[at:at + k]
        at += k
    check(lens, 16, table, ids[at:], pages)


@pytest.mark.parametrize("what", ["height", "low", "twice", "outside", "negative", "long"])
def test_nothing_moves(what):
    rng = np.random.default_rng(8)
    lens, table, stack = scene(40, 2, 20, 16, rng)
    stack, height = stack.copy(), None
    if what == "height":
        height = 41
    elif what == "low":
        height = -1
    elif what == "twice":
        stack[3] = stack[9]
    elif what == "outside":
        stack[3] = 40
    elif what == "negative":
        lens[0] = -1
    else:
        lens[0] = table.shape[1] * 16 + 1
    got, free, n, start, _ = call(lens, 16, table, stack, 40, height=height)
    assert F.fmha_check_status() == F.FMHA_ERR_PAGES and F.fmha_check_status() == F.FMHA_OK
    assert np.array_equal(got["new_ids"], np.arange(40)) and got["moves"] == 0 and (got["src"] == -1).all() and (got["dst"] == -1).all()
    k = min(max(n, 0), 40)
    assert np.array_equal(got["free_out"][:k], free[:k]) and np.array_equal(got["free_out"][k:], start["free_out"][k:])
    for b, c in enumerate(lens):
        k = up(min(max(c, 0), table.shape[1] * 16), 16)
        assert np.array_equal(got["new_table"][b, :k], table[b, :k])


def test_entries_that_are_no_used_page():
    table = np.array([[9, 2, 50, -3]], np.int32)           # 2 is free
    got, free, n, start, copies = call([64], 16, table, [0, 2, 4], 10)
    assert F.fmha_check_status() == F.FMHA_ERR_PAGES
    want = compact_ref([64], 16, table, free, n, start["new_table"], start["free_out"], copies)
    for k, v in want.items():
        assert np.array_equal(got[k], v if k != "moves" else [v]), k


def test_the_data_follows():
    rng = np.random.default_rng(2)
    lens, table, stack = scene(64, 3, 30, 16, rng)
    k, v = (torch.randn(64, 2, 16, 64, device="cuda").to(torch.bfloat16) for _ in range(2))
    before = [[x[table[b, j]].clone() for b in range(3) for j in range(up(lens[b], 16))] for x in (k, v)]
    got = check(lens, 16, table, stack, 64)
    i32 = dict(dtype=torch.int32, device="cuda")
    F.fmha_page_copy([F.make_kv_cache(k, v)], torch.tensor(got["src"], **i32), torch.tensor(got["dst"], **i32), None, torch.tensor(got["moves"], **i32))
    new = got["new_table"]
    after = [[x[new[b, j]] for b in range(3) for j in range(up(lens[b], 16))] for x in (k, v)]
    assert all(torch.equal(x, y) for p, q in zip(before, after) for x, y in zip(p, q))
    assert new[0, 0] < 30 and max(int(new[b, j]) for b in range(3) for j in range(up(lens[b], 16))) < 30


def test_captured():
    """The graph of a compaction and its copies, replayed over other tables and stacks."""
    rng = np.random.default_rng(12)
    pages, P = 40_000, 16     # two launches
    i32 = dict(dtype=torch.int32, device="cuda")
    scenes = [scene(pages, 30, used, P, rng) for used in (17_000, 25_000, 39_999)]
    width = max(s[1].shape[1] for s in scenes)
    lens, n = torch.zeros(30, **i32), torch.zeros(1, **i32)
    table, new = torch.full((30, width), -1, **i32), torch.zeros(30, width, **i32)
    stack, ids, out, src, dst, moves = (torch.zeros(k, **i32) for k in (pages, pages, pages, pages // 2, pages // 2, 1))
    k, v = (torch.zeros(pages, 1, P, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache = F.make_kv_cache(k, v)

    def step():
        F.fmha_page_compact(lens, P, table, stack, n, ids, new, src, dst, moves, out)
        F.fmha_page_copy([cache], src, dst, None, moves)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for s in scenes:
        lens.copy_(torch.tensor(s[0]))
        table[:, :s[1].shape[1]] = torch.tensor(s[1], **i32)
        stack[:len(s[2])] = torch.tensor(s[2], **i32)
        n.fill_(len(s[2]))
        k.copy_(torch.randint(-128, 128, k.shape, device="cuda"))
        v.copy_(-k)
        before = k.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert F.fmha_check_status() == F.FMHA_OK
        used = pages - len(s[2])
        for b in range(30):
            h = up(s[0][b], P)
            assert h == 0 or int(new[b, :h].max()) < used
            assert torch.equal(k[new[b, :h].long()], before[table[b, :h].long()]) and torch.equal(v[new[b, :h].long()], -before[table[b, :h].long()])
        assert out[:pages - used].tolist() == list(range(pages - 1, used - 1, -1))


def test_longest_row():
    """A row of nearly 2^31 entries, all of the pool's only page."""
    i32 = dict(dtype=torch.int32, device="cuda")
    width = (1 << 31) - 300
    table, new = torch.zeros(1, width, **i32), torch.full((1, width), -9, **i32)
    ids, moves, n = torch.zeros(1, **i32), torch.zeros(1, **i32), torch.zeros(1, **i32)
    src, dst, stack, out = (torch.zeros(4, **i32) for _ in range(4))
    F.fmha_page_compact(torch.tensor([width - 1], **i32), 1, table, stack[:1], n, ids, new, src, dst, moves, out[:1])
    assert F.fmha_check_status() == F.FMHA_OK
    assert int(new[0, -1]) == -9 and not any(bool(c.any()) for c in new[0, :-1].split(1 << 28))
