"""fmha_page_fork against its plain statement."""
import numpy as np
import pytest
import torch

import attention_tensor_cores_gb300 as F
from paged_util import up
from shared_util import fork_ref

pytestmark = pytest.mark.gpu


def shared_rows(lens, prefix, members, P, rng, pages, width, junk=-9):
    """A table whose groups of `members` rows have their first prefix pages in common, and the ids left."""
    ids = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), width), junk, np.int32)
    at = 0
    for g in range(0, len(lens), members):
        common = ids[at:at + prefix[g // members] // P]
        at += len(common)
        for b in range(g, min(g + members, len(lens))):
            k = min(len(common), up(lens[b], P))
            mine = up(lens[b], P) - k
            table[b, :k] = common[:k]
            table[b, k:k + mine] = ids[at:at + mine]
            at += mine
    assert at <= pages
    return table, ids[at:]


def call(parents, ctx, P, table, stack, pages, height=None, in_place=False, stream=None):
    dev = dict(dtype=torch.int32, device="cuda")
    free = np.full(pages, -5, np.int32)
    free[:len(stack)] = stack
    n = len(stack) if height is None else height
    B = len(parents)
    new = np.full((B, table.shape[1]), -9, np.int32)
    t = {k: torch.full((B,), -77, **dev) for k in ("seqlens", "src", "dst", "tokens")}
    t |= {"free": torch.tensor(free, **dev), "n": torch.tensor([n], **dev), "new_table": torch.tensor(new, **dev)}
    n_out = t["n"] if in_place else torch.full((1,), -77, **dev)
    F.fmha_page_fork(torch.tensor(parents, **dev), torch.tensor(ctx, **dev), P, torch.tensor(table, **dev), t["free"], t["n"], t["new_table"],
                     t["seqlens"], t["src"], t["dst"], t["tokens"], n_out, stream=stream)
    got = {k: v.cpu().numpy() for k, v in t.items()} | {"n": int(n_out)}
    return got, free, n, new


def check(parents, ctx, P, table, stack, pages, **kw):
    got, free, n, new = call(parents, ctx, P, table, stack, pages, **kw)
    assert F.fmha_check_status() == F.FMHA_OK
    want = fork_ref(parents, ctx, P, table, free, n, new)
    for k, v in want.items():
        assert np.array_equal(got[k], v), k
    # a page is free or held, never both; and a partly filled page has one holder
    held = {int(x) for b in range(len(parents)) for x in got["new_table"][b, :up(int(got["seqlens"][b]), P)]}
    assert not held & set(got["free"][:got["n"]].tolist())
    part = [int(got["new_table"][b, c // P]) for b, c in enumerate(got["seqlens"]) if c % P]
    assert len(part) == len(set(part))
    return got


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("parents", [[0], [0, 0], [0, 0, 0, 1], [1, 0], [1, 1], [-1, 1], [-1, -5], [], [0, 1, 0, 1, 0, 1]])
def test_small(parents, in_place):
    table, left = shared_rows([37, 40], [32], 2, 16, np.random.default_rng(1), 20, 6)
    check(parents, [37, 40], 16, table, left, 20, in_place=in_place)


@pytest.mark.parametrize("lens", [[0, 0], [1, 16], [16, 16], [15, 17], [96, 96], [0, 96]])
def test_page_borders(lens):
    table, left = shared_rows(lens, [0], 2, 16, np.random.default_rng(2), 40, 6)
    for parents in ([0, 0, 1, 1], [1, 1, 1], [0]):
        check(parents, lens, 16, table, left, 40)


@pytest.mark.parametrize("P", [1, 7, 16, 64])
@pytest.mark.parametrize("groups, members", [(1, 1), (2, 4), (40, 3), (33, 1), (300, 4)])
def test_beams(groups, members, P):
    rng = np.random.default_rng(P + groups)
    prefix = [int(x) // P * P for x in rng.integers(0, 300, groups)]
    lens = [prefix[i // members] + int(rng.integers(0, 60)) for i in range(groups * members)]
    pages = sum(prefix) // P + sum(up(x, P) for x in lens) + groups * members
    width = max(up(x, P) for x in lens) + 3
    table, left = shared_rows(lens, prefix, members, P, rng, pages, width)
    parents = [int(g * members + rng.integers(0, members)) if rng.random() > 0.1 else -1 for g in range(groups) for _ in range(members)]
    check(parents, lens, P, table, left, pages)


def test_a_step_at_a_time():
    """Beams of two requests over many steps: pages never leak."""
    P, members, pages = 8, 4, 200
    rng = np.random.default_rng(5)
    lens = [43] * members + [90] * members
    table, stack = shared_rows(lens, [40, 88], members, P, rng, pages, 30)
    stack = list(stack)
    for step in range(40):
        parents = [g * members + int(rng.integers(0, members)) for g in range(2) for _ in range(members)]
        got = check(parents, lens, P, table, stack, pages)
        lens, table, stack = [int(x) for x in got["seqlens"]], got["new_table"], list(got["free"][:got["n"]])
        for b in range(len(lens)):      # a token each, with a new page where one is full
            if lens[b] % P == 0:
                table[b, lens[b] // P] = stack.pop()
            lens[b] += 1
        held = {int(x) for b, c in enumerate(lens) for x in table[b, :up(c, P)]}
        assert len(held) + len(stack) == pages and not held & set(stack)


def test_no_free_page_is_needed_that_comes_back():
    # the stack is empty: the ended request's page goes to the copy
    table = np.array([[0, 1], [0, 2]], np.int32)
    got = check([1, 1], [20, 20], 16, table, [], 3)
    assert got["n"] == 0 and got["src"].tolist() == [-1, 2] and got["dst"].tolist() == [-1, 1]


@pytest.mark.parametrize("what", ["parent", "negative", "long", "height", "low", "few", "overflow"])
def test_refused(what):
    rng = np.random.default_rng(3)
    table, left = shared_rows([37, 40], [32], 2, 16, rng, 20, 6)
    parents, lens, height = [0, 0, 1], [37, 40], None
    if what == "parent":
        parents = [0, 2, 1]
    elif what == "negative":
        lens = [37, -1]
    elif what == "long":
        lens = [97, 40]
    elif what == "height":
        height = 21
    elif what == "low":
        height = -1
    elif what == "few":
        height = 0
    else:
        parents, height = [0], 20
    got, free, n, _ = call(parents, lens, 16, table, left, 20, height=height)
    assert F.fmha_check_status() == F.FMHA_ERR_PAGES and F.fmha_check_status() == F.FMHA_OK
    assert np.array_equal(got["free"], free) and got["n"] == n
    assert not got["seqlens"].any() and (got["src"] == -1).all() and (got["dst"] == -1).all() and not got["tokens"].any()


def test_ids_outside_the_pool():
    table = np.array([[0, 1 << 20, 2], [0, 3, -4]], np.int32)
    got, free, n, new = call([0, 0], [40, 40], 16, table, [5, 6], 8)
    assert F.fmha_check_status() == F.FMHA_ERR_PAGES
    want = fork_ref([0, 0], [40, 40], 16, table, free, n, new)
    for k, v in want.items():
        assert np.array_equal(got[k], v), k
    assert got["n"] == 2 + 1 - 1       # page 3 came back, -4 did not


@pytest.mark.parametrize("pages", [1, 31, 32, 33, 255, 256, 257, 100_000, 1 << 19])
def test_pools(pages):
    rng = np.random.default_rng(pages)
    k = min(pages, 500)
    ids = rng.permutation(pages)[:k].astype(np.int32)
    table = np.full((2, k + 1), -1, np.int32)
    table[1, :k] = ids
    table[0, 0] = ids[0]
    got = check([0], [1, k], 1, table, [], pages)
    assert got["n"] == k - 1


def test_large_batch():
    rng = np.random.default_rng(9)
    B, P = 8192, 16
    lens = [int(x) for x in rng.integers(0, 100, B)]
    pages = sum(up(x, P) for x in lens) + B
    table, left = shared_rows(lens, [0] * B, 1, P, rng, pages, 8)
    parents = rng.integers(-1, B, B)
    check([int(x) for x in parents], lens, P, table, left, pages)


def test_longest_row():
    """A row of nearly 2^31 entries, all of the pool's only page: handed on, then given back."""
    i32 = dict(dtype=torch.int32, device="cuda")
    width = (1 << 31) - 300
    table, new = torch.zeros(1, width, **i32), torch.full((1, width), -9, **i32)
    lens, seqlens, src, dst, tok, n = torch.tensor([width - 1], **i32), *(torch.zeros(1, **i32) for _ in range(5))
    stack = torch.full((1,), -5, **i32)
    F.fmha_page_fork(torch.zeros(1, **i32), lens, 1, table, stack, n, new, seqlens, src, dst, tok, n)
    assert F.fmha_check_status() == F.FMHA_OK
    assert seqlens.item() == width - 1 and n.item() == 0 and src.item() == -1
    assert int(new[0, -1]) == -9 and not any(bool(c.any()) for c in new[0, :-1].split(1 << 28))
    F.fmha_page_fork(torch.full((1,), -1, **i32), lens, 1, table, stack, n, new, seqlens, src, dst, tok, n)
    assert F.fmha_check_status() == F.FMHA_OK
    assert n.item() == 1 and stack.item() == 0 and seqlens.item() == 0
