"""Helpers for the tests of pages that requests share: plain statements of the operators, and shared caches."""
from __future__ import annotations

import numpy as np
import torch

from paged_util import make_pools, up

I32 = np.int32


# ------------------------------------------------------------------------------------------------
# forking, compacting
# ------------------------------------------------------------------------------------------------
def fork_ref(parents, ctx, P, table, free, n, new_table):
    """fmha_page_fork, one child after another (numpy int arrays; free and new_table are copied)."""
    free, new_table = free.copy(), new_table.copy()
    parents = [int(p) for p in parents]
    rows = [[int(x) for x in table[i, :up(int(c), P)]] for i, c in enumerate(ctx)]
    kept = {x for p in parents if p >= 0 for x in rows[p]}
    for x in sorted({x for i, r in enumerate(rows) if i not in parents for x in r} - kept):
        if 0 <= x < len(free):
            free[n] = x
            n += 1
    out = {k: [] for k in ("seqlens", "src", "dst", "tokens")}
    for b, p in enumerate(parents):
        c = int(ctx[p]) if p >= 0 else 0
        row = list(rows[p]) if p >= 0 else []
        src = dst = -1
        if c % P and p in parents[:b]:
            n -= 1
            src, dst = row[-1], int(free[n])
            row[-1] = dst
        new_table[b, :len(row)] = row
        for k, v in zip(out, (c, src, dst, c % P if src != -1 or dst != -1 else 0)):
            out[k].append(v)
    return {k: np.array(v, I32) for k, v in out.items()} | {"new_table": new_table, "free": free, "n": n}


def compact_ref(lens, P, table, free, n, new_table, free_out, copies):
    """fmha_page_compact (numpy int arrays; the last two tables are copied)."""
    new_table, free_out = new_table.copy(), free_out.copy()
    N = len(free)
    stack = {int(x) for x in free[:n]}
    holes = [x for x in range(N - n) if x in stack]
    ids = [-1 if x in stack else x for x in range(N)]
    moving = [x for x in range(N - n, N) if x not in stack]
    assert len(moving) == len(holes)
    for a, b in zip(moving, holes):
        ids[a] = b
    for b, c in enumerate(lens):
        for j in range(up(int(c), P)):
            x = int(table[b, j])
            new_table[b, j] = ids[x] if 0 <= x < N and x not in stack else x
    free_out[:n] = np.arange(N - 1, N - 1 - n, -1)
    pad = [-1] * (copies - len(moving))
    return {"new_ids": np.array(ids, I32), "new_table": new_table, "src": np.array(moving + pad, I32), "dst": np.array(holes + pad, I32),
            "moves": len(moving), "free_out": free_out}


# ------------------------------------------------------------------------------------------------
# groups of requests behind common pages
# ------------------------------------------------------------------------------------------------
class Groups:
    """Requests lens[g][i] of each group whose first prefix[g] tokens (whole pages of P) are in the same pages; pools with NaN
    wherever no key is, table entries behind a request's pages `junk`.  A wide table has room for more than 6000 key tiles,
    the fewest for which keys are read once for a group."""

    def __init__(self, lens, prefix, P, Hkv, D, layout="hnd", seed=0, scale=1.0, junk=-3, device="cuda", wide=True):
        g = torch.Generator().manual_seed(seed)
        self.members = [len(x) for x in lens]
        self.lens = [n for group in lens for n in group]
        self.prefix, self.P = prefix, P
        B = len(self.lens)
        assert all(p % P == 0 for p in prefix)
        held = [up(n, P) for n in self.lens]
        width = max(held + [1]) + 2
        if wide:
            width = max(width, up((6000 // (B * Hkv) + 1) * 128, P))
        total = sum(p // P for p in prefix) + sum(held)
        ids = torch.randperm(total + 5, generator=g)
        self.k, self.v = make_pools(total + 5, Hkv, P, D, layout, device="cpu")
        table = torch.full((B, width), junk, dtype=torch.int32)
        S = max(self.lens + [1])
        self.dense = [torch.zeros(B, Hkv, S, D, dtype=torch.bfloat16) for _ in range(2)]
        at, b = 0, 0
        for group, p in zip(lens, prefix):
            m = p // P
            common = ids[at:at + m]
            at += m
            reach = min(max(group + [0]), p)
            ckv = [torch.randn(Hkv, reach, D, generator=g).mul(scale).to(torch.bfloat16) for _ in range(2)]
            for n in group:
                c = min(m, up(n, P))
                mine = up(n, P) - c
                table[b, :c] = common[:c]
                table[b, c:c + mine] = ids[at:at + mine]
                at += mine
                rest = max(n - p, 0)
                for dense, pool, com in zip(self.dense, (self.k, self.v), ckv):
                    dense[b, :, :min(n, p)] = com[:, :min(n, p)]
                    dense[b, :, p:p + rest] = torch.randn(Hkv, rest, D, generator=g).mul(scale).to(torch.bfloat16)
                    for j in range(up(n, P)):
                        t = min(P, (reach if j < m else n) - j * P)   # a common page is as full as the longest request has it
                        src = com if j < m else dense[b]
                        pool[int(table[b, j]), :, :t] = src[:, j * P:j * P + t]
                b += 1
        self.table = table.to(device)
        if device != "cpu":
            self.k, self.v = (_to(x, device) for x in (self.k, self.v))
        self.seqlens = torch.tensor(self.lens, dtype=torch.int32, device=device)
        cu = np.concatenate([[0], np.cumsum(self.members)])
        self.cu = torch.tensor(cu, dtype=torch.int32, device=device)
        self.prefix_lens = torch.tensor(prefix, dtype=torch.int32, device=device)


def _to(pool, device):
    """The pool on the device, with its strides."""
    out = torch.empty_strided(pool.shape, pool.stride(), dtype=pool.dtype, device=device)
    return out.copy_(pool)
