"""Helpers for the tests of the paged key/value cache: plain 64-bit statements of its three operators."""
from __future__ import annotations

import math

import numpy as np
import torch


def up(n: int, m: int) -> int:
    return -(-n // m)


# ------------------------------------------------------------------------------------------------
# page tables
# ------------------------------------------------------------------------------------------------
def page_table_ref(ctx, new, P, free, n, table, T):
    """The page table step, one request after another (numpy int arrays; table and free are copied)."""
    table, free = table.copy(), free.copy()
    for b in range(len(ctx)):
        if new[b] < 0:
            k = up(int(ctx[b]), P)
            free[n:n + k] = table[b, :k]
            n += k
    cu, pos, slots, lens = [0], [], [], []
    for b in range(len(ctx)):
        c, a = int(ctx[b]), max(int(new[b]), 0)
        if new[b] >= 0:
            for j in range(up(c, P), up(c + a, P)):
                n -= 1
                table[b, j] = free[n]
        for x in range(c, c + a):
            pos.append(x)
            slots.append(int(table[b, x // P]) * P + x % P)
        cu.append(cu[-1] + a)
        lens.append(0 if new[b] < 0 else c + a)
    pad = T - cu[-1]
    i32 = np.int32
    return {"table": table, "free": free, "n": n, "cu": np.array(cu, i32), "seqlens": np.array(lens, i32),
            "positions": np.array(pos + [0] * pad, i32), "slots": np.array(slots + [-1] * pad, np.int64)}


def fill_tables(lens, P, pages, width, rng, junk=-1):
    """A block table of `width` columns with distinct pages for each request's tokens, and the pages left."""
    ids = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), width), junk, np.int32)
    at = 0
    for b, x in enumerate(lens):
        k = up(int(x), P)
        table[b, :k] = ids[at:at + k]
        at += k
    assert at <= pages
    return table, ids[at:]


# ------------------------------------------------------------------------------------------------
# pools
# ------------------------------------------------------------------------------------------------
def make_pools(pages, H, P, D, layout, device="cuda", fill=float("nan")):
    """K and V pools [pages, H, P, D] (views): hnd and nhd are pools of their own, kv is one allocation
    with K and V of a page side by side."""
    if layout == "kv":
        both = torch.full((pages, 2, H, P, D), fill, dtype=torch.bfloat16, device=device)
        return both[:, 0], both[:, 1]
    shape = (pages, H, P, D) if layout == "hnd" else (pages, P, H, D)
    a, b = (torch.full(shape, fill, dtype=torch.bfloat16, device=device) for _ in range(2))
    return (a, b) if layout == "hnd" else (a.permute(0, 2, 1, 3), b.permute(0, 2, 1, 3))


def scatter(pool, table, lens, P, dense):
    """dense [B, H, S, D] into the pages of each request's first lens[b] tokens."""
    for b, n in enumerate(lens):
        for i in range(up(int(n), P)):
            m = min(P, int(n) - i * P)
            pool[int(table[b, i]), :, :m] = dense[b, :, i * P:i * P + m].to(pool.device)


# ------------------------------------------------------------------------------------------------
# attention
# ------------------------------------------------------------------------------------------------
def attention_ref(q, k, v, lens, scale, causal):
    """(o, lse, a) in FP64: the output, its log-sum-exp and sum_j p_j |v_j|, which bounds what roundings of p
    can change.  q [B, Hq, Sq, D], k, v [B, Hkv, S, D] on the CPU."""
    B, Hq, Sq, D = q.shape
    g = Hq // k.shape[1]
    o, a = torch.zeros(B, Hq, Sq, D, dtype=torch.float64), torch.zeros(B, Hq, Sq, D, dtype=torch.float64)
    lse = torch.full((B, Hq, Sq), -math.inf, dtype=torch.float64)
    for b in range(B):
        for s in range(Sq):
            n = max(0, int(lens[b]) - Sq + 1 + s) if causal else int(lens[b])
            if n == 0:
                continue
            kk = k[b, :, :n].double().repeat_interleave(g, 0)
            vv = v[b, :, :n].double().repeat_interleave(g, 0)
            x = torch.einsum("hd,hnd->hn", q[b, :, s].double(), kk) * scale
            lse[b, :, s] = torch.logsumexp(x, -1)
            p = torch.softmax(x, -1)
            o[b, :, s] = torch.einsum("hn,hnd->hd", p, vv)
            a[b, :, s] = torch.einsum("hn,hnd->hd", p, vv.abs())
    return o, lse, a


# Tolerance of the output, from the roundings that the kernel makes: each p_j to two BF16 (what the first leaves,
# 2^-8 of p_j, rounded to half a step of its own: 2^-16 a in all), the output to BF16 (2^-8 |o|), and FP32 sums.
# The scores' FP32 sums over D <= 128 features err by at most 128 * 2^-23 * |q|.|k| scale <= 2^-16 * 16 for unit
# normals (|q|.|k| scale < 16 at D <= 128), 2^-12 of each p_j; the sums over keys, split by tiles of 128, by less
# than 2^-13 a.  So a (2^-12 + 2^-13 + 2^-16) + 2^-8 |o|, and for the log-sum-exp 2^-12 + a few 2^-22 |lse|.
def check_attention(out, lse, ref, bf16=True, what=""):
    o, l, a = ref
    out = out.double().cpu().view_as(o)
    assert torch.isfinite(out).all(), f"{what}: non-finite output"
    tol = a * (2.0 ** -12 + 2.0 ** -13 + 2.0 ** -16) + (2.0 ** -8 * o.abs() if bf16 else 0)
    over = (out - o).abs() - tol
    assert over.max() <= 0, f"{what}: off by {(out - o).abs().flatten()[over.argmax()]:.3e}, {over.max():.3e} too much"
    if lse is not None:
        lse = lse.double().cpu().view_as(l)
        none = l == -math.inf
        assert torch.equal(lse == -math.inf, none), f"{what}: empty rows"
        d = (lse - l)[~none].abs()
        assert d.numel() == 0 or (d - 2.0 ** -12 - 2.0 ** -20 * l[~none].abs()).max() <= 0, f"{what}: lse off by {d.max():.3e}"
