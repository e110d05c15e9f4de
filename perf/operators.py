"""The operators of the paged key/value cache and their measured cases.

Three operators serve requests of growing lengths:

  table   pages handed out and taken back, block table, positions and slots from request lengths;
  append  RMS norm of each query and key head, position rotation, and the store of k and v in the cache;
  attend  attention of each request's last tokens over the pages of the cache.

run() computes a case either through the library's entry points (own) or in plain torch operations in
32 bits.  exact() states the same results in 64 bits, from the definitions.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # a decoding step of a small batch: one token each, now and then a new page
        dict(name="table decode B8", op="table", B=8, ctx=4096, new=1, page=16, done=0, pad=0, lens=11),
        # a decoding step of a large batch, padded to its captured size, an eighth of the requests finished
        dict(name="table decode B256 padded", op="table", B=256, ctx=8191, new=1, page=64, done=32, pad=77, lens=12),
        # prompts of differing lengths that join a batch at once
        dict(name="table prompts B32", op="table", B=32, ctx=2000, new=8191, page=16, done=0, pad=501, lens=13),
        # a decoding step of a small batch (grouped heads, norm and full rotation)
        dict(name="append decode T8 D128", op="append", T=8, Hq=32, Hkv=8, D=128, rope=128, pairs=False, norm=True, page=16,
             layout="hnd", Sq=1, pad=0, pool=4096),
        # four proposed tokens for each of 33 requests, padded; half of each head rotated in neighbouring pairs, no norm
        dict(name="append verify T132 D64", op="append", T=132, Hq=16, Hkv=4, D=64, rope=32, pairs=True, norm=False, page=32,
             layout="nhd", Sq=4, pad=28, pool=8192),
        # a long prompt, or a chunk of several
        dict(name="append prompt T8192 D128", op="append", T=8192, Hq=32, Hkv=8, D=128, rope=128, pairs=False, norm=True, page=64,
             layout="hnd", Sq=1, pad=0, pool=16384),
        # one short request: latency
        dict(name="attend B1 500 keys", op="attend", B=1, Hq=32, Hkv=8, Sq=1, D=128, most=500, least=500, page=16, layout="hnd",
             causal=False, lens=21),
        # the decode workload of the library's benchmark, paged
        dict(name="attend B8 H32 4096 keys", op="attend", B=8, Hq=32, Hkv=32, Sq=1, D=128, most=4096, least=4096, page=64,
             layout="hnd", causal=False, lens=22),
        # proposed tokens of a batch with empty slots, tokens outermost in a page, odd lengths
        dict(name="attend verify B17 Sq4 D64", op="attend", B=17, Hq=16, Hkv=4, Sq=4, D=64, most=5001, least=0, page=32,
             layout="nhd", causal=True, lens=23),
        # one long request, split over its length
        dict(name="attend B1 131071 keys", op="attend", B=1, Hq=32, Hkv=8, Sq=1, D=128, most=131071, least=131071, page=64,
             layout="hnd", causal=False, lens=24),
        # the ragged grouped-query workload of the library's benchmark, in small pages
        dict(name="attend ragged B64 32768 keys", op="attend", B=64, Hq=32, Hkv=8, Sq=1, D=128, most=32768, least=1, page=16,
             layout="hnd", causal=False, lens=25),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["table", "append", "append", "attend", "attend", "attend"])
    page = rng.choice([8, 16, 32, 48, 64, 128, 256])
    layout = rng.choice(["hnd", "nhd"])
    if op == "table":
        B = _log(rng, 1, 1024)
        new = 1 if rng.random() < 0.5 else _log(rng, 2, max(2, min(8191, 120000 // B)))
        return dict(op=op, B=B, ctx=_log(rng, 1, 16384), new=new, page=page, done=rng.randint(0, B // 4), pad=rng.choice([0, rng.randint(0, 600)]),
                    lens=rng.randint(0, 1 << 30))
    Hkv, D = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([64, 128])
    if op == "append":
        group = rng.choice([1, 2, 3, 4, 8])
        Sq = rng.choice([1, 1, 2, 4])
        most = 8192 * 48 * 128 // ((group + 2) * Hkv * D)
        T = Sq * max(1, _log(rng, 1, min(8192, most)) // Sq)
        return dict(op=op, T=T, Hq=Hkv * group, Hkv=Hkv, D=D, rope=rng.choice([0, 16, 32, D // 2, D, D]), pairs=rng.random() < 0.4,
                    norm=rng.random() < 0.7, page=page, layout=layout, Sq=Sq, pad=Sq * rng.choice([0, 0, rng.randint(0, 9)]),
                    pool=T + rng.randint(1, 4096))
    Sq = rng.choice([1, 1, 1, 2, 4])
    group = rng.choice([g for g in (1, 2, 3, 4, 7, 8, 16) if g * Sq <= 16])
    B = _log(rng, 1, 128)
    room = 64 * 32768 // 2 * 8 * 128 // (B * Hkv * D)     # mean keys of a request that cost as much as the largest case
    most = _log(rng, 1, max(2, min(131071, 2 * room)))
    least = most if rng.random() < 0.3 and most <= room else 0
    return dict(op=op, B=B, Hq=Hkv * group, Hkv=Hkv, Sq=Sq, D=D, most=most, least=least, page=page, layout=layout,
                causal=Sq > 1 and rng.random() < 0.7, lens=rng.randint(0, 1 << 30))


def _up(n, m):
    return -(-n // m)


def _table_lens(c):
    """(tokens held, tokens to come or -1) of each request."""
    r = random.Random(c["lens"])
    ctx = [r.randint(0, c["ctx"]) for _ in range(c["B"])]
    new = [c["new"] if c["new"] == 1 else r.randint(1, c["new"]) for _ in range(c["B"])]
    for b in r.sample(range(c["B"]), c["done"]):
        new[b] = -1
    return ctx, new


def _attend_lens(c):
    r = random.Random(c["lens"])
    return [r.randint(c["least"], c["most"]) for _ in range(c["B"])]


def work(case):
    c = case
    if c["op"] == "table":
        ctx, new = _table_lens(c)
        P = c["page"]
        T = sum(n for n in new if n > 0) + c["pad"]
        back = sum(_up(x, P) for x, n in zip(ctx, new) if n < 0)
        need = sum(_up(x + n, P) - _up(x, P) for x, n in zip(ctx, new) if n >= 0)
        part = sum(1 for x, n in zip(ctx, new) if n > 0 and x % P)       # pages a request goes on filling
        return {"bytes": 12 * T + 16 * c["B"] + 8 * (back + need) + 4 * part + 12, "flops": 0}
    if c["op"] == "append":
        rows = c["T"] * (c["Hq"] + 2 * c["Hkv"])
        qk = c["T"] * (c["Hq"] + c["Hkv"]) * c["D"]
        table = min(c["T"], c["pool"]) * c["rope"] * 4
        return {"bytes": 4 * rows * c["D"] + 12 * c["T"] + 8 * c["pad"] + table + (4 * c["D"] if c["norm"] else 0),
                "flops": qk * ((4 if c["norm"] else 0) + 3)}
    lens = _attend_lens(c)
    q = c["B"] * c["Hq"] * c["Sq"]
    pages = sum(_up(n, c["page"]) for n in lens)
    return {"bytes": 4 * sum(lens) * c["Hkv"] * c["D"] + 4 * q * c["D"] + 4 * q + 4 * pages + 4 * c["B"],
            "flops": 4 * sum(lens) * c["Hq"] * c["Sq"] * c["D"]}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _pool(c, pages, g):
    """K and V pools of `pages` pages, logical order [pages][Hkv][page][D]."""
    H, P, D = c["Hkv"], c["page"], c["D"]
    shape = (pages, H, P, D) if c["layout"] == "hnd" else (pages, P, H, D)
    pools = [torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=g) for _ in range(2)]
    return pools if c["layout"] == "hnd" else [p.permute(0, 2, 1, 3) for p in pools]


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c = case
    g = torch.Generator(DEV).manual_seed(seed)
    s = {"case": c}
    if c["op"] == "table":
        ctx, new = _table_lens(c)
        P, B = c["page"], c["B"]
        held = [_up(x, P) for x in ctx]
        need = sum(_up(x + n, P) - h for x, n, h in zip(ctx, new, held) if n >= 0)
        width = max(_up(x + max(n, 0), P) for x, n in zip(ctx, new)) + 3
        N = sum(held) + need + 100
        ids = torch.randperm(N, generator=g, device=DEV, dtype=torch.int32)
        first = [0] * B
        for b in range(1, B):
            first[b] = first[b - 1] + held[b - 1]
        col = torch.arange(width, device=DEV)[None, :]
        at = (_int32(first)[:, None] + col).clamp(max=N - 1).long()
        s["table"] = torch.where(col < _int32(held)[:, None], ids[at], -1).to(torch.int32).contiguous()
        n = N - sum(held)
        s["free"] = torch.full((N,), -1, dtype=torch.int32, device=DEV)
        s["free"][:n] = ids[sum(held):]
        s["n"] = _int32([n])
        s["ctx"], s["new"] = _int32(ctx), _int32(new)
        T = sum(x for x in new if x > 0) + c["pad"]
        s["seqlens"], s["cu"], s["n_out"] = _int32([0] * B), _int32([0] * (B + 1)), _int32([0])
        s["positions"] = torch.zeros(T, dtype=torch.int32, device=DEV)
        s["slots"] = torch.zeros(T, dtype=torch.int64, device=DEV)
        return s
    H, D = c["Hkv"], c["D"]
    if c["op"] == "append":
        T, Hq = c["T"] + c["pad"], c["Hq"]
        pages = _up(c["pool"], c["page"])
        s["k_pool"], s["v_pool"] = _pool(c, pages, g)
        # one row of the projection's output for each token: queries, keys, values
        qkv = torch.empty(T, Hq + 2 * H, D, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        s["wq"] = s["wk"] = None
        if c["norm"]:
            s["wq"], s["wk"] = [(1 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16) for _ in range(2)]
        slots = torch.randperm(pages * c["page"], generator=g, device=DEV)[:c["T"]]
        s["slots"] = torch.cat([slots, slots.new_full((c["pad"],), -1)])
        s["positions"] = torch.cat([torch.randint(0, c["pool"], (c["T"],), generator=g, device=DEV), slots.new_zeros(c["pad"])]).int()
        s["cos_sin"] = None
        if c["rope"]:
            freq = 10000.0 ** (-torch.arange(0, c["rope"], 2, device=DEV, dtype=torch.float64) / c["rope"])
            angle = torch.arange(c["pool"], device=DEV, dtype=torch.float64)[:, None] * freq
            s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["q_out"] = torch.zeros(T // c["Sq"], Hq, c["Sq"], D, dtype=torch.bfloat16, device=DEV)
        return s
    lens, P, B = _attend_lens(c), c["page"], c["B"]
    held = [_up(n, P) for n in lens]
    pages = sum(held) + 7
    s["k_pool"], s["v_pool"] = _pool(c, pages, g)
    ids = torch.randperm(pages, generator=g, device=DEV, dtype=torch.int32)
    width = max(held) + 2
    first = [0] * B
    for b in range(1, B):
        first[b] = first[b - 1] + held[b - 1]
    col = torch.arange(width, device=DEV)[None, :]
    at = (_int32(first)[:, None] + col).clamp(max=pages - 1).long()
    s["table"] = torch.where(col < _int32(held)[:, None], ids[at], -1).to(torch.int32).contiguous()
    s["seqlens"] = _int32(lens)
    s["q"] = torch.empty(B, c["Hq"], c["Sq"], D, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(B, c["Hq"], c["Sq"], dtype=torch.float32, device=DEV)
    return s


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"table": _own_table, "append": _own_append, "attend": _own_attend}[op](state)
    return {"table": _plain_table, "append": _plain_append, "attend": _plain_attend}[op](state)


def _table_outputs(s):
    return {k: s[k] for k in ("table", "free", "n_out", "seqlens", "cu", "positions", "slots")}


def _own_table(s):
    import attention_tensor_cores_gb300 as F
    F.fmha_page_table(s["ctx"], s["new"], s["case"]["page"], s["free"], s["n"], s["table"], s["seqlens"], s["cu"], s["positions"],
                      s["slots"], s["n_out"])
    return _table_outputs(s)


def _own_append(s):
    import attention_tensor_cores_gb300 as F
    if "cache" not in s:
        s["cache"] = F.make_kv_cache(s["k_pool"], s["v_pool"])
    F.fmha_rope_append(s["q"], s["k"], s["v"], s["wq"], s["wk"], 1e-6, s["cos_sin"], s["positions"], s["slots"], s["q_out"], s["cache"],
                       interleaved=s["case"]["pairs"])
    return {"q": s["q_out"], "k": s["k_pool"], "v": s["v_pool"]}


def _own_attend(s):
    import attention_tensor_cores_gb300 as F
    c = s["case"]
    if "cache" not in s:     # what a program keeps from step to step: the cache's descriptor, the options and their workspace
        s["cache"] = F.make_kv_cache(s["k_pool"], s["v_pool"])
        need = F.fmha_paged_workspace_size(c["B"], c["Hq"], c["Sq"], s["cache"], F.make_opts(causal=c["causal"]))
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)
        s["opts"] = F.make_opts(workspace=s["workspace"], causal=c["causal"])
    F.fmha_fwd_paged(s["q"], s["cache"], s["table"], s["seqlens"], s["out"], s["lse"], c["D"] ** -0.5, s["opts"])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_table(s):
    P, table, free = s["case"]["page"], s["table"], s["free"]
    B, width = table.shape
    ctx, new, n = s["ctx"].long(), s["new"].long(), s["n"].long()
    done, add = new < 0, new.clamp(min=0)
    held = (ctx + P - 1) // P
    back = torch.where(done, held, 0)
    need = torch.where(done, 0, (ctx + add + P - 1) // P - held)
    back_end, need_end, cu = back.cumsum(0), need.cumsum(0), add.cumsum(0)
    # finished requests' pages onto the stack, in request order
    r = torch.arange(free.numel(), device=DEV) - n
    b = torch.searchsorted(back_end, r.clamp(min=0), right=True).clamp(max=B - 1)
    given = table[b, (r - (back_end - back)[b]).clamp(0, width - 1)]
    s["free"] = free = torch.where((r >= 0) & (r < back_end[-1]), given, free)
    # new pages from its top, in request order
    top = n + back_end[-1]
    j = torch.arange(width, device=DEV)[None, :] - held[:, None]
    at = (top - 1 - (need_end - need)[:, None] - j).clamp(0, free.numel() - 1)
    s["table"] = table = torch.where((j >= 0) & (j < need[:, None]), free[at], table)
    # each new token's request, position and slot
    t = torch.arange(s["slots"].numel(), device=DEV)
    b = torch.searchsorted(cu, t, right=True).clamp(max=B - 1)
    real = t < cu[-1]
    pos = torch.where(real, ctx[b] + t - (cu - add)[b], 0)
    slot = table[b, (pos // P).clamp(max=width - 1)].long() * P + pos % P
    s["slots"] = torch.where(real, slot, -1)
    s["positions"] = pos.int()
    s["seqlens"] = torch.where(done, 0, ctx + add).int()
    s["cu"] = torch.cat([cu.new_zeros(1), cu]).int()
    s["n_out"] = (top - need_end[-1]).int()
    return _table_outputs(s)


def _plain_norm(x, w):
    y = x.float()
    return y if w is None else y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()


def _plain_turn(y, cos_sin, pos, pairs):
    if cos_sin is None:
        return y
    R = cos_sin.shape[1]
    c, d = cos_sin[pos][:, None, :R // 2], cos_sin[pos][:, None, R // 2:]
    if pairs:
        a, b = y[..., 0:R:2], y[..., 1:R:2]
        turned = torch.stack([a * c - b * d, b * c + a * d], -1).flatten(-2)
    else:
        a, b = y[..., :R // 2], y[..., R // 2:R]
        turned = torch.cat([a * c - b * d, b * c + a * d], -1)
    return torch.cat([turned, y[..., R:]], -1)


def _plain_append(s):
    c = s["case"]
    T, P, Sq = c["T"], c["page"], c["Sq"]
    pos, slots = s["positions"][:T].long(), s["slots"][:T]
    q = _plain_turn(_plain_norm(s["q"][:T], s["wq"]), s["cos_sin"], pos, c["pairs"]).to(torch.bfloat16)
    k = _plain_turn(_plain_norm(s["k"][:T], s["wk"]), s["cos_sin"], pos, c["pairs"]).to(torch.bfloat16)
    s["q_out"][:T // Sq] = q.view(T // Sq, Sq, c["Hq"], c["D"]).transpose(1, 2)
    s["k_pool"][slots // P, :, slots % P] = k
    s["v_pool"][slots // P, :, slots % P] = s["v"][:T]
    return {"q": s["q_out"], "k": s["k_pool"], "v": s["v_pool"]}


def _plain_attend(s):
    c = s["case"]
    B, H, Sq, D = c["B"], c["Hkv"], c["Sq"], c["D"]
    pages = s["table"].clamp(min=0).long()
    n = s["seqlens"][:, None, None, None]
    kv = [p[pages].permute(0, 2, 1, 3, 4).reshape(B, H, -1, D).float() for p in (s["k_pool"], s["v_pool"])]
    j = torch.arange(kv[0].shape[2], device=DEV)
    q = s["q"].view(B, H, -1, D).float()                       # columns of a key/value head: its query heads' tokens
    last = torch.arange(q.shape[2], device=DEV)[:, None] % Sq - Sq if c["causal"] else -1
    seen = j <= n + last
    x = torch.where(seen, torch.matmul(q, kv[0].transpose(-1, -2)) * D ** -0.5, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = torch.exp(x - m)
    l = e.sum(-1, keepdim=True)
    o = torch.matmul(e, kv[1]) / torch.where(l == 0, 1.0, l)
    s["out"] = o.to(torch.bfloat16).view_as(s["q"])
    s["lse"] = (torch.log(l) + m).view_as(s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------------------------------------
# the definitions, in 64 bits
# ------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"table": _exact_table, "append": _exact_append, "attend": _exact_attend}[case["op"]](s)


def _exact_table(s):
    P = s["case"]["page"]
    table, free = s["table"].cpu().clone(), s["free"].cpu().clone()
    ctx, new, n = s["ctx"].tolist(), s["new"].tolist(), int(s["n"])
    T = s["slots"].numel()
    for b, x in enumerate(ctx):
        if new[b] < 0:
            k = _up(x, P)
            free[n:n + k] = table[b, :k]
            n += k
    cu, pos, slots, lens = [0], [], [], []
    for b, x in enumerate(ctx):
        add = max(new[b], 0)
        if new[b] >= 0:
            for j in range(_up(x, P), _up(x + add, P)):
                n -= 1
                table[b, j] = free[n]
        at = torch.arange(x, x + add)
        pos.append(at)
        slots.append(table[b][at // P].long() * P + at % P)
        cu.append(cu[-1] + add)
        lens.append(0 if new[b] < 0 else x + add)
    pad = T - cu[-1]
    pos.append(torch.zeros(pad, dtype=torch.int64))
    slots.append(torch.full((pad,), -1))
    return {"table": table, "free": free, "n_out": torch.tensor([n], dtype=torch.int32), "seqlens": torch.tensor(lens, dtype=torch.int32),
            "cu": torch.tensor(cu, dtype=torch.int32), "positions": torch.cat(pos).int(), "slots": torch.cat(slots)}


def _exact_append(s):
    c = s["case"]
    T, P, Sq, R = c["T"], c["page"], c["Sq"], c["rope"]

    def head(x, w):
        y = x[:T].double()
        if w is not None:
            y = y / (y.pow(2).sum(-1, keepdim=True) / c["D"] + 1e-6).sqrt() * w.double()
        if R:
            row = s["cos_sin"].double()[s["positions"][:T].long()].unsqueeze(1)
            z = torch.complex(row[..., :R // 2], row[..., R // 2:])
            i = torch.arange(R // 2, device=y.device)
            i, k = (2 * i, 2 * i + 1) if c["pairs"] else (i, i + R // 2)
            turned = torch.complex(y[..., i], y[..., k]) * z
            y[..., i], y[..., k] = turned.real, turned.imag
        return y

    q = s["q_out"].double()
    for i in range(Sq):
        q[:T // Sq, :, i] = head(s["q"], s["wq"])[i::Sq]
    pools = []
    for pool, new in ((s["k_pool"], head(s["k"], s["wk"])), (s["v_pool"], s["v"][:T].double())):
        rows = pool.double().transpose(1, 2).reshape(-1, c["Hkv"], c["D"])
        rows[s["slots"][:T]] = new
        pools.append(rows.view(-1, P, c["Hkv"], c["D"]).transpose(1, 2))
    return {"q": q, "k": pools[0], "v": pools[1]}


def _exact_attend(s):
    c = s["case"]
    P, H, Sq, D = c["page"], c["Hkv"], c["Sq"], c["D"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=s["q"].device)
    for b, n in enumerate(s["seqlens"].tolist()):
        page = s["table"][b, torch.arange(n, device=out.device) // P].long()
        at = torch.arange(n, device=out.device) % P
        k, v = s["k_pool"][page, :, at].double(), s["v_pool"][page, :, at].double()     # [n][Hkv][D]
        for i in range(Sq):
            see = max(0, n - Sq + 1 + i) if c["causal"] else n
            if see:
                q = s["q"][b, :, i].double().view(H, -1, D)
                x = torch.einsum("hgd,nhd->hgn", q, k[:see]) / math.sqrt(D)
                lse[b, :, i] = torch.logsumexp(x, -1).flatten()
                out[b, :, i] = torch.einsum("hgn,nhd->hgd", torch.softmax(x, -1), v[:see]).reshape(-1, D)
    return {"out": out, "lse": lse}
