"""The operators of pages that requests share, and their measured cases.

Several continuations of one prompt (parallel samples, beams, requests behind one system prompt) hold the
pages of their common beginning together.  Four operators serve them on the paged key/value cache:

  attend   attention of groups of requests whose first pages are the same
  fork     next step's requests as children of this step's: block table, freed pages, pages to be copied
  copy     pages copied inside the pools of all layers
  compact  used pages to the low ids: block table, moves and the stack of free pages

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
        # four beams of one request: latency
        dict(name="attend 4 beams 1000 keys", op="attend", groups=1, members=4, Hq=32, Hkv=8, Sq=1, D=128, most=900, least=900, own=100,
             page=16, layout="hnd", causal=False, empty=0, lens=41),
        # sixteen requests of four beams each, proposed tokens, tokens outermost in a page, odd lengths, empty slots
        dict(name="attend 16x4 verify Sq4 D64", op="attend", groups=16, members=4, Hq=16, Hkv=4, Sq=4, D=64, most=5001, least=100, own=333,
             page=32, layout="nhd", causal=True, empty=3, lens=42),
        # many samples of one long prompt
        dict(name="attend 64 samples 8192 prompt", op="attend", groups=1, members=64, Hq=32, Hkv=8, Sq=1, D=128, most=8192, least=8192,
             own=1000, page=64, layout="hnd", causal=False, empty=0, lens=43),
        # a batch of mixed lengths behind four long common documents
        dict(name="attend 4x64 32768 prefix", op="attend", groups=4, members=64, Hq=32, Hkv=8, Sq=1, D=128, most=32768, least=32768, own=2000,
             page=64, layout="hnd", causal=False, empty=0, lens=44),
        # a step of beam search: two requests of four beams
        dict(name="fork 2x4 beams", op="fork", groups=2, members=4, into=4, prefix=2000, own=100, page=16, done=0, spare=16, lens=51),
        # one prompt forked into 64 samples
        dict(name="fork 1 into 64", op="fork", groups=1, members=1, into=64, prefix=5001, own=0, page=32, done=0, spare=100, lens=52),
        # a step of beam search over a large batch, an eighth of the requests finished
        dict(name="fork 128x4 beams 16384 keys", op="fork", groups=128, members=4, into=4, prefix=15000, own=1384, page=64, done=16, spare=1000,
             lens=53),
        # the partly filled pages of a beam search's step, in every layer
        dict(name="copy 64 partial 32 layers", op="copy", pairs=64, count=64, layers=32, Hkv=8, D=128, page=16, layout="hnd", partial=True,
             skip=40, pages=256, lens=61),
        # whole pages after a compaction, tokens outermost; the list is longer than what is to be moved
        dict(name="copy 1501 pages 12 layers", op="copy", pairs=2500, count=1501, layers=12, Hkv=8, D=128, page=64, layout="nhd", partial=False,
             skip=0, pages=5000, lens=62),
        # a small pool, half in use
        dict(name="compact 1000 pages", op="compact", pages=1000, B=8, held=64, width=70, lens=71),
        # a pool of small pages that fills the device
        dict(name="compact 300000 pages", op="compact", pages=300000, B=512, held=400, width=1024, lens=72),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "fork", "copy", "compact"])
    page = rng.choice([8, 16, 32, 48, 64, 128])
    layout = rng.choice(["hnd", "nhd"])
    lens = rng.randint(0, 1 << 30)
    if op == "attend":
        Hkv, D, Sq = rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 128]), rng.choice([1, 1, 1, 2, 4])
        group = rng.choice([g for g in (1, 2, 3, 4, 7, 8, 16) if g * Sq <= 16])
        groups, members = _log(rng, 1, 16), _log(rng, 1, 64)
        # no more keys to read, nor products to take, than in the largest case
        part = groups * members * D * max(Hkv * 32, Hkv * group * Sq * 8)
        room, own_room = (256 * n * 128 * 8 * 32 // part for n in (32768, 2000))
        most = _log(rng, 1, max(1, min(32768, room)))
        return dict(op=op, groups=groups, members=members, Hq=Hkv * group, Hkv=Hkv, Sq=Sq, D=D, most=most, least=rng.choice([0, most // 2, most]),
                    own=_log(rng, 1, max(1, min(2000, own_room))), page=page, layout=layout, causal=Sq > 1 and rng.random() < 0.7,
                    empty=rng.choice([0, 0, rng.randint(0, groups * members // 4)]), lens=lens)
    if op == "fork":
        groups, members = _log(rng, 1, 128), rng.choice([1, 2, 4, 4])
        return dict(op=op, groups=groups, members=members, into=rng.choice([members, members, rng.randint(1, min(64, 512 // groups))]),
                    prefix=_log(rng, 1, 234 * page), own=rng.randint(0, 21 * page), page=page, done=rng.randint(0, groups // 2),
                    spare=rng.randint(0, 500), lens=lens)
    if op == "copy":
        Hkv, D, layers = rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 128]), rng.randint(1, 32)
        most = 3000 * 12 * 64 * 8 * 128 // (layers * page * Hkv * D)     # twice the pages that the largest case copies
        pages = _log(rng, 8, max(9, min(5000, most)))
        pairs = rng.randint(1, min(1500, pages // 2))
        return dict(op=op, pairs=pairs, count=rng.randint(0, pairs), layers=layers, Hkv=Hkv, D=D, page=page, layout=layout,
                    partial=rng.random() < 0.5, skip=rng.randint(0, pairs // 2), pages=pages, lens=lens)
    B = _log(rng, 1, 512)
    held = _log(rng, 1, 400)
    used = B * held
    return dict(op=op, pages=min(300000, used + _log(rng, 1, 100000)) if used < 300000 else 300000, B=B, held=min(held, 300000 // B),
                width=held + rng.randint(0, 200), lens=lens)


def _up(n, m):
    return -(-n // m)


def _attend_lens(c):
    """Tokens of each request, and of each group's common pages."""
    r = random.Random(c["lens"])
    prefix = [r.randint(c["least"], c["most"]) // c["page"] * c["page"] for _ in range(c["groups"])]
    lens = [p + r.randint(1, c["own"]) for p in prefix for _ in range(c["members"])]
    for b in r.sample(range(len(lens)), c["empty"]):
        lens[b] = 0
    return lens, prefix


def _fork_plan(c):
    """(tokens of each request, common tokens of each group, parent of each child)."""
    r = random.Random(c["lens"])
    prefix = [r.randint(1, c["prefix"]) for _ in range(c["groups"])]
    lens = [p + r.randint(0, c["own"]) for p in prefix for _ in range(c["members"])]
    done = set(r.sample(range(c["groups"]), c["done"]))
    parents = [-1 if g in done else g * c["members"] + r.randrange(c["members"]) for g in range(c["groups"]) for _ in range(c["into"])]
    return lens, prefix, parents


def _copy_plan(c):
    """(source, destination, tokens) of each pair; a skipped pair is all -1."""
    r = random.Random(c["lens"])
    ids = r.sample(range(c["pages"]), 2 * c["pairs"])
    pairs = [[ids[2 * i], ids[2 * i + 1], r.randint(1, c["page"]) if c["partial"] else c["page"]] for i in range(c["pairs"])]
    for i in r.sample(range(c["pairs"]), c["skip"]):
        pairs[i] = [-1, -1, 0]
    return pairs


def work(case):
    c = case
    if c["op"] == "attend":
        lens, prefix = _attend_lens(c)
        m = c["members"]
        shared = own_keys = 0
        for g, p in enumerate(prefix):
            of = [n for n in lens[g * m:(g + 1) * m] if n]
            shared += p if of else 0
            own_keys += sum(n - p for n in of)
        rows = len(lens) * c["Hq"] * c["Sq"]
        pages = sum(_up(n, c["page"]) for n in lens)
        return {"bytes": 4 * (shared + own_keys) * c["Hkv"] * c["D"] + 4 * rows * c["D"] + 4 * rows + 4 * pages + 4 * len(lens) + 8 * c["groups"],
                "flops": 4 * sum(lens) * c["Hq"] * c["Sq"] * c["D"]}
    if c["op"] == "fork":
        lens, _, parents = _fork_plan(c)
        used = {p for p in parents if p >= 0}
        read = sum(_up(n, c["page"]) for n in lens)
        written = sum(_up(lens[p], c["page"]) for p in parents if p >= 0)
        own_pages = sum(_up(n, c["page"]) for i, n in enumerate(lens) if i not in used)
        return {"bytes": 4 * (read + written) + 4 * own_pages + 4 * len(lens) + 20 * len(parents) + 8, "flops": 0}
    if c["op"] == "copy":
        tokens = sum(t for _, _, t in _copy_plan(c)[:c["count"]])
        return {"bytes": 2 * 2 * 2 * tokens * c["Hkv"] * c["D"] * c["layers"] + 12 * c["count"], "flops": 0}
    N, held = c["pages"], c["B"] * c["held"]
    free = N - held
    return {"bytes": 4 * free + 4 * N + 8 * (N // 2) + 8 * held + 4 * free + 4 * c["B"] + 8, "flops": 0}


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


def _shared_tables(lens, prefix, members, P, spare, g):
    """Block table of groups that hold the full pages of their first `prefix` tokens together, and the ids left over.
    Each request has a partly filled page and what follows to itself."""
    width = max(_up(n, P) for n in lens) + 2
    common = [p // P for p in prefix]
    rows, at = [], 0
    for i, p in enumerate(common):
        rows.append((at, p))
        at += p
    place = torch.full((len(lens), width), -1, dtype=torch.int64)
    for b, n in enumerate(lens):
        first, k = rows[b // members]
        k = min(k, _up(n, P))
        place[b, :k] = torch.arange(first, first + k)
        rest = _up(n, P) - k
        place[b, k:k + rest] = torch.arange(at, at + rest)
        at += rest
    ids = torch.randperm(at + spare, generator=g, device=DEV, dtype=torch.int32)
    place = place.to(DEV)
    return torch.where(place >= 0, ids[place.clamp(min=0)], -1).to(torch.int32).contiguous(), ids, at


def prepare(case, seed):
    c = case
    g = torch.Generator(DEV).manual_seed(seed)
    s = {"case": c}
    if c["op"] == "attend":
        lens, prefix = _attend_lens(c)
        s["table"], ids, _ = _shared_tables(lens, prefix, c["members"], c["page"], 7, g)
        s["k_pool"], s["v_pool"] = _pool(c, ids.numel(), g)
        B = len(lens)
        s["seqlens"], s["prefix"] = _int32(lens), _int32(prefix)
        s["cu"] = _int32([i * c["members"] for i in range(c["groups"] + 1)])
        s["q"] = torch.empty(B, c["Hq"], c["Sq"], c["D"], dtype=torch.bfloat16, device=DEV).normal_(generator=g)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(B, c["Hq"], c["Sq"], dtype=torch.float32, device=DEV)
        return s
    if c["op"] == "fork":
        lens, prefix, parents = _fork_plan(c)
        B = len(parents)
        s["table"], ids, used = _shared_tables(lens, prefix, c["members"], c["page"], c["spare"] + B, g)
        N = ids.numel()
        s["free"] = torch.full((N,), -1, dtype=torch.int32, device=DEV)
        s["free"][:N - used] = ids[used:]
        s["n"], s["parents"], s["ctx"] = _int32([N - used]), _int32(parents), _int32(lens)
        s["new_table"] = torch.full((B, s["table"].shape[1]), -1, dtype=torch.int32, device=DEV)
        for name in ("seqlens", "src", "dst", "tokens"):
            s[name] = torch.zeros(B, dtype=torch.int32, device=DEV)
        s["n_out"] = _int32([0])
        return s
    if c["op"] == "copy":
        s["pools"] = [_pool(c, c["pages"], g) for _ in range(c["layers"])]
        pairs = _int32(_copy_plan(c))
        s["src"], s["dst"], s["tokens"] = [pairs[:, i].contiguous() for i in range(3)]
        s["count"] = _int32([c["count"]])
        return s
    N, B, held, width = c["pages"], c["B"], c["held"], c["width"]
    ids = torch.randperm(N, generator=g, device=DEV, dtype=torch.int32)
    s["table"] = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    s["table"][:, :held] = ids[:B * held].view(B, held)
    n = N - B * held
    s["free"] = torch.full((N,), -1, dtype=torch.int32, device=DEV)
    s["free"][:n] = ids[B * held:]
    s["n"] = _int32([n])
    r = random.Random(c["lens"])
    s["seqlens"] = _int32([held * 16 - r.randint(0, 15) for _ in range(B)])      # pages of 16 tokens
    s["new_table"] = torch.full_like(s["table"], -1)
    s["new_ids"], s["free_out"] = torch.zeros_like(s["free"]), torch.full_like(s["free"], -1)
    s["src"], s["dst"] = (torch.zeros(N // 2, dtype=torch.int32, device=DEV) for _ in range(2))
    s["moves"] = _int32([0])
    return s


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"attend": _own_attend, "fork": _own_fork, "copy": _own_copy, "compact": _own_compact}[op](state)
    return {"attend": _plain_attend, "fork": _plain_fork, "copy": _plain_copy, "compact": _plain_compact}[op](state)


FORK = ("new_table", "seqlens", "src", "dst", "tokens", "free", "n_out")
COMPACT = ("new_ids", "new_table", "src", "dst", "moves", "free_out")


def _own_attend(s):
    import attention_tensor_cores_gb300 as F
    c = s["case"]
    if "cache" not in s:     # what a program keeps from step to step: the cache's descriptor, the options and their workspace
        s["cache"] = F.make_kv_cache(s["k_pool"], s["v_pool"])
        need = F.fmha_prefix_workspace_size(s["q"].shape[0], c["Hq"], c["Sq"], s["cache"], F.make_opts(causal=c["causal"]))
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)
        s["opts"] = F.make_opts(workspace=s["workspace"], causal=c["causal"])
    F.fmha_fwd_prefix(s["q"], s["cache"], s["table"], s["seqlens"], s["cu"], s["prefix"], s["out"], s["lse"], c["D"] ** -0.5, s["opts"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_fork(s):
    import attention_tensor_cores_gb300 as F
    F.fmha_page_fork(s["parents"], s["ctx"], s["case"]["page"], s["table"], s["free"], s["n"], s["new_table"], s["seqlens"], s["src"],
                     s["dst"], s["tokens"], s["n_out"])
    return {k: s[k] for k in FORK}


def _own_copy(s):
    import attention_tensor_cores_gb300 as F
    if "caches" not in s:
        s["caches"] = [F.make_kv_cache(k, v) for k, v in s["pools"]]
    F.fmha_page_copy(s["caches"], s["src"], s["dst"], s["tokens"], s["count"])
    return {"pools": s["pools"]}


def _own_compact(s):
    import attention_tensor_cores_gb300 as F
    F.fmha_page_compact(s["seqlens"], 16, s["table"], s["free"], s["n"], s["new_ids"], s["new_table"], s["src"], s["dst"], s["moves"],
                        s["free_out"])
    return {k: s[k] for k in COMPACT}


def _plain_attend(s):
    c = s["case"]
    H, Sq, D = c["Hkv"], c["Sq"], c["D"]
    out, lse = torch.empty_like(s["q"]), torch.empty_like(s["lse"])
    for b in range(s["q"].shape[0]):
        pages = s["table"][b].clamp(min=0).long()
        k, v = (p[pages].permute(1, 0, 2, 3).reshape(H, -1, D).float() for p in (s["k_pool"], s["v_pool"]))
        q = s["q"][b].view(H, -1, D).float()                   # rows of a key/value head: its query heads' tokens
        j = torch.arange(k.shape[1], device=DEV)
        last = torch.arange(q.shape[1], device=DEV)[:, None] % Sq - Sq if c["causal"] else -1
        x = torch.where(j <= s["seqlens"][b] + last, torch.matmul(q, k.transpose(-1, -2)) * D ** -0.5, -math.inf)
        m = x.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, 0.0, m)
        e = torch.exp(x - m)
        l = e.sum(-1, keepdim=True)
        o = torch.matmul(e, v) / torch.where(l == 0, 1.0, l)
        out[b] = o.to(torch.bfloat16).view_as(out[b])
        lse[b] = (torch.log(l) + m).view_as(lse[b])
    return {"out": out, "lse": lse}


def _plain_fork(s):
    P, table, free, n = s["case"]["page"], s["table"], s["free"], s["n"].long()
    Bo, width = table.shape
    N, B = free.numel(), s["parents"].numel()
    p, ctx = s["parents"].long(), s["ctx"].long()
    live, pc = p >= 0, p.clamp(min=0)
    children = torch.zeros(Bo, dtype=torch.int64, device=DEV).scatter_add_(0, pc, live.long())
    col = torch.arange(width, device=DEV)[None, :]
    held = col < ((ctx + P - 1) // P)[:, None]

    def named(rows):     # pages that these rows hold
        at = torch.where(held & rows[:, None], table.long(), N)
        return torch.zeros(N + 1, dtype=torch.bool, device=DEV).scatter_(0, at.flatten(), True)[:N]
    freed = named(children == 0) & ~named(children > 0)
    rank = freed.long().cumsum(0)
    given = rank[-1]
    # freed pages onto the stack, in the order of their ids
    at = torch.where(freed, n + rank - 1, N)
    ids = torch.arange(N, device=DEV, dtype=torch.int32)
    free = torch.cat([free, free.new_zeros(1)]).scatter_(0, at, ids)[:N]
    # children behind their parent's first take a page from its top in place of a partly filled one
    b = torch.arange(B, device=DEV)
    first = torch.full((Bo + 1,), B, device=DEV).scatter_reduce_(0, torch.where(live, p, Bo), b, "amin")
    lens = torch.where(live, ctx[pc], 0)
    part, last = lens % P, (lens // P).clamp(max=width - 1)
    copies = live & (part > 0) & (first[pc] != b)
    a = copies.long().cumsum(0) - 1
    page = free[(n + given - 1 - a).clamp(0, N - 1)]
    new = torch.where(live[:, None] & held[pc], table[pc], s["new_table"])
    s["new_table"] = torch.where(copies[:, None] & (col == last[:, None]), page[:, None], new)
    s["free"], s["seqlens"] = free, lens.int()
    s["src"] = torch.where(copies, table[pc, last], -1)
    s["dst"] = torch.where(copies, page, -1)
    s["tokens"] = torch.where(copies, part, 0).int()
    s["n_out"] = (n + given - copies.sum()).int()
    return {k: s[k] for k in FORK}


def _plain_copy(s):
    c = s["case"]
    N, P = c["pages"], c["page"]
    real = (torch.arange(c["pairs"], device=DEV) < s["count"]) & (s["src"] >= 0)
    at = torch.where(real, s["dst"], N).long()
    source = torch.arange(N + 1, device=DEV).scatter_(0, at, s["src"].clamp(min=0).long())[:N]
    tokens = torch.zeros(N + 1, dtype=torch.int32, device=DEV).scatter_(0, at, s["tokens"])[:N]
    over = (torch.arange(P, device=DEV) < tokens[:, None])[:, None, :, None]
    for pools in s["pools"]:
        for pool in pools:
            pool.copy_(torch.where(over, pool[source], pool))
    return {"pools": s["pools"]}


def _plain_compact(s):
    table, n = s["table"], s["n"].long()
    N, width = s["free"].numel(), table.shape[1]
    ids = torch.arange(N, device=DEV)
    at = torch.where(ids < n, s["free"].long(), N)
    free = torch.zeros(N + 1, dtype=torch.bool, device=DEV).scatter_(0, at, True)[:N]
    used = N - n                                               # ids below it will be used, the others free
    low, high = free & (ids < used), ~free & (ids >= used)
    lists = []
    for which in (high, low):
        k = torch.where(which, which.long().cumsum(0) - 1, N // 2)
        lists.append(torch.full((N // 2 + 1,), -1, device=DEV).scatter_(0, k, ids)[:N // 2].int())
    s["src"], s["dst"] = lists
    s["moves"] = high.sum().int().view(1)
    rank = (high.long().cumsum(0) - 1).clamp(0, max(N // 2 - 1, 0))
    moved = s["dst"][rank] if N > 1 else ids.int()
    s["new_ids"] = torch.where(free, -1, torch.where(high, moved, ids.int()))
    held = torch.arange(width, device=DEV)[None, :] < ((s["seqlens"] + 15) // 16)[:, None]
    s["new_table"] = torch.where(held, s["new_ids"][table.clamp(min=0).long()], s["new_table"])
    s["free_out"] = torch.where(ids < n, (N - 1 - ids).int(), s["free_out"])
    return {k: s[k] for k in COMPACT}


# ------------------------------------------------------------------------------------------------
# the definitions, in 64 bits
# ------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "fork": _exact_fork, "copy": _exact_copy, "compact": _exact_compact}[case["op"]](s)


def _exact_attend(s):
    c = s["case"]
    P, H, Sq, D = c["page"], c["Hkv"], c["Sq"], c["D"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["seqlens"].tolist()):
        at = torch.arange(n, device=DEV)
        page = s["table"][b, at // P].long()
        k, v = s["k_pool"][page, :, at % P].double(), s["v_pool"][page, :, at % P].double()     # [n][Hkv][D]
        for i in range(Sq):
            see = max(0, n - Sq + 1 + i) if c["causal"] else n
            if see:
                q = s["q"][b, :, i].double().view(H, -1, D)
                x = torch.einsum("hgd,nhd->hgn", q, k[:see]) / math.sqrt(D)
                lse[b, :, i] = torch.logsumexp(x, -1).flatten()
                out[b, :, i] = torch.einsum("hgn,nhd->hgd", torch.softmax(x, -1), v[:see]).reshape(-1, D)
    return {"out": out, "lse": lse}


def _exact_fork(s):
    P = s["case"]["page"]
    table, free, new = s["table"].tolist(), s["free"].tolist(), s["new_table"].tolist()
    ctx, parents, n = s["ctx"].tolist(), s["parents"].tolist(), int(s["n"])
    going_on = {p for p in parents if p >= 0}
    kept = {x for i in going_on for x in table[i][:_up(ctx[i], P)]}
    for x in sorted({x for i in range(len(ctx)) if i not in going_on for x in table[i][:_up(ctx[i], P)]} - kept):
        free[n] = x
        n += 1
    lens, src, dst, tokens, seen = [], [], [], [], set()
    for b, p in enumerate(parents):
        lens.append(ctx[p] if p >= 0 else 0)
        k, part = _up(lens[b], P), lens[b] % P
        new[b][:k] = table[p][:k]
        copy = part > 0 and p in seen
        if copy:
            n -= 1
            new[b][k - 1] = free[n]
        src.append(table[p][k - 1] if copy else -1)
        dst.append(free[n] if copy else -1)
        tokens.append(part if copy else 0)
        seen.add(p)
    values = dict(new_table=new, seqlens=lens, src=src, dst=dst, tokens=tokens, free=free, n_out=[n])
    return {k: torch.tensor(values[k], dtype=torch.int32) for k in FORK}


def _exact_copy(s):
    c = s["case"]
    for k, v in s["pools"]:
        for a, b, t in _copy_plan(c)[:c["count"]]:
            if a >= 0:
                k[b, :, :t] = k[a, :, :t]
                v[b, :, :t] = v[a, :, :t]
    return {"pools": s["pools"]}


def _exact_compact(s):
    n, N = int(s["n"]), s["free"].numel()
    free = s["free"][:n].tolist()
    out = set(free)
    used = N - n
    holes = [i for i in range(used) if i in out]
    new = [-1 if i in out else i for i in range(N)]
    moving = [i for i in range(used, N) if i not in out]
    for a, b in zip(moving, holes):
        new[a] = b
    table = s["table"].cpu()
    new_table = s["new_table"].cpu().clone()
    new_ids = torch.tensor(new, dtype=torch.int32)
    for b, x in enumerate(s["seqlens"].tolist()):
        k = _up(x, 16)
        new_table[b, :k] = new_ids[table[b, :k].long()]
    pad = [-1] * (N // 2 - len(moving))
    values = dict(new_ids=new, src=moving + pad, dst=holes + pad, moves=[len(moving)],
                  free_out=[N - 1 - i for i in range(n)] + s["free_out"][n:].tolist())
    return {k: new_table if k == "new_table" else torch.tensor(values[k], dtype=torch.int32) for k in COMPACT}
