"""fmha_rope_append on the GPU against its definition in 64 bits."""
import pytest
import torch

import attention_tensor_cores_gb300 as F
from paged_util import make_pools, up

pytestmark = pytest.mark.gpu

EPS = 1e-6


def table_of(max_pos, R):
    f = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    x = torch.arange(max_pos, dtype=torch.float64)[:, None] * f
    return torch.cat([x.cos(), x.sin()], 1).float()


def ref_heads(x, w, cos_sin, pos, pairs):
    """(y, size) in FP64: the heads, and for each feature the magnitude its FP32 roundings are relative to."""
    y = x.double()
    D = y.shape[-1]
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * w.double()
    size = y.abs()
    if cos_sin is not None:
        R = cos_sin.shape[1]
        c, s = cos_sin.double()[pos.long()][:, None, :R // 2], cos_sin.double()[pos.long()][:, None, R // 2:]
        i = torch.arange(R // 2)
        i, j = (2 * i, 2 * i + 1) if pairs else (i, i + R // 2)
        a, b = y[..., i], y[..., j]
        y = y.clone()
        y[..., i], y[..., j] = a * c - b * s, b * c + a * s
        size[..., i] = size[..., j] = a.abs() + b.abs()
    return y, size


# Each output is rounded once to BF16 (half a step: 2^-8 of it).  Before that, FP32: a sum of D <= 128 squares
# and its root (relative error below (D / 2 + 8) 2^-24 < 2^-17), three products and a sum (4 * 2^-24): all below
# 2^-16 of the magnitudes that enter.  2^-134 covers outputs below BF16's normal range.
def near(got, ref, size, what):
    d = (got.double().cpu() - ref).abs() - (2.0 ** -8 * ref.abs() + 2.0 ** -16 * size * (1 + 2.0 ** -8) + 2.0 ** -134)
    assert (d <= 0).all(), f"{what}: {d.max():.3e} too much"


def case(T, Hq, Hkv, D, R, pairs, wq, wk, P, layout, Sq=1, pad=(), seed=0, split=False, sigma=1.0, max_pos=500, pages=None):
    g = torch.Generator().manual_seed(seed)
    n = T * 3 + 40
    pages = pages or up(n, P)
    qkv = (torch.randn(T, Hq + 2 * Hkv, D, generator=g) * sigma).to(torch.bfloat16)
    d = qkv.cuda()
    q, k, v = d[:, :Hq], d[:, Hq:Hq + Hkv], d[:, Hq + Hkv:]
    if split:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    ws = [(1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16) if on else None for on in (wq, wk)]
    table = table_of(max_pos, R) if R else None
    pos = torch.randint(0, max_pos, (T,), generator=g).int()
    slots = torch.randperm(pages * P, generator=g)[:T]
    for t in pad:
        slots[t], pos[t] = -1 - t, -5
    kp, vp = make_pools(pages, Hkv, P, D, layout, fill=-3.0)
    cache = F.make_kv_cache(kp, vp)
    out = torch.full((T // Sq, Hq, Sq, D), -3.0, dtype=torch.bfloat16, device="cuda")
    dev = lambda x: None if x is None else x.cuda()   # noqa: E731
    F.fmha_rope_append(q, k, v, dev(ws[0]), dev(ws[1]), EPS, dev(table), dev(pos) if R else None, slots.cuda(), out, cache,
                       interleaved=pairs)
    assert F.fmha_check_status() == 0
    real = slots >= 0
    ref_pos = pos.clamp(min=0)
    rq, size_q = ref_heads(qkv[:, :Hq], ws[0], table, ref_pos, pairs)
    rk, size_k = ref_heads(qkv[:, Hq:Hq + Hkv], ws[1], table, ref_pos, pairs)
    got = out.transpose(1, 2).reshape(T, Hq, D)
    near(got[real.cuda()], rq[real], size_q[real], "q")
    assert (got[~real.cuda()] == -3).all(), "padding was written"
    st = slots[real].cuda()
    near(kp[st // P, :, st % P], rk[real], size_k[real], "k")
    assert torch.equal(vp[st // P, :, st % P].cpu(), qkv[:, Hq + Hkv:][real]), "v"
    untouched = torch.ones(pages * P, dtype=torch.bool)
    untouched[slots[real]] = False
    u = untouched.nonzero()[:, 0].cuda()
    assert (kp[u // P, :, u % P] == -3).all() and (vp[u // P, :, u % P] == -3).all(), "another slot was written"


@pytest.mark.parametrize("D, R", [(64, 0), (64, 16), (64, 48), (64, 64), (128, 0), (128, 32), (128, 96), (128, 112), (128, 128)])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("norm", [(True, True), (False, False), (True, False), (False, True)])
def test_heads(D, R, pairs, norm):
    case(5, 6, 2, D, R, pairs, *norm, 16, "hnd", seed=D + R)


@pytest.mark.parametrize("T, Hq, Hkv, P, layout, Sq, split", [
    (1, 1, 1, 16, "hnd", 1, False), (1, 32, 8, 16, "nhd", 1, False), (7, 5, 5, 1, "hnd", 1, True), (8, 32, 8, 64, "kv", 4, False),
    (33, 7, 1, 48, "nhd", 3, True), (129, 16, 4, 8, "hnd", 1, False), (130, 12, 2, 5, "kv", 2, False), (1000, 4, 1, 24, "nhd", 1, False),
    (2049, 3, 1, 16, "hnd", 1, False), (513, 9, 3, 256, "hnd", 1, True)])
@pytest.mark.parametrize("D, pairs", [(64, True), (128, False)])
def test_layouts(T, Hq, Hkv, P, layout, Sq, split, D, pairs):
    case(T, Hq, Hkv, D, D, pairs, True, True, P, layout, Sq, split=split, seed=T)


def test_padding_is_left_alone():
    case(12, 4, 2, 64, 32, False, True, True, 16, "hnd", 2, pad=(0, 5, 10, 11))
    case(6, 4, 2, 128, 128, True, True, True, 16, "nhd", 1, pad=range(6))


@pytest.mark.parametrize("sigma", [1e-18, 1e-6, 1e6, 1e15])
def test_magnitudes(sigma):
    case(9, 4, 2, 128, 64, False, sigma < 1e10, sigma < 1e10, 16, "hnd", sigma=sigma)


def test_far_positions():
    case(9, 4, 2, 64, 64, False, True, True, 16, "hnd", max_pos=200001)


def test_one_token_of_any_stride():
    x = torch.ones(1, 2, 64, dtype=torch.bfloat16, device="cuda").as_strided((1, 2, 64), (3, 64, 1))
    kp, vp = make_pools(1, 2, 16, 64, "hnd", fill=0.0)
    out = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    F.fmha_rope_append(x, x, x, None, None, EPS, None, None, torch.tensor([5], device="cuda"), out, F.make_kv_cache(kp, vp))
    assert F.fmha_check_status() == 0 and (out == 1).all() and (kp[0, :, 5] == 1).all() and (vp[0, :, 5] == 1).all()


def test_no_tokens():
    case(0, 4, 2, 64, 64, False, True, True, 16, "hnd")


def test_out_of_bounds_tokens_are_left_out():
    """A slot behind the pool or a position behind the table: the token is left out and reported."""
    q = torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.ones(4, 1, 64, dtype=torch.bfloat16, device="cuda")
    for slots, pos in (([0, 32, 1, 1 << 40], [0, 0, 9, 0]), ([0, 3, 1, 4], [0, 10, 9, -1])):
        kp, vp = make_pools(2, 1, 16, 64, "hnd", fill=0.0)
        out = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
        F.fmha_rope_append(q, k, k, None, None, EPS, table_of(10, 64).cuda(), torch.tensor(pos, dtype=torch.int32, device="cuda"),
                           torch.tensor(slots, device="cuda"), out, F.make_kv_cache(kp, vp))
        assert F.fmha_check_status() == F.FMHA_ERR_PAGES
        assert [bool((out[t] != 0).any()) for t in range(4)] == [True, False, True, False]
        assert (vp != 0).sum() == 128 and (vp[0, 0, :2] == 1).all()


def test_nan_stays_in_its_head():
    q = torch.ones(2, 4, 128, dtype=torch.bfloat16, device="cuda")
    q[0, 1, 5] = float("nan")
    q[1, 2, 7] = float("inf")
    k = torch.ones(2, 2, 128, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    kp, vp = make_pools(1, 2, 16, 128, "hnd", fill=0.0)
    out = torch.zeros(2, 4, 128, dtype=torch.bfloat16, device="cuda")
    F.fmha_rope_append(q, k, k, w, w, EPS, table_of(10, 128).cuda(), torch.tensor([1, 2], dtype=torch.int32, device="cuda"),
                       torch.tensor([3, 4], device="cuda"), out, F.make_kv_cache(kp, vp))
    fine = torch.isfinite(out).all(-1)
    assert fine.tolist() == [[True, False, True, True], [True, True, False, True]]
    assert torch.isfinite(kp).all() and F.fmha_check_status() == 0


def test_refuses_wrong_shapes():
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    kp, vp = make_pools(2, 1, 16, 64, "hnd", fill=0.0)
    cache = F.make_kv_cache(kp, vp)
    slots = torch.arange(4, device="cuda")
    args = lambda **kw: {**dict(q=q, k=q[:, :1], v=q[:, :1], q_weight=None, k_weight=None, eps=EPS, cos_sin=None, positions=None,   # noqa: E731
                                slots=slots, q_out=torch.zeros_like(q), cache=cache), **kw}
    F.fmha_rope_append(**args())
    for bad in (dict(k=q), dict(q=q.float()), dict(q_out=q[:2].contiguous()), dict(slots=slots.int()), dict(slots=slots[:3]),
                dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)), dict(q_weight=q[0, 0, :32].contiguous()), dict(v=q.cpu()[:, :1])):
        with pytest.raises(F.FmhaError):
            F.fmha_rope_append(**args(**bad))
