"""Scores that are not finite, dense and paged decode: a row that sees one is NaN whatever its keys' split, as in
the formula; rows that do not see it keep their values."""
import math

import pytest
import torch

import attention_tensor_cores_gb300 as F
from paged_util import attention_ref

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")

SHAPES = [  # B, Hq, Hkv, Sq, S, D
    (1, 2, 2, 1, 300, 64),       # one column, up to four pieces a unit
    (1, 2, 2, 1, 9000, 128),     # one column, more pieces
    (2, 8, 2, 2, 500, 128),      # eight columns
    (1, 16, 1, 1, 6000, 64)]     # sixteen columns, more than four pieces


def outputs(q, k, v, lens, causal, how):
    """(o, lse) in FP32 of one way to the same attention."""
    B, Hq, Sq, D = q.shape
    Hkv, S = k.shape[1:3]
    dev = [x.cuda().contiguous() for x in (q, k, v)]
    out, lse = torch.full(q.shape, -3.0, device="cuda"), torch.full(q.shape[:3], -3.0, device="cuda")
    ns = 1 if how.endswith("whole") else 0
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if how.startswith("paged"):
        P = 24 if S % 24 == 0 else 8
        pad = -S % P
        pools = [torch.nn.functional.pad(x, (0, 0, 0, pad)).view(B, Hkv, -1, P, D).transpose(1, 2).reshape(-1, Hkv, P, D) for x in dev[1:]]
        cache = F.make_kv_cache(*pools)
        table = torch.arange(pools[0].shape[0], dtype=torch.int32, device="cuda").view(B, -1).contiguous()
        n = F.fmha_paged_workspace_size(B, Hq, Sq, cache, F.make_opts(F.FMHA_OUT_F32, num_splits=ns))
        ws = torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device="cuda")
        F.fmha_fwd_paged(dev[0], cache, table, lens_d, out, lse, D ** -0.5, F.make_opts(F.FMHA_OUT_F32, num_splits=ns, workspace=ws, causal=causal))
    else:
        o = F.make_opts(F.FMHA_OUT_F32, lens_d if "ragged" in how else None, ns, causal=causal)
        ws = torch.full((max(256, F.fmha_workspace_size(B, Hq, Hkv, Sq, S, D, o)),), 0xFF, dtype=torch.uint8, device="cuda")
        F.fmha_fwd_ex(*dev, out, lse, D ** -0.5, F.make_opts(F.FMHA_OUT_F32, lens_d if "ragged" in how else None, ns, ws, causal=causal))
    torch.cuda.synchronize()
    assert F.fmha_check_status() == 0
    return out.cpu(), lse.cpu()


@pytest.mark.parametrize("how", ["dense", "dense whole", "dense ragged", "paged", "paged whole"])
@pytest.mark.parametrize("shape", SHAPES)
def test_rows_that_see_it_are_nan(shape, how):
    B, Hq, Hkv, Sq, S, D = shape
    g = torch.Generator().manual_seed(S)
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)   # noqa: E731
    q, k, v = rnd(B, Hq, Sq, D).abs(), rnd(B, Hkv, S, D), rnd(B, Hkv, S, D)   # positive queries: infinite keys give one sign
    lens, group, causal = [S] * B, Hq // Hkv, Sq > 1
    o_ref, l_ref, a = attention_ref(q, k, v, lens, D ** -0.5, causal)

    def expect(q, k, sees, what):
        """NaN in the rows of sees [B, Hq, Sq], the reference's values in the others."""
        out, lse = outputs(q, k, v, lens, causal, how)
        assert torch.isnan(out[sees]).all() and torch.isnan(lse[sees]).all(), f"{what}: {out[sees].flatten()[:3]}, {lse[sees][:3]}"
        fine = ~sees
        # dense weights are rounded to BF16 (2^-8), paged ones to 2^-16; FP32 sums as in check_attention
        tol = a[fine] * (2.0 ** -8 + 2.0 ** -11)
        assert ((out[fine].double() - o_ref[fine]).abs() <= tol).all(), what
        assert ((lse[fine].double() - l_ref[fine]).abs() <= 2.0 ** -12 + 2.0 ** -20 * l_ref[fine].abs()).all(), what

    none = torch.zeros(B, Hq, Sq, dtype=torch.bool)
    x, sees = q.clone(), none.clone()
    x[-1, Hq - 1, Sq - 1, 3] = NAN
    sees[-1, Hq - 1, Sq - 1] = True
    expect(x, k, sees, "a query")
    for at in (0, S // 2, S - 1):
        x, sees = k.clone(), none.clone()
        x[0, Hkv - 1, at, 7] = NAN
        seen = [i for i in range(Sq) if not causal or at <= i + S - Sq]
        sees[0, (Hkv - 1) * group:, seen] = True
        expect(q, x, sees, f"key {at}")
        x[0, Hkv - 1, at] = INF
        expect(q, x, sees, f"infinite key {at}")
    x = k.clone()
    x[0, 0] = NAN
    sees = none.clone()
    sees[0, :group] = True
    expect(q, x, sees, "every key of a head")


@pytest.mark.parametrize("how", ["dense", "paged"])
def test_a_score_of_minus_infinity_weighs_nothing(how):
    g = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)   # noqa: E731
    q, k, v = rnd(1, 4, 1, 64).abs() + 1, rnd(1, 2, 700, 64), rnd(1, 2, 700, 64)
    k[0, 1, 100:690] = -INF
    left = torch.cat([torch.arange(100), torch.arange(690, 700)])
    ref = [torch.cat(x, 1) for x in zip(attention_ref(q[:, :2], k[:, :1], v[:, :1], [700], 0.125, False),
                                        attention_ref(q[:, 2:], k[:, 1:, left], v[:, 1:, left], [110], 0.125, False))]
    out, lse = outputs(q, k, v, [700], False, how)
    o, l, a = ref
    assert ((out.double() - o).abs() <= a * (2.0 ** -8 + 2.0 ** -11)).all()
    assert ((lse.double() - l).abs() <= 2.0 ** -12 + 2.0 ** -20 * l.abs()).all()
    k[0, 1] = -INF     # nothing left: as a row without keys
    out, lse = outputs(q, k, v, [700], False, how)
    assert (out[0, 2:] == 0).all() and (lse[0, 2:] == -math.inf).all() and torch.isfinite(out[0, :2]).all()
