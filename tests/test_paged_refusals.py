"""CPU checks of the paged cache's entry points: what they refuse, before they touch a device."""
import ctypes

import pytest
import torch

import attention_tensor_cores_gb300 as F
from attention_tensor_cores_gb300 import build as B

OK, A, B8 = 0x10000, 0x10000, 0x10008


@pytest.fixture(scope="module")
def lib():
    B.build()
    return F.load()


def cache(**kw):
    c = F.fmha_kv_cache()
    base = dict(k=OK, v=OK, num_pages=10, page_size=16, Hkv=2, D=64, page_stride=2048, head_stride=1024, token_stride=64)
    for k, v in (base | kw).items():
        setattr(c, k, v)
    return c


BAD_CACHES = [(dict(k=None), F.FMHA_ERR_INVALID), (dict(v=None), F.FMHA_ERR_INVALID), (dict(k=B8), F.FMHA_ERR_INVALID),
              (dict(num_pages=0), F.FMHA_ERR_INVALID), (dict(page_size=0), F.FMHA_ERR_INVALID), (dict(Hkv=0), F.FMHA_ERR_INVALID),
              (dict(num_pages=1 << 27), F.FMHA_ERR_UNSUPPORTED), (dict(D=96), F.FMHA_ERR_UNSUPPORTED), (dict(D=512), F.FMHA_ERR_UNSUPPORTED), (dict(token_stride=60), F.FMHA_ERR_INVALID),
              (dict(token_stride=56), F.FMHA_ERR_INVALID), (dict(head_stride=-1024), F.FMHA_ERR_INVALID),
              (dict(page_stride=1 << 38), F.FMHA_ERR_INVALID)]


def paged(lib, c=None, q=A, table=A, pages=4, lens=A, out=A, lse=None, B=2, Hq=4, Sq=1, scale=0.125, opts=None):
    return lib.fmha_fwd_paged(q, c or cache(), table, pages, lens, out, lse, B, Hq, Sq, scale, None, opts)


def opts(**kw):
    o = F.fmha_opts()
    for k, v in kw.items():
        setattr(o, k, v)
    return o


@pytest.mark.parametrize("bad, code", BAD_CACHES)
def test_cache_descriptor(lib, bad, code):
    assert paged(lib, cache(**bad)) == code
    assert append(lib, cache(**bad)) == code


@pytest.mark.parametrize("bad, code", [
    (dict(q=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(out=None), 1), (dict(q=B8), 1), (dict(out=B8), 1),
    (dict(table=0x10002), 1), (dict(lens=0x10001), 1), (dict(lse=0x10002), 1), (dict(B=-1), 1), (dict(Sq=-1), 1), (dict(Hq=3), 1),
    (dict(Hq=0), 1), (dict(pages=0), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(c=cache(D=128, token_stride=128, head_stride=2048, page_stride=4608)), 2),
    (dict(c=cache(D=128, token_stride=128, head_stride=2048, page_stride=1024)), 2), (dict(c=cache(page_size=12)), 2), (dict(c=cache(page_size=4)), 2), (dict(pages=1 << 28), 2), (dict(B=1 << 30), 2),
    (dict(opts=opts(out_kind=7)), 1), (dict(opts=opts(num_splits=-1)), 1), (dict(opts=opts(seqlens_k=A)), 1),
    (dict(opts=opts(out_kind=2)), 1), (dict(opts=opts(workspace=0x10010, workspace_bytes=1 << 20)), 1)])
def test_fwd_paged(lib, bad, code):
    assert paged(lib, **bad) == code
    assert b"fmha_fwd_paged" in lib.fmha_last_error()


def test_paged_workspace_size(lib):
    c = cache()
    assert lib.fmha_paged_workspace_size(2, 4, 1, c, None) == 0
    size = lib.fmha_paged_workspace_size(2, 4, 1, c, opts())
    assert size > 0 and size % 256 == 0
    assert lib.fmha_paged_workspace_size(2, 4, 1, c, opts(num_splits=1)) == 0
    assert lib.fmha_paged_workspace_size(2, 4, 1, c, opts(num_splits=1, out_kind=2)) > 0
    assert lib.fmha_paged_workspace_size(2, 3, 1, c, None) == 0
    assert lib.fmha_paged_workspace_size(2, 4, 1, None, None) == 0
    assert lib.fmha_paged_workspace_size(1 << 29, 4, 1, c, opts()) == 0
    # more than 16 rows per key/value head: chunks of rows, each with partials of its own
    assert lib.fmha_paged_workspace_size(1 << 30, 4, 0, c, opts()) == lib.fmha_paged_workspace_size(0, 4, 1, c, opts()) == 0
    assert lib.fmha_paged_workspace_size(2, 64, 1, c, opts()) > lib.fmha_paged_workspace_size(2, 32, 1, c, opts())


def append(lib, c=None, q=A, k=A, v=A, qs=256, wq=None, wk=None, eps=1e-6, table=A, max_pos=100, rope=64, pos=A, slots=A, out=A, T=8,
           Hq=4, Sq=1):
    return lib.fmha_rope_append(q, qs, k, 128, v, 128, wq, wk, eps, table, max_pos, rope, 0, pos, slots, out, c or cache(), T, Hq, Sq, None)


@pytest.mark.parametrize("bad, code", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(slots=None), 1), (dict(out=None), 1), (dict(table=None), 1),
    (dict(pos=None), 1), (dict(q=B8), 1), (dict(wq=B8), 1), (dict(wk=0x10004), 1), (dict(table=B8), 1), (dict(out=B8), 1),
    (dict(pos=0x10002), 1), (dict(slots=0x10004), 1), (dict(qs=260), 1), (dict(qs=-256), 1), (dict(T=-1), 1), (dict(Hq=3), 1),
    (dict(Hq=0), 1), (dict(Sq=0), 1), (dict(Sq=3), 1), (dict(rope=-16), 1), (dict(rope=80), 1), (dict(max_pos=0), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(rope=24), 2), (dict(T=1 << 30), 2)])
def test_append(lib, bad, code):
    assert append(lib, **bad) == code
    assert b"fmha_rope_append" in lib.fmha_last_error()


def table_call(lib, ctx=A, new=A, B=2, page=16, free=A, count=A, pages=10, table=A, width=4, lens=A, cu=A, pos=A, slots=A, T=2, out=A):
    return lib.fmha_page_table(ctx, new, B, page, free, count, pages, table, width, lens, cu, pos, slots, T, out, None)


@pytest.mark.parametrize("bad, code", [
    (dict(ctx=None), 1), (dict(new=None), 1), (dict(free=None), 1), (dict(count=None), 1), (dict(table=None), 1), (dict(lens=None), 1),
    (dict(cu=None), 1), (dict(pos=None), 1), (dict(slots=None), 1), (dict(out=None), 1), (dict(ctx=0x10002), 1), (dict(slots=0x10004), 1),
    (dict(B=-1), 1), (dict(page=0), 1), (dict(pages=0), 1), (dict(width=0), 1), (dict(T=-1), 1), (dict(B=8193), 2),
    (dict(width=1 << 28), 2), (dict(T=(1 << 30) + 1), 2), (dict(pages=(1 << 30) + 1), 2)])
def test_page_table(lib, bad, code):
    assert table_call(lib, **bad) == code
    assert b"fmha_page_table" in lib.fmha_last_error()


def test_binding_refuses_cpu_tensors_and_bad_pools():
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(F.FmhaError):
        F.make_kv_cache(k, k)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(F.FmhaError):
        F.fmha_page_table(i, i, 16, i, i, i, i, i, i, i, i)


def test_pages_error_has_a_text(lib):
    assert lib.fmha_error_string(F.FMHA_ERR_PAGES).decode().startswith("FMHA_ERR_PAGES")
    assert ctypes.sizeof(F.fmha_kv_cache) == 56
