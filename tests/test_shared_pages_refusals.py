"""CPU checks of the entry points for shared pages: what they refuse, before they touch a device."""
import ctypes

import pytest
import torch

import attention_tensor_cores_gb300 as F
from attention_tensor_cores_gb300 import build as B
from test_paged_refusals import BAD_CACHES, cache, opts

A, ODD = 0x10000, 0x10002
WS = dict(workspace=0x20000, workspace_bytes=1 << 40)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return F.load()


def prefix(lib, c=None, q=A, table=A, pages=4, lens=A, cu=A, pre=A, N=1, out=A, lse=None, B=2, Hq=4, Sq=1, scale=0.125, o=None):
    return lib.fmha_fwd_prefix(q, c or cache(), table, pages, lens, cu, pre, N, out, lse, B, Hq, Sq, scale, None, o or opts(**WS))


@pytest.mark.parametrize("bad, code", BAD_CACHES)
def test_cache_descriptor(lib, bad, code):
    assert prefix(lib, cache(**bad)) == code
    assert copy(lib, [cache(**bad)]) == code


@pytest.mark.parametrize("bad, code", [
    (dict(q=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(cu=None), 1), (dict(pre=None), 1), (dict(out=None), 1),
    (dict(q=0x10008), 1), (dict(out=0x10008), 1), (dict(table=ODD), 1), (dict(lens=ODD), 1), (dict(cu=ODD), 1), (dict(pre=ODD), 1),
    (dict(lse=ODD), 1), (dict(B=-1), 1), (dict(Sq=-1), 1), (dict(Hq=3), 1), (dict(Hq=0), 1), (dict(pages=0), 1), (dict(N=0), 1), (dict(N=-1), 1),
    (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(N=8193), 2),
    (dict(c=cache(D=128, token_stride=128, head_stride=2048, page_stride=4608)), 2), (dict(c=cache(page_size=12)), 2),
    (dict(pages=1 << 28), 2), (dict(B=1 << 28), 2), (dict(B=1 << 22, pages=1 << 20), 2),
    (dict(o=opts(out_kind=7, **WS)), 1), (dict(o=opts(num_splits=-1, **WS)), 1), (dict(o=opts(num_splits=1, **WS)), 2),
    (dict(o=opts(seqlens_k=A, **WS)), 1), (dict(o=opts(out_kind=2, **WS)), 1), (dict(o=opts(workspace=0x10010, workspace_bytes=1 << 30)), 1),
    (dict(o=opts(out_kind=2, out_scales=A, out_tensor_scale=A, out_f32=0x10008, **WS)), 1)])
def test_fwd_prefix(lib, bad, code):
    assert prefix(lib, **bad) == code
    assert b"fmha_fwd_prefix" in lib.fmha_last_error()


def test_prefix_workspace_size(lib):
    c = cache()
    size = lib.fmha_prefix_workspace_size(2, 4, 1, c, None)
    assert size > 0 and size % 256 == 0 and size == lib.fmha_prefix_workspace_size(2, 4, 1, c, opts())
    # partials of up to 64 rows per key/value head are shared: more rows have fewer partials
    assert lib.fmha_prefix_workspace_size(2, 130, 1, c, None) < 2 * lib.fmha_prefix_workspace_size(2, 128, 1, c, None)
    assert lib.fmha_prefix_workspace_size(2, 4, 1, c, opts(out_kind=2)) > size
    assert lib.fmha_prefix_workspace_size(2, 4, 1, c, opts(out_kind=2, out_f32=A)) == size + 256
    for bad in ((2, 3, 1, c), (2, 4, 1, None), (1 << 28, 4, 1, c), (-1, 4, 1, c), (2, 4, 1, cache(D=96)), (0, 4, 1, c), (2, 4, 0, c)):
        assert lib.fmha_prefix_workspace_size(*bad, opts()) == 0


def fork(lib, parents=A, B=2, ctx=A, old=2, page=16, table=A, width=4, free=A, count=A, pages=10, new=0x30000, lens=A, src=A, dst=A, tok=A, out=A):
    return lib.fmha_page_fork(parents, B, ctx, old, page, table, width, free, count, pages, new, lens, src, dst, tok, out, None)


@pytest.mark.parametrize("bad, code", [(dict([(k, None)]), 1) for k in "parents ctx table free count new lens src dst tok out".split()] +
                         [(dict([(k, ODD)]), 1) for k in "parents ctx table free count new lens src dst tok out".split()] +
                         [(dict(B=-1), 1), (dict(old=-1), 1), (dict(page=0), 1), (dict(pages=0), 1), (dict(width=0), 1), (dict(new=A), 1),
                          (dict(B=8193), 2), (dict(old=8193), 2), (dict(width=1 << 28), 2), (dict(pages=(1 << 19) + 1), 2)])
def test_page_fork(lib, bad, code):
    assert fork(lib, **bad) == code
    assert b"fmha_page_fork" in lib.fmha_last_error()


def copy(lib, caches=None, n_caches=None, src=A, dst=A, tok=None, n=2, count=None):
    caches = [cache()] if caches is None else caches
    array = (F.fmha_kv_cache * max(len(caches), 1))(*caches)
    return lib.fmha_page_copy(array if caches else None, len(caches) if n_caches is None else n_caches, src, dst, tok, n, count, None)


@pytest.mark.parametrize("bad, code", [
    (dict(src=None), 1), (dict(dst=None), 1), (dict(src=ODD), 1), (dict(dst=ODD), 1), (dict(tok=ODD), 1), (dict(count=ODD), 1), (dict(n=-1), 1),
    (dict(n_caches=-1), 1), (dict(caches=[], n_caches=1), 1), (dict(caches=[cache(), cache(num_pages=11)]), 1),
    (dict(caches=[cache(), cache(page_stride=4096)]), 1), (dict(caches=[cache(), cache(token_stride=128)]), 1), (dict(caches=[cache(), cache(k=None)]), 1),
    (dict(caches=[cache(page_size=1 << 21, num_pages=1)]), 2)])
def test_page_copy(lib, bad, code):
    assert copy(lib, **bad) == code
    assert b"fmha_page_copy" in lib.fmha_last_error()


def test_page_copy_of_nothing(lib):
    assert copy(lib, caches=[]) == F.FMHA_OK
    assert copy(lib, n=0, src=None, dst=None) == F.FMHA_OK


def compact(lib, lens=A, B=2, page=16, table=A, width=4, free=A, count=A, pages=10, ids=A, new=0x30000, src=A, dst=A, n=5, moves=A, out=0x30000):
    return lib.fmha_page_compact(lens, B, page, table, width, free, count, pages, ids, new, src, dst, n, moves, out, None)


@pytest.mark.parametrize("bad, code", [(dict([(k, None)]), 1) for k in "lens table free count ids new src dst moves out".split()] +
                         [(dict([(k, ODD)]), 1) for k in "lens table free count ids new src dst moves out".split()] +
                         [(dict(B=-1), 1), (dict(page=0), 1), (dict(pages=0), 1), (dict(width=0), 1), (dict(n=4), 1), (dict(new=A), 1), (dict(out=A), 1),
                          (dict(width=1 << 28), 2), (dict(pages=(1 << 20) + 1, n=1 << 20), 2), (dict(B=(1 << 24) + 1), 2), (dict(n=(1 << 30) + 1), 2)])
def test_page_compact(lib, bad, code):
    assert compact(lib, **bad) == code
    assert b"fmha_page_compact" in lib.fmha_last_error()


def test_binding_refuses_cpu_tensors_and_wrong_types():
    i = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(2, 4, 1, 64, dtype=torch.bfloat16)
    c = F.fmha_kv_cache()
    for call in (lambda: F.fmha_page_fork(i, i, 16, i, i, i, i, i, i, i, i, i), lambda: F.fmha_page_copy([c], i, i),
                 lambda: F.fmha_page_compact(i, 16, i, i, i, i, i, i, i, i, i), lambda: F.fmha_fwd_prefix(x, c, i, i, i, i, x, None, 1.0),
                 lambda: F.fmha_page_copy(c, None, i), lambda: F.fmha_fwd_prefix(3, c, i, i, i, i, x, None, 1.0)):
        with pytest.raises(F.FmhaError) as e:
            call()
        assert e.value.code == F.FMHA_ERR_INVALID
    assert ctypes.sizeof(F.fmha_kv_cache) == 56
