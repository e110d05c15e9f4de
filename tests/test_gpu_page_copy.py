"""fmha_page_copy: exact."""
import pytest
import torch

import attention_tensor_cores_gb300 as F
from paged_util import make_pools

pytestmark = pytest.mark.gpu


def pools(layers, pages, H, P, D, layout, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for _ in range(layers):
        kv = make_pools(pages, H, P, D, layout)
        for x in kv:
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        out.append(kv)
    return out


def expect(kv, pairs):
    want = [[x.clone() for x in layer] for layer in kv]
    for s, d, t in pairs:
        if s >= 0 and d >= 0:
            for layer, w in zip(kv, want):
                for x, y in zip(layer, w):
                    y[d, :, :t] = x[s, :, :t]
    return want


def same(kv, want):
    return all(torch.equal(x, y) for layer, w in zip(kv, want) for x, y in zip(layer, w))


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("layout", ["hnd", "nhd", "kv"])
@pytest.mark.parametrize("H, P, D", [(1, 1, 64), (1, 16, 128), (3, 17, 64), (8, 64, 128), (2, 1000, 64), (40, 5, 128)])
@pytest.mark.parametrize("layers", [1, 3])
def test_pairs(H, P, D, layout, layers):
    kv = pools(layers, 20, H, P, D, layout)
    pairs = [(0, 10, P), (1, 11, 1), (2, 12, max(1, P // 2)), (2, 13, P), (-1, -1, 0), (3, 14, 0), (-1, 15, P), (4, -2, P)]
    want = expect(kv, pairs)
    caches = [F.make_kv_cache(*x) for x in kv]
    src, dst, tok = (i32([p[i] for p in pairs]) for i in range(3))
    F.fmha_page_copy(caches, src, dst, tok)
    assert F.fmha_check_status() == F.FMHA_OK and same(kv, want)


def test_whole_pages_and_count():
    kv = pools(2, 20, 2, 16, 64, "hnd")
    pairs = [(0, 10, 16), (1, 11, 16), (2, 12, 16)]
    src, dst = i32([0, 1, 2]), i32([10, 11, 12])
    caches = [F.make_kv_cache(*x) for x in kv]
    for count in (0, 2, 3):
        want = expect(kv, pairs[:count])
        F.fmha_page_copy(caches, src, dst, count=i32([count]))
        assert F.fmha_check_status() == F.FMHA_OK and same(kv, want), count
    want = expect(kv, pairs)
    F.fmha_page_copy(tuple(caches), src, dst)
    assert same(kv, want)
    for none in ([], caches):
        F.fmha_page_copy(none, i32([]), i32([]))
    assert F.fmha_check_status() == F.FMHA_OK and same(kv, want)


def test_out_of_bounds():
    kv = pools(1, 20, 2, 16, 64, "nhd")
    caches = [F.make_kv_cache(*x) for x in kv]
    for src, dst, tok, count, pairs in (([20], [3], [16], None, []), ([3], [1 << 30], [16], None, []), ([3], [4], [17], None, [(3, 4, 16)]),
                                        ([3], [4], [-1], None, []), ([3, 5], [4, 6], [16, 16], 3, [(3, 4, 16), (5, 6, 16)]), ([3], [4], [16], -1, [])):
        want = expect(kv, pairs)
        F.fmha_page_copy(caches, i32(src), i32(dst), i32(tok), None if count is None else i32([count]))
        assert F.fmha_check_status() == F.FMHA_ERR_PAGES and same(kv, want), (src, dst, tok, count)
    assert F.fmha_check_status() == F.FMHA_OK


def test_more_layers_than_a_launch_takes():
    kv = pools(130, 4, 1, 8, 64, "hnd")
    want = expect(kv, [(1, 2, 5)])
    F.fmha_page_copy([F.make_kv_cache(*x) for x in kv], i32([1]), i32([2]), i32([5]))
    assert F.fmha_check_status() == F.FMHA_OK and same(kv, want)


def test_far_pages():
    # offsets past 2^32 bytes and 2^31 elements
    kv = pools(1, 3, 1, 8, 64, "hnd")
    big = torch.empty((1 << 32) + 4096, dtype=torch.bfloat16, device="cuda")
    k = big.as_strided((3, 1, 8, 64), ((1 << 31), 512, 64, 1))
    v = big.as_strided((3, 1, 8, 64), ((1 << 31), 512, 64, 1), 1024)
    k.copy_(kv[0][0])
    v.copy_(kv[0][1])
    F.fmha_page_copy([F.make_kv_cache(k, v)], i32([0, 2]), i32([1, -1]), i32([7, 8]))
    F.fmha_page_copy([F.make_kv_cache(k, v)], i32([1]), i32([2]), i32([8]))
    want = expect(kv, [(0, 1, 7)])
    want = expect(want, [(1, 2, 8)])
    assert F.fmha_check_status() == F.FMHA_OK and same([(k, v)], want)
