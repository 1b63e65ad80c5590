"""The paged 4-bit cache's host checks at the ends of their ranges, without a GPU."""
import ctypes

import pytest

from block_discrete_diffusion_b200 import build, dg


@pytest.fixture(scope="module")
def lib():
    build.build()
    return dg.lib()


def cache(**kw):
    c = dict(n_layers=2, n_kv=2, d_head=64, n_pages=5, n_seq=3, max_pages=4)
    c.update(kw)
    return dg.dg_kv4_cache_t(*(c[k] for k in ("n_layers", "n_kv", "d_head", "n_pages", "n_seq", "max_pages")), 4096,
                             (1 << 64) - 1, 8192, (1 << 64) - 1)


@pytest.mark.parametrize("n_layers,n_kv,d_head,n_pages", [(1 << 30, 65535, 128, 1 << 24), ((1 << 31) - 1, 65535, 64, 1 << 24),
                                                          (1 << 26, 1, 64, 1 << 20), (1 << 29, 512, 128, 1 << 24)])
def test_pools_whose_bytes_no_size_holds_are_refused(lib, n_layers, n_kv, d_head, n_pages):
    """Sizes that are each allowed, and whose product is not (in 64 bits it may come out small)."""
    c = cache(n_layers=n_layers, n_kv=n_kv, d_head=d_head, n_pages=n_pages, n_seq=1)
    assert dg.dg_kv4_pool_bytes(c) == 0 and dg.dg_kv4_book_bytes(c) == 0
    assert lib.dg_kv4_init(ctypes.byref(c), None) == dg.DG_ERR_INVALID_ARG


def test_the_largest_pools_are_counted_whole(lib):
    c = cache(n_layers=100, n_kv=512, d_head=128, n_pages=1 << 24, n_seq=1)
    assert dg.dg_kv4_pool_bytes(c) == 100 * 512 * 72 * 128 << 24


@pytest.mark.parametrize("stride", [0, 32, -56])
@pytest.mark.parametrize("dim", ["seq", "row", "head"])
def test_outputs_on_one_another_are_refused(lib, dim, stride):
    """(An expanded tensor, a sliding window.)  Inputs may be broadcast, and a dimension of one may have any stride."""
    c = cache()
    far = dict(seq=1024, row=256, head=64)
    far[dim] = stride
    s = (far["seq"], far["row"], far["head"])
    good = (1024, 256, 64)
    bad = dg.DG_ERR_INVALID_ARG
    for k, v in ((s, good), (good, s)):
        rows = dg.dg_kv4_rows(4096, 1 << 20, *k, *v, None, 4, 0)
        assert lib.dg_kv4_read(ctypes.byref(c), 0, ctypes.byref(rows), None) == bad
        assert b"overlap" in lib.dg_last_error()
    attn = dg.dg_kv4_attn(4096, 1 << 20, None, None, *good, *s, 4, 4, 0, 0, 1.0)
    assert lib.dg_kv4_attend(ctypes.byref(c), 0, ctypes.byref(attn), 4096, 1 << 40, None) == bad
    assert b"overlap" in lib.dg_last_error()
    # past the checks of arguments: a workspace that is too small is found after them
    ok = dg.dg_kv4_attn(4096, 1 << 20, None, None, *s, *good, 4, 4, 0, 0, 1.0)
    assert lib.dg_kv4_attend(ctypes.byref(c), 0, ctypes.byref(ok), 4096, 1, None) == dg.DG_ERR_CAPACITY
    one = cache(n_seq=1, n_kv=1)
    ok = dg.dg_kv4_attn(4096, 1 << 20, None, None, *good, stride, stride, stride, 1, 1, 0, 0, 1.0)
    assert lib.dg_kv4_attend(ctypes.byref(one), 0, ctypes.byref(ok), 4096, 1, None) == dg.DG_ERR_CAPACITY
