"""Limits of the cache's further forms on the CPU: arguments that a kernel could not take are refused before any HIP
call."""
import pytest

from .test_kvcache_forms_abi import L, _append, _attend, _cache, _said  # noqa: F401 (L: a fixture)


@pytest.mark.parametrize("lw", [None, 0x10000])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scales_over_small_caps(L, sign, lw):  # noqa: F811
    """scale / cap times 2 log2(e), the factor that a product takes to its tanh, has to be a float: with an infinite one
    a product of 0 would be NaN.  3.4028e38 / 2.8854 = 1.1793e38."""
    weights = dict(lw=lw, lws=(64, 32)) if lw else {}
    for scale, cap in ((1.2e30, 1e-8), (1e30, 5e-9), (1.19e38, 1.0), (3.3e38, 2.0)):
        assert _attend(L, scale=sign * scale, cap=cap, **weights) == 1 and "cap" in _said(L)
    for scale, cap in ((1.17e30, 1e-8), (1.17e38, 1.0)):
        assert _attend(L, scale=sign * scale, cap=cap, ws=None, nb=0, **weights) == 3


# 10 pages of 32 slots of 2 heads of 64 codes, in the order of their strides
@pytest.mark.parametrize("strides", [(4096, 64, 64), (64, 128, 64), (4096, 128, 128), (4032, 128, 64), (64, 64, 64),
                                     (4096, 64, 2032), (2048, 64, 4096), (128, 1216, 64), (192, 64, 64)])
def test_caches_that_overlap(L, strides):  # noqa: F811
    """Strides of at least dim each, and yet two slots in one place: the move of older codes writes what another reads."""
    for name in "kv":
        c = _cache(**{f"{name}_{n}": s for n, s in zip(("page", "slot", "head"), strides)})
        assert _append(L, c, T=0) == 1 and "overlap" in _said(L)
        assert _append(L, c, T=0, **({} if name == "k" else dict(v=None))) == (1 if name == "k" else 0)


@pytest.mark.parametrize("strides", [(4096, 128, 64), (4096, 64, 2048), (64, 1280, 640), (128, 1280, 64),
                                     (2048, 64, 20480), (64, 640, 20480), (1 << 39, 128, 64), (8192, 256, 128),
                                     (4096, 1 << 39, 64 + 9 * 4096)])
def test_caches_of_any_order(L, strides):  # noqa: F811
    c = _cache(**{f"{k}_{n}": s for k in "kv" for n, s in zip(("page", "slot", "head"), strides)})
    assert _append(L, c, T=0) == 0, _said(L)


def test_strides_of_what_there_is_one_of_are_free(L):  # noqa: F811
    for bad in (dict(pages=1, k_page=0), dict(heads=1, k_head=16), dict(pages=1, heads=1, k_page=64, k_head=64)):
        assert _append(L, _cache(**bad), T=0) == 0, _said(L)
