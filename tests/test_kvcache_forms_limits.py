"""Limits of the cache's further forms on the CPU: arguments that a kernel could not take are refused before any HIP
call."""
import pytest

from .test_kvcache_forms_abi import L, _attend, _said  # noqa: F401 (L: a fixture)


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
