"""Softmax scales of the windowed calls whose product with log2(e) (and with an
e4m3 pool's k_scale) leaves fp32: refused before a launch (no GPU needed)."""

import ctypes

import pytest

from tests.test_boundary_steps import NULL, P, _shape, pa  # noqa: F401  (pa: the fixture)


def calls(pa):
    L, s = pa.lib(), ctypes.byref(_shape(pa))
    return (lambda scale, ks=1.0: L.pa_varlen_fwd_sinks(P, P, P, P, P, 4, 2, s, scale, 8, 2, P,
                                                        NULL, NULL),
            lambda scale, ks=1.0: L.pa_decode_window(P, P, P, P, s, scale, 8, 2, P, NULL, NULL),
            lambda scale, ks=1.0: L.pa_decode_window_fp8(P, P, P, P, s, scale, ks, 1.0, 8, 2, P,
                                                         NULL, NULL))


@pytest.mark.parametrize("scale", [3e38, 2.4e38, 3.4028234663852886e38])
def test_scales_past_fp32_are_refused(pa, scale):  # noqa: F811
    for call in calls(pa):
        assert call(scale) == pa.PA_ERR_INVALID


def test_products_past_fp32_are_refused(pa):  # noqa: F811
    fp8 = calls(pa)[2]
    for scale, ks in ((1e30, 1e30), (1e20, 2.5e18), (2.0, 3.4e38), (3.4e38, 3.4e38)):
        assert fp8(scale, ks) == pa.PA_ERR_INVALID, (scale, ks)
