"""Scales that the attention over 4-bit caches cannot hold: refused on the host,
before anything is enqueued."""
import math

import pytest

import sparse_attention_top_gb300 as gb
from test_prefill_host import selected4, tree4


@pytest.mark.parametrize("f", [tree4, selected4])
@pytest.mark.parametrize("scale,unit", [(2.0 ** 113, 1.0), (-2.0 ** 113, 1.0), (2.0 ** 53, 2.0 ** 60), (math.inf, 1.0), (3e38, 2.0 ** -10)])
def test_scales_beyond_the_products_range(f, scale, unit):
    """(their factor was infinite, and a score of 0 a NaN)"""
    assert f(scale=scale, ks=unit) == gb.EUNSUPPORTED
