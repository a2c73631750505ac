"""Limits of the paged cache's calls, decided before a launch: no GPU needed."""

import ctypes

import pytest

from coreset_attention_approximation_b200 import wildcat
from test_cache_cpu import BIG, OK, lib, shape  # noqa: F401  (lib: a fixture)


@pytest.mark.parametrize("dtype,tile", [(wildcat.WC_BF16, 16), (wildcat.WC_F32, 8)])
def test_attend_refuses_tables_whose_places_pass_32_bits(lib, dtype, tile):
    """Units x (tiles + 4) places of full tables: up to 2^31 - 1 they can be
    counted, but not rounded up to a multiple of some two thousand warps."""
    for places in ((1 << 31) - 1, (1 << 31) + (1 << 20)):
        units = 64
        tiles = places // units - 4
        s = shape(batch=units // 2, hq=2, hkv=2, dtype=dtype, page=tile, max_pages=tiles)
        assert lib.wc_cache_workspace_bytes(ctypes.byref(s), 0) > 0
        for r in (0, 64):
            assert lib.wc_cache_attend(ctypes.byref(s), OK, 128, 64, OK, OK, OK, OK, r, OK, OK, None, OK, OK, None,
                                       OK, BIG, None) == 4
