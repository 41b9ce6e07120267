"""Sizes that the key/value cache's entry points refuse before they touch a device."""
import pytest

import moe_expert_cache_gb300 as ft


def _init(L=1, Hq=4, Hkv=2, D=64, page=16, n_pages=8, n_rows=1, row_pages=4, T_max=4, B_max=1):
    return ft.kv_init(L, Hq, Hkv, D, page, n_pages, n_rows, row_pages, ft.FT_KV_BF16, T_max, B_max, 1 << 20, 1 << 20, 1 << 20,
                      1 << 20, None)


@pytest.mark.parametrize("sizes", [
    # rows of partial results: a short row tile for each head and request, 2^31 rows of 128 and more
    dict(Hq=1 << 21, Hkv=1 << 21, T_max=1, B_max=1024),
    dict(Hq=1 << 14, Hkv=1 << 14, T_max=1, B_max=1024),
    dict(Hq=1 << 22, Hkv=1 << 22, T_max=255, B_max=1024),
    # ... and one for each query row on top of its partial result
    dict(Hq=1, Hkv=1, T_max=(1 << 30) - 1),
    # banks of the pool whose number passes 64 bits
    dict(L=1 << 30, n_pages=1 << 30, Hq=8, Hkv=8),
    dict(L=1 << 30, Hq=1 << 20, Hkv=1 << 20),
])
def test_sizes_whose_rows_have_no_number(sizes):
    assert _init(**sizes) == (ft.FT_ERR_ARG, None)


def test_page_bytes_of_a_record_that_no_pool_holds():
    assert ft.kv_page_bytes((1 << 31) - 1, (1 << 31) - 1, 256, 128) == 0
    assert ft.kv_page_bytes(1 << 30, 1, 64, 16) == 0
    assert ft.kv_page_bytes((1 << 30) - 1, 1, 64, 16) == ((1 << 30) - 1) * 2 * 16 * 64 * 2
