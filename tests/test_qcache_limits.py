"""Sizes of the attention over the 4-bit cache whose work would not be counted in 32 bits."""
import pytest

import tree_speculative_verify_tv_gb300 as tv


@pytest.fixture(scope="module", autouse=True)
def _lib():
    tv.build()
    tv.load()


def need(B, nodes, H, Hkv, max_pages):
    return tv.tv_qcache_attention_workspace_bytes(B, nodes, nodes, H, Hkv, 128, max_pages)


def test_a_request_of_too_many_tiles_is_refused():
    # 512 groups of 64 rows, 8 heads: 2^19 tiles of context alone are 2^31
    assert need(1, 256, 1024, 8, 1 << 20) == 0
    # 2^19 - 8 tiles of context, 2 of the tree and the unit's constant of 3 are below
    assert need(1, 256, 1024, 8, (1 << 20) - 16) > 0


def test_many_requests_of_long_tables_are_taken():
    assert need(300, 1, 64, 8, 1 << 14) > 0
    assert need(1024, 16, 32, 8, 1 << 15) > 0
