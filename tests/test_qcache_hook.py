"""The test hook of tv_qcache_attention's waits: an addition to out_dtype, refused with any type
that is refused without it."""
import os
import re

import pytest

import tree_speculative_verify_tv_gb300 as tv

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "treeverify.h")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    tv.build()
    tv.load()


def rc(dtype, q=0x10000):
    p = [0x20000 + 0x1000 * i for i in range(10)]
    return tv.tv_qcache_attention(2, 5, 4, 4, 2, 128, 9, 4, p[0], p[1], p[2], p[3], 0, 0, q, 512, p[4], p[5],
                                  p[6], 256, 0.1, dtype, p[7], p[8], 0, p[9], stream=0, check=False)


def test_the_hook_is_the_headers():
    m = re.search(r"#define TV_QCACHE_TEST_EXPIRE_WAIT\s+(0x[0-9a-fA-F]+)", open(HEADER).read())
    assert m and int(m.group(1), 16) == tv.TV_QCACHE_TEST_EXPIRE_WAIT


def test_types_are_checked_with_it():
    hook = tv.TV_QCACHE_TEST_EXPIRE_WAIT
    for bad in (2, 7, 0x200, -1, 1 << 30):
        assert rc(bad) == rc(bad | hook) == tv.TV_ERR_DTYPE
    for good in (tv.TV_BF16, tv.TV_F32):
        assert rc(good, q=None) == rc(good | hook, q=None) == tv.TV_ERR_NULL
        # a call that would run, but for its workspace of 0 bytes
        assert rc(good) == rc(good | hook) == tv.TV_ERR_SHAPE
