"""Tree attention without a GPU: calls that have nothing to do."""

from __future__ import annotations

import pytest

from quantized_cross_loop_gb300 import build as kbuild
from quantized_cross_loop_gb300 import kvq
from tests.test_paged_tree_abi import BAD, P, _cache, _tree


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return kvq.lib()


def test_a_mask_of_no_rows_needs_no_address(L):
    c = _cache(L)
    assert _tree(L, c, n=0, mask=None, words=1, q=None, out=None, ws=None, size=0) == 0
    assert _tree(L, c, n=0, mask=None, words=0, q=None, out=None, ws=None, size=0) == 0
    assert _tree(L, c, n=0, mask=None, words=33) == BAD
    assert _tree(L, c, n=0, mask=P, words=0) == BAD
    assert _tree(L, c, n=9, mask=None, words=1) == BAD
