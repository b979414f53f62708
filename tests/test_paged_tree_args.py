"""Tree attention without a GPU: calls that have nothing to do; what its kernel does when a wait runs out, by its source."""

from __future__ import annotations

import os
import re

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


def _functions(text):
    """Bodies of a source file's functions (and of its types' members) by name."""
    out = {}
    for m in re.finditer(r"(\w+)\([^;{}]*\)\s*(?:const )?(?::[^{;]*)?\{", text):
        depth, i = 0, m.end() - 1
        while True:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
            if depth == 0:
                break
        out.setdefault(m.group(1), []).append(text[m.end():i - 1])
    return out


def test_no_wait_of_the_tree_kernel_leaves_another_behind():
    """A wait that runs out must not keep anybody from a barrier or a collective that others are at: softmax warps, which
    share a barrier without a limit, have no way out of their tiles; the other roles leave by whole warps and share none."""
    with open(os.path.join(kbuild.CSRC, "kvq_paged_tree.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    bodies = _functions(text)
    softmax = text[text.index("struct Softmax"):text.index("struct Tiles")]
    rest = text.replace(softmax, "")
    assert softmax.count("bar.sync") == 1 and "bar.sync" not in rest and "barrier.sync" not in text
    for name in ("run", "weigh", "summed", "finish", "finish_copies", "load_queries"):
        for body in (b for b in bodies[name] if b in softmax):
            assert re.search(r"return( true| false)?;", body) is None, name
    assert "warp_wait" not in softmax  # (nobody votes there: nobody leaves)
    roles = rest[rest.index("struct Tiles"):rest.index("tree_kernel(")]
    assert re.search(r"(?<!warp_)\bwait_long|\bmbar_wait\(|mbar_try_wait\(", roles) is None
    assert "__syncthreads" not in roles and "__syncthreads" not in softmax
    # the kernel's own: the last one is behind all roles
    kernel = text[text.index("tree_kernel(const"):text.index("constexpr int kJoinWarps")]
    assert kernel.rindex("__syncthreads") > kernel.rindex("screen_values") and "return" not in kernel[kernel.index("tcgen05.alloc"):]
    # and each wait ends: a counted loop around the try
    (long,) = bodies["mbar_wait_long"]
    assert re.search(r"for \(int i = 0; i < kWaitTries; \+\+i\)", long) and "while" not in long


def test_copies_under_way_land_before_the_tree_kernel_ends():
    """Those of 16-bit rows are in no group that a wait for groups knows of."""
    with open(os.path.join(kbuild.CSRC, "kvq_paged_tree.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    kernel = text[text.index("tree_kernel(const"):text.index("constexpr int kJoinWarps")]
    behind = kernel[kernel.index("produce<F"):]
    assert "wait_copies();" in behind[:behind.index("} else {")] and _functions(text)["wait_copies"][0].count("cp.async.wait_all")
