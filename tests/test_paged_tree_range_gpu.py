"""Drafted tokens over the paged cache at the ends of their ranges: scales, weights far apart, workspaces of other sizes,
calls without rows, offsets out of order; against implementations in 64 bits, with the tolerances derived there."""

from __future__ import annotations

import math

import pytest
import torch

from tests.test_paged_tree_gpu import D, Cache, _attend, _exact, _gen, _offsets, _query, _tree

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ scales


@pytest.mark.parametrize("lens,rows", [([700, 0, 33], [1, 1, 1]), ([700, 90], [9, 130]), ([20011], [40])])
@pytest.mark.parametrize("scale", [2.0**-126, 2.0**-120, 1.5 * 2.0**118])
def test_value_scales_per_head_to_the_ends_of_their_range(lens, rows, scale):
    """Sums over many tokens divided by the weights' sum stay in FP32's range with any scale; the scale divided by that
    sum does not (units that a block finishes, in copies and not, and units that several share). BF16 rounds results below
    its normal range by up to 2^-134."""
    c = Cache(lens, rows, 16, 2, "e4m3", seed=3)
    for b, T in enumerate(x + y for x, y in zip(lens, rows)):
        x = 256 + 64 * torch.randn((T, 2, D), generator=_gen(b), device="cuda")
        c.put(b, 0, c.v, c.v_scale, x.clamp(1, 448))
    c.v_scale[0], c.v_scale[1] = scale, 1.0
    n = sum(rows)
    q = _query(n, 8, "bf16")
    seen, mask = _tree(rows, 6)
    out, lse = _attend(c, q, _offsets(rows), mask)
    at = 0
    for b, (T, r) in enumerate(zip(lens, rows)):
        K, V = c.values(b, 0, T + r)
        see = torch.cat([torch.ones((r, T), dtype=torch.bool, device="cuda"), seen[b]], 1)
        for j in range(8):
            o, l, to, tl = _exact(q[at:at + r, j], K[:, j // 4], V[:, j // 4], see, 1 / math.sqrt(D), "e4m3", "bf16",
                                  c.value_scales(b, j // 4, T + r))
            assert (out[at:at + r, j].double() - o).abs().le(to + 2.0**-134).all(), (b, j)
            assert (lse[at:at + r, j].double() - l).abs().le(tl).all(), (b, j)
        at += r
