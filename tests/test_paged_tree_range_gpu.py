"""Drafted tokens over the paged cache at the ends of their ranges: scales, weights far apart, workspaces of other sizes,
calls without rows, offsets out of order; against implementations in 64 bits, with the tolerances derived there."""

from __future__ import annotations

import math

import pytest
import torch

from quantized_cross_loop_gb300 import kvq
from tests.test_paged_tree_gpu import (D, Cache, _all_bits, _attend, _chain, _compare, _exact, _gen, _offsets,
                                       _query, _raw, _tree)

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


@pytest.mark.parametrize("act", ["bf16", "fp16"])
@pytest.mark.parametrize("B,H,n", [(24, 8, 1), (24, 8, 20), (8, 4, 70)])
def test_many_light_tokens_of_large_scales_beside_a_heavy_one(act, B, H, n):
    """One token has nearly all of the weight and the smallest scale of its tile, just under 2^8 below the others'. The
    others' products of weight and scale are 2^-24.6 of its own each: 8000 of them count, and what is left out lies below
    2^-31 of the largest product, whatever the tile's scales are."""
    T = 8000
    c = Cache([T] * B, [n] * B, 64, H, "e4m3t", seed=3)
    c.k_scale.fill_(1.0)
    c.v_scale.fill_(1.0)
    _raw(c.k)[:] = 0
    light, heavy, one = (_raw(torch.tensor([x], device="cuda").to(c.v.dtype)) for x in (448.0, 1.0, 1.0))
    _raw(c.v)[:] = light
    for b in range(B):
        page, place = c.where(b, torch.tensor([5], device="cuda"))
        _raw(c.k)[page, place, :, 0] = one
        _raw(c.v)[page, place] = heavy
        c.v_scale[page, :, place] = 2.0**-7.9
    q = _query(n * B, 2 * H, act)
    q[..., 0] = 22.5  # (2^32.5 in base 2)
    seen, mask = _tree([n] * B, 2)
    out, lse = _attend(c, q, _offsets([n] * B), mask, softmax_scale=1.0)
    _compare(c, q, out, lse, seen, 1.0)


@pytest.mark.parametrize("act", ["bf16", "fp16"])
@pytest.mark.parametrize("rows", [[1], [9], [50], [140]])
def test_products_with_scales_rise_and_fall(act, rows):
    """Tile by tile the heaviest token and the largest scale are others, so that their products, the weights and the scales
    all have other maxima: nothing overflows FP16, nothing that counts is lost."""
    T = 128 * 40
    c = Cache([T], rows, 32, 1, "e4m3t", seed=5)
    t = torch.arange(T + rows[0], device="cuda")
    page, place = c.where(0, t)
    k = torch.zeros((T + rows[0], 1, D), device="cuda")
    k[:, 0, 0] = (t // 128 * 7 % 16).float() / 2 + (t % 5 == 0) * 3.0 * (t // 128 % 3 == 1)
    c.k_scale[page, :, place] = 1.0
    _raw(c.k)[page, place] = _raw(k.to(c.k.dtype))
    e = (t // 128 * 5 % 9).float() - 4 - torch.where(t % 5 == 0, (t // 128 % 9).float(), 0.0)
    c.v_scale[page, :, place] = torch.exp2(e)[:, None]
    q = _query(rows[0], 4, act)
    q[..., 0] = 1.75
    seen, mask = _tree(rows, 3)
    out, lse = _attend(c, q, _offsets(rows), mask, softmax_scale=1.0)
    _compare(c, q, out, lse, seen, 1.0)


@pytest.mark.parametrize("act", ["bf16", "fp16"])
@pytest.mark.parametrize("rows", [[3], [20], [60], [140], [9, 50]])
@pytest.mark.parametrize("low,high", [(-126, 100), (-126, 60), (-100, 110)])
def test_hidden_scales_far_above_those_of_the_tokens_seen(act, rows, low, high):
    """A drafted token of the largest scales does not reach the rows that do not see it: they see the smallest ones, which
    the way from weights to products has to bridge (BF16 holds results down to 2^-134, FP16 none of these)."""
    lens = [70, 0][:len(rows)]
    c = Cache(lens, rows, 16, 2, "e4m3t", seed=3)
    for b, T in enumerate(x + y for x, y in zip(lens, rows)):
        page, place = c.where(b, torch.arange(T, device="cuda"))
        _raw(c.v)[page, place] = _raw((200 + 50 * torch.randn((T, 2, D), generator=_gen(b), device="cuda")).to(c.v.dtype))
        c.v_scale[page, :, place] = 2.0**low
        page, place = c.where(b, torch.tensor([lens[b] + 1], device="cuda"))
        c.v_scale[page, :, place] = 2.0**high
    n = sum(rows)
    q = _query(n, 8, act)
    seen, mask = _tree(rows, 6)
    hidden = torch.cat([~s[:, 1] for s in seen])
    assert hidden.any() and not hidden.all()
    out, lse = _attend(c, q, _offsets(rows), mask)
    at = 0
    for b, (T, r) in enumerate(zip(lens, rows)):
        K, V = c.values(b, 0, T + r)
        see = torch.cat([torch.ones((r, T), dtype=torch.bool, device="cuda"), seen[b]], 1)
        for j in range(8):
            o, l, to, tl = _exact(q[at:at + r, j], K[:, j // 4], V[:, j // 4], see, 1 / math.sqrt(D), "e4m3t", act,
                                  c.value_scales(b, j // 4, T + r))
            x = out[at:at + r, j].double()
            assert ((x - o).abs().le(to + 2.0**-134) | (x.isinf() if act == "fp16" else torch.zeros_like(x) > 0)).all(), (b, j)
            assert (lse[at:at + r, j].double() - l).abs().le(tl).all(), (b, j)
        at += r
    assert torch.isfinite(out[hidden]).all()


# ------------------------------------------------------------------ values that are not finite


@pytest.mark.parametrize("cache,act", [("bf16", "bf16"), ("fp16", "fp16"), ("e4m3", "fp16"), ("e4m3t", "bf16"),
                                       ("e4m3t", "fp16")])
@pytest.mark.parametrize("rows", [[12, 40], [1, 9], [70, 140]])
def test_finite_channels_beside_values_that_are_not(cache, act, rows):
    """The channels that stay finite are as exact as without such values."""
    c = Cache([70, 129], rows, 16, 2, cache, seed=4)
    seen, mask = _tree(rows, 6)
    bad = [math.nan] if cache.startswith("e4m3") else [math.nan, math.inf, -math.inf]
    for i, (b, t) in enumerate(((0, 70), (0, 70 + rows[0] // 2), (1, 129), (1, 129 + rows[1] - 1))):
        page, place = c.where(b, torch.tensor([t], device="cuda"))
        for d in (3 * i, 64 + i):
            _raw(c.v)[page, place, 1, d] = _raw(torch.tensor([bad[(i + d) % len(bad)]], device="cuda").to(c.v.dtype))
    q = _query(sum(rows), 8, act)
    out, lse = _attend(c, q, _offsets(rows), mask)
    _compare(c, q, out, lse, seen)
    assert not torch.isfinite(out[:, 4:]).all() and torch.isfinite(out[:, :4]).all()


# ------------------------------------------------------------------ sizes


@pytest.mark.parametrize("H,Hq", [(8, 32), (1, 16), (2, 2)])
def test_workspace_of_the_largest_sizes_is_enough(H, Hq):
    """A workspace for some requests and rows serves every call of no more of either."""
    cache = kvq.PagedCache.empty(4, 16, H)
    B, n = [0, 1, 2, 7, 8, 64, 1000], [0, 1, 8, 9, 63, 129, 1024, 5000]
    size = [[cache.tree_workspace_bytes(b, Hq, r) for r in n] for b in B]
    for i in range(len(B)):
        for j in range(len(n)):
            assert size[i][j] >= max(size[x][y] for x in range(i + 1) for y in range(j + 1)), (B[i], n[j])


def test_a_workspace_serves_smaller_batches():
    rows = [300, 129, 0, 83]
    c = Cache([40, 0, 7, 1000], rows, 16, 8, "bf16", seed=4)
    ws = torch.empty(c.cache.tree_workspace_bytes(64, 32, sum(rows)), dtype=torch.uint8, device="cuda")
    q = _query(sum(rows), 32, "bf16")
    out, lse = _attend(c, q, _offsets(rows), None, workspace=ws)
    _compare(c, q, out, lse, _chain(rows))


@pytest.mark.parametrize("cache,act", [("bf16", "bf16"), ("fp16", "fp16"), ("e4m3", "bf16"), ("e4m3t", "bf16")])
@pytest.mark.parametrize("mask", [False, True])
def test_a_long_chunk_among_single_rows(cache, act, mask):
    """The mean of the rows is small, one request's are many: it goes through many units of the form for few rows."""
    rows = [1] * 30 + [700] + [1] * 5 + [0, 2]
    lens = [(37 * b) % 300 for b in range(30)] + [500] + [0, 1, 128, 1000, 63] + [9, 0]
    c = Cache(lens, rows, 16, 2, cache, seed=6)
    q = _query(sum(rows) + 1, 8, act)
    seen, bits = _tree(rows, 5, 0.1) if mask else (_chain(rows), None)
    if mask:
        bits = torch.cat([bits, bits[:1]])
    out, lse = _attend(c, q, _offsets(rows), bits)
    _compare(c, q, out, lse, seen)
    assert c.cache.error_word() == 0


def test_a_step_without_rows():
    """Nothing is drafted: a mask of no rows is no less valid than none."""
    c = Cache([20, 30], [0, 0], 16, 2, "bf16", seed=1)
    q, off = _query(0, 8, "bf16"), _offsets([0, 0])
    for mask in (None, torch.empty((0, 1), dtype=torch.int32, device="cuda")):
        out, lse = _attend(c, q, off, mask)
        assert out.shape == (0, 8, D) and lse.shape == (0, 8)
    assert c.cache.error_word() == 0


# ------------------------------------------------------------------ offsets out of order


@pytest.mark.parametrize("cache", ["bf16", "e4m3t"])
def test_read_reports_requests_whose_offsets_are_out_of_range(cache):
    c = Cache([200, 30, 40], [0] * 3, 16, 2, cache, seed=1)
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")

    def read(B, offsets, n):
        k, v = (torch.full((n, 2, D), 7.0, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        c.cache.clear_error()
        off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        kvq.kvq_paged_read(c.cache, c.table[:B].contiguous(), zero[:B].contiguous(), k, v, offsets=off)
        return k, v, c.cache.error_word()

    for offsets in ([0, 100], [-1, 64], [5, 4]):  # beyond the rows, in front of them, backwards
        k, v, error = read(1, offsets, 64)
        assert (k == 7).all() and (v == 7).all() and error == kvq.PAGED_ERR_LENGTH
    k, v, error = read(3, [0, 3, 3, 1000], 10)  # the last request's
    want = [x.float().bfloat16() for x in c.values(0, 0, 3)]
    assert torch.equal(k[:3], want[0]) and torch.equal(v[:3], want[1])
    assert (k[3:] == 7).all() and (v[3:] == 7).all() and error == kvq.PAGED_ERR_LENGTH
    k, v, error = read(3, [0, 3, 2, 2], 10)  # request 1 goes backwards, request 2 has no rows
    assert torch.equal(k[:3], want[0]) and (k[3:] == 7).all() and error == kvq.PAGED_ERR_LENGTH
    k, v, error = read(3, [2, 5, 5, 7], 10)  # rows in front of the first and behind the last are nobody's
    assert torch.equal(k[2:5], want[0]) and (k[:2] == 7).all() and (k[7:] == 7).all() and error == 0
    assert torch.equal(k[5:7], c.values(2, 0, 2)[0].float().bfloat16())


def test_read_of_few_rows_of_many_requests():
    """The rows of three among 200000 requests; then the last but one's offsets are out of order, too."""
    B, H = 200000, 2
    cache = kvq.PagedCache.empty(8, 16, H)
    cache.k.copy_(torch.arange(8 * 16 * H * D, device="cuda").view(8, 16, H, D) % 251)
    cache.v.copy_(cache.k + 1)
    table = torch.full((B, 1), 1 << 30, dtype=torch.int32, device="cuda")
    rows = torch.zeros(B, dtype=torch.int32)
    at = {0: (3, 2), 123456: (0, 1), B - 1: (7, 5)}  # page, rows
    for b, (page, n) in at.items():
        table[b, 0], rows[b] = page, n
    off = torch.cat([torch.zeros(1, dtype=torch.int32), rows.cumsum(0).to(torch.int32)]).cuda()
    start = torch.full((B,), 2, dtype=torch.int32, device="cuda")
    want = torch.cat([cache.k[page, 2:2 + n] for page, n in at.values()])
    k, v = (torch.full((9, H, D), 7.0, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    kvq.kvq_paged_read(cache, table, start, k, v, offsets=off)
    assert torch.equal(k[:8], want) and torch.equal(v[:8], want + 1) and (k[8] == 7).all() and cache.error_word() == 0
    off[B - 1] = 1
    kvq.kvq_paged_read(cache, table, start, k, v, offsets=off)
    assert cache.error_word() == kvq.PAGED_ERR_LENGTH


@pytest.mark.parametrize("cache,bounds", [("bf16", True), ("e4m3t", False)])
def test_commit_leaves_requests_of_such_offsets_alone(cache, bounds):
    """Requests 1 and 2 have no list, one's beyond the end and one's backwards; request 0's and 3's tokens move."""
    lens = [20, 20, 20, 20]
    c = Cache(lens, [10] * 4, 16, 2, cache, seed=4, bounds=bounds)
    accepted = torch.tensor([2, 5, 1, 4, 7], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 2, 900, 2, 5], dtype=torch.int32, device="cuda")
    want = _all_bits(c)
    for b, a in ((0, [2, 5]), (3, [1, 4, 7])):
        src, dst = c.where(b, 20 + torch.tensor(a, device="cuda")), c.where(b, 20 + torch.arange(len(a), device="cuda"))
        for x in want[:2]:
            x[dst] = x[src].clone()
        if cache == "e4m3t":
            for x in want[2:]:
                x[dst[0], :, dst[1]] = x[src[0], :, src[1]].clone()
        else:  # (20 tokens and those: the second page)
            k = want[0].view(c.k.dtype)[c.table[b, 1].long(), :4 + len(a)].float()
            want[-1][c.table[b, 1].long()] = torch.stack([k.amin(0), k.amax(0)], 1).to(c.bounds.dtype)
    kvq.kvq_paged_tree_commit(c.cache, c.table, c.seq, accepted, off)
    for x, y in zip(want, _all_bits(c)):
        assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
    assert c.cache.error_word() == kvq.PAGED_ERR_LENGTH
