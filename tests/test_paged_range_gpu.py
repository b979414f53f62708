"""The paged cache's operators at the ends of their types' ranges, against plain
64-bit implementations: queries and scales of very different sizes, scores in the
subnormal range, ties of the 8-bit rounding, infinities beside masked places.

Tolerances are those of the arithmetic: a sum of 128 exact products in FP32 is off
by at most 132 * 2^-23 of the sum of the terms' magnitudes, whatever the query's
channels that meet zero keys are (their products are zero). Orders and stored
codes have no tolerance.
"""

from __future__ import annotations

import math

import pytest
import torch

from quantized_cross_loop_gb300 import kvq
from tests.test_paged_gpu import D, DT, Batch, _attend, _bounds_only, _check_selection, _compare, _gen, _query, _raw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("g", [4, 12])
@pytest.mark.parametrize("ratio", [0, 16, 24, 30, 31, 32, 33, 34, 40, 64, 66, 67, 90, 120])
def test_e4m3_attention_of_queries_with_channels_far_apart(ratio, g):
    """Channels of 2^ratio and many sizes below, which meet zero keys, leave the logits to ordinary channels: no bit of
    those may be lost beside them. Heads of one group differ in their channels' spread."""
    b = Batch([100, 64, 900, 3], 16, 2, "e4m3", seed=ratio)
    zero = D // 2
    _raw(b.k)[..., :zero] = 0
    for k in b.K:
        k[..., :zero] = 0
    q = _query(4, 2 * g)
    steps = torch.arange(zero, 0, -1, device="cuda") * (ratio / zero)
    large = (torch.randn((4, 2 * g, zero), generator=_gen(ratio), device="cuda").double() * 2.0 ** steps).bfloat16()
    large[..., 0] = 2.0**ratio
    q[:, 1:, :zero] = large[:, 1:]  # (head 0 stays as it is)
    q[1, 2] = 0
    out, lse = _attend(b, q)
    _compare(b, q, out, lse, 1 / math.sqrt(D))


def test_e4m3_attention_of_queries_over_the_whole_range_of_bf16():
    """One channel at BF16's end, ordinary ones, and channels down to BF16's smallest subnormal on keys of a large
    scale: the largest meets zero keys, so that what counts lies up to 2^260 below it."""
    b = Batch([70, 200], 16, 1, "e4m3", seed=2)
    _raw(b.k)[..., 0] = 0
    b.k_scale.fill_(2.0**120)
    b.K = [k.clone() for k in b.K]
    for i, t in enumerate(b.lens):
        at = torch.arange(t, device="cuda")
        k = _raw(b.k)[b.table[i].long()[at // 16], at % 16].view(b.dt).double()
        b.K[i] = k * 2.0**120
    q = torch.zeros((2, 4, D), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 2.0**127
    q[:, 0, 1:40] = (torch.randn((2, 39), generator=_gen(1), device="cuda").double() * 2.0**-126).bfloat16()
    q[:, 1, 1:40] = 2.0**-133  # the smallest BF16 number
    q[:, 2, 1:40] = -(2.0**-130)
    q[:, 3, 0] = 0
    q[:, 3, 5:9] = 2.0**-133
    out, lse = _attend(b, q, softmax_scale=1.0)
    _compare(b, q, out, lse, 1.0)


@pytest.mark.parametrize("g,requests", [(4, 4), (4, 170), (16, 170), (1, 700), (3, 5000)])
def test_e4m3_attention_of_far_apart_channels_in_some_heads(g, requests):
    """Heads whose channels need more than FP16, here and there in batches of fewer and of many more units than blocks,
    over all pages and over selected ones; beside a refused request, one without tokens, and a bad selection."""
    lens = [(29 * i) % 170 for i in range(requests)]
    lens[:4] = [3000, 40, 0, 75]
    b = Batch(lens, 16, 2, "e4m3", seed=g, bounds=False)
    _raw(b.k)[..., 0] = 0
    for k in b.K:
        k[..., 0] = 0
    q = _query(requests, 2 * g)
    i = torch.arange(requests * 2 * g, device="cuda").view(requests, 2 * g)
    q[..., 0] = torch.where(i % 5 == 2, 2.0**60, q[..., 0].float()).bfloat16()
    check = list(range(4)) + list(range(4, requests, max(1, requests // 40)))
    some = Batch.__new__(Batch)
    some.lens, some.ps, some.H = [lens[x] for x in check], 16, 2
    some.K, some.V = [b.K[x] for x in check], [b.V[x] for x in check]
    out, lse = _attend(b, q)
    _compare(some, q[check], out[check], lse[check], 1 / math.sqrt(D))
    sel = torch.full((requests, 2, 4), -1, dtype=torch.int32, device="cuda")
    pages = torch.tensor([-(-t // 16) for t in lens], device="cuda")
    for h in range(2):
        for e in range(3):
            sel[:, h, e] = torch.where(pages > 2 * e + h, 2 * e + h, -1)
    out = kvq.kvq_paged_sparse_attn(b.cache, b.table, b.seq, q, sel, lse=lse)
    _compare(some, q[check], out[check], lse[check], 1 / math.sqrt(D), sel=sel[check])
    assert b.cache.error_word() == 0
    b.seq[1] = -1
    b.table[3, 2] = b.cache.n_pages
    out, lse = _attend(b, q)
    _compare(some, q[check], out[check], lse[check], 1 / math.sqrt(D), skip=(1, 3))
    b.seq[1], sel[0, 1, 1] = 40, 0
    out = kvq.kvq_paged_sparse_attn(b.cache, b.table, b.seq, q, sel, lse=lse)
    assert torch.isnan(out[0, g:]).all() and torch.isfinite(out[0, :g]).all()


def test_captured_e4m3_attention_follows_the_queries():
    """A captured call replayed with queries that FP16 holds and queries that it does not; two streams at once."""
    b = Batch([700, 40, 90], 16, 2, "e4m3", seed=1)
    _raw(b.k)[..., 0] = 0
    for k in b.K:
        k[..., 0] = 0
    q, out, lse = _query(3, 8), torch.empty((3, 8, D), device="cuda"), torch.empty((3, 8), device="cuda")
    ws = torch.empty(b.cache.workspace_bytes(3, 8, 0), dtype=torch.uint8, device="cuda")
    kvq.kvq_paged_decode_attn(b.cache, b.table, b.seq, q, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.kvq_paged_decode_attn(b.cache, b.table, b.seq, q, out=out, lse=lse, workspace=ws)
    seen = []
    for turn, large in enumerate((1.0, 2.0**70, 1.0, 2.0**40)):
        q.copy_(_query(3, 8, seed=turn))
        q[turn % 3, turn::2, 0] = large
        graph.replay()
        torch.cuda.synchronize()
        _compare(b, q, out, lse, 1 / math.sqrt(D))
        seen.append((q.clone(), out.clone()))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [(want, kvq.kvq_paged_decode_attn(b.cache, b.table, b.seq, x, stream=streams[i % 2]))
           for i, (x, want) in enumerate(seen * 5)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in got)


@pytest.mark.parametrize("gain,k_scale,softmax_scale", [
    (2.0**-115, 2.0**-33, 0.1),      # the scales' product is below FP32's smallest number: all tokens weigh the same
    (2.0**126, 2.0**-78, 2.0**-78),  # ... beside queries of BF16's other end
    (2.0**-133, 2.0**35, 2.0**95),   # above FP32's largest, and the smallest queries bring the logits back
])
def test_e4m3_attention_of_scales_whose_product_leaves_fp32(gain, k_scale, softmax_scale):
    b = Batch([77, 200, 64], 16, 2, "e4m3", seed=4, spread=20.0)
    stored = [k / b.k_scale.double()[:, None] for k in b.K]
    b.k_scale.fill_(k_scale)
    b.K = [k * k_scale for k in stored]
    q = (torch.sign(torch.randn((3, 8, D), generator=_gen(3), device="cuda")).double() * gain).bfloat16()
    assert (q != 0).all()
    out, lse = _attend(b, q, softmax_scale=softmax_scale)
    _compare(b, q, out, lse, softmax_scale)


@pytest.mark.parametrize("v_scale", [2.0**110, 2.0**-126])
def test_e4m3_attention_of_large_and_small_value_scales(v_scale):
    """Values whose sum lies within FP32's range, in requests that one block and several blocks attend to."""
    b = Batch([5000, 40], 16, 1, "e4m3", seed=6)
    stored = [v / b.v_scale.double()[:, None] for v in b.V]
    b.v_scale.fill_(v_scale)
    b.V = stored
    q = _query(2, 4)
    out, lse = _attend(b, q)
    _compare(b, q, out.double() / v_scale, lse, 1 / math.sqrt(D))


@pytest.mark.parametrize("cache,act", [("bf16", "bf16"), ("fp16", "fp16"), ("e4m3", "bf16"), ("e4m3", "fp16")])
@pytest.mark.parametrize("channel", [7, 23])
def test_infinite_queries_beside_masked_places(cache, act, channel):
    """A query whose products with all keys are -inf finds nothing, also where the last tile has places without a
    token."""
    b = Batch([16, 40, 3, 70], 16, 1, cache)
    _raw(b.k)[..., channel] = _raw(torch.full((1,), -2.0, device="cuda").to(b.dt))
    q = _query(4, 4, act)
    q[:, 1, channel] = math.inf
    out, lse = _attend(b, q)
    assert (out[:, 1] == 0).all() and torch.isneginf(lse[:, 1]).all()
    assert torch.isfinite(out).all() and torch.isfinite(lse[:, [0, 2, 3]]).all()


@pytest.mark.parametrize("lens,H", [([300], 2), ([3000], 1)])  # one launch, two launches
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("size", [-130, -142, -147])
def test_selection_of_scores_below_fp32s_normal_range(lens, H, cache, size):
    """Products that FP32 rounds to a few bits or to nothing (those of FP16 numbers are never that small): the order is
    that of the exact scores all the same."""
    b = _bounds_only(lens, 1, H, "bf16", seed=-size)
    g = _gen(-size)
    n = b.bounds.shape[0]
    small = torch.rand((n, H, 2, D), generator=g, device="cuda")
    small[::3, :, :, 5:] = 0  # pages of few large terms beside pages of many small ones
    small[::3] *= 60
    e_bounds = size // 2 if cache == "bf16" else -6
    b.dt = DT[cache]
    b.bounds = (small.double() * 2.0**e_bounds).to(b.dt)
    b.cache = kvq.PagedCache(1, H, key_bounds=b.bounds)
    q = torch.randn((len(lens), 2 * H, D), generator=g, device="cuda").abs()
    q = (q.double() * 2.0 ** (size - e_bounds)).bfloat16()
    _check_selection(b, q, 40, 0, 0)
    _check_selection(b, -q, 41, 1, 1)


def test_selection_of_a_page_of_many_terms_below_the_smallest_number():
    """A score of 51 * 2^-149 whose terms FP32 rounds to zero, beside one of 2^-149 that it does not."""
    b = _bounds_only([2], 1, 1, "bf16")
    first, second = (int(b.table[0, i]) for i in (0, 1))
    b.bounds.zero_()
    b.bounds[first, 0, 1] = 1.6 * 2.0**-76
    b.bounds[second, 0, 1, 9] = 2.0**-74
    q = torch.full((1, 1, D), 2.0**-75, dtype=torch.bfloat16, device="cuda")
    sel = kvq.kvq_paged_select(b.cache, b.table, b.seq, q, 1, n_first=0, n_last=0)
    assert sel.flatten().tolist() == [0]


@pytest.mark.parametrize("wide", [False, True])
def test_selection_that_takes_all_pages_checks_them(wide):
    """A page outside the pool sets the error bit also where no page has to be scored (one launch, two launches)."""
    b = Batch([100, 90, 1600], 16, 2, "bf16")
    if wide:
        pad = torch.full((3, 3000 - b.table.shape[1]), 1 << 30, dtype=torch.int32, device="cuda")
        b.table = torch.cat([b.table, pad], 1).contiguous()
    q = _query(3, 8)
    good = kvq.kvq_paged_select(b.cache, b.table, b.seq, q, 9)
    assert b.cache.error_word() == 0
    for bad in (b.cache.n_pages, -1):
        table = b.table.clone()
        table[1, 5] = bad  # the last of six
        sel = kvq.kvq_paged_select(b.cache, table, b.seq, q, 9)
        assert torch.equal(sel, good) and b.cache.error_word() == kvq.PAGED_ERR_PAGE
        b.cache.clear_error()


SCALES = [7.0, 49.0, 3.0, 5.0, 9.0, 11.0, 13.0, 1.0, 0.5, 0.1, 0.3, 1e-30, 3.1e30, 3.0e38, 1.2e-38, 2.0**127]


@pytest.mark.parametrize("act", ["bf16", "fp16"])
@pytest.mark.parametrize("rows", [1, 64])
def test_e4m3_append_of_every_number(act, rows):
    """Every 16-bit number, keys and values, by scales with and without an exact reciprocal: the stored code is that of
    the FP32 quotient rounded to nearest even and saturated; the page's bounds are of the codes stored."""
    H = len(SCALES)
    x = torch.arange(-(1 << 15), 1 << 15, dtype=torch.int32).to(torch.int16).view(DT[act]).view(-1, 1, D).expand(-1, H, D)
    n = x.shape[0]
    B = n // rows
    ks, vs = torch.tensor(SCALES), torch.tensor(SCALES[::-1])
    cache = kvq.PagedCache.empty(B, rows, H, torch.float8_e4m3fn, key_bounds=True, k_scale=ks.cuda(), v_scale=vs.cuda())
    table = torch.randperm(B, generator=torch.Generator().manual_seed(1)).int()
    off = None if rows == 1 else torch.arange(0, n + 1, rows, dtype=torch.int32, device="cuda")
    dev = x.contiguous().cuda()
    start = torch.zeros(B, dtype=torch.int32, device="cuda")
    kvq.kvq_paged_append(cache, table.cuda().view(B, 1), start, dev, dev, offsets=off)
    assert cache.error_word() == 0
    for pool, s in ((cache.k, ks), (cache.v, vs)):
        want = (x.float() / s[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(B, rows, H, D)
        got = _raw(pool).cpu()[table.long()].view(torch.float8_e4m3fn)
        nan = torch.isnan(want.float())
        assert torch.equal(torch.isnan(got.float()), nan)
        same = _raw(got) == _raw(want)
        assert (same | nan).all(), [(SCALES, i) for i in (~(same | nan)).nonzero()[:4].tolist()]
        if pool is cache.k:
            lo, hi = cache.key_bounds.float().cpu()[table.long()].unbind(2)
            w = want.float()
            assert torch.equal(torch.nan_to_num(lo, 999.0), torch.nan_to_num(w.amin(1), 999.0))
            assert torch.equal(torch.nan_to_num(hi, 999.0), torch.nan_to_num(w.amax(1), 999.0))


def test_attention_needs_its_own_workspace_only():
    """A table of many pages costs the attention nothing: its workspace is that of a table without pages."""
    b = Batch([300, 40], 16, 2, "bf16")
    q = _query(2, 8)
    out, lse = _attend(b, q)
    small, large = (b.cache.workspace_bytes(2, 8, w) for w in (0, 1 << 20))
    assert 0 < small < large // 4
    ws = torch.empty(small, dtype=torch.uint8, device="cuda")
    wide = torch.full((2, 1 << 16), -5, dtype=torch.int32, device="cuda")
    wide[:, :b.table.shape[1]] = b.table
    got = kvq.kvq_paged_decode_attn(b.cache, wide, b.seq, q, workspace=ws)
    assert torch.equal(got, out)
    sel = kvq.kvq_paged_select(b.cache, wide, b.seq, q, 5)
    want = kvq.kvq_paged_sparse_attn(b.cache, b.table, b.seq, q, sel)
    assert torch.equal(want, kvq.kvq_paged_sparse_attn(b.cache, wide, b.seq, q, sel, workspace=ws))
    with pytest.raises(kvq.KvqError, match="WORKSPACE"):
        kvq.kvq_paged_decode_attn(b.cache, wide, b.seq, q, workspace=ws[:small - 16])
    with pytest.raises(kvq.KvqError, match="WORKSPACE"):
        kvq.kvq_paged_select(b.cache, wide, b.seq, q, 5, workspace=ws)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    kvq.kvq_paged_decode_attn(b.cache, wide, b.seq, q)
    assert torch.cuda.max_memory_allocated() - before < small + 4 * out.numel() * 4 + (1 << 16)


def test_workspace_bytes_of_sizes_beyond_any_call():
    b = Batch([64, 3], 16, 2, "bf16")
    assert b.cache.workspace_bytes(2, 8, 2**31 - 65536) > 0
    for n, hq, width in ((2, 8, 2**31 - 65535), (2, 8, 2**31 - 1), (1 << 26, 8, 0), (2**31 - 1, 2, 0)):
        assert b.cache.workspace_bytes(n, hq, width) == 0


@pytest.mark.parametrize("cache", ["bf16", "fp16", "e4m3"])
def test_softmax_weights_keep_their_bits(cache):
    """Two tokens a request, values 0 and 1, logits 0 and s (one channel, exact): out is the second weight.

    Errors, relative to it, s in (-8, 0]: the scale's log2 e and the argument of exp2 (below 16, or 2^4, in FP16's and
    E4M3's shifted form, half a step of 2^-20 times ln 2): 2^-24 |s| 2 + 2^-21; exp2 itself 2^-22; all that for both
    weights; the split 2^-22 (FP16, E4M3: two parts of 11 bits) or none (BF16: three of 8); sums of two terms in the
    tensor cores, cut off by a step of 2^-23 each, the merge of four warps, division and product: 8 * 2^-23 in all.
    A weight without its last part is off by up to 2^-16 (BF16) or 2^-11."""
    n = 64
    g = _gen(9)
    logit = torch.linspace(-7.9, 0.0, n, device="cuda")
    act = "fp16" if cache == "fp16" else "bf16"
    b = Batch([2] * n, 2, 1, cache, seed=1, bounds=False)
    b.cache.k.copy_(torch.zeros_like(b.cache.k.float()).to(b.dt))
    if cache == "e4m3":  # few codes: the logits' spread comes from the query
        b.k_scale.fill_(1.0)
        b.v_scale.fill_(1.0)
    pages = b.table[:, 0].long()
    keys = torch.full((n,), -1.0, device="cuda").to(b.dt)
    _raw(b.k)[pages, 1, 0, 3] = _raw(keys)
    one = torch.ones((n, D), device="cuda").to(b.dt)
    _raw(b.v)[pages, 0, 0] = 0
    _raw(b.v)[pages, 1, 0] = _raw(one)
    q = torch.zeros((n, 2, D), device="cuda").to(DT[act])
    q[:, 0, 3] = (-logit).to(DT[act])
    q[:, 1, 3] = (-logit * torch.rand(n, generator=g, device="cuda")).to(DT[act])
    out, lse = _attend(b, q, softmax_scale=1.0)
    s = -q[..., 3].double()
    p = s.exp()
    want = p / (1 + p)
    tol = 2 * (2.0**-23 * s.abs() + 2.0**-21 + 2.0**-22) + (0 if cache == "bf16" else 2.0**-22) + 8 * 2.0**-23
    err = (out.double() - want[..., None]).abs() / want[..., None]
    assert (err <= tol[..., None]).all(), (err / tol[..., None]).max()
    assert ((lse.double() - torch.log1p(p)).abs() <= tol + 2.0**-22).all()
    # the tolerance tells a weight whose last part is missing: the definition with such weights is outside of it
    bits = 16 if cache == "bf16" else 11
    unit = torch.exp2(torch.floor(torch.log2(p)) + 1 - bits)
    cut = (torch.floor(p / unit) if cache == "bf16" else torch.round(p / unit)) * unit
    assert ((cut / (1 + p) - want).abs() / want > tol).sum() > n // 2
