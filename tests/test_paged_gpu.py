"""The paged cache through the C ABI against plain 64-bit implementations:
append with rotation, decode attention over the pages, page selection, and
attention over selected pages.

Tolerances are bounds of the arithmetic, taken from the inputs:

- A stored key or rotated query differs from the exact rotation x cos - y sin by
  the FP32 evaluation, at most e32 = 3 * 2^-24 (|x cos| + |y sin|) (two products
  and a sum, each off by half a step), and by one rounding to the stored type, at
  most eps/2 of the value or half the smallest subnormal.
- An attention logit is a sum of 128 exact products accumulated in FP32. Tensor
  cores may cut off where a sum would round, a whole step of 2^-23 for each of
  128 additions, and scaling adds two: |delta| <= 132 * 2^-23 * scale * sum |q k|.
  A weight e^(s - m) then is off by the factor 1 + delta, by the rounding of its
  argument (R * 2^-22 for arguments down to -R, which weigh e^-R, so that
  R e^-R <= 1/e and one step of 2^-22 covers it; two are taken) and by its split
  into two BF16 parts (2^-16). Numerator and denominator both carry that factor,
  and a running sum over T tokens in steps of 16 cuts off at most T/16 + 64 times
  2^-23 (64: merging warps, blocks and rescaling). Element by element:
  |out - exact| <= (2 (delta + 2^-21 + 2^-16) + 2 (T/16 + 64) 2^-23) * sum p |v| / l.
- lse: delta + 2^-21 + (T/16 + 64) 2^-23, and 2^-22 of the value (log, sum, scaling).
- Key bounds are the exact minimum and maximum of the stored keys, selections the
  exact order of the scores: no tolerance.
"""

from __future__ import annotations

import math
import random

import pytest
import torch

from quantized_cross_loop_gb300 import kvq

pytestmark = pytest.mark.gpu

D = 128
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
BITS = {torch.bfloat16: torch.int16, torch.float16: torch.int16, torch.float8_e4m3fn: torch.uint8}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _raw(t):
    return t.view(BITS[t.dtype])


class Batch:
    """A cache whose every place that no request owns holds NaN (also behind each request's last token), the table of
    shuffled pages, and each request's keys and values in 64 bits as stored."""

    def __init__(self, lens, ps, H, dtype, seed=0, layout="token", spread=1.0, room=0, bounds=True, spare=2):
        g = _gen(seed)
        dt = DT[dtype]
        self.lens, self.ps, self.H, self.dt = lens, ps, H, dt
        pages = [-(-(t + room) // ps) for t in lens]
        n = sum(pages) + spare
        shape = (n, H, ps, D) if layout == "head" else (n, ps, H, D)
        if layout == "interleaved":  # K and V of a place side by side in one allocation
            both = torch.full((n, ps, 2, H, D), math.nan, device="cuda").to(dt)
            self.k, self.v = both[:, :, 0], both[:, :, 1]
        else:
            self.k, self.v = (torch.full(shape, math.nan, device="cuda").to(dt) for _ in range(2))
            if layout == "head":
                self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.k_scale = self.v_scale = None
        if dtype == "e4m3":
            self.k_scale, self.v_scale = (0.3 + torch.rand(H, generator=g, device="cuda") for _ in range(2))
        perm = torch.randperm(n, generator=g, device="cuda").tolist()
        W = max(1, max(pages, default=1)) + 1
        table = torch.full((len(lens), W), 1 << 30, dtype=torch.int32)  # behind the last page: never looked at
        self.K, self.V = [], []
        at = 0
        for b, T in enumerate(lens):
            mine = perm[at:at + pages[b]]
            at += pages[b]
            table[b, :len(mine)] = torch.tensor(mine, dtype=torch.int32)
            k = (torch.randn((T, H, D), generator=g, device="cuda") * spread).to(dt)
            v = torch.randn((T, H, D), generator=g, device="cuda").to(dt)
            t = torch.arange(T, device="cuda")
            page = torch.tensor(mine, device="cuda", dtype=torch.long)[t // ps] if T else t
            _raw(self.k)[page, t % ps] = _raw(k)
            _raw(self.v)[page, t % ps] = _raw(v)
            self.K.append(self._scaled(k, self.k_scale))
            self.V.append(self._scaled(v, self.v_scale))
        self.table = table.cuda()
        self.seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.bounds = torch.full((n, H, 2, D), math.nan, device="cuda").to(dt) if bounds else None
        if bounds:
            self.refresh_bounds()
        self.cache = kvq.PagedCache(ps, H, self.k, self.v, self.bounds, self.k_scale, self.v_scale)

    def _scaled(self, x, s):
        return x.double() if s is None else x.double() * s.double()[:, None]

    def refresh_bounds(self):
        for b, T in enumerate(self.lens):
            for p in range(-(-T // self.ps)):
                page = int(self.table[b, p])
                rows = self.k[page, :min(self.ps, T - p * self.ps)].float()
                new = torch.stack([rows.amin(0), rows.amax(0)], 1).to(self.dt)
                _raw(self.bounds)[page] = _raw(new)


def _exact(q, K, V, scale, tokens=None):
    """out, lse and the tolerance terms in 64 bits: q [g, D], K, V [T, D]."""
    if tokens is not None:
        K, V = K[tokens], V[tokens]
    T = K.shape[0]
    if T == 0:
        z = torch.zeros((q.shape[0], D), dtype=torch.float64, device="cuda")
        return z, torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device="cuda"), z, z[:, 0]
    q = q.double()
    s = q @ K.T * scale
    delta = 132 * 2.0**-23 * scale * (q.abs() @ K.abs().T).amax(1)
    p = torch.softmax(s, 1)
    seq = (T / 16 + 64) * 2.0**-23
    tol = (2 * (delta + 2.0**-21 + 2.0**-16) + 2 * seq)[:, None] * (p @ V.abs())
    lse = torch.logsumexp(s, 1)
    return p @ V, lse, tol, delta + 2.0**-21 + seq + 2.0**-22 * lse.abs()


def _compare(batch, q, out, lse, scale, sel=None, skip=()):
    H, g = batch.H, q.shape[1] // batch.H
    for b, T in enumerate(batch.lens):
        if b in skip:
            assert torch.isnan(out[b]).all() and torch.isnan(lse[b]).all()
            continue
        for h in range(H):
            tokens = None
            if sel is not None:
                pg = sel[b, h][sel[b, h] >= 0].long()
                tokens = (pg[:, None] * batch.ps + torch.arange(batch.ps, device="cuda")).flatten()
                tokens = tokens[tokens < T]
            r = slice(h * g, (h + 1) * g)
            o, l, to, tl = _exact(q[b, r], batch.K[b][:, h], batch.V[b][:, h], scale, tokens)
            assert (out[b, r].double() - o).abs().le(to + 1e-30).all(), (b, h, (out[b, r] - o).abs().max())
            same = lse[b, r].double() == l
            assert (same | (lse[b, r].double() - l).abs().le(tl)).all(), (b, h, lse[b, r], l)


def _attend(batch, q, **kw):
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out = kvq.kvq_paged_decode_attn(batch.cache, batch.table, batch.seq, q, lse=lse, **kw)
    return out, lse


def _query(B, Hq, act="bf16", seed=5, gain=1.0):
    return (torch.randn((B, Hq, D), generator=_gen(seed), device="cuda") * gain).to(DT[act])


# ------------------------------------------------------------------ attention over all pages


@pytest.mark.parametrize("cache,act", [("bf16", "bf16"), ("fp16", "fp16"), ("e4m3", "bf16"), ("e4m3", "fp16")])
@pytest.mark.parametrize("lens,ps,H,g,layout", [
    ([1], 64, 1, 1, "token"),
    ([0, 1, 63, 64, 65, 0, 129, 1000], 64, 8, 4, "token"),
    ([5, 17, 100], 1, 2, 3, "token"),
    ([31, 33, 200], 7, 3, 5, "head"),
    ([300, 12], 48, 2, 8, "interleaved"),
    ([700, 1, 90], 16, 1, 16, "head"),
    ([257], 1024, 4, 11, "token"),
    ([9001], 32, 8, 4, "token"),
])
def test_attention(cache, act, lens, ps, H, g, layout):
    b = Batch(lens, ps, H, cache, seed=sum(lens) + g, layout=layout)
    q = _query(len(lens), H * g, act)
    out, lse = _attend(b, q)
    _compare(b, q, out, lse, 1 / math.sqrt(D))
    assert b.cache.error_word() == 0


def test_attention_many_requests_and_long_one():
    """More (request, head) pairs than blocks, lengths from 0 to long, so that ranges cross many requests."""
    rng = random.Random(3)
    lens = [rng.choice([0, 0, 1, rng.randint(1, 90), rng.randint(1, 700)]) for _ in range(500)] + [20011]
    b = Batch(lens, 16, 2, "bf16", seed=1, bounds=False)
    q = _query(len(lens), 8)
    out, lse = _attend(b, q)
    _compare(b, q, out, lse, 1 / math.sqrt(D))


@pytest.mark.parametrize("cache", ["bf16", "fp16", "e4m3"])
def test_attention_of_large_logits(cache):
    """Logits of hundreds: single tokens take nearly all weight, the running maximum moves by more than FP32's exponent."""
    b = Batch([333, 64, 2000], 16, 2, cache, seed=8, spread=12.0)
    act = "fp16" if cache == "fp16" else "bf16"
    q = _query(3, 8, act, gain=6.0)
    out, lse = _attend(b, q, softmax_scale=0.5)
    _compare(b, q, out, lse, 0.5)


@pytest.mark.parametrize("gain", [2.0**-60, 2.0**-20, 2.0**10, 2.0**40])
def test_attention_e4m3_with_small_and_large_queries(gain):
    """BF16 queries beyond FP16's range against 8-bit keys: the scale brings the logits back."""
    b = Batch([200, 77], 16, 2, "e4m3", seed=9)
    q = _query(2, 8, gain=gain)
    q[0, 3] = 0
    out, lse = _attend(b, q, softmax_scale=0.1 / gain if gain < 2.0**30 else 2.0**-44)
    _compare(b, q, out, lse, 0.1 / gain if gain < 2.0**30 else 2.0**-44)


def test_attention_strided_queries_own_buffers_and_no_lse():
    b = Batch([100, 37, 0], 16, 2, "bf16")
    wide = torch.randn((3, 12, D), generator=_gen(1), device="cuda").bfloat16()  # q | k | v of a projection
    q = wide[:, :8]
    out = torch.full((3, 8, D), 3.0, device="cuda")
    ws = torch.full((b.cache.workspace_bytes(3, 8, b.table.shape[1]),), 0xAB, dtype=torch.uint8, device="cuda")
    r = kvq.kvq_paged_decode_attn(b.cache, b.table, b.seq, q, out=out, workspace=ws)
    assert r is out
    lse = torch.empty((3, 8), device="cuda")
    again = kvq.kvq_paged_decode_attn(b.cache, b.table, b.seq, q, lse=lse, workspace=ws)
    assert torch.equal(out, again)  # the same call gives the same bits
    _compare(b, q, out, lse, 1 / math.sqrt(D))
    one = kvq.kvq_paged_decode_attn(b.cache, b.table[:1], b.seq[:1], q[:1])
    assert torch.equal(one, kvq.kvq_paged_decode_attn(b.cache, b.table[:1], b.seq[:1], q[:1].contiguous()))


def test_nan_key_stays_in_its_request_and_head():
    b = Batch([100, 90, 80], 16, 2, "bf16")
    b.k[int(b.table[1, 2]), 3, 1, 7] = math.nan
    q = _query(3, 8)
    out, lse = _attend(b, q)
    assert torch.isnan(out[1, 4:]).all() and torch.isnan(lse[1, 4:]).all()
    b.K[1][:, 1] = 0
    keep = torch.isfinite(out)
    assert keep[0].all() and keep[2].all() and keep[1, :4].all()


def test_refused_requests_are_nan_and_flagged():
    """A negative length, one beyond the table, a page outside the pool (both ends): only those requests are NaN."""
    b = Batch([100, 90, 80, 70, 60], 16, 2, "bf16")
    q = _query(5, 8)
    b.seq[0] = -1
    b.seq[2] = b.table.shape[1] * 16 + 1
    _compare(b, q, *_attend(b, q), 1 / math.sqrt(D), skip=(0, 2))
    assert b.cache.error_word() == kvq.PAGED_ERR_LENGTH
    b.cache.clear_error()
    b.seq[0], b.seq[2] = 100, 80
    b.table[1, 5] = b.cache.n_pages
    b.table[3, 0] = -7
    _compare(b, q, *_attend(b, q), 1 / math.sqrt(D), skip=(1, 3))
    assert b.cache.error_word() == kvq.PAGED_ERR_PAGE


def test_offsets_beyond_32_bits():
    """Pages more than 2^32 bytes (and 2^31 elements) into the pool, read and written."""
    ps, H, n = 64, 8, 36000  # 36000 * 64 * 8 * 128 * 2 bytes = 4.7 GB each
    k, v = (torch.empty((n, ps, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bounds = torch.zeros((n, H, 2, D), dtype=torch.bfloat16, device="cuda")
    cache = kvq.PagedCache(ps, H, k, v, bounds)
    table = torch.tensor([[n - 1, 3, n - 2]], dtype=torch.int32, device="cuda")
    T = 150
    kn, vn = (torch.randn((T, H, D), generator=_gen(s), device="cuda").bfloat16() for s in (1, 2))
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvq.kvq_paged_append(cache, table, zero, kn, vn, offsets=torch.tensor([0, T], dtype=torch.int32, device="cuda"))
    assert torch.equal(k[n - 1], kn[:64]) and torch.equal(v[n - 2, :22], vn[128:])
    assert torch.equal(bounds[n - 2, :, 1], kn[128:].amax(0))
    q = _query(1, 32)
    lse = torch.empty((1, 32), device="cuda")
    out = kvq.kvq_paged_decode_attn(cache, table, zero + T, q, lse=lse)
    for h in range(H):
        r = slice(4 * h, 4 * h + 4)
        o, l, to, tl = _exact(q[0, r], kn[:, h].double(), vn[:, h].double(), 1 / math.sqrt(D))
        assert (out[0, r] - o).abs().le(to).all() and (lse[0, r] - l).abs().le(tl).all()


# ------------------------------------------------------------------ selection


def _scores(batch, q, b, h):
    """Exact scores of a request's pages, products of 8-bit and 11-bit significands summed in 64 bits: a positive query
    channel takes the page's largest key, a negative one the smallest (the larger product wherever lo <= hi)."""
    g = q.shape[1] // batch.H
    x = q[b, h * g:(h + 1) * g].double()
    pages = -(-batch.lens[b] // batch.ps)
    bd = batch.bounds.view(BITS[batch.dt])[batch.table[b, :pages].long()].view(batch.dt).double()[:, h]
    return torch.where(x[None] < 0, x[None] * bd[:, None, 0], x[None] * bd[:, None, 1]).sum((1, 2))


def _expected(score, n, first, last):
    P = score.numel()
    if P <= n:
        return list(range(P)) + [-1] * (n - P)
    s = torch.where(torch.isfinite(score), score, torch.full_like(score, 1e300)).clone()
    s[:first] = math.inf
    if last:
        s[P - last:] = math.inf
    return sorted(s.sort(descending=True, stable=True).indices[:n].tolist())


def _check_selection(batch, q, n, first, last, **kw):
    sel = kvq.kvq_paged_select(batch.cache, batch.table, batch.seq, q, n, n_first=first, n_last=last, **kw)
    for b in range(len(batch.lens)):
        for h in range(batch.H):
            assert sel[b, h].tolist() == _expected(_scores(batch, q, b, h), n, first, last), (b, h)
    return sel


@pytest.mark.parametrize("cache,act", [("bf16", "bf16"), ("fp16", "fp16"), ("e4m3", "bf16"), ("e4m3", "fp16")])
@pytest.mark.parametrize("lens,ps,H,g,n,first,last", [
    ([1], 16, 1, 1, 1, 0, 0),
    ([0, 3, 500, 17, 1000], 8, 2, 4, 5, 1, 1),
    ([4000, 900], 7, 3, 5, 40, 0, 0),
    ([5000, 64], 16, 8, 8, 33, 1, 2),
    ([20000], 4, 1, 16, 700, 3, 4),
    ([640], 64, 2, 2, 10, 5, 5),
])
def test_selection(cache, act, lens, ps, H, g, n, first, last):
    b = Batch(lens, ps, H, cache, seed=n)
    _check_selection(b, _query(len(lens), H * g, act), n, first, last)
    assert b.cache.error_word() == 0


@pytest.mark.parametrize("case", ["all", "most", "two"])
def test_selection_ties_take_the_lower_page(case):
    """Pages with the same bounds score the same; pages that differ in one channel by the smallest step are told apart."""
    b = Batch([3000], 8, 2, "bf16")
    ids = b.table[0, :375].long()
    one = torch.randn((2, 2, D), generator=_gen(4), device="cuda").bfloat16()
    if case == "all":
        b.bounds[ids] = one
    elif case == "most":
        b.bounds[ids[::2]] = one
    else:
        b.bounds[ids] = one
        up = _raw(b.bounds)  # one channel's bounds a step up or down, on a few pages
        for i, p in enumerate((371, 200, 37, 3)):
            up[ids[p], :, :, 5 + i] += 1
    _check_selection(b, _query(1, 8), 50, 0, 0)
    _check_selection(b, _query(1, 8, seed=6), 51, 1, 1)


def test_selection_of_scores_that_cancel():
    """Scores near zero from large terms: FP32 sums lose what the order depends on, the order is exact all the same."""
    b = Batch([8 * 600], 8, 1, "bf16")
    ids = b.table[0, :600].long()
    g = _gen(11)
    x = torch.randn((600, 1, 1, D // 2), generator=g, device="cuda").bfloat16() * 256
    small = torch.randn((600, 1, 1, D // 2), generator=g, device="cuda").bfloat16()
    b.bounds[ids, :, :, :D // 2] = x.expand(-1, 1, 2, -1)
    b.bounds[ids, :, :, D // 2:] = -x.expand(-1, 1, 2, -1)
    b.bounds[ids, :, :, 3] += small[..., 3]
    q = _query(1, 2)
    q[..., D // 2:] = q[..., :D // 2]
    _check_selection(b, q, 100, 0, 0)


def test_selection_of_infinite_and_nan_bounds_and_bad_pages():
    b = Batch([1600], 16, 2, "bf16")
    ids = b.table[0, :100].long()
    b.bounds[ids[40], 0, 1, 3] = math.inf
    b.bounds[ids[70], 0, 0, 9] = math.nan
    q = _query(1, 8)
    q[..., 3] = q[..., 3].abs()
    sel = _check_selection(b, q, 7, 0, 1)
    assert 40 in sel[0, 0].tolist() and 70 in sel[0, 0].tolist()
    b.table[0, 55] = b.cache.n_pages  # outside the pool: never chosen by its score
    sel = kvq.kvq_paged_select(b.cache, b.table, b.seq, q, 99, n_first=0, n_last=0)
    assert 55 not in sel[0].unique().tolist() and b.cache.error_word() == kvq.PAGED_ERR_PAGE
    b.cache.clear_error()
    b.seq[0] = -3
    sel = kvq.kvq_paged_select(b.cache, b.table, b.seq, q, 9)
    assert (sel == -1).all() and b.cache.error_word() == kvq.PAGED_ERR_LENGTH


def test_selection_of_many_pages():
    b = Batch([70001, 12], 1, 1, "bf16", seed=3)
    _check_selection(b, _query(2, 2), 513, 2, 2)


# ------------------------------------------------------------------ attention over selected pages


@pytest.mark.parametrize("cache", ["bf16", "fp16", "e4m3"])
@pytest.mark.parametrize("lens,ps,H,g,n", [
    ([1, 0, 16, 17, 500], 16, 2, 4, 3),
    ([1000, 64, 640], 64, 8, 4, 4),
    ([333, 90], 7, 3, 5, 20),
    ([4000], 24, 1, 16, 100),
    ([900], 1, 2, 8, 300),
])
def test_sparse_attention(cache, lens, ps, H, g, n):
    b = Batch(lens, ps, H, cache, seed=n)
    q = _query(len(lens), H * g, "fp16" if cache == "fp16" else "bf16")
    sel = kvq.kvq_paged_select(b.cache, b.table, b.seq, q, n)
    lse = torch.empty(q.shape[:2], device="cuda")
    out = kvq.kvq_paged_sparse_attn(b.cache, b.table, b.seq, q, sel, lse=lse)
    _compare(b, q, out, lse, 1 / math.sqrt(D), sel=sel)
    # every page selected: the whole attention, to the bit of the tolerance's terms
    P = max(1, max(-(-t // ps) for t in lens))
    every = torch.full((len(lens), H, P), -1, dtype=torch.int32, device="cuda")
    for i, t in enumerate(lens):
        m = -(-t // ps)
        every[i, :, :m] = torch.arange(m, device="cuda")
    out = kvq.kvq_paged_sparse_attn(b.cache, b.table, b.seq, q, every, lse=lse)
    _compare(b, q, out, lse, 1 / math.sqrt(D))
    assert b.cache.error_word() == 0


def test_sparse_attention_of_no_pages_and_of_bad_selections():
    b = Batch([500, 400, 300, 200, 100], 16, 2, "bf16")
    q = _query(5, 8)
    sel = torch.tensor([0, 3, 5, -1], dtype=torch.int32, device="cuda").repeat(5, 2, 1).contiguous()
    sel[0, 1] = -1  # nothing selected
    sel[1, 0] = torch.tensor([3, 3, 5, -1])  # the same page twice
    sel[2, 1] = torch.tensor([0, 19, -1, -1])  # behind the last page (300 tokens: pages 0..18)
    sel[3, 0] = torch.tensor([5, 2, -1, -1])  # not ascending
    sel[4, 1] = torch.tensor([-1, 2, -1, -1])  # a page behind the end of the list
    lse = torch.empty((5, 8), device="cuda")
    out = kvq.kvq_paged_sparse_attn(b.cache, b.table, b.seq, q, sel, lse=lse)
    assert b.cache.error_word() == kvq.PAGED_ERR_SELECTION
    assert (out[0, 4:] == 0).all() and torch.isneginf(lse[0, 4:]).all()
    bad = {(1, 0), (2, 1), (3, 0), (4, 1)}
    for r in range(5):
        for h in range(2):
            x, l = out[r, 4 * h:4 * h + 4], lse[r, 4 * h:4 * h + 4]
            if (r, h) in bad:
                assert torch.isnan(x).all() and torch.isnan(l).all(), (r, h)
            elif (r, h) != (0, 1):
                t = (torch.tensor([0, 3, 5], device="cuda")[:, None] * 16 + torch.arange(16, device="cuda")).flatten()
                o, le, to, tl = _exact(q[r, 4 * h:4 * h + 4], b.K[r][:, h], b.V[r][:, h], 1 / math.sqrt(D), t)
                assert (x - o).abs().le(to).all() and (l - le).abs().le(tl).all(), (r, h)


# ------------------------------------------------------------------ append


def _rope(n, R):
    ang = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (
        -torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


def _rotated(x, rope, pos, inter):
    """Exact rotation of x [n, heads, D] and its FP32 error bound."""
    x = x.double()
    R = rope.shape[1]
    c, s = rope[pos].double()[:, None, :R // 2], rope[pos].double()[:, None, R // 2:]
    y, e = x.clone(), torch.zeros_like(x)
    i = (torch.arange(0, R, 2), torch.arange(1, R, 2)) if inter else (torch.arange(R // 2), torch.arange(R // 2, R))
    a, b = x[..., i[0]], x[..., i[1]]
    y[..., i[0]], y[..., i[1]] = a * c - b * s, b * c + a * s
    e[..., i[0]] = 3 * 2.0**-24 * ((a * c).abs() + (b * s).abs())
    e[..., i[1]] = 3 * 2.0**-24 * ((b * c).abs() + (a * s).abs())
    return y, e


HALF = {torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11, torch.float8_e4m3fn: 2.0**-4}
TINY = {torch.bfloat16: 2.0**-134, torch.float16: 2.0**-25, torch.float8_e4m3fn: 2.0**-10}


def _near(stored, exact, e32):
    dt = stored.dtype
    return (stored.double() - exact).abs().le((HALF[dt] * (exact.abs() + e32)).clamp(min=TINY[dt]) + e32).all()


@pytest.mark.parametrize("cache,act", [("bf16", "bf16"), ("fp16", "fp16"), ("e4m3", "bf16"), ("e4m3", "fp16")])
@pytest.mark.parametrize("lens,rows,ps,H,g,R,inter,layout", [
    ([0], [1], 64, 1, 1, 128, False, "token"),
    ([0, 5, 63, 64, 100], None, 64, 8, 4, 128, False, "token"),
    ([0, 5, 63, 64, 100], [0, 1, 2, 65, 200], 64, 8, 4, 128, False, "token"),
    ([7, 0, 30], [33, 0, 1], 16, 3, 2, 64, True, "head"),
    ([7, 0, 30], [33, 100, 1], 5, 2, 5, 96, False, "interleaved"),
    ([0, 11], [700, 3], 48, 1, 16, 0, False, "head"),
    ([3, 9, 1], [4, 2, 1], 2, 2, 1, 8, True, "token"),
])
def test_append(cache, act, lens, rows, ps, H, g, R, inter, layout):
    per = rows or [1] * len(lens)
    room = max(per)
    b = Batch(lens, ps, H, cache, seed=len(lens) + ps, layout=layout, room=room)
    n, pad = sum(per), 0 if rows is None else 3
    wide = (torch.randn((n + pad, (g + 2) * H, D), generator=_gen(2), device="cuda") * (40 if cache == "e4m3" else 1)
            ).to(DT[act])
    q, kn, vn = wide[:, :g * H], wide[:, g * H:(g + 1) * H], wide[:, (g + 1) * H:]
    off = torch.tensor([0] + per).cumsum(0)
    rope = _rope(max(l + r for l, r in zip(lens, per)), R) if R else None
    q_out = torch.full((n + pad, g * H, D), 9.0, device="cuda").to(DT[act])
    k0, v0, b0 = (_raw(t).clone() for t in (b.k, b.v, b.bounds))
    r = kvq.kvq_paged_append(b.cache, b.table, b.seq, kn, vn, offsets=None if rows is None else off.int().cuda(), q=q,
                             q_out=q_out, rope=rope, interleaved=inter)
    assert r is q_out and b.cache.error_word() == 0
    assert torch.equal(b.seq.cpu(), torch.tensor(lens, dtype=torch.int32))
    assert (q_out[n:] == 9.0).all()  # padding rows
    for i, (T, m) in enumerate(zip(lens, per)):
        if m == 0:
            continue
        rr = slice(int(off[i]), int(off[i]) + m)
        pos = torch.arange(T, T + m, device="cuda")
        page, slot = b.table[i].long()[pos // ps], pos % ps
        ek, e32 = _rotated(kn[rr], rope, pos, inter) if R else (kn[rr].double(), torch.zeros_like(kn[rr].double()))
        eq, eq32 = _rotated(q[rr], rope, pos, inter) if R else (q[rr].double(), torch.zeros_like(q[rr].double()))
        ev = vn[rr].double()
        ev32 = torch.zeros_like(ev)
        if b.k_scale is not None:  # the division adds half a step of FP32
            ks, vs = b.k_scale.double()[:, None], b.v_scale.double()[:, None]
            ek, e32, ev = ek / ks, e32 / ks + 2.0**-23 * (ek / ks).abs(), ev / vs
            ev32 = 2.0**-23 * ev.abs()
            ek, ev = ek.clamp(-448, 448), ev.clamp(-448, 448)
        dt = b.k.dtype
        sk, sv = (_raw(t)[page, slot].view(dt) for t in (b.k, b.v))
        assert _near(sk, ek, e32) and _near(q_out[rr], eq, eq32) and _near(sv, ev, ev32)
        if b.k_scale is None:
            assert torch.equal(sv, vn[rr])
        for p in range(T // ps, (T + m - 1) // ps + 1):  # bounds: exactly those of all keys on the page now
            pid = int(b.table[i, p])
            keys = b.k[pid, :min(ps, T + m - p * ps)].float()
            got = b.bounds[pid].float()
            assert torch.equal(got[:, 0], keys.amin(0)) and torch.equal(got[:, 1], keys.amax(0))
            _raw(b.bounds)[pid] = b0[pid]
        _raw(b.k)[page, slot] = k0[page, slot]
        _raw(b.v)[page, slot] = v0[page, slot]
    for now, was in ((b.k, k0), (b.v, v0), (b.bounds, b0)):  # and nothing else has changed
        assert torch.equal(_raw(now), was)


def test_append_in_place_queries_and_given_positions():
    b = Batch([10, 20], 16, 2, "bf16", room=40)
    n = 50
    kn, vn = (torch.randn((n, 2, D), generator=_gen(s), device="cuda").bfloat16() for s in (1, 2))
    q = torch.randn((n, 8, D), generator=_gen(3), device="cuda").bfloat16()
    pos = torch.randint(0, 500, (n,), generator=_gen(4), device="cuda").int()
    rope = _rope(500, 128)
    off = torch.tensor([0, 13, 50], dtype=torch.int32, device="cuda")
    for inter in (False, True):
        x = q.clone()
        kvq.kvq_paged_append(b.cache, b.table, b.seq, kn, vn, offsets=off, q=x, q_out=x, rope=rope, positions=pos,
                             interleaved=inter)
        y, e = _rotated(q, rope, pos.long(), inter)
        assert _near(x, y, e)
        y, e = _rotated(kn, rope, pos.long(), inter)
        t = torch.arange(37, device="cuda") + 20
        assert _near(b.k[b.table[1].long()[t // 16], t % 16], y[13:], e[13:])


def test_append_refusals_leave_everything_alone():
    b = Batch([10, 20, 30, 40], 16, 2, "bf16", room=64)
    kn, vn = (torch.randn((8, 2, D), generator=_gen(s), device="cuda").bfloat16() for s in (1, 2))
    q = torch.randn((8, 2, D), generator=_gen(3), device="cuda").bfloat16()
    rope = _rope(60, 128)
    off = torch.tensor([0, 2, 4, 6, 8], dtype=torch.int32, device="cuda")

    def run(start, off, table=None, positions=None, expect=0, untouched=()):
        k0 = _raw(b.k).clone()
        v0 = _raw(b.v).clone()
        qo = torch.full_like(q, 5.0)
        b.cache.clear_error()
        kvq.kvq_paged_append(b.cache, b.table if table is None else table, start, kn, vn, offsets=off, q=q, q_out=qo,
                             rope=rope, positions=positions)
        assert b.cache.error_word() == expect
        for r in range(8):
            assert ((qo[r] == 5.0).all() == (r in untouched)), r
        changed = (_raw(b.k) != k0).flatten(1).any(1).sum() + (_raw(b.v) != v0).flatten(1).any(1).sum()
        _raw(b.k).copy_(k0)
        _raw(b.v).copy_(v0)
        return int(changed)

    assert run(b.seq, off) > 0
    bad = b.seq.clone()
    bad[1] = -1
    bad[2] = b.table.shape[1] * 16 - 1  # two rows from the last place on
    run(bad, off, expect=kvq.PAGED_ERR_LENGTH, untouched=(2, 3, 4, 5))
    worse = torch.tensor([0, 2, 1, 6, 9], dtype=torch.int32, device="cuda")  # falls; ends behind the rows
    assert run(b.seq, worse, expect=kvq.PAGED_ERR_LENGTH, untouched=(6, 7)) > 0
    neg = torch.tensor([-2, 2, 4, 6, 8], dtype=torch.int32, device="cuda")
    run(b.seq, neg, expect=kvq.PAGED_ERR_LENGTH, untouched=(0, 1))
    table = b.table.clone()
    table[0, 0] = b.cache.n_pages
    table[3, 2] = -1
    run(b.seq, off, table=table, expect=kvq.PAGED_ERR_PAGE, untouched=(0, 1, 6, 7))
    pos = torch.tensor([0, 60, 1, -1, 2, 3, 4, 59], dtype=torch.int32, device="cuda")
    run(b.seq, off, positions=pos, expect=kvq.PAGED_ERR_POSITION, untouched=(1, 3))


def test_append_nan_and_infinite_keys():
    """NaN keys make the page's bounds NaN (the selection then ranks the page first); E4M3 saturates infinities."""
    for cache in ("bf16", "e4m3"):
        b = Batch([5], 16, 1, cache, room=4)
        kn = torch.randn((1, 1, D), generator=_gen(1), device="cuda").bfloat16()
        kn[0, 0, 3], kn[0, 0, 4], kn[0, 0, 5] = math.nan, math.inf, -math.inf
        kvq.kvq_paged_append(b.cache, b.table, b.seq, kn, kn)
        page = int(b.table[0, 0])
        got = b.k[page, 5, 0].float()
        top = 448.0 if cache == "e4m3" else math.inf
        assert torch.isnan(got[3]) and got[4] == top and got[5] == -top
        bd = b.bounds[page, 0].float()
        assert torch.isnan(bd[:, 3]).all() and bd[1, 4] == top and bd[0, 5] == -top


# ------------------------------------------------------------------ as they are used


def test_serving_run():
    """Prompts of three requests appended in two chunks, then decode steps: append, select, sparse and full attention, all
    on one workspace; at the end the full 64-token pages are packed and the rest is a BF16 tail of the packed attention."""
    H, Hq, ps, W = 2, 8, 64, 8
    cache = kvq.PagedCache.empty(40, ps, H, key_bounds=True)
    table = torch.randperm(40, generator=_gen(0), device="cuda")[:3 * W].int().view(3, W).contiguous()
    rope = _rope(W * ps, 128)
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    K, V = [[], [], []], [[], [], []]
    ws = torch.empty(cache.workspace_bytes(3, Hq, W), dtype=torch.uint8, device="cuda")
    seed = 0
    for per in ([130, 1, 64], [7, 90, 0]) + ([1, 1, 1],) * 40:
        seed += 1
        n = sum(per)
        kn, vn = (torch.randn((n, H, D), generator=_gen(100 * seed + i), device="cuda").bfloat16() for i in (0, 1))
        q = torch.randn((n, Hq, D), generator=_gen(100 * seed + 2), device="cuda").bfloat16()
        off = torch.tensor([0] + per).cumsum(0)
        qr = kvq.kvq_paged_append(cache, table, lens, kn, vn, offsets=off.int().cuda(), q=q, rope=rope)
        for b in range(3):
            pos = torch.arange(per[b], device="cuda") + int(lens[b])
            K[b].append(_rotated(kn[off[b]:off[b + 1]], rope, pos, False)[0])
            V[b].append(vn[off[b]:off[b + 1]].double())
        lens += torch.tensor(per, dtype=torch.int32, device="cuda")
    assert cache.error_word() == 0
    q = qr
    lse, lse_s = torch.empty((3, Hq), device="cuda"), torch.empty((3, Hq), device="cuda")
    out = kvq.kvq_paged_decode_attn(cache, table, lens, q, lse=lse, workspace=ws)
    sel = kvq.kvq_paged_select(cache, table, lens, q, 2, workspace=ws)
    sparse = kvq.kvq_paged_sparse_attn(cache, table, lens, q, sel, lse=lse_s, workspace=ws)
    for b in range(3):
        T = int(lens[b])
        pos = torch.arange(T, device="cuda")
        page, slot = table[b].long()[pos // ps], pos % ps
        k, v = torch.cat(K[b]), torch.cat(V[b])
        ks = cache.k[page, slot].double()
        assert (ks - k).abs().le(2.0**-8 * k.abs() + 1e-5).all() and torch.equal(cache.v[page, slot].double(), v)
        for h in range(H):
            r = slice(4 * h, 4 * h + 4)
            o, l, to, tl = _exact(q[b, r], ks[:, h], v[:, h], 1 / math.sqrt(D))
            assert (out[b, r] - o).abs().le(to).all() and (lse[b, r] - l).abs().le(tl).all()
            chosen = sel[b, h].tolist()
            assert 0 in chosen and (T - 1) // ps in chosen
            t = torch.cat([torch.arange(p * ps, min(T, p * ps + ps), device="cuda") for p in chosen if p >= 0])
            o, l, to, tl = _exact(q[b, r], ks[:, h], v[:, h], 1 / math.sqrt(D), t)
            assert (sparse[b, r] - o).abs().le(to).all() and (lse_s[b, r] - l).abs().le(tl).all()
    # flush: request 0's full pages into a packed base, page by page; the pages are kvq_append_tile's tiles as they lie
    T = int(lens[0])
    full = T // 64
    first = int(table[0, 0])
    chains = []
    for kind, pool in ((kvq.KVQ_K, cache.k), (kvq.KVQ_V, cache.v)):
        s = kvq.kvq_encode_base(pool[first], kind, token_cap=64 * full)
        for p in range(1, full):
            kvq.kvq_append_tile([s], [pool[int(table[0, p])]], [None])
        whole = torch.cat([pool[int(table[0, p])] for p in range(full)])
        want = kvq.kvq_encode_base(whole.contiguous(), kind)
        assert torch.equal(s.codes_view(), want.codes_view()) and torch.equal(s.scales_view(), want.scales_view())
        chains.append(s)
    last = int(table[0, full])
    seg = (None, None, cache.k[last, :T - 64 * full], cache.v[last, :T - 64 * full])
    packed = kvq.RequestTable([[chains[0]]], [[chains[1]]], segments=[seg])
    got = kvq.kvq_decode_attn_packed(packed, q[:1].contiguous(), 1, H)
    kh, vh = (kvq.kvq_reconstruct([c], 1).double() for c in chains)
    kx = torch.cat([kh, cache.k[last, :T - 64 * full].double()])
    vx = torch.cat([vh, cache.v[last, :T - 64 * full].double()])
    for h in range(H):
        o = _exact(q[0, 4 * h:4 * h + 4], kx[:, h], vx[:, h], 1 / math.sqrt(D))[0]
        # the packed reader's own tolerance (2e-3 + 1e-2 |x|), and as much for the BF16 rounding of the reconstruction
        assert (got[0, 4 * h:4 * h + 4] - o).abs().le(4e-3 + 2e-2 * o.abs()).all()


def test_joining_by_lse():
    """Attention over two disjoint parts joined by their lse is attention over all."""
    b = Batch([600], 16, 2, "bf16")
    q = _query(1, 8)
    out, lse = _attend(b, q)
    P = 38
    parts = []
    for pages in (range(0, 20), range(20, P)):
        sel = torch.tensor(list(pages), dtype=torch.int32, device="cuda").expand(1, 2, -1).contiguous()
        l = torch.empty((1, 8), device="cuda")
        parts.append((kvq.kvq_paged_sparse_attn(b.cache, b.table, b.seq, q, sel, lse=l), l))
    w = torch.softmax(torch.stack([parts[0][1], parts[1][1]]).double(), 0)[..., None]
    joined = parts[0][0].double() * w[0] + parts[1][0].double() * w[1]
    for h in range(2):
        r = slice(4 * h, 4 * h + 4)
        _, _, to, tl = _exact(q[0, r], b.K[0][:, h], b.V[0][:, h], 1 / math.sqrt(D))
        assert (joined[0, r] - out[0, r]).abs().le(4 * to).all()  # three results, weights off by the lse's tolerance


def test_captured_step_follows_lengths_and_tables():
    """A captured step replayed with other lengths, tables and rows; two graphs on one stream share a workspace."""
    b = Batch([300, 40, 0, 7], 16, 2, "bf16", room=200)
    n = 4
    kn, vn = (torch.randn((n, 2, D), generator=_gen(s), device="cuda").bfloat16() for s in (1, 2))
    q = _query(n, 8)
    rope = _rope(b.table.shape[1] * 16, 128)
    ws = torch.empty(b.cache.workspace_bytes(n, 8, b.table.shape[1]), dtype=torch.uint8, device="cuda")
    start, after = b.seq.clone(), b.seq + 1
    out, lse, qr = torch.empty((n, 8, D), device="cuda"), torch.empty((n, 8), device="cuda"), torch.empty_like(q)
    sel = torch.empty((n, 2, 3), dtype=torch.int32, device="cuda")
    out_s, lse_s = torch.empty_like(out), torch.empty_like(lse)

    def step():
        kvq.kvq_paged_append(b.cache, b.table, start, kn, vn, q=q, q_out=qr, rope=rope)
        kvq.kvq_paged_decode_attn(b.cache, b.table, after, qr, out=out, lse=lse, workspace=ws)

    def sparse():
        kvq.kvq_paged_select(b.cache, b.table, after, qr, 3, sel=sel, workspace=ws)
        kvq.kvq_paged_sparse_attn(b.cache, b.table, after, qr, sel, out=out_s, lse=lse_s, workspace=ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
        sparse()
    torch.cuda.synchronize()
    graphs = []
    for f in (step, sparse):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        graphs.append(g)
    for lens in ([300, 40, 0, 7], [17, 239, 100, 1], [0, 0, 499, 63]):
        kn.normal_(generator=_gen(sum(lens)))
        start.copy_(torch.tensor(lens, dtype=torch.int32))
        after.copy_(start + 1)
        perm = torch.randperm(b.cache.n_pages, generator=_gen(lens[0]), device="cuda").int()
        b.table.copy_(perm[torch.arange(b.table.numel(), device="cuda").view(b.table.shape) % b.cache.n_pages])
        for t in (b.k, b.v, b.bounds):  # finite everywhere: the table now points at any page
            t.copy_(torch.randn(t.shape, generator=_gen(9), device="cuda"))
        for o in (out, lse, out_s, lse_s):
            o.fill_(3.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        want_lse = torch.empty_like(lse)
        want = kvq.kvq_paged_decode_attn(b.cache, b.table, after, qr, lse=want_lse)
        assert torch.equal(want, out) and torch.equal(want_lse, lse)
        want_sel = kvq.kvq_paged_select(b.cache, b.table, after, qr, 3)
        assert torch.equal(want_sel, sel)
        assert torch.equal(kvq.kvq_paged_sparse_attn(b.cache, b.table, after, qr, sel), out_s)
    assert b.cache.error_word() == 0


def test_two_streams_at_once():
    """Calls on two streams, each with buffers that the binding allocates for it, while the default stream works too."""
    b = Batch([3000, 500, 90], 16, 4, "bf16")
    q1, q2 = _query(3, 16, seed=1), _query(3, 16, seed=2)
    want = [kvq.kvq_paged_decode_attn(b.cache, b.table, b.seq, q) for q in (q1, q2)]
    sel = [kvq.kvq_paged_select(b.cache, b.table, b.seq, q, 9) for q in (q1, q2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i in range(20):
        for s, q in zip(streams, (q1, q2)):
            got.append((kvq.kvq_paged_decode_attn(b.cache, b.table, b.seq, q, stream=s),
                        kvq.kvq_paged_select(b.cache, b.table, b.seq, q, 9, stream=s)))
        torch.empty(1 << 20, device="cuda").fill_(float(i))
    torch.cuda.synchronize()
    for i, (o, s) in enumerate(got):
        assert torch.equal(o, want[i % 2]) and torch.equal(s, sel[i % 2])


def test_empty_batch_and_zero_width_table():
    b = Batch([64], 16, 2, "bf16")
    none = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    z = torch.empty((0,), dtype=torch.int32, device="cuda")
    q = torch.empty((0, 8, D), dtype=torch.bfloat16, device="cuda")
    kv = torch.empty((0, 2, D), dtype=torch.bfloat16, device="cuda")
    assert kvq.kvq_paged_decode_attn(b.cache, none, z, q).shape == (0, 8, D)
    assert kvq.kvq_paged_select(b.cache, none, z, q, 3).shape == (0, 2, 3)
    kvq.kvq_paged_append(b.cache, none, z, kv, kv)
    wide = torch.empty((2, 0), dtype=torch.int32, device="cuda")
    lens = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    out = kvq.kvq_paged_decode_attn(b.cache, wide, lens, _query(2, 8))
    assert (out[0] == 0).all() and torch.isnan(out[1]).all()
    assert (kvq.kvq_paged_select(b.cache, wide, lens, _query(2, 8), 3) == -1).all()
    assert b.cache.error_word() == kvq.PAGED_ERR_LENGTH


def test_binding_refusals():
    b = Batch([64, 3], 16, 2, "bf16", room=16)
    q = _query(2, 8)
    E = kvq.KvqError
    with pytest.raises(E, match="float16"):
        kvq.kvq_paged_decode_attn(b.cache, b.table, b.seq, q.float())
    with pytest.raises(E, match="dtype"):
        kvq.kvq_paged_decode_attn(b.cache, b.table, b.seq, q.half())  # FP16 queries of a BF16 cache
    with pytest.raises(E, match="n_q_heads"):
        kvq.kvq_paged_decode_attn(b.cache, b.table, b.seq, q[:, :7].contiguous())
    with pytest.raises(E, match="seq_lens"):
        kvq.kvq_paged_decode_attn(b.cache, b.table, b.seq.long(), q)
    with pytest.raises(E, match="page_table"):
        kvq.kvq_paged_decode_attn(b.cache, b.table.t(), b.seq, q)
    with pytest.raises(E, match="heads of a row"):
        kvq.kvq_paged_decode_attn(b.cache, b.table, b.seq, _query(8, 2).transpose(0, 1))
    with pytest.raises(E, match="WORKSPACE"):
        kvq.kvq_paged_decode_attn(b.cache, b.table, b.seq, q, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(E, match="softmax_scale"):
        kvq.kvq_paged_decode_attn(b.cache, b.table, b.seq, q, softmax_scale=0.0)
    with pytest.raises(E, match="out must be"):
        kvq.kvq_paged_decode_attn(b.cache, b.table, b.seq, q, out=torch.empty((2, 8, D), device="cuda").bfloat16())
    with pytest.raises(E, match="n_first"):
        kvq.kvq_paged_select(b.cache, b.table, b.seq, q, 2, n_first=2, n_last=1)
    with pytest.raises(E, match="sel must be"):
        kvq.kvq_paged_sparse_attn(b.cache, b.table, b.seq, q, torch.zeros((2, 2, 1), device="cuda"))
    bare = kvq.PagedCache(16, 2, b.k, b.v)
    with pytest.raises(E, match="key_bounds"):
        kvq.kvq_paged_select(bare, b.table, b.seq, q, 2)
    kn = torch.zeros((2, 2, D), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(E, match="n_rows"):
        kvq.kvq_paged_append(b.cache, b.table, b.seq, kn[:1], kn[:1])  # one row for two requests, no offsets
    with pytest.raises(E, match="rotary_dim"):
        kvq.kvq_paged_append(b.cache, b.table, b.seq, kn, kn, rope=_rope(8, 12))
    with pytest.raises(E, match="dtype"):
        kvq.kvq_paged_append(b.cache, b.table, b.seq, kn.half(), kn.half())
    with pytest.raises(E, match="bounds alone"):
        kvq.kvq_paged_append(kvq.PagedCache(16, 2, key_bounds=b.bounds), b.table, b.seq, kn, kn)
    with pytest.raises(E, match="overlap"):  # the same row for every place
        one = torch.zeros((1, 1, 2, D), dtype=torch.bfloat16, device="cuda").expand(3, 16, 2, D)
        kvq.kvq_paged_append(kvq.PagedCache(16, 2, one, one), b.table, b.seq, kn, kn)
    with pytest.raises(E, match="scales belong"):
        s = torch.ones(2, device="cuda")
        kvq.kvq_paged_decode_attn(kvq.PagedCache(16, 2, b.k, b.v, None, s, s), b.table, b.seq, q)


def _bounds_only(lens, ps, H, dtype, seed=0):
    """A cache of key bounds alone, finite random bounds lo <= hi, for selections over more pages than a pool would hold."""
    g = _gen(seed)
    b = Batch.__new__(Batch)
    b.lens, b.ps, b.H, b.dt = lens, ps, H, DT[dtype]
    pages = [-(-t // ps) for t in lens]
    n, W = sum(pages) + 1, max(pages)
    mid = torch.randn((n, H, D), generator=g, device="cuda")
    w = torch.rand((n, H, D), generator=g, device="cuda") + 1
    b.bounds = torch.stack([mid - w, mid + w], 2).to(b.dt)
    perm = torch.randperm(n, generator=g, device="cuda").int()
    b.table = torch.full((len(lens), W), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, m in enumerate(pages):
        b.table[i, :m] = perm[at:at + m]
        at += m
    b.seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    b.cache = kvq.PagedCache(ps, H, key_bounds=b.bounds)
    return b


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,H,n,first,last", [
    ([1500] * 12, 8, 40, 1, 1),        # a launch in which a block has a unit, more than 512 pages
    ([300, 12, 4000, 90], 3, 12, 6, 6),  # nothing but the forced pages of the long ones
    ([3000], 1, 2999, 0, 0),
    ([40000, 700], 1, 100, 1, 1),      # more pages than the bit map and the staged keys hold
])
def test_selection_over_many_pages(cache, lens, H, n, first, last):
    b = _bounds_only(lens, 1, H, cache, seed=n)
    _check_selection(b, _query(len(lens), 4 * H), n, first, last)


@pytest.mark.parametrize("lens,H", [([3000], 1), ([1800] * 12, 7), ([40000], 1)])
@pytest.mark.parametrize("differing", [0, 5])
def test_selection_ties_beyond_the_list(lens, H, differing):
    """More pages of the same score than are ranked in shared memory."""
    b = _bounds_only(lens, 1, H, "bf16")
    one = b.bounds[:1].clone()
    b.bounds.copy_(one.expand_as(b.bounds))
    up = _raw(b.bounds)
    for i in range(differing):
        up[b.table[0, 700 + 211 * i].long(), :, :, 3 * i] += 1 + i
    _check_selection(b, _query(len(lens), 2 * H), 1300, 0, 0)
    _check_selection(b, _query(len(lens), 2 * H, seed=7), 60, 2, 3)


@pytest.mark.parametrize("g", [3, 12])
def test_attention_many_units(g):
    """More (request, KV head) pairs than blocks, for either width of the query operand."""
    lens = [(37 * i) % 300 for i in range(170)] + [5000]
    b = Batch(lens, 16, 2, "bf16", seed=g, bounds=False)
    q = _query(len(lens), 2 * g)
    out, lse = _attend(b, q)
    _compare(b, q, out, lse, 1 / math.sqrt(D))


@pytest.mark.parametrize("H,g,cache", [(6, 4, "bf16"), (16, 2, "e4m3"), (64, 1, "fp16"), (160, 1, "bf16"), (7, 16, "bf16")])
def test_attention_head_counts(H, g, cache):
    """Head counts that share the device's blocks out in different ways (lanes of one head, of several, or one lane)."""
    lens = [700, 0, 33, 128, 1, 400]
    b = Batch(lens, 16, H, cache, seed=H, bounds=False)
    q = _query(len(lens), H * g, "fp16" if cache == "fp16" else "bf16")
    out, lse = _attend(b, q)
    _compare(b, q, out, lse, 1 / math.sqrt(D))
    sel = torch.full((len(lens), H, 5), -1, dtype=torch.int32, device="cuda")
    for i, t in enumerate(lens):
        for h in range(H):
            n = min(5, -(-t // 16))
            sel[i, h, :n] = torch.randperm(-(-t // 16), generator=torch.Generator().manual_seed(h))[:n].sort().values.int()
    out = kvq.kvq_paged_sparse_attn(b.cache, b.table, b.seq, q, sel, lse=lse)
    _compare(b, q, out, lse, 1 / math.sqrt(D), sel=sel)


def test_attention_of_keys_that_are_minus_infinity():
    """Logits of -inf weigh nothing; a request of nothing else has no sum."""
    b = Batch([40, 20], 16, 1, "bf16")
    q = _query(2, 4).abs()  # every product with -inf is -inf
    for i in range(2):
        n = 30 if i == 0 else 20  # request 0 keeps ten tokens
        t = torch.arange(n, device="cuda")
        b.k[b.table[i].long()[t // 16], t % 16] = -math.inf
    out, lse = _attend(b, q)
    o, l, to, tl = _exact(q[0], b.K[0][:, 0], b.V[0][:, 0], 1 / math.sqrt(D), torch.arange(30, 40, device="cuda"))
    assert (out[0] - o).abs().le(to).all() and (lse[0] - l).abs().le(tl).all()
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()


def test_more_requests_than_lanes_and_threads():
    """Batches around the sizes at which a block finds its range another way (32 requests, 128 threads)."""
    for n in (31, 32, 33, 127, 128, 129, 400):
        lens = [(13 * i) % 61 for i in range(n)]
        b = Batch(lens, 8, 1, "bf16", seed=n, room=2)
        q = _query(n, 2)
        out, lse = _attend(b, q)
        _compare(b, q, out, lse, 1 / math.sqrt(D))
        _check_selection(b, q, 3, 1, 1)
        per = [(i % 3) for i in range(n)]
        kn = torch.randn((sum(per), 1, D), generator=_gen(n), device="cuda").bfloat16()
        off = torch.tensor([0] + per).cumsum(0)
        kvq.kvq_paged_append(b.cache, b.table, b.seq, kn, kn, offsets=off.int().cuda())
        for i in range(0, n, 7):
            pos = torch.arange(per[i], device="cuda") + lens[i]
            got = b.k[b.table[i].long()[pos // 8], pos % 8]
            assert torch.equal(got, kn[off[i]:off[i + 1]])
        assert b.cache.error_word() == 0


def test_append_without_rotation_has_no_use_for_positions():
    """Without a rotation table no position can be outside it."""
    b = Batch([3], 16, 2, "bf16", room=8)
    kn, vn = (torch.randn((4, 2, D), generator=_gen(s), device="cuda").bfloat16() for s in (1, 2))
    pos = torch.tensor([-1, -5, 1 << 30, 0], dtype=torch.int32, device="cuda")
    for off in (None, torch.tensor([0, 4], dtype=torch.int32, device="cuda")):
        n = 1 if off is None else 4
        q = torch.randn((n, 4, D), generator=_gen(3), device="cuda").bfloat16()
        b.k.zero_()
        got = kvq.kvq_paged_append(b.cache, b.table, b.seq, kn[:n], vn[:n], offsets=off, q=q, positions=pos[:n])
        assert b.cache.error_word() == 0 and torch.equal(got, q)
        page = int(b.table[0, 0])
        assert torch.equal(b.k[page, 3:3 + n], kn[:n]) and torch.equal(b.v[page, 3:3 + n], vn[:n])


@pytest.mark.parametrize("pages", [400, 600])
def test_selection_of_scores_that_cancel_beside_infinite_bounds(pages):
    """A page with an infinite bound in a channel where the query is zero (0 * inf: not finite, so it is taken) stands
    beside pages whose order FP32 loses: theirs is exact all the same."""
    b = Batch([8 * pages], 8, 1, "bf16")
    ids = b.table[0, :pages].long()
    g = _gen(12)
    q = _query(1, 2)
    q[..., 7] = 0.0
    q[..., 3] = q[..., 3].abs()
    perm = torch.randperm(D // 2, generator=g, device="cuda")
    q[..., D // 2:] = q[..., perm]
    b.bounds[ids] = 0.0
    b.bounds[ids, :, :, 3] = -100.0
    infinite = [0, 64, 128]
    near = [p for i in infinite for p in range(i + 1, i + 8)]  # their scores: terms of 2^4 to 2^24, sums below 1
    x = torch.randn((len(near), 1, 1, D // 2), generator=g, device="cuda")
    x = (x * 2.0 ** (4 + 20 * torch.rand(x.shape, generator=g, device="cuda"))).bfloat16()
    b.bounds[ids[near]] = torch.cat([x, -x[..., perm]], 3).expand(-1, 1, 2, -1)
    for c in (3, 7):
        b.bounds[ids[near], :, :, c] = 0.0
        b.bounds[ids[near], :, :, D // 2 + int((perm == c).nonzero())] = 0.0
    b.bounds[ids[near], :, :, 3] = (torch.randn((len(near), 1, 1), generator=g, device="cuda") / 4).bfloat16()
    b.bounds[ids[infinite], :, :, 7] = math.inf
    _check_selection(b, q, 13, 0, 0)


@pytest.mark.parametrize("cache,inter,layout", [("bf16", False, "token"), ("e4m3", True, "head")])
@pytest.mark.parametrize("ps", [8, 32, 33, 64, 256, 1024])
def test_append_of_prompts_among_single_rows(cache, inter, layout, ps):
    """Units of every size side by side: pages that a warp takes, pages that a block takes, requests without rows."""
    rng = random.Random(ps)
    lens = [rng.choice([0, ps - 1, ps, rng.randint(0, 90)]) for _ in range(45)]
    rows = [rng.choice([0, 1, 1, 1, 2, 31, 32, 33]) for _ in range(45)]
    rows[7], rows[8], rows[30], rows[44] = 600, 1, 300, 0
    test_append(cache, "bf16", lens, rows, ps, 3, 2, 128, inter, layout)


def test_workspace_bytes_of_sizes_that_no_call_takes():
    b = Batch([64, 3], 16, 2, "bf16")
    assert b.cache.workspace_bytes(2, 32, 4) > 0
    for n, hq, width in ((-1, 8, 4), (2, 7, 4), (2, 1, 4), (2, 34, 4), (2, 8, -1)):
        assert b.cache.workspace_bytes(n, hq, width) == 0
