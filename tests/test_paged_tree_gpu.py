"""The paged cache's operators for drafted tokens and for 8-bit caches with a scale per token, on the GPU: tree
attention, commit, appending with scales per token, reading back; against implementations in 64 bits."""

from __future__ import annotations

import math
import random

import pytest
import torch

from quantized_cross_loop_gb300 import kvq

pytestmark = pytest.mark.gpu

D = 128
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn, "e4m3t": torch.float8_e4m3fn}
ALL = [("bf16", "bf16"), ("fp16", "fp16"), ("e4m3", "bf16"), ("e4m3", "fp16"), ("e4m3t", "bf16"), ("e4m3t", "fp16")]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _raw(t):
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16)


def _offsets(rows):
    return torch.tensor([0] + rows).cumsum(0).to(torch.int32).cuda()


class Cache:
    """A cache of lens[b] + rows[b] tokens per request: NaN in every place that no token has (scales there too), a table
    of shuffled pages, the tokens' values in 64 bits."""

    def __init__(self, lens, rows, ps, H, dtype, seed=0, layout="token", spread=1.0, room=0, bounds=False):
        g = _gen(seed)
        self.lens, self.rows, self.ps, self.H, self.dtype, dt = list(lens), list(rows), ps, H, dtype, DT[dtype]
        total = [t + n for t, n in zip(lens, rows)]
        pages = [-(-(t + room) // ps) for t in total]
        n = sum(pages) + 2
        if layout == "interleaved":  # K and V of a place side by side in one allocation
            both = torch.full((n, ps, 2, H, D), math.nan, device="cuda").to(dt)
            self.k, self.v = both[:, :, 0], both[:, :, 1]
        else:
            shape = (n, H, ps, D) if layout == "head" else (n, ps, H, D)
            self.k, self.v = (torch.full(shape, math.nan, device="cuda").to(dt) for _ in range(2))
            if layout == "head":
                self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.k_scale = self.v_scale = None
        if dtype == "e4m3":
            self.k_scale, self.v_scale = (0.3 + torch.rand(H, generator=g, device="cuda") for _ in range(2))
        if dtype == "e4m3t":
            self.k_scale, self.v_scale = (torch.full((n, H, ps), math.nan, device="cuda") for _ in range(2))
        perm = torch.randperm(n, generator=g, device="cuda").tolist()
        table = torch.full((len(lens), max([1] + pages) + 1), 1 << 30, dtype=torch.int32)  # behind the last: not read
        at = 0
        for b, p in enumerate(pages):
            table[b, :p] = torch.tensor(perm[at:at + p], dtype=torch.int32)
            at += p
        self.table = table.cuda()
        self.bounds = torch.full((n, H, 2, D), math.nan, device="cuda").to(dt) if bounds else None
        for b, T in enumerate(total):
            for pool, scale in ((self.k, self.k_scale), (self.v, self.v_scale)):
                x = torch.randn((T, H, D), generator=g, device="cuda") * (spread if pool is self.k else 1.0)
                self.put(b, 0, pool, scale, x, g)
        self.seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.cache = kvq.PagedCache(ps, H, self.k, self.v, self.bounds, self.k_scale, self.v_scale)

    def where(self, b, t):
        page = self.table[b].long().clamp(max=self.k.shape[0] - 1)
        return page[t // self.ps], t % self.ps

    def put(self, b, t0, pool, scale, x, g=None):
        t = torch.arange(t0, t0 + x.shape[0], device="cuda")
        page, place = self.where(b, t)
        if self.dtype == "e4m3t":  # scales over several powers of two, not of the rows' own magnitude
            s = torch.exp2(torch.rand((x.shape[0], self.H), generator=g, device="cuda") * 6 - 8)
            scale[page, :, place] = s
            x = (x / s[..., None]).clamp(-448, 448)
        _raw(pool)[page, place] = _raw(x.to(pool.dtype))

    def values(self, b, t0, t1):
        """K and V of tokens t0 .. t1 - 1 in 64 bits."""
        page, place = self.where(b, torch.arange(t0, t1, device="cuda"))
        r = []
        for pool, scale in ((self.k, self.k_scale), (self.v, self.v_scale)):
            x = _raw(pool)[page, place].view(pool.dtype).double()
            if self.dtype == "e4m3":
                x = x * scale.double()[:, None]
            if self.dtype == "e4m3t":
                x = x * scale[page, :, place].double()[..., None]
            r.append(x)
        return r

    def value_scales(self, b, h, T):
        """The scales that are not the same for all of a head's values."""
        if self.dtype != "e4m3t":
            return torch.ones(T, dtype=torch.float64, device="cuda")
        page, place = self.where(b, torch.arange(T, device="cuda"))
        return self.v_scale[page, h, place].double()


def _tree(rows, seed, holes=0.0, words=None):
    """Visibility [n, n] of each request's drafted tokens, and the mask's words."""
    rng = random.Random(seed)
    W = words or max(1, -(-max([1] + rows) // 32))
    seen, out = [], []
    for n in rows:
        s = torch.zeros((n, n), dtype=torch.bool)
        for i in range(n):
            p = rng.randint(max(-1, i - 6), i - 1)
            if p >= 0:
                s[i] = s[p]
            s[i, i] = True
        s &= torch.tensor([rng.random() >= holes for _ in range(n)])[:, None].expand(-1, n) if n else s
        seen.append(s.cuda())
        bits = torch.zeros((n, W * 32), dtype=torch.int64)
        bits[:, :n] = s[:, :W * 32]
        out.append((bits.view(n, W, 32) << torch.arange(32)).sum(2).to(torch.int32))
    return seen, torch.cat(out).cuda() if out else None


def _chain(rows):
    return [torch.ones((n, n), device="cuda").tril() > 0 for n in rows]


def _exact(q, K, V, seen, scale, cache, act, vs):
    """out, lse of rows q [n, D] in 64 bits, and their tolerances. A product of 128 channels summed in FP32 is off by
    `delta`, which moves a logarithmic weight by as much (twice: also the sum's); a weight (times vs [T], its value's
    scale, where tokens have one) is rounded to 16 bits: BF16 by 2^-8 of it, FP16 by 2^-11, or half of FP16's smallest
    step, 2^-25, where the largest weight is at least 2^7: 2^-32 of that one; tensor-core sums cut off up to 2^-23 per 16
    tokens; out is rounded once."""
    q = q.double()
    s = (q @ K.T * scale).masked_fill(~seen, -math.inf)
    none = (s == -math.inf).all(1)
    lse = torch.logsumexp(s, 1)
    p = torch.softmax(s, 1).masked_fill(none[:, None], 0.0)
    Kf, Vf = K.nan_to_num(0, 0, 0), V.nan_to_num(0, 0, 0)
    delta = 136 * 2.0**-23 * scale * (q.abs() @ Kf.abs().T).masked_fill(~seen, 0).amax(1) + 2.0**-20
    seq = (K.shape[0] / 16 + 64) * 2.0**-23
    half = cache != "bf16"
    pv = torch.where(seen[..., None] & (p[..., None] >= 0), p[..., None] * V, 0.0).sum(1)
    pa = p.nan_to_num(0) @ Vf.abs()
    tol = (2 * delta + 2 * seq)[:, None] * pa + (2.0**-11 if half else 2.0**-8) * pa
    if half:
        vs = vs.nan_to_num(0, 0, 0)
        codes = (Vf / torch.where(vs == 0, 1.0, vs)[:, None]).abs()
        tol = tol + 2.0**-32 * (p.nan_to_num(0) * vs).amax(1)[:, None] * codes.sum(0)
    u = 2.0**-11 if act == "fp16" else 2.0**-8
    tol = tol + u * (pv.abs() + tol) + (2.0**-24 if act == "fp16" else 0)
    return pv, lse, tol, delta + seq + 2.0**-21 * lse.abs()


def _attend(c, q, offsets, mask, **kw):
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out = torch.full(q.shape, 7.0, device="cuda", dtype=q.dtype)
    kvq.kvq_paged_tree_attn(c.cache, c.table, c.seq, q, offsets=offsets, mask=mask, out=out, lse=lse, **kw)
    return out, lse


def _compare(c, q, out, lse, seen, scale=1 / math.sqrt(D), refused=()):
    act = "bf16" if q.dtype == torch.bfloat16 else "fp16"
    H, g, at = c.H, q.shape[1] // c.H, 0
    for b, (T, n) in enumerate(zip(c.lens, c.rows)):
        r = slice(at, at + n)
        at += n
        if b in refused:
            assert torch.isnan(out[r]).all() and torch.isnan(lse[r]).all()
            continue
        if n == 0:
            continue
        K, V = c.values(b, 0, T + n)
        see = torch.cat([torch.ones((n, T), dtype=torch.bool, device="cuda"), seen[b]], 1)
        for h in range(H):
            for j in range(h * g, h * g + g):
                o, l, to, tl = _exact(q[r, j], K[:, h], V[:, h], see, scale, c.dtype, act, c.value_scales(b, h, T + n))
                x, y = out[r, j].double(), lse[r, j].double()
                fine = torch.isfinite(o)
                assert ((x == o) | (x.isnan() & o.isnan()) | fine).all(), (b, h, j, "not finite")
                assert (x - o).abs()[fine].le(to[fine] + 1e-30).all(), (b, h, j, ((x - o).abs() / to)[fine].max())
                assert ((y == l) | (y.isnan() & l.isnan()) | (y - l).abs().le(tl)).all(), (b, h, j, y, l)
    assert (out[at:] == 7).all() and (lse[at:] == 7).all()  # padding


def _query(n, Hq, act, seed=5, gain=1.0, wide=0):
    x = (torch.randn((n, Hq + wide, D), generator=_gen(seed), device="cuda") * gain).to(DT[act])
    return x[:, :Hq]


# ------------------------------------------------------------------ tree attention


@pytest.mark.parametrize("cache,act", ALL)
@pytest.mark.parametrize("lens,rows,ps,H,g,layout,kind", [
    ([1], [1], 64, 1, 1, "token", "tree"),
    ([0, 5, 64, 63], [3, 1, 0, 65], 64, 2, 4, "token", "tree"),
    ([100, 0, 257, 128], [8, 16, 31, 33], 16, 2, 4, "token", "tree"),
    ([0, 0, 40], [1, 7, 5], 7, 3, 5, "head", "holes"),
    ([300, 12, 999], [64, 3, 40], 48, 1, 8, "interleaved", "tree"),
    ([130, 700], [17, 129], 16, 1, 16, "head", "holes"),
    ([257], [200], 1024, 2, 3, "token", "none"),
    ([0, 77, 5], [300, 129, 1], 32, 2, 4, "token", "none"),
    ([6000], [20], 32, 2, 4, "token", "tree"),
    ([0], [1024], 64, 1, 2, "token", "none"),
])
def test_tree_attention(cache, act, lens, rows, ps, H, g, layout, kind):
    c = Cache(lens, rows, ps, H, cache, seed=sum(lens) + g, layout=layout)
    q = _query(sum(rows) + 3, H * g, act, wide=2)
    if kind == "none":
        seen, mask = _chain(rows), None
    else:
        seen, mask = _tree(rows, 7, 0.3 if kind == "holes" else 0.0)
        mask = torch.cat([mask, torch.full((3, mask.shape[1]), -1, dtype=torch.int32, device="cuda")])
    out, lse = _attend(c, q, _offsets(rows), mask)
    _compare(c, q, out, lse, seen)
    assert c.cache.error_word() == 0


@pytest.mark.parametrize("cache,act", ALL)
def test_one_row_per_request(cache, act):
    """A decode step: no offsets, no mask; lengths around the tile's."""
    lens = [0, 1, 126, 127, 128, 129, 255, 1000, 3]
    c = Cache(lens, [1] * 9, 16, 2, cache, seed=3)
    q = _query(9, 8, act)
    out, lse = _attend(c, q, None, None)
    _compare(c, q, out, lse, _chain([1] * 9))


def test_many_requests_and_a_long_one():
    """More units than blocks, ranges that cross many requests, and units that many blocks share."""
    rng = random.Random(3)
    lens = [rng.choice([0, 1, rng.randint(1, 90), rng.randint(1, 700)]) for _ in range(300)] + [40011]
    rows = [rng.choice([0, 1, 4, rng.randint(1, 40)]) for _ in range(300)] + [35]
    c = Cache(lens, rows, 16, 2, "bf16", seed=1)
    q = _query(sum(rows), 8, "bf16")
    seen, mask = _tree(rows, 2)
    out, lse = _attend(c, q, _offsets(rows), mask)
    _compare(c, q, out, lse, seen)


@pytest.mark.parametrize("cache,act", ALL)
@pytest.mark.parametrize("rows", [(1, 3), (20, 33), (30, 70)])
def test_many_short_units(cache, act, rows):
    """Units of one or two tiles, many to a block: queries, rings and flags are used anew at every turn."""
    rng = random.Random(5)
    B = 700 if rows[1] < 10 else 300
    lens = [rng.randint(0, 200) for _ in range(B)]
    n = [rng.randint(*rows) for _ in range(B)]
    c = Cache(lens, n, 32, 2, cache, seed=2)
    q = _query(sum(n), 8, act)
    seen, mask = _tree(n, 4, 0.1)
    out, lse = _attend(c, q, _offsets(n), mask)
    for b in range(0, B, 23):  # (a sample, the same of every form)
        r = slice(sum(n[:b]), sum(n[:b + 1]))
        K, V = c.values(b, 0, lens[b] + n[b])
        see = torch.cat([torch.ones((n[b], lens[b]), dtype=torch.bool, device="cuda"), seen[b]], 1)
        for j in range(8):
            o, l, to, tl = _exact(q[r, j], K[:, j // 4], V[:, j // 4], see, 1 / math.sqrt(D), cache, act,
                                  c.value_scales(b, j // 4, lens[b] + n[b]))
            assert (out[r, j].double() - o).abs().le(to + 1e-30).all(), (b, j)
            y = lse[r, j].double()
            assert ((y == l) | (y - l).abs().le(tl)).all(), (b, j)
    assert c.cache.error_word() == 0
    again, lse2 = _attend(c, q, _offsets(n), mask)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("cache", ["e4m3", "e4m3t", "bf16"])
def test_queries_of_channels_far_apart(cache):
    """The largest channel meets keys of zero there: what the small ones find is all that counts."""
    c = Cache([300, 70], [5, 40], 16, 2, cache, seed=3)
    _raw(c.k)[..., 7] = 0
    q = _query(45, 8, "bf16")
    q[..., 7] = 2.0**70
    q[::2] = q[::2] * 2.0**-3
    seen, mask = _tree([5, 40], 2)
    out, lse = _attend(c, q, _offsets([5, 40]), mask)
    _compare(c, q, out, lse, seen)


@pytest.mark.parametrize("cache,act", [("bf16", "bf16"), ("e4m3t", "bf16"), ("fp16", "fp16")])
def test_long_shared_units(cache, act):
    """One request whose units' tokens are cut among all blocks, with two row tiles."""
    c = Cache([30001], [50], 16, 1, cache, seed=2)
    q = _query(50, 4, act)
    seen, mask = _tree([50], 4)
    out, lse = _attend(c, q, _offsets([50]), mask)
    _compare(c, q, out, lse, seen)


@pytest.mark.parametrize("cache,act", ALL)
def test_large_logits(cache, act):
    """Logits of hundreds: the running maximum moves by more than FP32's exponent, single tokens take nearly all."""
    c = Cache([333, 2000], [9, 30], 16, 2, cache, seed=8, spread=12.0 if cache != "e4m3t" else 1.0)
    q = _query(39, 8, act, gain=6.0)
    seen, mask = _tree([9, 30], 1)
    out, lse = _attend(c, q, _offsets([9, 30]), mask, softmax_scale=0.5)
    _compare(c, q, out, lse, seen, 0.5)


@pytest.mark.parametrize("cache,act", ALL)
def test_rising_maximum(cache, act):
    """Every tile's largest score far above the last one's: the sums are rescaled at every step."""
    c = Cache([1500], [5], 16, 1, cache, seed=9)
    for t in range(1500):
        page, place = c.where(0, torch.tensor([t], device="cuda"))
        x = torch.full((1, 1, D), (t // 100 + 1) * 0.25, device="cuda")
        c.put(0, t, c.k, c.k_scale, x, _gen(t))
    q = torch.ones((5, 4, D), device="cuda").to(DT[act])
    out, lse = _attend(c, q, _offsets([5]), None)
    _compare(c, q, out, lse, _chain([5]))


@pytest.mark.parametrize("cache,act", ALL)
@pytest.mark.parametrize("what", ["k", "v"])
def test_values_that_are_not_finite(cache, act, what):
    """A drafted token that is not finite counts for the rows that see it, not for the others."""
    rows = [12, 40]
    c = Cache([70, 0], rows, 16, 2, cache, seed=4)
    seen, mask = _tree(rows, 6)
    pool, scale = (c.k, c.k_scale) if what == "k" else (c.v, c.v_scale)
    bad = [math.nan] if cache.startswith("e4m3") else [math.nan, math.inf, -math.inf]
    for b, t in ((0, 73), (0, 79), (1, 5), (1, 20)):
        page, place = c.where(b, torch.tensor([t], device="cuda"))
        if cache == "e4m3t" and t in (73, 5):
            scale[page, 1, place] = math.inf if what == "v" and t == 5 else math.nan
        else:
            _raw(pool)[page, place, 1, t] = _raw(torch.tensor([bad[t % len(bad)]], device="cuda").to(pool.dtype))
    q = _query(sum(rows), 8, act)
    out, lse = _attend(c, q, _offsets(rows), mask)
    at = 0
    for b, n in enumerate(rows):
        K, V = c.values(b, 0, c.lens[b] + n)
        for i in range(n):
            t = [x for x in range(c.lens[b] + n) if x < c.lens[b] or seen[b][i, x - c.lens[b]]]
            for j in range(8):
                h = j // 4
                s = q[at + i, j].double() @ K[t, h].T / math.sqrt(D)
                o, ok = torch.softmax(s, 0) @ V[t, h], True
                x, l = out[at + i, j].double(), lse[at + i, j].double()
                if torch.isnan(s).any() or torch.isposinf(s).any():
                    assert torch.isnan(x).all() and (torch.isnan(l) or what == "k")
                else:
                    ok = torch.isfinite(o)
                    assert ((x == o) | (x.isnan() & o.isnan()) | ok).all(), (b, i, j, x[~ok], o[~ok])
                    assert ((x - o)[ok].abs() <= 0.05).all(), (b, i, j)
        at += n
    assert torch.isfinite(out[:, :4]).all()  # the other KV head


@pytest.mark.parametrize("act", ["bf16", "fp16"])
@pytest.mark.parametrize("low,high", [(-126, -100), (-60, 60), (-110, 0), (30, 100)])
def test_scales_far_apart(act, low, high):
    """Values' scales over many powers of two, against the keys' order: the tokens that weigh most have the smallest."""
    c = Cache([700, 90], [9, 130], 16, 2, "e4m3t", seed=3)
    for b, T in enumerate([709, 220]):
        page, place = c.where(b, torch.arange(T, device="cuda"))
        e = torch.linspace(high, low, T, device="cuda").round()
        c.v_scale[page, :, place] = torch.exp2(e)[:, None]
    q = _query(139, 8, act)
    seen, mask = _tree([9, 130], 6)
    out, lse = _attend(c, q, _offsets([9, 130]), mask)
    if act == "bf16" or high < 0:
        _compare(c, q, out, lse, seen)
    else:  # (FP16 cannot hold such results: infinite, but the sums are right)
        fine = torch.full_like(lse, 0.0)
        at = 0
        for b, n in enumerate(c.rows):
            K, _ = c.values(b, 0, c.lens[b] + n)
            see = torch.cat([torch.ones((n, c.lens[b]), dtype=torch.bool, device="cuda"), seen[b]], 1)
            for j in range(8):
                s = (q[at:at + n, j].double() @ K[:, j // 4].T / math.sqrt(D)).masked_fill(~see, -math.inf)
                fine[at:at + n, j] = torch.logsumexp(s, 1)
            at += n
        assert (lse - fine).abs().max() < 1e-4


def test_keys_of_minus_infinite_score_weigh_nothing():
    c = Cache([3], [2], 16, 1, "bf16", seed=2)
    for t in range(5):
        page, place = c.where(0, torch.tensor([t], device="cuda"))
        c.k[page, place, 0, 0] = -math.inf
    q = _query(2, 2, "bf16").abs() + 1
    out, lse = _attend(c, q, _offsets([2]), None)
    assert (out == 0).all() and (lse == -math.inf).all()


def test_refused_requests():
    rows = [2, 3, 4, 5, 33]
    c = Cache([20, 30, 40, 50, 10], rows, 16, 2, "bf16", seed=4)
    q = _query(sum(rows) + 2, 8, "bf16")
    seen, mask = _tree(rows, 1, words=1)  # (one word: 33 rows are too many)
    mask = torch.cat([mask, mask[:2]])
    off = _offsets(rows)
    c.seq[0] = -1
    c.seq[1] = c.table.shape[1] * 16 - 2  # two of three rows fit
    c.table[2, 1] = c.k.shape[0]
    out, lse = _attend(c, q, off, mask)
    _compare(c, q, out, lse, seen, refused=(0, 1, 2, 4))
    assert c.cache.error_word() == kvq.PAGED_ERR_LENGTH | kvq.PAGED_ERR_PAGE
    c.cache.clear_error()
    c.seq[:] = torch.tensor(c.lens, dtype=torch.int32)
    c.table[2, 1] = -5
    out, lse = _attend(c, q, off, None)
    _compare(c, q, out, lse, _chain(rows), refused=(2,))
    assert c.cache.error_word() == kvq.PAGED_ERR_PAGE
    c.cache.clear_error()
    bad = off.clone()
    bad[2] = 1000  # requests 1 and 2 have no rows then
    out, lse = _attend(c, q, bad, None)
    assert (out[2:9] == 7).all() and (lse[2:9] == 7).all() and torch.isfinite(out[9:47]).all()
    assert c.cache.error_word() == kvq.PAGED_ERR_LENGTH


def test_too_many_rows_are_refused():
    rows = [1025, 2]
    c = Cache([5, 6], rows, 64, 1, "fp16", seed=4)
    q = _query(1027, 1, "fp16")
    out, lse = _attend(c, q, _offsets(rows), None)
    _compare(c, q, out, lse, _chain(rows), refused=(0,))
    assert c.cache.error_word() == kvq.PAGED_ERR_LENGTH


@pytest.mark.parametrize("cache,act", [("bf16", "bf16"), ("e4m3t", "fp16")])
def test_captured_calls_follow_lengths_tables_and_masks(cache, act):
    """Two captured calls share a workspace; replays read the lengths, offsets, masks and pages of the time."""
    rows = [6, 30, 9]
    c = Cache([100, 900, 300], rows, 16, 2, cache, seed=6)
    n = sum(rows)
    q = _query(n, 8, act)
    seen, mask = _tree(rows, 3)
    off = _offsets(rows)
    ws = torch.empty(c.cache.tree_workspace_bytes(3, 8, n), dtype=torch.uint8, device="cuda")
    outs = [(torch.full(q.shape, 7.0, device="cuda", dtype=q.dtype), torch.full((n, 8), 7.0, device="cuda"))
            for _ in range(2)]

    def call(i, m):
        kvq.kvq_paged_tree_attn(c.cache, c.table, c.seq, q, offsets=off, mask=m, out=outs[i][0], lse=outs[i][1],
                                workspace=ws)

    call(0, mask)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0, mask)
        call(1, None)
    for step in range(3):
        graph.replay()
        torch.cuda.synchronize()
        _compare(c, q, *outs[0], seen)
        _compare(c, q, *outs[1], _chain(rows))
        # other requests, other trees: what was request 1 is request 0 now
        order = [(b + 1) % 3 for b in range(3)]
        c.table.copy_(c.table[order].clone())
        c.lens, c.rows = [c.lens[b] for b in order], [c.rows[b] for b in order]
        c.seq.copy_(torch.tensor(c.lens, dtype=torch.int32))
        seen, new = _tree(c.rows, 20 + step)
        rows = c.rows
        mask.copy_(new)
        off.copy_(_offsets(c.rows))


def test_two_streams():
    """Calls with workspaces of their own on two streams at once give what they give alone."""
    c = Cache([3000, 500], [20, 64], 16, 2, "bf16", seed=6)
    seen, mask = _tree([20, 64], 3)
    off = _offsets([20, 64])
    q = [_query(84, 8, "bf16", seed=s) for s in (1, 2)]
    alone = [_attend(c, x, off, mask) for x in q]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for i, s in enumerate(streams):
            lse = torch.empty((84, 8), device="cuda")
            with torch.cuda.stream(s):
                lse = torch.empty((84, 8), device="cuda")
            got[i].append((kvq.kvq_paged_tree_attn(c.cache, c.table, c.seq, q[i], offsets=off, mask=mask, lse=lse,
                                                   stream=s), lse))
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(out, alone[i][0]) and torch.equal(lse, alone[i][1])


# ------------------------------------------------------------------ appending with a scale per token


def _token_cache(pages, ps, H, layout="token"):
    shape = (pages, H, ps, D) if layout == "head" else (pages, ps, H, D)
    k, v = (torch.full(shape, 0.5, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    if layout == "head":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    ks, vs = (torch.full((pages, H, ps), 7.0, device="cuda") for _ in range(2))
    return kvq.PagedCache(ps, H, k, v, None, ks, vs)


def _codes(x):
    """Scale and E4M3 code of rows x (FP32 [..., D]), as documented."""
    top = x.abs().amax(-1)
    s = top / torch.full_like(top, 448.0)  # (by a plain number it would be a product with the reciprocal)
    s = torch.where(s < 2.0**-126, torch.full_like(s, 2.0**-126), s)
    return s, (x / s[..., None]).to(torch.float8_e4m3fn)


@pytest.mark.parametrize("act", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,start,ps,H,layout", [
    ([1, 1, 1], [0, 15, 77], 16, 3, "token"),
    ([5, 0, 40, 1], [3, 9, 0, 63], 16, 2, "head"),
    ([200, 33], [0, 1], 64, 8, "token"),
    ([70], [1000], 1024, 1, "token"),
])
def test_append_with_scales_per_token(act, rows, start, ps, H, layout):
    """Without a rotation scale and codes are exactly those of the FP32 quotients; nothing else is written."""
    g = _gen(sum(rows))
    n, B = sum(rows), len(rows)
    W = max(-(-(t + r) // ps) for t, r in zip(start, rows))
    cache = _token_cache(B * W + 1, ps, H, layout)
    table = torch.randperm(B * W + 1, generator=g, device="cuda")[:B * W].view(B, W).to(torch.int32)
    x = torch.randn((n + 2, 2 * H, D), generator=g, device="cuda")
    x = (x * torch.exp2(torch.rand((n + 2, 2 * H, 1), generator=g, device="cuda") * 12 - 6)).to(DT[act])
    x[0, 0] = 0  # a row of zeros, and one with a single value
    x[n - 1, H] = 0
    x[n - 1, H, 77] = -3.25
    off = None if rows == [1] * B else _offsets(rows)
    if off is None:
        x = x[:n]
    before = [t.clone() for t in (_raw(cache.k), _raw(cache.v), cache.k_scale, cache.v_scale)]
    kvq.kvq_paged_append(cache, table, torch.tensor(start, dtype=torch.int32, device="cuda"), x[:, :H], x[:, H:],
                         offsets=off)
    at = 0
    for b, (t0, r) in enumerate(zip(start, rows)):
        t = torch.arange(t0, t0 + r, device="cuda")
        page, place = table[b].long()[t // ps], t % ps
        for i, pool in enumerate((before[0], before[1])):
            s, c = _codes(x[at:at + r, i * H:i * H + H].float())
            pool[page, place] = _raw(c)
            before[2 + i][page, :, place] = s
        at += r
    for want, got in zip(before, (_raw(cache.k), _raw(cache.v), cache.k_scale, cache.v_scale)):
        assert torch.equal(want, got)
    assert cache.error_word() == 0


@pytest.mark.parametrize("R,inter", [(128, False), (64, True), (32, False)])
@pytest.mark.parametrize("rows", [[1, 1], [30, 7]])
def test_append_with_rotation_and_scales_per_token(R, inter, rows):
    """Rotated keys: FP32 sums of two products are off by 2^-22 of their terms, the scale by as much and its own rounding;
    a code by half a step (2^-4 of it, or 2^-10) and what the quotient is off."""
    g = _gen(R)
    H, ps, n = 2, 16, sum(rows)
    cache = _token_cache(8, ps, H)
    table = torch.arange(8, device="cuda").view(2, 4).to(torch.int32)
    start = torch.tensor([3, 17], dtype=torch.int32, device="cuda")
    k, v, q = (torch.randn((n, h, D), generator=g, device="cuda").to(torch.bfloat16) for h in (H, H, 4))
    ang = torch.rand((64, R // 2), generator=g, device="cuda") * 6
    rope = torch.cat([ang.cos(), ang.sin()], 1).contiguous()
    off = None if rows == [1, 1] else _offsets(rows)
    qr = kvq.kvq_paged_append(cache, table, start, k, v, offsets=off, q=q, rope=rope, interleaved=inter)
    plain = kvq.PagedCache.empty(8, ps, H)
    q16 = kvq.kvq_paged_append(plain, table, start, k, v, offsets=off, q=q, rope=rope, interleaved=inter)
    assert torch.equal(qr, q16)
    at = 0
    for b, r in enumerate(rows):
        t = torch.arange(int(start[b]), int(start[b]) + r, device="cuda")
        page, place = table[b].long()[t // ps], t % ps
        x = k[at:at + r].double()
        c, s = rope[t, None, :R // 2].double(), rope[t, None, R // 2:].double()
        i, j = (slice(0, R, 2), slice(1, R, 2)) if inter else (slice(0, R // 2), slice(R // 2, R))
        y, mag = x.clone(), x.abs()
        y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., j] * c + x[..., i] * s
        mag[..., i], mag[..., j] = (z := x[..., i].abs() + x[..., j].abs()), z
        got = _raw(cache.k)[page, place].view(torch.float8_e4m3fn).double()
        sc = cache.k_scale[page, :, place].double()
        assert ((sc - y.abs().amax(2) / 448) / sc).abs().max() <= 2.0**-20
        err = (got * sc[..., None] - y).abs()
        assert (err <= y.abs() * (2.0**-4 + 2.0**-18) + sc[..., None] * 2.0**-10 + mag * 2.0**-20).all()
        sv, cv = _codes(v[at:at + r].float())
        assert torch.equal(_raw(cache.v)[page, place], _raw(cv)) and torch.equal(cache.v_scale[page, :, place], sv)
        at += r


def test_append_of_rows_at_the_ends_of_the_range():
    """Rows whose scale would be below FP32's normal range, and rows that are not finite."""
    cache = _token_cache(2, 16, 1)
    x = torch.zeros((7, 1, D), device="cuda")
    x[0, 0, 3] = 2.0**-130  # (below the smallest scale's 448ths)
    x[1, 0, :2] = torch.tensor([2.0**-118, -(2.0**-126)])
    x[2, 0, :3] = torch.tensor([3.3e38, -1.0, 1e30])
    x[3, 0, :2] = torch.tensor([math.inf, 1.0])
    x[4, 0, 9] = -math.inf
    x[5, 0, 0] = math.nan
    x[6, 0, :] = 1.0
    x = x.to(torch.bfloat16)
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvq.kvq_paged_append(cache, table, zero, x, x, offsets=_offsets([7]))
    s, c = _codes(x.float())
    for pool, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        for i in (0, 1, 2, 6):
            assert torch.equal(_raw(pool)[1, i], _raw(c)[i]) and scale[1, 0, i] == s[i, 0]
    out = [torch.empty((7, 1, D), device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    kvq.kvq_paged_read(cache, table, zero, *out, offsets=_offsets([7]))
    for o in out:
        assert torch.isnan(o[3:6]).all() and torch.isfinite(o[[0, 1, 2, 6]]).all() and (o[6] == 1).all()


# ------------------------------------------------------------------ reading back


@pytest.mark.parametrize("cache,act", [(c, a) for c in ("bf16", "fp16", "e4m3", "e4m3t") for a in ("bf16", "fp16")])
@pytest.mark.parametrize("lens,start,ps,H,layout", [
    ([64, 64], [0, 0], 64, 8, "token"),
    ([5, 0, 300, 1, 77], [3, 0, 111, 0, 76], 7, 3, "head"),
    ([1000], [1], 16, 1, "interleaved"),
    ([3000, 2000], [0, 500], 1, 2, "token"),
    ([70, 100], [2, 90], 1024, 17, "token"),
])
def test_read(cache, act, lens, start, ps, H, layout):
    c = Cache(lens, [0] * len(lens), ps, H, cache, seed=len(lens), layout=layout)
    rows = [t - s for t, s in zip(lens, start)]
    n = sum(rows)
    both = torch.full((n + 3, 2, H, D), 7.0, device="cuda").to(DT[act])  # strided rows
    k, v = kvq.kvq_paged_read(c.cache, c.table, torch.tensor(start, dtype=torch.int32, device="cuda"), both[:, 0],
                              both[:, 1], offsets=_offsets(rows))
    at = 0
    for b, (s, t) in enumerate(zip(start, lens)):
        K, V = c.values(b, s, t)  # (8-bit values times FP32 scales: FP32 rounds the product before the type does)
        assert torch.equal(k[at:at + t - s], K.float().to(DT[act])) and torch.equal(v[at:at + t - s], V.float().to(DT[act]))
        at += t - s
    assert (both[n:] == 7).all() and c.cache.error_word() == 0


def test_read_one_row_per_request_and_refusals():
    c = Cache([20, 30, 40], [0] * 3, 16, 2, "e4m3t", seed=1)
    k, v = (torch.full((3, 2, D), 7.0, device="cuda", dtype=torch.float16) for _ in range(2))
    start = torch.tensor([19, 0, 33], dtype=torch.int32, device="cuda")
    kvq.kvq_paged_read(c.cache, c.table, start, k, v)
    for b in range(3):
        K, V = c.values(b, int(start[b]), int(start[b]) + 1)
        assert torch.equal(k[b], K[0].float().half()) and torch.equal(v[b], V[0].float().half())
    start[0], start[1] = -1, c.table.shape[1] * 16
    c.table[2, 2] = 999
    kvq.kvq_paged_read(c.cache, c.table, start, k, v)
    assert torch.isnan(k).all() and torch.isnan(v).all()
    assert c.cache.error_word() == kvq.PAGED_ERR_LENGTH | kvq.PAGED_ERR_PAGE
    c.cache.clear_error()
    k.fill_(7)
    off = torch.tensor([0, 2, 1, 3], dtype=torch.int32, device="cuda")  # request 1 has no range
    kvq.kvq_paged_read(c.cache, c.table, torch.zeros_like(start), k, v, offsets=off)
    assert torch.isfinite(k[0]).all()


@pytest.mark.parametrize("cache", ["bf16", "fp16", "e4m3", "e4m3t"])
def test_rows_read_back_are_packed(cache):
    """64 tokens of any cache, read to BF16, are a tile of the packed chain."""
    c = Cache([200], [0], 16, 2, cache, seed=1, layout="head")
    k, v = (torch.empty((128, 2, D), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    kvq.kvq_paged_read(c.cache, c.table, torch.zeros(1, dtype=torch.int32, device="cuda"), k, v, offsets=_offsets([128]))
    K, V = c.values(0, 0, 128)
    for x, want, kind in ((k, K, kvq.KVQ_K), (v, V, kvq.KVQ_V)):
        whole = kvq.kvq_encode_base(want.float().bfloat16(), kind)
        mine = kvq.kvq_encode_base(x, kind)
        assert torch.equal(whole.codes_view(), mine.codes_view())


# ------------------------------------------------------------------ commit


def _all_bits(c):
    return [x.clone() for x in (_raw(c.k), _raw(c.v), c.k_scale, c.v_scale, c.bounds) if x is not None]


@pytest.mark.parametrize("cache,bounds", [("bf16", True), ("fp16", True), ("e4m3", True), ("e4m3t", False), ("bf16", False)])
@pytest.mark.parametrize("lens,accepted,ps,H,layout", [
    ([5], [[0]], 16, 1, "token"),
    ([0, 15, 16, 40], [[], [1, 3, 4], [0, 1, 2], [7]], 16, 2, "token"),
    ([0, 100, 7], [[2, 3, 5, 90], [], list(range(0, 99, 2))], 7, 3, "head"),
    ([63, 1], [list(range(1, 140)), list(range(64)) + [99]], 64, 1, "interleaved"),
    ([500], [[9]], 1024, 8, "token"),
])
def test_commit(cache, bounds, lens, accepted, ps, H, layout):
    rows = [140] * len(lens)
    c = Cache(lens, rows, ps, H, cache, seed=sum(lens), layout=layout, bounds=bounds)
    if bounds:  # with the drafted tokens in them
        for b in range(len(lens)):
            for p in range(-(-(lens[b] + 140) // ps)):
                k = c.k[c.table[b, p].long(), :min(ps, lens[b] + 140 - p * ps)].float()
                c.bounds[c.table[b, p].long()] = torch.stack([k.amin(0), k.amax(0)], 1).to(c.bounds.dtype)
    want = _all_bits(c)
    for b, (T, acc) in enumerate(zip(lens, accepted)):
        if acc:
            src, dst = c.where(b, T + torch.tensor(acc, device="cuda")), c.where(b, T + torch.arange(len(acc), device="cuda"))
            for x in want[:2]:
                x[dst] = x[src].clone()
            if cache == "e4m3t":
                for x in want[2:]:
                    x[dst[0], :, dst[1]] = x[src[0], :, src[1]].clone()
        end = T + len(acc)
        for p in range(T // ps, -(-end // ps) if bounds else 0):
            k = want[0].view(c.k.dtype)[c.table[b, p].long(), :min(ps, end - p * ps)].float()
            want[-1][c.table[b, p].long()] = torch.stack([k.amin(0), k.amax(0)], 1).to(c.bounds.dtype)
    flat = torch.tensor([x for a in accepted for x in a], dtype=torch.int32, device="cuda")
    kvq.kvq_paged_tree_commit(c.cache, c.table, c.seq, flat, _offsets([len(a) for a in accepted]))
    for x, y in zip(want, _all_bits(c)):
        assert torch.equal(_raw(x) if x.dtype == DT["e4m3"] else x.view(torch.int32 if x.element_size() == 4 else x.dtype),
                           _raw(y) if y.dtype == DT["e4m3"] else y.view(torch.int32 if y.element_size() == 4 else y.dtype)) \
            or torch.equal(torch.nan_to_num(x.float()), torch.nan_to_num(y.float()))
    assert c.cache.error_word() == 0


def test_commit_leaves_refused_requests_alone():
    lens = [20] * 8
    c = Cache(lens, [10] * 8, 16, 2, "bf16", seed=4)
    lists = [[3, 2], [-1, 2], [4, 4], [1, 200], [2, 5], [0, 6], [1], [2, 3]]
    c.seq[5] = -1
    c.table[6, 1] = 5000
    want = _all_bits(c)
    src, dst = c.where(4, torch.tensor([22, 25], device="cuda")), c.where(4, torch.tensor([20, 21], device="cuda"))
    src7, dst7 = c.where(7, torch.tensor([22, 23], device="cuda")), c.where(7, torch.tensor([20, 21], device="cuda"))
    for x in want:
        x[dst] = x[src].clone()
        x[dst7] = x[src7].clone()
    flat = torch.tensor([x for a in lists for x in a], dtype=torch.int32, device="cuda")
    kvq.kvq_paged_tree_commit(c.cache, c.table, c.seq, flat, _offsets([len(a) for a in lists]))
    assert all(torch.equal(x, y) for x, y in zip(want, _all_bits(c)))
    assert c.cache.error_word() == kvq.PAGED_ERR_LENGTH | kvq.PAGED_ERR_SELECTION | kvq.PAGED_ERR_PAGE
    c.cache.clear_error()
    off = _offsets([len(a) for a in lists])
    off[3] = 1000
    off[2] = 3
    kvq.kvq_paged_tree_commit(c.cache, c.table, c.seq, flat[:0], torch.zeros_like(off))  # nothing accepted
    assert c.cache.error_word() == kvq.PAGED_ERR_LENGTH  # (request 5's length)


# ------------------------------------------------------------------ together


@pytest.mark.parametrize("cache", ["bf16", "e4m3t"])
def test_a_serving_run(cache):
    """A prompt in two chunks, then steps of drafting, verifying and committing; each attention against the tokens that a
    plain list of keys and values holds."""
    H, Hq, ps, B = 2, 8, 16, 3
    g = _gen(11)
    W = 20
    if cache == "e4m3t":
        pool = kvq.PagedCache.empty(B * W + 2, ps, H, dtype=torch.float8_e4m3fn, token_scales=True)
    else:
        pool = kvq.PagedCache.empty(B * W + 2, ps, H, key_bounds=True)
    table = torch.randperm(B * W, generator=g, device="cuda").view(B, W).to(torch.int32)
    view = Cache.__new__(Cache)
    view.k, view.v, view.k_scale, view.v_scale, view.bounds = pool.k, pool.v, pool.k_scale, pool.v_scale, pool.key_bounds
    view.table, view.ps, view.H, view.dtype, view.cache = table, ps, H, cache, pool
    pos = torch.arange(400, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (
        -torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
    rope = torch.cat([pos.cos(), pos.sin()], 1).float().contiguous()
    lens = [0] * B
    kept = [[] for _ in range(B)]  # stored keys of each request's tokens, as read back

    def step(rows, seen, mask, positions):
        n = sum(rows)
        k, v = (torch.randn((n, H, D), generator=g, device="cuda").bfloat16() for _ in range(2))
        q = torch.randn((n, Hq, D), generator=g, device="cuda").bfloat16()
        seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
        off = _offsets(rows)
        q = kvq.kvq_paged_append(pool, table, seq, k, v, offsets=off, q=q, rope=rope, positions=positions)
        lse = torch.empty((n, Hq), device="cuda")
        out = kvq.kvq_paged_tree_attn(pool, table, seq, q, offsets=off, mask=mask, lse=lse)
        view.lens, view.rows, view.seq = list(lens), rows, seq
        for b in range(B):  # the cached part is what was kept
            if lens[b]:
                assert torch.equal(view.values(b, 0, lens[b])[0], torch.stack(kept[b]))
        _compare(view, q, out, lse, seen)
        return seq

    for rows in ([100, 33, 64], [30, 1, 0]):
        step(rows, _chain(rows), None, None)
        for b, r in enumerate(rows):
            kept[b] += list(view.values(b, lens[b], lens[b] + r)[0])
            lens[b] += r
    for i in range(4):
        rows = [8, 16, 1 + i]
        seen, mask = _tree(rows, 30 + i)
        depth = torch.cat([s.sum(1) for s in seen]).int() - 1
        positions = depth + torch.cat([torch.full((r,), t, device="cuda") for t, r in zip(lens, rows)])
        seq = step(rows, seen, mask, positions.int())
        taken = []
        for b, r in enumerate(rows):  # the path to a leaf
            leaf = r - 1 if i % 2 else r // 2
            taken.append([j for j in range(r) if seen[b][leaf, j]])
            K = view.values(b, lens[b], lens[b] + r)[0]
            kept[b] += [K[j].clone() for j in taken[b]]
        flat = torch.tensor([x for a in taken for x in a], dtype=torch.int32, device="cuda")
        kvq.kvq_paged_tree_commit(pool, table, seq, flat, _offsets([len(a) for a in taken]))
        lens[:] = [t + len(a) for t, a in zip(lens, taken)]
        if cache == "bf16":  # bounds of exactly the tokens that are there
            for b in range(B):
                for p in range(-(-lens[b] // ps)):
                    K = pool.k[table[b, p].long(), :min(ps, lens[b] - p * ps)]
                    assert torch.equal(pool.key_bounds[table[b, p].long()], torch.stack([K.amin(0), K.amax(0)], 1))
    assert pool.error_word() == 0


@pytest.mark.parametrize("cache", ["bf16", "e4m3t"])
def test_a_captured_step_follows_its_inputs(cache):
    """A step of appending, attending, committing and reading back, captured once and replayed with other lengths, rows,
    trees and paths, leaves in one cache what the same calls leave in another, bit for bit."""
    H, Hq, ps, B, W, n = 2, 8, 16, 3, 12, 24
    g = _gen(12)

    def pool():
        if cache == "e4m3t":
            p = kvq.PagedCache.empty(B * W + 1, ps, H, dtype=torch.float8_e4m3fn, token_scales=True)
        else:
            p = kvq.PagedCache.empty(B * W + 1, ps, H, key_bounds=True)
        return p

    pools = [pool(), pool()]
    for p in pools:
        for t in (p.k, p.v, p.k_scale, p.v_scale, p.key_bounds):
            if t is not None:
                t.view(torch.uint8).zero_()
    table = torch.zeros((B, W), dtype=torch.int32, device="cuda")
    start = torch.zeros(B, dtype=torch.int32, device="cuda")
    off, taken_off = (torch.zeros(B + 1, dtype=torch.int32, device="cuda") for _ in range(2))
    taken = torch.zeros(n, dtype=torch.int32, device="cuda")
    mask = torch.zeros((n, 1), dtype=torch.int32, device="cuda")
    k, v = (torch.zeros((n, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros((n, Hq, D), dtype=torch.bfloat16, device="cuda")
    ws = [torch.empty(p.tree_workspace_bytes(B, Hq, n), dtype=torch.uint8, device="cuda") for p in pools]
    outs = [[torch.zeros((n, Hq, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((n, Hq), device="cuda"),
             torch.zeros((n, H, D), dtype=torch.bfloat16, device="cuda"),
             torch.zeros((n, H, D), dtype=torch.bfloat16, device="cuda")] for _ in pools]

    def step(i):
        p, (out, lse, rk, rv) = pools[i], outs[i]
        kvq.kvq_paged_append(p, table, start, k, v, offsets=off)
        kvq.kvq_paged_tree_attn(p, table, start, q, offsets=off, mask=mask, out=out, lse=lse, workspace=ws[i])
        kvq.kvq_paged_tree_commit(p, table, start, taken, taken_off)
        kvq.kvq_paged_read(p, table, start, rk, rv, offsets=taken_off)

    step(0)  # (no rows yet: nothing but the first calls' set-up)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(0)
    lens = [0, 7, 100]
    for rows in ([8, 1, 15], [0, 20, 4], [3, 3, 3], [8, 8, 8]):
        seen, m = _tree(rows, sum(lens))
        paths = [[j for j in range(r) if seen[b][r // 2, j]] if r else [] for b, r in enumerate(rows)]
        flat = [x for a in paths for x in a]
        table.copy_(torch.randperm(B * W, generator=g, device="cuda").view(B, W).to(torch.int32))
        start.copy_(torch.tensor(lens, dtype=torch.int32))
        off.copy_(_offsets(rows))
        taken_off.copy_(_offsets([len(a) for a in paths]))
        taken[:len(flat)] = torch.tensor(flat, dtype=torch.int32, device="cuda")
        mask.zero_()
        mask[:m.shape[0]] = m
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        step(1)
        torch.cuda.synchronize()
        for a, b in zip(*outs):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        for name in ("k", "v", "k_scale", "v_scale", "key_bounds"):
            a, b = (getattr(p, name) for p in pools)
            assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert flat and bool((outs[0][2][:len(flat)] != 0).any())
        lens = [t + len(a) for t, a in zip(lens, paths)]
    assert [p.error_word() for p in pools] == [0, 0]


def test_arguments_of_the_binding():
    c = Cache([20, 30], [2, 3], 16, 2, "e4m3t", seed=1)
    b = Cache([20, 30], [2, 3], 16, 2, "bf16", seed=1)
    q, off = _query(5, 8, "bf16"), _offsets([2, 3])
    E = kvq.KvqError
    with pytest.raises(E, match="kvq_paged_tree_attn"):
        kvq.kvq_paged_decode_attn(c.cache, c.table, c.seq, q[:2].contiguous())
    with pytest.raises(E, match="mask"):
        kvq.kvq_paged_tree_attn(b.cache, b.table, b.seq, q, offsets=off, mask=torch.zeros((5, 1), device="cuda"))
    with pytest.raises(E, match="n_rows"):
        kvq.kvq_paged_tree_attn(b.cache, b.table, b.seq, q)
    with pytest.raises(E, match="q_dtype"):
        kvq.kvq_paged_tree_attn(b.cache, b.table, b.seq, q.half(), offsets=off)
    with pytest.raises(E, match="out"):
        kvq.kvq_paged_tree_attn(b.cache, b.table, b.seq, q, offsets=off, out=torch.empty((5, 8, D), device="cuda"))
    with pytest.raises(E, match="workspace"):
        kvq.kvq_paged_tree_attn(b.cache, b.table, b.seq, q, offsets=off,
                                workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(E, match="key_bounds"):
        kvq.PagedCache(16, 2, c.k, c.v, torch.empty((c.k.shape[0], 2, 2, D), device="cuda").to(torch.float8_e4m3fn),
                       c.k_scale, c.v_scale)
    with pytest.raises(E, match="come together"):
        kvq.PagedCache(16, 2, c.k, c.v, None, c.k_scale, None)
    with pytest.raises(E, match="float8"):
        kvq.PagedCache(16, 2, b.k, b.v, None, *(torch.empty((b.k.shape[0], 2, 16), device="cuda") for _ in range(2)))
    with pytest.raises(E, match="k_out"):
        kvq.kvq_paged_read(b.cache, b.table, b.seq, torch.empty((5, 2, D), device="cuda"), torch.empty((5, 2, D), device="cuda"))
    with pytest.raises(E, match="accepted"):
        kvq.kvq_paged_tree_commit(b.cache, b.table, b.seq, off.long(), off)
    # nothing to do
    out = kvq.kvq_paged_tree_attn(b.cache, b.table, b.seq, q[:0], offsets=torch.zeros_like(off))
    assert out.shape == (0, 8, D)
