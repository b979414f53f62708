"""Workloads of the paged cache's operators for drafted tokens and for 8-bit
caches with a scale per token: quantising keys and values as they are written,
reading a cache back, attention of a tree of drafted tokens (or of a chunk of
tokens) over the cache, and committing the accepted ones.

With ``own`` false ``run`` computes an operator from elementary torch
operations in FP32; with ``own`` true it makes the calls of
``quantized_cross_loop_gb300.kvq``.
"""

from __future__ import annotations

import math
import random

import torch

own = False

D = 128  # channels of a head, as everywhere in the library
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn, "e4m3t": torch.float8_e4m3fn}
E4M3_MAX = 448.0
SMALLEST_SCALE = 2.0**-126


def listed():
    return [
        # one request that verifies a few drafted tokens: latency
        dict(name="tree_one", op="tree", B=1, lo=256, T=256, n=8, same=True, H=8, Hq=32, ps=64, cache="bf16", act="bf16",
             mask="tree", heads_first=False, empty=False, pad=0),
        # a serving batch that verifies small trees over ragged requests
        dict(name="tree_batch", op="tree", B=64, lo=512, T=4095, n=16, same=False, H=8, Hq=32, ps=64, cache="bf16",
             act="bf16", mask="tree", heads_first=False, empty=False, pad=5),
        # wide trees, eight query heads a KV head: the products count, not the cache
        dict(name="tree_wide", op="tree", B=8, lo=16384, T=16384, n=64, same=True, H=8, Hq=64, ps=64, cache="bf16",
             act="bf16", mask="tree", heads_first=False, empty=False, pad=0),
        # long requests in an 8-bit cache of small pages with a scale per token
        dict(name="tree_long_e4m3t", op="tree", B=4, lo=30001, T=65535, n=24, same=False, H=8, Hq=32, ps=16,
             cache="e4m3t", act="bf16", mask="tree", heads_first=True, empty=False, pad=0),
        # plain decoding over such a cache: one token per request
        dict(name="decode_e4m3t", op="tree", B=64, lo=512, T=16383, n=1, same=True, H=8, Hq=32, ps=64, cache="e4m3t",
             act="bf16", mask="none", heads_first=False, empty=True, pad=0),
        # chunks of prompts behind what is cached already
        dict(name="chunk_fp16", op="tree", B=4, lo=1000, T=8192, n=1000, same=False, H=8, Hq=32, ps=64, cache="fp16",
             act="fp16", mask="none", heads_first=False, empty=False, pad=0),
        # one new token per request, quantised as it is written
        dict(name="append_step_e4m3t", op="append", B=64, lo=512, T=2047, H=8, Hq=32, ps=64, cache="e4m3t", act="bf16",
             rows=1, rotary=128, inter=False, pad=0, heads_first=False, empty=False),
        # four long prompts, quantised as they are written
        dict(name="append_prompts_e4m3t", op="append", B=4, lo=0, T=0, H=8, Hq=64, ps=64, cache="e4m3t", act="bf16",
             rows=8192, rotary=128, inter=False, pad=0, heads_first=False, empty=False),
        # the oldest 64 tokens of each request on their way into the packed chain
        dict(name="read_tiles", op="read", B=64, lo=64, T=64, H=8, ps=64, cache="e4m3t", act="bf16", rows=64,
             heads_first=False, empty=False, pad=0),
        # whole requests out of a head-major cache
        dict(name="read_requests", op="read", B=8, lo=1, T=8191, H=8, ps=16, cache="fp16", act="bf16", rows=8191,
             heads_first=True, empty=False, pad=3),
        # the accepted tokens of a serving batch, key bounds kept right
        dict(name="commit_batch", op="commit", B=64, lo=512, T=2047, n=16, take=5, H=8, ps=64, cache="bf16",
             bounds=True, heads_first=False, empty=False),
        # long accepted paths of many requests
        dict(name="commit_long", op="commit", B=256, lo=100, T=2000, n=64, take=32, H=8, ps=16, cache="e4m3t",
             bounds=False, heads_first=True, empty=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "append", "read", "commit"])
    H = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 8, 8, 12, 16] if H < 8 else [1, 2, 3, 4, 5, 8])
    cache = rng.choice(["bf16", "fp16", "e4m3", "e4m3t", "e4m3t"])
    act = cache if cache in ("bf16", "fp16") else rng.choice(["bf16", "fp16"])
    ps = rng.choice([8, 16, 24, 32, 48, 64, 64, 128])
    case = dict(op=op, H=H, ps=ps, cache=cache, act=act, heads_first=rng.random() < 0.4, empty=rng.random() < 0.3)
    if op == "append":
        rows = _log(rng, 1, 4000)
        case.update(cache="e4m3t", act=rng.choice(["bf16", "fp16"]), Hq=H * g, rows=rows,
                    B=max(1, min(_log(rng, 1, 256), 16000 // rows)), T=_log(rng, 1, 1500),
                    rotary=rng.choice([0, 32, 64, 96, 128, 128]), inter=rng.random() < 0.3, pad=rng.choice([0, 0, 1, 50]))
        case.update(lo=rng.choice([0, case["T"] // 2, case["T"]]))
        return case
    if op == "read":
        rows = _log(rng, 1, 8000)
        case.update(act=rng.choice(["bf16", "fp16"]), rows=rows, B=max(1, min(_log(rng, 1, 256), 60000 // rows)),
                    T=rows + _log(rng, 1, 2000), pad=rng.choice([0, 0, 1, 50]))
        case.update(lo=case["T"])
        return case
    if op == "commit":
        n = _log(rng, 1, 128)
        T = _log(rng, 1, 4000)
        case.update(B=max(1, min(_log(rng, 1, 400), 200000 // T)), T=T, lo=rng.choice([0, T // 8, T]), n=n,
                    take=rng.randint(0, n), bounds=cache != "e4m3t" and rng.random() < 0.6)
        return case
    mask = rng.choice(["tree", "tree", "holes", "none"])
    n = _log(rng, 1, 256 if mask != "none" else 1000)
    # no more products, and no more scores for a plain form to hold, than the largest listed case
    most = 500000000 // (n * g * H)
    T = max(1, min(_log(rng, 1, 60000), most - n))
    T += 1 - T % 2 if rng.random() < 0.7 else 0
    B = max(1, min(_log(rng, 1, 300), 250000 // (T + n), most // (T + n)))
    case.update(B=B, lo=rng.choice([T, max(1, T // 8), 0]), T=T, n=n, same=rng.random() < 0.4, Hq=H * g, mask=mask,
                pad=rng.choice([0, 0, 1, 50]))
    return case


# ------------------------------------------------------------------ sizes of a case (from its fields alone)


def _lengths(c):
    """Tokens that each request has cached: T for lo == T, else spread over lo..T by their logarithm; `empty`: every
    fifth has none."""
    rng = random.Random(c["B"] * 1000003 + c["T"] * 31 + c["lo"])
    n = [c["T"] if c["lo"] == c["T"] else min(c["T"], max(c["lo"], _log(rng, c["lo"] + 1, c["T"] + 1) - 1))
         for _ in range(c["B"])]
    return [0 if c["empty"] and b % 5 == 3 else t for b, t in enumerate(n)]


def _rows(c):
    """Rows of each request: drafted tokens, new tokens, or tokens to be read."""
    rng = random.Random(c["B"] * 7919 + c.get("n", 0) * 13 + c.get("rows", 0))
    if c["op"] == "tree":
        n = [c["n"] if c["same"] else rng.randint(max(1, c["n"] // 2), c["n"]) for _ in range(c["B"])]
        return [0 if c["empty"] and b % 7 == 4 and c["n"] > 1 else r for b, r in enumerate(n)]
    if c["op"] == "commit":
        return [c["n"]] * c["B"]
    if c["op"] == "read":
        return [min(t, c["rows"]) for t in _lengths(c)]
    n = [c["rows"] if c["rows"] == 1 or c["B"] == 4 else rng.randint(max(1, c["rows"] // 2), c["rows"])
         for _ in range(c["B"])]
    return n if c["rows"] == 1 else [0 if c["empty"] and b % 5 == 3 else r for b, r in enumerate(n)]


def _accepted(c):
    """Accepted nodes of each request, ascending. They lie behind the places that they move to, or stay where they
    are, so that a second pass over the same pages finds the same tokens."""
    rng = random.Random(c["B"] * 104729 + c["n"] * 31 + c["take"])
    out = []
    for _ in range(c["B"]):
        m = rng.randint(0, c["take"])
        out.append(sorted(rng.sample(range(m, c["n"]), m)) if 2 * m <= c["n"] else list(range(m)))
    return out


def _cdiv(a, b):
    return -(-a // b)


def _words(c):
    return _cdiv(max(1, c["n"]), 32)


def work(case):
    c = case
    cb = 1 if c["cache"].startswith("e4m3") else 2
    row = c["H"] * 2 * (D * cb + (4 if c["cache"] == "e4m3t" else 0))  # a token's keys, values and scales
    lens = _lengths(c)
    if c["op"] == "commit":
        acc = _accepted(c)
        moved = sum(sum(1 for k, x in enumerate(a) if k != x) for a in acc)
        by = 2 * moved * row
        if c["bounds"]:
            for t, a in zip(lens, acc):
                e = t + len(a)
                if e > t // c["ps"] * c["ps"]:
                    by += (e - t // c["ps"] * c["ps"]) * c["H"] * D * cb
                    by += (_cdiv(e, c["ps"]) - t // c["ps"]) * c["H"] * 2 * D * cb
        return {"bytes": max(by, 1), "flops": 0}
    n = sum(_rows(c))
    if c["op"] == "append":
        return {"bytes": n * c["H"] * D * 4 + n * row + n * c["Hq"] * D * 4 + n * c["rotary"] * 4,
                "flops": n * (3 * (c["H"] + c["Hq"]) * c["rotary"] + 6 * c["H"] * D)}
    if c["op"] == "read":
        return {"bytes": n * row + n * c["H"] * D * 4, "flops": 2 * n * c["H"] * D}
    rows = _rows(c)
    by = sum(t + r for t, r in zip(lens, rows) if r) * row + n * c["Hq"] * (D * 4 + 4)
    by += n * _words(c) * 4 if c["mask"] != "none" else 0
    pairs = sum(r * t + (r * (r + 1) // 2 if c["mask"] == "none" else r) for t, r in zip(lens, rows))
    return {"bytes": by, "flops": 4 * D * c["Hq"] * pairs}


# ------------------------------------------------------------------ inputs


def _bits(t):
    return torch.uint8 if t.element_size() == 1 else torch.int16


def _pool(g, c, n_pages):
    """A K or V pool [n_pages][page][H][D] of the cache's type, normal values around a mean of each page, and its
    scales; head-major in memory where the case says so."""
    H, ps = c["H"], c["ps"]
    dt = DTYPES[c["cache"]]
    out = torch.empty((n_pages, H, ps, D) if c["heads_first"] else (n_pages, ps, H, D), dtype=dt, device="cuda")
    scale = None
    if c["cache"] == "e4m3":
        scale = 0.05 + 0.02 * torch.rand(H, generator=g, device="cuda")
    if c["cache"] == "e4m3t":
        scale = torch.empty((n_pages, H, ps), device="cuda")
    for a in range(0, n_pages, 4096):
        e = min(n_pages, a + 4096)
        x = torch.randn((e - a, ps, H, D), generator=g, device="cuda")
        x += torch.randn((e - a, 1, H, D), generator=g, device="cuda") * 0.5
        if c["cache"] == "e4m3":
            x *= 16
        if c["cache"] == "e4m3t":
            s = (x.abs().amax(3) / E4M3_MAX).clamp(min=SMALLEST_SCALE)
            scale[a:e] = s.transpose(1, 2)
            x = (x / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
        out[a:e] = (x.transpose(1, 2) if c["heads_first"] else x).to(dt)
    return (out.transpose(1, 2) if c["heads_first"] else out), scale


def _offsets(rows):
    return torch.tensor([0] + rows, device="cuda").cumsum(0).to(torch.int32)


def _tree_mask(g, c, rows):
    """Bits of the drafted tokens that each row may attend to: its ancestors in a random tree and itself; "holes": some
    rows have none of them."""
    B, N, W = c["B"], max(1, c["n"]), _words(c)
    i = torch.arange(N, device="cuda")
    # a parent within the eight nodes before, or the cached tokens (-1)
    up = (torch.rand((B, N), generator=g, device="cuda") * 9).long() + 1
    parent = (i - up).clamp(min=-1)
    sees = torch.eye(N, device="cuda").repeat(B, 1, 1)
    sees.scatter_add_(2, parent.clamp(min=0)[..., None], (parent >= 0).float()[..., None])
    for _ in range(max(1, (N - 1).bit_length())):
        sees = (sees @ sees).clamp(max=1)
    sees = sees > 0
    if c["mask"] == "holes":
        sees &= (torch.rand((B, N, 1), generator=g, device="cuda") > 0.25)
    bits = torch.zeros((B, N, W * 32), dtype=torch.int64, device="cuda")
    bits[..., :N] = sees
    words = (bits.view(B, N, W, 32) << torch.arange(32, device="cuda")).sum(3).to(torch.int32)
    live = i < torch.tensor(rows, device="cuda")[:, None]
    return torch.cat([words[live], words.new_zeros((c["pad"], W))]).contiguous()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, H, ps = c["B"], c["H"], c["ps"]
    act = DTYPES[c.get("act", "bf16")]
    lens, rows = _lengths(c), _rows(c)
    start = [t - r for t, r in zip(lens, rows)] if c["op"] == "read" else lens  # (read: the last rows of a request)
    pages = [_cdiv(t + r, ps) for t, r in zip(start, rows)]
    n_pages = sum(pages) + 3  # some pages belong to nobody
    width = max(1, max(pages))
    # a table of shuffled pages, as a long-running server has it; entries behind a request's last page are not looked at
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor([0] + pages, device="cuda").cumsum(0)[:-1]
    at = first[:, None] + torch.arange(width, device="cuda")[None]
    live = torch.arange(width, device="cuda")[None] < torch.tensor(pages, device="cuda")[:, None]
    table = torch.where(live, perm[at.clamp(max=n_pages - 1)], torch.full_like(perm[:1], -1)).contiguous()
    s = dict(case=c, table=table, lens=torch.tensor(start, dtype=torch.int32, device="cuda"), n_live=sum(rows),
             counts=torch.tensor(rows, device="cuda"), most=max(1, max(rows)), bounds=None)
    (s["k"], s["k_scale"]), (s["v"], s["v_scale"]) = _pool(g, c, n_pages), _pool(g, c, n_pages)
    n = sum(rows) + c.get("pad", 0)
    s["offsets"] = _offsets(rows)
    if c["op"] == "tree":
        Hq = c["Hq"]
        if c["n"] == 1 and c["same"] and not c["pad"]:
            s["offsets"] = None
        # one projection's output: q | k | v side by side in a row, the operator gets a view of it
        s["q"] = torch.randn((n, Hq + 2 * H, D), generator=g, device="cuda").to(act)[:, :Hq]
        s["mask"] = None if c["mask"] == "none" else _tree_mask(g, c, rows)
        s["out"], s["lse"] = torch.zeros((n, Hq, D), dtype=act, device="cuda"), torch.zeros((n, Hq), device="cuda")
    if c["op"] == "append":
        Hq, R = c["Hq"], c["rotary"]
        if c["rows"] == 1 and not c["pad"]:
            s["offsets"] = None
        qkv = torch.randn((n, Hq + 2 * H, D), generator=g, device="cuda")
        qkv *= torch.exp(torch.randn((n, Hq + 2 * H, 1), generator=g, device="cuda"))  # tokens of unlike magnitude
        qkv = qkv.to(act)
        s["q"], s["k_new"], s["v_new"] = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        s["q_out"] = torch.zeros((n, Hq, D), dtype=act, device="cuda")
        s["rope"] = None
        if R:
            pos = torch.arange(max(1, max(t + r for t, r in zip(lens, rows))), dtype=torch.float64, device="cuda")
            ang = pos[:, None] * 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
            s["rope"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
    if c["op"] == "read":
        s["k_out"], s["v_out"] = (torch.zeros((n, H, D), dtype=act, device="cuda") for _ in range(2))
    if c["op"] == "commit":
        acc = _accepted(c)
        s["taken"] = torch.tensor([len(a) for a in acc], device="cuda")
        s["most"] = max(1, max(len(a) for a in acc))
        s["offsets"] = _offsets([len(a) for a in acc])
        s["accepted"] = torch.tensor([x for a in acc for x in a], dtype=torch.int32, device="cuda")
        if c["bounds"]:  # (with the drafted tokens' keys in them, as an append leaves them)
            b = torch.stack([s["k"].float().amin(1), s["k"].float().amax(1)], 2)
            s["bounds"] = b.to(s["k"].dtype)
    if own:
        from quantized_cross_loop_gb300 import kvq

        s["cache"] = kvq.PagedCache(page_size=ps, n_heads=H, k=s["k"], v=s["v"], key_bounds=s["bounds"],
                                    k_scale=s["k_scale"], v_scale=s["v_scale"])
        if c["op"] == "tree":
            s["workspace"] = torch.empty(s["cache"].tree_workspace_bytes(B, c["Hq"], n), dtype=torch.uint8,
                                         device="cuda")
    return s


# ------------------------------------------------------------------ one pass


def run(state):
    s = state
    c = s["case"]
    if own:
        from quantized_cross_loop_gb300 import kvq

        if c["op"] == "tree":
            kvq.kvq_paged_tree_attn(s["cache"], s["table"], s["lens"], s["q"], offsets=s["offsets"], mask=s["mask"],
                                    out=s["out"], lse=s["lse"], workspace=s["workspace"])
        elif c["op"] == "append":
            kvq.kvq_paged_append(s["cache"], s["table"], s["lens"], s["k_new"], s["v_new"], offsets=s["offsets"],
                                 q=s["q"], q_out=s["q_out"], rope=s["rope"], interleaved=c["inter"])
        elif c["op"] == "read":
            kvq.kvq_paged_read(s["cache"], s["table"], s["lens"], s["k_out"], s["v_out"], offsets=s["offsets"])
        else:
            kvq.kvq_paged_tree_commit(s["cache"], s["table"], s["lens"], s["accepted"], s["offsets"])
        return _written(s)
    {"tree": _plain_tree, "append": _plain_append, "read": _plain_read, "commit": _plain_commit}[c["op"]](s)
    return _written(s)


def _written(s):
    """What an operator writes (all of it the caller's own buffers)."""
    op = s["case"]["op"]
    if op == "tree":
        return {"out": s["out"], "lse": s["lse"]}
    if op == "read":
        return {"k": s["k_out"], "v": s["v_out"]}
    r = {"k": s["k"], "v": s["v"]}
    if s["case"]["cache"] == "e4m3t":
        r.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
    if op == "append":
        r["q"] = s["q_out"]
    if s["bounds"] is not None:
        r["bounds"] = s["bounds"]
    return r


# ------------------------------------------------------------------ the plain forms


def _requests(s):
    """The request of each live row, and the row's number within it."""
    row = torch.arange(s["n_live"], device="cuda")
    if s["offsets"] is None:
        return row, torch.zeros_like(row)
    off = s["offsets"].long()
    req = torch.searchsorted(off[1:], row, right=True)
    return req, row - off[req]


def _take(pool, scale, c, page, slot):
    """FP32 values [..., H, D] of tokens at (page, slot)."""
    x = pool.view(_bits(pool))[page, slot].view(pool.dtype).float()
    if c["cache"] == "e4m3":
        x = x * scale[:, None]
    if c["cache"] == "e4m3t":
        x = x * scale[page, :, slot][..., None]
    return x


def _plain_tree(s):
    c = s["case"]
    B, H, Hq, ps, N = c["B"], c["H"], c["Hq"], c["ps"], s["most"]
    n = s["n_live"]
    req, i = _requests(s)
    t = torch.arange(s["table"].shape[1] * ps, device="cuda")
    page = s["table"].long().clamp(min=0)[:, t // ps]
    slot = (t % ps).expand_as(page)
    k, v = (_take(s[x], s[x + "_scale"], c, page, slot).transpose(1, 2) for x in ("k", "v"))  # [B, H, tokens, D]
    j = t - s["lens"].long()[:, None]  # the drafted token's number
    drafted = (j >= 0) & (j < s["counts"][:, None])
    if s["mask"] is None:
        sees = drafted[:, None] & (j[:, None] <= torch.arange(N, device="cuda")[:, None])
    else:
        words = s["mask"].new_zeros((B, N, s["mask"].shape[1]))
        words[req, i] = s["mask"][:n]
        jj = j.clamp(0, words.shape[2] * 32 - 1)[:, None].expand(-1, N, -1)
        sees = drafted[:, None] & ((torch.gather(words, 2, jj // 32) >> (jj % 32)) & 1).bool()
    sees = (sees | (j < 0)[:, None]).repeat_interleave(Hq // H, dim=1)[:, None]  # [B, 1, rows, tokens]
    q = torch.zeros((B, N, Hq, D), device="cuda")
    q[req, i] = s["q"][:n].float()
    q = q.view(B, N, H, Hq // H, D).transpose(1, 2).reshape(B, H, -1, D)
    x = (q @ k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    x = torch.where(sees, x, torch.full_like(x, -math.inf))
    v = torch.where((j < s["counts"][:, None])[:, None, :, None], v, torch.zeros_like(v))
    m = x.amax(3, keepdim=True)
    x = (x - torch.where(torch.isinf(m), torch.zeros_like(m), m)).exp()
    l = x.sum(3, keepdim=True)
    out = (x @ v) / torch.where(l == 0, torch.ones_like(l), l)
    lse = torch.where(l == 0, torch.full_like(l, -math.inf), m + l.log())
    back = lambda y: y.view(B, H, N, Hq // H, -1).transpose(1, 2).reshape(B, N, Hq, -1)[req, i]  # noqa: E731
    s["out"][:n] = back(out).to(s["out"].dtype)
    s["lse"][:n] = back(lse)[..., 0]


def _plain_rotate(x, s, pos):
    R = s["case"]["rotary"]
    x = x.float()
    if not R:
        return x
    cs = s["rope"][pos]
    cos, sin = cs[:, None, :R // 2], cs[:, None, R // 2:]
    y = x.clone()
    if s["case"]["inter"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y[..., 0:R:2], y[..., 1:R:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y[..., :R // 2], y[..., R // 2:R] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_append(s):
    c = s["case"]
    ps, n = c["ps"], s["n_live"]
    req, i = _requests(s)
    pos = s["lens"].long()[req] + i
    page, slot = s["table"].long()[req, pos // ps], pos % ps
    s["q_out"][:n] = _plain_rotate(s["q"][:n], s, pos).to(s["q_out"].dtype)
    for name, x in (("k", _plain_rotate(s["k_new"][:n], s, pos)), ("v", s["v_new"][:n].float())):
        scale = (x.abs().amax(2) / E4M3_MAX).clamp(min=SMALLEST_SCALE)
        x = (x / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(s[name].dtype)
        s[name].view(torch.uint8)[page, slot] = x.view(torch.uint8)
        s[name + "_scale"][page, :, slot] = scale


def _plain_read(s):
    c = s["case"]
    req, i = _requests(s)
    pos = s["lens"].long()[req] + i
    page, slot = s["table"].long()[req, pos // c["ps"]], pos % c["ps"]
    for name in ("k", "v"):
        s[name + "_out"][:s["n_live"]] = _take(s[name], s[name + "_scale"], c, page, slot).to(s[name + "_out"].dtype)


def _plain_commit(s):
    c = s["case"]
    ps, taken, lens = c["ps"], s["taken"], s["lens"].long()
    table = s["table"].long()
    off = s["offsets"].long()
    row = torch.arange(s["accepted"].numel(), device="cuda")
    req = torch.searchsorted(off[1:], row, right=True)
    here, there = lens[req] + s["accepted"].long(), lens[req] + row - off[req]
    page, slot, to_page, to_slot = table[req, here // ps], here % ps, table[req, there // ps], there % ps
    for name in ("k", "v"):
        pool = s[name].view(_bits(s[name]))
        pool[to_page, to_slot] = pool[page, slot]
        if c["cache"] == "e4m3t":
            scale = s[name + "_scale"]
            scale[to_page, :, to_slot] = scale[page, :, slot]
    if s["bounds"] is None:
        return
    # the pages from the first drafted token's on, as far as they hold tokens now
    p = (lens // ps)[:, None] + torch.arange(_cdiv(s["most"], ps) + 1, device="cuda")
    end = (lens + taken)[:, None]
    live = p * ps < end
    phys = table[torch.arange(c["B"], device="cuda")[:, None].expand_as(p)[live], p[live]]
    k = s["k"].view(_bits(s["k"]))[phys].view(s["k"].dtype).float()
    t = (p * ps)[live][:, None] + torch.arange(ps, device="cuda")
    there = (t < end.expand_as(p)[live][:, None])[..., None, None]
    lo = torch.where(there, k, torch.full_like(k, math.inf)).amin(1)
    hi = torch.where(there, k, torch.full_like(k, -math.inf)).amax(1)
    new = torch.stack([lo, hi], 2).to(s["bounds"].dtype)
    s["bounds"].view(_bits(new))[phys] = new.view(_bits(new))


# ------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    lens, rows = s["lens"].tolist(), _rows(c)
    # a token's stored values in 64 bits, from the pools and scales as they are
    pools = {}
    for name in ("k", "v"):
        x = s[name].double()
        if c["op"] in ("tree", "read"):
            if c["cache"] == "e4m3":
                x = x * s[name + "_scale"].double()[:, None]
            if c["cache"] == "e4m3t":
                x = x * s[name + "_scale"].double().transpose(1, 2)[..., None]
        pools[name] = x
    if c["op"] == "tree":
        return _exact_tree(s, pools, lens, rows)
    if c["op"] == "read":
        out = {x: s[x + "_out"].double() for x in ("k", "v")}
        at = 0
        for b, (t0, r) in enumerate(zip(lens, rows)):
            t = torch.arange(t0, t0 + r, device="cuda")
            for x in ("k", "v"):
                out[x][at:at + r] = pools[x][s["table"][b].long()[t // c["ps"]], t % c["ps"]]
            at += r
        return out
    return _exact_append(s, pools, lens, rows) if c["op"] == "append" else _exact_commit(s, pools, lens)


def _exact_tree(s, pools, lens, rows):
    c = s["case"]
    H, g, ps = c["H"], c["Hq"] // c["H"], c["ps"]
    out, lse = s["out"].double(), s["lse"].double()
    at = 0
    for b, (T, n) in enumerate(zip(lens, rows)):
        if n == 0:
            continue
        t = torch.arange(T + n, device="cuda")
        page = s["table"][b].long()[t // ps]
        if s["mask"] is None:
            seen = torch.ones((n, n), device="cuda").tril() > 0
        else:
            bit = torch.arange(n, device="cuda")
            seen = ((s["mask"][at:at + n].long()[:, bit // 32] >> (bit % 32)) & 1) > 0
        seen = torch.cat([torch.ones((n, T), device="cuda") > 0, seen], 1)
        none = ~seen.any(1)
        for h in range(H):
            k, v = pools["k"][page, t % ps, h], pools["v"][page, t % ps, h]
            for j in range(h * g, h * g + g):
                x = (s["q"][at:at + n, j].double() @ k.T / math.sqrt(D)).masked_fill(~seen, -math.inf)
                out[at:at + n, j] = (torch.softmax(x, 1) @ v).masked_fill(none[:, None], 0.0)
                lse[at:at + n, j] = torch.logsumexp(x, 1)
        at += n
    return {"out": out, "lse": lse}


def _exact_append(s, pools, lens, rows):
    c = s["case"]
    ps, R = c["ps"], c["rotary"]
    scales = {x: s[x + "_scale"].double() for x in ("k", "v")}
    q = s["q_out"].double()
    at = 0
    for b, (t0, n) in enumerate(zip(lens, rows)):
        if n == 0:
            continue
        t = torch.arange(t0, t0 + n, device="cuda")
        page = s["table"][b].long()[t // ps]
        new = {x: s[x][at:at + n].double() for x in ("q", "k_new", "v_new")}
        if R:
            z = torch.complex(*s["rope"][t0:t0 + n].double().unsqueeze(1).chunk(2, dim=2))
            for x in (new["q"], new["k_new"]):
                if c["inter"]:
                    pair = x[..., :R].unflatten(2, (R // 2, 2))
                    w = torch.complex(pair[..., 0].contiguous(), pair[..., 1].contiguous()) * z
                    x[..., :R] = torch.view_as_real(w).flatten(2)
                else:
                    w = torch.complex(x[..., :R // 2].contiguous(), x[..., R // 2:R].contiguous()) * z
                    x[..., :R] = torch.cat([w.real, w.imag], 2)
        q[at:at + n] = new["q"]
        for x in ("k", "v"):
            y = new[x + "_new"]
            scale = y.abs().amax(2).div(E4M3_MAX).clamp(min=SMALLEST_SCALE)
            pools[x][page, t % ps] = y / scale[..., None]
            scales[x][page, :, t % ps] = scale
        at += n
    return {"k": pools["k"], "v": pools["v"], "k_scale": scales["k"], "v_scale": scales["v"], "q": q}


def _exact_commit(s, pools, lens):
    c = s["case"]
    ps = c["ps"]
    r = {x: pools[x] for x in ("k", "v")}
    if c["cache"] == "e4m3t":
        r.update({x + "_scale": s[x + "_scale"].double() for x in ("k", "v")})
    if s["bounds"] is not None:
        r["bounds"] = s["bounds"].double()
    for b, (t0, taken) in enumerate(zip(lens, _accepted(c))):
        page = s["table"][b].long()
        if taken:
            src = t0 + torch.tensor(taken, device="cuda")
            dst = t0 + torch.arange(len(taken), device="cuda")
            for x in ("k", "v"):
                r[x][page[dst // ps], dst % ps] = r[x][page[src // ps], src % ps].clone()
                if c["cache"] == "e4m3t":
                    y = r[x + "_scale"]
                    y[page[dst // ps], :, dst % ps] = y[page[src // ps], :, src % ps].clone()
        if s["bounds"] is not None:
            end = t0 + len(taken)
            for p in range(t0 // ps, _cdiv(end, ps)):
                k = r["k"][page[p], :min(ps, end - p * ps)]
                r["bounds"][page[p], :, 0], r["bounds"][page[p], :, 1] = k.amin(0), k.amax(0)
    return r
